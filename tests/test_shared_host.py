"""CPU checks of the shared-latent calls: the oracle against hand cases and a second formulation,
the description's checks, and the refusals that happen before anything touches a GPU."""
import ctypes
import itertools

import numpy as np
import pytest

from oracle import shared as S


def test_e4m3_values():
    v = S.e4m3_values()
    assert len(v) == 127 and v[0] == 0 and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6 and v[-1] == 448.0
    assert np.all(np.diff(v) > 0)


@pytest.mark.parametrize("top,e", [(448.0, 0), (449.0, 1), (1.75, -8), (1.7500001, -7), (1.0, -8), (2.0, -7),
                                   (3.5, -7), (0.0, 0)])
def test_group_scale_is_the_smallest_power_of_two(top, e):
    g = np.zeros(32)
    g[5] = top
    y = S.quantize_e4m3(g)
    # the stored maximum is the nearest of 16 significands at this scale: off by at most 2^-4
    assert abs(y[5] - top) <= 2.0 ** -4 * top
    if top:
        assert top <= 448 * 2.0 ** e and not top <= 448 * 2.0 ** (e - 1)


def test_quantiser_ties_subnormals_and_bad_groups():
    g = np.zeros(32)
    g[0] = 448.0                                  # e = 0
    g[1], g[2], g[3] = 17.0, 19.0, -17.0          # halfway between 16, 18, 20: to even mantissas
    g[4], g[5] = 2.0 ** -10, 3 * 2.0 ** -10       # halfway: 0 | 2^-9, 2^-9 | 2 * 2^-9
    y = S.quantize_e4m3(g)
    assert list(y[:6]) == [448.0, 16.0, 20.0, -16.0, 0.0, 2.0 ** -8]
    for bad in (np.nan, np.inf, -np.inf):
        b = np.ones(64)
        b[7] = bad
        y = S.quantize_e4m3(b)
        assert np.all(np.isnan(y[:32])) and np.all(y[32:] == 1.0)


def test_rotation_keeps_norms_and_relative_angles():
    rng = np.random.default_rng(0)
    a, b = rng.standard_normal((2, 1, 32))
    for s, t in ((0, 0), (3, 11), (1000, 70000)):
        ra, rb = S.rotate(a, [s], 1e4)[0], S.rotate(b, [t], 1e4)[0]
        ra2, rb2 = S.rotate(a, [s + 5], 1e4)[0], S.rotate(b, [t + 5], 1e4)[0]
        assert np.isclose(np.linalg.norm(ra), np.linalg.norm(a)) and np.isclose(ra @ rb, ra2 @ rb2)
    assert np.array_equal(S.rotate(a, [9], 0.0), a)


def test_attention_equals_the_rank_space_form():
    """q . [c B_k | kr] = (B_k q) . c + q_r . kr, and sum p (c B_v) = (sum p c) B_v."""
    rng = np.random.default_rng(1)
    T, r, hq, hkv, dn, dr, dv = 9, 12, 4, 2, 5, 4, 3
    c, kr = rng.standard_normal((T, r)), rng.standard_normal((T, dr))
    Bk, Bv = rng.standard_normal((r, hkv * dn)), rng.standard_normal((r, hkv * dv))
    q = rng.standard_normal((3, hq, dn + dr))
    out, lse, _ = S.attention(q, S.expand(c, Bk, hkv), kr, S.expand(c, Bv, hkv), 0.3)
    for i, j in itertools.product(range(3), range(hq)):
        h = j // 2
        qt = Bk[:, h * dn:(h + 1) * dn] @ q[i, j, :dn]
        n = T - 2 + i
        s = 0.3 * (c[:n] @ qt + kr[:n] @ q[i, j, dn:])
        p = np.exp(s - s.max())
        assert np.allclose(out[i, j], (p @ c[:n] / p.sum()) @ Bv[:, h * dv:(h + 1) * dv])
        assert np.isclose(lse[i, j], s.max() + np.log(p.sum()))


def test_attention_rows_without_keys():
    q = np.ones((3, 1, 4))
    out, lse, _ = S.attention(q, np.ones((1, 1, 2)), np.ones((1, 2)), np.full((1, 1, 2), 7.0), 1.0)
    assert np.all(out[:2] == 0) and np.all(np.isneginf(lse[:2])) and np.all(out[2] == 7.0)


def _desc(lib, **kw):
    base = dict(batch=2, n_q_heads=4, n_kv_heads=2, dim_nope=128, dim_rope=64, dim_v=128, rank=128, capacity=256)
    base.update(kw)
    return lib.make_shared_desc(**base)


def test_desc_size_matches_binding(lib):
    assert lib.lr_shared_desc_size() == ctypes.sizeof(lib.lr_shared_desc)


@pytest.mark.parametrize("field,value,status", [
    ("batch", 0, 1), ("batch", 1025, 2), ("n_q_heads", 5, 1), ("n_q_heads", 130, 2), ("n_kv_heads", 0, 1),
    ("dim_nope", 96, 1), ("dim_rope", 16, 1), ("dim_rope", 0, 1), ("dim_v", 256, 1), ("rank", 0, 1),
    ("rank", 96, 1), ("rank", 576, 1), ("capacity", 0, 1), ("capacity", 200, 1), ("capacity", (1 << 24) + 128, 1),
    ("n_pages", -1, 1), ("n_pages", (1 << 22) + 1, 1), ("quant_bits", 4, 1), ("dtype", 0, 2), ("dtype", 5, 1),
    ("max_queries", 0, 1), ("max_queries", 9, 2), ("rope_theta", -1.0, 1), ("rope_theta", float("nan"), 1),
    ("rope_theta", float("inf"), 1), ("softmax_scale", -0.5, 1), ("softmax_scale", float("nan"), 1)])
def test_bad_descriptions_are_refused_before_the_device(lib, field, value, status):
    d = _desc(lib, **{field: value})
    out = ctypes.c_void_p()
    st = lib.raw_status("lr_shared_create", ctypes.byref(d), ctypes.c_void_p(16), ctypes.c_void_p(16), None,
                        ctypes.byref(out))
    assert st == status and not out.value


def test_reserved_words_and_null_arguments(lib):
    d = _desc(lib)
    d.reserved[1] = 1
    out = ctypes.c_void_p()
    ptr = ctypes.c_void_p(16)
    assert lib.raw_status("lr_shared_create", ctypes.byref(d), ptr, ptr, None, ctypes.byref(out)) == 1
    d = _desc(lib)
    assert lib.raw_status("lr_shared_create", ctypes.byref(d), None, ptr, None, ctypes.byref(out)) == 1
    assert lib.raw_status("lr_shared_create", ctypes.byref(d), ptr, None, None, ctypes.byref(out)) == 1
    assert lib.raw_status("lr_shared_create", ctypes.byref(d), ptr, ptr, None, None) == 1
    assert lib.raw_status("lr_shared_create", None, ptr, ptr, None, ctypes.byref(out)) == 1
    assert lib.raw_status("lr_shared_destroy", None) == 0
    for name, args in (("lr_shared_append", (ptr, 64, ptr, 64, ptr, ptr, 1, None)),
                       ("lr_shared_read", (ptr, None, 1, ptr, ptr, None)),
                       ("lr_shared_decode", (ptr, 1, ptr, ptr, None, None)),
                       ("lr_shared_expand", (ptr, None, 1, ptr, ptr, ptr, None)),
                       ("lr_shared_attn", (ptr, ptr, ptr, ptr, ptr, ptr, 1, 1, 1, 1, ptr, None, None)),
                       ("lr_shared_set_block_table", (ptr, None)), ("lr_shared_set_block_table_device", (ptr, None)),
                       ("lr_shared_set_wait_limit", (0,)), ("lr_shared_device_error", (None,))):
        assert lib.raw_status(name, None, *args) == 1, name
