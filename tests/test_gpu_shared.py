"""Shared-latent caches on the GPU against the fp64 oracle: writing and reading back (bf16 exact,
8-bit codes exact), the absorbed decode, expansion and ragged attention, at the lengths, page
boundaries, head layouts and masks where they can go wrong; refusals; streams and graphs.

Tolerances come from the arithmetic (u = 2^-8, half a bf16 step; fp32 half step 2^-24)."""
import ctypes

import numpy as np
import pytest

from oracle import shared as S

pytestmark = pytest.mark.gpu

U, F = 2.0 ** -8, 2.0 ** -24


def bf16(x):
    import torch
    return torch.tensor(np.asarray(x), dtype=torch.float32).to(torch.bfloat16).cuda()


def f64(t):
    return t.detach().cpu().double().numpy()


def i32(x):
    import torch
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Layer:
    """A cache filled with seeded tokens through a permuted page table, and its fp64 contents."""

    def __init__(self, lib, lens, hq=4, hkv=4, dn=128, dr=64, dv=128, r=128, bits=0, new=1, cap=None, seed=0,
                 theta=0.0, spare=2, stale=True, scale=0.0):
        import torch
        rng = np.random.default_rng(seed)
        self.lib, self.lens, B = lib, list(lens), len(lens)
        self.hq, self.hkv, self.dn, self.dr, self.dv, self.r, self.bits = hq, hkv, dn, dr, dv, r, bits
        cap = cap or max(128, -(-max(lens) // 128) * 128)
        self.cap, pps = cap, cap // 128
        n_pages = B * pps + spare
        self.desc = lib.make_shared_desc(B, hq, hkv, dn, dr, dv, r, cap, n_pages=n_pages, quant_bits=bits,
                                         max_queries=new, rope_theta=theta, softmax_scale=scale)
        self.scale = scale or (dn + dr) ** -0.5
        sp = np.arange(1, r + 1) ** -0.3
        self.Bk, self.Bv = bf16(rng.standard_normal((r, hkv * dn)) / r ** 0.5), bf16(
            rng.standard_normal((r, hkv * dv)) / r ** 0.5)
        self.cache = lib.lr_shared_create(self.desc, self.Bk, self.Bv)
        self.table = rng.permutation(n_pages)[:B * pps].reshape(B, pps).astype(np.int32)
        if stale:                      # every row of the pool first holds non-finite leftovers
            junk = bf16(np.full((cap, r), np.inf)), bf16(np.full((cap, dr), np.nan))
            for k in range(0, n_pages, pps):
                t = (np.arange(B * pps) % n_pages + k) % n_pages
                lib.lr_shared_set_block_table(self.cache, t.reshape(B, pps).astype(np.int32))
                lib.lr_shared_append(self.cache, *junk, i32(np.zeros(cap)), i32(np.arange(cap)))
        lib.lr_shared_set_block_table(self.cache, self.table)
        n = sum(lens)
        self.c = bf16(rng.standard_normal((n, r)) * sp * 1.5)
        self.kr = bf16(rng.standard_normal((n, dr)))
        seq = np.repeat(np.arange(B), lens)
        pos = np.concatenate([np.arange(x) for x in lens]) if n else np.zeros(0)
        if n:
            lib.lr_shared_append(self.cache, self.c, self.kr, i32(seq), i32(pos))
        self.cu = np.concatenate([[0], np.cumsum(lens)])
        c = f64(self.c)
        self.c64 = S.quantize_e4m3(c) if bits else c
        self.kr64 = S.rotate(f64(self.kr), pos, theta)
        self.Bk64, self.Bv64 = f64(self.Bk), f64(self.Bv)
        self.rng = rng
        torch.cuda.synchronize()

    def rows(self, b):
        return slice(self.cu[b], self.cu[b + 1])

    def query(self, n_tok, amp=1.5):
        return bf16(self.rng.standard_normal((len(self.lens), n_tok, self.hq, self.dn + self.dr)) * amp)

    def decode(self, q, lens=None):
        import torch
        B, n = q.shape[:2]
        out = torch.full((B, n, self.hq, self.dv), 777.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((B, n, self.hq), 777.0, dtype=torch.float32, device="cuda")
        self.lib.lr_shared_decode(self.cache, q, i32(self.lens if lens is None else lens), out, lse)
        torch.cuda.synchronize()
        assert self.lib.lr_shared_device_error(self.cache) == 0
        return out, lse

    def check_decode(self, q, out, lse, lens=None):
        """out and lse against the oracle, within what the roundings can add up to.

        Scores: q~ has K = dn fp32 steps, then two bf16 halves (residual u^2 of it), the dot product
        r + dr fp32 steps: E = scale ((u^2 + (dn + r + dr + 8) F) sum |q~_i c_i|-like terms); log2
        and exp2 in fp32 add 2^-20 of the score.  Weights: one bf16 rounding (u) in the numerator
        and in the normaliser.  Rank-space sums: (T + r + 64) F and the split halves u^2 of
        sum_i (sum_t p |c_ti|) |B_i|.  The output: u of its value."""
        n_tok = q.shape[1]
        q64, g = f64(q), self.hq // self.hkv
        lens = self.lens if lens is None else lens
        for b, n in enumerate(lens):
            c, kr = self.c64[self.rows(b)][:n], self.kr64[self.rows(b)][:n]
            ro, rl, mix = S.attention(q64[b], S.expand(c, self.Bk64, self.hkv), kr, S.expand(c, self.Bv64, self.hkv),
                                      self.scale)
            if self.rope_stored:
                kr_err = U * np.abs(kr)
            for s in range(n_tok):
                seen = n - (n_tok - 1 - s)
                go, gl = f64(out[b, s]), f64(lse[b, s])
                if seen <= 0:
                    assert np.all(go == 0) and np.all(np.isneginf(gl)), (b, s)
                    continue
                for j in range(self.hq):
                    h = j // g
                    Bk, Bv = self.Bk64[:, h * self.dn:(h + 1) * self.dn], self.Bv64[:, h * self.dv:(h + 1) * self.dv]
                    aq = np.abs(Bk) @ np.abs(q64[b, s, j, :self.dn])
                    mag = np.abs(c[:seen]) @ aq + np.abs(kr[:seen]) @ np.abs(q64[b, s, j, self.dn:])
                    E = self.scale * (U * U + (self.dn + self.r + self.dr + 8) * F) * mag.max() + 2.0 ** -20 * (
                        self.scale * mag.max())
                    if self.rope_stored:
                        E += self.scale * (kr_err[:seen] @ np.abs(q64[b, s, j, self.dn:])).max()
                    assert abs(gl[j] - rl[s, j]) <= E + (seen + 64) * F + 2.0 ** -21 * abs(rl[s, j]), (b, s, j)
                    w = np.exp(self.scale * (c[:seen] @ (Bk @ q64[b, s, j, :self.dn]) + kr[:seen] @ q64[
                        b, s, j, self.dn:]) - rl[s, j])
                    A = (w @ np.abs(c[:seen])) @ np.abs(Bv)
                    tol = U * np.abs(ro[s, j]) + (2 * U + 2 * E) * mix[s, j] + (U * U + (seen + self.r + 64) * F) * A
                    err = np.abs(go[j] - ro[s, j])
                    assert np.all(err <= tol), (b, s, j, (err / tol).max())

    rope_stored = False


# ---------------------------------------------------------------------------
# write and read back
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("bits", [0, 8])
@pytest.mark.parametrize("r,dr", [(64, 32), (192, 64), (512, 64)])
def test_write_reads_back_what_it_stands_for(lib, bits, r, dr):
    import torch
    lens = [1, 127, 128, 129, 300]
    m = Layer(lib, lens, r=r, dr=dr, bits=bits, theta=1e4)
    c = torch.full((sum(lens) + 3, r), 5.0, dtype=torch.bfloat16, device="cuda")
    kr = torch.full((sum(lens) + 3, dr), 5.0, dtype=torch.bfloat16, device="cuda")
    lib.lr_shared_read(m.cache, i32(m.cu), c, kr)
    assert np.array_equal(f64(c)[:-3], m.c64)
    a = np.abs(f64(m.kr))
    pair = np.concatenate([a[:, :dr // 2] + a[:, dr // 2:]] * 2, axis=1)
    assert np.all(np.abs(f64(kr)[:-3] - m.kr64) <= U * np.abs(m.kr64) + 4 * F * pair)
    assert np.all(f64(c)[-3:] == 5) and np.all(f64(kr)[-3:] == 5)   # behind the last sequence: untouched


def test_every_code_and_extreme_groups(lib):
    """All finite e4m3 values at several scales, and groups at the edges of the range."""
    import torch
    vals = S.e4m3_values()
    rows = []
    for e in (-100, -60, -7, 0, 7, 60, 112):
        x = np.zeros(256)
        x[:127], x[128:255] = vals, -vals
        x = x.reshape(8, 32).copy()
        x[:, 31] = 448.0                                       # pins every group's scale to 2^e
        rows.append((x * 2.0 ** e).reshape(-1))
    rows.append(np.full(256, 2.0 ** -126))                     # below the smallest scale's normal codes
    top = np.zeros(256)
    top[::32] = 2.0 ** 127
    rows.append(top)
    bad = np.ones(256)
    bad[[3, 70, 140]] = np.inf, np.nan, -np.inf
    rows.append(bad)
    x = bf16(np.array(rows))
    d = lib.make_shared_desc(1, 1, 1, 64, 32, 64, 256, 128, quant_bits=8)
    cache = lib.lr_shared_create(d, bf16(np.zeros((256, 64))), bf16(np.zeros((256, 64))))
    n = len(rows)
    kr = bf16(np.zeros((n, 32)))
    lib.lr_shared_append(cache, x, kr, i32(np.zeros(n)), i32(np.arange(n)))
    c, k = torch.zeros_like(x), torch.zeros_like(kr)
    lib.lr_shared_read(cache, i32([0, n]), c, k)
    want = S.quantize_e4m3(f64(x))
    assert np.array_equal(f64(c)[:7], f64(x)[:7])              # every value is its own code
    assert np.array_equal(f64(c), want, equal_nan=True)


def test_far_positions_rotate_with_exact_angles(lib):
    import torch
    d = lib.make_shared_desc(1, 1, 1, 64, 64, 64, 64, 1 << 20, n_pages=3, rope_theta=1e6)
    cache = lib.lr_shared_create(d, bf16(np.zeros((64, 64))), bf16(np.zeros((64, 64))))
    pos = np.array([0, 1, 999_999, (1 << 20) - 1])
    table = np.zeros((1, 8192), np.int32)
    table[0, 999_999 // 128], table[0, -1] = 1, 2
    lib.lr_shared_set_block_table(cache, table)
    kr = bf16(np.random.default_rng(0).standard_normal((4, 64)))
    lib.lr_shared_append(cache, bf16(np.zeros((4, 64))), kr, i32(np.zeros(4)), i32(pos))
    want = S.rotate(f64(kr), pos, 1e6)
    for i, p in enumerate(pos):
        c, k = torch.zeros((1, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros_like(kr[:1])
        lib.lr_shared_read(cache, i32([0, 1]), c, k, start=i32([p]))
        assert np.all(np.abs(f64(k)[0] - want[i]) <= U * np.abs(want[i]) + 1e-6)


def test_spaced_rows_padding_and_partial_reads(lib):
    """Columns of one wider projection output as c and kr; padded tokens write nothing; reads that
    start inside a page, skip sequences, and run past what may be read."""
    import torch
    rng = np.random.default_rng(3)
    d = lib.make_shared_desc(3, 2, 2, 64, 32, 64, 128, 256)
    cache = lib.lr_shared_create(d, bf16(np.zeros((128, 128))), bf16(np.zeros((128, 128))))
    wide = bf16(rng.standard_normal((40, 8 + 128 + 32 + 8)))
    c, kr = wide[:, 8:136], wide[:, 136:168]
    seq = np.array([0, 2] * 20)
    pos = np.arange(40) // 2 + 120                             # crosses a page
    seq[4], seq[5], pos[6], pos[7] = -1, 3, -1, 256            # padding of each kind
    lib.lr_shared_append(cache, c, kr, i32(seq), i32(pos))
    got_c = torch.full((30, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    got_k = torch.full((30, 32), 9.0, dtype=torch.bfloat16, device="cuda")
    # sequence 0: tokens 120..139; sequence 1: none; sequence 2: tokens 250..259, six of them past the capacity
    lib.lr_shared_read(cache, i32([2, 22, 22, 32]), got_c, got_k, start=i32([120, 0, 250]))
    g, k = f64(got_c), f64(got_k)
    assert np.all(g[:2] == 9) and np.all(k[:2] == 9)
    for t in range(20):
        i = 2 * t
        want = (f64(c)[i], f64(kr)[i]) if i not in (4, 6) else (np.zeros(128), np.zeros(32))
        assert np.array_equal(g[2 + t], want[0]) and np.array_equal(k[2 + t], want[1]), t
    assert np.all(g[22:28] == 0) and np.all(g[28:] == 9) and np.all(k[28:] == 9)


# ---------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------

LENS = [0, 1, 2, 127, 128, 129, 300, 517]


@pytest.mark.parametrize("bits", [0, 8])
@pytest.mark.parametrize("hq,hkv,r,dn,dr,dv,new", [
    (4, 4, 128, 128, 64, 128, 1), (28, 4, 256, 128, 64, 128, 1), (28, 28, 512, 128, 64, 128, 1),
    (16, 1, 64, 64, 32, 64, 1), (5, 5, 192, 128, 32, 64, 3), (40, 8, 448, 64, 64, 128, 2), (1, 1, 320, 64, 32, 128, 8),
    (17, 17, 384, 64, 64, 64, 1), (64, 16, 320, 64, 64, 64, 2)])
def test_decode_matches_the_oracle(lib, bits, hq, hkv, r, dn, dr, dv, new):
    m = Layer(lib, LENS, hq=hq, hkv=hkv, r=r, dn=dn, dr=dr, dv=dv, bits=bits, new=new)
    q = m.query(new)
    m.check_decode(q, *m.decode(q))


@pytest.mark.parametrize("bits", [0, 8])
@pytest.mark.parametrize("r", [128, 512])
def test_decode_many_heads_and_uneven_lengths(lib, bits, r):
    m = Layer(lib, [1500, 3, 0, 900], hq=128, hkv=128, r=r, bits=bits, new=2, dn=64, dv=64)
    q = m.query(2)
    m.check_decode(q, *m.decode(q))


@pytest.mark.parametrize("r,bits", [(128, 8), (448, 8), (512, 0)])
def test_decode_long_context_over_many_splits(lib, r, bits):
    m = Layer(lib, [20000, 5], hq=6, hkv=3, r=r, bits=bits)
    q = m.query(1)
    m.check_decode(q, *m.decode(q))


@pytest.mark.parametrize("r,bits", [(r, 8) for r in range(64, 513, 64)] + [(192, 0), (512, 0)])
def test_decode_runs_that_use_every_slot_again(lib, r, bits):
    """Runs of 9 tiles over several sequences (1024 query rows leave 4 CTA columns), more than there are
    slots at any rank, and tiles that differ in sign and size: latents of one tile under the weights of
    another would show.  Twice the same."""
    import torch
    m = Layer(lib, [1500, 300, 129, 1, 100], hq=128, hkv=2, r=r, bits=bits, new=8, dn=64, dv=64)
    pos = np.concatenate([np.arange(n) for n in m.lens])
    tile = pos // 64
    f = np.where(tile % 2, -1.0, 1.0) * 2.0 ** (tile % 3)      # exact in bf16, and in the codes' scales
    m.c = m.c * bf16(f)[:, None]
    m.c64 *= f[:, None]
    lib.lr_shared_append(m.cache, m.c, m.kr, i32(np.repeat(np.arange(5), m.lens)), i32(pos))
    q = m.query(8, 0.5)
    a = m.decode(q)
    m.check_decode(q, *a)
    for _ in range(4):
        b = m.decode(q)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_decode_of_rotated_keys_and_own_scale(lib):
    m = Layer(lib, [200, 129], r=128, theta=1e4, scale=0.21)
    m.rope_stored = True
    q = m.query(1)
    m.check_decode(q, *m.decode(q))


@pytest.mark.parametrize("amp", [0.0, 30.0])
@pytest.mark.parametrize("r", [256, 512])
def test_decode_equal_and_sharp_weights(lib, amp, r):
    m = Layer(lib, [700, 128], hq=16, hkv=16, r=r)
    q = m.query(1, amp)
    m.check_decode(q, *m.decode(q))


@pytest.mark.parametrize("hq,r,bits,new", [(4, 128, 0, 1), (28, 512, 0, 1), (28, 512, 8, 1), (128, 256, 8, 2)])
def test_decode_of_equal_weights_other_than_one(lib, hq, r, bits, new):
    """Every 64th token has weight 1, the others all the same weight, which bf16 rounds by nearly half a
    step.  One latent throughout: the common rounding of the weights (u at most, their sum is of the
    unrounded ones), then that of the output, u of a value itself up to u larger; sums, the halves."""
    w = 0.5 * (1 + 2.0 ** -8 - 2.0 ** -13)
    m = Layer(lib, [640, 64, 1], hq=hq, hkv=hq, r=r, bits=bits, new=new, dn=64, dv=64, scale=-float(np.log(w)))
    pos = np.concatenate([np.arange(n) for n in m.lens])
    m.c[:] = m.c[:1].clone()
    m.kr.zero_()
    m.kr[:, 3] = bf16(np.where(pos % 64 == 0, 0.0, -1.0))
    lib.lr_shared_append(m.cache, m.c, m.kr, i32(np.repeat([0, 1, 2], m.lens)), i32(pos))
    q = m.query(new, 0.0)
    q[..., 64 + 3] = 1.0
    out, lse = map(f64, m.decode(q))
    want = (m.c64[0] @ m.Bv64).reshape(hq, 64)
    A = (np.abs(m.c64[0]) @ np.abs(m.Bv64)).reshape(hq, 64)
    for b, n in enumerate(m.lens):
        for s in range(new):
            seen = n - (new - 1 - s)
            if seen <= 0:
                continue
            high = (seen + 63) // 64
            assert np.all(np.abs(lse[b, s] - np.log(high + (seen - high) * w)) <= 2.0 ** -18)
            assert np.all(np.abs(out[b, s] - want) <= U * (2 + U) * np.abs(want) + (U * U + (n + r + 64) * F) * A)


@pytest.mark.parametrize("hq,r,bits,new", [(4, 128, 0, 1), (28, 512, 8, 2), (6, 192, 8, 1), (28, 512, 0, 2)])
def test_decode_over_visible_infinities_and_nans(lib, hq, r, bits, new):
    """A score of -infinity weighs nothing; one of +infinity, and a NaN, make NaN of the queries that see
    them; other sequences, before and behind in the same run or not, are as without."""
    import torch
    m = Layer(lib, [200, 700, 130, 64], hq=hq, hkv=hq, r=r, bits=bits, new=new, dn=64, dv=64)
    q = m.query(new)
    q[..., 64:] = 0.0
    q[..., 64 + 5] = 1.0
    want, wl = m.decode(q)

    def put(b, t, c=None, kr=None):
        """Token t of sequence b once more, some of its elements replaced."""
        i = int(m.cu[b]) + t
        x, y = m.c[i:i + 1].clone(), m.kr[i:i + 1].clone()
        if c is not None:
            x[0, r - 3] = c
        if kr is not None:
            y[0, 5] = kr
        lib.lr_shared_append(m.cache, x, y, i32([b]), i32([t]))

    # tokens of a very low score, then of none at all
    for t in (0, 63, 64, 699 - new):
        put(1, t, kr=-3e38)
    low, ll = m.decode(q)
    assert torch.isfinite(low.float()).all() and torch.isfinite(ll).all() and not torch.equal(low[1], want[1])
    for t in (0, 63, 64, 699 - new):
        put(1, t, kr=-np.inf)
    out, lse = m.decode(q)
    assert torch.equal(out, low) and torch.equal(lse, ll)
    for kw in (dict(kr=np.inf), dict(kr=np.nan), dict(c=np.nan), dict(c=np.inf), dict(c=-np.inf)):
        put(1, 300, **kw)
        out, lse = m.decode(q)
        assert torch.isnan(out[1].float()).all(), kw
        # (an infinite latent's score may be -infinity: no weight, but 0 times its value is NaN still)
        assert torch.isnan(lse[1]).all() or kw.get("c") in (np.inf, -np.inf), kw
        for b in (0, 2, 3):
            assert torch.equal(out[b], want[b]) and torch.equal(lse[b], wl[b]), kw
    for t in (0, 63, 64, 300, 699 - new):
        put(1, t)
    out, lse = m.decode(q)
    assert torch.equal(out, want) and torch.equal(lse, wl)


def test_decode_shorter_lengths_and_clamping(lib):
    """row_len picks a prefix; values outside 0..capacity are clamped."""
    import torch
    m = Layer(lib, [300, 384, 10])
    q = m.query(1)
    m.check_decode(q, *m.decode(q, [17, 384, 0]), lens=[17, 384, 0])
    a, b = m.decode(q, [300, 9999, -4]), m.decode(q, [300, 384, 0])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_decode_without_lse_and_twice_the_same(lib):
    import torch
    m = Layer(lib, [513, 77, 1000], hq=28, hkv=28, r=512)
    q = m.query(1)
    a = m.decode(q)
    out = torch.zeros_like(a[0])
    lib.lr_shared_decode(m.cache, q, i32(m.lens), out)
    assert torch.equal(out, a[0])
    b = m.decode(q)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("hq,r,new", [(28, 256, 1), (28, 512, 1), (64, 512, 1)])
def test_decode_rising_scores_raise_the_maximum_often(lib, hq, r, new):
    """Scores that grow along the context: the running maxima move in every tile of every run, and
    with them every accumulator is rescaled."""
    import torch
    m = Layer(lib, [3000, 1000], hq=hq, hkv=hq, r=r, dn=64, dv=64, scale=1.0, stale=False)
    ramp = np.concatenate([np.arange(n) for n in m.lens]) / 20.0
    m.kr[:, 0] = bf16(ramp)
    seq = np.repeat([0, 1], m.lens)
    lib.lr_shared_append(m.cache, m.c, m.kr, i32(seq), i32(np.concatenate([np.arange(n) for n in m.lens])))
    m.kr64 = f64(m.kr)
    q = m.query(1, 0.3)
    q[..., 64] = 1.0
    m.check_decode(q, *m.decode(q))


@pytest.mark.parametrize("r", [128, 320])
def test_decode_captured_and_replayed_with_other_lengths_and_pages(lib, r):
    import torch
    m = Layer(lib, [260, 300], hq=8, hkv=8, r=r)
    q = m.query(1)
    lens = i32([260, 300])
    out = torch.zeros((2, 1, 8, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((2, 1, 8), dtype=torch.float32, device="cuda")
    table = i32(m.table)
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        lib.lr_shared_decode(m.cache, q, lens, out, lse)      # first launches outside the capture
    torch.cuda.current_stream().wait_stream(s)
    with torch.cuda.graph(g):
        lib.lr_shared_set_block_table_device(m.cache, table)
        lib.lr_shared_decode(m.cache, q, lens, out, lse)
    for new in ([260, 300], [1, 129], [0, 256]):
        lens.copy_(i32(new))
        g.replay()
        torch.cuda.synchronize()
        m.check_decode(q, out, lse, lens=new)
    # swapped pages: sequence 0 now reads sequence 1's tokens
    table.copy_(i32(m.table[::-1].copy()))
    lens.copy_(i32([300, 260]))
    g.replay()
    torch.cuda.synchronize()
    swapped = out.clone()
    lib.lr_shared_set_block_table(m.cache, m.table)
    again, _ = m.decode(torch.flip(q, [0]).contiguous(), [260, 300])
    assert torch.equal(swapped, torch.flip(again, [0]))


def test_decode_on_another_stream(lib):
    import torch
    m = Layer(lib, [130, 60])
    q = m.query(1)
    want = m.decode(q)
    s = torch.cuda.Stream()
    out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    lens = i32(m.lens)
    s.wait_stream(torch.cuda.current_stream())
    lib.lr_shared_decode(m.cache, q, lens, out, lse, stream=s)
    s.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_bad_device_pages_are_clamped(lib):
    """Entries outside the pool read some page of it, never memory outside."""
    import torch
    m = Layer(lib, [200, 100], stale=False)
    lib.lr_shared_set_block_table_device(m.cache, i32([[-5, 1 << 30], [7, -(1 << 31)]]))
    q = m.query(1)
    out, lse = m.decode(q)
    assert torch.isfinite(out.float()).all()
    lib.lr_shared_set_block_table(m.cache, m.table)
    m.check_decode(q, *m.decode(q))


@pytest.mark.parametrize("r,bits", [(256, 0), (512, 0), (512, 8)])
def test_waits_that_give_up_are_reported_and_the_cache_recovers(lib, r, bits):
    m = Layer(lib, [500, 129], hq=8, hkv=8, r=r, bits=bits)
    q = m.query(1)
    import torch
    out, lens = torch.zeros((2, 1, 8, 128), dtype=torch.bfloat16, device="cuda"), i32(m.lens)
    lib.lr_shared_set_wait_limit(m.cache, 4)
    lib.lr_shared_decode(m.cache, q, lens, out)
    torch.cuda.synchronize()
    assert lib.lr_shared_device_error(m.cache) == lib.LR_ERR_TIMEOUT
    assert lib.lr_shared_device_error(m.cache) == 0
    lib.lr_shared_set_wait_limit(m.cache, 0)
    m.check_decode(q, *m.decode(q))


@pytest.mark.parametrize("r,bits", [(64, 0), (512, 0), (512, 8)])
def test_steps_without_a_pause(lib, r, bits):
    """Appends, lengths and decodes follow one another on a stream with nothing between: each decode
    reads what the calls before it wrote, as it does when the GPU is waited for after every call."""
    import torch
    B, hq, steps = 3, 16, 96
    got = []
    for pause in (False, True):
        m = Layer(lib, [100, 1, 250], hq=hq, hkv=hq, r=r, bits=bits, cap=512)
        rng = np.random.default_rng(5)
        c, kr = bf16(rng.standard_normal((steps, B, r)) * 3), bf16(rng.standard_normal((steps, B, 64)))
        q = bf16(rng.standard_normal((steps, B, 1, hq, 192)))
        out = torch.zeros((steps, B, 1, hq, 128), dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros((steps, B, 1, hq), dtype=torch.float32, device="cuda")
        seq, lens = i32(np.arange(B)), i32(m.lens)
        torch.cuda.synchronize()
        for i in range(steps):
            for call in (lambda: lib.lr_shared_append(m.cache, c[i], kr[i], seq, lens), lambda: lens.add_(1),
                         lambda: lib.lr_shared_decode(m.cache, q[i], lens, out[i], lse[i])):
                call()
                if pause:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert lib.lr_shared_device_error(m.cache) == 0
        got.append((out, lse))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert got[0][0].abs().sum() > 0


def test_decodes_of_two_caches_at_once(lib):
    """Caches own their scratch: decodes of two of them may overlap, on two streams."""
    import torch
    ms = [Layer(lib, lens, hq=28, hkv=28, r=r, bits=bits) for lens, r, bits in (([900, 31, 400], 512, 0), ([700, 1200], 320, 8))]
    qs, streams = [m.query(1) for m in ms], [torch.cuda.Stream() for _ in ms]
    want = [m.decode(q) for m, q in zip(ms, qs)]
    lens = [i32(m.lens) for m in ms]
    got = [[(torch.zeros_like(w[0]), torch.zeros_like(w[1])) for _ in range(8)] for w in want]
    torch.cuda.synchronize()
    for n in range(8):
        for m, q, s, l, g in zip(ms, qs, streams, lens, got):
            lib.lr_shared_decode(m.cache, q, l, *g[n], stream=s)
    torch.cuda.synchronize()
    for m, q, w, g in zip(ms, qs, want, got):
        assert lib.lr_shared_device_error(m.cache) == 0
        m.check_decode(q, *w)
        assert all(torch.equal(o, w[0]) and torch.equal(e, w[1]) for o, e in g)


# Scores from the rotary part alone, 8 bits times a power of two and so exact in fp32: far from zero on
# either side.  (sign, power): sign 2^power or, where its product with log2(e) rounds, 165/128 of it.
FAR = [(s * f, p) for f in (1.0, 165 / 128) for s, p in ((-1, 110), (-1, 60), (-1, 35), (1, 35), (1, 110))] + [
    (s * 165 / 128, p) for s, p in ((-1, 32), (-1, 30), (1, 29), (-1, 25))]


def far_scores(n, sign, power):
    """Scores of n keys and which of them carry all the weight: half of the keys, in no order, stand at
    sign 2^power; the others at twice (half) that where that is less."""
    pick = np.random.default_rng(n).random(n) < 0.5
    pick[0] = True
    low = sign * 2.0 ** (power + (1 if sign < 0 else -1))
    return np.where(pick, sign * 2.0 ** power, low), pick


@pytest.mark.parametrize("sign,power", FAR)
@pytest.mark.parametrize("hq,r,bits,n", [(4, 128, 0, 700), (28, 512, 0, 129), (28, 512, 8, 129), (6, 256, 8, 3000)])
def test_decode_of_scores_far_from_zero(lib, hq, r, bits, n, sign, power):
    """A maximum of -2^110 is a maximum as any other: equal scores weigh the same, lower ones nothing."""
    m = Layer(lib, [n], hq=hq, hkv=hq, r=r, bits=bits, dn=64, dv=64, scale=1.0)
    s, pick = far_scores(n, sign, power)
    m.kr.zero_()
    m.kr[:, 3] = bf16(s / 2.0 ** 60)
    lib.lr_shared_append(m.cache, m.c, m.kr, i32(np.zeros(n)), i32(np.arange(n)))
    q = m.query(1, 0.0)
    q[..., 64 + 3] = 2.0 ** 60
    out, lse = map(f64, m.decode(q))
    # the lse: scale log2(e) and its product each round once, as do log2(e) itself and the factor back
    want = sign * 2.0 ** power + np.log(pick.sum())
    assert np.all(np.abs(lse - want) <= 8 * F * abs(want) + 2.0 ** -20)
    # equal weights 2^x of one rounding (u), in the numerator; sums of n + r fp32 steps, two halves; the output
    rows = S.expand(m.c64[pick], m.Bv64, hq)
    A = (np.abs(m.c64[pick]).mean(axis=0) @ np.abs(m.Bv64)).reshape(hq, 64)
    tol = U * np.abs(rows.mean(axis=0)) + U * np.abs(rows).mean(axis=0) + (U * U + (n + r + 64) * F) * A
    assert np.all(np.abs(out[0, 0] - rows.mean(axis=0)) <= tol)


# ---------------------------------------------------------------------------
# expansion
# ---------------------------------------------------------------------------

def run_expand(m, first, lens, spare=3):
    """Packed expansion of tokens first[b] .. first[b] + lens[b] - 1, with rows to spare behind."""
    import torch
    T = sum(lens) + spare
    k = torch.full((T, m.hkv, m.dn), 55.0, dtype=torch.bfloat16, device="cuda")
    v = torch.full((T, m.hkv, m.dv), 55.0, dtype=torch.bfloat16, device="cuda")
    kr = torch.full((T, m.dr), 55.0, dtype=torch.bfloat16, device="cuda")
    cu = i32(np.concatenate([[0], np.cumsum(lens)]))
    m.lib.lr_shared_expand(m.cache, cu, k, v, kr, start=None if first is None else i32(first))
    assert m.lib.lr_shared_device_error(m.cache) == 0
    return k, v, kr, cu


def check_expand(m, first, lens, k, v, kr):
    """One rounding to bf16 (u) of an fp32 sum of r products."""
    idx = np.concatenate([m.cu[b] + f + np.arange(n) for b, (f, n) in enumerate(zip(first, lens))]).astype(int)
    c, n = m.c64[idx], len(idx)
    for got, B, w in ((k, m.Bk64, m.hkv * m.dn), (v, m.Bv64, m.hkv * m.dv)):
        want, mag = c @ B, np.abs(c) @ np.abs(B)
        err = np.abs(f64(got)[:n].reshape(n, w) - want)
        assert np.all(err <= U * np.abs(want) + (m.r + 8) * F * mag)
        assert np.all(f64(got)[n:] == 55)
    assert np.array_equal(f64(kr)[:n], m.kr64[idx]) and np.all(f64(kr)[n:] == 55)


@pytest.mark.parametrize("bits", [0, 8])
@pytest.mark.parametrize("hkv,r,dn,dr,dv", [(1, 64, 64, 32, 64), (3, 192, 128, 64, 64), (5, 448, 64, 32, 128),
                                            (28, 512, 128, 64, 128)])
def test_expand_matches_the_oracle(lib, bits, hkv, r, dn, dr, dv):
    m = Layer(lib, LENS, hq=hkv, hkv=hkv, r=r, dn=dn, dr=dr, dv=dv, bits=bits)
    k, v, kr, _ = run_expand(m, None, m.lens)
    check_expand(m, [0] * len(LENS), m.lens, k, v, kr)


@pytest.mark.parametrize("bits", [0, 8])
def test_expand_parts_that_start_and_end_inside_pages(lib, bits):
    m = Layer(lib, [300, 257, 129, 600], hq=2, hkv=2, r=128, bits=bits)
    first, lens = [127, 256, 60, 1], [2, 1, 0, 599]
    k, v, kr, _ = run_expand(m, first, lens)
    check_expand(m, first, lens, k, v, kr)


def test_expand_many_tiles_per_run(lib):
    """Runs that cross tiles and sequences: more (page, column block) units than SMs."""
    m = Layer(lib, [2000, 3000, 1, 4000], hq=10, hkv=10, r=320)
    k, v, kr, _ = run_expand(m, None, m.lens)
    check_expand(m, [0] * 4, m.lens, k, v, kr)


def test_expand_outside_the_cache_writes_nothing(lib):
    m = Layer(lib, [128, 128], hq=2, hkv=2, r=64, dn=64, dv=64)
    k, v, kr, _ = run_expand(m, [-3, 126], [5, 6], spare=0)
    got = f64(k)
    assert np.all(got[:3] == 55) and np.all(got[7:] == 55)      # positions -3..-1, and 128..131
    want = m.c64[[0, 1, 254, 255]] @ m.Bk64
    assert np.allclose(got[3:7].reshape(4, -1), want, atol=0.02)
    assert np.array_equal(f64(kr)[3:7], m.kr64[[0, 1, 254, 255]])


def test_expand_of_fewer_rows_than_the_parts_hold(lib):
    """total bounds the rows, however many tokens cu speaks of (here 2 million, in a few zero pages)."""
    import torch
    d = lib.make_shared_desc(8, 1, 1, 64, 32, 64, 64, 1 << 18, n_pages=4)
    cache = lib.lr_shared_create(d, bf16(np.ones((64, 64))), bf16(np.ones((64, 64))))
    cu = i32(np.arange(9) << 18)
    k, v, kr = (torch.full((n, *x), 55.0, dtype=torch.bfloat16, device="cuda") for n, x in
                ((20001, (1, 64)), (20001, (1, 64)), (20001, (32,))))
    lib.lr_shared_expand(cache, cu, k[:20000], v[:20000], kr[:20000])
    assert lib.lr_shared_device_error(cache) == 0
    for x in (k, v, kr):
        assert not x[:20000].any() and (x[20000] == 55).all()


@pytest.mark.parametrize("bits", [0, 8])
def test_expand_of_parts_that_do_not_ascend_is_bounded_and_reported(lib, bits):
    """64 parts that all claim the same 20000 rows: far more tiles than those rows can have."""
    import torch
    d = lib.make_shared_desc(128, 1, 1, 64, 32, 64, 64, 1 << 15, n_pages=4, quant_bits=bits)
    cache = lib.lr_shared_create(d, bf16(np.ones((64, 64))), bf16(np.ones((64, 64))))
    k, v, kr = (torch.full((20001, *x), 55.0, dtype=torch.bfloat16, device="cuda") for x in ((1, 64), (1, 64), (32,)))
    lib.lr_shared_expand(cache, i32([0, 20000] * 64 + [0]), k[:20000], v[:20000], kr[:20000])
    assert lib.lr_shared_device_error(cache) == lib.LR_ERR_INVALID_ARG
    assert all((x[20000] == 55).all() for x in (k, v, kr))
    lib.lr_shared_expand(cache, i32([0] + [20000] * 128), k[:20000], v[:20000], kr[:20000])
    assert lib.lr_shared_device_error(cache) == 0
    assert not any(x[:20000].any() for x in (k, v, kr)) and all((x[20000] == 55).all() for x in (k, v, kr))


@pytest.mark.parametrize("bits", [0, 8])
def test_expand_captured_and_replayed_with_other_parts(lib, bits):
    import torch
    m = Layer(lib, [300, 513, 40], hq=3, hkv=3, r=192, bits=bits)
    cu, start = i32([0, 0, 0, 0]), i32([0, 0, 0])
    k, v, kr = (torch.zeros((600, *x), dtype=torch.bfloat16, device="cuda") for x in ((3, 128), (3, 128), (64,)))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        lib.lr_shared_expand(m.cache, cu, k, v, kr, start=start)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.lr_shared_expand(m.cache, cu, k, v, kr, start=start)
    for first, lens in (([0, 0, 0], [300, 260, 40]), ([299, 100, 39], [1, 400, 1]), ([0, 0, 5], [0, 0, 3])):
        start.copy_(i32(first)), cu.copy_(i32(np.concatenate([[0], np.cumsum(lens)])))
        for x in (k, v, kr):
            x.fill_(55.0)
        g.replay()
        check_expand(m, first, lens, k, v, kr)


@pytest.mark.parametrize("bits", [0, 8])
def test_expansions_at_once_and_one_that_gives_up(lib, bits):
    """Two caches expanded on two streams again and again; then waits that give up are reported, and
    the cache recovers."""
    import torch
    ms = [Layer(lib, lens, hq=4, hkv=4, r=r, dn=64, dv=64, bits=bits) for lens, r in (([700, 300], 64), ([1, 129, 500], 512))]
    outs = [run_expand(m, None, m.lens) for m in ms]
    streams = [torch.cuda.Stream() for _ in ms]
    got = [[torch.zeros_like(x) for x in o[:3]] for o in outs]
    torch.cuda.synchronize()
    for _ in range(8):
        for m, s, o, g in zip(ms, streams, outs, got):
            lib.lr_shared_expand(m.cache, o[3], *g, stream=s)
    torch.cuda.synchronize()
    for m, o, g in zip(ms, outs, got):
        check_expand(m, [0] * len(m.lens), m.lens, *o[:3])
        assert all(torch.equal(x[:sum(m.lens)], y[:sum(m.lens)]) for x, y in zip(g, o))
    m = ms[1]
    lib.lr_shared_set_wait_limit(m.cache, 4)
    lib.lr_shared_expand(m.cache, outs[1][3], *got[1])
    assert lib.lr_shared_device_error(m.cache) == lib.LR_ERR_TIMEOUT
    assert lib.lr_shared_device_error(m.cache) == 0
    lib.lr_shared_set_wait_limit(m.cache, 0)
    check_expand(m, [0] * 3, m.lens, *run_expand(m, None, m.lens)[:3])


# ---------------------------------------------------------------------------
# ragged attention
# ---------------------------------------------------------------------------

def attn_case(lib, nq, nk, hq=4, hkv=4, dn=128, dr=64, dv=128, seed=0, amp=1.5, behind=5, scale=0.0):
    """Inputs of ragged attention, with non-finite rows behind the last sequence."""
    rng = np.random.default_rng(seed)
    Tq, Tk = sum(nq), sum(nk)
    q = bf16(rng.standard_normal((Tq + 2, hq, dn + dr)) * amp)
    k, kr, v = (rng.standard_normal(x) for x in ((Tk + behind, hkv, dn), (Tk + behind, dr), (Tk + behind, hkv, dv)))
    if behind:
        k[Tk:], kr[Tk:], v[Tk:] = np.nan, np.inf, np.inf
    d = lib.make_shared_desc(1, hq, hkv, dn, dr, dv, 64, 128, softmax_scale=scale)
    cache = lib.lr_shared_create(d, bf16(np.zeros((64, hkv * dn))), bf16(np.zeros((64, hkv * dv))))
    cu = [i32(np.concatenate([[0], np.cumsum(x)])) for x in (nq, nk)]
    return cache, q, bf16(k), bf16(kr), bf16(v), cu


def run_attn(lib, cache, q, k, kr, v, cu, causal):
    import torch
    d = cache.desc
    out = torch.full((q.shape[0], d.n_q_heads, d.dim_v), 33.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((q.shape[0], d.n_q_heads), 33.0, dtype=torch.float32, device="cuda")
    lib.lr_shared_attn(cache, q, k, kr, v, cu[0], cu[1], out, lse, causal=causal)
    assert lib.lr_shared_device_error(cache) == 0
    return out, lse


def check_attn(q, k, kr, v, nq, nk, causal, scale, out, lse):
    """Scores: dn + dr fp32 steps, log2 / exp2 in fp32 (2^-20 of their size): E.  Weights: one bf16
    rounding; sums: (m + 64) fp32 steps; the output: u of its value."""
    q64, k64, kr64, v64, o64, l64 = map(f64, (q, k, kr, v, out, lse))
    a = b = 0
    for n, m in zip(nq, nk):
        Q, K, R, V = q64[a:a + n], k64[b:b + m], kr64[b:b + m], v64[b:b + m]
        g = Q.shape[1] // K.shape[1]
        for j in range(Q.shape[1]):
            key = np.concatenate([K[:, j // g], R], axis=1)
            s = Q[:, j] @ key.T * scale
            if causal:
                s = np.where(np.arange(m) <= np.arange(n)[:, None] + m - n, s, -np.inf)
            none = ~np.any(np.isfinite(s), axis=1) if m else np.ones(n, bool)
            assert np.all(o64[a:a + n, j][none] == 0) and np.all(np.isneginf(l64[a:a + n, j][none]))
            if np.all(none):
                continue
            s = s[~none]
            top = s.max(axis=1, keepdims=True)
            p = np.exp(s - top)
            tot = p.sum(axis=1, keepdims=True)
            rl = (top + np.log(tot))[:, 0]
            p /= tot
            ro, mix = p @ V[:, j // g], p @ np.abs(V[:, j // g])
            mag = (np.abs(Q[:, j][~none]) @ np.abs(key).T).max(axis=1) * scale
            E = ((key.shape[1] + 8) * F + 2.0 ** -20) * mag
            assert np.all(np.abs(l64[a:a + n, j][~none] - rl) <= E + (m + 64) * F + 2.0 ** -21 * np.abs(rl)), (n, m, j)
            tol = U * np.abs(ro) + (U + 2 * E[:, None] + (m + 64) * F) * mix
            err = np.abs(o64[a:a + n, j][~none] - ro)
            assert np.all(err <= tol), (n, m, j, (err / tol).max())
        a, b = a + n, b + m
    assert np.all(o64[a:] == 33) and np.all(l64[a:] == 33)       # rows behind the last sequence: untouched


RAGGED = [([1, 127, 128, 129, 0, 257, 300], [1, 127, 128, 129, 0, 257, 300]),      # prompts
          ([1, 5, 130, 256, 1], [300, 128, 700, 1000, 129]),                         # chunks of longer contexts
          ([200, 3, 300, 2], [5, 0, 129, 1])]                                        # fewer keys than queries


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,nk", RAGGED)
@pytest.mark.parametrize("hq,hkv,dn,dr,dv", [(4, 4, 128, 64, 128), (6, 2, 64, 32, 64), (3, 3, 128, 32, 64),
                                             (4, 1, 64, 64, 128)])
def test_attn_matches_the_oracle(lib, nq, nk, causal, hq, hkv, dn, dr, dv):
    case = attn_case(lib, nq, nk, hq, hkv, dn, dr, dv)
    out, lse = run_attn(lib, *case, causal)
    check_attn(*case[1:5], nq, nk, causal, (dn + dr) ** -0.5, out, lse)


@pytest.mark.parametrize("amp", [0.0, 40.0])
def test_attn_equal_and_sharp_weights(lib, amp):
    nq = nk = [700, 130]
    case = attn_case(lib, nq, nk, amp=amp)
    out, lse = run_attn(lib, *case, True)
    check_attn(*case[1:5], nq, nk, True, 192 ** -0.5, out, lse)


@pytest.mark.parametrize("hq,nq,nk", [(4, 300, 700), (2, 5, 5000)])
def test_attn_of_equal_weights_other_than_one(lib, hq, nq, nk):
    """As for the decode: every 64th key has weight 1, the others one that rounds by nearly half a step."""
    w = 0.5 * (1 + 2.0 ** -8 - 2.0 ** -13)
    cache, q, k, kr, v, cu = attn_case(lib, [nq], [nk], hq, hq, 64, 64, 64, behind=0, scale=-float(np.log(w)))
    q.zero_(), kr.zero_()
    q[:, :, 64 + 3], kr[:, 3] = 1.0, bf16(np.where(np.arange(nk) % 64 == 0, 0.0, -1.0))
    v[:] = v[:1].clone()
    out, lse = map(f64, run_attn(lib, cache, q, k, kr, v, cu, True))
    seen = np.arange(nq) + nk - nq + 1
    high = (seen + 63) // 64
    assert np.all(np.abs(lse[:nq] - np.log(high + (seen - high) * w)[:, None]) <= 2.0 ** -18)
    want = f64(v)[0]
    assert np.all(np.abs(out[:nq] - want) <= (U * (2 + U) + (nk + 64) * F) * np.abs(want))


def test_attn_rising_scores_raise_the_maximum_often(lib):
    """Keys that grow along the sequence: every key tile raises the running maximum, so O is
    rescaled again and again."""
    import torch
    nq, nk = [260], [1500]
    cache, q, k, kr, v, cu = attn_case(lib, nq, nk, 2, 2, 64, 64, 64, behind=0, scale=1.0)
    ramp = torch.arange(1500, device="cuda").float() / 10
    q[:, :, 0], k[:, :, 0] = 1.0, ramp[:, None].to(torch.bfloat16)
    out, lse = run_attn(lib, cache, q, k, kr, v, cu, True)
    check_attn(q, k, kr, v, nq, nk, True, 1.0, out, lse)


@pytest.mark.parametrize("sign,power", FAR)
@pytest.mark.parametrize("hq,hkv,nq,nk", [(4, 4, 300, 700), (28, 28, 260, 260), (2, 1, 5, 5000)])
def test_attn_of_scores_far_from_zero(lib, hq, hkv, nq, nk, sign, power):
    """As for the decode: plain, causal and split over a cluster."""
    cache, q, k, kr, v, cu = attn_case(lib, [nq], [nk], hq, hkv, 64, 64, 64, behind=0, scale=1.0)
    s, pick = far_scores(nk, sign, power)
    q.zero_(), kr.zero_()
    q[:, :, 64 + 3], kr[:, 3] = 2.0 ** 60, bf16(s / 2.0 ** 60)
    out, lse = map(f64, run_attn(lib, cache, q, k, kr, v, cu, True))
    seen = pick & (np.arange(nk) <= np.arange(nq)[:, None] + nk - nq)
    n = seen.sum(axis=1, keepdims=True)
    want = sign * 2.0 ** power + np.log(n)
    assert np.all(np.abs(lse[:nq] - want) <= 8 * F * np.abs(want) + 2.0 ** -20)
    v64 = np.repeat(f64(v), hq // hkv, axis=1)
    ro, mix = (np.einsum("ij,jhd->ihd", seen / n, x) for x in (v64, np.abs(v64)))
    assert np.all(np.abs(out[:nq] - ro) <= U * np.abs(ro) + (U + (nk + 64) * F) * mix)


@pytest.mark.parametrize("hq,hkv,nq,nk", [(4, 4, [100, 300, 40], [100, 600, 40]), (28, 7, [5, 260, 3], [70, 260, 3]),
                                          (2, 1, [3, 9, 7], [130, 5000, 900])])
def test_attn_over_visible_infinities_and_nans(lib, hq, hkv, nq, nk):
    """A score of -infinity weighs nothing; one of +infinity, or NaN, makes NaN of the queries that see it and
    of no other (those of its sequence may be rescaled along with them: both results are within u |out| + u of
    the mean of |v|, and a little, of the truth); an infinite value is infinite in its column for the queries that see it; other sequences
    are as without."""
    import torch
    cache, q, k, kr, v, cu = attn_case(lib, nq, nk, hq, hkv, 64, 32, 64)
    q[..., 64:] = 0.0
    q[..., 64 + 5] = 1.0
    want, wl = run_attn(lib, cache, q, k, kr, v, cu, True)
    a, b = nq[0], nk[0]
    t = nk[1] - nq[1] // 2                                     # a key of the second sequence
    mine = np.arange(a, a + nq[1])
    sees = torch.tensor(mine[np.arange(nq[1]) + nk[1] - nq[1] >= t]).cuda()
    not_ = torch.tensor(np.setdiff1d(np.arange(q.shape[0]), sees.cpu().numpy())).cuda()
    other = torch.tensor(np.setdiff1d(np.arange(q.shape[0]), mine)).cuda()
    low = kr.clone()
    low[b + t, 5] = -3e38
    none = kr.clone()
    none[b + t, 5] = -np.inf
    x, y = run_attn(lib, cache, q, k, low, v, cu, True), run_attn(lib, cache, q, k, none, v, cu, True)
    assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1]) and not torch.equal(x[0][sees], want[sees])
    for bad in (np.inf, np.nan):
        z = kr.clone()
        z[b + t, 5] = bad
        out, lse = run_attn(lib, cache, q, k, z, v, cu, True)
        assert torch.isnan(out[sees].float()).all() and torch.isnan(lse[sees]).all()
        assert torch.equal(out[other], want[other]) and torch.equal(lse[other], wl[other])
        assert (out[not_].float() - want[not_].float()).abs().max() <= 4.1 * U * v[:sum(nk)].abs().max()
        assert torch.allclose(lse[not_], wl[not_], rtol=2.0 ** -18, atol=2.0 ** -18)
    for bad in (np.inf, -np.inf, np.nan):
        z = v.clone()
        z[b + t, hkv - 1, 7] = bad
        out, lse = run_attn(lib, cache, q, k, kr, z, cu, True)
        g = hq // hkv
        hit = out[sees][:, hq - g:, 7].float()
        assert torch.isnan(hit).all() if np.isnan(bad) else (hit == bad).all()
        assert torch.equal(lse, wl) and torch.equal(out[other], want[other])
        rest = [c for c in range(64) if c != 7]
        assert torch.equal(out[..., rest], want[..., rest]) and torch.equal(out[:, :hq - g], want[:, :hq - g])


def test_attn_without_keys_or_queries(lib):
    import torch
    cache, q, k, kr, v, cu = attn_case(lib, [3, 4], [0, 0], behind=0)
    out, lse = run_attn(lib, cache, q, k, kr, v, cu, False)
    assert torch.all(out[:7] == 0) and torch.all(torch.isneginf(lse[:7])) and torch.all(out[7:] == 33)
    lib.lr_shared_attn(cache, q[:0], k, kr, v, i32([0]), i32([0]), out[:0], lse[:0])


def test_attn_joins_over_key_ranges_by_lse(lib):
    """A chunk against its context in two calls (the context whole, itself causal) equals one call."""
    import torch
    n, ctx = 150, 400
    cache, q, k, kr, v, cu = attn_case(lib, [n], [ctx + n], behind=0)
    q = q[:n].contiguous()
    whole, wl = run_attn(lib, cache, q, k, kr, v, cu, True)
    a, al = run_attn(lib, cache, q, k[:ctx], kr[:ctx], v[:ctx], (cu[0], i32([0, ctx])), False)
    b, bl = run_attn(lib, cache, q, k[ctx:], kr[ctx:], v[ctx:], (cu[0], i32([0, n])), True)
    l = torch.logaddexp(al, bl)
    joined = a.float() * (al - l).exp()[..., None] + b.float() * (bl - l).exp()[..., None]
    assert torch.allclose(l, wl, atol=1e-5, rtol=1e-5)
    # each side is within u (|o| + mix) of the truth; |v| <= 6 here
    assert (joined - whole.float()).abs().max() <= 4 * U * 6


def test_attn_captured_and_replayed_with_other_lengths(lib):
    import torch
    nq, nk = [100, 300], [300, 301]
    cache, q, k, kr, v, cu = attn_case(lib, nq, nk)
    out = torch.zeros((q.shape[0], 4, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((q.shape[0], 4), dtype=torch.float32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        lib.lr_shared_attn(cache, q, k, kr, v, cu[0], cu[1], out, lse)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.lr_shared_attn(cache, q, k, kr, v, cu[0], cu[1], out, lse)
    for nq, nk in (([100, 300], [300, 301]), ([257, 143], [600, 1]), ([0, 1], [5, 600 - 5])):
        cu[0].copy_(i32(np.concatenate([[0], np.cumsum(nq)])))
        cu[1].copy_(i32(np.concatenate([[0], np.cumsum(nk)])))
        out.fill_(33.0), lse.fill_(33.0)
        g.replay()
        check_attn(q, k, kr, v, nq, nk, True, 192 ** -0.5, out, lse)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hkv,dn,dr,dv", [(1, 1, 128, 64, 128), (2, 2, 64, 32, 64), (3, 1, 64, 64, 128), (5, 5, 128, 32, 64)])
@pytest.mark.parametrize("nq,nk", [([1], [4097]), ([50], [5000]), ([257], [2050]), ([300, 40], [3000, 129]),
                                   ([130, 1], [1, 4000]), ([5, 0, 200], [0, 900, 3500]), ([400], [1100])])
def test_attn_of_few_queries_over_many_keys(lib, nq, nk, causal, hq, hkv, dn, dr, dv):
    """Few CTAs' worth of queries: the keys are split over a cluster, parts may be empty or see nothing."""
    cache, q, k, kr, v, cu = attn_case(lib, nq, nk, hq=hq, hkv=hkv, dn=dn, dr=dr, dv=dv, seed=3)
    check_attn(q, k, kr, v, nq, nk, causal, (dn + dr) ** -0.5, *run_attn(lib, cache, q, k, kr, v, cu, causal))


@pytest.mark.parametrize("amp", [0.0, 30.0])
def test_attn_split_with_equal_and_sharp_weights(lib, amp):
    nq, nk = [70], [4500]
    cache, q, k, kr, v, cu = attn_case(lib, nq, nk, amp=amp)
    check_attn(q, k, kr, v, nq, nk, True, 192 ** -0.5, *run_attn(lib, cache, q, k, kr, v, cu, True))


@pytest.mark.parametrize("hq,dn,dr,dv", [(1, 128, 64, 128), (4, 64, 32, 64)])
@pytest.mark.parametrize("nq,nk", [([256], [4608]), ([130], [2306]), ([130, 256], [1, 4608])])
def test_attn_split_whose_last_part_is_the_second_query_tiles_alone(lib, nq, nk, hq, dn, dr, dv):
    """36 (19) key tiles in 8 parts of 5 (3), causal: the last part holds a key tile that the first 128
    queries do not see, so their tile is neither loaded nor read there."""
    import torch
    cache, q, k, kr, v, cu = attn_case(lib, nq, nk, hq=hq, hkv=hq, dn=dn, dr=dr, dv=dv, seed=4)
    want = run_attn(lib, cache, q, k, kr, v, cu, True)
    check_attn(q, k, kr, v, nq, nk, True, (dn + dr) ** -0.5, *want)
    for _ in range(20):
        got = run_attn(lib, cache, q, k, kr, v, cu, True)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_attn_split_captured_and_replayed_with_other_lengths(lib):
    import torch
    nq, nk = [40, 20], [3000, 2000]
    cache, q, k, kr, v, cu = attn_case(lib, nq, nk)
    out = torch.zeros((q.shape[0], 4, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((q.shape[0], 4), dtype=torch.float32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        lib.lr_shared_attn(cache, q, k, kr, v, cu[0], cu[1], out, lse)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.lr_shared_attn(cache, q, k, kr, v, cu[0], cu[1], out, lse)
    for nq, nk in (([40, 20], [3000, 2000]), ([1, 59], [5000, 0]), ([0, 60], [4, 4996]), ([30, 2], [129, 1])):
        cu[0].copy_(i32(np.concatenate([[0], np.cumsum(nq)])))
        cu[1].copy_(i32(np.concatenate([[0], np.cumsum(nk)])))
        out.fill_(33.0), lse.fill_(33.0)
        g.replay()
        kk, rr, vv = (x[:sum(nk)] for x in (k, kr, v))
        check_attn(q, kk, rr, vv, nq, nk, True, 192 ** -0.5, out, lse)


def test_attn_split_waits_that_give_up_are_reported(lib):
    import torch
    nq, nk = [300], [9000]
    cache, q, k, kr, v, cu = attn_case(lib, nq, nk)
    out = torch.zeros((q.shape[0], 4, 128), dtype=torch.bfloat16, device="cuda")
    lib.lr_shared_set_wait_limit(cache, 4)
    lib.lr_shared_attn(cache, q, k, kr, v, cu[0], cu[1], out)
    assert lib.lr_shared_device_error(cache) == lib.LR_ERR_TIMEOUT
    lib.lr_shared_set_wait_limit(cache, 0)
    check_attn(q, k, kr, v, nq, nk, True, 192 ** -0.5, *run_attn(lib, cache, q, k, kr, v, cu, True))


def test_attn_waits_that_give_up_are_reported(lib):
    nq, nk = [300, 40], [700, 129]
    cache, q, k, kr, v, cu = attn_case(lib, nq, nk)
    import torch
    out = torch.zeros((q.shape[0], 4, 128), dtype=torch.bfloat16, device="cuda")
    lib.lr_shared_set_wait_limit(cache, 4)
    lib.lr_shared_attn(cache, q, k, kr, v, cu[0], cu[1], out)
    assert lib.lr_shared_device_error(cache) == lib.LR_ERR_TIMEOUT
    lib.lr_shared_set_wait_limit(cache, 0)
    check_attn(q, k, kr, v, nq, nk, True, 192 ** -0.5, *run_attn(lib, cache, q, k, kr, v, cu, True))


# ---------------------------------------------------------------------------
# as they are used together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("bits", [0, 8])
def test_prompts_then_steps(lib, bits):
    """Two prompts written, expanded and attended; then three decode steps, each writing its token
    first.  Every result against full attention over what the cache stands for."""
    import torch
    H, r, dn, dr, dv, theta = 6, 192, 128, 64, 128, 1e4
    scale, lens, steps = (dn + dr) ** -0.5, [200, 126], 3
    rng = np.random.default_rng(5)
    T = [n + steps for n in lens]
    c = [bf16(rng.standard_normal((n, r))) for n in T]
    kr = [bf16(rng.standard_normal((n, dr))) for n in T]
    q = [bf16(rng.standard_normal((n, H, dn + dr))) for n in T]
    Bk, Bv = bf16(rng.standard_normal((r, H * dn)) / r ** 0.5), bf16(rng.standard_normal((r, H * dv)) / r ** 0.5)
    d = lib.make_shared_desc(2, H, H, dn, dr, dv, r, 256, quant_bits=bits, rope_theta=theta)
    cache = lib.lr_shared_create(d, Bk, Bv)
    lib.lr_shared_set_block_table(cache, np.array([[3, 0], [1, 2]]))
    lib.lr_shared_append(cache, torch.cat([x[:n] for x, n in zip(c, lens)]),
                         torch.cat([x[:n] for x, n in zip(kr, lens)]),
                         i32(np.repeat([0, 1], lens)), i32(np.concatenate([np.arange(n) for n in lens])))
    cu = i32([0, lens[0], sum(lens)])
    k = torch.zeros((sum(lens), H, dn), dtype=torch.bfloat16, device="cuda")
    v, kx = torch.zeros_like(k), torch.zeros((sum(lens), dr), dtype=torch.bfloat16, device="cuda")
    lib.lr_shared_expand(cache, cu, k, v, kx)
    qp = torch.cat([x[:n] for x, n in zip(q, lens)])
    out, lse = torch.zeros((sum(lens), H, dv), dtype=torch.bfloat16, device="cuda"), torch.zeros(
        (sum(lens), H), dtype=torch.float32, device="cuda")
    lib.lr_shared_attn(cache, qp, k, kx, v, cu, cu, out, lse)
    got = [[f64(out[:lens[0]])], [f64(out[lens[0]:])]]
    for s in range(steps):
        pos = [n + s for n in lens]
        lib.lr_shared_append(cache, torch.stack([x[p] for x, p in zip(c, pos)]),
                             torch.stack([x[p] for x, p in zip(kr, pos)]), i32([0, 1]), i32(pos))
        o = torch.zeros((2, 1, H, dv), dtype=torch.bfloat16, device="cuda")
        lib.lr_shared_decode(cache, torch.stack([x[p:p + 1] for x, p in zip(q, pos)]), i32([p + 1 for p in pos]), o)
        for b in range(2):
            got[b].append(f64(o[b]))
    for b, n in enumerate(T):
        z = f64(c[b])
        z = S.quantize_e4m3(z) if bits else z
        ref, _, mix = S.attention(f64(q[b]), S.expand(z, f64(Bk), H), S.rotate(f64(kr[b]), np.arange(n), theta),
                                  S.expand(z, f64(Bv), H), scale)
        # stored rotary keys and expanded keys are rounded to bf16: scores move by at most
        # u scale sum |q| |k|, which here stays below 0.2; values by u
        err = np.abs(np.concatenate(got[b]) - ref)
        assert np.sqrt((err ** 2).mean()) <= 2 * U * np.sqrt((mix ** 2).mean())
        assert err.max() <= 0.25 * mix.max()


@pytest.mark.parametrize("bits", [0, 8])
def test_pools_past_32_bits(lib, bits):
    """Pages whose first element (code) lies past 2^32 give what pages at the pool's start give."""
    import torch
    r, hq, lens = 512, 4, [200, 256]
    rng = np.random.default_rng(8)
    c, kr, q = bf16(rng.standard_normal((456, r))), bf16(rng.standard_normal((456, 64))), bf16(
        rng.standard_normal((2, 1, hq, 192)))
    B = bf16(rng.standard_normal((r, hq * 128)) / r ** 0.5)
    seq, pos = i32(np.repeat([0, 1], lens)), i32(np.concatenate([np.arange(n) for n in lens]))
    got = []
    for n in (4, (1 << 16) + 4):                               # 2^16 pages of 128 x 512
        cache = lib.lr_shared_create(lib.make_shared_desc(2, hq, hq, 128, 64, 128, r, 256, n_pages=n, quant_bits=bits), B, B)
        lib.lr_shared_set_block_table(cache, np.array([[n - 1, n - 3], [n - 4, n - 2]]))
        lib.lr_shared_append(cache, c, kr, seq, pos)
        x, y, out = torch.zeros_like(c), torch.zeros_like(kr), torch.zeros((2, 1, hq, 128), dtype=torch.bfloat16, device="cuda")
        k, v, z = torch.zeros((456, hq, 128), dtype=torch.bfloat16, device="cuda"), torch.zeros(
            (456, hq, 128), dtype=torch.bfloat16, device="cuda"), torch.zeros_like(kr)
        cu = i32([0, 200, 456])
        lib.lr_shared_read(cache, cu, x, y)
        lib.lr_shared_decode(cache, q, i32(lens), out)
        lib.lr_shared_expand(cache, cu, k, v, z)
        assert lib.lr_shared_device_error(cache) == 0
        got.append((x, y, out, k, v, z))
        lib.lr_shared_destroy(cache)
    assert all(torch.equal(a, b) and a.any() for a, b in zip(*got))
    assert np.array_equal(f64(got[1][0]), S.quantize_e4m3(f64(c)) if bits else f64(c))


def test_results_past_32_bits(lib):
    """Expanded rows, queries and outputs past element 2^31."""
    import torch
    H, n, parts = 128, 16900, 8
    d = lib.make_shared_desc(parts, H, H, 128, 64, 128, 64, 17024, n_pages=133)        # all sequences share the pages
    rng = np.random.default_rng(9)
    Bk, Bv = bf16(rng.standard_normal((64, H * 128)) / 8), bf16(rng.standard_normal((64, H * 128)) / 8)
    cache = lib.lr_shared_create(d, Bk, Bv)
    c, kr = bf16(rng.standard_normal((n, 64))), bf16(rng.standard_normal((n, 64)))
    lib.lr_shared_append(cache, c, kr, i32(np.zeros(n)), i32(np.arange(n)))
    T = n * parts
    k, v = (torch.zeros((T, H, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x = torch.zeros((T, 64), dtype=torch.bfloat16, device="cuda")
    lib.lr_shared_expand(cache, i32(np.arange(parts + 1) * n), k, v, x)
    assert lib.lr_shared_device_error(cache) == 0 and k.numel() > 1 << 31
    c64 = f64(c[-70:])
    for got, B in ((k, Bk), (v, Bv)):
        assert all(torch.equal(got[i * n:(i + 1) * n], got[:n]) for i in range(1, parts))
        want, mag = c64 @ f64(B), np.abs(c64) @ np.abs(f64(B))
        assert np.all(np.abs(f64(got[-70:]).reshape(70, -1) - want) <= U * np.abs(want) + (64 + 8) * F * mag)
    assert torch.equal(x, kr.repeat(parts, 1))
    k, v, x = k[:340].clone(), v[:340].clone(), x[:340].clone()
    nq = [131100, 100]
    q = torch.randn((sum(nq), H, 192), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros((sum(nq), H, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((sum(nq), H), dtype=torch.float32, device="cuda")
    lib.lr_shared_attn(cache, q, k, x, v, i32([0, nq[0], sum(nq)]), i32([0, 40, 340]), out, lse, causal=False)
    assert lib.lr_shared_device_error(cache) == 0 and out.numel() > 1 << 31
    for rows, keys in ((slice(0, 30), slice(0, 40)), (slice(131050, 131100), slice(0, 40)), (slice(131100, 131200), slice(40, 340))):
        check_attn(q[rows], k[keys], x[keys], v[keys], [rows.stop - rows.start], [keys.stop - keys.start], False,
                   192 ** -0.5, out[rows], lse[rows])


@pytest.mark.parametrize("bits", [0, 8])
def test_the_largest_batch(lib, bits):
    """1024 sequences, most of them empty or of a few tokens."""
    rng = np.random.default_rng(10)
    lens = rng.integers(0, 4, 1024)
    lens[[0, 31, 32, 500, 1023]] = 129, 0, 200, 256, 65
    m = Layer(lib, [int(n) for n in lens], hq=2, hkv=1, r=64, dn=64, dr=32, dv=64, bits=bits, new=2, stale=False)
    q = m.query(2)
    m.check_decode(q, *m.decode(q))
    k, v, kr, _ = run_expand(m, None, m.lens)
    check_expand(m, [0] * 1024, m.lens, k, v, kr)
    nq, nk = [int(n) for n in rng.integers(0, 3, 1024)], [int(n) for n in rng.integers(0, 4, 1024)]
    nq[7], nk[7], nk[900] = 300, 400, 1000
    case = attn_case(lib, nq, nk, 2, 2, 64, 32, 64)
    check_attn(*case[1:5], nq, nk, True, 96 ** -0.5, *run_attn(lib, *case, True))


@pytest.mark.parametrize("hq,r,bits", [(1, 64, 8), (7, 192, 8), (5, 512, 0)])
def test_decode_of_fewer_tokens_than_the_cache_allows(lib, hq, r, bits):
    m = Layer(lib, [300, 7, 64, 1], hq=hq, hkv=hq, r=r, dn=64, dv=64, bits=bits, new=8)
    for n in range(1, 9):
        q = m.query(n)
        m.check_decode(q, *m.decode(q))


def test_all_operators_at_once(lib):
    """Decode, expansion, attention with split keys and without, each on a stream of its own, again and
    again: they share SMs, shared memory and tensor memory, and wait for nobody but themselves."""
    import torch
    dec = Layer(lib, [900, 31, 400], hq=28, hkv=28, r=64, bits=8, dn=64, dr=32, dv=64)
    exp = Layer(lib, [700, 1200], hq=4, hkv=4, r=64, dn=64, dr=32, dv=64, seed=1)
    few = attn_case(lib, [200], [5000], 2, 2, 64, 32, 64)
    many = attn_case(lib, [300, 700], [300, 700], 28, 28, 64, 32, 64)
    q, lens, cu, main = dec.query(1), i32(dec.lens), i32(exp.cu), torch.cuda.current_stream()

    def calls(s):
        o = torch.zeros((3, 1, 28, 64), dtype=torch.bfloat16, device="cuda")
        e = [torch.zeros((1900, *x), dtype=torch.bfloat16, device="cuda") for x in ((4, 64), (4, 64), (32,))]
        a, b = (torch.zeros((c[1].shape[0], c[1].shape[1], 64), dtype=torch.bfloat16, device="cuda") for c in (few, many))
        for t in s:
            t.wait_stream(main)
        lib.lr_shared_decode(dec.cache, q, lens, o, stream=s[0])
        lib.lr_shared_expand(exp.cache, cu, *e, stream=s[1])
        for c, y, t in ((few, a, s[2]), (many, b, s[3])):
            lib.lr_shared_attn(*c[:5], *c[5], y, stream=t)
        return [o, *e, a, b]

    want = calls([main] * 4)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = [calls(streams) for _ in range(20)]
    torch.cuda.synchronize()
    for c in (dec.cache, exp.cache, few[0], many[0]):
        assert lib.lr_shared_device_error(c) == 0
    assert all(torch.equal(x, y) and y.any() for g in got for x, y in zip(g, want))


@pytest.mark.parametrize("r,bits", [(192, 8), (512, 0), (512, 8)])
def test_steps_captured_and_replayed(lib, r, bits):
    """Two steps (append, lengths, decode) in one graph, replayed, against the same steps one by one."""
    import torch
    B, hq, reps = 3, 16, 20
    rng = np.random.default_rng(6)
    c, kr = bf16(rng.standard_normal((reps, 2, B, r)) * 3), bf16(rng.standard_normal((reps, 2, B, 64)))
    q = bf16(rng.standard_normal((reps, 2, B, 1, hq, 192)))
    got = []
    for graph in (False, True):
        m = Layer(lib, [100, 1, 250], hq=hq, hkv=hq, r=r, bits=bits, cap=512)
        seq, lens = i32(np.arange(B)), i32(m.lens)
        x, y, w = c[0].clone(), kr[0].clone(), q[0].clone()
        out = torch.zeros((2, B, 1, hq, 128), dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros((2, B, 1, hq), dtype=torch.float32, device="cuda")

        def steps():
            for i in range(2):
                lib.lr_shared_append(m.cache, x[i], y[i], seq, lens)
                lens.add_(1)
                lib.lr_shared_decode(m.cache, w[i], lens, out[i], lse[i])

        m.decode(m.query(1))                                   # first launches outside the capture
        if graph:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                steps()
        res = []
        for i in range(reps):
            x.copy_(c[i]), y.copy_(kr[i]), w.copy_(q[i])
            g.replay() if graph else steps()
            res += [out.clone(), lse.clone()]
        torch.cuda.synchronize()
        assert lib.lr_shared_device_error(m.cache) == 0
        got.append(res)
    assert all(torch.equal(a, b) and a.any() for a, b in zip(*got))


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------

def test_refusals(lib):
    import torch
    m = Layer(lib, [5, 6], r=128, new=2)
    q = m.query(2)
    out = torch.zeros((2, 2, 4, 128), dtype=torch.bfloat16, device="cuda")
    lens = i32(m.lens)
    with pytest.raises(ValueError):
        lib.lr_shared_decode(m.cache, q.float(), lens, out)
    with pytest.raises(ValueError):
        lib.lr_shared_decode(m.cache, q, lens.cpu(), out)
    with pytest.raises(ValueError):
        lib.lr_shared_decode(m.cache, q, lens, out[:, :1])
    with pytest.raises(ValueError):
        lib.lr_shared_append(m.cache, m.c[:, :64], m.kr, i32(np.zeros(11)), i32(np.zeros(11)))
    with pytest.raises(ValueError):
        lib.lr_shared_append(m.cache, m.c.T.contiguous().T, m.kr, i32(np.zeros(11)), i32(np.zeros(11)))
    with pytest.raises(lib.LRError) as e:          # rows 129 elements apart: not 16-byte aligned
        w = torch.zeros((11, 129), dtype=torch.bfloat16, device="cuda")
        lib.lr_shared_append(m.cache, w[:, :128], m.kr, i32(np.zeros(11)), i32(np.zeros(11)))
    assert e.value.status == lib.LR_ERR_INVALID_ARG
    with pytest.raises(lib.LRError) as e:
        w = torch.zeros((11, 136), dtype=torch.bfloat16, device="cuda")
        lib.lr_shared_append(m.cache, w[:, 4:132], m.kr, i32(np.zeros(11)), i32(np.zeros(11)))
    assert e.value.status == lib.LR_ERR_INVALID_ARG
    q3 = torch.zeros((2, 3, 4, 192), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(lib.LRError) as e:
        lib.lr_shared_decode(m.cache, q3, lens, torch.zeros((2, 3, 4, 128), dtype=torch.bfloat16, device="cuda"))
    assert e.value.status == lib.LR_ERR_CAPACITY
    with pytest.raises(lib.LRError) as e:
        lib.lr_shared_set_block_table(m.cache, np.array([[0], [4]]))
    assert e.value.status == lib.LR_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        lib.lr_shared_set_block_table(m.cache, np.array([[0, 1], [0, 1]]))
    off = torch.zeros(q.numel() + 1, dtype=torch.bfloat16, device="cuda")[1:].reshape(q.shape)
    with pytest.raises(lib.LRError) as e:
        lib.lr_shared_decode(m.cache, off, lens, out)
    assert e.value.status == lib.LR_ERR_INVALID_ARG


def test_nothing_to_do(lib):
    import torch
    m = Layer(lib, [5, 6])
    none = torch.zeros((0, 128), dtype=torch.bfloat16, device="cuda")
    lib.lr_shared_append(m.cache, none, none[:, :64], i32([]), i32([]))
    lib.lr_shared_read(m.cache, i32([0, 0, 0]), none, torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda"))


def test_failed_allocations_leave_nothing_behind(lib):
    import torch
    d = lib.make_shared_desc(2, 4, 4, 128, 64, 128, 128, 256, quant_bits=8, rope_theta=1e4)
    Bk, Bv = bf16(np.zeros((128, 512))), bf16(np.zeros((128, 512)))
    lib.lr_shared_destroy(lib.lr_shared_create(d, Bk, Bv))
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    n = 0
    while True:
        lib.lr_debug_inject_fault(lib.LR_FAULT_ALLOC, n)
        try:
            cache = lib.lr_shared_create(d, Bk, Bv)
            break
        except lib.LRError as e:
            assert e.status == lib.LR_ERR_OOM
            assert torch.cuda.mem_get_info()[0] == free
        n += 1
    lib.lr_debug_inject_fault(lib.LR_FAULT_ALLOC, -1)
    assert n == 11
    lib.lr_shared_destroy(cache)
    assert torch.cuda.mem_get_info()[0] == free


def test_failed_launches_are_reported(lib):
    m = Layer(lib, [130, 60])
    q = m.query(1)
    for n in range(3):
        lib.lr_debug_inject_fault(lib.LR_FAULT_LAUNCH, n)
        with pytest.raises(lib.LRError) as e:
            m.decode(q)
        assert e.value.status == lib.LR_ERR_CUDA
    lib.lr_debug_inject_fault(lib.LR_FAULT_LAUNCH, -1)
    m.check_decode(q, *m.decode(q))
