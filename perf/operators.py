"""The shared-latent operators as they are measured: cases, inputs, plain forms and exact values.

A shared-latent cache keeps ONE latent c of rank r and one rotary key of dim_rope elements per
token.  Head h's key is [c B_k,h | rotary key], its value c B_v,h.  Four operators work on it:

write    lr_shared_append + lr_shared_read: tokens rotated, (for 8 bits) quantised, written to
         their pages, and read back
decode   lr_shared_decode: a few query tokens per sequence against the paged latents, absorbed
expand   lr_shared_expand: stored tokens read back as per-head keys and values
prefill  lr_shared_attn: ragged attention of expanded keys and values

In 8 bits a group of 32 ranks shares a power-of-two scale 2^e, the smallest with
max|c| <= 448 * 2^e, and every element is the nearest e4m3 value of c / 2^e.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

PAGE = 128
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _case(op, name=None, **kw):
    c = dict(op=op, heads=28, kv_heads=28, nope=128, rope=64, dv=128, rank=512, bits=0)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one decode step of a batch of 16: one token per sequence, latency-bound
        _case("write", "write_step16", batch=16, low=1, high=1, tokens=16, theta=1e6),
        # ragged prompts arriving together, held in 8 bits
        _case("write", "write_ragged_e4m3", batch=9, low=1, high=2000, tokens=6001, rank=448, bits=8, theta=1e4),
        # bulk prompts: 16 sequences of 4096 tokens, in 8 bits
        _case("write", "write_bulk_e4m3", batch=16, low=4096, high=4096, tokens=65536, bits=8, theta=1e6),
        # a single short conversation: latency of the whole call
        _case("decode", "decode_one517", batch=1, low=517, high=517, tokens=517, rank=256, new=1),
        # the batch of 16 at 4096 tokens, one layer of 28 query heads
        _case("decode", "decode_16x4k", batch=16, low=4096, high=4096, tokens=65536, new=1),
        # the batch of 16 at 32768 tokens, latents in 8 bits
        _case("decode", "decode_16x32k_e4m3", batch=16, low=32768, high=32768, tokens=524288, bits=8, new=1),
        # a serving batch at very different lengths, many heads, two draft tokens checked at once
        _case("decode", "decode_ragged_128h", batch=12, low=1, high=16000, tokens=50007, heads=128, kv_heads=128,
              new=2),
        # part of two contexts (starting inside a page) expanded for a chunk of a prompt
        _case("expand", "expand_chunk_e4m3", batch=3, low=1, high=900, tokens=1411, heads=16, kv_heads=16, rank=448,
              bits=8, skip=77),
        # a 32768-token context expanded for a long prompt
        _case("expand", "expand_32k", batch=2, low=12000, high=20768, tokens=32768, skip=0),
        # short ragged prompts
        _case("prefill", "prefill_short", batch=7, low=1, high=400, tokens=1203, ahead=0, causal=True),
        # two prompts of 8192 tokens
        _case("prefill", "prefill_2x8k", batch=2, low=8192, high=8192, tokens=16384, ahead=0, causal=True),
        # a chunk of new tokens against long contexts already held
        _case("prefill", "prefill_chunk", batch=2, low=200, high=823, tokens=1023, ahead=14001, causal=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["write", "decode", "expand", "prefill"])
    kv = rng.choice([1, 2, 4, 7, 8, 16, 20, 28, 32, 64, 128])
    group = rng.choice([g for g in (1, 1, 1, 2, 4, 7, 16) if kv * g <= 128])
    kw = dict(heads=kv * group, kv_heads=kv, nope=rng.choice([64, 128, 128]), rope=rng.choice([32, 64, 64]),
              dv=rng.choice([64, 128, 128]), rank=64 * rng.randint(1, 8), bits=rng.choice([0, 8]))
    batch = _log_int(rng, 1, 48)
    if op == "write":
        high = _log_int(rng, 1, max(1, 65536 // batch))
        kw.update(theta=rng.choice([1e4, 1e6]))
    elif op == "decode":
        high = _log_int(rng, 1, min(100000, 400000 // batch))
        kw.update(new=rng.choice([1, 1, 1, 2, 3, 4]))
    elif op == "expand":
        high = _log_int(rng, 1, max(1, min(16000, 900000 // (batch * kw["kv_heads"]))))
        kw.update(skip=rng.choice([0, 0, 128, rng.randint(1, 700)]))
    else:
        kw["bits"] = 0
        high = _log_int(rng, 1, max(1, min(4000, 300000 // (batch * kw["heads"]))))
        kw.update(ahead=rng.choice([0, 0, rng.randint(1, 4000)]), causal=rng.choice([True, True, False]))
    low = rng.choice([1, 1, max(1, high // 2), high])
    kw.update(batch=batch, low=low, high=high, tokens=_total(batch, low, high, rng))
    return _case(op, **kw)


def _total(batch, low, high, rng):
    """A total that lengths between low and high (or 1 and high) can reach."""
    return low if batch == 1 else (batch * high if low == high else rng.randint(batch * low, batch * high))


def _lengths(case):
    """Ragged lengths in [low, high] that add up to `tokens`; the same for every seed."""
    n, lo, hi, total = case["batch"], case["low"], case["high"], case["tokens"]
    rng = np.random.default_rng([n, lo, hi, total])
    w = rng.exponential(1.0, n)
    x = np.clip(np.floor(w / w.sum() * total), lo, hi).astype(np.int64)
    i = 0
    while x.sum() != total:                       # spread what is left over
        d = int(total - x.sum())
        k = i % n
        x[k] = min(max(x[k] + d, lo), hi)
        i += 1
        if i > 2 * n:
            break
    return [int(v) for v in x]


def work(case):
    L = _lengths(case)
    T, H, G = sum(L), case["heads"], case["kv_heads"]
    dn, dr, dv, r = case["nope"], case["rope"], case["dv"], case["rank"]
    stored = (r * 2 if case["bits"] == 0 else r + r // 32) + dr * 2
    op = case["op"]
    if op == "write":
        # tokens in, their stored form written and read once, tokens out; positions
        return {"bytes": T * (2 * (r + dr) * 2 + 2 * stored + 8), "flops": T * 6 * dr}
    if op == "decode":
        rows = case["batch"] * case["new"] * H
        weights = G * r * (dn + dv) * 2
        bytes_ = T * stored + weights + rows * ((dn + dr + dv) * 2 + 4)
        seen = sum(max(0, n - case["new"] + 1 + s) for n in L for s in range(case["new"]))
        return {"bytes": bytes_, "flops": 2 * seen * H * (2 * r + dr) + 2 * rows * r * (dn + dv)}
    if op == "expand":
        return {"bytes": T * (stored + (G * (dn + dv) + dr) * 2) + G * r * (dn + dv) * 2,
                "flops": 2 * T * r * G * (dn + dv)}
    keys = sum(n + case["ahead"] for n in L)
    pairs = sum((n * (case["ahead"] + (n + 1) / 2) if case["causal"] else n * (n + case["ahead"])) for n in L)
    return {"bytes": T * H * ((dn + dr + dv) * 2 + 4) + keys * (G * (dn + dv) + dr) * 2,
            "flops": 2 * pairs * H * (dn + dr + dv)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed((seed * 1000003 + salt) % (2 ** 62))
    return g


def _randn(shape, seed, salt, scale=1.0):
    return (torch.randn(shape, generator=_gen(seed, salt), device="cuda", dtype=F32) * scale).to(BF16)


def _latents(case, n, seed):
    """Normalised latents with a decaying spectrum and rotary keys of unit scale."""
    r = case["rank"]
    sp = torch.arange(1, r + 1, device="cuda", dtype=F32) ** -0.3
    sp = sp / sp.square().mean().sqrt()
    c = (torch.randn((n, r), generator=_gen(seed, 1), device="cuda", dtype=F32) * sp).to(BF16)
    return c, _randn((n, case["rope"]), seed, 2)


def _bases(case, seed):
    r, G = case["rank"], case["kv_heads"]
    return (_randn((r, G * case["nope"]), seed, 3, r ** -0.5), _randn((r, G * case["dv"]), seed, 4, r ** -0.5))


def _cu(lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")


def _cache_plan(case):
    """Lengths held per sequence, page table and pool size of a case's cache."""
    L = _lengths(case)
    held = [n + case.get("skip", 0) for n in L]
    pps = max(1, -(-max(held) // PAGE))
    return L, held, pps


def prepare(case, seed):
    op = case["op"]
    st = {"case": case}
    if op == "prefill":
        L = _lengths(case)
        K = [n + case["ahead"] for n in L]
        H, G = case["heads"], case["kv_heads"]
        st.update(L=L, K=K, cu_q=_cu(L), cu_k=_cu(K),
                  q=_randn((sum(L), H, case["nope"] + case["rope"]), seed, 5, 1.5),
                  k=_randn((sum(K), G, case["nope"]), seed, 6), kr=_randn((sum(K), case["rope"]), seed, 7),
                  v=_randn((sum(K), G, case["dv"]), seed, 8))
        if own:
            import rank_kv_cache_lr_b200 as lr
            B_k, B_v = _bases(case, seed)
            st["lr"], st["cache"] = lr, lr.lr_shared_create(_desc(lr, case, 1, 1), B_k, B_v)
            st["out"] = torch.empty((sum(L), H, case["dv"]), dtype=BF16, device="cuda")
            st["lse"] = torch.empty((sum(L), H), dtype=F32, device="cuda")
        return st
    L, held, pps = _cache_plan(case)
    B = case["batch"]
    perm = np.random.default_rng([seed, B, pps]).permutation(B * pps).astype(np.int32).reshape(B, pps)
    seq = torch.tensor(np.repeat(np.arange(B), held), dtype=torch.int32, device="cuda")
    pos = torch.tensor(np.concatenate([np.arange(n) for n in held]), dtype=torch.int32, device="cuda")
    c, kr = _latents(case, sum(held), seed)
    table = torch.tensor(perm, device="cuda")
    st.update(L=L, cu=_cu(L), table=table, pps=pps)
    if op == "write":
        st.update(c=c, kr=kr, seq=seq, pos=pos)
        if own:
            st.update(c_out=torch.empty_like(c), kr_out=torch.empty_like(kr))
    else:
        st["B_k"], st["B_v"] = _bases(case, seed)
        if not own:
            st["pool"] = _store(case, c, kr, seq, pos, table, B * pps)
    if own:
        import rank_kv_cache_lr_b200 as lr
        B_k, B_v = (st["B_k"], st["B_v"]) if op != "write" else _bases(case, seed)
        cache = lr.lr_shared_create(_desc(lr, case, B, pps), B_k, B_v)
        lr.lr_shared_set_block_table(cache, perm)
        st.update(lr=lr, cache=cache)
        if op != "write":
            lr.lr_shared_append(cache, c, kr, seq, pos)
    if op == "decode":
        new, H = case["new"], case["heads"]
        st["q"] = _randn((B, new, H, case["nope"] + case["rope"]), seed, 5, 1.5)
        st["row_len"] = torch.tensor(L, dtype=torch.int32, device="cuda")
        if own:
            st["out"] = torch.empty((B, new, H, case["dv"]), dtype=BF16, device="cuda")
            st["lse"] = torch.empty((B, new, H), dtype=F32, device="cuda")
    if op == "expand":
        st["start"] = torch.full((B,), case["skip"], dtype=torch.int32, device="cuda")
        if own:
            T, G = sum(L), case["kv_heads"]
            st.update(k=torch.empty((T, G, case["nope"]), dtype=BF16, device="cuda"),
                      v=torch.empty((T, G, case["dv"]), dtype=BF16, device="cuda"),
                      kr_out=torch.empty((T, case["rope"]), dtype=BF16, device="cuda"))
    return st


def _desc(lr, case, batch, pps):
    return lr.make_shared_desc(batch=batch, n_q_heads=case["heads"], n_kv_heads=case["kv_heads"],
                               dim_nope=case["nope"], dim_rope=case["rope"], dim_v=case["dv"], rank=case["rank"],
                               capacity=pps * PAGE, quant_bits=case["bits"], max_queries=case.get("new", 1),
                               rope_theta=case.get("theta", 0.0))


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _pow2(e):
    """2^e exactly (float32), from the exponent's bits; pow() is not exact on every device."""
    return ((e.to(torch.int32) + 127) << 23).view(F32)


def _quantise(c):
    """Values (float32) that the 8-bit form of c [n][r] stands for."""
    x = c.to(F32).reshape(c.shape[0], -1, 32)
    mant, ex = torch.frexp(x.abs().amax(-1, keepdim=True))          # max = mant 2^ex, mant in [0.5, 1)
    e = torch.where(mant > 0.875, ex - 8, ex - 9)
    e = torch.where(mant == 0, torch.zeros_like(e), e).clamp(min=-100)
    codes = (x * _pow2(-e)).to(torch.float8_e4m3fn)
    return (codes.to(F32) * _pow2(e)).reshape(c.shape)


def _rotate(kr, pos, theta):
    if not theta:
        return kr
    half = kr.shape[-1] // 2
    om = theta ** (-2.0 * torch.arange(half, device=kr.device, dtype=F64) / kr.shape[-1])
    ang = pos.to(F64)[:, None] * om
    cs, sn = ang.cos().to(F32), ang.sin().to(F32)
    a, b = kr[:, :half].to(F32), kr[:, half:].to(F32)
    return torch.cat([a * cs - b * sn, a * sn + b * cs], 1).to(BF16)


def _store(case, c, kr, seq, pos, table, n_pages):
    """A pool of pages [n_pages][128][r | rope], in what each element stands for."""
    if case["bits"] == 8:
        c = _quantise(c).to(BF16)
    pool = torch.zeros((n_pages * PAGE, c.shape[1] + kr.shape[1]), dtype=BF16, device="cuda")
    rows = table[seq.long(), (pos // PAGE).long()].long() * PAGE + (pos % PAGE).long()
    pool[rows] = torch.cat([c, _rotate(kr, pos, case.get("theta", 0.0))], 1)
    return pool


def _rows(st, b, first, n):
    t = torch.arange(first, first + n, device="cuda")
    return st["table"][b, t // PAGE].long() * PAGE + t % PAGE


def _softmax_lse(s):
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    return p / l.clamp(min=1e-30), (m + l.log()).squeeze(-1)


def _plain_write(st):
    case = st["case"]
    pool = _store(case, st["c"], st["kr"], st["seq"], st["pos"], st["table"], st["table"].numel())
    rows = st["table"][st["seq"].long(), (st["pos"] // PAGE).long()].long() * PAGE + (st["pos"] % PAGE).long()
    out = pool[rows]
    return {"c": out[:, :case["rank"]].contiguous(), "kr": out[:, case["rank"]:].contiguous()}


def _plain_decode(st):
    case = st["case"]
    H, G, dn, dv, r, new = (case[k] for k in ("heads", "kv_heads", "nope", "dv", "rank", "new"))
    B_k = st["B_k"].to(F32).reshape(r, G, dn)
    B_v = st["B_v"].to(F32).reshape(r, G, dv)
    scale = (dn + case["rope"]) ** -0.5
    q = st["q"].to(F32)
    out, lse = [], []
    for b, n in enumerate(st["L"]):
        z = st["pool"][_rows(st, b, 0, n)].to(F32)                          # [n][r + rope]
        qn = torch.einsum("sgjd,rgd->sgjr", q[b, :, :, :dn].reshape(new, G, H // G, dn), B_k).reshape(new, H, r)
        qa = torch.cat([qn, q[b, :, :, dn:]], -1)
        s = torch.matmul(qa, z.T) * scale                                   # [new][H][n]
        last = n - new + torch.arange(new, device="cuda")[:, None, None]
        s = s.masked_fill(torch.arange(n, device="cuda") > last, float("-inf"))
        p, l = _softmax_lse(s)
        o = torch.matmul(p, z[:, :r])
        out.append(torch.einsum("sgjr,rgd->sgjd", o.reshape(new, G, H // G, r), B_v).reshape(new, H, dv))
        lse.append(l)
    return {"out": torch.stack(out).to(BF16), "lse": torch.stack(lse)}


def _plain_expand(st):
    case = st["case"]
    G, r = case["kv_heads"], case["rank"]
    z = torch.cat([st["pool"][_rows(st, b, case["skip"], n)] for b, n in enumerate(st["L"])])
    c = z[:, :r].to(F32)
    return {"k": (c @ st["B_k"].to(F32)).to(BF16).reshape(-1, G, case["nope"]),
            "v": (c @ st["B_v"].to(F32)).to(BF16).reshape(-1, G, case["dv"]), "kr": z[:, r:].contiguous()}


def _plain_prefill(st):
    case = st["case"]
    H, G, dn = case["heads"], case["kv_heads"], case["nope"]
    scale = (dn + case["rope"]) ** -0.5
    T = st["q"].shape[0]
    out = torch.empty((T, H, case["dv"]), dtype=BF16, device="cuda")
    lse = torch.empty((T, H), dtype=F32, device="cuda")
    q0 = k0 = 0
    for n, m in zip(st["L"], st["K"]):
        kr = st["kr"][k0:k0 + m].to(F32)
        hidden = torch.arange(m, device="cuda") > torch.arange(n, device="cuda")[:, None] + (m - n)
        for h in range(H):
            g = h // (H // G)
            k = torch.cat([st["k"][k0:k0 + m, g].to(F32), kr], 1)
            s = st["q"][q0:q0 + n, h].to(F32) @ k.T * scale
            if case["causal"]:
                s = s.masked_fill(hidden, float("-inf"))
            p, l = _softmax_lse(s)
            out[q0:q0 + n, h] = (p @ st["v"][k0:k0 + m, g].to(F32)).to(BF16)
            lse[q0:q0 + n, h] = l
        q0 += n
        k0 += m
    return {"out": out, "lse": lse}


def run(st):
    op = st["case"]["op"]
    if not own:
        return {"write": _plain_write, "decode": _plain_decode, "expand": _plain_expand,
                "prefill": _plain_prefill}[op](st)
    lr, cache = st["lr"], st["cache"]
    if op == "write":
        lr.lr_shared_append(cache, st["c"], st["kr"], st["seq"], st["pos"])
        lr.lr_shared_read(cache, st["cu"], st["c_out"], st["kr_out"])
        return {"c": st["c_out"], "kr": st["kr_out"]}
    if op == "decode":
        lr.lr_shared_decode(cache, st["q"], st["row_len"], st["out"], st["lse"])
        return {"out": st["out"], "lse": st["lse"]}
    if op == "expand":
        lr.lr_shared_expand(cache, st["cu"], st["k"], st["v"], st["kr_out"], start=st["start"])
        return {"k": st["k"], "v": st["v"], "kr": st["kr_out"]}
    lr.lr_shared_attn(cache, st["q"], st["k"], st["kr"], st["v"], st["cu_q"], st["cu_k"], st["out"], st["lse"],
                      causal=st["case"]["causal"])
    return {"out": st["out"], "lse": st["lse"]}


# ---------------------------------------------------------------------------
# exact values: the definitions in 64 bits, with full keys and values
# ---------------------------------------------------------------------------

def _exact_e4m3(c):
    """c [n][r] in float64 -> what its 8-bit form stands for, by search among the e4m3 values."""
    vals = torch.tensor([(m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
                         for e in range(16) for m in range(8)][:127], dtype=F64, device=c.device)
    out = torch.empty_like(c)
    for g in range(0, c.shape[1], 32):
        x = c[:, g:g + 32]
        top = x.abs().max(1, keepdim=True).values
        e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -140) / 448.0)).to(torch.int64)
        two = lambda k: ((k + 1023) << 52).view(F64)                        # noqa: E731  2^k, exactly
        e = torch.where(top > 448.0 * two(e), e + 1, e)
        e = torch.where(top <= 448.0 * two(e - 1), e - 1, e)
        e = torch.where(top == 0, torch.zeros_like(e), e.clamp(min=-100))
        y = (x.abs() / two(e)).contiguous()
        hi = torch.searchsorted(vals, y).clamp(max=126)
        lo = (hi - 1).clamp(min=0)
        dh, dl = vals[hi] - y, y - vals[lo]
        pick = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
        out[:, g:g + 32] = torch.sign(x) * vals[pick] * two(e)
    return out


def exact(case, seed):
    op = case["op"]
    if op == "prefill":
        return _exact_prefill(case, seed)
    L, held, _ = _cache_plan(case)
    c, kr = _latents(case, sum(held), seed)
    z = torch.empty(c.shape, dtype=F64, device="cuda")
    for i in range(0, len(c), 65536):
        z[i:i + 65536] = c[i:i + 65536].to(F64)
        if case["bits"] == 8:
            z[i:i + 65536] = _exact_e4m3(z[i:i + 65536])
    kr = kr.to(F64)
    dr = case["rope"]
    if op == "write":
        pos = torch.cat([torch.arange(n, device="cuda", dtype=F64) for n in held])
        j = torch.arange(dr // 2, device="cuda", dtype=F64)
        ang = pos[:, None] * torch.exp(-2.0 * j / dr * math.log(case["theta"]))
        w = torch.complex(kr[:, :dr // 2], kr[:, dr // 2:]) * torch.polar(torch.ones_like(ang), ang)
        return {"c": z, "kr": torch.cat([w.real, w.imag], 1)}
    B_k, B_v = (x.to(F64) for x in _bases(case, seed))
    G, H, dn, dv = case["kv_heads"], case["heads"], case["nope"], case["dv"]
    if op == "expand":
        keep = torch.cat([torch.arange(n, device="cuda") >= case["skip"] for n in held])
        z, kr = z[keep], kr[keep]
        return {"k": torch.mm(z, B_k).reshape(-1, G, dn), "v": torch.mm(z, B_v).reshape(-1, G, dv), "kr": kr}
    q = _randn((case["batch"], case["new"], H, dn + dr), seed, 5, 1.5).to(F64)
    out = torch.zeros((case["batch"], case["new"], H, dv), dtype=F64, device="cuda")
    lse = torch.full((case["batch"], case["new"], H), float("-inf"), dtype=F64, device="cuda")
    a = 0
    for b, n in enumerate(L):
        for g in range(G):
            key = torch.cat([z[a:a + n] @ B_k[:, g * dn:(g + 1) * dn], kr[a:a + n]], 1)
            val = z[a:a + n] @ B_v[:, g * dv:(g + 1) * dv]
            hs = slice(g * (H // G), (g + 1) * (H // G))
            for s in range(case["new"]):
                m = n - case["new"] + 1 + s
                if m <= 0:
                    continue
                logit = q[b, s, hs] @ key[:m].T / math.sqrt(dn + dr)
                lse[b, s, hs] = torch.logsumexp(logit, 1)
                out[b, s, hs] = torch.exp(logit - lse[b, s, hs][:, None]) @ val[:m]
        a += n
    return {"out": out, "lse": lse}


def _exact_prefill(case, seed):
    L = _lengths(case)
    K = [n + case["ahead"] for n in L]
    H, G, dn, dr, dv = (case[k] for k in ("heads", "kv_heads", "nope", "rope", "dv"))
    q = _randn((sum(L), H, dn + dr), seed, 5, 1.5)
    k, kr = _randn((sum(K), G, dn), seed, 6), _randn((sum(K), dr), seed, 7)
    v = _randn((sum(K), G, dv), seed, 8)
    out = torch.empty((sum(L), H, dv), dtype=F64, device="cuda")
    lse = torch.empty((sum(L), H), dtype=F64, device="cuda")
    q0 = k0 = 0
    for n, m in zip(L, K):
        for h in range(H):
            g = h * G // H
            key, val = torch.cat([k[k0:k0 + m, g], kr[k0:k0 + m]], 1).to(F64), v[k0:k0 + m, g].to(F64)
            for i in range(0, n, 2048):                                     # rows in blocks
                e = min(n, i + 2048)
                seen = m - n + e if case["causal"] else m
                logit = q[q0 + i:q0 + e, h].to(F64) @ key[:seen].T / math.sqrt(dn + dr)
                if case["causal"]:
                    logit += torch.full((e - i, seen), float("-inf"), dtype=F64, device="cuda").triu(m - n + i + 1)
                lse[q0 + i:q0 + e, h] = torch.logsumexp(logit, 1)
                out[q0 + i:q0 + e, h] = torch.exp(logit - lse[q0 + i:q0 + e, h][:, None]) @ val[:seen]
        q0 += n
        k0 += m
    return {"out": out, "lse": lse}
