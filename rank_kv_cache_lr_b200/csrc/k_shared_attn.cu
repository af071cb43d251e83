// Ragged attention over expanded keys and values (the form of shared-latent attention for
// prompts): head j's key is [k_h | kr] with kr shared by the heads, its value v_h.
//
//   S = Q [K | Kr]^T       M = 128 queries, N = 128 keys, K = dn + dr (rounded up to 64)
//   P = 2^(S c - m)        online softmax, lazy running max; c = scale log2 e
//   O += P V               M = 128 queries, N = dv, K = 128 keys; P (bf16) as A operand in TMEM
//
// A CTA holds two 128-query tiles of one head, so the tensor pipe works on one tile while the
// other is in its softmax: S0 S1 | PV0 S0' PV1 S1' | ...  Each tile has its own warpgroup
// (thread = query row = TMEM lane: row maxima and sums need no shuffles).  P overlays S in
// TMEM; the MMAs of one CTA run in issue order, so S' of a tile is written after its PV has
// read P.  Keys and values stream through one ring of 16 KB boxes (64 columns x 128 rows).
//
// Bound: the tensor pipe, 2 x 128 x 128 (dn + dr + dv) MACs per tile pair and key tile
// (2560 clocks at 192 + 128) against 2048 clocks of exponentials on the same SM.
//
// Roundings: P to bf16 (half a step, 2^-8 relative, at random over the keys, below the output's
// own); sums of the unrounded weights in fp32; the output once.  A running max may be stale by
// 2^8 before it is raised (fp32 sums hold that easily), which saves most rescales of O.
#include "shared_internal.cuh"
#include "tc_common.cuh"

#include <algorithm>

namespace {

using tc::drain_wait;
using tc::kLazy;

constexpr int kBox = 128 * 128;        // 128 rows x 64 columns x 2 B
constexpr int kRing = 8;
constexpr int kThreads = 320;
constexpr int kAuxBytes = 1024;
constexpr float kNoMax = -1e30f;

struct AttArgs {
  unsigned long long wait_ns;
  const int32_t* cu_q; const int32_t* cu_k;
  int nseq, total_q, total_k, Hq, g, dn, dv, dq, causal, slots;   // slots: tile pairs in the grid
  float scale_log2;
  __nv_bfloat16* out;
  float* lse;
  int* err;
};

// Barriers (arrival count; who arrives -> who waits):
//   q_full          1 + tx   producer -> MMA
//   full/empty[s]   1 + tx / 1   boxes of K, Kr, V in the order of use
//   s_full[t]       1        MMA commit of S of tile t -> its softmax warps
//   p_full[t]       4        softmax warps (P stored) -> MMA
//   pv_done[t]      1        MMA commit of PV -> softmax warps (O rescale, epilogue)
struct Aux {
  uint64_t q_full, full[kRing], empty[kRing], s_full[2], p_full[2], pv_done[2], done;
  uint32_t tmem_base;
  int abort_flag;
  int b, pair;
  unsigned long long wait_ns;
};
static_assert(sizeof(Aux) <= kAuxBytes, "aux block");

__device__ __forceinline__ bool wait_b(uint64_t* bar, uint32_t parity, Aux* aux, int* err) {
  return tc::wait_b(bar, parity, &aux->abort_flag, err, aux->wait_ns);
}
__device__ __forceinline__ bool wait_w(uint64_t* bar, uint32_t parity, Aux* aux, int* err) {
  return __all_sync(0xffffffffu, wait_b(bar, parity, aux, err));
}

// Rows of sequence b in a packed array of `total` rows.
struct Rows {
  int first, n;
};
__device__ __forceinline__ Rows rows_of(const int32_t* cu, int b, int total) {
  const int a = min(max(__ldg(cu + b), 0), total), e = min(max(__ldg(cu + b + 1), a), total);
  return Rows{a, e - a};
}

__global__ void __launch_bounds__(kThreads, 1)
    k_shared_attn(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_kr, const __grid_constant__ CUtensorMap tm_v,
                  const AttArgs p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (ptx::smem_u32(smem_raw) & 1023) {
    if (threadIdx.x == 0) atomicExch(p.err, (int)LR_ERR_UNSUPPORTED);
    return;
  }
  Aux* aux = reinterpret_cast<Aux*>(smem_raw);
  uint8_t* q_s = smem_raw + kAuxBytes;                 // 2 tiles x nqb boxes
  const int nqb = (p.dq + 63) >> 6;                    // 64-column boxes of a query row
  const int nkb = (p.dn >> 6) + 1, nvb = p.dv >> 6;    // boxes of a key tile (rotary last), of a value tile
  uint8_t* ring = q_s + 2 * nqb * kBox;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int head = blockIdx.x % p.Hq, kvh = head / p.g;

  pdl_wait();
  pdl_trigger();
  if (warp == 9) {
    // the longest tile pairs (causal: the last ones) start first
    auto pairs = [&](int b) { return (rows_of(p.cu_q, b, p.total_q).n + 255) >> 8; };
    const int want = p.slots - 1 - (int)(blockIdx.x / p.Hq);
    int b = p.nseq, pair = 0;
    if (want < tile_total(pairs, p.nseq)) tile_find(pairs, p.nseq, want, &b, &pair);
    if (lane == 0) {
      aux->b = b;
      aux->pair = pair;
    }
  }
  if (threadIdx.x == 0) {
    ptx::mbar_init(&aux->q_full, 1);
    for (int s = 0; s < kRing; ++s) {
      ptx::mbar_init(&aux->full[s], 1);
      ptx::mbar_init(&aux->empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      ptx::mbar_init(&aux->s_full[t], 1);
      ptx::mbar_init(&aux->p_full[t], 4);
      ptx::mbar_init(&aux->pv_done[t], 1);
    }
    ptx::mbar_init(&aux->done, 1);
    aux->abort_flag = 0;
    aux->wait_ns = tc::wait_limit(p.wait_ns);
    ptx::fence_mbar_init();
  }
  if (warp == 8) {
    ptx::tmem_alloc(&aux->tmem_base, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = aux->tmem_base;
  const int b = aux->b;
  const bool any = b < p.nseq;
  const Rows rq = any ? rows_of(p.cu_q, b, p.total_q) : Rows{0, 0};
  const Rows rk = any ? rows_of(p.cu_k, b, p.total_k) : Rows{0, 0};
  const int q0 = aux->pair * 256;
  // key tiles of each query tile: up to the last key its last query sees
  int nt[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int lo = q0 + t * 128, hi = min(rq.n, lo + 128) - 1;
    const int last = p.causal ? min(rk.n - 1, hi + rk.n - rq.n) : rk.n - 1;
    nt[t] = lo < rq.n && last >= 0 ? (last >> 7) + 1 : 0;
  }
  const int ntk = max(nt[0], nt[1]);

  if (warp == 9) {
    // ------------------------------------------------------------- TMA producer
    if (lane == 0 && ntk > 0) {
      const int tiles = rq.n - q0 > 128 ? 2 : 1;
      ptx::mbar_arrive_expect_tx(&aux->q_full, (uint32_t)(tiles * nqb * kBox));
      for (int t = 0; t < tiles; ++t)
        for (int c = 0; c < nqb; ++c)
          ptx::tma_load_3d(q_s + (t * nqb + c) * kBox, &tm_q, &aux->q_full, c * 64, head, rq.first + q0 + t * 128);
      int pos = 0;
      bool ok = true;
      for (int j = 0; j < ntk && ok; ++j) {
        const int row = rk.first + j * 128;
        for (int c = 0; c < nkb + nvb; ++c) {
          const int s = pos % kRing;
          if (pos >= kRing && !(ok = wait_b(&aux->empty[s], (pos / kRing - 1) & 1, aux, p.err))) break;
          ptx::mbar_arrive_expect_tx(&aux->full[s], kBox);
          uint8_t* dst = ring + s * kBox;
          if (c < nkb - 1) ptx::tma_load_3d(dst, &tm_k, &aux->full[s], c * 64, kvh, row);
          else if (c == nkb - 1) ptx::tma_load_2d(dst, &tm_kr, &aux->full[s], 0, row);
          else ptx::tma_load_3d(dst, &tm_v, &aux->full[s], (c - nkb) * 64, kvh, row);
          ++pos;
        }
      }
      // every copy this thread issued has landed before the CTA can exit
      drain_wait(&aux->q_full, 0);
      for (int k = max(0, pos - kRing); k < pos; ++k) drain_wait(&aux->full[k % kRing], (k / kRing) & 1);
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------- MMA issuer (warp-wide)
    if (ntk > 0) {
      const uint32_t ids = ptx::idesc_f16(1, 0, 0, 128, 128);                  // S: K-major x K-major
      const uint32_t idv = ptx::idesc_f16(1, 0, 1, 128, (uint32_t)p.dv);       // PV: TMEM x MN-major
      const uint64_t qd0 = ptx::smem_desc(ptx::smem_u32(q_s), 16, 1024, 2);
      const uint64_t kd0 = ptx::smem_desc(ptx::smem_u32(ring), 16, 1024, 2);
      const uint64_t vd0 = ptx::smem_desc(ptx::smem_u32(ring), kBox, 1024, 2);
      const int per = nkb + nvb;
      auto scores = [&](int t, int j, bool wait) -> bool {
        for (int c = 0; c < nkb; ++c) {
          const int pos = j * per + c, s = pos % kRing;
          if (wait && !wait_w(&aux->full[s], (pos / kRing) & 1, aux, p.err)) return false;
          ptx::tc_fence_after();
          // the query boxes: dn, then the rotary columns (dn and dn + 64 are box borders)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            ptx::mma_f16_elect(tmem + t * 128, qd0 + (uint64_t)(((t * nqb + c) * kBox >> 4) + kk * 2),
                               kd0 + (uint64_t)((s * kBox >> 4) + kk * 2), ids, (c | kk) ? 1u : 0u);
        }
        ptx::mma_commit_elect(&aux->s_full[t]);
        return true;
      };
      auto values = [&](int t, int j, bool wait) -> bool {
        if (!wait_w(&aux->p_full[t], j & 1, aux, p.err)) return false;
        const int pos0 = j * per + nkb;
        if (wait)
          for (int c = 0; c < nvb; ++c)
            if (!wait_w(&aux->full[(pos0 + c) % kRing], ((pos0 + c) / kRing) & 1, aux, p.err)) return false;
        ptx::tc_fence_after();
        // a box at a time along N: the boxes of a tile need not be neighbours in the ring
        const uint32_t idh = ptx::idesc_f16(1, 0, 1, 128, 64);
        const int s0 = pos0 % kRing;
        if (nvb == 2 && s0 + 1 < kRing) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            ptx::mma_f16_ta_elect(tmem + 256 + t * 128, tmem + t * 128 + kk * 8,
                                  vd0 + (uint64_t)((s0 * kBox + kk * 2048) >> 4), idv, (j | kk) ? 1u : 0u);
        } else {
          for (int c = 0; c < nvb; ++c) {
            const int s = (pos0 + c) % kRing;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              ptx::mma_f16_ta_elect(tmem + 256 + t * 128 + c * 64, tmem + t * 128 + kk * 8,
                                    vd0 + (uint64_t)((s * kBox + kk * 2048) >> 4), idh, (j | kk) ? 1u : 0u);
          }
        }
        ptx::mma_commit_elect(&aux->pv_done[t]);
        return true;
      };
      auto release = [&](int pos, int n) {
        for (int c = 0; c < n; ++c) ptx::mma_commit_elect(&aux->empty[(pos + c) % kRing]);
      };
      bool ok = wait_w(&aux->q_full, 0, aux, p.err);
      if (ok && nt[0] > 0) ok = scores(0, 0, true);
      if (ok && nt[1] > 0) ok = scores(1, 0, nt[0] == 0);
      if (ok) release(0, nkb);
      for (int j = 0; j < ntk && ok; ++j) {
        const bool first_v = j < nt[0], first_k = j + 1 < nt[0];
        if (ok && first_v) ok = values(0, j, true);
        if (ok && first_k) ok = scores(0, j + 1, true);
        if (ok && j < nt[1]) ok = values(1, j, !first_v);
        if (ok) release(j * per + nkb, nvb);
        if (ok && j + 1 < nt[1]) ok = scores(1, j + 1, !first_k);
        if (ok && j + 1 < ntk) release((j + 1) * per, nkb);
      }
      ptx::mma_commit_elect(&aux->done);
      drain_wait(&aux->done, 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------- softmax and epilogue, tile t
    const int t = warp >> 2, qd = warp & 3;
    const int row = qd * 32 + lane, i = q0 + t * 128 + row;
    const uint32_t s_col = tmem + ((uint32_t)(qd * 32) << 16) + t * 128, o_col = s_col + 256;
    const int last = p.causal ? min(rk.n - 1, i + rk.n - rq.n) : rk.n - 1;   // last key this query sees
    const int wlast = __shfl_sync(0xffffffffu, last, 0);                     // the warp's smallest
    float m = kNoMax, l = 0.f;
    bool ok = true;
    for (int j = 0; j < nt[t]; ++j) {
      if (!(ok = wait_w(&aux->s_full[t], j & 1, aux, p.err))) break;
      ptx::tc_fence_after();
      const int lim = last - j * 128;              // columns 0..lim are visible
      const bool edge = wlast - j * 128 < 127;     // some row of the warp masks columns here
      float mx = -INFINITY;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t v[32];
        ptx::tmem_ld32(s_col + 32 * c, v);
        ptx::tmem_wait_ld();
        if (edge) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (32 * c + e <= lim) mx = fmaxf(mx, __uint_as_float(v[e]));
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) mx = fmaxf(mx, __uint_as_float(v[e]));
        }
      }
      mx *= p.scale_log2;
      if (__any_sync(0xffffffffu, mx > m + kLazy)) {
        const float mn = fmaxf(m, mx), a = ptx::ex2_approx(m - mn);
        m = mn;
        l *= a;
        if (j > 0) {
          if (!(ok = wait_w(&aux->pv_done[t], (j - 1) & 1, aux, p.err))) break;
          ptx::tc_fence_after();
          for (int c = 0; c < p.dv; c += 32) {
            uint32_t v[32];
            ptx::tmem_ld32(o_col + c, v);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * a);
            ptx::tmem_st32(o_col + c, v);
          }
        }
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t v[32], w[16];
        ptx::tmem_ld32(s_col + 32 * c, v);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float p0 = ptx::ex2_approx(fmaf(__uint_as_float(v[2 * e]), p.scale_log2, -m));
          float p1 = ptx::ex2_approx(fmaf(__uint_as_float(v[2 * e + 1]), p.scale_log2, -m));
          if (edge) {
            if (32 * c + 2 * e > lim) p0 = 0.f;
            if (32 * c + 2 * e + 1 > lim) p1 = 0.f;
          }
          l += p0;
          l += p1;
          const __nv_bfloat162 h = __floats2bfloat162_rn(p0, p1);
          w[e] = *reinterpret_cast<const uint32_t*>(&h);
        }
        ptx::tmem_st16(s_col + 16 * c, w);
      }
      if (j * 128 + 128 > rk.n) {
        // the rows behind the last key belong to the next sequence: weight 0, but 0 times an
        // infinity there would be NaN, so their values become 0 (each tile clears them before it
        // hands over its weights; both store the same)
        const int pos0 = j * (nkb + nvb) + nkb;
        for (int c = 0; c < nvb; ++c)
          if (!(ok = wait_w(&aux->full[(pos0 + c) % kRing], ((pos0 + c) / kRing) & 1, aux, p.err))) break;
        if (!ok) break;
        if (j * 128 + row >= rk.n)
          for (int c = 0; c < nvb; ++c) {
            const uint32_t base = ptx::smem_u32(ring + ((pos0 + c) % kRing) * kBox + row * 128);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(base + e * 16), "r"(0) : "memory");
          }
        ptx::fence_proxy_async_smem();
        __syncwarp();
      }
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&aux->p_full[t]);
    }
    if (ok && nt[t] > 0) ok = wait_w(&aux->pv_done[t], (nt[t] - 1) & 1, aux, p.err);
    ptx::tc_fence_after();
    if (ok) {
      const size_t o = ((size_t)rq.first + i) * p.Hq + head;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      if (i < rq.n && p.lse) p.lse[o] = l == 0.f ? -INFINITY : (m + log2f(l)) * LR_LN2;
      __syncwarp();
      for (int c = 0; c < p.dv; c += 32) {
        uint32_t v[32];
        if (nt[t] > 0) {
          ptx::tmem_ld32(o_col + c, v);
          ptx::tmem_wait_ld();
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            // a row that saw no key has weight sum 0: its output is 0
            const float x0 = l == 0.f ? 0.f : __uint_as_float(v[16 * h + 2 * e]) * inv;
            const float x1 = l == 0.f ? 0.f : __uint_as_float(v[16 * h + 2 * e + 1]) * inv;
            const __nv_bfloat162 b2 = __floats2bfloat162_rn(x0, x1);
            w[e] = *reinterpret_cast<const uint32_t*>(&b2);
          }
          if (i < rq.n) ptx::st_global_v8(p.out + o * p.dv + c + 16 * h, w);
        }
        __syncwarp();                  // the next TMEM load wants the whole warp
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

bool map3d(CUtensorMap* m, const void* ptr, uint64_t d0, uint64_t d1, uint64_t d2) {
  const cuuint64_t dims[3] = {d0, d1, d2}, st[2] = {d0 * 2, d0 * d1 * 2};
  const cuuint32_t box[3] = {64, 1, 128};
  return tc::make_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, ptr, 3, dims, st, box);
}

}  // namespace

cudaError_t launch_shared_attn(lr_shared* c, const void* q, const void* k, const void* kr, const void* v,
                               const int32_t* cu_q, const int32_t* cu_k, int nseq, int total_q, int total_k,
                               int causal, void* out, float* lse, cudaStream_t s) {
  const lr_shared_desc& d = c->desc;
  AttArgs a;
  a.wait_ns = c->wait_ns;
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.nseq = nseq;
  a.total_q = total_q;
  a.total_k = total_k;
  a.Hq = d.n_q_heads;
  a.g = d.n_q_heads / d.n_kv_heads;
  a.dn = d.dim_nope;
  a.dv = d.dim_v;
  a.dq = d.dim_nope + d.dim_rope;
  a.causal = causal;
  a.scale_log2 = c->scale_log2;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.err = c->dev_err;
  const long long slots = (long long)total_q / 256 + std::min(nseq, total_q);
  if (slots * a.Hq > 0x7FFFFFFF) return cudaErrorNotSupported;
  a.slots = (int)slots;
  CUtensorMap tq, tk, tkr, tv;
  if (total_k == 0) k = kr = v = q;      // no key tile is ever loaded; the maps need an address
  const cuuint64_t rows = std::max(total_k, 1);
  if (!map3d(&tq, q, a.dq, a.Hq, total_q) || !map3d(&tk, k, a.dn, d.n_kv_heads, rows) ||
      !map3d(&tv, v, a.dv, d.n_kv_heads, rows))
    return cudaErrorInvalidValue;
  {
    const cuuint64_t dims[2] = {(cuuint64_t)d.dim_rope, rows}, st[1] = {(cuuint64_t)d.dim_rope * 2};
    const cuuint32_t box[2] = {64, 128};
    if (!tc::make_map(&tkr, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, kr, 2, dims, st, box)) return cudaErrorInvalidValue;
  }
  const size_t smem = kAuxBytes + (size_t)(2 * ((a.dq + 63) / 64) + kRing) * kBox;
  static std::atomic<uint32_t> optin{0};
  cudaError_t e = smem_optin(k_shared_attn, optin);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_shared_attn, dim3((unsigned)(slots * a.Hq)), dim3(kThreads), smem, s, tq, tk, tkr, tv, a);
}
