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
// read P.  Keys and values pass through one ring of 16 KB slots
// (what the query tiles leave of shared memory; 8 slots against 5 a tile at 192 + 128), so a
// tile's values load as soon as the scores of the tile before are done.
//
// Few CTAs over many keys (a few heads or short chunks): up to 8 CTAs, a cluster, take equal parts of
// the key tiles of one query tile pair and join (m, l, O) through distributed shared memory.
//
// Bound: the tensor pipe, 2 x 128 x 128 (dn + dr + dv) MACs per tile pair and key tile
// (2560 clocks at 192 + 128) against 2048 clocks of exponentials on the same SM.  Measured: ~4300
// clocks (per query tile: 1200 from the first MMA of S to its softmax, 1700 of softmax, 300 to
// the last MMA of PV, and the keys of the next tile, which wait on values of the last).  Two
// sequences of 8192 tokens, 28 heads, causal: 1.02 ms, 1.18 PFLOP/s in a short burst, 1.19 ms run
// continuously, at the card's power limit (1000 W).  In bursts, with two fixed stages for
// keys and one for values 1.22 ms; with a barrier per 64-column box of keys 1.24 ms (a test between
// MMAs costs more than the earlier start gains).
//
// Roundings: P to bf16 (half a step, 2^-8 relative at most: at random over the keys, but alike for equal
// weights that are no powers of two, and then 2^-8 of the output before its own rounding); sums of the
// unrounded weights in fp32 (a second sum, of the rounded ones, would take three more instructions
// for every two weights); the output once.  A running max may be stale by
// 2^8 before it is raised (fp32 sums hold that easily), which saves most rescales of O.
#include "shared_internal.cuh"
#include "tc_common.cuh"

#include <algorithm>
#include <cmath>

namespace {

using tc::drain_wait;
using tc::kLazy;

constexpr int kBox = 128 * 128;        // 128 rows x 64 columns x 2 B
constexpr int kVBox = kBox / 2;        // 64 rows x 64 columns x 2 B
// Three warpgroups: 0 and 1 softmax of tiles 0 and 1, 2 MMA issuers (warps 8 and 10), TMA producer
// (warp 9) and an idle warp.  Launched at 168 registers, rebalanced so that a softmax thread holds its
// row of 128 scores (read from TMEM once).
constexpr int kThreads = 384;
constexpr int kLaunchRegs = 168, kSoftmaxRegs = 200, kCtlRegs = 104;
static_assert(256 * kSoftmaxRegs + 128 * kCtlRegs <= kThreads * kLaunchRegs, "register split exceeds the launch");
constexpr int kAuxBytes = 1024;
constexpr float kNoMax = -3.402823466e38f;   // running max before any visible key: finite, and below every score
constexpr int kMaxSplit = 8;
constexpr int kPartMl = 256 * 8;       // (m, l) of a part's rows, then their sums (rows padded by 16 bytes)

struct AttArgs {
  unsigned long long wait_ns;
  const int32_t* cu_q; const int32_t* cu_k;
  int nseq, total_q, total_k, Hq, g, dn, dv, dq, causal, stagger, slots, ring, split;   // slots: tile pairs a head; ring: 16 KB slots for keys and values;
                                                                                // split: CTAs a tile pair
  float scale_log2, scale_pow2;   // softmax scale times log2 e, and the largest power of two that is no larger
  __nv_bfloat16* out;
  float* lse;
  int* err;
};

// Barriers (arrival count; who arrives -> who waits).  [2]: by the parity of the key tile, so that a
// waiter may be one key tile behind the arriver.
//   q_full[t]         1 + tx   producer -> MMA
//   k_full, v_full[2] 1 + tx   producer -> MMA (values also -> softmax, which clears what lies behind the last key)
//   s_full[t][2]      1        MMA commit of S of tile t -> its softmax warps, producer (the keys' slots)
//   p_full[t][h][2]   4        softmax warps (P of keys 64 h .. 64 h + 63 stored) -> MMA
//   pv_done[t][h][2]  1        MMA commit of PV of key half h -> producer (the values' slots), epilogue
//   done              2        final commits of both MMA warps
struct Aux {
  uint64_t q_full[2], k_full[2], v_full[2], s_full[2][2], p_full[2][2][2], pv_done[2][2][2], done;
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

// A warp-uniform value, known as such to the compiler: MMA operands then stay in uniform registers
// (an MMA issues at the tensor core's pace; without, every ~160 cycles).
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

// Rows of sequence b in a packed array of `total` rows.
struct Rows {
  int first, n;
};
__device__ __forceinline__ Rows rows_of(const int32_t* cu, int b, int total) {
  const int a = min(max(__ldg(cu + b), 0), total), e = min(max(__ldg(cu + b + 1), a), total);
  return Rows{a, e - a};
}

template <bool kSplit>
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
  // slots of a key tile (rotary last): 128 keys x 64 columns each; of a value tile: all columns of 64
  // keys (dv = 128) or of 128 keys (dv = 64), so that half h of the keys is one operand
  const int nkb = (p.dn >> 6) + 1, nvb = p.dv >> 6, unit = nkb + nvb;
  [[maybe_unused]] uint8_t* part_s = q_s;              // a part's sums, at its end
  uint8_t* kv_s = q_s + 2 * nqb * kBox;                // the ring: K0 V0 K1 V1 ..., p.ring slots of kBox
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int work = kSplit ? blockIdx.x / p.split : blockIdx.x;           // (a split's CTAs are a cluster)
  const int part = kSplit ? blockIdx.x % p.split : 0;
  const int head = work % p.Hq, kvh = head / p.g;

  pdl_wait();
  if (warp == 9) {
    // the longest tile pairs (causal: the last ones) start first
    auto pairs = [&](int b) { return (rows_of(p.cu_q, b, p.total_q).n + 255) >> 8; };
    const int want = p.slots - 1 - work / p.Hq;
    int b = p.nseq, pair = 0;
    if (want < tile_total(pairs, p.nseq)) tile_find(pairs, p.nseq, want, &b, &pair);
    if (lane == 0) {
      aux->b = b;
      aux->pair = pair;
    }
  }
  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) ptx::mbar_init(&aux->q_full[t], 1);
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(&aux->k_full[s], 1);
      ptx::mbar_init(&aux->v_full[s], 1);
      for (int t = 0; t < 2; ++t) {
        ptx::mbar_init(&aux->s_full[t][s], 1);
        ptx::mbar_init(&aux->p_full[t][0][s], 4);
        ptx::mbar_init(&aux->p_full[t][1][s], 4);
        ptx::mbar_init(&aux->pv_done[t][0][s], 1);
        ptx::mbar_init(&aux->pv_done[t][1][s], 1);
      }
    }
    ptx::mbar_init(&aux->done, 2);
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
  pdl_trigger();              // (once TMEM is held, see k_shared_decode)
  const uint32_t tmem = aux->tmem_base;
  const int b = aux->b;
  const bool any = b < p.nseq;
  const Rows rq = any ? rows_of(p.cu_q, b, p.total_q) : Rows{0, 0};
  Rows rk = any ? rows_of(p.cu_k, b, p.total_k) : Rows{0, 0};
  const int q0 = aux->pair * 256;
  // key tiles of each query tile: up to the last key its last query sees
  int nt[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int lo = q0 + t * 128, hi = min(rq.n, lo + 128) - 1;
    const int last = p.causal ? min(rk.n - 1, hi + rk.n - rq.n) : rk.n - 1;
    nt[t] = lo < rq.n && last >= 0 ? (last >> 7) + 1 : 0;
  }
  int shift = rk.n - rq.n;               // causal: query i sees keys up to i + shift (of this part)
  if constexpr (kSplit) {
    const int per = (max(nt[0], nt[1]) + p.split - 1) / p.split, j0 = part * per;
    for (int t = 0; t < 2; ++t) nt[t] = min(max(nt[t] - j0, 0), per);
    rk.first += j0 * 128;
    rk.n -= j0 * 128;
    shift -= j0 * 128;
  }
  const int ntk = max(nt[0], nt[1]);

  if (warp >= 8) {
    ptx::setmaxnreg_dec<kCtlRegs>();
    if (warp == 9) {
      // ------------------------------------------------------------- TMA producer
      if (lane == 0 && ntk > 0) {
        auto queries = [&](int t) {
          ptx::mbar_arrive_expect_tx(&aux->q_full[t], (uint32_t)(nqb * kBox));
          for (int c = 0; c < nqb; ++c)
            ptx::tma_load_3d(q_s + (t * nqb + c) * kBox, &tm_q, &aux->q_full[t], c * 64, head, rq.first + q0 + t * 128);
        };
        // (a tile that sees no key here has no reader, and a part's sums take its place; the second tile's
        // come behind the first keys)
        if (nt[0] > 0) queries(0);
        // Slots are taken and given back in one order, K0 V0 K1 V1 ..., so V_j goes where K_{j-1} was (free
        // early: its scores are done) and K_{j+1} partly where V_{j-1} was, half by half.
        bool ok = true;
        int at = 0, left = p.ring;                     // next slot, free slots
        int fi = 0, fu = 0;                            // next slot to be freed: unit fu of tile fi (keys, then values)
        auto slot = [&]() -> uint8_t* {                // the next slot, once both query tiles are done with what it held
          if (left == 0) {
            const int s = fi & 1, h = fu - nkb + 2 - nvb;
            for (int t = 0; t < 2 && ok; ++t)
              if (fi < nt[t]) ok = wait_b(h >= 0 ? &aux->pv_done[t][h][s] : &aux->s_full[t][s], (fi >> 1) & 1, aux, p.err);
            const int run = fu == 0 ? nkb : 1;         // a key tile is free as a whole
            left = run;
            fu += run;
            if (fu == unit) {
              fu = 0;
              ++fi;
            }
          }
          uint8_t* const dst = kv_s + at * kBox;
          if (++at == p.ring) at = 0;
          --left;
          return dst;
        };
        int nk = 0, nv = 0;                            // key and value tiles begun
        for (int j = 0; j < ntk && ok; ++j) {
          const int row = rk.first + j * 128, s = j & 1;
          for (int c = 0; c < nkb; ++c) {
            uint8_t* dst = slot();
            if (!ok) break;
            if (c == 0) {
              ptx::mbar_arrive_expect_tx(&aux->k_full[s], (uint32_t)(nkb * kBox));
              ++nk;
            }
            if (c < nkb - 1) ptx::tma_load_2d(dst, &tm_k, &aux->k_full[s], kvh * p.dn + c * 64, row);
            else ptx::tma_load_2d(dst, &tm_kr, &aux->k_full[s], 0, row);
          }
          if (j == 0 && nt[1] > 0) queries(1);
          for (int c = 0; c < nvb && ok; ++c) {
            uint8_t* dst = slot();
            if (!ok) break;
            if (c == 0) {
              ptx::mbar_arrive_expect_tx(&aux->v_full[s], (uint32_t)(nvb * kBox));
              ++nv;
            }
            for (int e = 0; e < 2; ++e)                // dv = 128: columns 64 e of key half c; else key half e
              ptx::tma_load_2d(dst + e * kVBox, &tm_v, &aux->v_full[s], kvh * p.dv + (nvb == 2 ? e * 64 : 0),
                               row + (nvb == 2 ? c : e) * 64);
          }
        }
        // every copy this thread issued has landed before the CTA can exit
        if (nt[0] > 0) drain_wait(&aux->q_full[0], 0);
        if (nt[1] > 0) drain_wait(&aux->q_full[1], 0);
        for (int j = max(0, nk - 2); j < nk; ++j) drain_wait(&aux->k_full[j & 1], (j >> 1) & 1);
        for (int j = max(0, nv - 2); j < nv; ++j) drain_wait(&aux->v_full[j & 1], (j >> 1) & 1);
      }
    } else if (warp != 11 && ntk > 0) {
      // ------------------------------------------------------------- MMA issuer of tile t (warp-wide)
      // A warp per tile: an MMA's issue waits for the tensor pipe, so whatever stands between two
      // MMAs of one warp (a barrier test costs ~130 cycles, a commit ~60, serial code ~8 an instruction
      // beside busy softmax warps) leaves the pipe idle unless the other tile's warp issues meanwhile.
      // So what S(j) needs is made ready before PV(j - 1)'s last wait.
      const int t = warp == 10 ? 1 : 0, ntt = nt[t];
      const uint32_t ids = ptx::idesc_f16(1, 0, 0, 128, 128);                  // S: K-major x K-major
      const uint32_t idv = ptx::idesc_f16(1, 0, 1, 128, (uint32_t)p.dv);       // PV: TMEM x MN-major
      const uint64_t qd = ptx::smem_desc(ptx::smem_u32(q_s + t * nqb * kBox), 16, 1024, 2);
      const uint64_t kd = ptx::smem_desc(ptx::smem_u32(kv_s), 16, 1024, 2);
      const uint64_t vd = ptx::smem_desc(ptx::smem_u32(kv_s), kVBox, 1024, 2);
      const uint32_t d_s = uniform(tmem + t * 128);
      int kp = 0;                                      // ring slot of key tile j
      uint64_t vb[2] = {vd, vd};                       // halves of value tile j - 1
      bool ok = ntt == 0 || wait_w(&aux->q_full[t], 0, aux, p.err);
#pragma unroll 1
      for (int j = 0; j <= ntt && ok; ++j) {
        const int s = j & 1, ph = (j >> 1) & 1;
        uint64_t kb[3];
        int vp = kp;
#pragma unroll
        for (int c = 0; c < 3; ++c)
          if (c < nkb) {
            kb[c] = kd + uniform((uint32_t)vp * (kBox >> 4));
            if (++vp == p.ring) vp = 0;
          }
        bool k_in = false;                             // key tile j has landed
        // PV(j - 1), in two halves of 64 keys: the first runs while the softmax works on the second
        if (j > 0) {
          const int si = s ^ 1, phi = ((j - 1) >> 1) & 1;
          const uint32_t more = uniform(j > 1 ? 1u : 0u);
          if (!(ok = wait_w(&aux->v_full[si], phi, aux, p.err))) break;
          if (!(ok = wait_w(&aux->p_full[t][0][si], phi, aux, p.err))) break;
          ptx::tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            ptx::mma_f16_ta_elect(d_s + 256, d_s + kk * 8, vb[0] + (uint64_t)(kk * 128), idv, kk ? 1u : more);
          ptx::mma_commit_elect(&aux->pv_done[t][0][si]);
          if (j < ntt) k_in = __all_sync(0xffffffffu, ptx::mbar_test_wait(&aux->k_full[s], ph));
          if (!(ok = wait_w(&aux->p_full[t][1][si], phi, aux, p.err))) break;
          ptx::tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            ptx::mma_f16_ta_elect(d_s + 256, d_s + 32 + kk * 8, vb[1] + (uint64_t)(kk * 128), idv, 1u);
          ptx::mma_commit_elect(&aux->pv_done[t][1][si]);
        }
        if (j == ntt) break;
        // S(j): the query boxes are dn, then the rotary columns (dn and dn + 64 are box borders).
        // Where all CTAs run at once, over many key tiles, tile 1 starts when tile 0 is half through its
        // softmax: in step, both would want the tensor pipe at one time and the exponentials at another
        // (512 new tokens over 4096: 100 us against 116; over 32768: 637 against 675; 1280 over 16000: 320
        // against 350).  In several waves the tiles drift apart by themselves and the wait costs (prompts of
        // 4096: 158 us with it, 141 without; 16384: 2.2 and 2.1 ms), and so it does over a few key tiles
        // (seven prompts of up to 400 tokens: 28.8 and 26.7 us; the border of four is from these and the above).
        if (!k_in && !(ok = wait_w(&aux->k_full[s], ph, aux, p.err))) break;
        if (t == 1 && p.stagger && ntk > 4 && j < nt[0] && !(ok = wait_w(&aux->p_full[0][0][s], ph, aux, p.err))) break;
        ptx::tc_fence_after();
#pragma unroll
        for (int c = 0; c < 3; ++c)
          if (c < nkb) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              ptx::mma_f16_elect(d_s, qd + (uint64_t)((c * kBox >> 4) + kk * 2), kb[c] + (uint64_t)(kk * 2), ids, c + kk ? 1u : 0u);
          }
        ptx::mma_commit_elect(&aux->s_full[t][s]);
        // value tile j lies behind key tile j
        const int v1 = vp + 1 == p.ring ? 0 : vp + 1;
        vb[0] = vd + uniform((uint32_t)vp * (kBox >> 4));
        vb[1] = nvb == 2 ? vd + uniform((uint32_t)v1 * (kBox >> 4)) : vb[0] + (kVBox >> 4);
        kp += unit;
        if (kp >= p.ring) kp -= p.ring;
      }
      ptx::mma_commit_elect(&aux->done);
      drain_wait(&aux->done, 0);
    }
    __syncwarp();
  } else {
    ptx::setmaxnreg_inc<kSoftmaxRegs>();
    // ------------------------------------------------------------- softmax and epilogue, tile t
    const int t = warp >> 2, qd = warp & 3;
    const int row = qd * 32 + lane, i = q0 + t * 128 + row;
    const uint32_t s_col = tmem + ((uint32_t)(qd * 32) << 16) + t * 128, o_col = s_col + 256;
    const int last = p.causal ? min(rk.n - 1, i + shift) : rk.n - 1;   // last key this query sees
    const int wlast = __shfl_sync(0xffffffffu, last, 0);                     // the warp's smallest
    // Weights are 2^(v cf + neg), by one fma a score v: with c = scale log2 e usually cf = c and neg = -m, m
    // the rounded product of c and the largest v.  The fma's product is exact, so all weights of a row share a
    // factor 2^x, |x| at most half a step of m, which their sum and so out and lse take part in.  From
    // |m| = 2^31 on it could leave fp32; there scores that differ do so by 2^7 or more, so weights are 1 or
    // nothing with any factor near c, and cf is a power of two, whose products are exact.
    float m = kNoMax, neg = -kNoMax, cf = p.scale_log2, l = 0.f;
    bool ok = true;
    for (int j = 0; j < nt[t]; ++j) {
      if (!(ok = wait_w(&aux->s_full[t][j & 1], (j >> 1) & 1, aux, p.err))) break;
      ptx::tc_fence_after();
      const int lim = last - j * 128;              // columns 0..lim are visible
      uint32_t v[4][32];                           // the row's scores, as fp32 bits
#pragma unroll
      for (int c = 0; c < 4; ++c) ptx::tmem_ld32(s_col + 32 * c, v[c]);
      ptx::tmem_wait_ld();
      if (wlast - j * 128 < 127) {                 // some row of the warp masks columns here
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int e = 0; e < 32; ++e) v[c][e] = 32 * c + e <= lim ? v[c][e] : 0xFF800000u;   // -inf
      }
      if (j * 128 + 128 > rk.n) {
        // the rows behind the last key belong to the next sequence: weight 0, but 0 times an
        // infinity there would be NaN, so their values become 0 (each tile clears them before it
        // hands over its weights; both store the same)
        if (!(ok = wait_w(&aux->v_full[j & 1], (j >> 1) & 1, aux, p.err))) break;
        if (j * 128 + row >= rk.n) {
          const int h = row >> 6;                      // key half: a slot of its own, or half of one
          uint8_t* vs = kv_s + ((j * unit + nkb + (nvb == 2 ? h : 0)) % p.ring) * kBox + (nvb == 2 ? 0 : h * kVBox);
          for (int c = 0; c < nvb; ++c) {
            const uint32_t base = ptx::smem_u32(vs + c * kVBox + (row & 63) * 128);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(base + e * 16), "r"(0) : "memory");
          }
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
      }
      float mx[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        mx[c] = fmaxf(__uint_as_float(v[c][0]), __uint_as_float(v[c][1]));
#pragma unroll
        for (int e = 2; e < 32; e += 2) mx[c] = ptx::max3(mx[c], __uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1]));
      }
      const float vmax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), top = vmax * p.scale_log2;
      if (__any_sync(0xffffffffu, top > m + kLazy)) {
        const float mn = fmaxf(m, top), a = ptx::ex2_approx(m - mn);
        if (top > m) {
          cf = fabsf(top) < 2147483648.f ? p.scale_log2 : p.scale_pow2;
          neg = -(vmax * cf);
        }
        m = mn;
        l *= a;
        if (j > 0) {                               // (PV(j - 1) came before S(j), which is complete)
          for (int c = 0; c < p.dv; c += 16) {
            uint32_t o[16];
            ptx::tmem_ld16(o_col + c, o);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
            ptx::tmem_st16(o_col + c, o);
          }
        }
      }
      const float2 sc = make_float2(cf, cf), nm = make_float2(neg, neg);
      float2 sum[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t w[16];
        sum[c] = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 x = ptx::fma2(make_float2(__uint_as_float(v[c][2 * e]), __uint_as_float(v[c][2 * e + 1])), sc, nm);
          const float2 y = make_float2(ptx::ex2_approx(x.x), ptx::ex2_approx(x.y));
          sum[c] = ptx::add2(sum[c], y);
          const __nv_bfloat162 h = __floats2bfloat162_rn(y.x, y.y);
          w[e] = *reinterpret_cast<const uint32_t*>(&h);
        }
        ptx::tmem_st16(s_col + 16 * c, w);
        if (c & 1) {
          ptx::tmem_wait_st();
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&aux->p_full[t][c >> 1][j & 1]);
        }
      }
      const float2 l2 = ptx::add2(ptx::add2(sum[0], sum[1]), ptx::add2(sum[2], sum[3]));
      l += l2.x + l2.y;
    }
    if (ok && nt[t] > 0) ok = wait_w(&aux->pv_done[t][1][(nt[t] - 1) & 1], ((nt[t] - 1) >> 1) & 1, aux, p.err);
    ptx::tc_fence_after();
    if constexpr (kSplit) {
      // this part's sums take the place of the operands, once both tiles are done with them
      ptx::named_bar_sync(1, 256);
      reinterpret_cast<float2*>(part_s)[t * 128 + row] = make_float2(m, ok ? l : 0.f);
      for (int c = 0; c < p.dv; c += 32) {
        uint32_t v[32];
        if (nt[t] > 0) {
          ptx::tmem_ld32(o_col + c, v);
          ptx::tmem_wait_ld();
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
          *reinterpret_cast<uint4*>(part_s + kPartMl + (t * 128 + row) * (p.dv * 4 + 16) + (c + 4 * e) * 4) =
              make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        __syncwarp();
      }
    } else if (ok) {
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
  if constexpr (kSplit) {
    __syncwarp();
    ptx::cluster_sync();                 // every part's sums are in place
    const int rows = 256 / p.split, vecs = p.dv >> 2;
    const uint32_t at = ptx::smem_u32(part_s);
    for (int idx = threadIdx.x; idx < rows * vecs; idx += kThreads) {
      const int r = part * rows + idx / vecs, c = idx % vecs * 4, i = q0 + r;
      if (i >= rq.n) continue;
      float2 ml[kMaxSplit];
      float top = kNoMax;
#pragma unroll
      for (int k = 0; k < kMaxSplit; ++k)
        if (k < p.split) {
          ml[k] = ptx::ld_cluster_f2(ptx::map_rank(at + r * 8, k));
          if (ml[k].y != 0.f) top = fmaxf(top, ml[k].x);
        }
      float l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kMaxSplit; ++k)
        if (k < p.split && ml[k].y != 0.f) {           // (a part that saw no key holds nothing)
          const float w = ptx::ex2_approx(ml[k].x - top);
          const float4 v = ptx::ld_cluster_f4(ptx::map_rank(at + kPartMl + r * (p.dv * 4 + 16) + c * 4, k));
          l += w * ml[k].y;
          o.x += w * v.x;
          o.y += w * v.y;
          o.z += w * v.z;
          o.w += w * v.w;
        }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const __nv_bfloat162 a = __floats2bfloat162_rn(o.x * inv, o.y * inv), b2 = __floats2bfloat162_rn(o.z * inv, o.w * inv);
      const size_t to = ((size_t)rq.first + i) * p.Hq + head;
      *reinterpret_cast<uint2*>(p.out + to * p.dv + c) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b2));
      if (c == 0 && p.lse) p.lse[to] = l == 0.f ? -INFINITY : (top + log2f(l)) * LR_LN2;
    }
    __syncwarp();
    ptx::cluster_sync();                 // none leaves while another reads its sums
  }
}

bool map2d(CUtensorMap* m, const void* ptr, uint64_t d0, uint64_t d1, uint32_t rows = 128) {
  const cuuint64_t dims[2] = {d0, d1}, st[1] = {d0 * 2};
  const cuuint32_t box[2] = {64, rows};
  return tc::make_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, ptr, 2, dims, st, box);
}
bool map3d(CUtensorMap* m, const void* ptr, uint64_t d0, uint64_t d1, uint64_t d2) {
  const cuuint64_t dims[3] = {d0, d1, d2}, st[2] = {d0 * 2, d0 * d1 * 2};
  const cuuint32_t box[3] = {64, 1, 128};
  return tc::make_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, ptr, 3, dims, st, box);
}

template <bool kSplit>
cudaError_t launch(const AttArgs& a, size_t smem, cudaStream_t s, const CUtensorMap& tq, const CUtensorMap& tk,
                   const CUtensorMap& tkr, const CUtensorMap& tv) {
  static std::atomic<uint32_t> optin{0};
  cudaError_t e = smem_optin(k_shared_attn<kSplit>, optin);
  if (e != cudaSuccess) return e;
  // the register split was sized for exactly this launch allocation (an increase beyond it waits)
  static std::atomic<int> regs{-1};
  if (regs.load() < 0) {
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, k_shared_attn<kSplit>) == cudaSuccess) regs.store(fa.numRegs);
  }
  if (regs.load() != kLaunchRegs) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)(a.slots * a.Hq * a.split));
  return kSplit ? launch_pdl_cluster(k_shared_attn<kSplit>, grid, dim3(kThreads), a.split, smem, s, tq, tk, tkr, tv, a)
                : launch_pdl(k_shared_attn<kSplit>, grid, dim3(kThreads), smem, s, tq, tk, tkr, tv, a);
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
  a.scale_pow2 = std::scalbn(1.f, std::ilogb(a.scale_log2));
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.err = c->dev_err;
  const long long slots = (long long)total_q / 256 + std::min(nseq, total_q);
  if (slots * a.Hq > 0x7FFFFFFF) return cudaErrorNotSupported;
  a.slots = (int)slots;
  a.stagger = ((long long)total_q + 255) / 256 * a.Hq <= c->num_sms;
  CUtensorMap tq, tk, tkr, tv;
  if (total_k == 0) k = kr = v = q;      // no key tile is ever loaded; the maps need an address
  const cuuint64_t rows = std::max(total_k, 1);
  if (!map3d(&tq, q, a.dq, a.Hq, total_q) || !map2d(&tk, k, (uint64_t)d.n_kv_heads * a.dn, rows) ||
      !map2d(&tv, v, (uint64_t)d.n_kv_heads * a.dv, rows, 64) || !map2d(&tkr, kr, d.dim_rope, rows))
    return cudaErrorInvalidValue;
  // the ring: what the query tiles leave of shared memory, at most two tiles of keys and values
  const int nqb = (a.dq + 63) / 64, unit = a.dn / 64 + 1 + a.dv / 64;
  a.ring = std::min(2 * unit, (int)((tc::kSmemLimit - kAuxBytes) / kBox) - 2 * nqb);
  const size_t smem = kAuxBytes + (size_t)(2 * nqb + a.ring) * kBox;
  // Split the keys while there are SMs for all parts and each keeps two key tiles (by the average).  Timed
  // alone, in short bursts: 4 heads, 512 new tokens over 8192: 158 us without, 38 with a split of 8; 28 heads,
  // 256 over 30000: 597 without, 325 in two parts.  (A cluster lies in one GPC: 15 of 8 CTAs run at once, so
  // 16 to 18 take two waves, and as long as in fours: 200 over 30000 with 15 heads 96 us, 16 to 18 187, 19 179.)
  a.split = 1;
  while (a.split < kMaxSplit && 2 * a.split * slots * a.Hq <= c->num_sms && total_k / (256 * nseq) >= 2 * a.split) a.split *= 2;
  return a.split > 1 ? launch<true>(a, smem, s, tq, tk, tkr, tv) : launch<false>(a, smem, s, tq, tk, tkr, tv);
}
