// Absorbed decode over a shared-latent cache: a few query tokens per sequence against every
// stored token, without rebuilding keys or values.
//
//   q~_j = B_k,h q_nope,j                              k_shared_qproj   (rank space, per head)
//   s_tj = scale (c_t . q~_j + kr_t . q_rope,j)        k_shared_decode  GEMM1, M = 64 tokens
//   o~_j = sum_t p_tj c_t,  p = softmax over visible t k_shared_decode  GEMM2, M = 128 ranks
//   out_j = o~_j B_v,h / l_j                           k_shared_out     (merges the splits)
//
// One tile of latents in shared memory serves as keys (rows of GEMM1's A operand, K-major) and,
// through a second descriptor of the same bytes, as values (GEMM2's A operand, MN-major): each
// stored byte crosses HBM once per block of query rows.  Heads are the N side of both MMAs, so a
// block of NR = 16 or 32 query rows pays for no empty rows of a 128-row operand.
//
// Tiles are 64 tokens, half a page: beside the query latents (64 KB at r = 512) two such tiles
// fit, so one is fetched while the other is at work.  With 128-token tiles only one fits, and its
// fetch, scores, softmax and value mix follow one another (4.1 us a tile of bf16, 6.2 us of 8
// bits, against 1.9 us of copies); splitting the rank over two CTAs instead costs two exchanges a
// tile and came out the same.  A GEMM1 step of 64 x 64 takes 33 clocks (128 x 64: 48), so smaller
// tiles cost the tensor pipe 1.4 times the time per token, ~1800 clocks a tile at r = 512, still
// below the 3300 that a bf16 tile takes from HBM.
//
// Measured (r = 512, 28 heads): a bf16 tile every ~3000 clocks (of its chain, fetch 2100, scores
// 1200, softmax 1000, value mix 1000, two tiles are under way); 16 x 4096 tokens 25 us, of which the
// first tile's way through the SM takes 6.  An 8-bit tile every ~3800 clocks: its codes' expansion
// (3000 clocks by 16 warps) takes the fetch's place in the chain; 16 x 32768 tokens 131 us, 2.6 TB/s.
//
// Roundings: q~ enters GEMM1 as two bf16 halves, hi and lo = q~ - hi, stacked on N and added in
// fp32: the scores, and so lse, carry ~16 bits of q~.  The rotary query is bf16 as given.  p enters
// GEMM2 as one bf16 (half a step, 2^-8 relative at most); its sum, for lse and the normaliser, is of the
// unrounded weights in fp32.  So weights that differ round at random over the tokens, but equal ones that
// are no powers of two alike: the output is then off by up to 2^-8 of its size before its own rounding.
// (Dividing by the sum of the rounded weights, which cancels that, beside the one for lse: 16 x 4096
// tokens 34.4 -> 35.0 us, 16 x 32768 of 8 bits 134.7 -> 139.7.)
//
// Work: the tiles of all sequences, in order, are cut into equal runs on the device (tile_run),
// one run per CTA column, so ragged batches stay balanced and a captured graph serves any
// lengths.  A run's part of one sequence is one partial (m, l, o~), joined by k_shared_out.
#include "shared_internal.cuh"
#include "tc_common.cuh"

#include <algorithm>

namespace {

using tc::drain_wait;
using tc::kLazy;
using tc::kSmemLimit;

constexpr int kTok = 64;               // tokens of a tile
constexpr int kSub = kTok * 128;       // 64 tokens x 64 ranks x 2 B (one TMA box)
constexpr int kWSub = 128 * 128;       // 128 rows x 64 columns x 2 B (the projections' operands)
constexpr int kAuxBytes = 2048;
constexpr int kMaxSlots = 4;
constexpr float kNoMax = -3.402823466e38f;   // running max before any visible token: finite (no inf - inf), and below every score
constexpr int kSCol = 0;               // TMEM: S of tile t and rank half h in columns [128 (t % 2) + 64 h, + 2 NR)
constexpr int kOCol = 256;             // TMEM: O~ of 128-rank block k in columns [256 + k NR, + NR)

struct DecArgs {
  unsigned long long wait_ns;
  const int32_t* row_len;
  RowMap map;
  int B, cap, r, Hq, n_tok, R, HB, X, nslot;
  float scale_log2;
  const uint8_t* codes;
  const uint8_t* scale;
  float* part_o;
  float* part_ml;
  int* err;
};

// A sequence's length and a page, read before the grid-dependency wait.  The kernel before (k_shared_qproj,
// or k_shared_decode for the join) let this one in only after its own wait, so all work before the call,
// whatever wrote lengths, pages and rows, is complete; only the query latents (the partials) are still on
// their way.  The reads go to L2, past whatever an SM's L1 may hold from before.
__device__ __forceinline__ int early_len(const int32_t* row_len, int b, int cap) {
  return min(max(__ldcg(row_len + b), 0), cap);
}
__device__ __forceinline__ int early_page(const RowMap& m, int b, int t) {
  return min(max(__ldcg(m.table + (long long)b * m.pps + (t >> 7)), 0), m.n_pages - 1);
}

// The next sequence part of a run: false at its end.  Every role walks its own copy.
struct Seg {
  int b, t0, nt, len;
};
__device__ __forceinline__ bool next_seg(TileRun* run, const DecArgs& p, Seg* s) {
  while (run->left > 0 && run->b < p.B) {
    const int len = early_len(p.row_len, run->b, p.cap);
    const int nt = (len + kTok - 1) / kTok - run->tile;
    if (nt <= 0) {
      ++run->b;
      run->tile = 0;
      continue;
    }
    s->b = run->b;
    s->t0 = run->tile;
    s->nt = min(nt, run->left);
    s->len = len;
    run->left -= s->nt;
    ++run->b;
    run->tile = 0;
    return true;
  }
  return false;
}

// Sixteen codes of one token (their words in the order in which they are stored), times 2^e, to
// two 16-byte columns of a swizzled row: w.x, w.y to address a0 and w.z, w.w to a1.
__device__ __forceinline__ void expand16(const uint4& w, uint32_t eb, uint32_t a0, uint32_t a1) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
  uint32_t o[8];
  shared_expand<4>(in, eb, o);
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a0), "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3])
               : "memory");
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a1), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
               : "memory");
}
// A warp-uniform value, known as such to the compiler: MMA operands then stay in uniform registers
// (an MMA issues at the tensor core's pace; without, every ~160 cycles).
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

// Sixteen codes of one token row of a 128-rank chunk, per thread of 256: 1 << sh = 8 threads a row, so
// 32 rows a step; in a last chunk of 64 ranks 4 threads a row, one step.  The codes lie at 16 tid in
// the chunk's rows; this is where the first of their two 16-byte bf16 columns goes in the chunk's
// boxes (the second is at ^ 16).  128-byte swizzle: column v of row tok sits at v ^ (tok % 8); the
// lanes of the second box take their two columns in the other order, so that the eight lanes of a row
// store to eight different columns.
__device__ __forceinline__ uint32_t code_place(int tid, int sh) {
  const int col = tid & ((1 << sh) - 1), tok = tid >> sh, swap = col >> 2;
  return (uint32_t)(swap * kSub + tok * 128) + ((((col & 3) * 2 + swap) ^ (tok & 7)) << 4);
}

// Barriers (arrival count; who arrives -> who waits); phase k is waited with parity k & 1.  NG =
// NR / 16 groups of four softmax warps.
//   full[s][h]      1 + tx   producer's boxes -> GEMM1 issuer; half h of the ranks (half_of_block), the
//                            rotary box with the second (8 bits: 16 expansion warps, after their blocks
//                            0 and 1 and after 2 and 3, + 1 + tx with the rotary box; at two blocks in all
//                            the second one is there early, with full[s][0])
//   empty[s][h]     1        GEMM2's commit on half h -> producer, expansion warps (each for the half of
//                            the block it writes)
//   q_full/q_empty  1 + tx / 2   per sequence of the run
//   s_full[2]       2        GEMM1's commits (one a half) -> softmax warps
//   s_empty[2]      4 NG     softmax warps (scores read) -> GEMM1 issuer
//   p_full[2]       4 NG     softmax warps -> GEMM2 issuer
//   p_empty[2]      1        GEMM2's commit -> softmax warps (P may be rewritten, O~ rescaled)
//   o_full          1        GEMM2's commit, last tile of a sequence -> softmax warps
//   o_empty         4 NG     softmax warps (O~ read) -> GEMM2 issuer
//   done            3        final commits of the issuers: every MMA complete before TMEM is freed
struct Aux {
  uint64_t full[kMaxSlots][2], empty[kMaxSlots][2];
  uint64_t q_full, q_empty, s_full[2], s_empty[2], p_full[2], p_empty[2], o_full, o_empty, done;
  uint32_t tmem_base;
  int abort_flag;
  unsigned long long wait_ns;
  TileRun run;
  float red[2][4][16];               // [group][lane quarter][row]
  alignas(16) float alpha[2][16];    // [group][row]: factors of a rescale
  int off_s[32];                     // row j sees tokens t < len + off_s[j]
};
static_assert(sizeof(Aux) <= kAuxBytes, "aux block");

__device__ __forceinline__ bool wait_b(uint64_t* bar, uint32_t parity, Aux* aux, int* err) {
  // (tc::wait_b with the barrier's own suspend time: with a longer hint a waiting warp takes part in
  // a software loop of short sleeps, and 27 warps wait here at times)
  if (ptx::mbar_test_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer();
  for (;;) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    if (*(volatile int*)&aux->abort_flag) return false;
    if (ptx::globaltimer() - t0 > aux->wait_ns) {
      *(volatile int*)&aux->abort_flag = 1;
      atomicExch(err, (int)LR_ERR_TIMEOUT);
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_w(uint64_t* bar, uint32_t parity, Aux* aux, int* err) {
  return __all_sync(0xffffffffu, wait_b(bar, parity, aux, err));
}

// A use count of a ring: slot and phase parity, without divisions.
struct Ring {
  int slot = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next(int n) {
    if (++slot == n) {
      slot = 0;
      ph ^= 1;
    }
  }
};

// Sum or maximum over the lanes that share lane % 4 (the same score columns).
template <bool kMax>
__device__ __forceinline__ float reduce_rows(float v) {
#pragma unroll
  for (int o = 4; o <= 16; o <<= 1) {
    const float got = __shfl_xor_sync(0xffffffffu, v, o);
    v = kMax ? fmaxf(v, got) : v + got;
  }
  return v;
}

// Warps: 0 TMA producer, 1 and 3 GEMM1 issuers, one for each half of the ranks (an MMA and what
// prepares it take a warp ~85 clocks here, 33 in the pipe, so two warps fill it better; each half
// has its own accumulator, as nothing orders the MMAs of two warps), 2 GEMM2 issuer; then NG groups of
// four softmax warps, 16 query rows each; (8 bits) 16 warps that expand codes to bf16.
template <int NR, bool kQuant>
constexpr int dec_threads() {
  return 128 + NR * 8 + (kQuant ? 512 : 0);
}
__host__ __device__ constexpr int dec_slot(int r) { return (r / 64 + 1) * kSub; }   // a tile, its rotary box last
// A tile's ranks in two halves that are filled and given back apart: the first (nch + 1) / 2 of its nch
// blocks of 128 ranks, and the others (at 64 and 128 ranks there are none).  In 64-rank boxes:
__host__ __device__ constexpr int first_boxes(int r) {
  const int all = r / 64, half = ((r + 127) / 128 + 1) / 2 * 2;
  return half < all ? half : all;
}
__host__ __device__ constexpr int half_of_block(int c, int r) { return 2 * c >= first_boxes(r); }

// Shared memory: [aux][q~: r/64 blocks of (2 NR rows hi | lo) x 128 B][q_rope: NR rows x 128 B]
// [P: 2 x 64 tokens x NR][slots].
template <int NR, bool kQuant>
__global__ void __launch_bounds__(dec_threads<NR, kQuant>(), 1)
    k_shared_decode(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_qr,
                    const __grid_constant__ CUtensorMap tm_c, const __grid_constant__ CUtensorMap tm_kr,
                    const DecArgs p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (ptx::smem_u32(smem_raw) & 1023) {      // layout precondition; uniform for the whole CTA
    if (threadIdx.x == 0) atomicExch(p.err, (int)LR_ERR_UNSUPPORTED);
    return;
  }
  constexpr int NG = NR / 16, kQSub = 2 * NR * 128, kPBuf = kTok * NR * 2;
  const int nsub = p.r >> 6, nch = (p.r + 127) >> 7;
  const int slot_bytes = dec_slot(p.r), nsub0 = first_boxes(p.r);
  Aux* aux = reinterpret_cast<Aux*>(smem_raw);
  uint8_t* q_s = smem_raw + kAuxBytes;
  uint8_t* qr_s = q_s + nsub * kQSub;
  uint8_t* p_s = qr_s + NR * 128;
  uint8_t* ring = p_s + 2 * kPBuf;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int x = blockIdx.x, hb = blockIdx.y;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.nslot; ++s) {
      ptx::mbar_init(&aux->full[s][0], kQuant ? 16 : 1);
      ptx::mbar_init(&aux->full[s][1], kQuant ? 17 : 1);
      ptx::mbar_init(&aux->empty[s][0], 1);
      ptx::mbar_init(&aux->empty[s][1], 1);
    }
    ptx::mbar_init(&aux->q_full, 1);
    ptx::mbar_init(&aux->q_empty, 2);
    for (int k = 0; k < 2; ++k) {
      ptx::mbar_init(&aux->s_full[k], 2);
      ptx::mbar_init(&aux->s_empty[k], 4 * NG);
      ptx::mbar_init(&aux->p_full[k], 4 * NG);
      ptx::mbar_init(&aux->p_empty[k], 1);
    }
    ptx::mbar_init(&aux->o_full, 1);
    ptx::mbar_init(&aux->o_empty, 4 * NG);
    ptx::mbar_init(&aux->done, 3);
    aux->abort_flag = 0;
    aux->wait_ns = tc::wait_limit(p.wait_ns);
    ptx::fence_mbar_init();
  }
  if (threadIdx.x >= 64 && threadIdx.x < 64 + NR) {   // query row j of this block belongs to token (hb NR + j) / Hq
    const int j = threadIdx.x - 64;
    aux->off_s[j] = min((hb * NR + j) / p.Hq, p.n_tok - 1) - (p.n_tok - 1);
  }
  if (warp == 0 && lane == 0) {
    ptx::prefetch_tmap(&tm_q);
    ptx::prefetch_tmap(&tm_qr);
    ptx::prefetch_tmap(&tm_c);
    ptx::prefetch_tmap(&tm_kr);
  }
  // TMEM: a CTA that held some while it waited for a grid could keep that grid from its own.  So a kernel
  // here lets dependents in once it holds its TMEM, and takes it after its wait; or before, as here, where
  // the grid to be waited for (k_shared_qproj) is known to hold its own by now.
  if (warp == 1) {
    ptx::tmem_alloc(&aux->tmem_base, 512);
    ptx::tmem_relinquish();
  }
  if (warp == 0) {
    int chunk;
    const TileRun run = tile_run([&](int b) { return (early_len(p.row_len, b, p.cap) + kTok - 1) / kTok; }, p.B,
                                 p.X, x, &chunk);
    if (lane == 0) aux->run = run;
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = aux->tmem_base;
  TileRun run = aux->run;
  Seg sg;

  if (warp == 0) {
    // ------------------------------------------------------------- TMA producer
    if (lane == 0) {
      int gt = 0, nseg = 0;              // tiles and sequences issued
      Ring w;
      bool ok = true;
      while (ok && next_seg(&run, p, &sg)) {
        for (int i = 0; i < sg.nt; ++i) {
          const int tok = (sg.t0 + i) * kTok, half = tok & 64;
          const long long page = early_page(p.map, sg.b, tok);
          uint8_t* dst = ring + w.slot * slot_bytes;
          const int row = (int)page * 128 + half;
          uint64_t* const full = aux->full[w.slot];
          // (an abort between the halves leaves the first one's copies to the drain below, whose wait for
          // the second half then runs into its limit)
          bool begun = false;
          if (!kQuant) {
            if (gt >= p.nslot && !(ok = wait_b(&aux->empty[w.slot][0], w.ph ^ 1, aux, p.err))) break;
            begun = true;
            ptx::mbar_arrive_expect_tx(&full[0], (uint32_t)(nsub0 * kSub));
            for (int s = 0; s < nsub0; ++s) ptx::tma_load_2d(dst + s * kSub, &tm_c, &full[0], s * 64, row);
          }
          if (gt < p.nslot || (ok = wait_b(&aux->empty[w.slot][1], w.ph ^ 1, aux, p.err))) {
            begun = true;
            ptx::mbar_arrive_expect_tx(&full[1], (uint32_t)((kQuant ? 1 : nsub - nsub0 + 1) * kSub));
            if (!kQuant)
              for (int s = nsub0; s < nsub; ++s) ptx::tma_load_2d(dst + s * kSub, &tm_c, &full[1], s * 64, row);
            ptx::tma_load_2d(dst + nsub * kSub, &tm_kr, &full[1], 0, row);
          }
          if (!begun) break;
          ++gt;
          w.next(p.nslot);
          if (!ok) break;
          if (i > 0) continue;
          // the query latents, behind the first tile: it has further to come
          pdl_wait();
          pdl_trigger();
          if (nseg > 0 && !(ok = wait_b(&aux->q_empty, (nseg - 1) & 1, aux, p.err))) break;
          ptx::mbar_arrive_expect_tx(&aux->q_full, (uint32_t)(nsub * kQSub + NR * 128));
          for (int s = 0; s < nsub; ++s)
            ptx::tma_load_2d(q_s + s * kQSub, &tm_q, &aux->q_full, s * 64, (sg.b * p.HB + hb) * 2 * NR);
          ptx::tma_load_3d(qr_s, &tm_qr, &aux->q_full, 0, hb * NR, sg.b);
          ++nseg;
        }
      }
      pdl_wait();          // (a CTA without work too: this grid must not end before the one it waits for)
      // every copy this thread issued has landed before the CTA can exit
      if (nseg > 0) drain_wait(&aux->q_full, (nseg - 1) & 1);
      for (int k = min(gt, p.nslot); k > 0; --k) {
        if (w.slot == 0) w.ph ^= 1;
        w.slot = w.slot ? w.slot - 1 : p.nslot - 1;
        if (!kQuant) drain_wait(&aux->full[w.slot][0], w.ph);
        drain_wait(&aux->full[w.slot][1], w.ph);
      }
    }
    __syncwarp();
  } else if (warp == 1 || warp == 3) {
    // ------------------------------------------------------------- GEMM1 issuer (warp-wide)
    const uint32_t id1 = ptx::idesc_f16(1, 0, 0, kTok, 2 * NR);  // K-major x K-major (hi | lo)
    const uint32_t idr = ptx::idesc_f16(1, 0, 0, kTok, NR);      // rotary part, into the hi columns
    const uint64_t kd0 = ptx::smem_desc(ptx::smem_u32(ring), 16, 1024, 2);
    const int h = warp == 3, s0 = h ? nsub0 : 0, s1 = h ? nsub : nsub0;   // half of the ranks, its boxes
    const uint64_t qb = ptx::smem_desc(ptx::smem_u32(q_s + s0 * kQSub), 16, 1024, 2);
    const uint64_t qrd = ptx::smem_desc(ptx::smem_u32(qr_s), 16, 1024, 2);
    int gt = 0, nseg = 0;
    Ring w;
    bool ok = true;
    while (ok && next_seg(&run, p, &sg)) {
      if (!(ok = wait_w(&aux->q_full, nseg & 1, aux, p.err))) break;
      for (int i = 0; i < sg.nt; ++i, ++gt, w.next(p.nslot)) {
        uint64_t a = kd0 + uniform((uint32_t)(w.slot * slot_bytes + s0 * kSub) >> 4), b = qb;
        const uint32_t d_s = uniform(tmem + kSCol + 128 * (gt & 1) + 64 * h);
        if (gt >= 2 && !(ok = wait_w(&aux->s_empty[gt & 1], ((gt >> 1) - 1) & 1, aux, p.err))) break;
        if (!(ok = wait_w(&aux->full[w.slot][h], w.ph, aux, p.err))) break;
        ptx::tc_fence_after();
#pragma unroll 1
        for (int s = s0; s < s1; ++s, a += kSub >> 4, b += kQSub >> 4) {
          const uint32_t more = s > s0 ? 1u : 0u;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            ptx::mma_f16_elect(d_s, a + (uint64_t)(kk * 2), b + (uint64_t)(kk * 2), id1, kk ? 1u : more);
        }
        if (h == 1) {                        // the rotary box follows the ranks' boxes
          const uint32_t more = s1 > s0 ? 1u : 0u;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)     // columns past dim_rope are 0 on both sides
            ptx::mma_f16_elect(d_s, a + (uint64_t)(kk * 2), qrd + (uint64_t)(kk * 2), idr, kk ? 1u : more);
        }
        ptx::mma_commit_elect(&aux->s_full[gt & 1]);
        if (i == sg.nt - 1) ptx::mma_commit_elect(&aux->q_empty);
      }
      ++nseg;
    }
    ptx::mma_commit_elect(&aux->done);
    drain_wait(&aux->done, 0);
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------------- GEMM2 issuer (warp-wide)
    const uint32_t id2 = ptx::idesc_f16(1, 1, 1, 128, NR);       // MN-major x MN-major
    const uint64_t vd0 = ptx::smem_desc(ptx::smem_u32(ring), kSub, 1024, 2);
    const uint64_t pd0 = ptx::smem_desc(ptx::smem_u32(p_s), 128, 1024, 0);
    int gt = 0, nseg = 0;
    Ring w;
    bool ok = true;
    while (ok && next_seg(&run, p, &sg)) {
      for (int i = 0; i < sg.nt; ++i, ++gt, w.next(p.nslot)) {
        const uint64_t vd = vd0 + uniform((uint32_t)(w.slot * slot_bytes) >> 4);
        const uint64_t pd = pd0 + uniform((uint32_t)((gt & 1) * kPBuf) >> 4);
        const uint32_t first = uniform(i ? 1u : 0u), d_o = uniform(tmem + kOCol);
        if (i == 0 && nseg > 0 && !(ok = wait_w(&aux->o_empty, (nseg - 1) & 1, aux, p.err))) break;
        if (!(ok = wait_w(&aux->p_full[gt & 1], (gt >> 1) & 1, aux, p.err))) break;
        ptx::tc_fence_after();
        // a last block of 64 ranks mixes the box behind it into rows that nobody reads
        uint64_t a = vd;
        uint32_t d = d_o;
#pragma unroll 1
        for (int c = 0; c < nch; ++c, a += 2 * kSub >> 4, d += NR) {
#pragma unroll
          for (int kt = 0; kt < 4; ++kt)
            ptx::mma_f16_elect(d, a + (uint64_t)(kt * 128), pd + (uint64_t)(kt * 16), id2, kt ? 1u : first);
          if (2 * c + 2 == (nsub0 + 1) / 2 * 2) ptx::mma_commit_elect(&aux->empty[w.slot][0]);
        }
        ptx::mma_commit_elect(&aux->empty[w.slot][1]);
        ptx::mma_commit_elect(&aux->p_empty[gt & 1]);
        if (i == sg.nt - 1) ptx::mma_commit_elect(&aux->o_full);
      }
      ++nseg;
    }
    ptx::mma_commit_elect(&aux->done);
    drain_wait(&aux->done, 0);
    __syncwarp();
  } else if (warp >= 4 && warp < 4 + 4 * NG) {
    // ------------------------------------------------------------- softmax / epilogue
    // Scores of 64 tokens stand in lanes 0..15 of each lane quarter; the fragment load spreads 16
    // lanes x 16 columns over the warp: lane l has tokens l / 4 and l / 4 + 8 of the quarter's 16,
    // columns 2 (l % 4), + 1, and the same + 8.
    const int qd = warp & 3, g = (warp - 4) >> 2;        // lane quarter, group of 16 query rows
    const uint32_t lane_off = (uint32_t)(qd * 32) << 16;
    const int tok0 = qd * 16 + (lane >> 2), col0 = 16 * g + 2 * (lane & 3);
    const uint32_t p_at = ptx::smem_u32(p_s + 2 * g * (kTok * 16) + tok0 * 16 + (lane & 3) * 4);
    int gt = 0, nseg = 0;
    Ring w;
    bool ok = true;
    while (ok && next_seg(&run, p, &sg)) {
      float m[4], l[4];                                  // of the columns; m in units of log2, alike in the whole group
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        m[k] = kNoMax;
        l[k] = 0.f;
      }
      for (int i = 0; i < sg.nt; ++i, ++gt, w.next(p.nslot)) {
        const int k2 = gt & 1, t = (sg.t0 + i) * kTok + tok0;
        const uint32_t s_col = tmem + lane_off + kSCol + 128 * k2 + 16 * g;
        // after an abort every wait returns at once: the warps finish the sequence in step (their
        // barriers stay matched) and leave at the verdict below
        (void)wait_w(&aux->s_full[k2], (gt >> 1) & 1, aux, p.err);
        ptx::tc_fence_after();
        uint32_t hi[8], lo[8], hi1[8], lo1[8];
        ptx::tmem_ld16x256_x2(s_col, hi);
        ptx::tmem_ld16x256_x2(s_col + NR, lo);
        ptx::tmem_ld16x256_x2(s_col + 64, hi1);
        ptx::tmem_ld16x256_x2(s_col + 64 + NR, lo1);     // (nothing there if all ranks are in the first half)
        ptx::tmem_wait_ld();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&aux->s_empty[k2]);
        float s[2][4];                                   // [token of the two][column]
#pragma unroll
        for (int e = 0; e < 8; ++e)
          s[(e >> 1) & 1][(e >> 2) * 2 + (e & 1)] =
              ((__uint_as_float(hi[e]) + __uint_as_float(hi1[e])) +
               (__uint_as_float(lo[e]) + (nsub > nsub0 ? __uint_as_float(lo1[e]) : 0.f))) *
              p.scale_log2;
        // a tile every row sees whole needs no masks; otherwise row j sees t < len + off
        if ((sg.t0 + i) * kTok + kTok > sg.len - (p.n_tok - 1)) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int end = sg.len + aux->off_s[col0 + 8 * (k >> 1) + (k & 1)];
            s[0][k] = t < end ? s[0][k] : -INFINITY;
            s[1][k] = t + 8 < end ? s[1][k] : -INFINITY;
          }
        }
        bool ex = false;
#pragma unroll
        for (int k = 0; k < 4; ++k) ex |= fmaxf(s[0][k], s[1][k]) > m[k] + kLazy;
        ex = ptx::named_bar_or(1 + g, 128, ex);
        if (ex) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float top = reduce_rows<true>(fmaxf(s[0][k], s[1][k]));
            if (lane < 4) aux->red[g][qd][col0 - 16 * g + 8 * (k >> 1) + (k & 1)] = top;   // read by all before the next vote
          }
          ptx::named_bar_sync(1 + g, 128);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int c = col0 - 16 * g + 8 * (k >> 1) + (k & 1);
            const float mn = fmaxf(m[k], fmaxf(fmaxf(aux->red[g][0][c], aux->red[g][1][c]),
                                               fmaxf(aux->red[g][2][c], aux->red[g][3][c])));
            const float a = ptx::ex2_approx(m[k] - mn);
            m[k] = mn;
            l[k] *= a;
            if (qd == 0 && lane < 4) aux->alpha[g][c] = a;
          }
          if (i > 0) {
            // the value mixes before have completed, then the group's 16 columns of O~ are rescaled
            ptx::named_bar_sync(1 + g, 128);
            (void)wait_w(&aux->p_empty[k2 ^ 1], ((gt - 1) >> 1) & 1, aux, p.err);
            ptx::tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 2 * nch; ++c) {            // 8 columns at a time
              uint32_t v[8];
              const int j0 = 8 * (c & 1);
              const uint32_t col = tmem + lane_off + kOCol + (c >> 1) * NR + 16 * g + j0;
              ptx::tmem_ld8(col, v);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 8; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * aux->alpha[g][j0 + j]);
              ptx::tmem_st8(col, v);
            }
            ptx::tmem_wait_st();
          }
        }
        if (!kQuant && sg.len - (sg.t0 + i) * kTok < kTok) {
          // rows behind the sequence hold whatever the page held: 0 weight times a stale
          // infinity would still be NaN, so their values become 0
          for (int c = warp - 4; c < nsub; c += 4 * NG)
            for (int rr = lane; rr < kTok; rr += 32)
              if ((sg.t0 + i) * kTok + rr >= sg.len) {
                const uint32_t base = ptx::smem_u32(ring + w.slot * slot_bytes + c * kSub + rr * 128);
#pragma unroll
                for (int v = 0; v < 8; ++v)
                  asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(base + v * 16), "r"(0) : "memory");
              }
          __syncwarp();
        }
        if (gt >= 2) (void)wait_w(&aux->p_empty[k2], ((gt >> 1) - 1) & 1, aux, p.err);   // this buffer's last use
#pragma unroll
        for (int tk = 0; tk < 2; ++tk)
#pragma unroll
          for (int cb = 0; cb < 2; ++cb) {
            const float p0 = ptx::ex2_approx(s[tk][2 * cb] - m[2 * cb]);
            const float p1 = ptx::ex2_approx(s[tk][2 * cb + 1] - m[2 * cb + 1]);
            const __nv_bfloat162 h = __floats2bfloat162_rn(p0, p1);
            l[2 * cb] += p0;
            l[2 * cb + 1] += p1;
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(p_at + k2 * kPBuf + cb * (kTok * 16) + tk * 128),
                         "r"(*reinterpret_cast<const uint32_t*>(&h))
                         : "memory");
          }
        // the weights become visible to the tensor core, then one arrival per warp
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&aux->p_full[k2]);
      }
      ok = ptx::named_bar_and(1 + g, 128, wait_b(&aux->o_full, nseg & 1, aux, p.err));
      if (!ok) break;
      ptx::tc_fence_after();
      const size_t base = ((size_t)(x + sg.b) * p.HB + hb) * NR;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float lt = reduce_rows<false>(l[k]);
        if (lane < 4) aux->red[g][qd][col0 - 16 * g + 8 * (k >> 1) + (k & 1)] = lt;
      }
      ptx::named_bar_sync(1 + g, 128);
      if (qd == 0 && lane < 4) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int c = col0 - 16 * g + 8 * (k >> 1) + (k & 1);
          const float l4 = (aux->red[g][0][c] + aux->red[g][1][c]) + (aux->red[g][2][c] + aux->red[g][3][c]);
          reinterpret_cast<float2*>(p.part_ml)[base + 16 * g + c] = make_float2(m[k], l4);
        }
      }
      __syncwarp();
      for (int c = 0; c < nch; ++c) {                    // thread = rank row
        const int e = c * 128 + qd * 32 + lane;
        uint32_t o[16];
        ptx::tmem_ld16(tmem + lane_off + kOCol + c * NR + 16 * g, o);
        ptx::tmem_wait_ld();
        if (e < p.r) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (hb * NR + 16 * g + j < p.R) p.part_o[(base + 16 * g + j) * p.r + e] = __uint_as_float(o[j]);
        }
        __syncwarp();
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&aux->o_empty);
      ++nseg;
    }
    __syncwarp();
  } else if (kQuant && warp >= 4 + 4 * NG) {
    // ------------------------------------------------------------- expansion of codes
    // Two groups of 8 warps take the even and the odd chunks.  The codes come straight to registers,
    // fetched anew as soon as a chunk is expanded, so neither their latency nor their copy holds up a
    // free slot.  The code is kept short: the roles of this kernel share the instruction caches, and
    // with addresses made anew for each step its warps waited for instructions more than for anything.
    const int tid = (threadIdx.x - (128 + NR * 8)) & 255, g = (warp - 4 - 4 * NG) >> 3;
    const uint32_t wide = code_place(tid, 3);
    const bool odd = (nsub & 1) != 0, swap = (lane & 4) != 0;
    // the next tile to fetch, its page's table entry, and the rows of the sequence in it
    pdl_wait();                                        // (plain loads, unlike the producer's copies)
    int i = 0, page_n = 0, valid_n = 0;
    bool more = next_seg(&run, p, &sg);
    auto peek = [&]() { page_n = __ldg(p.map.table + (long long)sg.b * p.map.pps + ((sg.t0 + i) * kTok >> 7)); };
    if (more) peek();
    int page = 0, half = 0;                            // of the tile being fetched
    // (past the run's end the last tile is fetched again: loads under a condition were waited for
    // where they were issued)
    auto advance = [&]() {
      if (!more) return false;
      page = min(max(page_n, 0), p.map.n_pages - 1);
      half = (sg.t0 + i) * kTok & 64;
      valid_n = sg.len - (sg.t0 + i) * kTok;           // (may exceed 64)
      if (++i == sg.nt) {
        i = 0;
        more = next_seg(&run, p, &sg);
      }
      if (more) peek();
      return true;
    };
    uint4 x[2][2];                                     // [chunk of the group][step]
    uint32_t eb[2][2];
    auto fetch = [&](int k) {                          // (a chunk that is not there: the group's first again)
      const int c = g + 2 * k < nch ? g + 2 * k : min(g, nch - 1);
      const bool l = odd && c == nch - 1;
      const int sh = l ? 2 : 3;
      const uint8_t* codes = p.codes + ((long long)page * 128 * p.r + (c * 16384 + half * (16 << sh) + tid * 16));
      const uint8_t* scale = p.scale + ((long long)page * nch * 512 +
                                        (c * 512 + (half + (tid >> sh)) * 4 + ((tid & ((1 << sh) - 1)) >> 1)));
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        // (each byte is used once: it has no place in the little L1 that is left)
        x[k][r] = ptx::ld_nc_stream(codes + (l ? 0 : r * 4096));
        eb[k][r] = __ldg(scale + (l ? 0 : r * 128));
      }
    };
    bool got = advance();                              // x holds a tile to expand
    int valid = valid_n;
    fetch(0);
    fetch(1);
    Ring w;
    int gt = 0;
    while (got) {
      got = advance();
      const uint32_t dst = ptx::smem_u32(ring + w.slot * slot_bytes);
      bool ok = true;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int c = g + 2 * k, h = c < nch ? half_of_block(c, p.r) : k;
        if (gt >= p.nslot && !(ok = wait_w(&aux->empty[w.slot][h], w.ph ^ 1, aux, p.err))) break;
        if (c < nch) {
          const bool l = odd && c == nch - 1;
          const uint32_t box = dst + 2 * c * kSub + (l ? code_place(tid, 2) : wide);
          const int tok = tid >> (l ? 2 : 3);
#pragma unroll
          for (int r = 0; r < 2; ++r)
            if (r == 0 || !l) {
              uint4 y = x[k][r];
              if (swap && !l) y = make_uint4(y.z, y.w, y.x, y.y);
              const bool in = tok + r * 32 < valid;        // rows behind the sequence hold whatever the page held
              if (!in) y = make_uint4(0, 0, 0, 0);
              expand16(y, in ? eb[k][r] : 127u, box + r * 4096, (box + r * 4096) ^ 16);
            }
        }
        fetch(k);
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&aux->full[w.slot][k]);
      }
      if (!ok) break;
      valid = valid_n;
      ++gt;
      w.next(p.nslot);
    }
    __syncwarp();
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// Query projection: q~ = B_k,h q_nope for nb (token, sequence) pairs x g heads of one KV head.
// M = 128 ranks (A: rows of B_k,h, K-major), N = the query rows, K = dim_nope.  Every element
// of B_k is read once per row block (a few MB in all): the launch is latency-bound, so one
// CTA does one MMA group straight from two copies, and the basis copy starts before the
// grid-dependency wait.
struct QpArgs {
  unsigned long long wait_ns;
  int r, dn, g, nb, BS, n_tok, Hq, HB, NR, ncols;   // ncols: MMA N (nb g rounded up to 16)
  uint32_t tcols;        // TMEM columns (a power of two)
  __nv_bfloat16* qt;     // [B][HB][2 NR][r]
  int* err;
};
struct QpAux {
  uint64_t w_full, q_full, done;
  uint32_t tmem_base;
  int abort_flag;
  long long at[128];     // element of qt where column m's hi half starts (rank 0), or -1: no such row
};

__global__ void __launch_bounds__(128)
    k_shared_qproj(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_q,
                   const QpArgs p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (ptx::smem_u32(smem_raw) & 1023) {
    if (threadIdx.x == 0) atomicExch(p.err, (int)LR_ERR_UNSUPPORTED);
    return;
  }
  uint8_t* w_s = smem_raw;                       // dn/64 blocks of 128 ranks x 128 B
  uint8_t* q_s = smem_raw + (p.dn >> 6) * kWSub;  // dn/64 blocks of ncols rows x 128 B
  QpAux& aux = *reinterpret_cast<QpAux*>(q_s + (p.dn >> 6) * p.ncols * 128);
  const int i0 = blockIdx.x * 128, h = blockIdx.y, bs0 = blockIdx.z * p.nb;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kb = p.dn >> 6;
  const uint32_t qblk = (uint32_t)p.ncols * 128;
  if (threadIdx.x == 0) {
    ptx::mbar_init(&aux.w_full, 1);
    ptx::mbar_init(&aux.q_full, 1);
    ptx::mbar_init(&aux.done, 1);
    aux.abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::mbar_arrive_expect_tx(&aux.w_full, kb * kWSub);
    for (int k = 0; k < kb; ++k) ptx::tma_load_2d(w_s + k * kWSub, &tm_w, &aux.w_full, h * p.dn + k * 64, i0);
  }
  {
    const int m = threadIdx.x, bs = bs0 + m / p.g;
    long long o = -1;
    if (m < p.nb * p.g && bs < p.BS) {
      const int b = bs / p.n_tok, row = (bs % p.n_tok) * p.Hq + h * p.g + m % p.g;
      o = (((long long)b * p.HB + row / p.NR) * 2 * p.NR + row % p.NR) * p.r;
    }
    aux.at[m] = o;
  }
  pdl_wait();
  if (warp == 1) {            // (after the wait, as in k_shared_decode)
    ptx::tmem_alloc(&aux.tmem_base, p.tcols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  pdl_trigger();
  const uint32_t tmem = aux.tmem_base;
  const uint64_t limit = tc::wait_limit(p.wait_ns);
  if (warp == 0) {
    if (lane == 0) {
      ptx::mbar_arrive_expect_tx(&aux.q_full, (uint32_t)(kb * p.nb * p.g * 128));
      for (int k = 0; k < kb; ++k)       // rows past the last (token, sequence) pair read as 0
        ptx::tma_load_3d(q_s + k * qblk, &tm_q, &aux.q_full, k * 64, h * p.g, bs0);
    }
    __syncwarp();
    const bool ok = __all_sync(0xffffffffu, tc::wait_b(&aux.w_full, 0, &aux.abort_flag, p.err, limit) &&
                                                tc::wait_b(&aux.q_full, 0, &aux.abort_flag, p.err, limit));
    if (ok) {
      ptx::tc_fence_after();
      const uint32_t id = ptx::idesc_f16(1, 0, 0, 128, (uint32_t)p.ncols);
      const uint64_t wd = ptx::smem_desc(ptx::smem_u32(w_s), 16, 1024, 2);
      const uint64_t qd = ptx::smem_desc(ptx::smem_u32(q_s), 16, 1024, 2);
      for (int k = 0; k < kb; ++k)
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          ptx::mma_f16_elect(tmem, wd + (uint64_t)((k * kWSub >> 4) + kk * 2),
                             qd + (uint64_t)((k * qblk >> 4) + kk * 2), id, (k | kk) ? 1u : 0u);
    }
    ptx::mma_commit_elect(&aux.done);
    drain_wait(&aux.w_full, 0);
    drain_wait(&aux.q_full, 0);
    drain_wait(&aux.done, 0);
    __syncwarp();
  }
  __syncthreads();          // warp 0 has seen every MMA complete
  ptx::tc_fence_after();
  const int i = i0 + warp * 32 + lane;
  const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
  if (!aux.abort_flag) {
    for (int c0 = 0; c0 < p.ncols; c0 += 16) {
      uint32_t v[16];
      ptx::tmem_ld16(tmem + lane_off + c0, v);
      ptx::tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const long long at = aux.at[c0 + j];
        if (at < 0 || i >= p.r) continue;
        const float f = __uint_as_float(v[j]);
        const __nv_bfloat16 hi = __float2bfloat16_rn(f);
        const __nv_bfloat16 lo = __float2bfloat16_rn(f - __bfloat162float(hi));
        p.qt[at + i] = hi;
        p.qt[at + (long long)p.NR * p.r + i] = lo;
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, p.tcols);
  }
}

// ---------------------------------------------------------------------------
// Join of the split partials and output projection, per KV head and block of RB (<= 32) query
// rows: o~ = sum_k w_k o~_k / sum_k w_k l_k with w_k = 2^(m_k - max m), then
// out = o~ B_v,h with M = dim_v (A: B_v,h columns, MN-major), N = 2 x 16 or 2 x 32 rows (bf16 hi | lo of o~,
// so that the projection adds no rounding of its own), K = r.  B_v,h is copied before the
// grid-dependency wait; partials come from L2.
struct OutArgs {
  unsigned long long wait_ns;
  const int32_t* row_len;
  int B, cap, r, dv, g, RB, rows, n_tok, Hq, HB, NR, X;   // rows = B n_tok g, of one KV head
  const float* part_o;
  const float* part_ml;
  __nv_bfloat16* out;
  float* lse;
  int* err;
};
constexpr int kOutThreads = 512;
constexpr int kMaxRuns = 160;          // slots one sequence can have: the CTA columns (<= SMs)
struct OutAux {
  uint64_t w_full, done;
  uint32_t tmem_base;
  int abort_flag;
  int first[32], count[32], row[32];   // per row: first slot, slots, row of its sequence,
  long long orow[32];                  // row of the outputs
  float inv[32];
  float w[32][kMaxRuns];
  float4 part[kOutThreads];            // sums over subsets of a row's slots
};

__global__ void __launch_bounds__(kOutThreads)
    k_shared_out(const __grid_constant__ CUtensorMap tm_w, const OutArgs p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (ptx::smem_u32(smem_raw) & 1023) {
    if (threadIdx.x == 0) atomicExch(p.err, (int)LR_ERR_UNSUPPORTED);
    return;
  }
  const int nsub = p.r >> 6;
  const int half = p.RB <= 16 ? 16 : 32;                 // rows of o~'s hi half, then its lo half
  const int oblk = 2 * half * 128;
  uint8_t* o_s = smem_raw;                               // nsub blocks of 2 half rows x 128 B
  uint8_t* w_s = o_s + nsub * oblk;                      // 2 column halves of r rows x 128 B
  OutAux* aux = reinterpret_cast<OutAux*>(w_s + 2 * p.r * 128);
  const int h = blockIdx.y, m0 = blockIdx.x * p.RB;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nv = p.dv >> 6;                              // 64-column halves of B_v,h
  if (threadIdx.x == 0) {
    ptx::mbar_init(&aux->w_full, 1);
    ptx::mbar_init(&aux->done, 1);
    aux->abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::mbar_arrive_expect_tx(&aux->w_full, (uint32_t)(nv * p.r * 128));
    for (int v = 0; v < nv; ++v)
      for (int k = 0; k < nsub; ++k)
        ptx::tma_load_2d(w_s + v * p.r * 128 + k * 64 * 128, &tm_w, &aux->w_full, h * p.dv + v * 64, k * 64);
  }
  if (threadIdx.x < 32) aux->count[threadIdx.x] = 0;
  __syncwarp();
  const int nrow = min(p.RB, p.rows - m0);               // rows m0 .. m0 + nrow - 1
  if (warp == 0) {
    // slots of the rows' sequences, from the same cut into runs as the decode's
    auto tiles = [&](int b) { return (early_len(p.row_len, b, p.cap) + kTok - 1) / kTok; };
    const int chunk = max(1, (tile_total(tiles, p.B) + p.X - 1) / p.X);
    int run = 0;
    const int bk = (m0 + lane) / p.g / p.n_tok;          // the sequence of row m0 + lane
    for (int base = 0; base < p.B; base += 32) {
      const int b = base + lane;
      const int v = b < p.B ? tiles(b) : 0;
      int inc = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
      }
      const int t0 = run + inc - v;
      // lane k: row k's sequence, if it is one of these 32
      const int tk = __shfl_sync(0xffffffffu, t0, (bk - base) & 31), vk = __shfl_sync(0xffffffffu, v, (bk - base) & 31);
      if (lane < nrow && bk >= base && bk < base + 32 && vk > 0) {
        const int x0 = tk / chunk, x1 = (tk + vk - 1) / chunk;
        aux->first[lane] = x0 + bk;
        aux->count[lane] = min(x1 - x0 + 1, kMaxRuns);
      }
      run += __shfl_sync(0xffffffffu, inc, 31);
    }
    __syncwarp();
    if (lane < nrow) {
      const int bs = (m0 + lane) / p.g;
      aux->row[lane] = (bs % p.n_tok) * p.Hq + h * p.g + (m0 + lane) % p.g;
      aux->orow[lane] = (long long)(bs / p.n_tok) * p.n_tok * p.Hq + aux->row[lane];
    }
  }
  pdl_wait();
  if (warp == 1) {            // (after the wait, see k_shared_decode)
    ptx::tmem_alloc(&aux->tmem_base, 64);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  pdl_trigger();
  const uint32_t tmem = aux->tmem_base;
  const size_t srow = (size_t)p.HB * p.NR;               // rows per slot
  for (int k = warp; k < nrow; k += kOutThreads / 32) {  // weights: a warp per row
    const int n = aux->count[k];
    const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + (size_t)aux->first[k] * srow + aux->row[k];
    float m = -INFINITY;
    for (int s = lane; s < n; s += 32) {
      const float2 v = ml[s * srow];
      if (v.y > 0.f || !(v.y == v.y)) m = fmaxf(m, v.x);  // a part that saw no token has no say
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float l = 0.f;
    for (int s = lane; s < n; s += 32) {
      const float2 v = ml[s * srow];
      const float w = v.y == 0.f ? 0.f : exp2f(v.x - m);
      aux->w[k][s] = w;
      l += w * v.y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) {
      aux->inv[k] = l == 0.f ? 0.f : 1.f / l;
      if (p.lse) p.lse[aux->orow[k]] = l == 0.f ? -INFINITY : (m + log2f(l)) * LR_LN2;
    }
  }
  __syncthreads();
  // A part of r/4 threads (4 ranks each) sums a row's slots; with fewer rows than parts, several
  // parts share a row, each with every sub-th slot.  The rows of o_s past nrow stay as they are:
  // they only reach accumulator columns that nobody reads.
  const int r4 = p.r >> 2, parts = kOutThreads / r4;
  const int part = (int)threadIdx.x / r4, e = ((int)threadIdx.x % r4) * 4;
  const int subs = max(1, parts / nrow);
  auto put = [&](int k, float4 acc) {                    // a row's sum, divided, as hi and lo
    const float inv = aux->inv[k];
    acc.x *= inv;
    acc.y *= inv;
    acc.z *= inv;
    acc.w *= inv;
    const __nv_bfloat162 h0 = __floats2bfloat162_rn(acc.x, acc.y), h1 = __floats2bfloat162_rn(acc.z, acc.w);
    const __nv_bfloat162 l0 = __floats2bfloat162_rn(acc.x - __low2float(h0), acc.y - __high2float(h0));
    const __nv_bfloat162 l1 = __floats2bfloat162_rn(acc.z - __low2float(h1), acc.w - __high2float(h1));
    // K-major, 128-byte swizzle: row k (hi) and half + k (lo; half % 8 = 0, the same swizzle)
    uint8_t* d = o_s + (e >> 6) * oblk + k * 128 + ((((e & 63) >> 3) ^ (k & 7)) << 4) + (e & 4) * 2;
    *reinterpret_cast<uint2*>(d) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1));
    *reinterpret_cast<uint2*>(d + half * 128) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&l0), *reinterpret_cast<const uint32_t*>(&l1));
  };
  auto add = [](float4& acc, float f, const float4& v) {
    acc.x += f * v.x;
    acc.y += f * v.y;
    acc.z += f * v.z;
    acc.w += f * v.w;
  };
  const size_t step = srow * p.r;
  auto src_of = [&](int k) { return p.part_o + ((size_t)aux->first[k] * srow + aux->row[k]) * p.r + e; };
  if (nrow <= parts) {
    const int k = part % nrow, sub = part / nrow;
    const bool in = part < parts && sub < subs;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (in) {
      const int n = aux->count[k];
      const float* src = src_of(k);
      for (int s = sub; s < n; s += 8 * subs) {
        float4 v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (s + q * subs < n) v[q] = *reinterpret_cast<const float4*>(src + (s + q * subs) * step);
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (s + q * subs < n) add(acc, aux->w[k][s + q * subs], v[q]);
      }
    }
    if (subs > 1) {
      aux->part[threadIdx.x] = acc;
      __syncthreads();
    }
    if (in && sub == 0) {
      for (int q = 1; q < subs; ++q) add(acc, 1.f, aux->part[threadIdx.x + q * nrow * r4]);
      put(k, acc);
    }
  } else if (part < parts) {
    // four rows at a time, two slots of each: eight loads in flight, as many rows have few slots
    for (int k0 = part; k0 < nrow; k0 += 4 * parts) {
      float4 acc[4];
      int n[4], most = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
        n[q] = k0 + q * parts < nrow ? aux->count[k0 + q * parts] : 0;
        most = max(most, n[q]);
      }
      for (int s = 0; s < most; s += 2) {
        float4 v[4][2];
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int u = 0; u < 2; ++u)
            if (s + u < n[q]) v[q][u] = *reinterpret_cast<const float4*>(src_of(k0 + q * parts) + (s + u) * step);
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int u = 0; u < 2; ++u)
            if (s + u < n[q]) add(acc[q], aux->w[k0 + q * parts][s + u], v[q][u]);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (k0 + q * parts < nrow) put(k0 + q * parts, acc[q]);
    }
  }
  ptx::fence_proxy_async_smem();
  __syncthreads();
  if (warp == 0) {
    const bool ok = __all_sync(
        0xffffffffu, tc::wait_b(&aux->w_full, 0, &aux->abort_flag, p.err, tc::wait_limit(p.wait_ns)));
    if (ok) {
      ptx::tc_fence_after();
      const uint32_t id = ptx::idesc_f16(1, 1, 0, 128, 2 * half);   // A MN-major, B K-major
      const uint64_t wd = ptx::smem_desc(ptx::smem_u32(w_s), (uint32_t)p.r * 128, 1024, 2);
      const uint64_t od = ptx::smem_desc(ptx::smem_u32(o_s), 16, 1024, 2);
      const uint32_t d = uniform(tmem), idu = uniform(id);
      for (int k = 0; k < nsub; ++k) {
        const uint64_t a = wd + uniform((uint32_t)(k * 64 * 128) >> 4), b = od + uniform((uint32_t)(k * oblk) >> 4);
        const uint32_t more = uniform(k ? 1u : 0u);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          ptx::mma_f16_elect(d, a + (uint64_t)(kk * 16 * 128 >> 4), b + (uint64_t)(kk * 2), idu, kk ? 1u : more);
      }
    }
    ptx::mma_commit_elect(&aux->done);
    drain_wait(&aux->w_full, 0);
    drain_wait(&aux->done, 0);
    __syncwarp();
  }
  __syncthreads();
  ptx::tc_fence_after();
  if (warp < 4 && !aux->abort_flag) {
    const int d = warp * 32 + lane;
    for (int k0 = 0; k0 < half; k0 += 16) {
      uint32_t hi[16], lo[16];
      ptx::tmem_ld16(tmem + ((uint32_t)(warp * 32) << 16) + k0, hi);
      ptx::tmem_ld16(tmem + ((uint32_t)(warp * 32) << 16) + half + k0, lo);
      ptx::tmem_wait_ld();
      if (d < p.dv) {
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (k0 + k < nrow) {
            p.out[aux->orow[k0 + k] * p.dv + d] = __float2bfloat16_rn(__uint_as_float(hi[k]) + __uint_as_float(lo[k]));
          }
      }
      __syncwarp();
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 64);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// How R query rows per sequence are cut: NR per block (16 when a sequence has no more, else 32),
// HB blocks, X runs of tiles.  (64 rows a block leave room for one tile only at r = 512.)
struct Cut {
  int NR, HB, X;
};
Cut cut_of(const lr_shared_desc& d, int n_tokens, int num_sms) {
  const int R = n_tokens * d.n_q_heads;
  Cut c;
  c.NR = R <= 16 ? 16 : 32;
  c.HB = (R + c.NR - 1) / c.NR;
  c.X = std::max(1, std::min(num_sms, kMaxRuns) / c.HB);
  return c;
}

size_t decode_smem(int r, int NR, int nslot) {
  return kAuxBytes + (size_t)(r / 64) * 2 * NR * 128 + (size_t)NR * 128 + 2 * kTok * NR * 2 +
         (size_t)nslot * dec_slot(r);
}

bool map2d(CUtensorMap* m, CUtensorMapDataType type, const void* ptr, uint64_t d0, uint64_t d1, uint64_t stride,
           uint32_t b0, uint32_t b1) {
  const cuuint64_t dims[2] = {d0, d1}, st[1] = {stride};
  const cuuint32_t box[2] = {b0, b1};
  return tc::make_map(m, type, ptr, 2, dims, st, box);
}

template <int NR, bool kQuant>
cudaError_t launch_dec(const lr_shared* c, const CUtensorMap& tqr, const DecArgs& a, size_t smem, cudaStream_t s) {
  static std::atomic<uint32_t> optin{0};
  cudaError_t e = smem_optin(k_shared_decode<NR, kQuant>, optin);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_shared_decode<NR, kQuant>, dim3(a.X, a.HB), dim3(dec_threads<NR, kQuant>()), smem, s,
                    c->tm_qt[NR / 32], tqr, c->tm_c64, c->tm_kr, a);
}

}  // namespace

size_t shared_qt_bytes(const lr_shared_desc* d) {
  size_t most = 0;
  for (int n = 1; n <= d->max_queries; ++n) {
    const Cut c = cut_of(*d, n, 148);
    most = std::max(most, (size_t)c.HB * 2 * c.NR);
  }
  return most * d->batch * d->rank * 2;
}

void shared_part_rows(const lr_shared_desc* d, int num_sms, size_t* rows) {
  *rows = 0;
  for (int n = 1; n <= d->max_queries; ++n) {
    const Cut c = cut_of(*d, n, num_sms);
    *rows = std::max(*rows, (size_t)(c.X + d->batch) * c.HB * c.NR);
  }
}

cudaError_t shared_decode_maps(lr_shared* c) {
  const lr_shared_desc& d = c->desc;
  const CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const uint64_t r = d.rank, rows = (uint64_t)c->n_pages * 128;
  const uint64_t wk = (uint64_t)d.n_kv_heads * d.dim_nope, wv = (uint64_t)d.n_kv_heads * d.dim_v;
  const uint64_t qrows = shared_qt_bytes(&d) / (r * 2);
  bool ok = map2d(&c->tm_w, bf, c->B, wk, r, (wk + wv) * 2, 64, 128) &&
            map2d(&c->tm_v, bf, static_cast<const __nv_bfloat16*>(c->B) + wk, wv, r, (wk + wv) * 2, 64, 64) &&
            map2d(&c->tm_kr, bf, c->kr, d.dim_rope, rows, (uint64_t)d.dim_rope * 2, 64, kTok) &&
            map2d(&c->tm_qt[0], bf, c->qt, r, qrows, r * 2, 64, 32) &&
            map2d(&c->tm_qt[1], bf, c->qt, r, qrows, r * 2, 64, 64);
  // (8 bits: the codes are copied without a map; any valid one stands in)
  if (ok && d.quant_bits) c->tm_c = c->tm_c64 = c->tm_kr;
  else if (ok)
    ok = map2d(&c->tm_c, bf, c->c, r, rows, r * 2, 64, 128) && map2d(&c->tm_c64, bf, c->c, r, rows, r * 2, 64, kTok);
  return ok ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t launch_shared_decode(lr_shared* c, const void* q, int n_tokens, const int32_t* row_len, void* out,
                                 float* lse, cudaStream_t s) {
  const lr_shared_desc& d = c->desc;
  const Cut cut = cut_of(d, n_tokens, c->num_sms);
  const int R = n_tokens * d.n_q_heads, NR = cut.NR, HB = cut.HB, X = cut.X;
  const int g = d.n_q_heads / d.n_kv_heads, r = d.rank, dq = d.dim_nope + d.dim_rope;
  const int BS = d.batch * n_tokens;
  const bool quant = d.quant_bits != 0;
  const CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;

  // query projection
  QpArgs qp;
  qp.wait_ns = c->wait_ns;
  qp.r = r;
  qp.dn = d.dim_nope;
  qp.g = g;
  qp.nb = std::max(1, std::min(BS, 32 / g));
  qp.BS = BS;
  qp.n_tok = n_tokens;
  qp.Hq = d.n_q_heads;
  qp.HB = HB;
  qp.NR = NR;
  qp.ncols = (qp.nb * g + 15) / 16 * 16;
  qp.tcols = qp.ncols <= 32 ? 32 : (qp.ncols <= 64 ? 64 : 128);
  qp.qt = static_cast<__nv_bfloat16*>(c->qt);
  qp.err = c->dev_err;
  CUtensorMap tq, tqr;
  {
    const cuuint64_t dims[3] = {(cuuint64_t)dq, (cuuint64_t)d.n_q_heads, (cuuint64_t)BS};
    const cuuint64_t st[2] = {(cuuint64_t)dq * 2, (cuuint64_t)d.n_q_heads * dq * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)g, (cuuint32_t)qp.nb};
    if (!tc::make_map(&tq, bf, q, 3, dims, st, box)) return cudaErrorInvalidValue;
  }
  static std::atomic<uint32_t> optin_q{0}, optin_o{0};
  cudaError_t e = smem_optin(k_shared_qproj, optin_q);
  if (e != cudaSuccess) return e;
  const size_t smem_q = (size_t)(d.dim_nope / 64) * (kWSub + qp.ncols * 128) + sizeof(QpAux);
  e = launch_pdl(k_shared_qproj, dim3((r + 127) / 128, d.n_kv_heads, (BS + qp.nb - 1) / qp.nb), dim3(128), smem_q, s,
                 c->tm_w, tq, qp);
  if (e != cudaSuccess) return e;

  // attention over the stored rows
  {
    const cuuint64_t dims[3] = {(cuuint64_t)d.dim_rope, (cuuint64_t)R, (cuuint64_t)d.batch};
    const cuuint64_t st[2] = {(cuuint64_t)dq * 2, (cuuint64_t)R * dq * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)NR, 1};
    if (!tc::make_map(&tqr, bf, static_cast<const __nv_bfloat16*>(q) + d.dim_nope, 3, dims, st, box))
      return cudaErrorInvalidValue;
  }
  DecArgs a;
  a.wait_ns = c->wait_ns;
  a.row_len = row_len;
  a.map = row_map(c);
  a.B = d.batch;
  a.cap = d.capacity;
  a.r = r;
  a.Hq = d.n_q_heads;
  a.n_tok = n_tokens;
  a.R = R;
  a.HB = HB;
  a.X = X;
  a.scale_log2 = c->scale_log2;
  a.codes = static_cast<const uint8_t*>(c->c);
  a.scale = c->scale;
  a.part_o = c->part_o;
  a.part_ml = c->part_ml;
  a.err = c->dev_err;
  a.nslot = 1;
  while (a.nslot < kMaxSlots && decode_smem(r, NR, a.nslot + 1) <= (size_t)kSmemLimit) ++a.nslot;
  const size_t smem = decode_smem(r, NR, a.nslot);
  if (NR == 16)
    e = quant ? launch_dec<16, true>(c, tqr, a, smem, s) : launch_dec<16, false>(c, tqr, a, smem, s);
  else
    e = quant ? launch_dec<32, true>(c, tqr, a, smem, s) : launch_dec<32, false>(c, tqr, a, smem, s);
  if (e != cudaSuccess) return e;

  // join and output projection
  OutArgs o;
  o.wait_ns = c->wait_ns;
  o.row_len = row_len;
  o.B = d.batch;
  o.cap = d.capacity;
  o.r = r;
  o.dv = d.dim_v;
  o.g = g;
  o.rows = BS * g;
  // the fewest rows a block whose grid still is one wave (each block reads B_v,h once more)
  o.RB = 32;
  while (o.RB > 1 && (o.rows + o.RB / 2 - 1) / (o.RB / 2) * d.n_kv_heads <= c->num_sms) o.RB /= 2;
  o.n_tok = n_tokens;
  o.Hq = d.n_q_heads;
  o.HB = HB;
  o.NR = NR;
  o.X = X;
  o.part_o = c->part_o;
  o.part_ml = c->part_ml;
  o.out = static_cast<__nv_bfloat16*>(out);
  o.lse = lse;
  o.err = c->dev_err;
  e = smem_optin(k_shared_out, optin_o);
  if (e != cudaSuccess) return e;
  const size_t smem_o = (size_t)(r / 64) * (o.RB <= 16 ? 4096 : 8192) + (size_t)2 * r * 128 + sizeof(OutAux);
  return launch_pdl(k_shared_out, dim3((o.rows + o.RB - 1) / o.RB, d.n_kv_heads), dim3(kOutThreads), smem_o, s, c->tm_v,
                    o);
}
