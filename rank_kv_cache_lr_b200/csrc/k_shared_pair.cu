// Absorbed decode over a shared-latent cache with r > 256, by pairs of CTAs that split the rank.
//
// The mathematics, roundings and runs are k_shared_decode's.  There a tile's latents (128 KB at
// r = 512) and the query latents (64 KB) fill an SM, so a tile's copies can only start as its
// predecessor's value mix ends: load, scores, softmax and value mix follow one another (4.1 us a
// tile of bf16, 6.2 us of 8 bits).  Here CTA 0 of a cluster of two holds ranks 0..255 and CTA 1
// the others and the rotary part, of the tiles and of q~ alike: half the bytes each, so two tiles
// fit (blocks of 16 and 32 query rows; 64 rows: one tile and a half) and the copies of tile i + 1
// run under the work on tile i.  Per tile the CTAs exchange, through distributed shared memory:
//   S: each has a partial sum over its ranks for all NR rows, finishes NR/2 of them, and gets the
//      other's partial sums for those (fp32, 128 x NR/2);
//   P: the weights of its rows, which the other's value mix needs too (bf16, 128 x NR/2);
//   alpha: the factors by which its rows' running maxima moved, for the other's accumulators.
// The value mix needs no exchange: each CTA owns its ranks of o~.
#include "shared_decode.cuh"

#include <algorithm>

namespace {

// Barriers (arrival count; who arrives -> who waits); phase k is waited with parity k & 1; GO =
// NR / 16 groups of 8 own rows, four warps each.
//   raw_full, slot_full, slot_empty, rope_full, rope_empty, q_full, q_empty, s_full[2]
//                   as in k_shared_decode.cu
//   s_empty[2] 4 GO  softmax warps (own and other's columns read) -> MMA issuer
//   x_full     1 + tx   the OTHER CTA's partial scores, stored here -> softmax warps
//   r_full     1 + tx   the OTHER CTA's P and alpha, stored here -> softmax warps
//                    (both armed one tile ahead; the other stores those of tile i + 1 only after
//                    every warp here is past the phase of tile i)
//   p_full     4 GO  softmax warps (own P written, the other's seen) -> MMA issuer
//   p_empty    2     MMA commits of GEMM2 in BOTH CTAs -> softmax warps (P may be rewritten in
//                    both, O~ rescaled)
//   o_full 1, o_empty 4 GO, done 1
struct PAux {
  uint64_t raw_full[kMaxSlots], slot_full[kMaxSlots], slot_empty[kMaxSlots];
  uint64_t rope_full, rope_empty, q_full, q_empty, s_full[2], s_empty[2], x_full, r_full, p_full, p_empty, o_full,
      o_empty, done;
  uint32_t tmem_base;
  int abort_flag;
  unsigned long long wait_ns;
  TileRun run;
  float red[4][4][8];          // [own group][lane quarter][row]
  alignas(16) float alpha_r[4][8];   // the other CTA's factors of this tile (written 16 bytes at a time)
  int off_s[64];               // row j sees tokens t < len + off_s[j]
};
static_assert(sizeof(PAux) <= kAuxBytes, "aux block");

__device__ __forceinline__ bool wait_b(uint64_t* bar, uint32_t parity, PAux* aux, int* err) {
  return tc::wait_b(bar, parity, &aux->abort_flag, err, aux->wait_ns);
}
__device__ __forceinline__ bool wait_w(uint64_t* bar, uint32_t parity, PAux* aux, int* err) {
  return __all_sync(0xffffffffu, wait_b(bar, parity, aux, err));
}
__device__ __forceinline__ bool wait_x(uint64_t* bar, uint32_t parity, PAux* aux, int* err) {
  return __all_sync(0xffffffffu, tc::wait_cluster(bar, parity, &aux->abort_flag, err, aux->wait_ns));
}

// Whether a phase is complete, for a whole warp.
__device__ __forceinline__ bool ready(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, ptx::mbar_test_wait(bar, parity));
}

constexpr int kOColP = 256;            // TMEM: S of tile t in columns [2 NR (t % 2), + 2 NR), O~ from 256

template <int NR, bool kQuant>
constexpr int pair_threads() {
  return 64 + NR * 8 + (kQuant ? 256 : 0);
}
template <int NR>
__host__ __device__ constexpr int pair_head_bytes() {   // q~ (256 ranks), rotary query, P, partial scores
  return (4 * 2 * NR * 128 + NR * 128 + 128 * NR * 2 + 128 * (NR / 2) * 4 + 1023) / 1024 * 1024;
}

// Shared memory: [aux][q~: 4 blocks of (2 NR rows hi | lo) x 128 B][q_rope: NR rows x 128 B]
// [P: 128 tokens x NR][recv: the other's partial scores, NR/16 groups of 2 x 128 x 16 B]
// [slots][rotary tile][8 bits: scales per slot].  Both CTAs have the same layout.
// Warps: 0 TMA producer, 1 MMA issuer, NR / 4 softmax warps (thread = token row of 8 own query
// rows, and carrier of 8 of the other's), (8 bits) 8 expansion warps.
template <int NR, bool kQuant>
__global__ void __launch_bounds__(pair_threads<NR, kQuant>(), 1)
    k_shared_pair(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_qr,
                  const __grid_constant__ CUtensorMap tm_c, const __grid_constant__ CUtensorMap tm_kr,
                  const DecArgs p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (ptx::smem_u32(smem_raw) & 1023) {      // layout precondition; uniform for the whole grid
    if (threadIdx.x == 0) atomicExch(p.err, (int)LR_ERR_UNSUPPORTED);
    return;
  }
  constexpr int GO = NR / 16, kQSub = 2 * NR * 128, kPBytes = 128 * NR * 2;
  constexpr uint32_t kXBytes = GO * 4096, kRBytes = GO * (2048 + 32);   // received per tile
  PAux* aux = reinterpret_cast<PAux*>(smem_raw);
  uint8_t* q_s = smem_raw + kAuxBytes;
  uint8_t* qr_s = q_s + 4 * kQSub;
  uint8_t* p_s = qr_s + NR * 128;
  uint8_t* recv = p_s + kPBytes;
  uint8_t* ring = smem_raw + kAuxBytes + pair_head_bytes<NR>();
  uint8_t* rope_s = ring + p.nslot * kSlot;
  uint8_t* sc_s = rope_s + kSub;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t cr = ptx::cluster_rank();
  const int x = blockIdx.x >> 1, hb = blockIdx.y;
  const int c_lo = cr ? 2 : 0, nloc = cr ? p.nch - 2 : 2;            // this CTA's 128-rank chunks
  const int r_loc = cr ? p.r - 256 : 256;                           // and ranks

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.nslot; ++s) {
      ptx::mbar_init(&aux->raw_full[s], 1);
      ptx::mbar_init(&aux->slot_full[s], kQuant ? 8 : 1);
      ptx::mbar_init(&aux->slot_empty[s], 1);
    }
    ptx::mbar_init(&aux->rope_full, 1);
    ptx::mbar_init(&aux->rope_empty, 1);
    ptx::mbar_init(&aux->q_full, 1);
    ptx::mbar_init(&aux->q_empty, 1);
    for (int k = 0; k < 2; ++k) {
      ptx::mbar_init(&aux->s_full[k], 1);
      ptx::mbar_init(&aux->s_empty[k], 4 * GO);
    }
    ptx::mbar_init(&aux->x_full, 1);
    ptx::mbar_init(&aux->r_full, 1);
    ptx::mbar_init(&aux->p_full, 4 * GO);
    ptx::mbar_init(&aux->p_empty, 2);
    ptx::mbar_init(&aux->o_full, 1);
    ptx::mbar_init(&aux->o_empty, 4 * GO);
    ptx::mbar_init(&aux->done, 1);
    aux->abort_flag = 0;
    aux->wait_ns = tc::wait_limit(p.wait_ns);
    ptx::fence_mbar_init();
    ptx::mbar_arrive_expect_tx(&aux->x_full, kXBytes);
    ptx::mbar_arrive_expect_tx(&aux->r_full, kRBytes);
  }
  if (threadIdx.x >= 64 && threadIdx.x < 128) {   // query row j of this block belongs to token (hb NR + j) / Hq
    const int j = threadIdx.x - 64;
    aux->off_s[j] = min((hb * NR + j) / p.Hq, p.n_tok - 1) - (p.n_tok - 1);
  }
  if (warp == 0 && lane == 0) {
    ptx::prefetch_tmap(&tm_q);
    ptx::prefetch_tmap(&tm_qr);
    ptx::prefetch_tmap(&tm_c);
    ptx::prefetch_tmap(&tm_kr);
  }
  if (warp == 1) {
    ptx::tmem_alloc(&aux->tmem_base, 512);
    ptx::tmem_relinquish();
  }
  pdl_wait();       // lengths, pages, rows and q~ may come from the work just before
  pdl_trigger();
  if (warp == 0) {
    int chunk;
    const TileRun run =
        tile_run([&](int b) { return (shared_len(p.row_len, b, p.cap) + 127) >> 7; }, p.B, p.X, x, &chunk);
    if (lane == 0) aux->run = run;
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();      // both CTAs' barriers are ready before any remote arrival
  ptx::tc_fence_after();
  const uint32_t tmem = aux->tmem_base;
  TileRun run = aux->run;
  Seg sg;
  int ntiles = 0;           // (MMA warp) tiles done

  if (warp == 0) {
    // ------------------------------------------------------------- TMA producer
    if (lane == 0) {
      const int nsub = r_loc >> 6;
      int gt = 0, pos = 0, nseg = 0;     // tiles, slot uses and sequences issued
      bool ok = true;
      while (ok && next_seg(&run, p, &sg)) {
        if (nseg > 0 && !(ok = wait_b(&aux->q_empty, (nseg - 1) & 1, aux, p.err))) break;
        ptx::mbar_arrive_expect_tx(&aux->q_full, (uint32_t)(nsub * kQSub + (cr ? NR * 128 : 0)));
        for (int s = 0; s < nsub; ++s)
          ptx::tma_load_2d(q_s + s * kQSub, &tm_q, &aux->q_full, (c_lo * 2 + s) * 64, (sg.b * p.HB + hb) * 2 * NR);
        if (cr) ptx::tma_load_3d(qr_s, &tm_qr, &aux->q_full, 0, hb * NR, sg.b);
        ++nseg;
        int next_page = p.map.page(sg.b, sg.t0 * 128);
        for (int i = 0; i < sg.nt && ok; ++i) {
          const int page = next_page;
          if (i + 1 < sg.nt) next_page = p.map.page(sg.b, (sg.t0 + i + 1) * 128);
          for (int lc = 0; lc < nloc; ++lc) {
            const int c = c_lo + lc, slot = pos % p.nslot, round = pos / p.nslot;
            if (round > 0 && !(ok = wait_b(&aux->slot_empty[slot], (round - 1) & 1, aux, p.err))) break;
            uint8_t* dst = ring + slot * kSlot;
            const bool full = c * 128 + 64 < p.r;
            if (kQuant) {
              const uint32_t bytes = full ? kSub : kSub / 2;
              ptx::mbar_arrive_expect_tx(&aux->raw_full[slot], bytes + kScaleBytes);
              ptx::bulk_load(dst + kSub, p.codes + (long long)page * 128 * p.r + c * kSub, bytes, &aux->raw_full[slot]);
              ptx::bulk_load(sc_s + slot * kScaleBytes, p.scale + ((long long)page * p.nch + c) * kScaleBytes,
                             kScaleBytes, &aux->raw_full[slot]);
            } else {
              const int nb = full ? 2 : 1;
              ptx::mbar_arrive_expect_tx(&aux->slot_full[slot], nb * kSub);
              for (int s = 0; s < nb; ++s)
                ptx::tma_load_2d(dst + s * kSub, &tm_c, &aux->slot_full[slot], c * 128 + s * 64, page * 128);
            }
            ++pos;
          }
          if (!ok) break;
          if (cr) {
            if (gt > 0 && !(ok = wait_b(&aux->rope_empty, (gt - 1) & 1, aux, p.err))) break;
            ptx::mbar_arrive_expect_tx(&aux->rope_full, kSub);
            ptx::tma_load_2d(rope_s, &tm_kr, &aux->rope_full, 0, page * 128);
            ++gt;
          }
        }
      }
      // every copy this thread issued has landed before the CTA can exit
      if (nseg > 0) drain_wait(&aux->q_full, (nseg - 1) & 1);
      for (int k = max(0, pos - p.nslot); k < pos; ++k)
        drain_wait(kQuant ? &aux->raw_full[k % p.nslot] : &aux->slot_full[k % p.nslot], (k / p.nslot) & 1);
      if (gt > 0) drain_wait(&aux->rope_full, (gt - 1) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------- MMA issuer (warp-wide)
    const uint32_t id1 = ptx::idesc_f16(1, 0, 0, 128, 2 * NR);   // GEMM1: K-major x K-major (hi | lo)
    const uint32_t idr = ptx::idesc_f16(1, 0, 0, 128, NR);       //        rotary part, into the hi columns
    const uint32_t id2 = ptx::idesc_f16(1, 1, 1, 128, NR);       // GEMM2: MN-major x MN-major
    const uint64_t kd0 = ptx::smem_desc(ptx::smem_u32(ring), 16, 1024, 2);
    const uint64_t vd0 = ptx::smem_desc(ptx::smem_u32(ring), kSub, 1024, 2);
    const uint64_t qd0 = ptx::smem_desc(ptx::smem_u32(q_s), 16, 1024, 2);
    const uint64_t rd0 = ptx::smem_desc(ptx::smem_u32(rope_s), 16, 1024, 2);
    const uint64_t qrd0 = ptx::smem_desc(ptx::smem_u32(qr_s), 16, 1024, 2);
    const uint64_t pd0 = ptx::smem_desc(ptx::smem_u32(p_s), 128, 2048, 0);
    int nseg = 0;
    bool ok = true;
    const uint64_t t_limit = aux->wait_ns;
    while (ok && next_seg(&run, p, &sg)) {
      if (!(ok = wait_w(&aux->q_full, nseg & 1, aux, p.err))) break;
      ptx::tc_fence_after();
      // Whatever is ready goes next: the value mix of tile vi (it frees slots) before the next
      // chunk kc of the scores of tile ki (chunk nloc: the rotary part).
      int ki = 0, kc = 0, vi = 0;
      uint64_t t0 = 0;                     // since when nothing was ready
      while (vi < sg.nt) {
        bool moved = false;
        if (vi < ki && ready(&aux->p_full, (ntiles + vi) & 1) &&
            (vi > 0 || nseg == 0 || ready(&aux->o_empty, (nseg - 1) & 1))) {
          const int gt = ntiles + vi;
          ptx::tc_fence_after();
          const uint32_t first = uniform(vi ? 1u : 0u);
          for (int lc = 0; lc < nloc; ++lc) {
            const int slot = (gt * nloc + lc) % p.nslot;
            const uint64_t a0 = vd0 + uniform((slot * kSlot) >> 4);
            const uint32_t d_o = uniform(tmem + kOColP + lc * NR);
#pragma unroll
            for (int kt = 0; kt < 8; ++kt)
              ptx::mma_f16_elect(d_o, a0 + (uint64_t)(kt * 128), pd0 + (uint64_t)(kt * 16), id2, kt ? 1u : first);
            ptx::mma_commit_elect(&aux->slot_empty[slot]);
          }
          ptx::mma_commit_mask_elect(&aux->p_empty, 3);
          if (vi == sg.nt - 1) ptx::mma_commit_elect(&aux->o_full);
          ++vi;
          moved = true;
        }
        if (ki < sg.nt) {
          const int gt = ntiles + ki, sb = gt & 1;
          const uint32_t d_s = uniform(tmem + 2 * NR * sb);
          if (kc < nloc) {
            const int pos = gt * nloc + kc, slot = pos % p.nslot;
            if ((kc > 0 || gt < 2 || ready(&aux->s_empty[sb], ((gt - 2) >> 1) & 1)) &&
                ready(&aux->slot_full[slot], (pos / p.nslot) & 1)) {
              ptx::tc_fence_after();
              const uint64_t a0 = kd0 + uniform((slot * kSlot) >> 4);
              const uint64_t b0 = qd0 + uniform((kc * 2 * kQSub) >> 4);
              const uint32_t first = uniform(kc ? 1u : 0u);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                ptx::mma_f16_elect(d_s, a0 + (uint64_t)(kk * 2), b0 + (uint64_t)(kk * 2), id1, kk ? 1u : first);
              if (kc * 128 + 64 < r_loc) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  ptx::mma_f16_elect(d_s, a0 + (uint64_t)((kSub >> 4) + kk * 2),
                                     b0 + (uint64_t)((kQSub >> 4) + kk * 2), id1, 1u);
              }
              ++kc;
              moved = true;
            }
          }
          if (kc == nloc && (!cr || ready(&aux->rope_full, gt & 1))) {
            if (cr) {
              ptx::tc_fence_after();
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)       // columns past dim_rope are 0 on both sides
                ptx::mma_f16_elect(d_s, rd0 + (uint64_t)(kk * 2), qrd0 + (uint64_t)(kk * 2), idr, 1u);
              ptx::mma_commit_elect(&aux->rope_empty);
            }
            if (ki == sg.nt - 1) ptx::mma_commit_elect(&aux->q_empty);
            ptx::mma_commit_elect(&aux->s_full[sb]);
            ++ki;
            kc = 0;
            moved = true;
          }
        }
        if (moved) {
          t0 = 0;
        } else {
          const uint64_t now = ptx::globaltimer();
          if (t0 == 0) t0 = now;
          const bool late = now - t0 > t_limit;
          if (__any_sync(0xffffffffu, late || *(volatile int*)&aux->abort_flag)) {
            if (late) {
              *(volatile int*)&aux->abort_flag = 1;
              atomicExch(p.err, (int)LR_ERR_TIMEOUT);
            }
            ok = false;
            break;
          }
        }
      }
      if (!ok) break;
      ntiles += sg.nt;
      ++nseg;
    }
    ptx::mma_commit_elect(&aux->done);
    drain_wait(&aux->done, 0);
    // the other CTA's last arrival here has come, so none is under way when this CTA exits (after
    // an abort it may never come)
    if (ok && ntiles > 0) drain_wait(&aux->p_empty, (ntiles - 1) & 1);
    __syncwarp();
  } else if (warp < 2 + NR / 4) {
    // ------------------------------------------------------------- softmax / epilogue
    const int qd = warp & 3, g = (warp - 2) >> 2;        // lane quarter, own group
    const int G = (int)cr * GO + g, Gx = (int)(1 - cr) * GO + g;   // its 8 query rows, and the other's carried here
    const int row = qd * 32 + lane;
    const uint32_t lane_off = (uint32_t)(qd * 32) << 16;
    const int bar = 1 + g;                               // the group's four warps
    const uint32_t peer = 1 - cr;
    const uint32_t recv_x = ptx::map_rank(ptx::smem_u32(recv + g * 4096 + row * 16), peer);
    const uint32_t p_x = ptx::map_rank(ptx::smem_u32(p_s + G * 2048 + row * 16), peer);
    const uint32_t alpha_x = ptx::map_rank(ptx::smem_u32(&aux->alpha_r[g][0]), peer);
    const uint32_t x_full_x = ptx::map_rank(ptx::smem_u32(&aux->x_full), peer);
    const uint32_t r_full_x = ptx::map_rank(ptx::smem_u32(&aux->r_full), peer);
    int gt = 0, nseg = 0;
    bool ok = true;
    // rescale 8 columns of every chunk of O~
    auto rescale = [&](int cols, const float (&a)[8]) {
      for (int lc = 0; lc < nloc; ++lc) {
        uint32_t v[8];
        const uint32_t col = tmem + lane_off + kOColP + lc * NR + cols;
        ptx::tmem_ld8(col, v);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * a[j]);
        ptx::tmem_st8(col, v);
      }
      ptx::tmem_wait_st();
    };
    while (ok && next_seg(&run, p, &sg)) {
      float m[8], l[8];                                  // in units of log2; alike in the whole group
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        m[j] = kNoMax;
        l[j] = 0.f;
      }
      for (int i = 0; i < sg.nt; ++i, ++gt) {
        const int k2 = gt & 1;
        const int t = (sg.t0 + i) * 128 + row;
        const uint32_t s_col = tmem + lane_off + 2 * NR * k2;
        // after an abort every wait returns at once: the warps finish the sequence in step (their
        // barriers stay matched) and leave at the verdict below
        (void)wait_w(&aux->s_full[k2], (gt >> 1) & 1, aux, p.err);
        ptx::tc_fence_after();
        float s[8];
        {
          // the partial sums of the other's rows go to it
          uint32_t a[8], b[8];
          ptx::tmem_ld8(s_col + 8 * Gx, a);
          ptx::tmem_ld8(s_col + NR + 8 * Gx, b);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 8; ++j) a[j] = __float_as_uint(__uint_as_float(a[j]) + __uint_as_float(b[j]));
          ptx::st_async_v4(recv_x, x_full_x, a[0], a[1], a[2], a[3]);
          ptx::st_async_v4(recv_x + 2048, x_full_x, a[4], a[5], a[6], a[7]);
          ptx::tmem_ld8(s_col + 8 * G, a);
          ptx::tmem_ld8(s_col + NR + 8 * G, b);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 8; ++j) s[j] = __uint_as_float(a[j]) + __uint_as_float(b[j]);
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&aux->s_empty[k2]);
        (void)wait_x(&aux->x_full, gt & 1, aux, p.err);
        if (threadIdx.x == 64) ptx::mbar_arrive_expect_tx(&aux->x_full, kXBytes);
        {
          const float4 u = *reinterpret_cast<const float4*>(recv + g * 4096 + row * 16);
          const float4 v = *reinterpret_cast<const float4*>(recv + g * 4096 + 2048 + row * 16);
          const float got[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 8; ++j) s[j] = (s[j] + got[j]) * p.scale_log2;
        }
        // a tile every row sees whole needs no masks; otherwise row j sees t < len + off_s[j]
        if ((sg.t0 + i) * 128 + 128 > sg.len - (p.n_tok - 1)) {
#pragma unroll
          for (int j = 0; j < 8; ++j) s[j] = t < sg.len + aux->off_s[8 * G + j] ? s[j] : -INFINITY;
        }
        bool ex = false;
#pragma unroll
        for (int j = 0; j < 8; ++j) ex |= s[j] > m[j] + kLazy;
        ex = ptx::named_bar_or(bar, 128, ex);
        if (gt > 0) {   // the value mixes before have completed: P may be rewritten, O~ rescaled
          (void)wait_x(&aux->p_empty, (gt - 1) & 1, aux, p.err);
          ptx::tc_fence_after();
        }
        if (!kQuant && t >= sg.len) {
          // rows behind the sequence hold whatever the page held: 0 weight times a stale
          // infinity would still be NaN, so their values become 0 (the groups share the boxes)
          for (int c = g; c < 2 * nloc; c += GO) {
            const uint32_t base =
                ptx::smem_u32(ring + ((gt * nloc + (c >> 1)) % p.nslot) * kSlot + (c & 1) * kSub + row * 128);
#pragma unroll
            for (int v = 0; v < 8; ++v)
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(base + v * 16), "r"(0) : "memory");
          }
        }
        __syncwarp();
        float a[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] = 1.f;
        if (ex) {
          float top[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) top[j] = s[j];
          const float mt = reduce_cols<true>(top, lane);
          if (lane < 8) aux->red[g][qd][lane] = mt;   // read by all before the next tile's vote
          ptx::named_bar_sync(bar, 128);
          bool need_o = false;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float mn = fmaxf(m[j], fmaxf(fmaxf(aux->red[g][0][j], aux->red[g][1][j]),
                                               fmaxf(aux->red[g][2][j], aux->red[g][3][j])));
            a[j] = ptx::ex2_approx(m[j] - mn);
            m[j] = mn;
            l[j] *= a[j];
            need_o |= a[j] < 1.f;
          }
          if (need_o && i > 0) rescale(8 * G, a);
        }
        uint32_t hw[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float p0 = ptx::ex2_approx(s[2 * e] - m[2 * e]);
          const float p1 = ptx::ex2_approx(s[2 * e + 1] - m[2 * e + 1]);
          const __nv_bfloat162 h = __floats2bfloat162_rn(p0, p1);
          l[2 * e] += p0;
          l[2 * e + 1] += p1;
          hw[e] = *reinterpret_cast<const uint32_t*>(&h);
        }
        ptx::st_async_v4(p_x, r_full_x, hw[0], hw[1], hw[2], hw[3]);
        if (qd == 0 && lane < 2)      // the same in every thread of the group
          ptx::st_async_v4(alpha_x + lane * 16, r_full_x, __float_as_uint(lane ? a[4] : a[0]),
                             __float_as_uint(lane ? a[5] : a[1]), __float_as_uint(lane ? a[6] : a[2]),
                             __float_as_uint(lane ? a[7] : a[3]));
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(ptx::smem_u32(p_s + G * 2048 + row * 16)),
                     "r"(hw[0]), "r"(hw[1]), "r"(hw[2]), "r"(hw[3])
                     : "memory");
        (void)wait_x(&aux->r_full, gt & 1, aux, p.err);
        if (threadIdx.x == 64) ptx::mbar_arrive_expect_tx(&aux->r_full, kRBytes);
        if (i > 0) {
          float b[8];
          bool need = false;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            b[j] = aux->alpha_r[g][j];
            need |= b[j] < 1.f;
          }
          if (__any_sync(0xffffffffu, need)) rescale(8 * Gx, b);
        }
        // own and received weights become visible to the tensor core, then one arrival per warp
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&aux->p_full);
      }
      ok = ptx::named_bar_and(bar, 128, wait_b(&aux->o_full, nseg & 1, aux, p.err));
      if (!ok) break;
      ptx::tc_fence_after();
      const size_t base = ((size_t)(x + sg.b) * p.HB + hb) * NR;
      const float lt = reduce_cols<false>(l, lane);
      if (lane < 8) aux->red[g][qd][lane] = lt;
      ptx::named_bar_sync(bar, 128);
      if (qd == 0 && lane < 8) {
        float mj = m[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) mj = lane == j ? m[j] : mj;
        const float l4 = (aux->red[g][0][lane] + aux->red[g][1][lane]) + (aux->red[g][2][lane] + aux->red[g][3][lane]);
        reinterpret_cast<float2*>(p.part_ml)[base + 8 * G + lane] = make_float2(mj, l4);
      }
      for (int lc = 0; lc < nloc; ++lc) {
        const int e = (c_lo + lc) * 128 + row;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int cols = 8 * (h ? Gx : G);
          uint32_t o[8];
          ptx::tmem_ld8(tmem + lane_off + kOColP + lc * NR + cols, o);
          ptx::tmem_wait_ld();
          if (e < p.r) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (hb * NR + cols + j < p.R) p.part_o[(base + cols + j) * p.r + e] = __uint_as_float(o[j]);
          }
          __syncwarp();
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&aux->o_empty);
      ++nseg;
    }
    __syncwarp();
  } else if (kQuant) {
    // ------------------------------------------------------------- expansion of codes
    const int tid = threadIdx.x - (64 + NR * 8);   // 0..255
    int pos = 0;
    bool ok = true;
    while (ok && next_seg(&run, p, &sg)) {
      for (int i = 0; i < sg.nt && ok; ++i) {
        const int valid = sg.len - (sg.t0 + i) * 128;      // token rows of this tile (may exceed 128)
        for (int lc = 0; lc < nloc; ++lc, ++pos) {
          const int slot = pos % p.nslot;
          if (!(ok = wait_w(&aux->raw_full[slot], (pos / p.nslot) & 1, aux, p.err))) break;
          expand_chunk(ring + slot * kSlot, sc_s + slot * kScaleBytes, tid, lc * 128 + 64 < r_loc, valid);
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&aux->slot_full[slot]);
        }
      }
    }
    __syncwarp();
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
  // neither CTA leaves while the other may still write into it (after an abort, stores that nobody
  // waited for have time to land)
  if (aux->abort_flag) __nanosleep(200000);
  ptx::cluster_sync();
}

template <int NR>
size_t pair_smem(int nslot, bool quant) {
  return (size_t)kAuxBytes + pair_head_bytes<NR>() + (size_t)nslot * kSlot + kSub +
         (quant ? (size_t)nslot * kScaleBytes : 0);
}

template <int NR, bool kQuant>
cudaError_t launch(const lr_shared* c, const CUtensorMap& tqr, DecArgs& a, cudaStream_t s) {
  static std::atomic<uint32_t> optin{0};
  cudaError_t e = smem_optin(k_shared_pair<NR, kQuant>, optin);
  if (e != cudaSuccess) return e;
  a.nslot = 0;
  while (a.nslot < 4 && pair_smem<NR>(a.nslot + 1, kQuant) <= (size_t)kSmemLimit) ++a.nslot;   // two tiles at most
  return launch_pdl_cluster(k_shared_pair<NR, kQuant>, dim3(2 * a.X, a.HB), dim3(pair_threads<NR, kQuant>()), 2,
                            pair_smem<NR>(a.nslot, kQuant), s, c->tm_qt[NR / 32], tqr, c->tm_c, c->tm_kr, a);
}

}  // namespace

cudaError_t launch_shared_pair(const lr_shared* c, const CUtensorMap& tqr, const int32_t* row_len, int n_tokens,
                               int R, int NR, int HB, int X, cudaStream_t s) {
  DecArgs a = dec_args(c, row_len, n_tokens, R, HB, X);
  if (c->desc.quant_bits)
    return NR == 16 ? launch<16, true>(c, tqr, a, s)
                    : (NR == 32 ? launch<32, true>(c, tqr, a, s) : launch<64, true>(c, tqr, a, s));
  return NR == 16 ? launch<16, false>(c, tqr, a, s)
                  : (NR == 32 ? launch<32, false>(c, tqr, a, s) : launch<64, false>(c, tqr, a, s));
}
