// Absorbed decode over a shared-latent cache: a few query tokens per sequence against every
// stored token, without rebuilding keys or values.
//
//   q~_j = B_k,h q_nope,j                              k_shared_qproj   (rank space, per head)
//   s_tj = scale (c_t . q~_j + kr_t . q_rope,j)        k_shared_decode  GEMM1, M = 128 tokens
//   o~_j = sum_t p_tj c_t,  p = softmax over visible t k_shared_decode  GEMM2, M = 128 ranks
//   out_j = o~_j B_v,h / l_j                           k_shared_out     (merges the splits)
//
// One 128-token tile of latents in shared memory serves as keys (rows of GEMM1's A operand,
// K-major) and, through a second descriptor of the same bytes, as values (GEMM2's A operand,
// MN-major): each stored byte crosses HBM once per step.  Heads are the N side of both MMAs, so
// a block of NR = 16 or 32 query rows pays for no empty rows of a 128-row operand.
//
// Roundings: q~ enters GEMM1 as two bf16 halves, hi and lo = q~ - hi, stacked on N (the
// A operand's shared-memory reads set the pace for N <= 64, so the second half is nearly
// free) and added in fp32: the scores, and so lse, carry ~16 bits of q~.  The rotary query is
// bf16 as given.  p enters GEMM2 as one bf16 (2^-8 relative at most, at random over the tokens,
// below the output's own rounding); its sum, for lse and the normaliser, is of the unrounded
// weights in fp32.
//
// Work: the 128-token tiles of all sequences, in order, are cut into equal runs on the device
// (tile_run), one run per CTA column, so ragged batches stay balanced and a captured graph
// serves any lengths.  A run's part of one sequence is one partial (m, l, o~), joined by
// k_shared_out.
#include "shared_decode.cuh"

#include <algorithm>

namespace {

constexpr int kSCol = 0;               // TMEM: S of tile t in columns [64 (t % 2), + 2 NR)
constexpr int kOCol = 128;             // TMEM: O~ of 128-rank chunk c in columns [128 + c NR, + NR)

// Barriers (arrival count; who arrives -> who waits); phase k is waited with parity k & 1.
//   raw_full[s]     1 + tx   8 bits: producer's codes and scales -> expansion warps
//   slot_full[s]    1 + tx / 8   producer's boxes (bf16) or the expansion warps -> MMA issuer
//   slot_empty[s]   1        MMA commit of GEMM2 -> producer
//   rope_full       1 + tx   producer -> MMA issuer
//   rope_empty      1        MMA commit of GEMM1 -> producer
//   q_full/q_empty  1 + tx / 1   per sequence of the run
//   s_full[2]       1        MMA commit of GEMM1 -> softmax warps
//   s_empty[2]      NR / 2   softmax warps (scores read) -> MMA issuer
//   p_full          NR / 2   softmax warps -> MMA issuer
//   p_empty         1        MMA commit of GEMM2 -> softmax warps
//   o_full          1        MMA commit, last tile of a sequence -> softmax warps
//   o_empty         NR / 2   softmax warps (O~ read) -> MMA issuer
//   done            1        final commit: every MMA complete before TMEM is freed
struct Aux {
  uint64_t raw_full[kMaxSlots], slot_full[kMaxSlots], slot_empty[kMaxSlots];
  uint64_t rope_full, rope_empty, q_full, q_empty, s_full[2], s_empty[2], p_full, p_empty, o_full, o_empty, done;
  uint32_t tmem_base;
  int abort_flag;
  unsigned long long wait_ns;
  TileRun run;
  float red[4][4][8];          // [column group][lane quarter][column]
  int off_s[32];               // row j sees tokens t < len + off_s[j]
};
static_assert(sizeof(Aux) <= kAuxBytes, "aux block");

__device__ __forceinline__ bool wait_b(uint64_t* bar, uint32_t parity, Aux* aux, int* err) {
  return tc::wait_b(bar, parity, &aux->abort_flag, err, aux->wait_ns);
}
__device__ __forceinline__ bool wait_w(uint64_t* bar, uint32_t parity, Aux* aux, int* err) {
  return __all_sync(0xffffffffu, wait_b(bar, parity, aux, err));
}

// Shared memory: [aux][q~: r/64 blocks of (2 NR rows hi | lo) x 128 B][q_rope: NR rows x 128 B]
// [P: 128 tokens x NR][slots][rotary tile][8 bits: scales per slot].
// Warps: 0 TMA producer, 1 MMA issuer, then NR / 2 softmax warps (thread = token row = TMEM lane
// of one group of 8 query rows; four warps a group; in the epilogue thread = rank row), then
// (8 bits) 8 warps that expand codes to bf16.  One warp per lane quarter for all 32 columns had
// taken ~4 us a tile: a single warp per scheduler cannot hide its own latencies.
template <int NR, bool kQuant>
constexpr int dec_threads() {
  return 64 + NR * 16 + (kQuant ? 256 : 0);
}
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
  constexpr int kQSub = 2 * NR * 128;
  constexpr int kPBytes = 128 * NR * 2;
  const int nsub = p.r >> 6;
  Aux* aux = reinterpret_cast<Aux*>(smem_raw);
  uint8_t* q_s = smem_raw + kAuxBytes;
  uint8_t* qr_s = q_s + nsub * kQSub;
  uint8_t* p_s = qr_s + NR * 128;
  uint8_t* ring = smem_raw + kAuxBytes + ((nsub * kQSub + NR * 128 + kPBytes + 1023) & ~1023);
  uint8_t* rope_s = ring + p.nslot * kSlot;
  uint8_t* sc_s = rope_s + kSub;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int x = blockIdx.x, hb = blockIdx.y;

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
      ptx::mbar_init(&aux->s_empty[k], NR / 2);
    }
    ptx::mbar_init(&aux->p_full, NR / 2);
    ptx::mbar_init(&aux->p_empty, 1);
    ptx::mbar_init(&aux->o_full, 1);
    ptx::mbar_init(&aux->o_empty, NR / 2);
    ptx::mbar_init(&aux->done, 1);
    aux->abort_flag = 0;
    aux->wait_ns = tc::wait_limit(p.wait_ns);
    ptx::fence_mbar_init();
  }
  if (threadIdx.x >= 64 && threadIdx.x < 96)   // query row j of this block belongs to token (hb NR + j) / Hq
    aux->off_s[lane] = min((hb * NR + lane) / p.Hq, p.n_tok - 1) - (p.n_tok - 1);
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
    const TileRun run = tile_run([&](int b) { return (shared_len(p.row_len, b, p.cap) + 127) >> 7; }, p.B, p.X, x, &chunk);
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
      int gt = 0, pos = 0, nseg = 0;     // tiles, slot uses and sequences issued
      bool ok = true;
      while (ok && next_seg(&run, p, &sg)) {
        if (nseg > 0 && !(ok = wait_b(&aux->q_empty, (nseg - 1) & 1, aux, p.err))) break;
        ptx::mbar_arrive_expect_tx(&aux->q_full, (uint32_t)(nsub * kQSub + NR * 128));
        for (int s = 0; s < nsub; ++s)
          ptx::tma_load_2d(q_s + s * kQSub, &tm_q, &aux->q_full, s * 64, (sg.b * p.HB + hb) * 2 * NR);
        ptx::tma_load_3d(qr_s, &tm_qr, &aux->q_full, 0, hb * NR, sg.b);
        ++nseg;
        int next_page = p.map.page(sg.b, sg.t0 * 128);
        for (int i = 0; i < sg.nt && ok; ++i, ++gt) {
          const int page = next_page;
          // the table is read one tile ahead, so that its latency is not between two copies
          if (i + 1 < sg.nt) next_page = p.map.page(sg.b, (sg.t0 + i + 1) * 128);
          for (int c = 0; c < p.nch; ++c) {
            const int slot = pos % p.nslot, round = pos / p.nslot;
            if (round > 0 && !(ok = wait_b(&aux->slot_empty[slot], (round - 1) & 1, aux, p.err))) break;
            uint8_t* dst = ring + slot * kSlot;
            if (kQuant) {
              // codes into the upper half of their slot, where the expansion reads them before
              // it writes
              const uint32_t bytes = c * 128 + 64 < p.r ? kSub : kSub / 2;
              ptx::mbar_arrive_expect_tx(&aux->raw_full[slot], bytes + kScaleBytes);
              ptx::bulk_load(dst + kSub, p.codes + (long long)page * 128 * p.r + c * kSub, bytes, &aux->raw_full[slot]);
              ptx::bulk_load(sc_s + slot * kScaleBytes, p.scale + ((long long)page * p.nch + c) * kScaleBytes,
                             kScaleBytes, &aux->raw_full[slot]);
            } else {
              const int nb = c * 128 + 64 < p.r ? 2 : 1;
              ptx::mbar_arrive_expect_tx(&aux->slot_full[slot], nb * kSub);
              for (int s = 0; s < nb; ++s)
                ptx::tma_load_2d(dst + s * kSub, &tm_c, &aux->slot_full[slot], c * 128 + s * 64, page * 128);
            }
            ++pos;
          }
          if (!ok) break;
          if (gt > 0 && !(ok = wait_b(&aux->rope_empty, (gt - 1) & 1, aux, p.err))) break;
          ptx::mbar_arrive_expect_tx(&aux->rope_full, kSub);
          ptx::tma_load_2d(rope_s, &tm_kr, &aux->rope_full, 0, page * 128);
        }
      }
      // every copy this thread issued has landed before the CTA can exit
      if (nseg > 0) drain_wait(&aux->q_full, (nseg - 1) & 1);
      for (int k = max(0, pos - p.nslot); k < pos; ++k)
        drain_wait(kQuant ? &aux->raw_full[k % p.nslot] : &aux->slot_full[k % p.nslot], (k / p.nslot) & 1);
      if (gt > 0) drain_wait(&aux->rope_full, (gt - 1) & 1);   // gt: tiles whose rotary part was issued
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------- MMA issuer (warp-wide)
    const uint32_t id1 = ptx::idesc_f16(1, 0, 0, 128, 2 * NR);   // GEMM1: K-major x K-major (hi | lo)
    const uint32_t idr = ptx::idesc_f16(1, 0, 0, 128, NR);       //        rotary part, into the hi columns
    const uint32_t id2 = ptx::idesc_f16(1, 1, 1, 128, NR);       // GEMM2: MN-major x MN-major
    // Operands go through `uniform`: the compiler then keeps them in uniform registers, and an
    // MMA issues every ~40 cycles (the pace of an operand read from shared memory) and not ~115.
    const uint64_t kd0 = ptx::smem_desc(ptx::smem_u32(ring), 16, 1024, 2);
    const uint64_t vd0 = ptx::smem_desc(ptx::smem_u32(ring), kSub, 1024, 2);
    const uint64_t qd0 = ptx::smem_desc(ptx::smem_u32(q_s), 16, 1024, 2);
    const uint64_t rd0 = ptx::smem_desc(ptx::smem_u32(rope_s), 16, 1024, 2);
    const uint64_t qrd0 = ptx::smem_desc(ptx::smem_u32(qr_s), 16, 1024, 2);
    const uint64_t pd0 = ptx::smem_desc(ptx::smem_u32(p_s), 128, 2048, 0);
    int gt0 = 0, nseg = 0;
    bool ok = true;
    // With slots for two tiles the scores of tile i + 1 go before the value mix of tile i, and
    // so run during its softmax; a tile's slots are held until its value mix.
    const bool ahead = p.nslot >= 2 * p.nch;
    while (ok && next_seg(&run, p, &sg)) {
      if (!(ok = wait_w(&aux->q_full, nseg & 1, aux, p.err))) break;
      ptx::tc_fence_after();
      for (int u = 0; u < 2 * sg.nt && ok; ++u) {
        int i = u >> 1;
        bool isv = u & 1;
        if (ahead) tc::unit_of(u, sg.nt, &i, &isv);
        const int gt = gt0 + i;
        if (!isv) {
          const int sb = gt & 1;
          if (gt >= 2 && !(ok = wait_w(&aux->s_empty[sb], ((gt - 2) >> 1) & 1, aux, p.err))) break;
          ptx::tc_fence_after();
          const uint32_t d_s = uniform(tmem + kSCol + 64 * sb);
          for (int c = 0; c < p.nch; ++c) {
            const int pos = gt * p.nch + c, slot = pos % p.nslot;
            if (!(ok = wait_w(&aux->slot_full[slot], (pos / p.nslot) & 1, aux, p.err))) break;
            ptx::tc_fence_after();
            const uint64_t a0 = kd0 + uniform((slot * kSlot) >> 4);
            const uint64_t b0 = qd0 + uniform((c * 2 * kQSub) >> 4);
            const uint32_t first = uniform(c ? 1u : 0u);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              ptx::mma_f16_elect(d_s, a0 + (uint64_t)(kk * 2), b0 + (uint64_t)(kk * 2), id1, kk ? 1u : first);
            if (c * 128 + 64 < p.r) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                ptx::mma_f16_elect(d_s, a0 + (uint64_t)((kSub >> 4) + kk * 2), b0 + (uint64_t)((kQSub >> 4) + kk * 2),
                                   id1, 1u);
            }
          }
          if (!ok || !(ok = wait_w(&aux->rope_full, gt & 1, aux, p.err))) break;
          ptx::tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)       // columns past dim_rope are 0 on both sides
            ptx::mma_f16_elect(d_s, rd0 + (uint64_t)(kk * 2), qrd0 + (uint64_t)(kk * 2), idr, 1u);
          ptx::mma_commit_elect(&aux->rope_empty);
          if (i == sg.nt - 1) ptx::mma_commit_elect(&aux->q_empty);
          ptx::mma_commit_elect(&aux->s_full[sb]);
        } else {
          if (!(ok = wait_w(&aux->p_full, gt & 1, aux, p.err))) break;
          if (i == 0 && nseg > 0 && !(ok = wait_w(&aux->o_empty, (nseg - 1) & 1, aux, p.err))) break;
          ptx::tc_fence_after();
          const uint32_t first = uniform(i ? 1u : 0u);
          for (int c = 0; c < p.nch; ++c) {
            const int slot = (gt * p.nch + c) % p.nslot;
            const uint64_t a0 = vd0 + uniform((slot * kSlot) >> 4);
            const uint32_t d_o = uniform(tmem + kOCol + c * NR);
#pragma unroll
            for (int kt = 0; kt < 8; ++kt)
              ptx::mma_f16_elect(d_o, a0 + (uint64_t)(kt * 128), pd0 + (uint64_t)(kt * 16), id2, kt ? 1u : first);
            ptx::mma_commit_elect(&aux->slot_empty[slot]);
          }
          ptx::mma_commit_elect(&aux->p_empty);
          if (i == sg.nt - 1) ptx::mma_commit_elect(&aux->o_full);
        }
      }
      gt0 += sg.nt;
      ++nseg;
    }
    ptx::mma_commit_elect(&aux->done);
    drain_wait(&aux->done, 0);
    __syncwarp();
  } else if (warp < 2 + NR / 2) {
    // ------------------------------------------------------------- softmax / epilogue
    const int qd = warp & 3, g = (warp - 2) >> 2;        // lane quarter, column group
    const int row = qd * 32 + lane;
    const uint32_t lane_off = (uint32_t)(qd * 32) << 16;
    const int bar = 1 + g;                               // the group's four warps
    int gt = 0, nseg = 0;
    bool ok = true;
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
        const uint32_t s_col = tmem + lane_off + kSCol + 64 * k2 + 8 * g;
        // after an abort every wait returns at once: the group's warps finish the sequence in step
        // (their barriers stay matched) and leave at the verdict below
        (void)wait_w(&aux->s_full[k2], (gt >> 1) & 1, aux, p.err);
        ptx::tc_fence_after();
        // a tile every row sees whole needs no masks; otherwise row j sees t < len + off_s[j]
        const bool edge = (sg.t0 + i) * 128 + 128 > sg.len - (p.n_tok - 1);
        float s[8];
        {
          uint32_t a[8], b[8];
          ptx::tmem_ld8(s_col, a);
          ptx::tmem_ld8(s_col + NR, b);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 8; ++j) s[j] = (__uint_as_float(a[j]) + __uint_as_float(b[j])) * p.scale_log2;
        }
        if (edge) {
#pragma unroll
          for (int j = 0; j < 8; ++j) s[j] = t < sg.len + aux->off_s[8 * g + j] ? s[j] : -INFINITY;
        }
        bool ex = false;
#pragma unroll
        for (int j = 0; j < 8; ++j) ex |= s[j] > m[j] + kLazy;
        ex = ptx::named_bar_or(bar, 128, ex);
        if (gt > 0) {   // the value mix before has completed: P may be rewritten, O~ rescaled
          (void)wait_w(&aux->p_empty, (gt - 1) & 1, aux, p.err);
          ptx::tc_fence_after();
        }
        if (!kQuant && t >= sg.len) {
          // rows behind the sequence hold whatever the page held: 0 weight times a stale
          // infinity would still be NaN, so their values become 0 (the groups share the boxes)
          for (int c = g; c < 2 * p.nch; c += NR / 8) {
            const uint32_t base =
                ptx::smem_u32(ring + ((gt * p.nch + (c >> 1)) % p.nslot) * kSlot + (c & 1) * kSub + row * 128);
#pragma unroll
            for (int v = 0; v < 8; ++v)
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(base + v * 16), "r"(0) : "memory");
          }
        }
        __syncwarp();
        if (ex) {
          float top[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) top[j] = s[j];
          const float mt = reduce_cols<true>(top, lane);
          if (lane < 8) aux->red[g][qd][lane] = mt;   // read by all before the next tile's vote
          ptx::named_bar_sync(bar, 128);
          float a[8];
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
          if (need_o && i > 0) {
            for (int c = 0; c < p.nch; ++c) {
              uint32_t v[8];
              const uint32_t col = tmem + lane_off + kOCol + c * NR + 8 * g;
              ptx::tmem_ld8(col, v);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 8; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * a[j]);
              ptx::tmem_st8(col, v);
            }
            ptx::tmem_wait_st();
          }
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
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(ptx::smem_u32(p_s + g * 2048 + row * 16)),
                     "r"(hw[0]), "r"(hw[1]), "r"(hw[2]), "r"(hw[3])
                     : "memory");
        // every lane makes its own stores visible to the tensor core, then one arrival per warp
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive(&aux->s_empty[k2]);
          ptx::mbar_arrive(&aux->p_full);
        }
      }
      ok = ptx::named_bar_and(bar, 128, wait_b(&aux->o_full, nseg & 1, aux, p.err));
      if (!ok) break;
      ptx::tc_fence_after();
      const size_t base = ((size_t)(x + sg.b) * p.HB + hb) * NR + 8 * g;
      const float lt = reduce_cols<false>(l, lane);
      if (lane < 8) aux->red[g][qd][lane] = lt;
      ptx::named_bar_sync(bar, 128);
      if (qd == 0 && lane < 8) {
        float mj = m[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) mj = lane == j ? m[j] : mj;
        const float l4 = (aux->red[g][0][lane] + aux->red[g][1][lane]) + (aux->red[g][2][lane] + aux->red[g][3][lane]);
        reinterpret_cast<float2*>(p.part_ml)[base + lane] = make_float2(mj, l4);
      }
      for (int c = 0; c < p.nch; ++c) {
        uint32_t o[8];
        ptx::tmem_ld8(tmem + lane_off + kOCol + c * NR + 8 * g, o);
        ptx::tmem_wait_ld();
        const int e = c * 128 + row;
        if (e < p.r) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (hb * NR + 8 * g + j < p.R) p.part_o[(base + j) * p.r + e] = __uint_as_float(o[j]);
        }
        __syncwarp();
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&aux->o_empty);
      ++nseg;
    }
  } else if (kQuant) {
    // ------------------------------------------------------------- expansion of codes
    const int tid = threadIdx.x - (64 + NR * 16);   // 0..255
    int pos = 0;
    bool ok = true;
    while (ok && next_seg(&run, p, &sg)) {
      for (int i = 0; i < sg.nt && ok; ++i) {
        const int valid = sg.len - (sg.t0 + i) * 128;      // token rows of this tile (may exceed 128)
        for (int c = 0; c < p.nch; ++c, ++pos) {
          const int slot = pos % p.nslot;
          if (!(ok = wait_w(&aux->raw_full[slot], (pos / p.nslot) & 1, aux, p.err))) break;
          uint8_t* dst = ring + slot * kSlot;
          const uint8_t* sc = sc_s + slot * kScaleBytes;
          expand_chunk(dst, sc, tid, c * 128 + 64 < p.r, valid);
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&aux->slot_full[slot]);
        }
      }
    }
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
  __nv_bfloat16* qt;     // [B][HB][2 NR][r]
  int* err;
};
struct QpAux {
  uint64_t w_full, q_full, done;
  uint32_t tmem_base;
  int abort_flag;
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
  uint8_t* q_s = smem_raw + (p.dn >> 6) * kSub;  // dn/64 blocks of ncols rows x 128 B
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
    ptx::mbar_arrive_expect_tx(&aux.w_full, kb * kSub);
    for (int k = 0; k < kb; ++k) ptx::tma_load_2d(w_s + k * kSub, &tm_w, &aux.w_full, h * p.dn + k * 64, i0);
  }
  if (warp == 1) {
    ptx::tmem_alloc(&aux.tmem_base, 128);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = aux.tmem_base;
  pdl_wait();
  pdl_trigger();
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
          ptx::mma_f16_elect(tmem, wd + (uint64_t)((k * kSub >> 4) + kk * 2),
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
        const int m = c0 + j, bs = bs0 + m / p.g;
        if (m >= p.nb * p.g || bs >= p.BS || i >= p.r) continue;
        const int b = bs / p.n_tok, row = (bs % p.n_tok) * p.Hq + h * p.g + m % p.g;
        const float f = __uint_as_float(v[j]);
        const __nv_bfloat16 hi = __float2bfloat16_rn(f);
        const __nv_bfloat16 lo = __float2bfloat16_rn(f - __bfloat162float(hi));
        const size_t o = (((size_t)b * p.HB + row / p.NR) * 2 * p.NR + row % p.NR) * p.r + i;
        p.qt[o] = hi;
        p.qt[o + (size_t)p.NR * p.r] = lo;
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 128);
  }
}

// ---------------------------------------------------------------------------
// Join of the split partials and output projection, per KV head and block of RB (<= 16) query
// rows: o~ = sum_k w_k o~_k / sum_k w_k l_k with w_k = 2^(m_k - max m), then
// out = o~ B_v,h with M = dim_v (A: B_v,h columns, MN-major), N = 32 rows (bf16 hi | lo of o~,
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
  int first[16], count[16], row[16];   // per row: first slot, slots, row of its sequence
  float inv[16];
  float w[16][kMaxRuns];
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
  uint8_t* o_s = smem_raw;                               // nsub blocks of 32 rows x 128 B
  uint8_t* w_s = o_s + nsub * 4096;                      // 2 column halves of r rows x 128 B
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
  if (warp == 1) {
    ptx::tmem_alloc(&aux->tmem_base, 32);
    ptx::tmem_relinquish();
  }
  if (threadIdx.x < 16) aux->count[threadIdx.x] = 0;
  pdl_wait();
  pdl_trigger();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = aux->tmem_base;
  const int nrow = min(p.RB, p.rows - m0);               // rows m0 .. m0 + nrow - 1
  if (warp == 0) {
    // slots of the rows' sequences, from the same cut into runs as the decode's
    auto tiles = [&](int b) { return (shared_len(p.row_len, b, p.cap) + 127) >> 7; };
    const int chunk = max(1, (tile_total(tiles, p.B) + p.X - 1) / p.X);
    int run = 0;
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
      if (v > 0) {
        const int x0 = t0 / chunk, x1 = (t0 + v - 1) / chunk;
        for (int k = 0; k < nrow; ++k)
          if ((m0 + k) / p.g / p.n_tok == b) {
            aux->first[k] = x0 + b;
            aux->count[k] = min(x1 - x0 + 1, kMaxRuns);
          }
      }
      run += __shfl_sync(0xffffffffu, inc, 31);
    }
    __syncwarp();
    if (lane < nrow) {
      const int bs = (m0 + lane) / p.g;
      aux->row[lane] = (bs % p.n_tok) * p.Hq + h * p.g + (m0 + lane) % p.g;
    }
  }
  __syncthreads();
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
      if (p.lse) {
        const int bs = (m0 + k) / p.g;
        p.lse[(size_t)(bs / p.n_tok) * p.n_tok * p.Hq + aux->row[k]] =
            l == 0.f ? -INFINITY : (m + log2f(l)) * LR_LN2;
      }
    }
  }
  __syncthreads();
  // A part of r/4 threads (4 ranks each) sums a row's slots; with fewer rows than parts, several
  // parts share a row, each with every sub-th slot.  The rows of o_s past nrow stay as they are:
  // they only reach accumulator columns that nobody reads.
  const int r4 = p.r >> 2, parts = kOutThreads / r4;
  const int part = (int)threadIdx.x / r4, e = ((int)threadIdx.x % r4) * 4;
  const int subs = max(1, parts / nrow);
  const int sub = subs > 1 ? part / nrow : 0;
  for (int k0 = 0; k0 < nrow; k0 += parts) {
    const int k = subs > 1 ? part % nrow : k0 + part;
    const bool in = part < parts && k < nrow && sub < subs;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (in) {
      const int n = aux->count[k];
      const float* src = p.part_o + ((size_t)aux->first[k] * srow + aux->row[k]) * p.r + e;
      const float* w = aux->w[k];
      const size_t step = srow * p.r;
      for (int s = sub; s < n; s += 8 * subs) {
        float4 v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (s + q * subs < n) v[q] = *reinterpret_cast<const float4*>(src + (s + q * subs) * step);
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (s + q * subs < n) {
            const float f = w[s + q * subs];
            acc.x += f * v[q].x;
            acc.y += f * v[q].y;
            acc.z += f * v[q].z;
            acc.w += f * v[q].w;
          }
      }
    }
    if (subs > 1) {
      aux->part[threadIdx.x] = acc;
      __syncthreads();
      if (in && sub == 0)
        for (int q = 1; q < subs; ++q) {
          const float4 v = aux->part[threadIdx.x + q * nrow * r4];
          acc.x += v.x;
          acc.y += v.y;
          acc.z += v.z;
          acc.w += v.w;
        }
    }
    if (in && sub == 0) {
      const float inv = aux->inv[k];
      acc.x *= inv;
      acc.y *= inv;
      acc.z *= inv;
      acc.w *= inv;
      const __nv_bfloat162 h0 = __floats2bfloat162_rn(acc.x, acc.y), h1 = __floats2bfloat162_rn(acc.z, acc.w);
      const __nv_bfloat162 l0 = __floats2bfloat162_rn(acc.x - __low2float(h0), acc.y - __high2float(h0));
      const __nv_bfloat162 l1 = __floats2bfloat162_rn(acc.z - __low2float(h1), acc.w - __high2float(h1));
      // K-major, 128-byte swizzle: row k (hi) and 16 + k (lo; 16 % 8 = 0, the same swizzle)
      uint8_t* d = o_s + (e >> 6) * 4096 + k * 128 + ((((e & 63) >> 3) ^ (k & 7)) << 4) + (e & 4) * 2;
      *reinterpret_cast<uint2*>(d) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1));
      *reinterpret_cast<uint2*>(d + 16 * 128) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&l0), *reinterpret_cast<const uint32_t*>(&l1));
    }
  }
  ptx::fence_proxy_async_smem();
  __syncthreads();
  if (warp == 0) {
    const bool ok = __all_sync(
        0xffffffffu, tc::wait_b(&aux->w_full, 0, &aux->abort_flag, p.err, tc::wait_limit(p.wait_ns)));
    if (ok) {
      ptx::tc_fence_after();
      const uint32_t id = ptx::idesc_f16(1, 1, 0, 128, 32);   // A MN-major, B K-major
      const uint64_t wd = ptx::smem_desc(ptx::smem_u32(w_s), (uint32_t)p.r * 128, 1024, 2);
      const uint64_t od = ptx::smem_desc(ptx::smem_u32(o_s), 16, 1024, 2);
      for (int k = 0; k < nsub; ++k)
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          ptx::mma_f16_elect(tmem, wd + (uint64_t)((k * 64 + kk * 16) * 128 >> 4),
                             od + (uint64_t)((k * 4096 >> 4) + kk * 2), id, (k | kk) ? 1u : 0u);
    }
    ptx::mma_commit_elect(&aux->done);
    drain_wait(&aux->w_full, 0);
    drain_wait(&aux->done, 0);
    __syncwarp();
  }
  __syncthreads();
  ptx::tc_fence_after();
  if (warp < 4 && !aux->abort_flag) {
    uint32_t v[32];
    ptx::tmem_ld32(tmem + ((uint32_t)(warp * 32) << 16), v);
    ptx::tmem_wait_ld();
    const int d = warp * 32 + lane;
    if (d < p.dv) {
#pragma unroll
      for (int k = 0; k < 16; ++k)
        if (k < nrow) {
          const int bs = (m0 + k) / p.g;
          const size_t o = (size_t)(bs / p.n_tok) * p.n_tok * p.Hq + aux->row[k];
          p.out[o * p.dv + d] = __float2bfloat16_rn(__uint_as_float(v[k]) + __uint_as_float(v[16 + k]));
        }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 32);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// How R query rows per sequence are cut: NR per block, HB blocks, X runs of tiles.  A block of
// 16 rows when a sequence has no more, else 32; pairs of CTAs (r > 256) also have blocks of 64.
struct Cut {
  int NR, HB, X;
};
Cut cut_of(const lr_shared_desc& d, int n_tokens, int num_sms) {
  const int R = n_tokens * d.n_q_heads;
  const bool pair = d.rank > 256;
  Cut c;
  c.NR = R <= 16 ? 16 : (pair && R > 32 ? 64 : 32);
  c.HB = (R + c.NR - 1) / c.NR;
  c.X = std::max(1, std::min(num_sms, kMaxRuns) / (pair ? 2 : 1) / c.HB);
  return c;
}

size_t decode_smem(int r, int NR, int nslot, bool quant) {
  const size_t head = (size_t)(r / 64) * 2 * NR * 128 + (size_t)NR * 128 + 128 * NR * 2;
  return kAuxBytes + ((head + 1023) & ~(size_t)1023) + (size_t)nslot * kSlot + kSub +
         (quant ? (size_t)nslot * kScaleBytes : 0);
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
                    c->tm_qt[NR / 32], tqr, c->tm_c, c->tm_kr, a);
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
            map2d(&c->tm_kr, bf, c->kr, d.dim_rope, rows, (uint64_t)d.dim_rope * 2, 64, 128) &&
            map2d(&c->tm_qt[0], bf, c->qt, r, qrows, r * 2, 64, 32) &&
            map2d(&c->tm_qt[1], bf, c->qt, r, qrows, r * 2, 64, 64) &&
            map2d(&c->tm_qt[2], bf, c->qt, r, qrows, r * 2, 64, 128);
  // (8 bits: the codes are copied without a map; any valid one stands in)
  if (ok && d.quant_bits) c->tm_c = c->tm_kr;
  else if (ok) ok = map2d(&c->tm_c, bf, c->c, r, rows, r * 2, 64, 128);
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
  const size_t smem_q = (size_t)(d.dim_nope / 64) * (kSub + qp.ncols * 128) + sizeof(QpAux);
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
  if (r > 256) {
    e = launch_shared_pair(c, tqr, row_len, n_tokens, R, NR, HB, X, s);
  } else {
    DecArgs a = dec_args(c, row_len, n_tokens, R, HB, X);
    while (a.nslot < kMaxSlots && decode_smem(r, NR, a.nslot + 1, quant) <= (size_t)kSmemLimit) ++a.nslot;
    const size_t smem = decode_smem(r, NR, a.nslot, quant);
    if (NR == 16)
      e = quant ? launch_dec<16, true>(c, tqr, a, smem, s) : launch_dec<16, false>(c, tqr, a, smem, s);
    else
      e = quant ? launch_dec<32, true>(c, tqr, a, smem, s) : launch_dec<32, false>(c, tqr, a, smem, s);
  }
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
  o.RB = 16;
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
  const size_t smem_o = (size_t)(r / 64) * 4096 + (size_t)2 * r * 128 + sizeof(OutAux);
  return launch_pdl(k_shared_out, dim3((o.rows + o.RB - 1) / o.RB, d.n_kv_heads), dim3(kOutThreads), smem_o, s, c->tm_v,
                    o);
}
