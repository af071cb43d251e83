// Stored tokens of a shared-latent cache as per-head keys and values: K = C B_k, V = C B_v,
// with C the latents read back from their pages, and the rotary keys copied along.
//
// One GEMM whose A operand is gathered by page: M = 256 tokens (two pages), N = 256 columns of
// [K | V], K = rank.  The tensor pipe bounds it (2 r flop per 2-byte output element: 512 flop
// per byte written at r = 512).  Two CTAs form a pair (cta_group::2): each keeps one page's whole
// latent tile in shared memory (r <= 512: 128 KB) and streams half of the bases' columns past both
// (from a copy transposed at creation, so both operands are K-major rows of 64 ranks).  So per 256 x
// 256 block only the bases cross L2, half by each: 32 B per SM and clock at full rate, where a single
// CTA's 128 x 256 blocks need 64 and an SM gets ~38.  The (page pair, column block) units of all
// sequences are cut into equal consecutive runs, one per pair: a run changes its tiles once or twice,
// and each 64-rank part of the next is fetched as soon as the last block has used the old one.
// Two TMEM accumulators let the epilogue of one block run under the MMAs of the next; it stores 32
// bytes per lane, whole sectors.  32768 tokens of r = 512, 28 heads of 128 + 128: 206 us, 1.17
// PFLOP/s in a short burst (259 us with single CTAs), 246 us run continuously: the card's power limit
// (1000 W, 1.6 GHz) then sets the pace, with 2 TB/s of writes beside the tensor pipe.
//
// 8-bit latents are expanded to bf16 (exactly) by eight warps straight from global memory into
// the swizzled tile, once per tile; the MMAs then run as for bf16.
#include "shared_internal.cuh"
#include "tc_common.cuh"


#include <algorithm>

namespace {

using tc::drain_wait;

constexpr int kSub = 128 * 128;        // 128 tokens x 64 ranks x 2 B
constexpr int kStage = kSub;           // 128 columns x 64 ranks x 2 B (this CTA's half of 256 columns)
constexpr int kStages = 6;
constexpr int kAuxBytes = 2048;

constexpr int kMaxTiles = 60;          // tiles of one CTA in a run

struct ExpArgs {
  unsigned long long wait_ns;
  const int32_t* cu; const int32_t* start;
  RowMap map;
  int B, cap, total, r, Wk, W, NB;   // columns: [0, Wk) of K, [Wk, W) of V; NB blocks of 256
  int dr;
  const uint8_t* codes; const uint8_t* scale;
  const __nv_bfloat16* kr_pool;
  __nv_bfloat16* k; __nv_bfloat16* v; __nv_bfloat16* kr;
  int* err;
};

// One tile of the run: token row i of it is row pool + i of the stored arrays and, for
// lo <= i < hi, row out + i of the results.
struct Tile {
  long long pool, out;
  int lo, hi;
};

// Barriers (arrival count; who arrives -> who waits).  CTA 0 issues all MMAs, so what they wait for is
// counted there, for both CTAs; what they free is announced in both:
//   a_full[s]   1 + tx / 16   producers (bf16) or expansion warps (8 bits) -> MMA; 64 ranks of the tiles
//   a_empty[s]  1        MMA commit in the tiles' last block -> producer / expansion warps
//   b_full/b_empty[s]    1 + tx / 1   basis stages (64 ranks)
//   d_full/d_empty[2]    1 / 8        accumulators
struct Aux {
  uint64_t a_full[8], a_empty[8], b_full[kStages], b_empty[kStages], d_full[2], d_empty[2], done;
  unsigned long long wait_ns;
  uint32_t tmem_base;
  int abort_flag;
  int blk0, units;       // first column block, units of this CTA
  Tile tiles[kMaxTiles];
};
static_assert(sizeof(Aux) <= kAuxBytes, "aux block");

__device__ __forceinline__ bool wait_b(uint64_t* bar, uint32_t parity, Aux* aux, int* err) {
  return tc::wait_b(bar, parity, &aux->abort_flag, err, aux->wait_ns);
}
__device__ __forceinline__ bool wait_w(uint64_t* bar, uint32_t parity, Aux* aux, int* err) {
  return __all_sync(0xffffffffu, wait_b(bar, parity, aux, err));
}
// As wait_w, for phases that the other CTA takes part in: what its threads did before is visible.
__device__ __forceinline__ bool wait_x(uint64_t* bar, uint32_t parity, Aux* aux, int* err) {
  const uint64_t t0 = ptx::globaltimer();
  bool ok = false;
  for (;;) {
    if (ptx::mbar_try_wait_cluster(bar, parity)) {
      ok = true;
      break;
    }
    if (*(volatile int*)&aux->abort_flag) break;
    if (ptx::globaltimer() - t0 > aux->wait_ns) {
      *(volatile int*)&aux->abort_flag = 1;
      atomicExch(err, (int)LR_ERR_TIMEOUT);
      break;
    }
  }
  return __all_sync(0xffffffffu, ok);
}

// Positions [lo, hi) of sequence b to expand, inside the cache and the results; position t goes to row
// t + off.  With an ascending cu there are then no more tiles than the host reckoned with, however many
// rows it speaks of; with another one there may be, and runs that do not fit are cut and reported.
struct Span {
  int lo, hi;
  long long off;
};
__device__ __forceinline__ Span span_at(const ExpArgs& p, int b) {
  const long long c0 = __ldg(p.cu + b), c1 = min(__ldg(p.cu + b + 1), p.total), st = p.start ? __ldg(p.start + b) : 0;
  Span s;
  s.off = c0 - st;
  s.lo = (int)min(max(max(c0, 0ll) - s.off, 0ll), (long long)p.cap);
  s.hi = (int)min(max(c1 - s.off, (long long)s.lo), (long long)p.cap);
  return s;
}
__device__ __forceinline__ int span_tiles(const ExpArgs& p, int b) {
  const Span s = span_at(p, b);
  return s.hi > s.lo ? ((s.hi + 127) >> 7) - (s.lo >> 7) : 0;
}

// A warp-uniform value, known as such to the compiler: MMA operands then stay in uniform registers
// (an MMA issues at the tensor core's pace; without, every ~160 cycles).
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

// A role's place in the run: unit u is column block blk of tile k.
struct Place {
  int u, k, blk;
  __device__ __forceinline__ bool fresh() const { return u == 0 || blk == 0; }
  __device__ __forceinline__ bool last(int units, int NB) const { return u == units - 1 || blk == NB - 1; }
  __device__ __forceinline__ void next(int NB) {
    ++u;
    if (++blk == NB) {
      blk = 0;
      ++k;
    }
  }
};

// Warps: 0 TMA producer, 1 MMA issuer (CTA 0), 2..5 epilogue, (8 bits) 6..13 expansion of codes; the
// last copies the rotary keys.
template <bool kQuant>
constexpr int exp_threads() {
  return kQuant ? 480 : 224;
}
template <bool kQuant>
__global__ void __launch_bounds__(exp_threads<kQuant>(), 1)
    k_shared_expand(const __grid_constant__ CUtensorMap tm_c, const __grid_constant__ CUtensorMap tm_w,
                    const ExpArgs p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (ptx::smem_u32(smem_raw) & 1023) {
    if (threadIdx.x == 0) atomicExch(p.err, (int)LR_ERR_UNSUPPORTED);
    return;
  }
  Aux* aux = reinterpret_cast<Aux*>(smem_raw);
  uint8_t* a_s = smem_raw + kAuxBytes;
  const int nsub = p.r >> 6;
  uint8_t* b_s = a_s + nsub * kSub;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t cr = ptx::cluster_rank();

  if (threadIdx.x == 0) {
    for (int s = 0; s < 8; ++s) {
      ptx::mbar_init(&aux->a_full[s], kQuant ? 16 : 1);
      ptx::mbar_init(&aux->a_empty[s], 1);
    }
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(&aux->b_full[s], 1);
      ptx::mbar_init(&aux->b_empty[s], 1);
    }
    for (int k = 0; k < 2; ++k) {
      ptx::mbar_init(&aux->d_full[k], 1);
      ptx::mbar_init(&aux->d_empty[k], 8);
    }
    ptx::mbar_init(&aux->done, 1);
    aux->abort_flag = 0;
    aux->wait_ns = tc::wait_limit(p.wait_ns);
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tm_c);
    ptx::prefetch_tmap(&tm_w);
  }
  pdl_wait();
  if (warp == 1) {            // (after the wait, as in k_shared_decode)
    ptx::tmem_alloc_pair(&aux->tmem_base, 512);
    ptx::tmem_relinquish_pair();
  }
  if (warp == 0) {
    // this CTA's run of units, and its tiles
    auto tiles = [&](int b) { return span_tiles(p, b); };
    const int total = tile_total(tiles, p.B);
    const unsigned G = gridDim.x / 2;                             // pairs
    const unsigned units = ((unsigned)total + 1) / 2 * (unsigned)p.NB;      // < 2^31 (host)
    const unsigned chunk = (units + G - 1) / G, first = chunk * (unsigned)(blockIdx.x >> 1);
    int n = 0, blk0 = 0;
    if (first < units) {
      n = (int)min(chunk, units - first);
      if (n > (kMaxTiles - 1) * p.NB) {        // more than the tile table holds: cu does not ascend
        n = (kMaxTiles - 1) * p.NB;
        if (lane == 0) atomicExch(p.err, (int)LR_ERR_INVALID_ARG);
      }
      blk0 = (int)(first % (unsigned)p.NB);
      const int t0 = (int)(first / (unsigned)p.NB), nt = (blk0 + n + p.NB - 1) / p.NB;
      for (int k = 0; k < nt; ++k) {
        int b, tile;
        const int t = 2 * (t0 + k) + (int)cr;
        if (t >= total) {            // an odd number of tiles: the last pair's second is any page, and not stored
          if (lane == 0) aux->tiles[k] = Tile{0, 0, 0, 0};
          continue;
        }
        tile_find(tiles, p.B, t, &b, &tile);
        if (lane == 0) {
          const Span s = span_at(p, b);
          const int tok = ((s.lo >> 7) + tile) << 7;
          aux->tiles[k].pool = (long long)p.map.page(b, tok) << 7;
          aux->tiles[k].out = tok + s.off;
          // rows inside the span, the results and the cache
          const long long o = tok + s.off;
          aux->tiles[k].lo = (int)max((long long)max(s.lo - tok, 0), min(-o, 128ll));
          aux->tiles[k].hi = (int)min((long long)min(s.hi - tok, 128), max((long long)p.total - o, 0ll));
        }
      }
    }
    if (lane == 0) {
      aux->blk0 = blk0;
      aux->units = n;
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();      // both CTAs' barriers are ready before any copy or arrival counts there
  ptx::tc_fence_after();
  pdl_trigger();
  const uint32_t tmem = aux->tmem_base;
  const int units = aux->units;
  Place w{0, 0, aux->blk0};

  if (warp == 0) {
    // ------------------------------------------------------------- TMA producer
    if (lane == 0) {
      int pos = 0, nt = 0;                  // basis stages and tiles issued
      int a_boxes = 0;                      // boxes issued of tile nt - 1
      bool ok = true;
      for (; ok && w.u < units; w.next(p.NB)) {
        const int c0 = w.blk * 256, n2 = min(256, p.W - c0) / 2;   // this CTA's columns of the block
        const bool fresh = w.fresh();
        const int row = (int)aux->tiles[w.k].pool;
        if (fresh) {
          ++nt;
          a_boxes = 0;
        }
        for (int h = 0; h < nsub; ++h) {
          if (!kQuant && fresh) {
            if (nt > 1 && !(ok = wait_b(&aux->a_empty[h], nt & 1, aux, p.err))) break;   // tile nt - 2's use
            if (cr == 0) ptx::mbar_arrive_expect_tx(&aux->a_full[h], 2 * kSub);
            ptx::tma_load_2d_pair(a_s + h * kSub, &tm_c, ptx::map_rank(ptx::smem_u32(&aux->a_full[h]), 0), h * 64, row);
            ++a_boxes;
          }
          const int st = pos % kStages;
          if (pos >= kStages && !(ok = wait_b(&aux->b_empty[st], (pos / kStages - 1) & 1, aux, p.err))) break;
          if (cr == 0) ptx::mbar_arrive_expect_tx(&aux->b_full[st], 2 * kStage);
          ptx::tma_load_2d_pair(b_s + st * kStage, &tm_w, ptx::map_rank(ptx::smem_u32(&aux->b_full[st]), 0), h * 64,
                                c0 + (int)cr * n2);        // rows past W read as 0
          ++pos;
        }
      }
      // every copy of either CTA has landed before the pair's last barrier (after an abort the other
      // CTA may not have issued its own: time to land is given there instead)
      if (cr == 0 && ok) {
        for (int k = max(0, pos - kStages); k < pos; ++k) drain_wait(&aux->b_full[k % kStages], (k / kStages) & 1);
        if (!kQuant)
          for (int s = 0; s < nsub; ++s) {
            const int n = s < a_boxes ? nt : nt - 1;      // tiles whose box s was issued
            if (n > 0) drain_wait(&aux->a_full[s], (n - 1) & 1);
          }
      }
    }
  } else if (warp == 1 && cr == 0) {
    // ------------------------------------------------------------- MMA issuer (warp-wide)
    const uint64_t ad0 = ptx::smem_desc(ptx::smem_u32(a_s), 16, 1024, 2);
    const uint64_t bd0 = ptx::smem_desc(ptx::smem_u32(b_s), 16, 1024, 2);
    int st = 0, nt = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (; ok && w.u < units; w.next(p.NB)) {
      const uint32_t id = uniform(ptx::idesc_f16(1, 0, 0, 256, (uint32_t)min(256, p.W - w.blk * 256)));
      const bool fresh = w.fresh(), last = w.last(units, p.NB);
      const int u = w.u;
      if (fresh) ++nt;
      const uint32_t d = uniform(tmem + (uint32_t)(u & 1) * 256);
      if (u >= 2 && !(ok = wait_x(&aux->d_empty[u & 1], ((u >> 1) - 1) & 1, aux, p.err))) break;
      for (int h = 0; h < nsub; ++h) {
        if (fresh && !(ok = wait_x(&aux->a_full[h], (nt - 1) & 1, aux, p.err))) break;
        if (!(ok = wait_w(&aux->b_full[st], ph, aux, p.err))) break;
        ptx::tc_fence_after();
        const uint64_t ad = ad0 + uniform((uint32_t)(h * kSub) >> 4);
        const uint64_t bd = bd0 + uniform((uint32_t)(st * kStage) >> 4);
        const uint32_t more = uniform(h ? 1u : 0u);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          ptx::mma_f16_pair_elect(d, ad + (uint64_t)(kk * 2), bd + (uint64_t)(kk * 2), id, kk ? 1u : more);
        ptx::mma_commit_pair_elect(&aux->b_empty[st]);
        if (last) ptx::mma_commit_pair_elect(&aux->a_empty[h]);
        if (++st == kStages) {
          st = 0;
          ph ^= 1;
        }
      }
      if (ok) ptx::mma_commit_pair_elect(&aux->d_full[u & 1]);
    }
    ptx::mma_commit_pair_elect(&aux->done);
    drain_wait(&aux->done, 0);
    __syncwarp();
  } else if (warp >= 2 && warp < 6) {
    // ------------------------------------------------------------- epilogue: thread = token row
    const int qd = warp & 3, row = qd * 32 + lane;
    const uint32_t lane_off = (uint32_t)(qd * 32) << 16;
    for (; w.u < units; w.next(p.NB)) {
      const Tile t = aux->tiles[w.k];
      const bool in = row >= t.lo && row < t.hi;
      const long long orow = t.out + row;
      const int c0 = w.blk * 256, n = min(256, p.W - c0), u = w.u;
      if (!wait_w(&aux->d_full[u & 1], (u >> 1) & 1, aux, p.err)) break;
      ptx::tc_fence_after();
      for (int c = 0; c < n; c += 32) {
        uint32_t v[32];
        ptx::tmem_ld32(tmem + lane_off + (uint32_t)(u & 1) * 256 + c, v);
        ptx::tmem_wait_ld();
        if (c + 32 >= n) {             // all read: the accumulator is free before the last stores
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive_cluster(ptx::map_rank(ptx::smem_u32(&aux->d_empty[u & 1]), 0));
        }
        // 32 columns lie in K or in V (both widths are multiples of 64)
        const int col = c0 + c;
        __nv_bfloat16* dst = col < p.Wk ? p.k + orow * p.Wk + col : p.v + orow * (p.W - p.Wk) + (col - p.Wk);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t o[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(v[16 * q + 2 * e]),
                                                            __uint_as_float(v[16 * q + 2 * e + 1]));
            o[e] = *reinterpret_cast<const uint32_t*>(&b2);
          }
          if (in) ptx::st_global_v8(dst + 16 * q, o);
        }
        __syncwarp();                  // the next TMEM load wants the whole warp
      }
    }
  } else if (warp == exp_threads<kQuant>() / 32 - 1) {
    // ------------------------------------------------------------- rotary keys, with a tile's first block
    const int sh = p.dr == 64 ? 3 : 2;                 // 16-byte parts of a row
    for (; w.u < units; w.next(p.NB)) {
      if (w.blk != 0) continue;
      const Tile t = aux->tiles[w.k];
      const uint4* src = reinterpret_cast<const uint4*>(p.kr_pool + (t.pool + t.lo) * p.dr);
      uint4* dst = reinterpret_cast<uint4*>(p.kr + (t.out + t.lo) * p.dr);
      const int n = (t.hi - t.lo) << sh;
      for (int i0 = lane; i0 < n; i0 += 8 * 32) {
        uint4 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (i0 + k * 32 < n) v[k] = __ldg(src + i0 + k * 32);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (i0 + k * 32 < n) dst[i0 + k * 32] = v[k];
      }
    }
    __syncwarp();
  } else if (kQuant && warp >= 6) {
    // ------------------------------------------------------------- expansion of codes
    const int tid = threadIdx.x - 192;
    int nt = 0;
    bool ok = true;
    for (; ok && w.u < units; w.next(p.NB)) {
      if (!w.fresh()) continue;
      ++nt;
      const long long row0 = aux->tiles[w.k].pool;
      const uint8_t* const codes = p.codes + shared_code_page(row0 >> 7, p.r);
      const uint8_t* const scale = p.scale + shared_scale_page(row0 >> 7, p.r);
      // four 64-rank parts at a time: a thread's 16-byte code runs are in flight together
      for (int s0 = 0; s0 < nsub; s0 += 4) {
        const int ns = min(4, nsub - s0);
        uint4 cd[8];
        uint32_t eb[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int idx = k * 256 + tid, tok = (idx >> 2) & 127, s = s0 + (idx >> 9), col = idx & 3;
          if ((idx >> 9) < ns) {
            cd[k] = __ldg(reinterpret_cast<const uint4*>(codes + shared_code_index(tok, p.r, s * 64 + col * 16)));
            eb[k] = __ldg(scale + shared_scale_index(tok, s * 2 + (col >> 1)));
          }
        }
        if (nt > 1)
          for (int q = 0; q < ns && ok; ++q) ok = wait_w(&aux->a_empty[s0 + q], nt & 1, aux, p.err);
        if (!ok) break;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int idx = k * 256 + tid, tok = (idx >> 2) & 127, s = s0 + (idx >> 9), col = idx & 3;
          if ((idx >> 9) < ns) {
            const uint32_t cw[4] = {cd[k].x, cd[k].y, cd[k].z, cd[k].w};
            uint32_t all[8];
            shared_expand<4>(cw, eb[k], all);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t* o = all + 4 * h;
              const uint32_t a = ptx::smem_u32(a_s + s * kSub + tok * 128) + (((col * 2 + h) ^ (tok & 7)) << 4);
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(o[0]), "r"(o[1]), "r"(o[2]),
                           "r"(o[3])
                           : "memory");
            }
          }
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0)
          for (int q = 0; q < ns; ++q) ptx::mbar_arrive_cluster(ptx::map_rank(ptx::smem_u32(&aux->a_full[s0 + q]), 0));
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  // neither CTA leaves while the other's MMAs, copies or arrivals may still reach it (after an abort,
  // those that nobody waited for have a millisecond to land, by the clock: a sleep may end at once)
  if (aux->abort_flag)
    for (const uint64_t t0 = ptx::globaltimer(); ptx::globaltimer() - t0 < 1000000;) __nanosleep(10000);
  __syncwarp();
  ptx::cluster_sync();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem, 512);
  }
}

bool map2d(CUtensorMap* m, const void* ptr, uint64_t d0, uint64_t d1, uint32_t b0, uint32_t b1) {
  const cuuint64_t dims[2] = {d0, d1}, st[1] = {d0 * 2};
  const cuuint32_t box[2] = {b0, b1};
  return tc::make_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, ptr, 2, dims, st, box);
}

}  // namespace

cudaError_t shared_expand_maps(lr_shared* c) {
  const lr_shared_desc& d = c->desc;
  const uint64_t W = (uint64_t)d.n_kv_heads * (d.dim_nope + d.dim_v);
  return map2d(&c->tm_bt, c->Bt, d.rank, W, 64, 128) ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t launch_shared_expand(lr_shared* c, const int32_t* cu, const int32_t* start, int total, void* k, void* v,
                                 void* kr, cudaStream_t s) {
  const lr_shared_desc& d = c->desc;
  ExpArgs a;
  a.wait_ns = c->wait_ns;
  a.cu = cu;
  a.start = start;
  a.map = row_map(c);
  a.B = d.batch;
  a.cap = d.capacity;
  a.total = total;
  a.r = d.rank;
  a.Wk = d.n_kv_heads * d.dim_nope;
  a.W = a.Wk + d.n_kv_heads * d.dim_v;
  a.NB = (a.W + 255) / 256;
  a.codes = static_cast<const uint8_t*>(c->c);
  a.scale = c->scale;
  a.dr = d.dim_rope;
  a.kr_pool = static_cast<const __nv_bfloat16*>(c->kr);
  a.kr = static_cast<__nv_bfloat16*>(kr);
  a.k = static_cast<__nv_bfloat16*>(k);
  a.v = static_cast<__nv_bfloat16*>(v);
  a.err = c->dev_err;
  const bool quant = d.quant_bits != 0;
  // One run per pair of SMs, no more runs than units there can be, and no run longer than its tile
  // table holds (beyond 60 tiles an SM, over a million tokens, the runs queue up).
  const long long tiles = (long long)total / 128 + 2 * std::min<long long>(d.batch, total), two = (tiles + 1) / 2;
  const long long grid = 2 * std::max(std::min<long long>(c->num_sms / 2, two * a.NB), (two + kMaxTiles - 3) / (kMaxTiles - 2));
  if (tiles * a.NB > 0x7FFFFFFF) return cudaErrorNotSupported;
  // (more than half an SM's shared memory at any rank: two pairs on the same two SMs could each hold one
  // SM's TMEM and wait for the other's)
  const size_t smem = std::max<size_t>(kAuxBytes + (size_t)(a.r / 64) * kSub + (size_t)kStages * kStage, 120 * 1024);
  static std::atomic<uint32_t> optin[2] = {{0}, {0}};
  cudaError_t e = quant ? smem_optin(k_shared_expand<true>, optin[1]) : smem_optin(k_shared_expand<false>, optin[0]);
  if (e != cudaSuccess) return e;
  return quant ? launch_pdl_cluster(k_shared_expand<true>, dim3((unsigned)grid), dim3(exp_threads<true>()), 2, smem, s, c->tm_c, c->tm_bt, a)
               : launch_pdl_cluster(k_shared_expand<false>, dim3((unsigned)grid), dim3(exp_threads<false>()), 2, smem, s, c->tm_c, c->tm_bt, a);
}
