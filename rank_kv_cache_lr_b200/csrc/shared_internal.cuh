// Internal definitions of the shared-latent cache (lr_shared_* in include/lr_kv.h): one latent
// and one rotary key per token, from which every head's key and value follow.
#pragma once

#include "lr_internal.cuh"

#include <cuda.h>

// Rows of the stored arrays are page * 128 + token % 128, page = table[b][token / 128].
struct lr_shared {
  lr_shared_desc desc;
  int pps, n_pages;      // pages per sequence, pages in the pool
  float scale_log2;      // softmax_scale * log2(e)
  int num_sms = 148, device = 0;
  cudaStream_t last_stream = nullptr;
  unsigned long long wait_ns = 0;
  std::vector<int32_t> host_table;

  void* c = nullptr;          // [rows][r] bf16, or e4m3 codes
                              // (8 bits: shared_code_index)
  uint8_t* scale = nullptr;   // 8 bits: [n_pages][ceil(r/128)][128][4] exponent bytes (shared_scale_index)
  void* kr = nullptr;         // [rows][dr] bf16
  int32_t* table = nullptr;   // [B][pps]
  void* B = nullptr;          // [r][Hkv*dn | Hkv*dv]: the bases side by side, so that one map covers both
  void* Bt = nullptr;         // [Hkv*dn | Hkv*dv][r]: B transposed (lr_shared_expand)
  float2* rope_cs = nullptr;  // [capacity][dr/2] (cos, sin), or null
  void* qt = nullptr;         // decode: query latents, hi and lo halves (k_shared_decode.cu)
  float* part_o = nullptr;    // decode: split partials [slots][rows][r]
  float* part_ml = nullptr;   // decode: [slots][rows][2] = m (log2), l
  int* dev_err = nullptr;

  // tensor maps of the cache's own storage, made once
  CUtensorMap tm_c, tm_c64;   // latents (bf16 caches) by stored row, in boxes of 128 and 64 tokens
  CUtensorMap tm_kr;          // rotary keys, 64 tokens
  CUtensorMap tm_w, tm_v;     // B_k: 128 ranks x 64 columns; B_v: 64 ranks x 64 columns
  CUtensorMap tm_bt;          // Bt: 128 columns x 64 ranks
  CUtensorMap tm_qt[2];       // query latents, hi | lo blocks of 2 x 16 and 2 x 32 rows
};

inline RowMap row_map(const lr_shared* c) {
  RowMap m;
  m.table = c->table;
  m.cap = c->desc.capacity;
  m.pps = c->pps;
  m.n_pages = c->n_pages;
  return m;
}

// The code of rank i of a stored row: a page holds its 128-rank chunks one after another, each
// [128 tokens][128 codes] (a last chunk of 64 ranks: [128][64]), so that a tile's chunk is one
// contiguous copy of 16 (8) KB.  (Boxes of 128 bytes from 512-byte rows took 1.0 us each with
// four in flight, 16 GB/s an SM.)
__host__ __device__ __forceinline__ long long shared_code_page(long long page, int r) { return page * (128ll * r); }
__host__ __device__ __forceinline__ uint32_t shared_code_index(int tok, int r, int i) {   // in its page
  const int c = i >> 7, left = r - (c << 7), w = left < 128 ? left : 128;
  return (uint32_t)((c << 14) + tok * w + (i & 127));
}

// The exponent byte (2^(byte - 127); 255: a group that held a NaN or an infinity) of ranks
// 32 g .. 32 g + 31 of a stored row.  A page's bytes of 128 ranks are contiguous, so that a
// tile side's scales are one 512-byte copy.
__host__ __device__ __forceinline__ long long shared_scale_page(long long page, int r) {
  return page * ((r + 127) >> 7) * 512;
}
__host__ __device__ __forceinline__ uint32_t shared_scale_index(int tok, int g) {   // in its page
  return (uint32_t)((g >> 2) * 512 + tok * 4 + (g & 3));
}

// Two e4m3 codes as bf16 before their scale: a code's sign, exponent and mantissa bits placed in
// a bf16 stand for its value times 2^-120 (subnormals included).  sel picks bytes (i, j) as
// halves with the sign replicated above each (selector bit 3).
template <uint32_t kSel>
__device__ __forceinline__ __nv_bfloat162 shared_place2(uint32_t w) {
  uint32_t a;
  asm("prmt.b32 %0, %1, %1, %2;" : "=r"(a) : "r"(w), "n"(kSel));
  a = (a << 4) & 0x87F087F0u;
  return *reinterpret_cast<const __nv_bfloat162*>(&a);
}
// 4 N codes of one group to bf16: times 2^e, byte eb (27..247, or 255).  e <= 7 (byte at most 134):
// 2^(120 + e) is a bf16, so one exact product; above, two products 2^(b1 - 127) 2^(b2 - 127) with
// 120 folded into the first; byte 255 (a group that held a NaN or an infinity) is NaN.
template <int N>
__device__ __forceinline__ void shared_expand(const uint32_t (&in)[N], uint32_t eb, uint32_t (&out)[2 * N]) {
  const uint32_t b1 = min(eb + 120u, 254u);
  const uint32_t h1 = eb == 255u ? 0x7FC07FC0u : b1 * 0x00800080u;
  const __nv_bfloat162 s1 = *reinterpret_cast<const __nv_bfloat162*>(&h1);
  __nv_bfloat162 x[2 * N];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    x[2 * k] = __hmul2(shared_place2<0x9180>(in[k]), s1);
    x[2 * k + 1] = __hmul2(shared_place2<0xB3A2>(in[k]), s1);
  }
  if (eb > 134u) {
    const uint32_t h2 = (eb + 247u - b1) * 0x00800080u;
    const __nv_bfloat162 s2 = *reinterpret_cast<const __nv_bfloat162*>(&h2);
#pragma unroll
    for (int k = 0; k < 2 * N; ++k) x[k] = __hmul2(x[k], s2);
  }
#pragma unroll
  for (int k = 0; k < 2 * N; ++k) out[k] = *reinterpret_cast<const uint32_t*>(&x[k]);
}

// Work of the paged kernels: the tiles of all sequences in order, cut into equal runs, run x for CTA column x of X.  A run may span several sequences, and a sequence
// several runs; (x, b) pairs form a staircase, so x + b numbers them without gaps in use.
struct TileRun {
  int b, tile, left;   // first sequence, first tile in it, tiles in the run
};

// By one whole warp: the sum of tiles(b) over the sequences.
template <typename Tiles>
__device__ __forceinline__ int tile_total(Tiles tiles, int B) {
  int total = 0;
  for (int i = threadIdx.x & 31; i < B; i += 32) total += tiles(i);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  return total;
}
// By one whole warp: the sequence and its tile that hold tile number `want` (< the total).
template <typename Tiles>
__device__ __forceinline__ void tile_find(Tiles tiles, int B, int want, int* b, int* tile) {
  const int lane = threadIdx.x & 31;
  int run = 0;
  for (int base = 0; base < B; base += 32) {
    const int i = base + lane;
    const int v = i < B ? tiles(i) : 0;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, run + inc > want);
    if (hit) {
      const int src = __ffs(hit) - 1;
      *b = base + src;
      *tile = want - __shfl_sync(0xffffffffu, run + inc - v, src);
      return;
    }
    run += __shfl_sync(0xffffffffu, inc, 31);
  }
  *b = B;
  *tile = 0;
}
// By one whole warp: run x of X equal runs of B sequences' tiles, and the runs' length.
template <typename Tiles>
__device__ __forceinline__ TileRun tile_run(Tiles tiles, int B, int X, int x, int* chunk_out) {
  const int total = tile_total(tiles, B);
  const int chunk = max(1, (total + X - 1) / X);
  *chunk_out = chunk;
  TileRun r{B, 0, 0};
  if ((long long)x * chunk >= total) return r;
  r.left = min(chunk, total - x * chunk);
  tile_find(tiles, B, x * chunk, &r.b, &r.tile);
  return r;
}

// Host side of each operator (checks done by shared_api.cu).
cudaError_t launch_shared_transpose(lr_shared* c, cudaStream_t s);
cudaError_t launch_shared_rope_table(lr_shared* c, cudaStream_t s);
cudaError_t launch_shared_append(lr_shared* c, const void* z, long long z_stride, const void* kr, long long kr_stride,
                                 const int32_t* seq, const int32_t* pos, int n, cudaStream_t s);
cudaError_t launch_shared_read(lr_shared* c, const int32_t* cu, const int32_t* start, int total, void* z, void* kr,
                               cudaStream_t s);
cudaError_t launch_shared_decode(lr_shared* c, const void* q, int n_tokens, const int32_t* row_len, void* out,
                                 float* lse, cudaStream_t s);
cudaError_t launch_shared_expand(lr_shared* c, const int32_t* cu, const int32_t* start, int total, void* k, void* v,
                                 void* kr, cudaStream_t s);
cudaError_t launch_shared_attn(lr_shared* c, const void* q, const void* k, const void* kr, const void* v,
                               const int32_t* cu_q, const int32_t* cu_k, int nseq, int total_q, int total_k,
                               int causal, void* out, float* lse, cudaStream_t s);
// tensor maps of the cache's storage (host only)
cudaError_t shared_decode_maps(lr_shared* c);
cudaError_t shared_expand_maps(lr_shared* c);
// Scratch of the decode, in bytes, for any n_tokens up to max_queries.
size_t shared_qt_bytes(const lr_shared_desc* d);
void shared_part_rows(const lr_shared_desc* d, int num_sms, size_t* rows);
