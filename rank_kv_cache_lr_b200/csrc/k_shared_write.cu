// Writing tokens into the shared-latent cache and reading them back.
//
// A token's row is its latent c (r elements) and its rotary key kr (dr elements).  On the way
// in kr is rotated (rotate-half) at the token's position with an fp32 (cos, sin) table made
// from fp64 angles; c is stored as it is, or in 8 bits: per group of 32 ranks the smallest
// power of two 2^e with max|c| <= 448 * 2^e, and the nearest e4m3 value of c / 2^e.  c / 2^e
// is exact, so the only rounding is to e4m3's 4 significant bits, and what a code stands for
// (4 bits times a power of two) is a bf16 value: reading back rounds nothing.
//
// Both directions move each byte once and are bound by HBM (one decode step: by latency).  A
// warp owns a token: its lanes hold 8 consecutive elements each (16 bytes in, 16 or 8 out), so
// every access is a full coalesced run and a group's maximum is two shuffles within 4 lanes.  With
// many tokens a warp owns two of them, all loads first (65536 tokens of r = 512 in 8 bits, written and
// read back: 53 us with one token a warp, 50 with two, 56 with four; 4.8 TB/s).
#include "shared_internal.cuh"

#include <cuda_fp8.h>

namespace {

constexpr int kWarps = 8, kMany = 2;
// Tokens a warp: kMany once that still fills the SMs (64 warps each), else 1, for the shortest way.
inline int per_warp(int n, int num_sms) { return n >= kMany * 64 * num_sms ? kMany : 1; }

__device__ __forceinline__ uint32_t warp_max4(uint32_t v) {   // over the 4 lanes of a group
  v = max(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return max(v, __shfl_xor_sync(0xffffffffu, v, 2));
}

__device__ __forceinline__ __nv_bfloat162 magnitudes(uint32_t two) {
  two &= 0x7FFF7FFFu;
  return *reinterpret_cast<const __nv_bfloat162*>(&two);
}

// Exponent byte of a group whose largest |element| has the bf16 magnitude bits `top`.
// 448 = 1.75 * 2^8: a maximum m * 2^x takes e = x - 8 while m <= 1.75 (mantissa bits <= 96).
// e >= -100 keeps 2^-e and every product inside fp32's and bf16's normal range.
__device__ __forceinline__ uint32_t shared_quant_exp(uint32_t top) {
  if (top >= 0x7F80u) return 255u;
  if (top == 0u) return 127u;
  const int e = (int)(top >> 7) - 127 - 8 + ((top & 127u) > 96u ? 1 : 0);
  return (uint32_t)(max(e, -100) + 127);
}

struct AppendArgs {
  const __nv_bfloat16* z; long long z_stride;
  const __nv_bfloat16* kr; long long kr_stride;
  const int32_t* seq; const int32_t* pos;
  int n, B, cap, r, dr;
  const float2* rope_cs;
  RowMap map;
  void* c; uint8_t* scale; __nv_bfloat16* kr_pool;
};

template <bool kQuant, int T>
__global__ void __launch_bounds__(32 * kWarps) k_shared_append(const AppendArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int i0 = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * T;
  const int nv = a.r >> 3;                                // 8-element runs, a multiple of 8
  const int half = a.dr >> 1;                             // rotary part: lane j holds the pair (j, j + dr/2)
  const bool has = lane < half;
  int b[T], t[T];
  uint4 w[T][2];
  __nv_bfloat16 x[T][2];
#pragma unroll
  for (int u = 0; u < T; ++u) {
    const int i = i0 + u;
    b[u] = t[u] = -1;
    if (i >= a.n) continue;
    b[u] = __ldg(a.seq + i);
    t[u] = __ldg(a.pos + i);
    const uint4* src = reinterpret_cast<const uint4*>(a.z + (long long)i * a.z_stride);
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (k * 32 + lane < nv) w[u][k] = __ldg(src + k * 32 + lane);
    if (has) {
      const __nv_bfloat16* kr = a.kr + (long long)i * a.kr_stride;
      x[u][0] = kr[lane];
      x[u][1] = kr[half + lane];
    }
  }
#pragma unroll
  for (int u = 0; u < T; ++u) {
    if (b[u] < 0 || b[u] >= a.B || t[u] < 0 || t[u] >= a.cap) continue;   // a padded row: writes nothing
    const long long row = a.map.row(b[u], t[u]);
    const int tok = (int)(row & 127);
    uint8_t* const codes = static_cast<uint8_t*>(a.c) + shared_code_page(row >> 7, a.r);
    uint8_t* const scale = a.scale + shared_scale_page(row >> 7, a.r);
    if (has) {
      float x0 = __bfloat162float(x[u][0]), x1 = __bfloat162float(x[u][1]);
      if (a.rope_cs) {
        const float2 cs = __ldg(a.rope_cs + (long long)t[u] * half + lane);
        const float y0 = x0 * cs.x - x1 * cs.y, y1 = x0 * cs.y + x1 * cs.x;
        x0 = y0;
        x1 = y1;
      }
      __nv_bfloat16* dst = a.kr_pool + row * a.dr;
      dst[lane] = __float2bfloat16_rn(x0);
      dst[half + lane] = __float2bfloat16_rn(x1);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int v = k * 32 + lane;
      const bool in = v < nv;
      if (!kQuant) {
        if (in) reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.c) + row * a.r)[v] = w[u][k];
        continue;
      }
      const uint32_t ww[4] = {w[u][k].x, w[u][k].y, w[u][k].z, w[u][k].w};
      uint32_t top = 0;
      if (in) {
        // magnitudes compared as pairs of bf16 (NaN wins)
        const __nv_bfloat162 m =
            __hmax2_nan(__hmax2_nan(magnitudes(ww[0]), magnitudes(ww[1])), __hmax2_nan(magnitudes(ww[2]), magnitudes(ww[3])));
        const uint32_t mb = *reinterpret_cast<const uint32_t*>(&m);
        top = max(mb & 0xFFFFu, mb >> 16);
      }
      top = warp_max4(top);
      const uint32_t eb = shared_quant_exp(top);
      // 2^-e, twice: the products are exact in bf16, but for some below 2^-126, whose code is 0 anyway
      const uint32_t ib = (254u - min(eb, 247u)) * 0x00800080u;
      const __nv_bfloat162 inv = *reinterpret_cast<const __nv_bfloat162*>(&ib);
      if (in) {
        uint32_t o[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float2 p = __bfloat1622float2(__hmul2(*reinterpret_cast<const __nv_bfloat162*>(&ww[2 * h]), inv));
          const float2 q = __bfloat1622float2(__hmul2(*reinterpret_cast<const __nv_bfloat162*>(&ww[2 * h + 1]), inv));
          const uint32_t lo = __nv_cvt_float2_to_fp8x2(p, __NV_SATFINITE, __NV_E4M3);
          const uint32_t hi = __nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
          o[h] = lo | (hi << 16);
        }
        *reinterpret_cast<uint2*>(codes + shared_code_index(tok, a.r, v * 8)) = make_uint2(o[0], o[1]);
        if ((lane & 3) == 0) scale[shared_scale_index(tok, v >> 2)] = (uint8_t)eb;
      }
    }
  }
}

struct ReadArgs {
  const int32_t* cu; const int32_t* start;
  int B, total, cap, r, dr;
  RowMap map;
  const void* c; const uint8_t* scale; const __nv_bfloat16* kr_pool;
  __nv_bfloat16* z; __nv_bfloat16* kr;
};

// Row i of the packed output belongs to the sequence b with cu[b] <= i < cu[b + 1] and holds
// its token start[b] + i - cu[b].  Each warp finds b by bisection of cu in shared memory.
template <bool kQuant, int T>
__global__ void __launch_bounds__(32 * kWarps) k_shared_read(const ReadArgs a) {
  extern __shared__ int32_t cu_s[];
  pdl_wait();
  pdl_trigger();
  for (int k = threadIdx.x; k <= a.B; k += blockDim.x) cu_s[k] = __ldg(a.cu + k);
  __syncthreads();
  const int lane = threadIdx.x & 31;
  const int i0 = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * T;
  long long found = -1;                         // lane u: the stored row of output row i0 + u, or none
  if (lane < T) {
    const int i = i0 + lane;
    int lo = 0, hi = a.B;                       // the last b in [0, B] with cu[b] <= i
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (cu_s[mid] <= i) lo = mid;
      else hi = mid - 1;
    }
    if (i < a.total && i >= cu_s[0] && lo < a.B) {      // (behind the last sequence: left as it is)
      const long long t = (long long)(a.start ? __ldg(a.start + lo) : 0) + ((long long)i - cu_s[lo]);
      if (t >= 0 && t < a.cap) found = a.map.row(lo, (int)t);
    }
  }
  const int nv = a.r >> 3;
  long long row[T];
  uint4 w[T][2], y[T];                          // latents (bf16) or their codes (x, y) and exponent bytes (z)
#pragma unroll
  for (int u = 0; u < T; ++u) {
    row[u] = __shfl_sync(0xffffffffu, found, u);
    if (row[u] < 0) continue;
    const int tok = (int)(row[u] & 127);
    const uint8_t* const codes = static_cast<const uint8_t*>(a.c) + shared_code_page(row[u] >> 7, a.r);
    const uint8_t* const scale = a.scale + shared_scale_page(row[u] >> 7, a.r);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int v = k * 32 + lane;
      if (v >= nv) continue;
      if (!kQuant) {
        w[u][k] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.c) + row[u] * a.r) + v);
      } else {
        const uint2 q = __ldg(reinterpret_cast<const uint2*>(codes + shared_code_index(tok, a.r, v * 8)));
        w[u][k].x = q.x;
        w[u][k].y = q.y;
        w[u][k].z = __ldg(scale + shared_scale_index(tok, v >> 2));
      }
    }
    if (lane < (a.dr >> 3)) y[u] = __ldg(reinterpret_cast<const uint4*>(a.kr_pool + row[u] * a.dr) + lane);
  }
#pragma unroll
  for (int u = 0; u < T; ++u) {
    if (row[u] < 0) continue;
    const long long i = i0 + u;
    uint4* dst = reinterpret_cast<uint4*>(a.z + i * a.r);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int v = k * 32 + lane;
      if (v >= nv) continue;
      if (!kQuant) {
        dst[v] = w[u][k];
        continue;
      }
      const uint32_t codes[2] = {w[u][k].x, w[u][k].y};
      uint32_t o[4];
      shared_expand<2>(codes, w[u][k].z, o);
      dst[v] = make_uint4(o[0], o[1], o[2], o[3]);
    }
    if (lane < (a.dr >> 3)) reinterpret_cast<uint4*>(a.kr + i * a.dr)[lane] = y[u];
  }
}

__global__ void k_shared_rope(float2* cs, int cap, int half, double log_theta) {
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= (long long)cap * half) return;
  const double ang = (double)(i / half) * exp(-log_theta * (double)(i % half) / (double)half);
  double sn, cn;
  sincos(ang, &sn, &cn);
  cs[i] = make_float2((float)cn, (float)sn);
}

// Bt [W][r] = B [r][W] transposed, in 32 x 32 tiles through shared memory (once, at creation).
__global__ void k_shared_transpose(const __nv_bfloat16* B, __nv_bfloat16* Bt, int r, int W) {
  __shared__ __nv_bfloat16 t[32][33];
  const int x = blockIdx.x * 32, y = blockIdx.y * 32;      // column of W, rank; both multiples of 32
  for (int j = threadIdx.y; j < 32; j += 8) t[j][threadIdx.x] = B[(size_t)(y + j) * W + x + threadIdx.x];
  __syncthreads();
  for (int j = threadIdx.y; j < 32; j += 8) Bt[(size_t)(x + j) * r + y + threadIdx.x] = t[threadIdx.x][j];
}

}  // namespace

cudaError_t launch_shared_transpose(lr_shared* c, cudaStream_t s) {
  const int W = c->desc.n_kv_heads * (c->desc.dim_nope + c->desc.dim_v);
  return launch_serial(k_shared_transpose, dim3(W / 32, c->desc.rank / 32), dim3(32, 8), 0, s,
                       static_cast<const __nv_bfloat16*>(c->B), static_cast<__nv_bfloat16*>(c->Bt), c->desc.rank, W);
}

cudaError_t launch_shared_rope_table(lr_shared* c, cudaStream_t s) {
  const int half = c->desc.dim_rope / 2;
  const long long n = (long long)c->desc.capacity * half;
  return launch_serial(k_shared_rope, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, c->rope_cs, c->desc.capacity,
                       half, log(c->desc.rope_theta));
}

cudaError_t launch_shared_append(lr_shared* c, const void* z, long long z_stride, const void* kr, long long kr_stride,
                                 const int32_t* seq, const int32_t* pos, int n, cudaStream_t s) {
  AppendArgs a;
  a.z = static_cast<const __nv_bfloat16*>(z);
  a.z_stride = z_stride;
  a.kr = static_cast<const __nv_bfloat16*>(kr);
  a.kr_stride = kr_stride;
  a.seq = seq;
  a.pos = pos;
  a.n = n;
  a.B = c->desc.batch;
  a.cap = c->desc.capacity;
  a.r = c->desc.rank;
  a.dr = c->desc.dim_rope;
  a.rope_cs = c->rope_cs;
  a.map = row_map(c);
  a.c = c->c;
  a.scale = c->scale;
  a.kr_pool = static_cast<__nv_bfloat16*>(c->kr);
  const bool many = per_warp(n, c->num_sms) > 1;
  const int per = kWarps * (many ? kMany : 1);
  const dim3 grid((n + per - 1) / per);
  if (many)
    return c->desc.quant_bits ? launch_pdl(k_shared_append<true, kMany>, grid, dim3(32 * kWarps), 0, s, a)
                              : launch_pdl(k_shared_append<false, kMany>, grid, dim3(32 * kWarps), 0, s, a);
  return c->desc.quant_bits ? launch_pdl(k_shared_append<true, 1>, grid, dim3(32 * kWarps), 0, s, a)
                            : launch_pdl(k_shared_append<false, 1>, grid, dim3(32 * kWarps), 0, s, a);
}

cudaError_t launch_shared_read(lr_shared* c, const int32_t* cu, const int32_t* start, int total, void* z, void* kr,
                               cudaStream_t s) {
  ReadArgs a;
  a.cu = cu;
  a.start = start;
  a.B = c->desc.batch;
  a.total = total;
  a.cap = c->desc.capacity;
  a.r = c->desc.rank;
  a.dr = c->desc.dim_rope;
  a.map = row_map(c);
  a.c = c->c;
  a.scale = c->scale;
  a.kr_pool = static_cast<const __nv_bfloat16*>(c->kr);
  a.z = static_cast<__nv_bfloat16*>(z);
  a.kr = static_cast<__nv_bfloat16*>(kr);
  const bool many = per_warp(total, c->num_sms) > 1;
  const int per = kWarps * (many ? kMany : 1);
  const dim3 grid((total + per - 1) / per);
  const size_t smem = (size_t)(a.B + 1) * sizeof(int32_t);
  if (many)
    return c->desc.quant_bits ? launch_pdl(k_shared_read<true, kMany>, grid, dim3(32 * kWarps), smem, s, a)
                              : launch_pdl(k_shared_read<false, kMany>, grid, dim3(32 * kWarps), smem, s, a);
  return c->desc.quant_bits ? launch_pdl(k_shared_read<true, 1>, grid, dim3(32 * kWarps), smem, s, a)
                            : launch_pdl(k_shared_read<false, 1>, grid, dim3(32 * kWarps), smem, s, a);
}
