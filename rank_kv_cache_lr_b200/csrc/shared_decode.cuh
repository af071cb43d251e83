// Pieces shared by the two decode kernels of the shared-latent cache (k_shared_decode.cu: one CTA
// per run of tiles; k_shared_pair.cu: two CTAs that split the rank).
#pragma once

#include "shared_internal.cuh"
#include "tc_common.cuh"

namespace {

using tc::drain_wait;
using tc::kLazy;
using tc::kSmemLimit;

constexpr int kSub = 128 * 128;        // 128 tokens x 64 ranks x 2 B (one TMA box)
constexpr int kSlot = 2 * kSub;        // 128 tokens x 128 ranks
constexpr int kScaleBytes = 512;       // 8 bits: exponent bytes of 128 tokens x 4 groups
constexpr int kAuxBytes = 2048;
constexpr int kMaxSlots = 6;
constexpr float kNoMax = -1e30f;       // running max before any visible token (finite: no inf - inf)

struct DecArgs {
  unsigned long long wait_ns;
  const int32_t* row_len;
  RowMap map;
  int B, cap, r, nch, Hq, n_tok, R, HB, X, nslot;
  float scale_log2;
  const uint8_t* codes;
  const uint8_t* scale;
  float* part_o;
  float* part_ml;
  int* err;
};

// The next sequence part of a run: false at its end.  Every role walks its own copy.
struct Seg {
  int b, t0, nt, len;
};
__device__ __forceinline__ bool next_seg(TileRun* run, const DecArgs& p, Seg* s) {
  while (run->left > 0 && run->b < p.B) {
    const int len = shared_len(p.row_len, run->b, p.cap);
    const int nt = ((len + 127) >> 7) - run->tile;
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

// Butterfly reduction of 8 columns over a warp: lane l holds op over all lanes of v[l % 8].
template <bool kMax>
__device__ __forceinline__ float reduce_cols(float (&v)[8], int lane) {
#pragma unroll
  for (int w = 4; w >= 1; w >>= 1) {
    const bool up = (lane & w) != 0;
#pragma unroll
    for (int k = 0; k < w; ++k) {
      const float keep = up ? v[k + w] : v[k];
      const float send = up ? v[k] : v[k + w];
      const float got = __shfl_xor_sync(0xffffffffu, send, w);
      v[k] = kMax ? fmaxf(keep, got) : keep + got;
    }
  }
  float r = v[0];
#pragma unroll
  for (int o = 8; o <= 16; o <<= 1) {
    const float got = __shfl_xor_sync(0xffffffffu, r, o);
    r = kMax ? fmaxf(r, got) : r + got;
  }
  return r;
}

// Two e4m3 codes as bf16 before their scale: a code's sign, exponent and mantissa bits placed in
// a bf16 stand for its value times 2^-120 (subnormals included).  sel picks bytes (i, j) as
// halves with the sign replicated above each (selector bit 3).
template <uint32_t kSel>
__device__ __forceinline__ __nv_bfloat162 place2(uint32_t w) {
  uint32_t a;
  asm("prmt.b32 %0, %1, %1, %2;" : "=r"(a) : "r"(w), "n"(kSel));
  a = (a << 4) & 0x87F087F0u;
  return *reinterpret_cast<const __nv_bfloat162*>(&a);
}
// Sixteen codes of one token (their words in the order in which they are stored), times 2^e, to
// two 16-byte columns of a swizzled row: w.x, w.y to address a0 and w.z, w.w to a1.  e <= 7
// (exponent byte at most 134): 2^(120 + e) is a bf16, so one exact product; kTwo: two products.
template <bool kTwo>
__device__ __forceinline__ void expand16(const uint4& w, uint32_t eb, uint32_t a0, uint32_t a1) {
  // 2^e = 2^(b1 - 127) 2^(b2 - 127) with 120 folded into the first; byte 255 (a group that held a
  // NaN or an infinity) is NaN
  const uint32_t b1 = kTwo ? min(eb + 120u, 254u) : eb + 120u;
  const uint32_t h1 = kTwo && eb == 255u ? 0x7FC07FC0u : b1 * 0x00800080u;
  const uint32_t h2 = (eb + 247u - b1) * 0x00800080u;
  const __nv_bfloat162 s1 = *reinterpret_cast<const __nv_bfloat162*>(&h1);
  const __nv_bfloat162 s2 = *reinterpret_cast<const __nv_bfloat162*>(&h2);
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
  uint32_t o[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    __nv_bfloat162 x = __hmul2(place2<0x9180>(in[k]), s1), y = __hmul2(place2<0xB3A2>(in[k]), s1);
    if (kTwo) {
      x = __hmul2(x, s2);
      y = __hmul2(y, s2);
    }
    o[2 * k] = *reinterpret_cast<const uint32_t*>(&x);
    o[2 * k + 1] = *reinterpret_cast<const uint32_t*>(&y);
  }
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a0), "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3])
               : "memory");
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a1), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
               : "memory");
}
// A warp-uniform value, known as such to the compiler.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

// Expand one 128-rank chunk of a tile by 256 threads (tid): codes in the upper half of the slot
// `dst`, exponent bytes `sc` [128][4], to bf16 boxes; `full`: 128 ranks (else 64); token rows at
// `valid` and beyond, which hold whatever the page held, become 0.
__device__ __forceinline__ void expand_chunk(uint8_t* dst, const uint8_t* sc, int tid, bool full, int valid) {
  // 16 codes a thread and step: 8 (a last chunk of 64 ranks: 4) threads per token row
  const int sh = full ? 3 : 2, steps = full ? 4 : 2;
  const int col = tid & ((1 << sh) - 1), tok0 = tid >> sh, dtok = 256 >> sh;
  uint4 w[4];
  uint32_t eb[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    eb[k] = 127u;
    if (k < steps) {
      w[k] = reinterpret_cast<const uint4*>(dst + kSub)[k * 256 + tid];
      eb[k] = sc[(k * dtok + tok0) * 4 + (col >> 1)];
    }
  }
  // A whole chunk's codes of a token lie where its second box row goes, and a warp holds
  // whole tokens: once its lanes have read, it may write.
  __syncwarp();
  // 128-byte swizzle: 16-byte column v of row tok sits at v ^ (tok % 8), and tok % 8 is
  // the same in every step; the lanes of the second box take their two columns in the
  // other order, so that the eight lanes of a row store to eight different columns
  const bool swap = col >= 4;
  const uint32_t base = ptx::smem_u32(dst + (col >> 2) * kSub + tok0 * 128);
  const uint32_t a0 = base + ((((col & 3) * 2 + swap) ^ (tok0 & 7)) << 4);
  const uint32_t a1 = base + ((((col & 3) * 2 + !swap) ^ (tok0 & 7)) << 4);
  const bool two = __any_sync(0xffffffffu, max(max(eb[0], eb[1]), max(eb[2], eb[3])) > 134u);
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (k < steps) {
      const uint32_t off = k * dtok * 128;
      uint4 x = w[k];
      if (swap) x = make_uint4(w[k].z, w[k].w, w[k].x, w[k].y);
      if (two) expand16<true>(x, eb[k], a0 + off, a1 + off);
      else expand16<false>(x, eb[k], a0 + off, a1 + off);
    }
  if (valid < 128) {                               // rows behind the sequence, as above
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < steps && k * dtok + tok0 >= valid) {
        const uint32_t off = k * dtok * 128;
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(a0 + off), "r"(0) : "memory");
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(a1 + off), "r"(0) : "memory");
      }
  }
}

inline DecArgs dec_args(const lr_shared* c, const int32_t* row_len, int n_tokens, int R, int HB, int X) {
  const lr_shared_desc& d = c->desc;
  DecArgs a;
  a.wait_ns = c->wait_ns;
  a.row_len = row_len;
  a.map = row_map(c);
  a.B = d.batch;
  a.cap = d.capacity;
  a.r = d.rank;
  a.nch = (d.rank + 127) / 128;
  a.Hq = d.n_q_heads;
  a.n_tok = n_tokens;
  a.R = R;
  a.HB = HB;
  a.X = X;
  a.nslot = 0;
  a.scale_log2 = c->scale_log2;
  a.codes = static_cast<const uint8_t*>(c->c);
  a.scale = c->scale;
  a.part_o = c->part_o;
  a.part_ml = c->part_ml;
  a.err = c->dev_err;
  return a;
}

}  // namespace
