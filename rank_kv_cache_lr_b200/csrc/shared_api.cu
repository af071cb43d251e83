// Host layer of the shared-latent calls (lr_shared_* in include/lr_kv.h): validation, lifetime
// and launches.
#include "shared_internal.cuh"

#include <algorithm>
#include <cmath>
#include <new>

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31) == 0; }

// Makes the cache's device current for a call and restores the caller's afterwards.
struct OnDevice {
  int before = -1;
  bool ok = true;
  explicit OnDevice(int dev) {
    ok = cudaGetDevice(&before) == cudaSuccess && (before == dev || cudaSetDevice(dev) == cudaSuccess);
    if (before == dev) before = -1;
  }
  ~OnDevice() {
    if (before >= 0) cudaSetDevice(before);
  }
};

lr_status validate(const lr_shared_desc* d) {
  if (!d) return LR_ERR_INVALID_ARG;
  if (d->batch < 1 || d->n_q_heads < 1 || d->n_kv_heads < 1 || d->capacity < 1) return LR_ERR_INVALID_ARG;
  if (d->n_q_heads % d->n_kv_heads) return LR_ERR_INVALID_ARG;
  if (d->quant_bits != 0 && d->quant_bits != 8) return LR_ERR_INVALID_ARG;
  if (d->dtype != LR_F32 && d->dtype != LR_BF16) return LR_ERR_INVALID_ARG;
  if (d->rank < 64 || d->rank % 64 || d->rank > 512) return LR_ERR_INVALID_ARG;
  if ((d->dim_nope != 64 && d->dim_nope != 128) || (d->dim_v != 64 && d->dim_v != 128) ||
      (d->dim_rope != 32 && d->dim_rope != 64))
    return LR_ERR_INVALID_ARG;
  if (d->capacity % kPageTokens || d->capacity > (1 << 24)) return LR_ERR_INVALID_ARG;
  if (d->n_pages < 0 || d->n_pages > (1 << 22)) return LR_ERR_INVALID_ARG;
  if (d->n_pages == 0 && (long long)d->batch * (d->capacity / kPageTokens) > (1 << 22)) return LR_ERR_INVALID_ARG;
  if (d->max_queries < 1) return LR_ERR_INVALID_ARG;
  if (!(d->rope_theta >= 0.0) || std::isinf(d->rope_theta)) return LR_ERR_INVALID_ARG;
  if (!(d->softmax_scale >= 0.0f) || std::isinf(d->softmax_scale)) return LR_ERR_INVALID_ARG;
  for (int32_t r : d->reserved)
    if (r != 0) return LR_ERR_INVALID_ARG;
  if (d->dtype != LR_BF16) return LR_ERR_UNSUPPORTED;
  if (d->n_q_heads > 128 || d->batch > 1024 || d->max_queries > 8) return LR_ERR_UNSUPPORTED;
  return LR_OK;
}

template <typename T>
cudaError_t dalloc(T** p, size_t bytes, bool zero) {
  *p = nullptr;
  if (bytes == 0) return cudaSuccess;
  cudaError_t e = lr_dev_malloc((void**)p, bytes);
  if (e == cudaSuccess && zero) e = cudaMemset(*p, 0, bytes);
  return e;
}

void free_all(lr_shared* c) {
  void* ptrs[] = {c->c, c->scale, c->kr, c->table, c->B, c->Bt, c->rope_cs, c->qt, c->part_o, c->part_ml, c->dev_err};
  for (void* p : ptrs)
    if (p) cudaFree(p);
}

lr_status status_of(cudaError_t e) {
  if (e == cudaSuccess) return LR_OK;
  if (e == cudaErrorMemoryAllocation) return LR_ERR_OOM;
  if (e == cudaErrorNotSupported) return LR_ERR_UNSUPPORTED;
  return LR_ERR_CUDA;
}

}  // namespace

extern "C" {

lr_status lr_shared_create(const lr_shared_desc* desc, const void* B_k, const void* B_v, void* stream,
                           lr_shared** out) {
  if (!out) return LR_ERR_INVALID_ARG;
  *out = nullptr;
  const lr_status st = validate(desc);
  if (st != LR_OK) return st;
  if (!B_k || !B_v) return LR_ERR_INVALID_ARG;
  lr_shared* c = new (std::nothrow) lr_shared();
  if (!c) return LR_ERR_OOM;
  c->desc = *desc;
  const lr_shared_desc& d = c->desc;
  c->pps = d.capacity / kPageTokens;
  c->n_pages = d.n_pages ? d.n_pages : d.batch * c->pps;
  const float scale = d.softmax_scale > 0.f ? d.softmax_scale : 1.0f / std::sqrt((float)(d.dim_nope + d.dim_rope));
  c->scale_log2 = scale * LR_LOG2E;
  c->last_stream = (cudaStream_t)stream;
  cudaError_t e = cudaGetDevice(&c->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&c->num_sms, cudaDevAttrMultiProcessorCount, c->device);
  const size_t rows = (size_t)c->n_pages * kPageTokens, r = d.rank;
  const size_t wk = (size_t)d.n_kv_heads * d.dim_nope * 2, wv = (size_t)d.n_kv_heads * d.dim_v * 2;   // bytes a basis row
  cudaStream_t s = (cudaStream_t)stream;
  if (e == cudaSuccess) e = dalloc(&c->c, rows * r * (d.quant_bits ? 1 : 2), true);
  if (e == cudaSuccess && d.quant_bits) e = dalloc(&c->scale, rows * ((r + 127) / 128) * 4, true);
  if (e == cudaSuccess) e = dalloc(&c->kr, rows * d.dim_rope * 2, true);
  if (e == cudaSuccess) e = dalloc(&c->table, (size_t)d.batch * c->pps * sizeof(int32_t), false);
  if (e == cudaSuccess) e = dalloc(&c->B, r * (wk + wv), false);
  if (e == cudaSuccess) e = dalloc(&c->Bt, r * (wk + wv), false);
  if (e == cudaSuccess && d.rope_theta > 0.0)
    e = dalloc(&c->rope_cs, (size_t)d.capacity * (d.dim_rope / 2) * sizeof(float2), false);
  if (e == cudaSuccess) e = dalloc(&c->qt, shared_qt_bytes(&d), true);
  size_t prows = 0;
  shared_part_rows(&d, c->num_sms, &prows);
  if (e == cudaSuccess) e = dalloc(&c->part_o, prows * r * sizeof(float), false);
  if (e == cudaSuccess) e = dalloc(&c->part_ml, prows * 2 * sizeof(float), false);
  if (e == cudaSuccess) e = dalloc(&c->dev_err, sizeof(int), true);
  if (e == cudaSuccess) {
    // span j of sequence b in page (b * pps + j) % n_pages until a table is set
    try {
      c->host_table.resize((size_t)d.batch * c->pps);
    } catch (...) {
      e = cudaErrorMemoryAllocation;
    }
    for (size_t i = 0; i < c->host_table.size(); ++i) c->host_table[i] = (int32_t)(i % (size_t)c->n_pages);
  }
  if (e == cudaSuccess)
    e = cudaMemcpy(c->table, c->host_table.data(), c->host_table.size() * sizeof(int32_t), cudaMemcpyHostToDevice);
  if (e == cudaSuccess) e = cudaMemcpy2DAsync(c->B, wk + wv, B_k, wk, wk, r, cudaMemcpyDeviceToDevice, s);
  if (e == cudaSuccess)
    e = cudaMemcpy2DAsync(static_cast<char*>(c->B) + wk, wk + wv, B_v, wv, wv, r, cudaMemcpyDeviceToDevice, s);
  if (e == cudaSuccess) e = shared_decode_maps(c);
  if (e == cudaSuccess) e = shared_expand_maps(c);
  if (e == cudaSuccess) e = launch_shared_transpose(c, s);
  if (e == cudaSuccess && c->rope_cs) e = launch_shared_rope_table(c, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(cudaStreamLegacy);   // the fills above
  if (e != cudaSuccess) {
    free_all(c);
    delete c;
    return status_of(e);
  }
  *out = c;
  return LR_OK;
}

lr_status lr_shared_destroy(lr_shared* c) {
  if (!c) return LR_OK;
  cudaError_t e;
  {
    OnDevice dev(c->device);
    e = cudaDeviceSynchronize();
    free_all(c);
  }
  delete c;
  return e == cudaSuccess ? LR_OK : LR_ERR_CUDA;
}

lr_status lr_shared_set_block_table(lr_shared* c, const int32_t* table, void* stream) {
  if (!c || !table) return LR_ERR_INVALID_ARG;
  const size_t n = (size_t)c->desc.batch * c->pps;
  for (size_t i = 0; i < n; ++i)
    if (table[i] < 0 || table[i] >= c->n_pages) return LR_ERR_INVALID_ARG;
  OnDevice dev(c->device);
  if (!dev.ok) return LR_ERR_CUDA;
  std::copy(table, table + n, c->host_table.begin());   // pageable: staged before the copy call returns
  c->last_stream = (cudaStream_t)stream;
  const cudaError_t e = cudaMemcpyAsync(c->table, c->host_table.data(), n * sizeof(int32_t), cudaMemcpyHostToDevice,
                                        (cudaStream_t)stream);
  return e == cudaSuccess ? LR_OK : LR_ERR_CUDA;
}

lr_status lr_shared_set_block_table_device(lr_shared* c, const int32_t* table, void* stream) {
  if (!c || !table) return LR_ERR_INVALID_ARG;
  OnDevice dev(c->device);
  if (!dev.ok) return LR_ERR_CUDA;
  c->last_stream = (cudaStream_t)stream;
  const cudaError_t e = cudaMemcpyAsync(c->table, table, (size_t)c->desc.batch * c->pps * sizeof(int32_t),
                                        cudaMemcpyDeviceToDevice, (cudaStream_t)stream);
  return e == cudaSuccess ? LR_OK : LR_ERR_CUDA;
}

lr_status lr_shared_append(lr_shared* c, const void* z, int64_t z_stride, const void* kr, int64_t kr_stride,
                           const int32_t* seq, const int32_t* pos, int32_t n, void* stream) {
  if (!c || n < 0) return LR_ERR_INVALID_ARG;
  if (n == 0) return LR_OK;
  if (!z || !kr || !seq || !pos) return LR_ERR_INVALID_ARG;
  if (!aligned16(z) || z_stride % 8 || (n > 1 && z_stride < c->desc.rank) || (n > 1 && kr_stride < c->desc.dim_rope))
    return LR_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(kr) & 1) return LR_ERR_INVALID_ARG;
  OnDevice dev(c->device);
  if (!dev.ok) return LR_ERR_CUDA;
  c->last_stream = (cudaStream_t)stream;
  return status_of(launch_shared_append(c, z, z_stride, kr, kr_stride, seq, pos, n, (cudaStream_t)stream));
}

lr_status lr_shared_read(lr_shared* c, const int32_t* cu, const int32_t* start, int32_t total, void* z, void* kr,
                         void* stream) {
  if (!c || total < 0) return LR_ERR_INVALID_ARG;
  if (total == 0) return LR_OK;
  if (!cu || !z || !kr || !aligned16(z) || !aligned16(kr)) return LR_ERR_INVALID_ARG;
  OnDevice dev(c->device);
  if (!dev.ok) return LR_ERR_CUDA;
  c->last_stream = (cudaStream_t)stream;
  return status_of(launch_shared_read(c, cu, start, total, z, kr, (cudaStream_t)stream));
}

lr_status lr_shared_decode(lr_shared* c, const void* q, int32_t n_tokens, const int32_t* row_len, void* out,
                           float* lse, void* stream) {
  if (!c || !q || !row_len || !out || n_tokens < 1) return LR_ERR_INVALID_ARG;
  if (!aligned16(q)) return LR_ERR_INVALID_ARG;
  if (n_tokens > c->desc.max_queries) return LR_ERR_CAPACITY;
  OnDevice dev(c->device);
  if (!dev.ok) return LR_ERR_CUDA;
  c->last_stream = (cudaStream_t)stream;
  return status_of(launch_shared_decode(c, q, n_tokens, row_len, out, lse, (cudaStream_t)stream));
}

lr_status lr_shared_expand(lr_shared* c, const int32_t* cu, const int32_t* start, int32_t total, void* k, void* v,
                           void* kr, void* stream) {
  if (!c || total < 0) return LR_ERR_INVALID_ARG;
  if (total == 0) return LR_OK;
  if (!cu || !k || !v || !kr || !aligned16(kr) || !aligned32(k) || !aligned32(v)) return LR_ERR_INVALID_ARG;
  OnDevice dev(c->device);
  if (!dev.ok) return LR_ERR_CUDA;
  c->last_stream = (cudaStream_t)stream;
  return status_of(launch_shared_expand(c, cu, start, total, k, v, kr, (cudaStream_t)stream));
}

lr_status lr_shared_attn(lr_shared* c, const void* q, const void* k, const void* kr, const void* v,
                         const int32_t* cu_q, const int32_t* cu_k, int32_t n_seq, int32_t total_q, int32_t total_k,
                         int32_t causal, void* out, float* lse, void* stream) {
  if (!c || n_seq < 0 || total_q < 0 || total_k < 0 || (causal != 0 && causal != 1)) return LR_ERR_INVALID_ARG;
  if (n_seq > 1024) return LR_ERR_UNSUPPORTED;
  if (n_seq == 0 || total_q == 0) return LR_OK;
  if (!q || !cu_q || !cu_k || !out || (total_k > 0 && (!k || !kr || !v))) return LR_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(kr) || !aligned16(v) || !aligned32(out)) return LR_ERR_INVALID_ARG;
  OnDevice dev(c->device);
  if (!dev.ok) return LR_ERR_CUDA;
  c->last_stream = (cudaStream_t)stream;
  return status_of(launch_shared_attn(c, q, k, kr, v, cu_q, cu_k, n_seq, total_q, total_k, causal, out, lse,
                                      (cudaStream_t)stream));
}

lr_status lr_shared_set_wait_limit(lr_shared* c, int64_t ns) {
  if (!c || ns < 0) return LR_ERR_INVALID_ARG;
  c->wait_ns = (unsigned long long)ns;
  return LR_OK;
}

lr_status lr_shared_device_error(lr_shared* c, int32_t* code) {
  if (!c || !code) return LR_ERR_INVALID_ARG;
  OnDevice dev(c->device);
  if (!dev.ok) return LR_ERR_CUDA;
  cudaError_t e = cudaStreamSynchronize(c->last_stream);
  if (e != cudaSuccess) return LR_ERR_CUDA;
  int h = 0;
  e = cudaMemcpy(&h, c->dev_err, sizeof(int), cudaMemcpyDeviceToHost);
  if (e == cudaSuccess) e = cudaMemset(c->dev_err, 0, sizeof(int));
  *code = h;
  return e == cudaSuccess ? LR_OK : LR_ERR_CUDA;
}

int32_t lr_shared_desc_size(void) { return (int32_t)sizeof(lr_shared_desc); }

}  // extern "C"
