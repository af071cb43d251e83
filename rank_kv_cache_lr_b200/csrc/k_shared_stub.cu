#include "shared_internal.cuh"
cudaError_t launch_shared_expand(lr_shared*, const int32_t*, const int32_t*, int, void*, void*, void*, cudaStream_t) { return cudaErrorNotSupported; }
cudaError_t launch_shared_attn(lr_shared*, const void*, const void*, const void*, const void*, const int32_t*, const int32_t*, int, int, int, int, void*, float*, cudaStream_t) { return cudaErrorNotSupported; }
