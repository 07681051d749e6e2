// Internal declarations of the paged-cache operators (page_slots.cu,
// norm_rope.cu, attend_paged.cu, attend_paged_tc.cu).
#pragma once

#include <string>

#include "internal.h"
#include "common.cuh"

namespace dspark {

inline bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline size_t dtype_bytes(int dtype) { return dtype == DSPARK_DTYPE_F32 ? 4 : 2; }
inline bool valid_dtype(int dtype) { return dtype == DSPARK_DTYPE_F32 || dtype == DSPARK_DTYPE_BF16 || dtype == DSPARK_DTYPE_F16; }

// Checks the sizes of a paged cache (not its pointers); 0 or an error code with the message set.
int check_paged_cache(const dspark_paged_cache* c);

// Elements of one layer's K (or V) storage.
inline int64_t paged_layer_elems(const dspark_paged_cache& c) {
    return (int64_t)c.num_pages * c.page_size * c.n_kv * c.head_dim;
}

__device__ __forceinline__ void set_status(int32_t* status, int32_t bits) {
    if (status) atomicOr(status, bits);
}

template <> __device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }

// The longest request an attention call takes: with it every key index and window edge fits 32 bits
// (2^30 keys of the smallest head are more than the GPU's memory).
constexpr int kMaxKeys = 1 << 30;

// Attention over a paged cache: what both kernels take.
struct PagedAttn {
    const void* q; void* out; float* lse;             // q, out [T][nH][hd] with row strides; lse [T][nH] or NULL
    int64_t q_stride, out_stride;                     // elements between tokens
    const void* k; const void* v;                     // this layer's pages
    const int32_t* table; const int32_t* cu; const int32_t* kv_len;
    int32_t* status;
    int T, B, nH, nKv, grp, hd, max_pages, num_pages, page_size, dtype;
    int max_new;
    float scale;
    int causal, window;
};
cudaError_t launch_attend_paged_simt(const PagedAttn& a, cudaStream_t s);
namespace tc {
bool attend_paged_tc_supported(const dspark_paged_cache& c, int n_heads);
int attend_paged_max_batch();
size_t attend_paged_tc_workspace(int hd);
cudaError_t launch_attend_paged_tc(const PagedAttn& a, void* ws, cudaStream_t s);
}  // namespace tc

}  // namespace dspark
