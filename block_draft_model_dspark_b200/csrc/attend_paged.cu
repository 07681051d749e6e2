// dspark_attend_paged: attention of each request's new tokens over its pages.
// The entry point, and the CUDA-core kernel for what the tensor-core kernel
// does not take (fp32 caches, head sizes that are no multiple of 64, pages
// whose size is no power of two or below eight).
//
//   out[t, h] = sum_j softmax_j(scale q[t, h] . K[j, g]) V[j, g],  g = h / (nH / nKv)
// over the keys j that query t sees. One warp per (token, query head): 32 keys
// at a time, a lane per key for the scores, then a lane per head dimension for
// the values; one pass with the running maximum and sum in 32 bits.
#include <algorithm>

#include "paged.h"

namespace dspark {
namespace {

constexpr int kWarps = 4;
constexpr int kMaxHd = 256;

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) attend_paged_simt_kernel(PagedAttn P) {
    __shared__ float s_q[kWarps][kMaxHd];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * kWarps + warp;
    pdl_trigger();
    pdl_wait();
    if (w >= (int64_t)P.T * P.nH) return;
    const int t = (int)(w / P.nH), h = (int)(w % P.nH), g = h / P.grp;
    // the request of token t: the last b with cu[b] <= t
    int b = 0, hi = P.B;
    while (hi - b > 1) {
        const int mid = (b + hi) >> 1;
        if (P.cu[mid] <= t) b = mid; else hi = mid;
    }
    const int c0 = P.cu[b], c1 = P.cu[b + 1];
    if (t < c0 || t >= c1) return;                     // a row of no request stays as it was
    int L = P.kv_len[b];
    const int cap = (int)min((int64_t)kMaxKeys, (int64_t)P.max_pages * P.page_size);
    if (L < 0 || L > cap) {
        if (lane == 0) set_status(P.status, DSPARK_DEV_BAD_LENGTH);
        L = min(max(L, 0), cap);
    }
    const int pos = L - (c1 - c0) + (t - c0);          // the query's own key
    const int end = P.causal ? min(L, pos + 1) : L;
    const int begin = P.window > 0 ? max(0, pos - P.window + 1) : 0;
    const T* q = static_cast<const T*>(P.q) + t * P.q_stride + (int64_t)h * P.hd;
    for (int d = lane; d < P.hd; d += 32) s_q[warp][d] = to_f(q[d]) * P.scale;
    __syncwarp();
    const T* K = static_cast<const T*>(P.k);
    const T* V = static_cast<const T*>(P.v);
    float acc[kMaxHd / 32];
#pragma unroll
    for (int i = 0; i < kMaxHd / 32; ++i) acc[i] = 0.f;
    float m = -INFINITY, l = 0.f;
    for (int j0 = begin; j0 < end; j0 += 32) {
        const int j = j0 + lane;
        int64_t row = -1;                              // row of the pages; -1: no key, or a page outside the pool
        float s = -INFINITY;
        if (j < end) {
            const int page = P.table[(int64_t)b * P.max_pages + j / P.page_size];
            s = 0.f;
            if (page < 0 || page >= P.num_pages) {
                set_status(P.status, DSPARK_DEV_BAD_PAGE);
            } else {
                row = (int64_t)page * P.page_size + j % P.page_size;
                const T* kr = K + (row * P.nKv + g) * P.hd;
                for (int d = 0; d < P.hd; ++d) s = fmaf(s_q[warp][d], to_f(kr[d]), s);
            }
        }
        float mx = s;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float mn = fmaxf(m, mx);
        const float at = mn == -INFINITY ? 0.f : mn;   // (scores of -infinity alone so far: weights 0; a NaN: a sum that is none)
        const float f = __expf(m - at), p = __expf(s - at);
        m = mn;
        l = l * f + warp_sum(p);
#pragma unroll
        for (int i = 0; i < kMaxHd / 32; ++i) acc[i] *= f;
        const int cnt = min(32, end - j0);
        for (int jj = 0; jj < cnt; ++jj) {
            const float pj = __shfl_sync(0xffffffffu, p, jj);
            const int64_t r = __shfl_sync(0xffffffffu, row, jj);
            if (r < 0) continue;
            const T* vr = V + (r * P.nKv + g) * P.hd;
#pragma unroll
            for (int i = 0; i < kMaxHd / 32; ++i)
                if (lane + 32 * i < P.hd) acc[i] = fmaf(pj, to_f(vr[lane + 32 * i]), acc[i]);
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;        // a query that sees no key: zeros, lse -infinity
    T* o = static_cast<T*>(P.out) + t * P.out_stride + (int64_t)h * P.hd;
#pragma unroll
    for (int i = 0; i < kMaxHd / 32; ++i)
        if (lane + 32 * i < P.hd) o[lane + 32 * i] = from_f<T>(acc[i] * inv);
    if (P.lse && lane == 0) P.lse[(int64_t)t * P.nH + h] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace

cudaError_t launch_attend_paged_simt(const PagedAttn& a, cudaStream_t s) {
    const int64_t warps = (int64_t)a.T * a.nH;
    const dim3 grid((unsigned)((warps + kWarps - 1) / kWarps)), block(kWarps * 32);
    return a.dtype == DSPARK_DTYPE_F32 ? launch_pdl(attend_paged_simt_kernel<float>, grid, block, 0, s, a)
         : a.dtype == DSPARK_DTYPE_F16 ? launch_pdl(attend_paged_simt_kernel<__half>, grid, block, 0, s, a)
                                       : launch_pdl(attend_paged_simt_kernel<__nv_bfloat16>, grid, block, 0, s, a);
}

}  // namespace dspark

using namespace dspark;

extern "C" size_t dspark_attend_paged_workspace_bytes(const dspark_paged_cache* c, int32_t T, int32_t n_heads, int32_t B) {
    if (check_paged_cache(c) != DSPARK_OK || T < 0 || n_heads < 1 || B < 0) return 0;
    return tc::attend_paged_tc_supported(*c, n_heads) ? tc::attend_paged_tc_workspace(c->head_dim) : 256;
}

extern "C" int dspark_attend_paged(const dspark_paged_cache* c, int32_t layer, const void* q, int64_t q_stride,
                                   int32_t n_heads, const int32_t* cu_new, const int32_t* kv_len, int32_t B, int32_t T,
                                   int32_t max_new, float scale, int32_t causal, int32_t window, void* out,
                                   int64_t out_stride, float* lse, void* ws, size_t ws_bytes, void* stream) {
    const int rc = check_paged_cache(c);
    if (rc != DSPARK_OK) return rc;
    if (layer < 0 || layer >= c->layers) DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "layer out of range");
    if (n_heads < 1 || n_heads % c->n_kv != 0)
        DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "n_heads must be a positive multiple of the cache's n_kv");
    if (B < 0 || B > c->batch) DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "B must be in [0, cache.batch]");
    if (B > tc::attend_paged_max_batch()) DSPARK_FAIL(DSPARK_ERR_UNSUPPORTED, "more than 4096 requests in one call");
    if (T < 0 || max_new < 0) DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "T and max_new must be >= 0");
    if (!(scale > 0.f) || scale > 3.0e38f) DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "scale must be positive and finite");
    if (window < 0) DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "window must be >= 0 (0: none)");
    if (T == 0 || B == 0) return DSPARK_OK;
    if (!c->k || !c->v || !q || !out || !cu_new || !kv_len || !ws)
        DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "cache.k, cache.v, q, out, cu_new, kv_len and ws must be non-NULL");
    const size_t es = dtype_bytes(c->dtype);
    if (!aligned_to(q, 16) || !aligned_to(out, 16) || !aligned_to(c->k, 16) || !aligned_to(c->v, 16) || !aligned_to(ws, 256))
        DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "q, out and the cache must be 16-byte aligned, ws 256-byte aligned");
    if ((q_stride * (int64_t)es) % 16 || (out_stride * (int64_t)es) % 16 || q_stride < 0 || out_stride < 0)
        DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "the token strides of q and out must be non-negative multiples of 16 bytes");
    const int64_t row = (int64_t)n_heads * c->head_dim;
    if (T > 1 && (q_stride < row || out_stride < row))
        DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "the token strides of q and out must be at least n_heads * head_dim");
    if (q_stride >= ((int64_t)1 << 38)) DSPARK_FAIL(DSPARK_ERR_UNSUPPORTED, "q_stride at or above 2^38");
    if ((int64_t)T * n_heads > ((int64_t)1 << 31) - 1) DSPARK_FAIL(DSPARK_ERR_UNSUPPORTED, "T * n_heads above 2^31 - 1");
    if (ws_bytes < dspark_attend_paged_workspace_bytes(c, T, n_heads, B))
        DSPARK_FAIL(DSPARK_ERR_WORKSPACE, "ws smaller than dspark_attend_paged_workspace_bytes()");
    PagedAttn a{};
    a.q = q; a.out = out; a.lse = lse; a.q_stride = T > 1 ? q_stride : row; a.out_stride = T > 1 ? out_stride : row;
    const size_t layer_bytes = (size_t)paged_layer_elems(*c) * es * layer;
    a.k = static_cast<const char*>(c->k) + layer_bytes;
    a.v = static_cast<const char*>(c->v) + layer_bytes;
    a.table = c->block_table; a.cu = cu_new; a.kv_len = kv_len; a.status = c->status;
    a.T = T; a.B = B; a.nH = n_heads; a.nKv = c->n_kv; a.grp = n_heads / c->n_kv; a.hd = c->head_dim;
    a.max_pages = c->max_pages; a.num_pages = c->num_pages; a.page_size = c->page_size; a.dtype = c->dtype;
    a.max_new = max_new; a.scale = scale; a.causal = causal != 0;
    a.window = window >= std::min((int64_t)kMaxKeys, (int64_t)c->max_pages * c->page_size) ? 0 : window;   // wider than any request: none
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = tc::attend_paged_tc_supported(*c, n_heads) ? tc::launch_attend_paged_tc(a, ws, s) : launch_attend_paged_simt(a, s);
    if (e != cudaSuccess) DSPARK_FAIL(DSPARK_ERR_CUDA, std::string("paged attention launch: ") + cudaGetErrorString(e));
    return DSPARK_OK;
}
