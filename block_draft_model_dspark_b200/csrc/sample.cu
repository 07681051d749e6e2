// dspark_sample: one token per row of logits by temperature, top-k, top-p and
// min-p from a given uniform number.
//
// With m the row's maximum and w_i = exp((x_i - m) / T), every filter keeps a
// prefix of the candidates in falling order (equal logits: the lower index
// first): top-k its first k; top-p, of those, the shortest prefix whose mass
// reaches p of theirs; min-p those with w_i >= min_p. The token is the first
// index i (in the vocabulary's order) whose cumulative kept mass exceeds
// u times the total.
//
// Weights are computed in 64 bits and summed as 64-bit fixed-point numbers (at
// 2^61 over a power of two above their sum): in a flat tail a token's share is
// about 10^-7 of the mass, so 32-bit sums would move the drawn token; integer
// sums are also the same in whatever order they are added.
#include "paged.h"

namespace dspark {
namespace {

constexpr int kThreads = 1024;
constexpr int kBins = 2048;

struct SampleParams {
    const void* logits; int64_t stride; int dtype, rows, V;
    const float* u; const float* temperature; const int32_t* top_k; const float* top_p; const float* min_p;
    int32_t* tokens; float* probs;
};

__device__ __forceinline__ float load_logit(const void* p, int64_t i, int dtype) {
    const float x = load_any(p, i, dtype);
    return x != x ? -INFINITY : x + 0.f;            // NaN counts as -infinity, -0 as 0
}
// Bits in the order of the values.
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t b = __float_as_uint(x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

struct Weights {
    double m, inv_t, scale;
    __device__ __forceinline__ double weight(float x) const {
        return (double)x == m ? 1.0 : exp(((double)x - m) * inv_t);
    }
    __device__ __forceinline__ uint64_t fixed(float x) const { return (uint64_t)__double2ull_rn(weight(x) * scale); }
};

template <typename T, typename Op>
__device__ __forceinline__ T block_reduce(T v, T* buf, Op op) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if (lane == 0) buf[wid] = v;
    __syncthreads();
    v = buf[lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
// Exclusive sum over the block's threads in order; *total gets the sum.
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* buf, uint64_t* total) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    uint64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) buf[wid] = x;
    __syncthreads();
    uint64_t wv = buf[lane], ws = wv;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, ws, o);
        if (lane >= o) ws += y;
    }
    *total = __shfl_sync(0xffffffffu, ws, 31);
    return __shfl_sync(0xffffffffu, ws - wv, wid) + x - v;
}

struct Hist {
    uint32_t cnt[kBins], lo[kBins], hi[kBins];      // elements, and their fixed-point mass
};

// A prefix of the falling order: every key above `key`, and the first `ties` of `key`.
struct Cut {
    uint32_t key;
    uint32_t ties;
    uint64_t above;                                 // fixed-point mass of the keys above
};

// The prefix that ends at the element where, from the top, `stop` first holds: by_count: the
// count reaches k; else: the mass before the next element is no longer below `mass`. `limit`
// bounds the elements looked at (a prefix found before).
__device__ Cut find_cut(const void* row, const SampleParams& P, const Weights& W, Hist& H, bool by_count, uint32_t k,
                        double mass, const Cut* limit, uint64_t* buf) {
    __shared__ uint32_t s_bin;
    __shared__ uint64_t s_above;
    __shared__ uint32_t s_cnt;
    const int tid = threadIdx.x;
    uint32_t prefix = 0, above_cnt = 0;
    uint64_t above = 0;
    const int shifts[3] = {21, 10, 0};
    uint32_t in_bin = 0;
    for (int level = 0; level < 3; ++level) {
        const int shift = shifts[level], bins = level == 2 ? 1024 : 2048;
        for (int i = tid; i < kBins; i += kThreads) H.cnt[i] = H.lo[i] = H.hi[i] = 0;
        __syncthreads();
        for (int i = tid; i < P.V; i += kThreads) {
            const float x = load_logit(row, i, P.dtype);
            const uint32_t key = order_key(x);
            if (level > 0 && (key >> (level == 1 ? 21 : 10)) != prefix) continue;
            if (limit && key < limit->key) continue;
            const uint32_t b = (key >> shift) & (bins - 1);
            atomicAdd(&H.cnt[b], 1u);
            const uint64_t f = W.fixed(x);
            const uint32_t lo = (uint32_t)f, old = atomicAdd(&H.lo[b], lo);
            const uint32_t hi = (uint32_t)(f >> 32) + (old + lo < old ? 1u : 0u);
            if (hi) atomicAdd(&H.hi[b], hi);
        }
        __syncthreads();
        if (tid == 0) s_bin = 0xffffffffu;
        // two bins per thread, from the top
        const int b0 = kBins - 1 - 2 * tid, b1 = b0 - 1;
        const uint32_t c0 = H.cnt[b0], c1 = H.cnt[b1];
        const uint64_t m0 = ((uint64_t)H.hi[b0] << 32) + H.lo[b0], m1 = ((uint64_t)H.hi[b1] << 32) + H.lo[b1];
        uint64_t tc, tm;
        const uint64_t pc = block_scan((uint64_t)c0 + c1, buf, &tc), pm = block_scan(m0 + m1, buf, &tm);
        auto crosses = [&](uint64_t c_before, uint32_t c, uint64_t m_before, uint64_t m) {
            if (c == 0) return false;
            if (by_count) return above_cnt + c_before < k && above_cnt + c_before + c >= k;
            // the boundary element lies in the last bin whose start is still below the mass
            return (double)(above + m_before) < mass && !((double)(above + m_before + m) < mass);
        };
        if (crosses(pc, c0, pm, m0)) { s_bin = b0; s_above = above + pm; s_cnt = above_cnt + (uint32_t)pc; }
        if (crosses(pc + c0, c1, pm + m0, m1)) { s_bin = b1; s_above = above + pm + m0; s_cnt = above_cnt + (uint32_t)pc + c0; }
        __syncthreads();
        if (s_bin == 0xffffffffu) return Cut{0u, 0xffffffffu, 0};    // no element crosses: everything stays
        const uint32_t bin = s_bin;
        above = s_above;
        above_cnt = s_cnt;
        in_bin = H.cnt[bin];
        prefix = level == 0 ? bin : (prefix << (level == 1 ? 11 : 10)) | bin;
        __syncthreads();
    }
    Cut c{prefix, 1u, above};
    if (limit && prefix == limit->key) in_bin = min(in_bin, limit->ties);
    if (by_count) {
        c.ties = k - above_cnt;
    } else {
        // ties i = 0, 1, .. stay while the mass before them is below `mass`
        const uint64_t f = W.fixed(key_value(prefix));
        uint32_t lo = 0, hi = in_bin;                                // the largest n <= in_bin with tie n - 1 staying
        while (lo < hi) {
            const uint32_t mid = (lo + hi + 1) >> 1;
            if ((double)(above + (uint64_t)(mid - 1) * f) < mass) lo = mid; else hi = mid - 1;
        }
        c.ties = max(lo, 1u);
    }
    return c;
}

__global__ void __launch_bounds__(kThreads) sample_kernel(SampleParams P) {
    __shared__ Hist H;
    __shared__ uint64_t buf[32];
    __shared__ int s_token;
    __shared__ uint64_t s_weight;
    const int tid = threadIdx.x, r = blockIdx.x;
    pdl_trigger();
    pdl_wait();
    const void* row = static_cast<const char*>(P.logits) + (int64_t)r * P.stride * (P.dtype == DSPARK_DTYPE_F32 ? 4 : 2);
    uint32_t best = 0;
    for (int i = tid; i < P.V; i += kThreads) best = max(best, order_key(load_logit(row, i, P.dtype)));
    best = block_reduce(best, reinterpret_cast<uint32_t*>(buf), [](uint32_t a, uint32_t b) { return max(a, b); });
    const float mx = key_value(best);
    if (mx == -INFINITY) {                                            // nothing to choose from
        if (tid == 0) { P.tokens[r] = -1; if (P.probs) P.probs[r] = 0.f; }
        return;
    }
    const float T = P.temperature ? P.temperature[r] : 1.f;
    if (!(T > 0.f)) {                                                 // greedy
        int at = 0x7fffffff;
        for (int i = tid; i < P.V; i += kThreads)
            if (load_logit(row, i, P.dtype) == mx) at = min(at, i);
        at = block_reduce(at, reinterpret_cast<int*>(buf), [](int a, int b) { return min(a, b); });
        if (tid == 0) { P.tokens[r] = at; if (P.probs) P.probs[r] = 1.f; }
        return;
    }
    Weights W{(double)mx, 1.0 / (double)T, 1.0};
    float z = 0.f;
    for (int i = tid; i < P.V; i += kThreads) z += (float)W.weight(load_logit(row, i, P.dtype));
    z = block_reduce(z, reinterpret_cast<float*>(buf), [](float a, float b) { return a + b; });
    int e;
    frexpf(z * 1.001f, &e);                                           // z < 2^e
    W.scale = ldexp(1.0, 61 - e);

    Cut cut{0u, 0xffffffffu, 0};                                      // everything
    const int k = P.top_k ? P.top_k[r] : 0;
    if (k > 0 && k < P.V) cut = find_cut(row, P, W, H, true, (uint32_t)k, 0.0, nullptr, buf);
    const float p = P.top_p ? P.top_p[r] : 1.f;
    if (p <= 0.f) cut = Cut{best, 1u, 0};
    else if (p < 1.f) {
        uint64_t total, mine = 0;
        for (int i = tid; i < P.V; i += kThreads) {
            const float x = load_logit(row, i, P.dtype);
            if (order_key(x) > cut.key || cut.ties == 0xffffffffu) mine += W.fixed(x);
        }
        block_scan(mine, buf, &total);
        if (cut.ties != 0xffffffffu) total += (uint64_t)cut.ties * W.fixed(key_value(cut.key));
        const Cut by_mass = find_cut(row, P, W, H, false, 0u, (double)p * (double)total,
                                     cut.ties == 0xffffffffu ? nullptr : &cut, buf);
        if (by_mass.ties != 0xffffffffu) cut = by_mass;
    }
    const double low = P.min_p ? (double)P.min_p[r] : 0.0;
    // a contiguous piece of the vocabulary per thread: its ties, then its kept mass
    const int per = (P.V + kThreads - 1) / kThreads, i0 = min(P.V, tid * per), i1 = min(P.V, i0 + per);
    uint64_t ties = 0, all;
    if (cut.ties != 0xffffffffu)
        for (int i = i0; i < i1; ++i) ties += order_key(load_logit(row, i, P.dtype)) == cut.key;
    const uint64_t tie0 = block_scan(ties, buf, &all);
    auto kept = [&](float x, uint64_t* tie) {
        const uint32_t key = order_key(x);
        if (key < cut.key) return false;
        if (key == cut.key && (*tie)++ >= cut.ties) return false;
        return W.weight(x) >= low || key == best;
    };
    uint64_t mass = 0, tie = tie0, total;
    int last = -1;
    for (int i = i0; i < i1; ++i) {
        const float x = load_logit(row, i, P.dtype);
        if (kept(x, &tie)) { mass += W.fixed(x); last = i; }
    }
    uint64_t cum = block_scan(mass, buf, &total);
    last = block_reduce(last, reinterpret_cast<int*>(buf), [](int a, int b) { return max(a, b); });
    if (tid == 0) { s_token = last; s_weight = 0; }
    __syncthreads();
    const double want = (double)P.u[r] * (double)total;
    if (mass > 0 && !((double)cum > want) && (double)(cum + mass) > want) {
        tie = tie0;
        for (int i = i0; i < i1; ++i) {
            const float x = load_logit(row, i, P.dtype);
            if (!kept(x, &tie)) continue;
            cum += W.fixed(x);
            if ((double)cum > want) { s_token = i; break; }
        }
    }
    __syncthreads();
    if (tid == 0) {
        P.tokens[r] = s_token;
        if (P.probs) P.probs[r] = (float)(W.weight(load_logit(row, s_token, P.dtype)) * W.scale / (double)total);
    }
}

}  // namespace
}  // namespace dspark

using namespace dspark;

extern "C" size_t dspark_sample_workspace_bytes(int32_t rows, int32_t vocab) {
    if (rows < 0 || vocab < 1) return 0;
    return 256;
}

extern "C" int dspark_sample(const void* logits, int32_t dtype, int64_t row_stride, int32_t rows, int32_t vocab,
                             const float* u, const float* temperature, const int32_t* top_k, const float* top_p,
                             const float* min_p, int32_t* tokens, float* probs, void* ws, size_t ws_bytes, void* stream) {
    if (!valid_dtype(dtype)) DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "dtype must be fp32, bf16 or fp16");
    if (rows < 0 || vocab < 1) DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "rows must be >= 0 and vocab >= 1");
    if (vocab > (1 << 24)) DSPARK_FAIL(DSPARK_ERR_UNSUPPORTED, "vocab above 2^24");
    if (row_stride < vocab && rows > 1) DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "row_stride below vocab");
    if (rows == 0) return DSPARK_OK;
    if (!logits || !u || !tokens || !ws) DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "logits, u, tokens and ws must be non-NULL");
    if (!aligned_to(logits, dtype_bytes(dtype))) DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "logits must be aligned to their type");
    if (!aligned_to(ws, 256)) DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "ws must be 256-byte aligned");
    if (ws_bytes < dspark_sample_workspace_bytes(rows, vocab))
        DSPARK_FAIL(DSPARK_ERR_WORKSPACE, "ws smaller than dspark_sample_workspace_bytes()");
    SampleParams P{};
    P.logits = logits; P.stride = row_stride; P.dtype = dtype; P.rows = rows; P.V = vocab; P.u = u;
    P.temperature = temperature; P.top_k = top_k; P.top_p = top_p; P.min_p = min_p; P.tokens = tokens; P.probs = probs;
    cudaError_t e = launch_pdl(sample_kernel, dim3(rows), dim3(kThreads), 0, static_cast<cudaStream_t>(stream), P);
    if (e != cudaSuccess) DSPARK_FAIL(DSPARK_ERR_CUDA, std::string("sample launch: ") + cudaGetErrorString(e));
    return DSPARK_OK;
}
