// dspark_norm_rope_paged: per-head RMS norms of q and k, the rotation at each
// token's position, and the write of k and v into the pages, in one pass.
//
//   y = x / sqrt(mean(x^2) + eps) * gain          (v: no gain, or v as it is)
//   (y1, y2) -> (y1 cos a - y2 sin a, y2 cos a + y1 sin a),  a = position * inv_freq[i]
// over the pairs (i, i + hd / 2). Bound by HBM: every element is read once and
// written once. A warp has the heads of one token (or a share of them when there are few
// tokens); `lanes` threads make a head, each with eight consecutive elements of its first
// half and the eight they turn with (two 16-byte loads of 16-bit rows), so the
// rotation needs no exchange and its eight cosines and sines stay in registers from head to head; the sum of squares is
// a shuffle over the head's lanes. The angles: the turn count is reduced in 64 bits (at position 10^6 a 32-bit angle
// is off by 0.03 rad), sine and cosine are taken of the fraction in 32 bits, each once a warp.
// 16384 tokens of 48 bf16 heads of 128: 85 us, 4.7 TB/s (of 6.55 measured for a copy); issue
// slots 62% used, 21 warps an SM (80 registers), most stalls on loads: a warp's loads stop while it computes. fp32 rows
// into fp16 pages: 114 us, 5.3 TB/s.
#include "paged.h"

namespace dspark {
namespace {

constexpr int kThreads = 256;
// Heads of a thread whose loads are in flight together, and the blocks an SM has registers for. Measured: 16384 tokens of 48
// bf16 heads of 128 take 85 us so, 7 to 57 us more with three or four heads, or the next round's loads ahead (registers);
// fp32 rows (twice the bytes a load) gain from two heads what a third block gives.
constexpr int kItems = 2;
template <typename X> constexpr int kBlocksOf = sizeof(X) == 4 ? 2 : 3;

struct NormRopeParams {
    const void* q; const void* k; const void* v; const void* q_norm; const void* k_norm;
    int64_t q_stride, k_stride, v_stride;      // elements between tokens
    const double* inv_freq; const int32_t* positions; const int64_t* slots;
    void* q_out; void* kc; void* vc;
    int32_t* status;
    int64_t num_slots;
    int T, nH, nKv, hd, lanes, log_lanes, v_norm, split, log_split;   // lanes: threads per head (a power of two, at most 16); split: warps per token
    float eps, inv_hd;
};

template <typename T> struct Raw8;             // eight elements as loaded
template <> struct Raw8<float> { float4 a, b; };
template <> struct Raw8<__half> { uint4 a; };
template <> struct Raw8<__nv_bfloat16> { uint4 a; };

__device__ __forceinline__ void load8(Raw8<float>& r, const float* p) {
    r.a = *reinterpret_cast<const float4*>(p);
    r.b = *reinterpret_cast<const float4*>(p + 4);
}
template <typename T>
__device__ __forceinline__ void load8(Raw8<T>& r, const T* p) { r.a = *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ void unpack8(const Raw8<float>& r, float (&x)[8]) {
    x[0] = r.a.x; x[1] = r.a.y; x[2] = r.a.z; x[3] = r.a.w;
    x[4] = r.b.x; x[5] = r.b.y; x[6] = r.b.z; x[7] = r.b.w;
}
__device__ __forceinline__ void unpack8(const Raw8<__half>& r, float (&x)[8]) {
    const __half2* h = reinterpret_cast<const __half2*>(&r.a);
#pragma unroll
    for (int i = 0; i < 4; ++i) { const float2 f = __half22float2(h[i]); x[2 * i] = f.x; x[2 * i + 1] = f.y; }
}
__device__ __forceinline__ void unpack8(const Raw8<__nv_bfloat16>& r, float (&x)[8]) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&r.a);
#pragma unroll
    for (int i = 0; i < 4; ++i) { const float2 f = __bfloat1622float2(h[i]); x[2 * i] = f.x; x[2 * i + 1] = f.y; }
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__half* p, const float (&x)[8]) {
    __half2 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(h);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
    __nv_bfloat162 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(h);
}

template <typename X, typename O>
__global__ void __launch_bounds__(kThreads, kBlocksOf<X>) norm_rope_kernel(NormRopeParams P) {
    const int lane = threadIdx.x & 31, half = P.hd / 2, groups = 32 >> P.log_lanes;
    const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    pdl_trigger();
    pdl_wait();
    const int t = (int)(w >> P.log_split), part = (int)w & (P.split - 1);
    if (t >= P.T) return;
    const int grp = lane >> P.log_lanes, l = lane & (P.lanes - 1), e = l * 8;
    const bool mine = e < half;                 // hd = 192 and the like leave lanes idle
    const int heads = P.nH + 2 * P.nKv;
    int64_t slot = P.slots[t];
    const X* q = static_cast<const X*>(P.q) + t * P.q_stride + e;
    const X* k = static_cast<const X*>(P.k) + t * P.k_stride + e;
    const X* v = static_cast<const X*>(P.v) + t * P.v_stride + e;
    const double pos = (double)P.positions[t];
    float cs[8], sn[8];
    bool ready = false;
    for (int i0 = part * groups + grp; i0 - grp < heads; i0 += P.split * groups * kItems) {
        // loads first, so that (the first time) the angles hide behind them
        Raw8<X> r1[kItems], r2[kItems];
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int h = i0 + i * P.split * groups;
            if (h >= heads || !mine) continue;
            const X* src = h < P.nH ? q + h * P.hd : h < P.nH + P.nKv ? k + (h - P.nH) * P.hd : v + (h - P.nH - P.nKv) * P.hd;
            load8(r1[i], src);
            load8(r2[i], src + half);
        }
        if (!ready) {
            ready = true;
            if (slot >= P.num_slots) {
                if (lane == 0) set_status(P.status, DSPARK_DEV_CAPACITY);
                slot = -1;
            }
            if (slot < 0) return;               // a padding row
            // a lane's eight pairs: its group finds 8 / groups of them, the groups tell each other
            const int shift = groups >= 8 ? 0 : groups == 4 ? 1 : 2, each = 1 << shift;
            float c[4], s[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                c[n] = 1.f;
                s[n] = 0.f;
                const int j = e + ((grp * each + n) & 7);
                if (n >= each || j >= half) continue;
                // turns = position * inv_freq / (2 pi), whole turns dropped in 64 bits
                const double turns = pos * P.inv_freq[j] * 0.15915494309189533576888376337251;
                sincospif((float)(2.0 * (turns - rint(turns))), &s[n], &c[n]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int from = (i >> shift) * P.lanes + l;
                const float ci = each == 4 ? c[i & 3] : each == 2 ? c[i & 1] : c[0], si = each == 4 ? s[i & 3] : each == 2 ? s[i & 1] : s[0];
                cs[i] = __shfl_sync(0xffffffffu, ci, from);
                sn[i] = __shfl_sync(0xffffffffu, si, from);
            }
        }
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int h = i0 + i * P.split * groups;
            const bool on = h < heads && mine;
            const int kind = h < P.nH ? 0 : h < P.nH + P.nKv ? 1 : 2;
            float x1[8], x2[8];
            float ss = 0.f;
            if (on) {
                unpack8(r1[i], x1);
                unpack8(r2[i], x2);
#pragma unroll
                for (int j = 0; j < 8; ++j) ss += x1[j] * x1[j] + x2[j] * x2[j];
            }
            for (int o = P.lanes >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (!on) continue;                  // lanes of a head agree except idle ones; the shuffle is behind
            // (rsqrtf is within 2^-22: far inside the one rounding to 16 bits, and 4 of the squares' roundings in fp32)
            const float r = kind == 2 && !P.v_norm ? 1.f : rsqrtf(ss * P.inv_hd + P.eps);
            if (kind == 2) {
#pragma unroll
                for (int j = 0; j < 8; ++j) { x1[j] *= r; x2[j] *= r; }
            } else {
                const X* gain = static_cast<const X*>(kind == 0 ? P.q_norm : P.k_norm);      // (from L1: not worth its registers)
                if (gain) {
                    Raw8<X> w1, w2;
                    float g1[8], g2[8];
                    load8(w1, gain + e);
                    load8(w2, gain + e + half);
                    unpack8(w1, g1);
                    unpack8(w2, g2);
#pragma unroll
                    for (int j = 0; j < 8; ++j) { x1[j] *= g1[j]; x2[j] *= g2[j]; }
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float a = x1[j] * r, b = x2[j] * r;
                    x1[j] = a * cs[j] - b * sn[j];
                    x2[j] = b * cs[j] + a * sn[j];
                }
            }
            O* dst = kind == 0 ? static_cast<O*>(P.q_out) + ((int64_t)t * P.nH + h) * P.hd
                               : static_cast<O*>(kind == 1 ? P.kc : P.vc) + (slot * P.nKv + (kind == 1 ? h - P.nH : h - P.nH - P.nKv)) * P.hd;
            store8(dst + e, x1);
            store8(dst + e + half, x2);
        }
    }
}

template <typename X, typename O>
cudaError_t launch(const NormRopeParams& P, cudaStream_t s) {
    const int64_t warps = (int64_t)P.T * P.split;
    return launch_pdl(norm_rope_kernel<X, O>, dim3((unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32))), dim3(kThreads), 0, s, P);
}
template <typename X>
cudaError_t launch_x(const NormRopeParams& P, int dtype, cudaStream_t s) {
    return dtype == DSPARK_DTYPE_F32 ? launch<X, float>(P, s)
         : dtype == DSPARK_DTYPE_F16 ? launch<X, __half>(P, s) : launch<X, __nv_bfloat16>(P, s);
}

}  // namespace
}  // namespace dspark

using namespace dspark;

extern "C" int dspark_norm_rope_paged(const dspark_paged_cache* c, int32_t layer, int32_t x_dtype, const void* q,
                                      int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                                      int32_t n_heads, const void* q_norm, const void* k_norm, const double* inv_freq,
                                      float eps, int32_t v_norm, const int32_t* positions, const int64_t* slots, int32_t T,
                                      void* q_out, void* stream) {
    const int rc = check_paged_cache(c);
    if (rc != DSPARK_OK) return rc;
    if (layer < 0 || layer >= c->layers) DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "layer out of range");
    if (!valid_dtype(x_dtype)) DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "x_dtype must be fp32, bf16 or fp16");
    if (n_heads < 1 || n_heads > (1 << 16)) DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "n_heads must be in [1, 2^16]");
    if (T < 0) DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "T must be >= 0");
    if (!(eps >= 0.f)) DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "eps must be >= 0");
    if (T == 0) return DSPARK_OK;
    if (!c->k || !c->v || !q || !k || !inv_freq || !positions || !slots || !q_out)
        DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "cache.k, cache.v, q, k, inv_freq, positions, slots and q_out must be non-NULL");
    if (!v) { v = k; v_stride = k_stride; }       // keys and values from one projection
    const size_t es = dtype_bytes(x_dtype);
    if (!aligned_to(q, 16) || !aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(q_out, 16) || !aligned_to(c->k, 16) ||
        !aligned_to(c->v, 16) || !aligned_to(q_norm, 16) || !aligned_to(k_norm, 16))
        DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "q, k, v, q_out, the gains and the cache must be 16-byte aligned");
    if ((q_stride * (int64_t)es) % 16 || (k_stride * (int64_t)es) % 16 || (v_stride * (int64_t)es) % 16)
        DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "the token strides of q, k and v must be multiples of 16 bytes");
    NormRopeParams P{};
    P.q = q; P.k = k; P.v = v; P.q_norm = q_norm; P.k_norm = k_norm;
    P.q_stride = q_stride; P.k_stride = k_stride; P.v_stride = v_stride;
    P.inv_freq = inv_freq; P.positions = positions; P.slots = slots; P.q_out = q_out;
    const size_t layer_bytes = (size_t)paged_layer_elems(*c) * dtype_bytes(c->dtype) * layer;
    P.kc = static_cast<char*>(c->k) + layer_bytes;
    P.vc = static_cast<char*>(c->v) + layer_bytes;
    P.status = c->status; P.num_slots = (int64_t)c->num_pages * c->page_size;
    P.T = T; P.nH = n_heads; P.nKv = c->n_kv; P.hd = c->head_dim; P.v_norm = v_norm != 0; P.eps = eps;
    P.inv_hd = 1.f / (float)c->head_dim;
    P.lanes = 1;
    while (P.lanes * 16 < P.hd) { P.lanes *= 2; ++P.log_lanes; }
    // few tokens: a token's heads over several warps, until the SMs have a block each or a warp has one round
    P.split = 1;
    while ((int64_t)T * P.split < 148 * 8 && P.split * (32 / P.lanes) < n_heads + 2 * c->n_kv) { P.split *= 2; ++P.log_split; }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = x_dtype == DSPARK_DTYPE_F32 ? launch_x<float>(P, c->dtype, s)
                  : x_dtype == DSPARK_DTYPE_F16 ? launch_x<__half>(P, c->dtype, s)
                                                : launch_x<__nv_bfloat16>(P, c->dtype, s);
    if (e != cudaSuccess) DSPARK_FAIL(DSPARK_ERR_CUDA, std::string("norm rope launch: ") + cudaGetErrorString(e));
    return DSPARK_OK;
}
