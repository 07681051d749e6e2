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
// A cluster of C CTAs owns a row, a contiguous slice each, and the CTAs exchange a few numbers
// through distributed shared memory: C = 1 when the rows alone fill the GPU (each pass then streams
// the row), more for fewer rows (a slice that fits is kept in shared memory). The first pass finds the maximum, and
// for rows whose total is needed the sum at the same time, relative to the thread's own running
// maximum. An unfiltered row then only looks into the piece of it that holds the token.
//
// top-k: the k-th largest of the threads' maxima is at most the k-th largest
// entry; the few entries at or above it (only threads whose maximum is look
// again) are listed, sorted and finished by one CTA, the others leave.
// top-p: a histogram over (m - x) / T in linear bins of 1/64 (as many elements a bin as
// the density has there: the adds rarely collide) of the entries with a weight above
// (1 - p) / V (the others together weigh less than 1 - p of the total). A bin also sums its
// elements' places within it: with their mean z its mass lies between n e^-z (Jensen) and n e^-z
// e^(h^2 / 8) (Hoeffding; h = 1/64), which leaves a bin or two for the prefix's end. If all entries down to
// there fit the list, one CTA finishes the row; else only those bins are listed, with the exact
// mass above them. What overflows the list (thousands of equal logits) is bisected.
//
// Weights and sums are 64-bit: in a flat tail a token's share is about 10^-7 of the mass,
// so 32-bit sums would move the drawn token. exp is 2^(k/16) from a table (16 doubles: no two
// of them share a bank) times the Taylor polynomial of degree 6 on |r| <= 1/32 octave, within
// 2^-46: 12 64-bit operations an element.
//
// 512 rows of 262144 fp32 logits: greedy 135 us (4.0 TB/s; 512 CTAs on 296 places), top-k 228 us (two passes over the row),
// unfiltered 290 us (issue slots 63%, 64-bit pipe 42%), top-p 480 to 790 us (a third and a fourth pass, or a fifth far
// down the tail). One such row:
// 8 to 42 us, the exchanges of its 16 CTAs.
#include <cfloat>
#include <type_traits>

#include "paged.h"
#include "tc_ptx.cuh"

namespace dspark {
namespace {

constexpr int NT = 512;                              // threads; two CTAs an SM
constexpr int kWarps = NT / 32;
constexpr int kBins = 2048;
constexpr int kList = 4096;
constexpr int kMaxCluster = 16;
constexpr int kPlaces = 1024;                        // steps of a place within a bin
constexpr int kSliceMax = (int)(0xffffffffu / (kPlaces - 1));         // 4.2 million entries
constexpr float kPerUnit = 64.f;                     // bins per unit of (m - x) / T
constexpr size_t kHeadBytes = kList * 8;             // the histogram, later the list
constexpr double kSlack = 3e-5;                      // above the relative rounding of a bin and its edge's weight (32 bits, (m - x) / T up to 32)
constexpr double kFixed = 2251799813685248.0;        // 2^51: sums of kList weights (at most 1) in 63 bits

struct SampleParams {
    const void* logits; int64_t stride; int rows, V, cluster, slice, resident;
    const float* u; const float* temperature; const int32_t* top_k; const float* top_p; const float* min_p;
    int32_t* tokens; float* probs;
};

// Numbers that the CTAs of a cluster tell each other: slot r is rank r's.
struct Exchange {
    uint64_t best[kMaxCluster];
    double total[kMaxCluster], above[kMaxCluster], kept[kMaxCluster];
    double share[kMaxCluster], cnt[kMaxCluster], listed[kMaxCluster], first_above[kMaxCluster];
    double bis_mass[2][kMaxCluster], bis_cnt[2][kMaxCluster];
    uint64_t cut;
    unsigned long long piece[kWarps];                // listed entries that stay, per warp's piece of the slice, in 1 / kFixed
    unsigned int n_list;
};
struct Scratch {
    Exchange x;
    double tab[16];
    double red[kWarps];
    double wsum[kWarps];
    uint64_t red64[kWarps];
    double cross_before, cross_upto;
    int cross_bin;
    int found;
};

// ------------------------------------------------------------------ distributed shared memory
__device__ __forceinline__ void put(uint64_t* p, int rank, uint64_t v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(tc::mapa_shared(p, rank)), "l"(v) : "memory");
}
__device__ __forceinline__ void put(double* p, int rank, double v) {
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(tc::mapa_shared(p, rank)), "d"(v) : "memory");
}
__device__ __forceinline__ uint32_t get_u32(const uint32_t* p, int rank) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(tc::mapa_shared(p, rank)) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t add_u32(unsigned int* p, int rank, uint32_t v) {
    uint32_t old;
    asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(tc::mapa_shared(p, rank)), "r"(v) : "memory");
    return old;
}

__device__ __forceinline__ void add_u64(unsigned long long* p, int rank, uint64_t v) {
    asm volatile("red.shared::cluster.add.u64 [%0], %1;" ::"r"(tc::mapa_shared(p, rank)), "l"(v) : "memory");
}

// ------------------------------------------------------------------ values
// Bits in the order of the values (-0 as 0).
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
// One number per candidate in the filters' order: the larger comes first.
__device__ __forceinline__ uint64_t rank_of(float x, int i) { return ((uint64_t)order_key(x) << 32) | (0xffffffffu - (uint32_t)i); }

struct Weights {
    double m, c16;
    float mf, cutoff, range, z_scale;
    const double* tab;
    __device__ __forceinline__ void set(float T, const double* t) {
        c16 = 16.0 * 1.4426950408889634073599 / (double)T;
        z_scale = kPerUnit / T;
        range = 55.f * T;                                                // weights below 2^-79 count as 0
        tab = t;
    }
    __device__ __forceinline__ void at(float mx) {
        mf = mx;
        m = (double)mx;
        cutoff = fmaxf(mx - range, -FLT_MAX);
    }
    // For x >= cutoff; any number for the others (NaN and -infinity among them).
    __device__ __forceinline__ double raw(float x) const {
        const double magic = 6755399441055744.0;                         // 1.5 2^52: the sum's low word is the rounded integer
        const double d = (double)x - m, t = fma(d, c16, magic);
        const int k = __double2loint(t);
        const double r = fma(d, c16, -(t - magic));                      // |r| <= 1/2 sixteenth of an octave
        double p = 9.181219573844436e-12;                                // (ln 2 / 16)^n / n!
        p = fma(p, r, 1.271587195055813e-9);
        p = fma(p, r, 1.467610032291943e-7);
        p = fma(p, r, 1.3550807779497455e-5);
        p = fma(p, r, 9.383847928089871e-4);
        p = fma(p, r, 4.332169878499658e-2);
        p = fma(p, r, 1.0);
        p *= tab[k & 15];
        return __hiloint2double(__double2hiint(p) + ((k >> 4) << 20), __double2loint(p));
    }
    __device__ __forceinline__ double operator()(float x) const { return x >= cutoff ? raw(x) : 0.0; }
    // m - x in bins, before rounding down; falls with x.
    __device__ __forceinline__ float z(float x) const { return fminf((mf - x) * z_scale, 4096.f); }
    __device__ __forceinline__ int bin(float x) const { return min((int)z(x), kBins - 1); }
};

// ------------------------------------------------------------------ block helpers
template <typename T, typename Op>
__device__ __forceinline__ T block_reduce(T v, T* buf, Op op) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if (lane == 0) buf[wid] = v;
    __syncthreads();
    v = buf[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) v = op(v, buf[w]);
    return v;
}
__device__ __forceinline__ double block_sum(double v, double* buf) {
    return block_reduce(v, buf, [](double a, double b) { return a + b; });
}
// Sum of v over the threads before this one; *total: over all.
__device__ __forceinline__ double block_scan(double v, double* buf, double* total) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    double x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) buf[wid] = x;
    double before = __shfl_up_sync(0xffffffffu, x, 1);
    if (lane == 0) before = 0.0;
    __syncthreads();
    double base = 0.0, all = 0.0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < wid) base += buf[w];
        all += buf[w];
    }
    *total = all;
    return base + before;
}
// Falling bitonic sort of n (a power of two, 64 .. kList) entries; a constant, so that the loops unroll, and a call,
// so that they do not crowd the passes' registers. Pairs at most 32 apart
// stay within one warp's 64 entries.
template <int n>
__device__ __noinline__ void sort_falling(uint64_t* a) {
    const int tid = threadIdx.x;
    __syncthreads();
    for (int k = 2; k <= n; k <<= 1) {
        for (int j = k >> 1; j > 0; j >>= 1) {
            for (int t = tid; t < n / 2; t += NT) {
                const int i = 2 * t - (t & (j - 1));
                const uint64_t x = a[i], y = a[i + j];
                if ((x < y) == ((i & k) == 0)) { a[i] = y; a[i + j] = x; }
            }
            if (j > 32 || (j == 1 && k >= 64)) __syncthreads(); else __syncwarp();
        }
    }
    __syncthreads();
}

// Adds the weights of a vector's entries >= thr that `pred` accepts; no branches, so that their 64-bit chains overlap.
template <int VEC, typename Pred>
__device__ __forceinline__ void add_mass(const Weights& W, const float (&x)[VEC], int i0, float thr, Pred pred, double& a, double& b) {
#pragma unroll
    for (int h = 0; h < VEC; h += 4) {                        // (four chains: eight do not fit the registers)
        double w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = W.raw(x[h + i]);
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            if (x[h + i] >= thr && pred(x[h + i], i0 + h + i, w[i])) a += w[i];
            if (x[h + i + 1] >= thr && pred(x[h + i + 1], i0 + h + i + 1, w[i + 1])) b += w[i + 1];
        }
    }
}

template <typename X>
__global__ void __launch_bounds__(NT, 2) sample_kernel(SampleParams P) {
    constexpr int VEC = 16 / (int)sizeof(X);
    using Light = std::integral_constant<int, 6>;             // vectors in flight a thread: passes that only compare,
    using Heavy = std::integral_constant<int, 2>;             // and those that sum weights
    extern __shared__ __align__(16) uint8_t smem[];
    uint32_t* hist = reinterpret_cast<uint32_t*>(smem);       // [kBins] elements
    uint32_t* place = hist + kBins;                           // [kBins] their places in the bin, in 1 / kPlaces; then the mean as a float
    uint64_t* list = reinterpret_cast<uint64_t*>(smem);
    uint4* data = reinterpret_cast<uint4*>(smem + kHeadBytes);
    __shared__ Scratch S;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, C = P.cluster;
    const int rank = C > 1 ? (int)tc::cluster_ctarank() : 0, r = blockIdx.x / C;
    if (tid == 0) S.x.n_list = 0;
    if (tid < kWarps) S.x.piece[tid] = 0;
    if (C > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");   // waited for before the first exchange
    if (tid < 16) S.tab[tid] = exp2((double)tid * 0.0625);
    pdl_trigger();
    pdl_wait();
    __syncthreads();                                          // the table: the first pass over a streamed row sums weights already
    const float T = P.temperature ? P.temperature[r] : 1.f, p = P.top_p ? P.top_p[r] : 1.f, mp = P.min_p ? P.min_p[r] : 0.f, u = P.u[r];
    const int k = P.top_k ? P.top_k[r] : 0;
    const bool alone = !(T > 0.f) || p <= 0.f || mp > 1.f || k == 1;                    // greedy, or a filter that leaves one
    const bool has_p = p < 1.f, has_k = k > 0 && k < P.V;
    const double low = mp > 0.f ? (double)mp : 0.0;
    const bool sum_now = !alone && !has_k && (has_p || low == 0.0);                     // the whole row's mass is needed
    Weights W;
    W.set(T, S.tab);

    // The slice, counted from the 16-byte boundary at or before the row: element j of it is entry s0 + j - off.
    const X* row = static_cast<const X*>(P.logits) + (int64_t)r * P.stride;
    const int off = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(X));
    const X* base = row - off;
    const int s0 = rank * P.slice, n_loc = min(max(off + P.V - s0, 0), P.slice);
    const int nvec = (n_loc + VEC - 1) / VEC, per_warp = (P.slice / VEC + kWarps - 1) / kWarps;
    const int v0 = min(nvec, wid * per_warp), v1 = min(nvec, v0 + per_warp);              // this warp's vectors
    auto fetch = [&](int v) {                                  // a vector of the row; -infinity outside it
        const int j = v * VEC;
        uint4 raw;
        if (s0 + j >= off && j + VEC <= n_loc) {
            raw = __ldg(reinterpret_cast<const uint4*>(base + s0 + j));
        } else {
            X* e = reinterpret_cast<X*>(&raw);
#pragma unroll
            for (int i = 0; i < VEC; ++i) e[i] = s0 + j + i >= off && j + i < n_loc ? base[s0 + j + i] : from_f<X>(-INFINITY);
        }
        return raw;
    };
    bool inf_max = false;                                      // the maximum is infinite: its candidates count as 0, the others as -infinity
    auto value = [&](X e) {
        const float x = to_f(e);
        return !inf_max ? x : x == INFINITY ? 0.f : -INFINITY;
    };
    // f(x[VEC], index of the first, their maximum (a NaN loses)) over vectors [a, b) of the slice, `step` apart
    auto scan = [&](auto batch, int a, int b, int step, bool first, auto f) {
        constexpr int BATCH = decltype(batch)::value;
        for (int v = a; v < b; v += BATCH * step) {
            uint4 raw[BATCH];
#pragma unroll
            for (int q = 0; q < BATCH; ++q)
                if (v + q * step < b) raw[q] = P.resident && !first ? data[v + q * step] : fetch(v + q * step);
#pragma unroll
            for (int q = 0; q < BATCH; ++q) {
                if (v + q * step >= b) break;
                if (P.resident && first) data[v + q * step] = raw[q];
                const X* e = reinterpret_cast<const X*>(&raw[q]);
                float x[VEC], hi = -INFINITY;
#pragma unroll
                for (int i = 0; i < VEC; ++i) { x[i] = value(e[i]); hi = fmaxf(hi, x[i]); }
                f(x, s0 + (v + q * step) * VEC - off, hi);
            }
        }
    };
    auto each = [&](auto batch, auto f) { scan(batch, v0 + lane, v1, 32, false, f); };      // over the slice, a contiguous piece per warp
    auto meet = [&] { if (C > 1) cluster_sync(); else __syncthreads(); };
    auto tell = [&](auto* slots, auto v) { if (tid < C) put(&slots[rank], tid, v); };   // this rank's number, to every CTA
    auto sum_of = [&](const double* slots) {
        double t = 0.0;
        for (int q = 0; q < C; ++q) t += slots[q];
        return t;
    };
    auto any = [](float, int, double) { return true; };

    // ---------------------------------------------------------------- the maximum, and the mass
    float best = -INFINITY;
    double sum0 = 0.0, sum1 = 0.0;
    if (sum_now && !P.resident) {
        W.at(best);
        constexpr int B = Heavy::value;
        for (int v = v0 + lane; v < v1; v += B * 32) {
            uint4 raw[B];
            float hi = -INFINITY;
#pragma unroll
            for (int q = 0; q < B; ++q)
                if (v + 32 * q < v1) raw[q] = fetch(v + 32 * q);
#pragma unroll
            for (int q = 0; q < B; ++q) {
                if (v + 32 * q >= v1) break;
                const X* e = reinterpret_cast<const X*>(&raw[q]);
#pragma unroll
                for (int i = 0; i < VEC; ++i) hi = fmaxf(hi, to_f(e[i]));      // (a NaN loses)
            }
            if (hi > best) {                                  // the sums so far, relative to the new maximum
                W.at(hi);
                const double f = W(best);
                sum0 *= f;
                sum1 *= f;
                best = hi;
            }
#pragma unroll
            for (int q = 0; q < B; ++q) {
                if (v + 32 * q >= v1) break;
                const X* e = reinterpret_cast<const X*>(&raw[q]);
                float x[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) x[i] = to_f(e[i]);
                add_mass<VEC>(W, x, 0, W.cutoff, any, sum0, sum1);
            }
        }
    } else {
        scan(Light{}, v0 + lane, v1, 32, true, [&](const float (&)[VEC], int, float hi) { best = fmaxf(best, hi); });
    }
    float mx = block_reduce(best, reinterpret_cast<float*>(S.red64), [](float x, float y) { return fmaxf(x, y); });
    if (C > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    // Lower bounds of the row's k-th largest: the k-th largest of the threads' maxima, of whichever CTA has the highest;
    // and, k / C of the candidates from each CTA, the lowest of their (k / C)-th.
    float bound = -INFINITY, share = -INFINITY;
    // (more than a thread's maximum each for k > NT: the maxima of eight parts of its vectors)
    const bool listable = has_k && !alone && k <= kList / 2;
    if (listable) {
        const int parts = k <= NT ? 1 : kList / NT;
        for (int i = tid; i < parts * NT; i += NT) list[i] = (uint64_t)order_key(parts == 1 ? best : -INFINITY) << 32;
        if (parts > 1) {
            int part = 0;
            scan(std::integral_constant<int, 1>{}, v0 + lane, v1, 32, !P.resident, [&](const float (&)[VEC], int, float hi) {
                uint64_t& most = list[part * NT + tid];
                most = max(most, (uint64_t)order_key(hi) << 32);
                part = part + 1 == parts ? 0 : part + 1;
            });
        }
        if (parts == 1) sort_falling<NT>(list); else sort_falling<kList>(list);
        bound = key_value((uint32_t)(list[k - 1] >> 32));
        share = key_value((uint32_t)(list[(k - 1) / C] >> 32));
        tell(S.x.share, (double)share);
    }
    tell(S.x.best, ((uint64_t)__float_as_uint(bound) << 32) | __float_as_uint(mx));
    meet();
    for (int q = 0; q < C; ++q) {
        mx = fmaxf(mx, __uint_as_float((uint32_t)S.x.best[q]));
        bound = fmaxf(bound, __uint_as_float((uint32_t)(S.x.best[q] >> 32)));
    }
    if (listable) {
        for (int q = 0; q < C; ++q) share = fminf(share, (float)S.x.share[q]);
        bound = fmaxf(bound, share);
    }
    // f(x, index) for the entries >= thr (no NaN); threads and vectors without one are skipped
    auto each_from = [&](float thr, auto f) {
        if (!(best >= thr)) return;
        each(Light{}, [&](const float (&x)[VEC], int i0, float hi) {
            if (hi >= thr) {
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (x[i] >= thr) f(x[i], i0 + i);
            }
        });
    };
    auto mass_of = [&](float thr, auto pred) {                // this thread's share of the weights of the entries >= thr
        double a = 0.0, b = 0.0;
        thr = fmaxf(thr, W.cutoff);
        if (best >= thr)
            each(Heavy{}, [&](const float (&x)[VEC], int i0, float hi) { if (hi >= thr) add_mass<VEC>(W, x, i0, thr, pred, a, b); });
        return a + b;
    };
    auto largest_alone = [&] {                                 // the lowest index of the maximum
        int at = 0x7fffffff;
        each_from(mx, [&](float, int i) { at = min(at, i); });
        at = block_reduce(at, reinterpret_cast<int*>(S.red64), [](int a, int b) { return min(a, b); });
        tell(S.x.cnt, (double)at);
        meet();
        if (rank == 0 && tid == 0) {
            double first = S.x.cnt[0];
            for (int q = 1; q < C; ++q) first = fmin(first, S.x.cnt[q]);
            P.tokens[r] = (int)first;
            if (P.probs) P.probs[r] = 1.f;
        }
    };
    if (mx == -INFINITY) {                                     // nothing to choose from
        if (rank == 0 && tid == 0) {
            P.tokens[r] = -1;
            if (P.probs) P.probs[r] = 0.f;
        }
        return;
    }
    if (alone) {
        largest_alone();
        return;
    }
    double mine = 0.0;                                        // this thread's mass
    if (mx == INFINITY) {
        inf_max = true;
        mx = 0.f;
        best = best == INFINITY ? 0.f : -INFINITY;
        bound = bound == INFINITY ? 0.f : -INFINITY;
        W.at(mx);
        if (sum_now) mine = mass_of(-FLT_MAX, any);
    } else {
        W.at(mx);
        if (sum_now) mine = P.resident ? mass_of(-FLT_MAX, any) : (sum0 + sum1) * W(best);
    }

    uint64_t cut = 0;                                         // candidates below it are dropped
    bool pieces = false;                                      // S.wsum: the kept mass of each warp's piece
    auto piece_sums = [&](double v) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        __syncthreads();
        if (lane == 0) S.wsum[wid] = v;
        __syncthreads();
        double t = 0.0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) t += S.wsum[w];
        return t;
    };
    // An entry's rank into the list of CTA 0; how many there are in all.
    int listed = 0;
    auto push = [&](float x, int i) {
        ++listed;
        const uint32_t at = C > 1 ? add_u32(&S.x.n_list, 0, 1u) : atomicAdd(&S.x.n_list, 1u);
        if (at < (uint32_t)kList) {
            if (C > 1) put(&list[at], 0, rank_of(x, i)); else list[at] = rank_of(x, i);
        }
    };
    auto count_list = [&] {
        tell(S.x.listed, (double)block_reduce(listed, reinterpret_cast<int*>(S.red64), [](int a, int b) { return a + b; }));
        meet();
        return sum_of(S.x.listed);
    };
    auto resort = [&](int m) {
        if (m == 256) sort_falling<256>(list);
        else if (m == 512) sort_falling<512>(list);
        else if (m == 1024) sort_falling<1024>(list);
        else if (m == 2048) sort_falling<2048>(list);
        else sort_falling<kList>(list);
    };
    auto sort_list = [&](int n) {
        int m = 256;
        while (m < n) m *= 2;
        for (int i = n + tid; i < m; i += NT) list[i] = 0;
        resort(m);
        return m;
    };
    // CTA 0 finishes the row from its list of n entries, the only ones that can stay; total: top-p's whole (without top-k).
    auto finish = [&](int n, double total) {
        const int m = sort_list(n), nk = has_k ? min(n, k) : n, per = (m + NT - 1) / NT;
        double mine = 0.0, all;
        for (int i = 0, q = tid * per; i < per && q < nk; ++i, ++q) mine += W(key_value((uint32_t)(list[q] >> 32)));
        double cum = block_scan(mine, S.red, &all);
        const double target = (double)p * (has_k ? all : total);
        for (int i = 0, q = tid * per; i < per && q < m; ++i, ++q) {
            const uint64_t e = list[q];
            const double w = q < nk ? W(key_value((uint32_t)(e >> 32))) : 0.0;
            const bool keep = q < nk && (q == 0 || ((!has_p || cum < target) && w >= low));
            cum += w;
            // next by rising index: complements fall
            list[q] = keep ? ~(((uint64_t)(0xffffffffu - (uint32_t)e) << 32) | (uint32_t)(e >> 32)) : 0;
        }
        resort(m);
        mine = 0.0;
        int last = -1;
        for (int i = 0, q = tid * per; i < per && q < m; ++i, ++q) {
            const uint64_t e = list[q];
            const double w = e ? W(key_value((uint32_t)~e)) : 0.0;
            if (w > 0.0) last = q;
            mine += w;
        }
        cum = block_scan(mine, S.red, &all);
        if (tid == 0) S.found = kList;
        __syncthreads();
        const double want = (double)u * all;
        if (last >= 0 && cum + mine > want) {
            for (int i = 0, q = tid * per; i < per && q < m; ++i, ++q) {
                const double w = list[q] ? W(key_value((uint32_t)~list[q])) : 0.0;
                cum += w;
                if (w > 0.0 && cum > want) { atomicMin(&S.found, q); break; }
            }
        }
        const int end = block_reduce(last, reinterpret_cast<int*>(S.red64), [](int a, int b) { return max(a, b); });
        __syncthreads();
        if (tid == 0) {
            const uint64_t v = ~list[S.found < kList ? S.found : end];
            P.tokens[r] = (int)(v >> 32);
            if (P.probs) P.probs[r] = (float)(W(key_value((uint32_t)v)) / all);
        }
    };

    bool bisect = false;
    if (has_k) {
        bisect = true;
        if (bound > -INFINITY) {
            each_from(bound, push);
            const double n = count_list();
            if (n <= (double)kList) {
                if (rank == 0) finish((int)n, 0.0);
                return;
            }
        }
    } else if (has_p) {
        // ------------------------------------------------------------ the prefix's end
        // At or below every x of bins 0 .. b.
        auto edge_x = [&](int b) {
            return b >= kBins - 1 ? -FLT_MAX : fmaxf(-FLT_MAX, mx - T * ((float)(b + 1) * (1.00002f / kPerUnit)) - 1e-6f * fabsf(mx));
        };
        bound = fmaxf(mx - T * (logf((float)P.V / (1.f - p)) + 0.01f), -FLT_MAX);
        tell(S.x.total, block_sum(mine, S.red));
        for (int i = tid; i < kBins; i += NT) hist[i] = place[i] = 0;
        __syncthreads();
        each_from(bound, [&](float x, int) {
            const float z = W.z(x);
            const int b = min((int)z, kBins - 1);
            atomicAdd(&hist[b], 1u);
            atomicAdd(&place[b], min((uint32_t)((z - (float)b) * kPlaces), kPlaces - 1u));
        });
        meet();
        const double total = sum_of(S.x.total), target = (double)p * total;
        // sums of the rank's share of the bins over the cluster
        const int nb = kBins / C;
        auto lower = [&](int b, uint32_t n, float mean) {     // bounds of a bin's mass
            return b == kBins - 1 ? 0.0 : (double)n * (1.0 - kSlack) * __expf(-((float)b + mean + 1.f / kPlaces) * (1.f / kPerUnit));
        };
        auto upper = [&](int b, uint32_t n, float mean) {     // (the last bin has no end)
            return (double)n * (1.0 + kSlack) * 1.000031 * __expf(-((float)b + (b == kBins - 1 ? 0.f : mean)) * (1.f / kPerUnit));
        };
        for (int b = rank * nb + tid; b < (rank + 1) * nb; b += NT) {
            uint32_t c = 0;
            double at = 0.0;
            for (int q = 0; q < C; ++q) {
                c += get_u32(&hist[b], q);
                at += get_u32(&place[b], q);
            }
            hist[b] = c;                                      // no other rank reads this rank's share before the next meeting
            place[b] = __float_as_uint(c > 0 ? (float)(at / ((double)kPlaces * c)) : 0.f);
        }
        meet();
        constexpr int PER = kBins / NT;                       // every CTA has all bins, a few a thread
        uint32_t c[PER];
        float mean[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int b = tid * PER + i;
            c[i] = get_u32(&hist[b], b / nb);
            mean[i] = __uint_as_float(get_u32(&place[b], b / nb));
        }
        // The first bin, from `from` on, at which the running sum of `measure`, `above` to start with, reaches the
        // target, or the last; *before: elements of the bins before it, *upto: with its own.
        auto cross = [&](auto measure, int from, double above, double* before, double* upto) {
            double v[PER], n = 0.0, sum = 0.0;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int b = tid * PER + i;
                v[i] = b >= from ? measure(b, c[i], mean[i]) : 0.0;
                sum += v[i];
                n += c[i];
            }
            double all_v, all_n;
            double pv = above + block_scan(sum, S.red, &all_v), pn = block_scan(n, S.red, &all_n);
            if (tid == 0) S.cross_bin = kBins - 1;
            __syncthreads();
            double at = pv;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                at += v[i];
                if (tid * PER + i >= from && at >= target) { atomicMin(&S.cross_bin, tid * PER + i); break; }
            }
            __syncthreads();
            const int bin = S.cross_bin;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                if (tid * PER + i == bin) { S.cross_before = pn; S.cross_upto = pn + c[i]; }
                pn += c[i];
            }
            __syncthreads();
            *before = S.cross_before;
            *upto = S.cross_upto;
            __syncthreads();
            return bin;
        };
        double before, upto, skip;
        int b_lo = cross(lower, 0, 0.0, &before, &upto);
        if (upto <= (double)kList) {
            meet();                                           // every rank has read the bins that the list overwrites
            each_from(fmaxf(bound, edge_x(b_lo)), [&](float x, int i) { if (W.bin(x) <= b_lo) push(x, i); });
            count_list();
            if (rank == 0) finish((int)upto, total);
            return;
        }
        int b_up = cross(upper, 0, 0.0, &before, &skip);
        // The mass above those bins stays, so without min_p it also is the start of the pieces' kept mass.
        double mass = 0.0;
        int from = 0;
        if (upto - before > (double)kList && b_up > 0) {      // far down the tail the bounds of the whole are too wide: again from the exact mass
            from = b_up;
            mass = mass_of(edge_x(from - 1), [&](float x, int, double) { return W.bin(x) < from; });
            tell(S.x.first_above, block_sum(mass, S.red));
            meet();
            const double above = sum_of(S.x.first_above);
            b_lo = cross(lower, from, above, &skip, &upto);
            b_up = cross(upper, from, above, &before, &skip);
        }
        if (upto - before <= (double)kList) {
            meet();
            // one pass for the exact mass of bins [from, b_up) and the list of bins [b_up, b_lo] (an x >= sure is above them
            // for sure: most need no bin)
            const float sure = from > 0 ? INFINITY : mx - T * ((float)b_up * (0.99998f / kPerUnit)) + 1e-6f * fabsf(mx);
            mass += mass_of(fmaxf(bound, edge_x(b_lo)), [&](float x, int i, double) {
                if (x >= sure && b_up > 0) return true;
                const int b = W.bin(x);
                if (b >= b_up && b <= b_lo) push(x, i);
                return b >= from && b < b_up;
            });
            tell(S.x.above, piece_sums(mass));
            const int n = (int)count_list();
            if (rank == 0) {
                const int per = (sort_list(n) + NT - 1) / NT;
                double own = 0.0, all;
                for (int i = 0, q = tid * per; i < per && q < n; ++i, ++q) own += W(key_value((uint32_t)(list[q] >> 32)));
                double cum = sum_of(S.x.above) + block_scan(own, S.red, &all);
                int stay = 0;                                 // the list's first `stay` entries stay
                for (int i = 0, q = tid * per; i < per && q < n; ++i, ++q) {
                    if (!(cum < target)) break;
                    const double w = W(key_value((uint32_t)(list[q] >> 32)));
                    ++stay;
                    cum += w;
                    const int j = (int)(0xffffffffu - (uint32_t)list[q]) + off, own_rank = j / P.slice;
                    add_u64(&S.x.piece[(j - own_rank * P.slice) / VEC / per_warp], own_rank, (uint64_t)__double2ull_rn(w * kFixed));
                }
                stay = block_reduce(stay, reinterpret_cast<int*>(S.red64), [](int a, int b) { return a + b; });
                const uint64_t c = n == 0 ? 0 : stay > 0 ? list[stay - 1] : list[0] + 1;
                if (tid < C) put(&S.x.cut, tid, c);
            }
            meet();
            cut = S.x.cut;
            pieces = low == 0.0;
        } else {
            bisect = true;
        }
    }
    if (bisect) {
        // ------------------------------------------------------------ too many equal or too close: bisection of the rank
        int turn = 0;
        const uint64_t top = rank_of(mx, 0);                  // no candidate comes before it
        auto measure = [&](uint64_t c, bool with_c, bool mass, double* n) {   // of the candidates above c (and not below `cut`)
            double nn = 0.0, mm = 0.0;
            each_from(-FLT_MAX, [&](float x, int i) {
                const uint64_t v = rank_of(x, i);
                if (v >= cut && (v > c || (with_c && v == c))) {
                    nn += 1.0;
                    if (mass) mm += W(x);
                }
            });
            nn = block_sum(nn, S.red);
            if (mass) mm = block_sum(mm, S.red);
            tell(S.x.bis_cnt[turn], nn);
            tell(S.x.bis_mass[turn], mm);
            meet();
            *n = sum_of(S.x.bis_cnt[turn]);
            const double t = sum_of(S.x.bis_mass[turn]);
            turn ^= 1;
            return t;
        };
        double n;
        if (has_k) {                                          // the largest c with k candidates at or above it
            measure(0, true, false, &n);
            if (n > (double)k) {
                uint64_t lo = 0, hi = top + 1;
                while (hi - lo > 1) {
                    const uint64_t mid = lo + ((hi - lo) >> 1);
                    measure(mid, true, false, &n);
                    if (n >= (double)k) lo = mid; else hi = mid;
                    if (n == (double)k) break;
                }
                cut = lo;
            }
        }
        if (has_p) {                                          // the smallest c with less than the target's mass above it
            const double target = (double)p * measure(0, true, true, &n);
            uint64_t lo = cut, hi = top;                      // hi always qualifies: nothing lies above it
            while (lo < hi) {
                const uint64_t mid = lo + ((hi - lo) >> 1);
                if (measure(mid, false, true, &n) < target) hi = mid; else lo = mid + 1;
            }
            cut = lo;
        }
    }

    // -------------------------------------------------------------------- the draw, in the vocabulary's order
    const float cut_x = key_value((uint32_t)(cut >> 32));
    const uint32_t cut_i = 0xffffffffu - (uint32_t)cut;
    // (a little below where the weight falls to min_p: the weight itself decides)
    const float thr = fmaxf(fmaxf(W.cutoff, cut != 0 ? cut_x : -FLT_MAX), low > 0.0 ? mx + 1.001f * T * logf(mp) - 1e-3f * T - 1e-6f * fabsf(mx) : -FLT_MAX);
    auto kept = [&](float x, int i, double w) { return w >= low && !(cut != 0 && x == cut_x && (uint32_t)i > cut_i); };
    double slice_sum;
    if (pieces) {
        if (tid < kWarps) S.wsum[tid] += (double)S.x.piece[tid] / kFixed;
        __syncthreads();
        slice_sum = 0.0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) slice_sum += S.wsum[w];
    } else {
        slice_sum = piece_sums(sum_now && !has_p ? mine : mass_of(thr, kept));
    }
    tell(S.x.kept, slice_sum);
    meet();
    const double all = sum_of(S.x.kept), want = (double)u * all;
    // the slice, then the warp's piece in it, then the element (the last with any mass where rounding finds none)
    double cum = 0.0, owner_cum = 0.0;
    int owner = -1;
    for (int q = 0; q < C; ++q) {
        const double s = S.x.kept[q];
        if (s > 0.0) {
            owner = q;
            owner_cum = cum;
            if (cum + s > want) break;
        }
        cum += s;
    }
    if (owner < 0) {                                          // (the filters always leave one)
        largest_alone();
        return;
    }
    if (rank != owner) return;
    cum = owner_cum;
    int piece = -1;
    double piece_cum = 0.0;
    for (int w = 0; w < kWarps; ++w) {
        const double s = S.wsum[w];
        if (s > 0.0) {
            piece = w;
            piece_cum = cum;
            if (cum + s > want) break;
        }
        cum += s;
    }
    const int a0 = min(nvec, piece * per_warp), a1 = min(nvec, a0 + per_warp), each_n = (a1 - a0 + NT - 1) / NT;
    const int t0 = min(a1, a0 + tid * each_n), t1 = min(a1, t0 + each_n);
    auto piece_scan = [&](auto f) {
        scan(Heavy{}, t0, t1, 1, false, [&](const float (&x)[VEC], int i0, float hi) {
            if (!(hi >= thr)) return;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const double w = x[i] >= thr ? W(x[i]) : 0.0;
                if (w > 0.0 && kept(x[i], i0 + i, w)) f(w, i0 + i);
            }
        });
    };
    mine = 0.0;
    int last = -1;
    piece_scan([&](double w, int i) { mine += w; last = i; });
    double part;
    cum = piece_cum + block_scan(mine, S.red, &part);
    if (tid == 0) S.found = 0x7fffffff;
    __syncthreads();
    if (last >= 0 && cum + mine > want) {
        int hit = 0x7fffffff;
        piece_scan([&](double w, int i) {
            cum += w;
            if (hit == 0x7fffffff && cum > want) hit = i;
        });
        atomicMin(&S.found, hit);
    }
    const int end = block_reduce(last, reinterpret_cast<int*>(S.red64), [](int a, int b) { return max(a, b); });
    __syncthreads();
    if (tid == 0) {
        const int at = S.found != 0x7fffffff ? S.found : end;
        P.tokens[r] = at;
        if (P.probs) P.probs[r] = (float)(W(value(row[at])) / all);
    }
}

template <typename X>
cudaError_t launch(SampleParams P, cudaStream_t s) {
    constexpr int VEC = 16 / (int)sizeof(X);
    auto slice = [&](int c) { return (int)(((int64_t)P.V + VEC - 1 + c - 1) / c + VEC - 1) / VEC * VEC; };
    // Rows are split while they leave SMs idle (148, two CTAs each) and a slice is long enough to pay for the exchanges;
    // and, whatever their number, down to slices whose places in one bin add up in 32 bits (four CTAs for 2^24 entries).
    int c = 1;
    while (c < kMaxCluster && (((int64_t)P.rows * c * 2 <= 296 && slice(c) > 4096) || slice(c) > kSliceMax)) c *= 2;
    P.cluster = c;
    P.slice = slice(c);
    // Shared memory for two CTAs an SM, or for one where there are no more CTAs than SMs.
    const size_t room = ((int64_t)P.rows * c <= 148 ? 208 * 1024 : 104 * 1024) - kHeadBytes;
    P.resident = P.slice * sizeof(X) <= room;
    const size_t smem = kHeadBytes + (P.resident ? P.slice * sizeof(X) : 0);
    auto kern = sample_kernel<X>;
    cudaError_t e = cudaSuccess;                              // (the attributes cost host time: only where the launch needs them)
    if (smem > 48 * 1024 - sizeof(Scratch)) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 208 * 1024);
    if (e == cudaSuccess && c > 8) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) e = launch_pdl_cluster(kern, dim3((unsigned)(P.rows * c)), dim3(NT), c, smem, s, P);
    return e;
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
    if (rows > (1 << 26)) DSPARK_FAIL(DSPARK_ERR_UNSUPPORTED, "more than 2^26 rows in one call");
    if (vocab > (1 << 24)) DSPARK_FAIL(DSPARK_ERR_UNSUPPORTED, "vocab above 2^24");
    if (row_stride < vocab && rows > 1) DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "row_stride below vocab");
    if (rows == 0) return DSPARK_OK;
    if (!logits || !u || !tokens || !ws) DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "logits, u, tokens and ws must be non-NULL");
    if (!aligned_to(logits, dtype_bytes(dtype))) DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "logits must be aligned to their type");
    if (!aligned_to(ws, 256)) DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "ws must be 256-byte aligned");
    if (ws_bytes < dspark_sample_workspace_bytes(rows, vocab))
        DSPARK_FAIL(DSPARK_ERR_WORKSPACE, "ws smaller than dspark_sample_workspace_bytes()");
    SampleParams P{};
    P.logits = logits; P.stride = row_stride; P.rows = rows; P.V = vocab; P.u = u;
    P.temperature = temperature; P.top_k = top_k; P.top_p = top_p; P.min_p = min_p; P.tokens = tokens; P.probs = probs;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = dtype == DSPARK_DTYPE_F32 ? launch<float>(P, s) : dtype == DSPARK_DTYPE_F16 ? launch<__half>(P, s) : launch<__nv_bfloat16>(P, s);
    if (e != cudaSuccess) DSPARK_FAIL(DSPARK_ERR_CUDA, std::string("sample launch: ") + cudaGetErrorString(e));
    return DSPARK_OK;
}
