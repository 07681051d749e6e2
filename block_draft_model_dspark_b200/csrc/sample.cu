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
// A cluster of C CTAs owns a row, a contiguous slice each, kept in shared memory: the row
// is read from HBM once, every later pass reads shared memory, and the CTAs exchange a few numbers
// through distributed shared memory. A filter's boundary is found from a
// histogram over (m - x) / T, linear bins of 1/64 (as many elements a bin as
// the density has there: the adds rarely collide), restricted to elements that
// can matter: for top-k those not below the smallest of k thread groups' maxima,
// for top-p those with a weight above (1 - p) / V (the others together weigh less than
// 1 - p of the total). If the elements down to the boundary fit a list of 1024,
// one CTA sorts it and finishes the row alone, the others leave. Else the
// boundary's bins are split 2048 ways once more and only the elements of the bins that
// still may hold it are sorted; what overflows even that (many equal logits) is bisected.
//
// Weights and sums are 64-bit: in a flat tail a token's share is about 10^-7 of the mass,
// so 32-bit sums would move the drawn token. exp is 2^(k/16) from a table (16 doubles: no two
// of them share a bank) times the Taylor polynomial of degree 6 on |r| <= 1/32 octave, within
// 2^-46; 12 64-bit operations an element, which is what bounds unfiltered rows.
#include <algorithm>
#include <cfloat>

#include "paged.h"
#include "tc_ptx.cuh"

namespace dspark {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kList = 1024;
constexpr int kMaxCluster = 16;
constexpr float kPerUnit = 64.f;                     // bins per unit of (m - x) / T
constexpr size_t kHeadBytes = 8192;                  // the histogram, later the list
constexpr double kSlack = 3e-5;                      // above the relative rounding of a bin and its edge's weight (32 bits, (m - x) / T up to 32)

struct SampleParams {
    const void* logits; int64_t stride; int rows, V, cluster, slice, resident;
    const float* u; const float* temperature; const int32_t* top_k; const float* top_p; const float* min_p;
    int32_t* tokens; float* probs;
};

// Numbers that the CTAs of a cluster tell each other: slot r is rank r's.
struct Exchange {
    uint64_t best[kMaxCluster];
    double total[kMaxCluster], above[kMaxCluster], above2[kMaxCluster], kept[kMaxCluster];
    double lo[kMaxCluster], up[kMaxCluster], cnt[kMaxCluster];          // of the rank's bins
    double bis_mass[2][kMaxCluster], bis_cnt[2][kMaxCluster];
    uint64_t cut;
    unsigned int n_list;
};
struct Scratch {
    Exchange x;
    double tab[16];
    double red[kWarps];
    double wsum[kWarps];
    uint64_t red64[kWarps];
    double cross_before;
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
    float mf, cutoff, inv_t;
    const double* tab;
    __device__ __forceinline__ void set(float mx, float T, const double* t) {
        mf = mx;
        m = (double)mx;
        c16 = 16.0 * 1.4426950408889634073599 / (double)T;
        inv_t = kPerUnit / T;
        cutoff = mx == INFINITY ? mx : fmaxf(mx - 55.f * T, -FLT_MAX);   // weights below 2^-79 count as 0
        tab = t;
    }
    __device__ __forceinline__ double operator()(float x) const {
        if (!(x >= cutoff)) return 0.0;
        if (x == mf) return 1.0;
        const double magic = 6755399441055744.0;                         // 1.5 2^52: the sum's low word is the rounded integer
        const double d = (double)x - m, t = fma(d, c16, magic);
        const int k = __double2loint(t);
        const double r = fma(d, c16, -(t - magic));                      // |r| <= 1/2 sixteenth of an octave
        // (ln 2 / 16)^n / n!
        double p = 9.181219573844436e-12;
        p = fma(p, r, 1.271587195055813e-9);
        p = fma(p, r, 1.467610032291943e-7);
        p = fma(p, r, 1.3550807779497455e-5);
        p = fma(p, r, 9.383847928089871e-4);
        p = fma(p, r, 4.332169878499658e-2);
        p = fma(p, r, 1.0);
        p *= tab[k & 15];
        return __hiloint2double(__double2hiint(p) + ((k >> 4) << 20), __double2loint(p));
    }
    // (m - x) / T in bins, before rounding down; falls with x.
    __device__ __forceinline__ float z(float x) const { return (mf - x) * inv_t; }
    __device__ __forceinline__ int bin(float x) const { return min((int)fminf(z(x), 4096.f), kBins - 1); }
};

template <typename X> __device__ __forceinline__ float clean(X v) {      // NaN counts as -infinity
    const float x = to_f(v);
    return x != x ? -INFINITY : x;
}

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
// Falling bitonic sort of n (a power of two, 64 .. kList) entries. Pairs at most 32 apart
// stay within one warp's 64 entries.
__device__ void sort_falling(uint64_t* a, int n) {
    const int tid = threadIdx.x;
    __syncthreads();
    for (int k = 2; k <= n; k <<= 1) {
        for (int j = k >> 1; j > 0; j >>= 1) {
            for (int t = tid; t < n / 2; t += kThreads) {
                const int i = 2 * t - (t & (j - 1));
                const uint64_t x = a[i], y = a[i + j];
                if ((x < y) == ((i & k) == 0)) { a[i] = y; a[i + j] = x; }
            }
            if (j > 32 || (j == 1 && k >= 64)) __syncthreads(); else __syncwarp();
        }
    }
    __syncthreads();
}

template <typename X>
__global__ void __launch_bounds__(kThreads, 3) sample_kernel(SampleParams P) {
    constexpr int VEC = 16 / (int)sizeof(X);
    extern __shared__ __align__(16) uint8_t smem[];
    uint32_t* hist = reinterpret_cast<uint32_t*>(smem);
    uint64_t* list = reinterpret_cast<uint64_t*>(smem);
    uint4* data = reinterpret_cast<uint4*>(smem + kHeadBytes);
    __shared__ Scratch S;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, C = P.cluster;
    const int rank = C > 1 ? (int)tc::cluster_ctarank() : 0, r = blockIdx.x / C;
    if (C > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");   // waited for before the first exchange
    if (tid == 0) S.x.n_list = 0;
    if (tid < 16) S.tab[tid] = exp2((double)tid * 0.0625);
    pdl_trigger();
    pdl_wait();
    const float T = P.temperature ? P.temperature[r] : 1.f, p = P.top_p ? P.top_p[r] : 1.f, mp = P.min_p ? P.min_p[r] : 0.f, u = P.u[r];
    const int k_in = P.top_k ? P.top_k[r] : 0;

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
    // f(x, index) over vectors [a, b) of the slice, `step` apart
    auto scan = [&](int a, int b, int step, auto f) {
        for (int v = a; v < b; v += step) {
            const uint4 raw = P.resident ? data[v] : fetch(v);
            const X* e = reinterpret_cast<const X*>(&raw);
#pragma unroll
            for (int i = 0; i < VEC; ++i) f(clean(e[i]), s0 + v * VEC + i - off);
        }
    };
    auto each = [&](auto f) { scan(v0 + lane, v1, 32, f); };   // over the slice, a contiguous piece per warp
    auto meet = [&] { if (C > 1) cluster_sync(); else __syncthreads(); };
    auto tell = [&](auto* slots, auto v) { if (tid < C) put(&slots[rank], tid, v); };   // this rank's number, to every CTA
    auto sum_of = [&](const double* slots) {
        double t = 0.0;
        for (int q = 0; q < C; ++q) t += slots[q];
        return t;
    };

    // ---------------------------------------------------------------- the slice, its maximum
    float best = -INFINITY;
    int best_i = 0x7fffffff;
    for (int v = v0 + lane; v < v1; v += 8 * 32) {
        uint4 raw[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (v + 32 * q < v1) raw[q] = fetch(v + 32 * q);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            if (v + 32 * q >= v1) break;
            if (P.resident) data[v + 32 * q] = raw[q];
            const X* e = reinterpret_cast<const X*>(&raw[q]);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float x = clean(e[i]);
                if (x > best) { best = x; best_i = s0 + (v + 32 * q) * VEC + i - off; }
            }
        }
    }
    uint64_t top = block_reduce(rank_of(best, best_i), S.red64, [](uint64_t a, uint64_t b) { return a > b ? a : b; });
    if (C > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    tell(S.x.best, top);
    meet();
    for (int q = 0; q < C; ++q) top = max(top, S.x.best[q]);
    const float mx = key_value((uint32_t)(top >> 32));
    const int top_i = (int)(0xffffffffu - (uint32_t)top);
    if (mx == -INFINITY || !(T > 0.f) || p <= 0.f) {          // nothing to choose from; greedy; the largest alone
        if (rank == 0 && tid == 0) {
            P.tokens[r] = mx == -INFINITY ? -1 : top_i;
            if (P.probs) P.probs[r] = mx == -INFINITY ? 0.f : 1.f;
        }
        return;
    }
    Weights W;
    W.set(mx, T, S.tab);
    const double low = mp > 0.f ? (double)mp : 0.0;
    const bool has_p = p < 1.f, has_k = k_in > 0 && k_in < P.V;
    const int k = k_in;
    uint64_t cut = 0;                                         // candidates below it are dropped

    if (has_p || has_k) {
        // ------------------------------------------------------------ the filters' boundary
        float bound = -INFINITY;                              // elements below it cannot stay
        double total = 0.0;
        if (has_k) {
            if (k <= kThreads) {
                int g = 1;
                while (g < 32 && kThreads / (2 * g) >= k) g *= 2;
                float b = best;
                for (int o = 1; o < g; o <<= 1) b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, o));
                bound = key_value((uint32_t)block_reduce((uint64_t)order_key(b), S.red64, [](uint64_t x, uint64_t y) { return x < y ? x : y; }));
            }
        } else {
            bound = mx - T * (logf((float)P.V / (1.f - p)) + 0.01f);
            double mine = 0.0;
            each([&](float x, int) { mine += W(x); });
            total = block_sum(mine, S.red);
            tell(S.x.total, total);
        }
        // a histogram of the slice, then sums of the rank's share of the bins over the cluster
        const int nb = kBins / C;
        auto histogram = [&](auto bin_of) {                   // bin_of: -1 for an element that takes no part
            for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
            __syncthreads();
            each([&](float x, int) {
                const int b = bin_of(x);
                if (b >= 0) atomicAdd(&hist[b], 1u);
            });
            meet();
        };
        // weight at the left edge of bin b: bins [z0, z0 + nz) of the first histogram over kBins
        float z0 = 0.f, dz = 1.f;
        auto edge = [&](int b) { return (double)__expf(-(z0 + dz * (float)b) * (1.f / kPerUnit)); };
        auto lower = [&](int b) { return b == kBins - 1 ? 0.0 : edge(b + 1) * (1.0 - kSlack); };   // the last bin has no end
        auto upper = [&](int b) { return edge(b) * (1.0 + kSlack); };
        auto gather_bins = [&] {
            double n = 0.0, lo = 0.0, up = 0.0;
            for (int b = rank * nb + tid; b < (rank + 1) * nb; b += kThreads) {
                uint32_t c = 0;
                for (int q = 0; q < C; ++q) c += get_u32(&hist[b], q);
                hist[b] = c;                                  // no other rank reads this rank's share before the next meeting
                n += c;
                if (!has_k) { lo += c * lower(b); up += c * upper(b); }
            }
            tell(S.x.cnt, block_sum(n, S.red));
            if (!has_k) {
                tell(S.x.lo, block_sum(lo, S.red));
                tell(S.x.up, block_sum(up, S.red));
            }
            meet();
        };
        // The first bin at which the running sum of `slots` (a bin's count times weight(b)) reaches
        // `want`, or the last; *before: elements of the bins before it, *upto: with its own.
        auto cross = [&](const double* slots, auto weight, double want, double* before, double* upto) {
            double sum = 0.0, cnt = 0.0;
            int q = 0;
            for (; q < C - 1 && !(sum + slots[q] >= want); ++q) { sum += slots[q]; cnt += S.x.cnt[q]; }
            const int per = (nb + kThreads - 1) / kThreads;
            uint32_t c[kBins / kThreads];
            double n = 0.0, v = 0.0;
#pragma unroll
            for (int i = 0; i < kBins / kThreads; ++i) {
                const int b = tid * per + i;
                c[i] = i < per && b < nb ? get_u32(&hist[q * nb + b], q) : 0u;
                n += c[i];
                v += c[i] * weight(q * nb + min(b, nb - 1));
            }
            double all_v, all_n;
            double pv = sum + block_scan(v, S.red, &all_v), pn = cnt + block_scan(n, S.red, &all_n);
            if (tid == 0) { S.cross_bin = kBins; }
            __syncthreads();
            int mine = kBins;
            double mine_n = 0.0;
#pragma unroll
            for (int i = 0; i < kBins / kThreads; ++i) {
                const int b = tid * per + i;
                if (i >= per || b >= nb) break;
                pv += c[i] * weight(q * nb + b);
                if (mine == kBins && pv >= want) { mine = q * nb + b; mine_n = pn; }
                pn += c[i];
            }
            if (mine < kBins) atomicMin(&S.cross_bin, mine);
            __syncthreads();
            const int bin = S.cross_bin;
            if (mine == bin && mine < kBins) {
                S.cross_before = mine_n;
                S.found = (int)c[0];
#pragma unroll
                for (int i = 1; i < kBins / kThreads; ++i)
                    if (tid * per + i == bin - q * nb) S.found = (int)c[i];
            }
            __syncthreads();
            if (bin == kBins) {                               // not reached in these bins: their last
                *before = cnt;
                *upto = cnt + all_n;
                return (q + 1) * nb - 1;
            }
            *before = S.cross_before;
            *upto = S.cross_before + S.found;
            return bin;
        };
        // The chosen elements' ranks into the list of CTA 0.
        auto gather = [&](auto chosen) {
            int n = 0;
            each([&](float x, int) { n += chosen(x); });
            int inc = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            uint32_t at = 0;
            if (lane == 31 && inc > 0) at = add_u32(&S.x.n_list, 0, (uint32_t)inc);
            at = __shfl_sync(0xffffffffu, at, 31) + (uint32_t)(inc - n);
            if (n > 0)
                each([&](float x, int i) {
                    if (chosen(x) && at < (uint32_t)kList) put(&list[at++], 0, rank_of(x, i));
                });
            meet();
        };
        auto sort_list = [&](int n) {
            int m = 64;
            while (m < n) m *= 2;
            for (int i = n + tid; i < m; i += kThreads) list[i] = 0;
            sort_falling(list, m);
            return m;
        };
        const double one = 1.0;
        histogram([&](float x) { return x >= bound && x > -INFINITY ? W.bin(x) : -1; });
        if (!has_k) total = sum_of(S.x.total);
        gather_bins();
        double before, upto;
        const int b_hi = has_k ? cross(S.x.cnt, [&](int) { return one; }, (double)k, &before, &upto)
                               : cross(S.x.lo, lower, (double)p * total, &before, &upto);
        bool bisect = false;
        if (upto <= (double)kList) {
            // -------------------------------------------------------- a short list: CTA 0 finishes the row
            meet();                                           // every rank has read the bins that the list overwrites
            gather([&](float x) { return x >= bound && x > -INFINITY && W.bin(x) <= b_hi; });
            if (rank != 0) return;
            const int n = (int)min(S.x.n_list, (unsigned)kList), m = sort_list(n);
            const int nk = has_k ? min(n, k) : n;
            constexpr int PER = kList / kThreads;
            uint64_t e[PER];
            double w[PER], mine = 0.0, all;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int q = tid * PER + i;
                e[i] = q < nk ? list[q] : 0;
                w[i] = q < nk ? W(key_value((uint32_t)(e[i] >> 32))) : 0.0;
                mine += w[i];
            }
            double cum = block_scan(mine, S.red, &all);
            const double target = (double)p * (has_k ? all : total);
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int q = tid * PER + i;
                const bool keep = q < nk && (q == 0 || ((!has_p || cum < target) && w[i] >= low));
                cum += w[i];
                // by rising index: the largest key first after the complement
                if (q < m) list[q] = keep ? ~(((uint64_t)(0xffffffffu - (uint32_t)e[i]) << 32) | (uint32_t)(e[i] >> 32)) : 0;
            }
            sort_falling(list, m);
            mine = 0.0;
            int last = -1;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int q = tid * PER + i;
                e[i] = q < m ? list[q] : 0;
                w[i] = e[i] ? W(key_value((uint32_t)~e[i])) : 0.0;
                if (w[i] > 0.0) last = q;
                mine += w[i];
            }
            cum = block_scan(mine, S.red, &all);
            if (tid == 0) S.found = kList;
            __syncthreads();
            const double want = (double)u * all;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                cum += w[i];
                if (w[i] > 0.0 && cum > want) { atomicMin(&S.found, tid * PER + i); break; }
            }
            const int end = (int)block_reduce((double)last, S.red, [](double a, double b) { return fmax(a, b); });
            __syncthreads();
            const int at = S.found < kList ? S.found : end;
            if (tid == at / PER) {
                const uint64_t v = ~list[at];
                P.tokens[r] = (int)(v >> 32);
                if (P.probs) P.probs[r] = (float)(W(key_value((uint32_t)v)) / all);
            }
            return;
        }
        if (!has_k) {
            // -------------------------------------------------------- a long prefix: the boundary's bins once more
            const double target = (double)p * total;
            double skip, skip2;
            const int b_lo = b_hi, b_up = cross(S.x.up, upper, target, &skip, &skip2);
            meet();
            z0 = (float)b_up;
            dz = (float)(b_lo + 1 - b_up) / (float)kBins;
            const float inv_dz = (float)kBins / (float)(b_lo + 1 - b_up);
            auto sub = [&](float x) {                         // -1: above, kBins: below, else the finer bin
                const int b = W.bin(x);
                if (b < b_up) return -1;
                if (b > b_lo || x == -INFINITY) return kBins;
                return min((int)fminf((W.z(x) - z0) * inv_dz, 4096.f), kBins - 1);
            };
            double mine = 0.0;
            histogram([&](float x) {
                const int b = sub(x);
                if (b < 0) mine += W(x);
                return b < kBins ? b : -1;
            });
            const double above0 = block_sum(mine, S.red);
            tell(S.x.above, above0);
            meet();
            const double above = sum_of(S.x.above);
            gather_bins();
            double n0, n1;
            const int s_up = cross(S.x.up, upper, target - above, &n0, &skip);
            const int s_lo = cross(S.x.lo, lower, target - above, &skip, &n1);
            if (n1 - n0 <= (double)kList) {
                meet();
                double m2 = 0.0;
                each([&](float x, int) {
                    const int b = sub(x);
                    if (b >= 0 && b < s_up) m2 += W(x);
                });
                tell(S.x.above2, block_sum(m2, S.red));
                gather([&](float x) { const int b = sub(x); return b >= s_up && b <= s_lo; });
                if (rank == 0) {
                    const double a2 = above + sum_of(S.x.above2);
                    const int n = (int)min(S.x.n_list, (unsigned)kList);
                    sort_list(n);
                    constexpr int PER = kList / kThreads;
                    double w[PER], own = 0.0, all;
#pragma unroll
                    for (int i = 0; i < PER; ++i) {
                        const int q = tid * PER + i;
                        w[i] = q < n ? W(key_value((uint32_t)(list[q] >> 32))) : 0.0;
                        own += w[i];
                    }
                    double cum = a2 + block_scan(own, S.red, &all);
                    int stay = 0;                             // the list's first `stay` entries stay
#pragma unroll
                    for (int i = 0; i < PER; ++i) {
                        stay += tid * PER + i < n && cum < target;
                        cum += w[i];
                    }
                    stay = (int)block_sum((double)stay, S.red);
                    const uint64_t c = n == 0 ? 0 : stay > 0 ? list[stay - 1] : list[0] + 1;
                    if (tid < C) put(&S.x.cut, tid, c);
                }
                meet();
                cut = min(S.x.cut, top);                      // the largest always stays
            } else {
                bisect = true;
            }
        } else {
            bisect = true;
        }
        if (bisect) {
            // -------------------------------------------------------- too many equal or too close: bisection of the rank
            int turn = 0;
            auto measure = [&](uint64_t c, bool with_c, bool mass, double* n) {   // of the candidates above c (and not below `cut`)
                double nn = 0.0, mm = 0.0;
                each([&](float x, int i) {
                    const uint64_t v = rank_of(x, i);
                    if (x > -INFINITY && v >= cut && (v > c || (with_c && v == c))) {
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
            if (has_k) {                                      // the largest c with k candidates at or above it
                measure(0, true, false, &n);
                if (n > (double)k) {
                    uint64_t lo = 0, hi = top + 1;
                    while (hi - lo > 1) {
                        const uint64_t mid = lo + ((hi - lo) >> 1);
                        measure(mid, true, false, &n);
                        if (n >= (double)k) lo = mid; else hi = mid;
                    }
                    cut = lo;
                }
            }
            if (has_p) {                                      // the smallest c with less than the target's mass above it
                const double target = (double)p * measure(0, true, true, &n);
                uint64_t lo = cut, hi = top;                  // hi always qualifies: nothing lies above it
                while (lo < hi) {
                    const uint64_t mid = lo + ((hi - lo) >> 1);
                    if (measure(mid, false, true, &n) < target) hi = mid; else lo = mid + 1;
                }
                cut = lo;
            }
        }
    }

    // -------------------------------------------------------------------- the draw, in the vocabulary's order
    const float cut_x = key_value((uint32_t)(cut >> 32));
    const uint32_t cut_i = 0xffffffffu - (uint32_t)cut;
    auto weight = [&](float x, int i) {                       // 0: dropped
        if (cut != 0 && !(x > cut_x || (x == cut_x && (uint32_t)i <= cut_i))) return 0.0;
        const double w = W(x);
        return w >= low || i == top_i ? w : 0.0;
    };
    double mine = 0.0;
    each([&](float x, int i) { mine += weight(x, i); });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    __syncthreads();
    if (lane == 0) S.wsum[wid] = mine;
    __syncthreads();
    double slice_sum = 0.0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) slice_sum += S.wsum[w];
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
    const int a0 = min(nvec, piece * per_warp), a1 = min(nvec, a0 + per_warp), each_n = (a1 - a0 + kThreads - 1) / kThreads;
    const int t0 = min(a1, a0 + tid * each_n), t1 = min(a1, t0 + each_n);
    mine = 0.0;
    int last = -1;
    scan(t0, t1, 1, [&](float x, int i) {
        const double w = weight(x, i);
        if (w > 0.0) { mine += w; last = i; }
    });
    double part;
    cum = piece_cum + block_scan(mine, S.red, &part);
    if (tid == 0) S.found = 0x7fffffff;
    __syncthreads();
    if (last >= 0 && cum + mine > want) {
        int hit = 0x7fffffff;
        scan(t0, t1, 1, [&](float x, int i) {
            const double w = weight(x, i);
            if (w <= 0.0) return;
            cum += w;
            if (hit == 0x7fffffff && cum > want) hit = i;
        });
        atomicMin(&S.found, hit);
    }
    const int end = (int)block_reduce((double)last, S.red, [](double a, double b) { return fmax(a, b); });
    __syncthreads();
    if (tid == 0) {
        const int at = S.found != 0x7fffffff ? S.found : end;
        P.tokens[r] = at;
        if (P.probs) P.probs[r] = (float)(W(clean(row[at])) / all);
    }
}

constexpr size_t kSliceBytes = 65536;                // three CTAs an SM
constexpr size_t kSliceMax = 196608;

template <typename X>
cudaError_t launch(SampleParams P, cudaStream_t s) {
    constexpr int VEC = 16 / (int)sizeof(X);
    // The row is split until a slice fits a third of an SM's shared memory, and further while the
    // rows alone leave SMs idle and a slice is long enough to pay for the exchanges.
    auto slice = [&](int c) { return (int)(((int64_t)P.V + VEC - 1 + c - 1) / c + VEC - 1) / VEC * VEC; };
    int c = 1;
    while (c < kMaxCluster && (slice(c) * sizeof(X) > kSliceBytes + 64 || ((int64_t)P.rows * c < 444 && slice(c) > 8192))) c *= 2;
    P.cluster = c;
    P.slice = slice(c);
    P.resident = P.slice * sizeof(X) <= kSliceMax;
    const size_t smem = kHeadBytes + (P.resident ? P.slice * sizeof(X) : 0);
    auto kern = sample_kernel<X>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(kHeadBytes + kSliceMax));
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) e = launch_pdl_cluster(kern, dim3((unsigned)(P.rows * c)), dim3(kThreads), c, smem, s, P);
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
