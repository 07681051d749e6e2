// dspark_attend_paged on the tcgen05 tensor cores (bf16 or fp16 caches, head_dim
// a multiple of 64, pages of a power of two >= 8 rows).
//
// A unit is up to NQ query tiles of one (request, kv head): the grp query heads
// that share the kv head times tpt = 128 / grp tokens fill the 128 rows of a tile
// (row r = token r / grp, head r % grp), so K and V are read once for all of them. Its
// key tiles of KT rows are gathered from the pages by TMA, a copy per page
// and 64 dimensions (one per page of 16 rows), into the swizzled layout the MMAs read.
//   S = Q K^T -> TMEM; P = exp2(scale log2(e) (S - m)) -> TMEM over
//   its S buffer, in the cache's type (both operands of an MMA have one type;
//   the sums take the unrounded P); O += P V -> TMEM.
// What the rounded P costs: over random keys the result's error is 1.3 to 1.4 times that of its own last rounding (bf16
// 0.0023 for 0.0017 relative, fp16 0.00029 for 0.00021); a second product for P's low half would double PV.
// The running maximum m is raised only when a tile's exceeds it by 8 (log2), so O
// is rarely rescaled; P stays below 256.
//
// Bound by the K and V bytes for few new tokens (64 requests of 8K to 32K keys, one token each: 860 us in a short run, 6.0
// TB/s, 925 to 1000 in a long one, by the GPU; 745 with pages of 64; head_dim 64 moves 32 KB a step and stays at 3.4 to 4.4
// TB/s), by the chain S -> softmax -> PV for prompt chunks (4 x 2048 tokens over up to 8K keys, head_dim 128: 450 us,
// 1000 TFLOP/s, tensor pipe 53% active; 510 to 520 us in a long run, at the power limit's clocks). head_dim 256 has the
// same chain with one query tile and 64 keys a step (8191 tokens in a window of 1024: 185 us, 200 in a long run, tensor pipe 43%, L2
// at 27% of its rate; units of 17 tiles pay their start and epilogue too: 690 to 750 TFLOP/s, 900 without the window). One
// request's 17 tokens over 4096 keys take 21 us: two launches, and a few microseconds each for finding the share, the
// first tile and the pieces' join.
//
// Steps: with NQ = 2 (prompt chunks, head_dim <= 128, KT = 128) step s is tile s / 2 of
// query tile s % 2, with NQ = 1 it is tile s; step s uses S buffer s % 2. The
// MMA thread issues S(0), S(1), then PV(s), S(s + 2): while one buffer is in the softmax
// the tensor cores work on the other. MMAs of one thread run in order, so S(s + 2) may
// overwrite the P that PV(s) reads. head_dim 192 and 256 keep Q in tensor memory (O, two
// S buffers of 64 columns and Q fill its 512 columns): with Q in shared
// memory the S product would read 192 bytes a cycle, above the 128 it can.
//
// Work split: the units' tiles (plus kUnitCost a unit for its fixed work), laid end to
// end, are cut into equal contiguous shares, one per CTA, whatever the
// requests' lengths (which only the device knows): each CTA finds its share's start, and the units that a cut crosses
// are listed. Those units' pieces write O / l (fp32) and (m, l)
// per row, which a merge kernel joins in order: results do not depend on timing.
//
// Warp roles: 8 softmax warps (TMEM lane = query row; NQ = 1: two threads to a row), then one warp
// each for the loads, the MMAs, and zeroing V rows outside the unit's keys (those
// rows may hold anything; P = 0 times NaN would poison O. K needs no care:
// masked scores are replaced). Every wait is bounded.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "paged.h"
#include "tc_ptx.cuh"

namespace dspark {
namespace tc {
namespace {

constexpr int kGrid = 148;           // shares: one CTA per SM of a B200
constexpr int kUnitCost = 4;         // a unit's fixed work (query tile, first load, epilogue) in tiles (2 to 4 measure alike, 1 and 6 worse)
constexpr int kRows = 128;           // rows of a query tile: the MMAs' M
constexpr int kMaxBatch = 4096;
constexpr float kRescale = 8.0f;     // log2 headroom before the running maximum is raised
constexpr size_t kSmemMax = 232448;

struct Share { int b, g, qt, x; int64_t len; };          // first unit, offset in it, total length (cost units)
struct MergeUnit { int b, g, qt, c0, odd, c1; };         // pieces: slot 2 c0 + odd, then slots 2 (c0 + 1) .. 2 c1; c1 < 0: none

struct Params {
    PagedAttn a;
    MergeUnit* merges;               // [kGrid]
    float4* part_o; float2* part_ml;  // [2 kGrid][NQ][hd / 4][128], [2 kGrid][NQ][128]
    int tpt, tpu;                    // tokens per query tile, per unit
    int page_shift;
    int32_t* status;
};

// Request b as every role sees it.
struct Req { int t0, n, L; };
__device__ __forceinline__ Req load_req(const PagedAttn& a, int b) {
    Req r;
    r.t0 = min(max(a.cu[b], 0), a.T);
    r.n = min(max(a.cu[b + 1], r.t0), a.T) - r.t0;
    r.L = (int)min((int64_t)min(max(a.kv_len[b], 0), kMaxKeys), (int64_t)a.max_pages * a.page_size);
    return r;
}
// The keys [lo, hi) that some query of unit qt sees (hi <= lo: none).
template <int KT>
__device__ __forceinline__ void unit_keys(const PagedAttn& a, const Req& r, int tpu, int qt, int* lo, int* hi) {
    const int i0 = qt * tpu, i1 = min(r.n, i0 + tpu) - 1;     // its tokens
    const int p0 = r.L - r.n + i0, p1 = r.L - r.n + i1;       // their keys
    *hi = a.causal ? min(r.L, p1 + 1) : r.L;
    *lo = a.window > 0 ? max(0, p0 - a.window + 1) : 0;
    if (*hi <= *lo) *hi = *lo = 0;
}
template <int KT>
__device__ __forceinline__ int unit_tiles(const PagedAttn& a, const Req& r, int tpu, int qt) {
    int lo, hi;
    unit_keys<KT>(a, r, tpu, qt, &lo, &hi);
    return hi > lo ? (hi + KT - 1) / KT - lo / KT : 0;
}

// A share's pieces, in order.
struct Piece {
    int b, g, qt;
    Req r;
    int lo, hi;          // the unit's keys
    int t0, nt;          // first key tile (of KT keys) and number of tiles
    bool whole;          // the unit's only piece: the output is written directly
    int slot;            // else the slot of its partial result
    int index;           // pieces with tiles before it in this share
};
template <int KT>
struct Walk {
    int b, g, qt, x, c, index;
    int64_t rem;
    bool first, have;
    Req r;
    __device__ __forceinline__ Walk(const Share& s, int cta) {
        b = s.b; g = s.g; qt = s.qt; x = s.x; rem = s.len; c = cta; index = 0; first = true; have = false;
    }
    __device__ __forceinline__ bool next(const Params& P, Piece* p) {
        while (rem > 0) {
            if (!have) {
                r = load_req(P.a, b);
                have = true;
                if (r.n == 0) {                                // no unit here
                    if (++b >= P.a.B) return false;
                    g = qt = x = 0; have = false;
                    continue;
                }
            }
            int lo, hi;
            unit_keys<KT>(P.a, r, P.tpu, qt, &lo, &hi);
            const int nt = hi > lo ? (hi + KT - 1) / KT - lo / KT : 0;
            const int cost = kUnitCost + nt;
            const int x0 = x, x1 = (int)min((int64_t)cost, x0 + rem);
            const int f0 = min(max(x0 - kUnitCost, 0), nt), f1 = min(max(x1 - kUnitCost, 0), nt);
            p->b = b; p->g = g; p->qt = qt; p->r = r; p->lo = lo; p->hi = hi;
            p->t0 = lo / KT + f0; p->nt = f1 - f0;
            p->whole = f1 - f0 == nt;
            p->slot = 2 * c + (first ? 0 : 1);
            p->index = index;
            rem -= x1 - x0;
            first = false;
            if (x1 == cost) {
                x = 0;
                if ((qt + 1) * P.tpu >= r.n) {
                    qt = 0;
                    if (++g == P.a.nKv) { g = 0; ++b; have = false; if (b >= P.a.B) rem = 0; }
                } else {
                    ++qt;
                }
            } else {
                x = x1;
            }
            if (f1 > f0) { ++index; return true; }
            if (nt == 0 && x1 == cost) return true;         // no keys: zeros to write
        }
        return false;
    }
};

// ------------------------------------------------------------------ plan
// Every CTA finds its own share (a kernel before this one would cost more than the few microseconds this takes): the
// requests' costs and their prefix sums over the block, then warp 0 places the share. It also lists the unit, if any,
// whose first cut between tiles is this share's start. pre: B + 1 numbers of scratch; buf: one per warp.
template <int KT>
__device__ __forceinline__ void plan_share(const Params& P, int64_t* pre, int64_t* buf, Share* share) {
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, B = P.a.B, threads = blockDim.x, warps = threads >> 5;
    const int cta = blockIdx.x;
    // a request's cost: a thread per request for few units each, a warp for many
    const bool by_warp = P.a.max_new > 4 * P.tpu;
    for (int b = by_warp ? wid : tid; b < B; b += by_warp ? warps : threads) {
        const Req r = load_req(P.a, b);
        int64_t cost = 0;
        const int units = (r.n + P.tpu - 1) / P.tpu;
        for (int qt = by_warp ? lane : 0; qt < units; qt += by_warp ? 32 : 1)
            cost += kUnitCost + unit_tiles<KT>(P.a, r, P.tpu, qt);
        if (by_warp) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) cost += __shfl_xor_sync(0xffffffffu, cost, o);
        }
        if (!by_warp || lane == 0) {
            pre[b] = cost;
            if (cta == 0 && (P.a.kv_len[b] != r.L || P.a.cu[b] != r.t0 || P.a.cu[b + 1] != r.t0 + r.n)) atomicOr(P.status, DSPARK_DEV_BAD_LENGTH);
        }
    }
    __syncthreads();
    // exclusive prefix sums, a contiguous run of requests per thread
    const int per = (B + threads - 1) / threads, b0 = min(B, tid * per), b1 = min(B, b0 + per);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += pre[b] * P.a.nKv;
    int64_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) buf[wid] = inc;
    __syncthreads();
    int64_t base = 0, W = 0;
    for (int w = 0; w < warps; ++w) {
        if (w < wid) base += buf[w];
        W += buf[w];
    }
    base += inc - mine;
    for (int b = b0; b < b1; ++b) {
        const int64_t cb = pre[b] * P.a.nKv;
        pre[b] = base;
        base += cb;
    }
    if (tid == 0) pre[B] = W;
    __syncthreads();
    if (wid == 0) {
        // shares of at least kUnitCost + 1: below that a piece is all fixed work
        const int64_t G = min((int64_t)kGrid, max((int64_t)1, W / (kUnitCost + 1)));
        auto start = [&](int64_t c) { return c >= G ? W : W * c / G; };
        const int64_t lo = start(cta), hi = start(cta + 1);
        Share s{0, 0, 0, 0, hi - lo};
        MergeUnit mu{0, 0, 0, 0, 0, -1};
        if (hi > lo) {
            int l = 0, h = B;                                // the last request that starts at or before lo and is not empty
            while (h - l > 1) {
                const int mid = (l + h) >> 1;
                if (pre[mid] <= lo) l = mid; else h = mid;
            }
            const Req r = load_req(P.a, l);
            const int64_t cg = (pre[l + 1] - pre[l]) / P.a.nKv;
            int64_t rest = lo - pre[l];
            s.b = l;
            s.g = (int)(rest / cg);
            rest -= s.g * cg;
            int cost = 0;
            for (int qt = 0;; qt += 32) {                    // 32 units at a time
                const int mine = kUnitCost + unit_tiles<KT>(P.a, r, P.tpu, min(qt + lane, (r.n - 1) / P.tpu));
                int64_t sum = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int64_t y = __shfl_up_sync(0xffffffffu, sum, o);
                    if (lane >= o) sum += y;
                }
                const unsigned over = __ballot_sync(0xffffffffu, sum > rest);
                if (over) {
                    const int k = __ffs(over) - 1;
                    s.qt = qt + k;
                    cost = __shfl_sync(0xffffffffu, mine, k);
                    s.x = (int)(rest - __shfl_sync(0xffffffffu, sum - mine, k));
                    break;
                }
                rest -= __shfl_sync(0xffffffffu, sum, 31);
            }
            const int64_t u0 = lo - s.x;                     // where the unit starts
            if (cta > 0 && s.x > kUnitCost && start(cta - 1) - u0 <= kUnitCost) {
                mu.b = s.b; mu.g = s.g; mu.qt = s.qt;
                mu.c0 = cta - 1;
                mu.odd = start(cta - 1) < u0;                // not the first region of that share
                int c1 = cta;
                while (c1 + 1 < G && start(c1 + 1) < u0 + cost) ++c1;
                mu.c1 = c1;
            }
        }
        if (lane == 0) {
            *share = s;
            P.merges[cta] = mu;
        }
    }
    __syncthreads();
}

// ------------------------------------------------------------------ PTX used here alone
__device__ __forceinline__ void tmem_ld_x32(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The largest; a NaN wins, so that a row's maximum tells of it (the polynomial below would hide one).
__device__ __forceinline__ float max2(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// Two fp32 lanes in one register pair: one instruction for both.
__device__ __forceinline__ uint64_t f2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void f2_out(uint64_t v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// 2^x for two x in [-126, 127) on the FMA pipe: the nearest integer goes into the exponent, 2^f on |f| <= 1/2 is a polynomial
// of degree 5 fitted for the relative error (2^-22.6 in exact arithmetic, within 2^-22 as evaluated here in fp32, which is
// what ex2.approx is good for: far inside the rounding of P to 16 bits). The special function unit does 16
// a clock, which is what a 128 x 128 tile's two products leave time for: some of them here make room.
__device__ __forceinline__ void exp2_poly(uint64_t x, float& p0, float& p1) {
    const uint64_t magic = f2(12582912.f, 12582912.f);          // 1.5 2^23: the sum's low bits are the integer
    const uint64_t t = add2(x, magic), n = add2(t, f2(-12582912.f, -12582912.f)), f = fma2(n, f2(-1.f, -1.f), x);
    uint64_t p = fma2(f2(1.327647129073739e-3f, 1.327647129073739e-3f), f, f2(9.675540961325169e-3f, 9.675540961325169e-3f));
    p = fma2(p, f, f2(5.550713092088699e-2f, 5.550713092088699e-2f));
    p = fma2(p, f, f2(0.24022120237350464f, 0.24022120237350464f));
    p = fma2(p, f, f2(0.6931469440460205f, 0.6931469440460205f));
    p = fma2(p, f, f2(1.0000001192092896f, 1.0000001192092896f));
    float a, b, ta, tb;
    f2_out(p, a, b);
    f2_out(t, ta, tb);
    p0 = __uint_as_float(__float_as_uint(a) + (__float_as_uint(ta) << 23));
    p1 = __uint_as_float(__float_as_uint(b) + (__float_as_uint(tb) << 23));
}
// Lane j of four has blocks 0 .. 3 (four words each) of row j; after this, block j of rows 0 .. 3.
__device__ __forceinline__ void transpose_blocks(uint32_t (&w)[16], int lane) {
#pragma unroll
    for (int x = 1; x <= 2; x *= 2) {
        const bool odd = lane & x;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            if (b & x) continue;                              // blocks b and b + x
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t t = __shfl_xor_sync(0xffffffffu, odd ? w[4 * b + i] : w[4 * (b + x) + i], x);
                if (odd) w[4 * b + i] = t; else w[4 * (b + x) + i] = t;
            }
        }
    }
}
// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
// A value that all lanes share, known as such to the compiler.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }
template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b);
template <> __device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T> __host__ __device__ constexpr uint32_t idesc(int M, int N, int b_mn_major);
template <> __host__ __device__ constexpr uint32_t idesc<__half>(int M, int N, int mn) { return idesc_f16(M, N, mn); }
template <> __host__ __device__ constexpr uint32_t idesc<__nv_bfloat16>(int M, int N, int mn) {
    return idesc_bf16(M, N) | (uint32_t(mn) << 16);
}

// ------------------------------------------------------------------ the kernel
template <int HD_, int NQ_, int KT_, bool QTMEM_, bool P16_ = false>
struct Cfg {
    static constexpr int HD = HD_, NQ = NQ_, KT = KT_;
    // Pages of 16 rows, one query tile: a page is one copy of all its chunks, [page][chunk][16 rows x 128 B] (a copy a chunk
    // is 2 KB, and their number then bounds the loads: 990 us for 64 long requests, against 750 with pages of 64). The
    // MMAs take eight rows at a fixed stride, so the keys go in two classes, rows 0 - 7 of every page, then rows 8 - 15.
    static constexpr bool P16 = P16_;
    static constexpr bool QTMEM = QTMEM_;                     // Q in tensor memory (staged through ring slots)
    static constexpr int NCH = HD / 64;                       // 64-dimension chunks
    static constexpr int kChunk = kRows * 128;                // a chunk of a query tile
    static constexpr int kTile = KT * HD * 2;                 // a K or V tile
    static constexpr int kQBytes = QTMEM ? 0 : NQ * NCH * kChunk;
    // Softmax threads per query row. With one query tile its softmax is the chain that the MMAs wait for, so
    // two threads share a row; with two tiles one's softmax runs beside the other's MMAs, and two
    // threads would not have the registers.
    static constexpr int SP = NQ == 1 ? 2 : 1;
    static constexpr int kSoft = NQ * SP * 128;
    static constexpr int kThreads = kSoft + 96;
    static constexpr int CH = KT / SP;                        // a thread's keys of a tile
    static constexpr int kTail = 512 + (SP == 2 ? kSoft * 8 : 0);   // barriers; two numbers per softmax thread
    static constexpr int kSlotsFit = (int)((kSmemMax - 1024 - kTail - kQBytes) / kTile);
    static constexpr int NS = kSlotsFit < 12 ? kSlotsFit : 12;
    static constexpr int kQPerSlot = kTile / kChunk;          // staged query chunks per slot
    static constexpr int kQSlots = QTMEM ? (NCH + kQPerSlot - 1) / kQPerSlot : 0;
    static constexpr int kOCol = 2 * KT, kQCol = 2 * KT + HD; // TMEM columns: S buffers, O tiles, Q
    static constexpr size_t kSmem = 1024 + kQBytes + (size_t)NS * kTile + kTail;
    static_assert(kSmem <= kSmemMax && (size_t)NS * kTile >= (kMaxBatch + 33) * 8, "shared memory");
    static_assert(2 * KT + NQ * HD + (QTMEM ? HD / 2 : 0) <= 512, "tensor memory");
};

struct Bars {
    uint64_t full[12], free_[12], vissued[12], vready[12];
    uint64_t sdone[2], pready[2], phalf[2], odone[2];
    uint64_t qfull, qfree, spare;
    Share share;
    uint32_t tmem;
    int abort;
};
constexpr int kBarBytes = 512;
static_assert(sizeof(Bars) <= kBarBytes, "barrier block");

// Ring entries before tile t's K and V within a piece of nt tiles: the order the MMAs take them in.
template <int NQ> __device__ __forceinline__ int k_entry(int t) { return NQ == 2 ? 2 * t : t == 0 ? 0 : 2 * t - 1; }
template <int NQ> __device__ __forceinline__ int v_entry(int t, int nt) {
    return NQ == 2 ? 2 * t + 1 : t == nt - 1 ? 2 * nt - 1 : 2 * t + 2;
}

template <typename T, typename C>
__global__ void __launch_bounds__(C::kThreads, 1)
attend_paged_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, Params P) {
    constexpr int HD = C::HD, NQ = C::NQ, KT = C::KT, NCH = C::NCH, NS = C::NS;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sQ = base;                                       // [NQ][NCH][128 rows x 128 B]
    uint8_t* ring = base + C::kQBytes;                        // NS tiles, [NCH][KT rows x 128 B]
    Bars& B = *reinterpret_cast<Bars*>(ring + (size_t)NS * C::kTile);
    float* s_half = reinterpret_cast<float*>(ring + (size_t)NS * C::kTile + kBarBytes);   // [2][SP][128]
    volatile int* abort_flag = &B.abort;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int kLoadWarp = C::kSoft / 32, kMmaWarp = kLoadWarp + 1, kFixWarp = kLoadWarp + 2;

    if (tid == 0) {
        for (int i = 0; i < NS; ++i) { mbar_init(&B.full[i], 1); mbar_init(&B.free_[i], 1); mbar_init(&B.vissued[i], 1); mbar_init(&B.vready[i], 1); }
        for (int i = 0; i < 2; ++i) { mbar_init(&B.sdone[i], 1); mbar_init(&B.pready[i], C::SP * 128); mbar_init(&B.phalf[i], C::SP * 128); mbar_init(&B.odone[i], 1); }
        mbar_init(&B.qfull, C::QTMEM ? C::SP * 128 : 1);
        mbar_init(&B.qfree, 1);
        mbar_init(&B.spare, 1);
        B.abort = 0;
        mbar_fence_init();
        prefetch_tmap(&tmQ); prefetch_tmap(&tmK); prefetch_tmap(&tmV);
    }
    if (warp == kMmaWarp) tmem_alloc(&B.tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = B.tmem;
    pdl_wait();

    int64_t* scratch = reinterpret_cast<int64_t*>(ring);
    plan_share<KT>(P, scratch, scratch + kMaxBatch + 1, &B.share);
    fence_async_shared();                                     // the ring was scratch: TMA writes it next
    __syncthreads();
    Walk<KT> walk(B.share, blockIdx.x);
    Piece p;
    int e = 0;                                                // ring entries before the piece
    int gs = 0;                                               // steps before the piece
    bool ok = true;

    if (warp == kLoadWarp) {
        // ------------------------------------------------------------ loads
        const int box = min(P.a.page_size, KT), per_tile = KT / box;
        const int sub = C::P16 ? lane : lane / NCH, ch = C::P16 ? 0 : lane % NCH;      // this lane's request of a tile: box `sub`, chunk `ch`
        auto acquire = [&](int entry) {                       // the slot's previous tile has been read
            const int s = entry % NS;
            if (entry >= NS && !__all_sync(0xffffffffu, mbar_wait(&B.free_[s], (uint32_t)(entry / NS - 1) & 1u, abort_flag, P.status)))
                return false;
            return true;
        };
        int issued = 0;
        while (ok && walk.next(P, &p)) {
            if (p.nt == 0) continue;
            const int tok = p.r.t0 + p.qt * P.tpu;
            const uint32_t qbytes = (uint32_t)(P.tpt * P.a.grp * 128);
            if (C::QTMEM) {
                for (int s = 0; s < C::kQSlots && ok; ++s) {
                    if (!acquire(e)) { ok = false; break; }
                    if (lane == 0) {
                        const int c0 = s * C::kQPerSlot, c1 = min(NCH, c0 + C::kQPerSlot);
                        mbar_arrive_expect_tx(&B.full[e % NS], qbytes * (c1 - c0));
                        for (int c = c0; c < c1; ++c)
                            tma_load_4d(ring + (size_t)(e % NS) * C::kTile + (c - c0) * C::kChunk, &tmQ, &B.full[e % NS], c * 64, 0, p.g, tok);
                    }
                    ++e;
                    issued = e;
                }
            } else {
                if (p.index > 0 && !__all_sync(0xffffffffu, mbar_wait(&B.qfree, (uint32_t)(p.index - 1) & 1u, abort_flag, P.status))) { ok = false; break; }
                if (lane == 0) {
                    mbar_arrive_expect_tx(&B.qfull, qbytes * NQ * NCH);
                    for (int q = 0; q < NQ; ++q)
                        for (int c = 0; c < NCH; ++c)
                            tma_load_4d(sQ + (q * NCH + c) * C::kChunk, &tmQ, &B.qfull, c * 64, 0, p.g, tok + q * P.tpt);
                }
            }
            // tile t's pages; boxes without a key of the unit are not loaded
            const int32_t* table = P.a.table + (int64_t)p.b * P.a.max_pages;
            auto page_of = [&](int t) {
                const int key = (p.t0 + t) * KT + sub * box;
                if (sub >= per_tile || t >= p.nt || key >= p.hi || key + box <= p.lo) return -2;
                int page = table[key >> P.page_shift];
                if (page < 0 || page >= P.a.num_pages) {
                    atomicOr(P.status, DSPARK_DEV_BAD_PAGE);
                    page = P.a.num_pages;                      // out of range: reads as zeros
                }
                return page;
            };
            auto load = [&](const CUtensorMap* m, bool v, int t, int page) {
                if (!acquire(e)) return false;
                const int s = e % NS;
                const unsigned act = __ballot_sync(0xffffffffu, page != -2);
                const int k0 = (p.t0 + t) * KT;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&B.full[s], (uint32_t)__popc(act) * (uint32_t)(box * 128 * (C::P16 ? NCH : 1)));
                    if (v && (k0 < p.lo || k0 + KT > p.hi)) mbar_arrive(&B.vissued[s]);
                }
                __syncwarp();
                if (page != -2) {
                    const int key = k0 + sub * box;
                    const int row = page * P.a.page_size + (key & (P.a.page_size - 1));
                    if (C::P16) tma_load_3d(ring + (size_t)s * C::kTile + sub * (NCH * 2048), m, &B.full[s], 0, row, p.g * NCH);
                    else tma_load_2d(ring + (size_t)s * C::kTile + ch * (KT * 128) + sub * (box * 128), m, &B.full[s], p.g * HD + ch * 64, row);
                }
                ++e;
                issued = e;
                return true;
            };
            int cur = page_of(0), prev = cur;
            for (int t = 0; t < p.nt && ok; ++t) {
                const int nxt = page_of(t + 1);                // in flight while this tile waits for its slot
                ok = load(&tmK, false, t, cur);
                if (NQ == 2) ok = ok && load(&tmV, true, t, cur);
                else if (t > 0) ok = ok && load(&tmV, true, t - 1, prev);
                prev = cur;
                cur = nxt;
            }
            if (NQ == 1 && ok) ok = load(&tmV, true, p.nt - 1, prev);
        }
        if (!ok) {                                            // copies in flight land before the block ends (bounded)
            const uint64_t deadline = global_timer_ns() + kWaitLimitNs;
            bool in = true;
            for (int i = max(0, issued - NS); i < issued && in; ++i)
                in = mbar_wait_until(&B.full[i % NS], (uint32_t)(i / NS) & 1u, deadline);
            if (!C::QTMEM && in && p.index >= 0) mbar_wait_until(&B.qfull, (uint32_t)p.index & 1u, global_timer_ns() + 1000000ull);
        }
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ MMAs
        // The whole warp runs the loop, so that what an MMA takes (descriptors, addresses) stays in uniform
        // registers; one elected thread issues.
        uint32_t vpar = 0;                                    // parity of each slot's next vready phase
        constexpr uint32_t id_qk = idesc<T>(kRows, C::P16 ? KT / 2 : KT, 0), id_pv = idesc<T>(kRows, HD, 1);
        const bool leader = elect_one();
        const uint32_t ring0 = smem_u32(ring), q0 = smem_u32(sQ);
        auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait(bar, parity, abort_flag, P.status); };
        while (ok && walk.next(P, &p)) {
            if (p.nt == 0) continue;
            const int e0 = uniform(e) + C::kQSlots, nt = uniform(p.nt), ns = nt * NQ, k_first = uniform(p.t0) * KT, lo = uniform(p.lo), hi = uniform(p.hi);
            const int g0 = uniform(gs);
            if (!__all_sync(0xffffffffu, wait(&B.qfull, (uint32_t)p.index & 1u))) { ok = false; break; }
            if (leader)
                for (int s = 0; s < C::kQSlots; ++s) mbar_arrive(&B.free_[(e + s) % NS]);
            auto issue_s = [&](int s) {
                const int t = s / NQ, q = s % NQ, en = e0 + k_entry<NQ>(t), sl = en % NS, buf = (g0 + s) & 1;
                if (q == 0 && !__all_sync(0xffffffffu, wait(&B.full[sl], (uint32_t)(en / NS) & 1u))) return false;
                tc_fence_after();
                if (leader) {
                    const uint32_t d = tmem + (uint32_t)(buf * KT);
                    constexpr int kChunkB = C::P16 ? 2048 : KT * 128;       // bytes between chunks of K
#pragma unroll
                    for (int h = 0; h < (C::P16 ? 2 : 1); ++h) {
                        const uint64_t bd = sdesc_k_sw128(ring0 + (uint32_t)sl * C::kTile + h * 1024, C::P16 ? NCH * 2048 : 1024);
                        const uint64_t ad = sdesc_k_sw128(q0 + (uint32_t)(q * NCH * C::kChunk));
#pragma unroll
                        for (int j = 0; j < HD / 16; ++j) {
                            const uint64_t bj = bd + (uint64_t)(((j >> 2) * kChunkB + (j & 3) * 32) >> 4);
                            if (C::QTMEM) mma_f16_ts(d + h * (KT / 2), tmem + (uint32_t)(C::kQCol + 8 * j), bj, id_qk, j > 0);
                            else mma_bf16(d + h * (KT / 2), ad + (uint64_t)(((j >> 2) * C::kChunk + (j & 3) * 32) >> 4), bj, id_qk, j > 0);
                        }
                    }
                    mma_commit(&B.sdone[buf]);
                    if (q == NQ - 1) mma_commit(&B.free_[sl]);
                    if (!C::QTMEM && s == ns - 1) mma_commit(&B.qfree);
                }
                return true;
            };
            if (!issue_s(0) || (ns > 1 && !issue_s(1))) { ok = false; break; }
            for (int s = 0; s < ns; ++s) {
                const int t = s / NQ, q = s % NQ, en = e0 + v_entry<NQ>(t, nt), sl = en % NS, buf = (g0 + s) & 1;
                if (q == 0) {
                    const int k0 = k_first + t * KT;
                    const bool part = k0 < lo || k0 + KT > hi;    // rows outside the unit's keys: zeroed first
                    uint64_t* bar = part ? &B.vready[sl] : &B.full[sl];
                    const uint32_t par = part ? (vpar >> sl) & 1u : (uint32_t)(en / NS) & 1u;
                    if (!__all_sync(0xffffffffu, wait(bar, par))) { ok = false; break; }
                    if (part) vpar ^= 1u << sl;
                }
                const uint32_t d = tmem + (uint32_t)(C::kOCol + q * HD), pa = tmem + (uint32_t)(buf * KT);
                const uint64_t bd = sdesc_mn_sw128(ring0 + (uint32_t)sl * C::kTile, C::P16 ? 2048 : KT * 128, C::P16 ? NCH * 2048 : 1024);
                // keys 16 j ..: with P16 rows 0 - 7 (then 8 - 15) of two pages
                auto v_at = [](int j) { return C::P16 ? 2 * (j % (KT / 32)) * NCH * 2048 + j / (KT / 32) * 1024 : j * 2048; };
                constexpr int J0 = NQ == 2 ? 4 : 0;           // MMAs on the half of P that is ready first
                if (NQ == 2) {
                    if (!__all_sync(0xffffffffu, wait(&B.phalf[buf], (uint32_t)((g0 + s) >> 1) & 1u))) { ok = false; break; }
                    tc_fence_after();
                    if (leader) {
#pragma unroll
                        for (int j = 0; j < J0; ++j)
                            mma_f16_ts(d, pa + (uint32_t)(8 * j), bd + (uint64_t)(v_at(j) >> 4), id_pv, t > 0 || j > 0);
                    }
                }
                if (!__all_sync(0xffffffffu, wait(&B.pready[buf], (uint32_t)((g0 + s) >> 1) & 1u))) { ok = false; break; }
                tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int j = J0; j < KT / 16; ++j)
                        mma_f16_ts(d, pa + (uint32_t)(j / (C::CH / 16) * C::CH + j % (C::CH / 16) * 8), bd + (uint64_t)(v_at(j) >> 4), id_pv, t > 0 || j > 0);
                    mma_commit(&B.odone[buf]);
                    if (q == NQ - 1) mma_commit(&B.free_[sl]);
                }
                if (s + 2 < ns && !issue_s(s + 2)) { ok = false; break; }
            }
            e = e0 + 2 * nt;
            gs = g0 + ns;
        }
        if (!ok && leader) {                                  // MMAs in flight end first (bounded)
            mma_commit(&B.spare);
            if (!mbar_wait_until(&B.spare, 0u, global_timer_ns() + kWaitLimitNs)) atomicOr(P.status, DSPARK_DEV_WAIT_TIMEOUT);
        }
        __syncwarp();
    } else if (warp == kFixWarp) {
        // ------------------------------------------------------------ V rows outside the unit's keys
        // (this warp skips entries, so a slot's load is first known to be issued: only then does the
        // parity of its full barrier name this load)
        uint32_t vpar = 0;
        while (ok && walk.next(P, &p)) {
            if (p.nt == 0) continue;
            const int e0 = e + C::kQSlots;
            for (int t = 0; t < p.nt; ++t) {
                const int k0 = (p.t0 + t) * KT, a = max(0, p.lo - k0), b = min(KT, p.hi - k0);   // rows [a, b) stay
                if (a == 0 && b == KT) continue;
                const int en = e0 + v_entry<NQ>(t, p.nt), sl = en % NS;
                const bool in = mbar_wait(&B.vissued[sl], (vpar >> sl) & 1u, abort_flag, P.status) &&
                                mbar_wait(&B.full[sl], (uint32_t)(en / NS) & 1u, abort_flag, P.status);
                vpar ^= 1u << sl;
                if (!__all_sync(0xffffffffu, in)) { ok = false; break; }
                uint8_t* tile = ring + (size_t)sl * C::kTile;
                const int dead = KT - (b - a);
                for (int i = lane; i < dead * 8; i += 32) {
                    const int row = (i >> 3) < a ? i >> 3 : (i >> 3) - a + b;
                    uint8_t* line = tile + (C::P16 ? row / 16 * (NCH * 2048) + row % 16 * 128 : row * 128) + (i & 7) * 16;
#pragma unroll
                    for (int c = 0; c < NCH; ++c) *reinterpret_cast<uint4*>(line + c * (C::P16 ? 2048 : KT * 128)) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_async_shared();                         // the MMAs read through the async proxy
                __syncwarp();
                if (lane == 0) mbar_arrive(&B.vready[sl]);
            }
            e = e0 + 2 * p.nt;
        }
    } else if (warp < kLoadWarp) {
        // ------------------------------------------------------------ softmax: SP threads per query row
        // SP = 2: threads r and r + 128 share row r, each takes half of the tile's keys and half of
        // the output's columns; they agree on the maximum through shared memory.
        constexpr int SP = C::SP, CH = C::CH, OH = HD / SP;
        const int q = SP == 2 ? 0 : tid >> 7, half = SP == 2 ? tid >> 7 : 0, r = tid & 127;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tO = tmem + (uint32_t)(C::kOCol + q * HD + half * OH) + lane_off;
        const float c = P.a.scale * 1.4426950408889634f;      // scores to log2
        float* mine = s_half + half * 128 + r;
        const float* other = s_half + (half ^ 1) * 128 + r;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, P.status));
        };
        auto agree = [&](bool good) { return SP == 1 ? good : !named_barrier_or(1, 256, !good); };   // a row's threads meet; false if one gave up
        const int grp = P.a.grp, tok_r = r / grp, head_r = r - tok_r * grp;
        // The loaded query rows of a piece (ring entries from e0) into tensor memory, two 16-bit values per column; the S
        // products of the piece before have all completed (their last was waited for).
        auto stage = [&](int e0) {
            const bool filled = r < P.tpt * grp;
            for (int s = 0; s < C::kQSlots; ++s) {
                const int en = e0 + s, sl = en % NS;
                if (!wait(&B.full[sl], (uint32_t)(en / NS) & 1u)) return false;
                const int c0 = s * C::kQPerSlot, c1 = min(NCH, c0 + C::kQPerSlot);
                for (int cc = c0; cc < c1; ++cc) {
                    const uint8_t* line = ring + (size_t)sl * C::kTile + (cc - c0) * C::kChunk + r * 128;
                    static_assert(!C::QTMEM || SP == 2, "each thread of a row stages half a line");
                    const int j0 = 4 * half;
                    uint32_t w[16];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint4 u = make_uint4(0u, 0u, 0u, 0u);
                        if (filled) u = *reinterpret_cast<const uint4*>(line + (((j0 + j) ^ (r & 7)) * 16));
                        w[4 * j] = u.x; w[4 * j + 1] = u.y; w[4 * j + 2] = u.z; w[4 * j + 3] = u.w;
                    }
                    tmem_st_x16(tmem + (uint32_t)(C::kQCol + cc * 32 + j0 * 4) + lane_off, w);
                }
            }
            tmem_st_wait();
            fence_async_shared();                             // reads done before the slots are loaded again
            tc_fence_before();
            mbar_arrive(&B.qfull);                            // the MMA warp then frees the slots
            return true;
        };
        bool more = walk.next(P, &p), staged = false;
        while (ok && more) {
            const int i = p.qt * P.tpu + q * P.tpt + tok_r;   // this row's token of the request
            const bool valid = tok_r < P.tpt && i < p.r.n;
            const int pos = p.r.L - p.r.n + i;
            const int row_hi = P.a.causal ? min(p.r.L, pos + 1) : p.r.L;
            const int row_lo = P.a.window > 0 ? max(0, pos - P.a.window + 1) : 0;
            // keys that every row of the tile sees (tokens of the whole query tile)
            const int i_first = p.qt * P.tpu + q * P.tpt, i_last = min(p.r.n, i_first + P.tpt) - 1;
            const int all_hi = P.a.causal ? min(p.r.L, p.r.L - p.r.n + i_first + 1) : p.r.L;
            const int all_lo = P.a.window > 0 ? max(0, p.r.L - p.r.n + i_last - P.a.window + 1) : 0;
            const bool live = __any_sync(0xffffffffu, valid);  // the warp has a row to compute (the MMAs read garbage for the others)
            float m = -INFINITY, l = 0.f;
            if (C::QTMEM && p.nt > 0 && !staged) ok = stage(e);
            bool good = ok;
            int last_step = -1;
            for (int t = 0; t < p.nt; ++t) {
                const int st = gs + t * NQ + q, buf = st & 1;
                const uint32_t tS = tmem + (uint32_t)(buf * KT + half * CH) + lane_off;
                good = good && wait(&B.sdone[buf], (uint32_t)(st >> 1) & 1u);
                tc_fence_after();
                const int k0 = (p.t0 + t) * KT;
                const bool edge = k0 < all_lo || k0 + KT > all_hi;   // some row does not see some key
                // At most 64 columns of scores at a time: 128 (SP = 1) are read once for the maximum and again
                // for the exponentials, as they would not stay in registers.
                constexpr int W = CH < 64 ? CH : 64;
                uint32_t u[W];
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                auto fetch = [&](int j) {                     // columns j .. j + W of this half
#pragma unroll
                    for (int i = 0; i < W; i += 32) tmem_ld_x32(tS + (uint32_t)(j + i), u + i);
                    tmem_ld_wait();
                    if (edge) {
                        // column i's key is k0 + first + place(i)
                        const int first = C::P16 ? half * 8 + 2 * j : half * CH + j, a = row_lo - k0 - first, b = row_hi - k0 - first;
#pragma unroll
                        for (int i = 0; i < W; ++i) {
                            const int place = C::P16 ? i / 8 * 16 + i % 8 : i;
                            if (place < a || place >= b) u[i] = 0xff800000u;
                        }
                    }
                };
#pragma unroll
                for (int j = CH - W; j >= 0 && live; j -= W) {
                    fetch(j);
#pragma unroll
                    for (int i = 0; i < W; i += 8)
#pragma unroll
                        for (int k = 0; k < 4; ++k) mx[k] = max3(mx[k], __uint_as_float(u[i + k]), __uint_as_float(u[i + 4 + k]));
                }
                float top = max2(max2(mx[0], mx[1]), max2(mx[2], mx[3]));
                if (SP == 2) mine[(t & 1) * 256] = top;       // two sets in turn: the other thread may still read the last
                if (!agree(good)) { ok = false; break; }
                if (SP == 2) top = max2(top, other[(t & 1) * 256]);
                top *= c;
                const bool need = m > -INFINITY && !(top <= m + kRescale);        // (a NaN becomes the maximum and stays it)
                if (__any_sync(0xffffffffu, need && live)) {
                    // O holds the tiles before at the old maximum: their PV must have landed
                    good = wait(&B.odone[last_step & 1], (uint32_t)(last_step >> 1) & 1u);
                    tc_fence_after();
                    const float f = need ? ex2(m - top) : 1.f;
                    if (need) { l *= f; m = top; }
#pragma unroll 1
                    for (int d = 0; d < OH; d += 16) {
                        uint32_t o[16];
                        tmem_ld_x16(tO + (uint32_t)d, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                        tmem_st_x16(tO + (uint32_t)d, o);
                    }
                    tmem_st_wait();
                }
                if (m == -INFINITY) m = top;                  // nothing summed yet
                const float neg = m == -INFINITY ? 0.f : -m;
                const uint64_t c2 = f2(c, c), neg2 = f2(neg, neg);
                uint64_t ls[2] = {0, 0};
                // poly: an eighth of the exponentials on the FMA pipe (scores of -infinity have no place there)
                auto exps = [&](int j0, auto poly) {
#pragma unroll
                    for (int j = 0; j < W; j += 16) {
                        uint32_t w[8];
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            const uint64_t x = fma2(f2(__uint_as_float(u[j + i]), __uint_as_float(u[j + i + 1])), c2, neg2);
                            float p0, p1, x0, x1;
                            f2_out(x, x0, x1);
                            if (poly.value && (i & 14) == 14) {
                                exp2_poly(f2(fmaxf(x0, -126.f), fmaxf(x1, -126.f)), p0, p1);
                            } else {
                                p0 = ex2(x0);
                                p1 = ex2(x1);
                            }
                            ls[(i >> 1) & 1] = add2(ls[(i >> 1) & 1], f2(p0, p1));
                            w[i >> 1] = pack2<T>(p0, p1);
                        }
                        tmem_st_x8(tS + (uint32_t)((j0 + j) / 2), w);       // (over scores already used)
                    }
                };
#pragma unroll
                for (int j = 0; j < CH && live; j += W) {
                    if (j > 0) fetch(j);
                    if (edge) exps(j, std::false_type{}); else exps(j, std::true_type{});
                    if (SP == 1 && j == 0) {
                        tmem_st_wait();
                        tc_fence_before();
                        mbar_arrive(&B.phalf[buf]);
                    }
                }
                if (SP == 1 && !live) mbar_arrive(&B.phalf[buf]);
                float l0, l1;
                f2_out(add2(ls[0], ls[1]), l0, l1);
                l += l0 + l1;
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&B.pready[buf]);
                last_step = st;
            }
            // ---- the piece's result
            if (!ok) break;                                   // (all of the tile's warps)
            // the next piece's queries first: its S products run beside this epilogue
            const Piece now = p;
            more = walk.next(P, &p);
            staged = C::QTMEM && more && p.nt > 0;
            if (staged) good = stage(e + (now.nt > 0 ? C::kQSlots + 2 * now.nt : 0)) && good;
            if (now.nt > 0) good = good && wait(&B.odone[last_step & 1], (uint32_t)(last_step >> 1) & 1u);
            tc_fence_after();
            if (SP == 2) mine[(now.nt & 1) * 256] = l;
            if (!agree(good)) { ok = false; break; }
            if (SP == 2) {
                l += other[(now.nt & 1) * 256];
                named_barrier_sync(1, 256);                   // both have read: the next piece may write
            }
            // l = 0: no key, or scores of -infinity alone (the polynomial's least value is 2^-126). A maximum that is NaN or
            // +infinity (a query with a NaN, a score that overflowed) has no softmax: the row becomes NaN.
            l = m == -INFINITY ? 0.f : m < INFINITY ? l : __int_as_float(0x7fffffff);
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const int64_t tok = now.r.t0 + i;
            const int h = now.g * grp + head_r;
            if (now.whole) {
                // A store of one row per lane would touch 32 lines. Four lanes exchange 16-byte blocks instead, so that
                // they write 64 bytes of one of their rows at a time.
                const int64_t at = valid ? tok * P.a.out_stride + (int64_t)h * HD + half * OH : -1;
                int64_t row_at[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) row_at[k] = __shfl_sync(0xffffffffu, at, (lane & ~3) + k);
                T* out = static_cast<T*>(P.a.out) + (lane & 3) * 8;
#pragma unroll
                for (int d = 0; d < OH; d += 32) {
                    uint32_t o[32], w[16];
                    if (now.nt > 0) {
                        tmem_ld_x32(tO + (uint32_t)d, o);
                        tmem_ld_wait();
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j) w[j] = l == 0.f ? 0u : pack2<T>(__uint_as_float(o[2 * j]) * inv, __uint_as_float(o[2 * j + 1]) * inv);
                    transpose_blocks(w, lane);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (row_at[k] >= 0) *reinterpret_cast<uint4*>(out + row_at[k] + d) = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
                }
                if (valid && half == 0 && P.a.lse) P.a.lse[tok * P.a.nH + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
            } else {
                // [slot][column / 4][row] float4: a warp's rows are neighbours
                const int64_t part = (int64_t)now.slot * NQ + q;
                if (valid && half == 0) P.part_ml[part * kRows + r] = make_float2(l > 0.f ? m : l == 0.f ? -INFINITY : l, l);     // (no number: the whole row is none)
                float4* po = P.part_o + (part * (HD / 4) + half * (OH / 4)) * kRows + r;
#pragma unroll
                for (int d = 0; d < OH; d += 32) {
                    uint32_t o[32];
                    tmem_ld_x32(tO + (uint32_t)d, o);
                    tmem_ld_wait();
                    if (valid) {
#pragma unroll
                        for (int j = 0; j < 32; j += 4)
                            po[(d + j) / 4 * kRows] =
                                make_float4(__uint_as_float(o[j]) * inv, __uint_as_float(o[j + 1]) * inv, __uint_as_float(o[j + 2]) * inv, __uint_as_float(o[j + 3]) * inv);
                    }
                }
            }
            tc_fence_before();                                // O read before the next piece's first PV (behind its P)
            if (now.nt > 0) {
                e += C::kQSlots + 2 * now.nt;
                gs += now.nt * NQ;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ merge
// out = sum_s w_s O_s / sum_s w_s, w_s = l_s exp2(m_s - M), over a unit's pieces in order. A thread has four columns
// of a row, neighbouring threads neighbouring rows (as the pieces lie): grid (units, row groups, column groups).
constexpr int kMergeCols = 16;                                // float4 columns per block
template <typename T, int HD, int NQ>
__global__ void __launch_bounds__(32 * kMergeCols) attend_paged_merge_kernel(Params P) {
    pdl_trigger();
    pdl_wait();
    const MergeUnit u = P.merges[blockIdx.x];
    if (u.c1 < 0) return;
    const int q = blockIdx.y / (kRows / 32), r = (blockIdx.y % (kRows / 32)) * 32 + (threadIdx.x & 31);
    const int col = blockIdx.z * kMergeCols + (threadIdx.x >> 5);
    const Req req = load_req(P.a, u.b);
    const int tr = r / P.a.grp, i = u.qt * P.tpu + q * P.tpt + tr;
    if (tr >= P.tpt || i >= req.n) return;
    const int h = u.g * P.a.grp + r - tr * P.a.grp, n = u.c1 - u.c0 + 1;
    auto part = [&](int s) { return (int64_t)(s == 0 ? 2 * u.c0 + u.odd : 2 * (u.c0 + s)) * NQ + q; };
    float M = -INFINITY, den = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int B = 8;                                      // pieces in flight
    for (int s0 = 0; s0 < n; s0 += B) {
        float2 ml[B];
        float4 o[B];
#pragma unroll
        for (int k = 0; k < B; ++k) {
            const int64_t p = part(min(s0 + k, n - 1));
            ml[k] = P.part_ml[p * kRows + r];
            o[k] = P.part_o[(p * (HD / 4) + col) * kRows + r];
        }
        float top = M;
#pragma unroll
        for (int k = 0; k < B; ++k) top = fmaxf(top, ml[k].x);
        const float f = M == -INFINITY ? 0.f : ex2(M - top);
        M = top;
        den *= f; acc.x *= f; acc.y *= f; acc.z *= f; acc.w *= f;
#pragma unroll
        for (int k = 0; k < B; ++k) {
            const float w = s0 + k >= n || ml[k].x == -INFINITY ? 0.f : ml[k].y * ex2(ml[k].x - M);
            den += w;
            acc.x = fmaf(w, o[k].x, acc.x); acc.y = fmaf(w, o[k].y, acc.y); acc.z = fmaf(w, o[k].z, acc.z); acc.w = fmaf(w, o[k].w, acc.w);
        }
    }
    const float inv = den == 0.f ? 0.f : 1.f / den;
    T* out = static_cast<T*>(P.a.out) + (int64_t)(req.t0 + i) * P.a.out_stride + (int64_t)h * HD + col * 4;
    *reinterpret_cast<uint2*>(out) = make_uint2(pack2<T>(acc.x * inv, acc.y * inv), pack2<T>(acc.z * inv, acc.w * inv));
    if (P.a.lse && col == 0) P.a.lse[(int64_t)(req.t0 + i) * P.a.nH + h] = den == 0.f ? -INFINITY : (M + log2f(den)) * 0.69314718055994531f;
}

// ------------------------------------------------------------------ host
PFN_cuTensorMapEncodeTiled_v12000 g_enc = nullptr;
std::once_flag g_enc_once;

template <int RANK>
bool make_map(CUtensorMap* tm, const void* ptr, int dtype, const cuuint64_t (&dims)[RANK], const cuuint64_t (&strides)[RANK - 1], const cuuint32_t (&box)[RANK]) {
    std::call_once(g_enc_once, [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            g_enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    });
    if (!g_enc) return false;
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    static_assert(RANK <= 4, "element strides");
    return g_enc(tm, dtype == DSPARK_DTYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, RANK,
                 const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                 CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Layout { size_t status, merges, ml, o, total; };
Layout layout(int hd) {
    const int rows = hd <= 128 ? 2 * kRows : kRows;
    Layout l{};
    size_t at = 0;
    auto take = [&](size_t n) { const size_t p = at; at = align_up(at + n, 256); return p; };
    l.status = take(4);
    l.merges = take(kGrid * sizeof(MergeUnit));
    l.ml = take((size_t)2 * kGrid * rows * 2 * sizeof(float));
    l.o = take((size_t)2 * kGrid * rows * hd * sizeof(float));
    l.total = at;
    return l;
}

template <typename T, typename C>
cudaError_t launch(Params P, cudaStream_t s) {
    const PagedAttn& a = P.a;
    P.tpt = kRows / a.grp;
    P.tpu = C::NQ * P.tpt;
    CUtensorMap tq, tk, tv;
    const cuuint64_t hb = (cuuint64_t)a.hd * 2;
    const cuuint64_t qd[4] = {(cuuint64_t)a.hd, (cuuint64_t)a.grp, (cuuint64_t)a.nKv, (cuuint64_t)a.T};
    const cuuint64_t qs[3] = {hb, hb * a.grp, (cuuint64_t)a.q_stride * 2};
    const cuuint32_t qb[4] = {64, (cuuint32_t)a.grp, 1, (cuuint32_t)P.tpt};
    // (a page is page_size rows of all kv heads: the fewer dimensions, the faster small boxes go)
    const cuuint64_t rows = (cuuint64_t)a.num_pages * a.page_size;
    bool ok = make_map(&tq, a.q, a.dtype, qd, qs, qb);
    if (C::P16) {
        const cuuint64_t kd[3] = {64, rows, (cuuint64_t)a.nKv * C::NCH}, ks[2] = {hb * a.nKv, 128};
        const cuuint32_t kb[3] = {64, 16, C::NCH};
        ok = ok && make_map(&tk, a.k, a.dtype, kd, ks, kb) && make_map(&tv, a.v, a.dtype, kd, ks, kb);
    } else {
        const cuuint64_t kd[2] = {(cuuint64_t)a.nKv * a.hd, rows}, ks[1] = {hb * a.nKv};
        const cuuint32_t kb[2] = {64, (cuuint32_t)std::min(a.page_size, C::KT)};
        ok = ok && make_map(&tk, a.k, a.dtype, kd, ks, kb) && make_map(&tv, a.v, a.dtype, kd, ks, kb);
    }
    if (!ok) return cudaErrorInvalidValue;
    auto kern = attend_paged_tc_kernel<T, C>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3(kGrid), dim3(C::kThreads), C::kSmem, s, tq, tk, tv, P);
    if (e == cudaSuccess)
        e = launch_pdl(attend_paged_merge_kernel<T, C::HD, C::NQ>, dim3(kGrid, C::NQ * kRows / 32, C::HD / 4 / kMergeCols), dim3(32 * kMergeCols), 0, s, P);
    return e;
}

template <typename T>
cudaError_t dispatch(const Params& P, cudaStream_t s) {
    // two query tiles per unit once a request's rows fill more than one: K and V tiles then feed twice the
    // MMAs and the softmax of one tile overlaps the MMAs of the other
    const bool two = (int64_t)P.a.max_new * P.a.grp > kRows;
    const bool p16 = P.a.page_size == 16;
    switch (P.a.hd) {
        case 64: return two ? launch<T, Cfg<64, 2, 128, false>>(P, s) : p16 ? launch<T, Cfg<64, 1, 128, false, true>>(P, s) : launch<T, Cfg<64, 1, 128, false>>(P, s);
        case 128: return two ? launch<T, Cfg<128, 2, 128, false>>(P, s) : p16 ? launch<T, Cfg<128, 1, 128, false, true>>(P, s) : launch<T, Cfg<128, 1, 128, false>>(P, s);
        case 192: return p16 ? launch<T, Cfg<192, 1, 64, true, true>>(P, s) : launch<T, Cfg<192, 1, 64, true>>(P, s);
        default: return p16 ? launch<T, Cfg<256, 1, 64, true, true>>(P, s) : launch<T, Cfg<256, 1, 64, true>>(P, s);
    }
}

}  // namespace

bool attend_paged_tc_supported(const dspark_paged_cache& c, int n_heads) {
    return c.dtype != DSPARK_DTYPE_F32 && c.head_dim % 64 == 0 && c.page_size >= 8 && (c.page_size & (c.page_size - 1)) == 0 &&
           n_heads / c.n_kv <= kRows && ((int64_t)c.num_pages + 1) * c.page_size < ((int64_t)1 << 31);
}
int attend_paged_max_batch() { return kMaxBatch; }
size_t attend_paged_tc_workspace(int hd) { return layout(hd).total; }

cudaError_t launch_attend_paged_tc(const PagedAttn& a, void* ws, cudaStream_t s) {
    const Layout l = layout(a.hd);
    char* w = static_cast<char*>(ws);
    Params P{};
    P.a = a;
    P.merges = reinterpret_cast<MergeUnit*>(w + l.merges);
    P.part_ml = reinterpret_cast<float2*>(w + l.ml);
    P.part_o = reinterpret_cast<float4*>(w + l.o);
    P.status = a.status ? a.status : reinterpret_cast<int32_t*>(w + l.status);
    while ((1 << P.page_shift) < a.page_size) ++P.page_shift;
    return a.dtype == DSPARK_DTYPE_F16 ? dispatch<__half>(P, s) : dispatch<__nv_bfloat16>(P, s);
}

}  // namespace tc
}  // namespace dspark
