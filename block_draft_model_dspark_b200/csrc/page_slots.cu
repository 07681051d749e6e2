// dspark_page_slots: from the requests' lengths to the pages they need, their
// block tables, and the slot and position of every new token.
//
// With ctx_b cached rows, n_b new ones and h_b pages held, request b wants
// w_b = max(ceil((ctx_b + n_b) / page), h_b) pages and takes w_b - h_b of them
// from the top of the free stack, in request order: the page of global rank r
// is free_pages[free_count - 1 - r]. Both exclusive sums (new tokens, pages
// taken) fix every output entry by itself, so the kernel is two scans and a
// fill. It is bound by latency (a few dependent loads and barriers): one launch
// of one cluster, each CTA scanning all requests (they sit in L2) into its own
// shared memory, then a share of the fill per CTA. The cluster barrier between
// the last read of a request's numbers and the first write lets the outputs
// be the inputs' own arrays (lengths and page counts advanced in place). One request takes
// 6 us in a graph, 512 requests with 65,000 tokens 11.7 us.
#include "paged.h"

namespace dspark {
namespace {

constexpr int kMaxBatch = 4096;
constexpr int kThreads = 512;
constexpr int kPer = kMaxBatch / kThreads;   // requests per thread
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kScanBytes = 2 * kWarps * (int)sizeof(int64_t);
constexpr int kTok = 4;                      // neighbouring tokens per thread

struct SlotsParams {
    const int32_t* ctx_len; const int32_t* n_new; const int32_t* n_pages; const int32_t* free_pages;
    const int32_t* free_count;
    int32_t* table; int32_t* n_pages_out; int32_t* free_count_out; int32_t* cu_new; int32_t* kv_len;
    int64_t* slots; int32_t* positions; int32_t* status;
    int B, n_free, max_tokens, max_pages, page_size, num_pages, cluster;
};

// Exclusive sum over the block of one value per thread; *total gets the sum.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* buf, int64_t* total) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) buf[wid] = x;
    __syncthreads();
    int64_t base = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < wid) base += buf[w];
        all += buf[w];
    }
    *total = all;
    return base + x - v;
}

// The last i in [0, n) with a[i] <= x (a ascending, a[0] <= x).
__device__ __forceinline__ int last_le(const int32_t* a, int n, int32_t x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kThreads) page_slots_kernel(SlotsParams P) {
    extern __shared__ int32_t sm[];
    int32_t* s_cu = sm;                       // [B + 1] first new token
    int32_t* s_first = sm + P.B + 1;          // [B + 1] rank of the first page taken
    int32_t* s_ctx = s_first + P.B + 1;       // [B]
    int32_t* s_held = s_ctx + P.B;            // [B]
    __shared__ int64_t buf[2][kWarps];        // kScanBytes
    static_assert(sizeof(buf) == kScanBytes, "the kernel's static shared memory");
    const int tid = threadIdx.x, rank = P.cluster > 1 ? (int)blockIdx.x : 0;
    pdl_trigger();
    pdl_wait();
    const int per = (P.B + kThreads - 1) / kThreads;   // <= kPer: requests [tid * per, ...)
    int32_t n[kPer], take[kPer], ctx[kPer], held[kPer];
    bool bad = false;
    int64_t sn = 0, st = 0;
    const int count = P.free_count[0];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int b = tid * per + i;
        n[i] = take[i] = ctx[i] = held[i] = 0;
        if (i >= per || b >= P.B) continue;
        ctx[i] = P.ctx_len[b];
        n[i] = P.n_new[b];
        held[i] = P.n_pages[b];
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int64_t kv = (int64_t)ctx[i] + n[i];
        if (ctx[i] < 0 || n[i] < 0 || held[i] < 0 || kv > (int64_t)P.max_pages * P.page_size || kv > 0x7fffffff ||
            held[i] > P.max_pages) {
            bad = true;
            n[i] = 0;
            continue;
        }
        const int want = (int)((kv + P.page_size - 1) / P.page_size);
        take[i] = max(want - held[i], 0);
        sn += n[i];
        st += take[i];
    }
    int64_t tot_n, tot_t;
    const int64_t pre_n = block_scan(sn, buf[0], &tot_n);
    const int64_t pre_t = block_scan(st, buf[1], &tot_t);
    bad = __syncthreads_or(bad || count < 0 || count > P.n_free || tot_t > count || tot_n > P.max_tokens);
    // refused: no page is taken, no token has a slot
    int32_t cn = (int32_t)pre_n, ct = (int32_t)pre_t;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int b = tid * per + i;
        if (i >= per || b >= P.B) continue;
        s_cu[b] = bad ? 0 : cn;
        s_first[b] = bad ? 0 : ct;
        s_ctx[b] = ctx[i];
        s_held[b] = held[i];
        cn += n[i];
        ct += take[i];
    }
    if (tid == 0) {
        s_cu[P.B] = bad ? 0 : (int32_t)tot_n;
        s_first[P.B] = bad ? 0 : (int32_t)tot_t;
    }
    if (P.cluster > 1) cluster_sync(); else __syncthreads();   // every CTA has read its inputs
    const int ntok = s_cu[P.B], ntake = s_first[P.B];
    if (rank == 0) {
        for (int b = tid; b <= P.B; b += kThreads) {
            P.cu_new[b] = s_cu[b];
            if (b == P.B) break;
            P.n_pages_out[b] = s_held[b] + s_first[b + 1] - s_first[b];
            P.kv_len[b] = s_ctx[b] + s_cu[b + 1] - s_cu[b];
        }
        if (tid == 0) {
            P.free_count_out[0] = count - ntake;
            if (bad) set_status(P.status, DSPARK_DEV_CAPACITY);
        }
    }
    const int stride = kThreads * P.cluster;
    for (int r = rank * kThreads + tid; r < ntake; r += stride) {
        const int b = last_le(s_first, P.B, r);               // the request that takes page r (ties: the last, which takes)
        const int page = P.free_pages[count - 1 - r];
        if (page < 0 || page >= P.num_pages) set_status(P.status, DSPARK_DEV_BAD_PAGE);       // (its tokens, if any, get no slot below)
        P.table[(int64_t)b * P.max_pages + s_held[b] + r - s_first[b]] = page;
    }
    // four neighbouring tokens a thread: one search, their pages fetched together
    for (int t0 = (rank * kThreads + tid) * kTok; t0 < P.max_tokens; t0 += stride * kTok) {
        int b = t0 < ntok ? last_le(s_cu, P.B, t0) : P.B, p[kTok], page[kTok];
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
            const int t = t0 + i;
            p[i] = 0;
            page[i] = -1;
            if (t >= ntok) continue;
            while (t >= s_cu[b + 1]) ++b;                     // (ends: ntok is the last entry)
            p[i] = s_ctx[b] + t - s_cu[b];
            const int j = p[i] / P.page_size;
            const int32_t* from = j < s_held[b] ? P.table + (int64_t)b * P.max_pages + j : P.free_pages + (count - 1 - (s_first[b] + j - s_held[b]));
            page[i] = *from;
            if (page[i] < 0 || page[i] >= P.num_pages) {
                set_status(P.status, DSPARK_DEV_BAD_PAGE);
                page[i] = -1;
            }
        }
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
            if (t0 + i >= P.max_tokens) break;
            P.slots[t0 + i] = page[i] < 0 ? -1 : (int64_t)page[i] * P.page_size + p[i] % P.page_size;
            P.positions[t0 + i] = p[i];
        }
    }
}

}  // namespace

int check_paged_cache(const dspark_paged_cache* c) {
    if (!c) DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "paged cache is NULL");
    if (c->layers < 1 || c->num_pages < 1 || c->page_size < 1 || c->n_kv < 1 || c->batch < 1 || c->max_pages < 1)
        DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "layers, num_pages, page_size, n_kv, batch and max_pages must be >= 1");
    if (!valid_dtype(c->dtype)) DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "paged cache dtype must be fp32, bf16 or fp16");
    if (c->head_dim < 16 || c->head_dim > 256 || c->head_dim % 16 != 0)
        DSPARK_FAIL(DSPARK_ERR_UNSUPPORTED, "head_dim must be a multiple of 16 in [16, 256]");
    if ((int64_t)c->num_pages * c->page_size > ((int64_t)1 << 40) || c->page_size > (1 << 20) || c->n_kv > (1 << 16))
        DSPARK_FAIL(DSPARK_ERR_UNSUPPORTED, "page_size above 2^20, n_kv above 2^16 or num_pages * page_size above 2^40");
    if (!c->block_table) DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "block_table must be non-NULL");
    return DSPARK_OK;
}

}  // namespace dspark

using namespace dspark;

extern "C" int dspark_page_slots(const dspark_paged_cache* c, const int32_t* ctx_len, const int32_t* n_new, int32_t B,
                                 const int32_t* n_pages, const int32_t* free_pages, int32_t n_free,
                                 const int32_t* free_count, int32_t max_tokens, int32_t* n_pages_out,
                                 int32_t* free_count_out, int32_t* cu_new, int32_t* kv_len, int64_t* slots,
                                 int32_t* positions, void* stream) {
    const int rc = check_paged_cache(c);
    if (rc != DSPARK_OK) return rc;
    if (B < 1 || B > c->batch) DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "B must be in [1, cache.batch]");
    if (B > kMaxBatch) DSPARK_FAIL(DSPARK_ERR_UNSUPPORTED, "more than 4096 requests in one call");
    if (max_tokens > (1 << 30)) DSPARK_FAIL(DSPARK_ERR_UNSUPPORTED, "max_tokens above 2^30");
    if (max_tokens < 0 || n_free < 0) DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "max_tokens and n_free must be >= 0");
    if (!ctx_len || !n_new || !n_pages || !free_count || !n_pages_out || !free_count_out || !cu_new || !kv_len ||
        (n_free > 0 && !free_pages) || (max_tokens > 0 && (!slots || !positions)))
        DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "every array of the call must be non-NULL");
    SlotsParams P{};
    P.ctx_len = ctx_len; P.n_new = n_new; P.n_pages = n_pages; P.free_pages = free_pages; P.free_count = free_count;
    P.table = c->block_table; P.n_pages_out = n_pages_out; P.free_count_out = free_count_out; P.cu_new = cu_new;
    P.kv_len = kv_len; P.slots = slots; P.positions = positions; P.status = c->status;
    P.B = B; P.n_free = n_free; P.max_tokens = max_tokens; P.max_pages = c->max_pages; P.page_size = c->page_size;
    P.num_pages = c->num_pages;
    // a CTA per 4096 tokens (two rounds of its threads): 512 requests with 65,000 tokens take 102 us with one CTA
    P.cluster = 1;
    while (P.cluster < kMaxCluster && (int64_t)P.cluster * 2 * kThreads * kTok < max_tokens) P.cluster *= 2;
    const size_t smem = (4 * (size_t)B + 2) * sizeof(int32_t);
    cudaError_t e = cudaSuccess;                      // (the attributes cost host time: only where the launch needs them)
    if (smem > 48 * 1024 - kScanBytes)                // (48 KB without asking, the scans' buffers among them)
        e = cudaFuncSetAttribute(page_slots_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)((4 * kMaxBatch + 2) * sizeof(int32_t)));
    if (e == cudaSuccess && P.cluster > 8) e = cudaFuncSetAttribute(page_slots_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess)
        e = launch_pdl_cluster(page_slots_kernel, dim3(P.cluster), dim3(kThreads), P.cluster, smem, static_cast<cudaStream_t>(stream), P);
    if (e != cudaSuccess) DSPARK_FAIL(DSPARK_ERR_CUDA, std::string("page slots launch: ") + cudaGetErrorString(e));
    return DSPARK_OK;
}
