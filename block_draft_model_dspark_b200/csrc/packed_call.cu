// dspark_packed_call: the paged calls with their arguments as 64-bit words, for bindings
// whose foreign calls cost by the argument (ctypes: 2.4 us for 20 arguments, 0.6 for one block of them,
// beside 5 us for the launch itself).
#include <string.h>

#include "paged.h"

using namespace dspark;

namespace {

struct Words {
    const int64_t* w;
    bool fit = true;                       // every 32-bit argument's word held one
    int64_t i() { return *w++; }
    int32_t i32() {
        const int64_t v = *w++;
        fit = fit && v == (int32_t)v;
        return (int32_t)v;
    }
    float f() { double d; memcpy(&d, w++, sizeof d); return (float)d; }
    template <typename T> T* p() { return reinterpret_cast<T*>(static_cast<uintptr_t>(*w++)); }
};

int unfit() { DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "an integer argument does not fit 32 bits"); }

}  // namespace

// Braced initialisers evaluate in order, so each call's words are read first to last.
extern "C" int dspark_packed_call(int32_t call, const int64_t* words) {
    if (!words) DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "words must be non-NULL");
    Words a{words};
    switch (call) {
        case DSPARK_CALL_PAGE_SLOTS: {
            struct { const dspark_paged_cache* c; const int32_t *ctx, *n; int32_t B; const int32_t *pages, *free_pages; int32_t n_free; const int32_t* count;
                     int32_t max_tokens; int32_t *pages_out, *count_out, *cu, *kv; int64_t* slots; int32_t* pos; void* stream; } v{
                a.p<const dspark_paged_cache>(), a.p<const int32_t>(), a.p<const int32_t>(), a.i32(), a.p<const int32_t>(), a.p<const int32_t>(), a.i32(),
                a.p<const int32_t>(), a.i32(), a.p<int32_t>(), a.p<int32_t>(), a.p<int32_t>(), a.p<int32_t>(), a.p<int64_t>(), a.p<int32_t>(), a.p<void>()};
            if (!a.fit) return unfit();
            return dspark_page_slots(v.c, v.ctx, v.n, v.B, v.pages, v.free_pages, v.n_free, v.count, v.max_tokens, v.pages_out, v.count_out, v.cu, v.kv,
                                     v.slots, v.pos, v.stream);
        }
        case DSPARK_CALL_NORM_ROPE_PAGED: {
            struct { const dspark_paged_cache* c; int32_t layer, dtype; const void* q; int64_t qs; const void* k; int64_t ks; const void* v; int64_t vs;
                     int32_t nH; const void *qn, *kn; const double* freq; float eps; int32_t v_norm; const int32_t* pos; const int64_t* slots; int32_t T;
                     void *out, *stream; } v{
                a.p<const dspark_paged_cache>(), a.i32(), a.i32(), a.p<const void>(), a.i(), a.p<const void>(), a.i(), a.p<const void>(), a.i(), a.i32(),
                a.p<const void>(), a.p<const void>(), a.p<const double>(), a.f(), a.i32(), a.p<const int32_t>(), a.p<const int64_t>(), a.i32(), a.p<void>(),
                a.p<void>()};
            if (!a.fit) return unfit();
            return dspark_norm_rope_paged(v.c, v.layer, v.dtype, v.q, v.qs, v.k, v.ks, v.v, v.vs, v.nH, v.qn, v.kn, v.freq, v.eps, v.v_norm, v.pos, v.slots,
                                          v.T, v.out, v.stream);
        }
        case DSPARK_CALL_ATTEND_PAGED: {
            struct { const dspark_paged_cache* c; int32_t layer; const void* q; int64_t qs; int32_t nH; const int32_t *cu, *kv; int32_t B, T, max_new;
                     float scale; int32_t causal, window; void* out; int64_t os; float* lse; void* ws; size_t ws_bytes; void* stream; } v{
                a.p<const dspark_paged_cache>(), a.i32(), a.p<const void>(), a.i(), a.i32(), a.p<const int32_t>(), a.p<const int32_t>(), a.i32(), a.i32(),
                a.i32(), a.f(), a.i32(), a.i32(), a.p<void>(), a.i(), a.p<float>(), a.p<void>(), (size_t)a.i(), a.p<void>()};
            if (!a.fit) return unfit();
            return dspark_attend_paged(v.c, v.layer, v.q, v.qs, v.nH, v.cu, v.kv, v.B, v.T, v.max_new, v.scale, v.causal, v.window, v.out, v.os, v.lse, v.ws,
                                       v.ws_bytes, v.stream);
        }
        case DSPARK_CALL_SAMPLE: {
            struct { const void* x; int32_t dtype; int64_t stride; int32_t rows, V; const float *u, *T; const int32_t* k; const float *p, *mp;
                     int32_t* tokens; float* probs; void* ws; size_t ws_bytes; void* stream; } v{
                a.p<const void>(), a.i32(), a.i(), a.i32(), a.i32(), a.p<const float>(), a.p<const float>(), a.p<const int32_t>(), a.p<const float>(),
                a.p<const float>(), a.p<int32_t>(), a.p<float>(), a.p<void>(), (size_t)a.i(), a.p<void>()};
            if (!a.fit) return unfit();
            return dspark_sample(v.x, v.dtype, v.stride, v.rows, v.V, v.u, v.T, v.k, v.p, v.mp, v.tokens, v.probs, v.ws, v.ws_bytes, v.stream);
        }
        default: DSPARK_FAIL(DSPARK_ERR_INVALID_ARGUMENT, "unknown call");
    }
}
