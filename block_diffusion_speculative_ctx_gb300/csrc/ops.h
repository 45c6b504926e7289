// Internal launchers of the serving operators (page tables, shared-prefix
// attention, logit rules): called by their C entries and by the session's
// passes in api.cu.
#pragma once

#include "dflash.h"
#include "launch.h"

namespace dfl {

// kv_tables.cu
void kv_tables(const Launch& L, const dflash_kv_tables_args& a);

// attention_shared.cu: false when a kernel could not be prepared (nothing queued).  With `tree`, rows see the own keys that
// their masks name instead of the causal ones.
struct TreeMasks {
    const uint32_t* masks;
    long long ld_mask;
    int words;
};
bool shared_prefix_attention(const Launch& L, const dflash_shared_prefix_args& a, const TreeMasks* tree = nullptr);

// logit_rules.cu
void process_logits(const Launch& L, const dflash_logits_args& a);

// ---- the session's own bookkeeping around them (session_ops.cu)
// A row that the rules leave without a token (bit of the device error word).
enum : uint32_t { ERR_NO_TOKEN = 8u };
// out[s] = a[s] + (b ? b[s] : 0) + add; with block set, start[s] = s * *block for s <= batch (a host value).
void own_lengths(const Launch& L, int batch, const int* a, const int* b, int add, int* out, int* start, const int* block);
// dst[i] = x row start[s0 + i + 1] - 1, i < n (fp32 rows of d).
void gather_last_rows(const Launch& L, const float* x, int d, const int* start, int s0, int n, float* dst);
// After a target pass: history[s][n - a .. n - 1] = the accepted drafts, history[s][n] = the anchor
// (accepted NULL: the anchor alone).  n is the new committed length.
void history_append(const Launch& L, int batch, int B, int ld, const int* n, const int* anchor, const int* accepted,
                    const int* proposal, int* history);
// index[i] >= n becomes -1 (no mask).
void drop_indices(const Launch& L, int* index, int rows, int n);
// Rows whose best logit is -inf have no token: the error word says so, and token 0 gets all of the row's
// mass, so that what follows stays defined.
void check_rows(const Launch& L, float* logits, long long ld, int rows, const int* best, uint32_t* err);

// The caches [layers][n_pages][n_kv_heads][64][head_dim] of a call: NULL, or which of the texts says what is wrong.
template <typename A>
const char* bad_caches(const A& a, const char* dtype, const char* layers, const char* sizes, const char* lie) {
    if (a.dtype != DFLASH_DTYPE_F32 && a.dtype != DFLASH_DTYPE_BF16) return dtype;
    if (a.layers < 1 || a.layers > 1024) return layers;
    const long long es = a.dtype == DFLASH_DTYPE_BF16 ? 2 : 4;
    // (token slots 64 * page + token are 32-bit)
    if (a.n_pages < 1 || a.n_pages > (1 << 24) || a.n_kv_heads < 1 || a.n_kv_heads > 1024 || a.head_dim < 1 ||
        a.head_dim > 4096 || a.head_dim * es % 16)
        return sizes;
    const long long layer = (long long)a.n_pages * a.n_kv_heads * 64 * a.head_dim;
    if (!a.k_cache || !a.v_cache || (((uintptr_t)a.k_cache | (uintptr_t)a.v_cache) & 15u) || a.ld_layer * es % 16 ||
        (a.layers > 1 && a.ld_layer < layer))
        return lie;
    return nullptr;
}

// Whether two such caches (of good sizes) share memory: layer i of one and layer i + j of the other, which may lie between
// each other.
template <typename A>
bool caches_overlap(const A& a) {
    const long long es = a.dtype == DFLASH_DTYPE_BF16 ? 2 : 4;
    const long long layer = (long long)a.n_pages * a.n_kv_heads * 64 * a.head_dim * es, between = a.ld_layer * es;
    const long long apart = (long long)((uintptr_t)a.v_cache - (uintptr_t)a.k_cache);
    for (long long j = 1 - a.layers; j < a.layers; ++j) {
        const long long d = apart + j * between;
        if (d > -layer && d < layer) return true;
    }
    return false;
}

// The entries' ends: a refused argument, and what f(L) queues on the caller's stream (failed_text: what to say where no CUDA
// error does).
inline dflash_status refuse(const char* why) {
    set_global_error(why);
    return DFLASH_E_INVAL;
}
template <typename F>
dflash_status queue(void* cuda_stream, const char* failed_text, F&& f) {
    bool failed = false;
    Launch L{(cudaStream_t)cuda_stream, nullptr};
    L.pdl = true;  // (each kernel waits for what runs before it ahead of its first read)
    L.failed = &failed;
    f(L);
    const cudaError_t e = cudaGetLastError();
    if (failed || e != cudaSuccess) {
        set_global_error(e != cudaSuccess ? cudaGetErrorString(e) : failed_text);
        return DFLASH_E_CUDA;
    }
    return DFLASH_OK;
}

// The entries' argument checks: DFLASH_OK, or E_INVAL with the reason in *why.
dflash_status check_shared_prefix(const dflash_shared_prefix_args& a, const char** why);
dflash_status check_logits(const dflash_logits_args& a, const char** why);

}  // namespace dfl
