// Internal launchers of the serving operators (page tables, shared-prefix
// attention, logit rules): called by their C entries and by the session's
// passes in api.cu.
#pragma once

#include "dflash.h"
#include "launch.h"

namespace dfl {

// kv_tables.cu
void kv_tables(const Launch& L, const dflash_kv_tables_args& a);

// attention_shared.cu: false when a kernel could not be prepared (nothing queued).
bool shared_prefix_attention(const Launch& L, const dflash_shared_prefix_args& a);

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

// The entries' argument checks: DFLASH_OK, or E_INVAL with the reason in *why.
dflash_status check_shared_prefix(const dflash_shared_prefix_args& a, const char** why);
dflash_status check_logits(const dflash_logits_args& a, const char** why);

}  // namespace dfl
