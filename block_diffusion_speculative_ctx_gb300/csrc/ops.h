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

// The entries' argument checks: DFLASH_OK, or E_INVAL with the reason in *why.
dflash_status check_shared_prefix(const dflash_shared_prefix_args& a, const char** why);
dflash_status check_logits(const dflash_logits_args& a, const char** why);

}  // namespace dfl
