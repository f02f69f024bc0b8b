// Library-internal helpers shared between the translation units of libatlaskv.
#pragma once

#include "atlaskv.h"

// Record `msg` as this thread's atlaskv_last_error() text and return `st`.
atlaskv_status akv_report(atlaskv_status st, const char *msg);

// Raise a kernel's dynamic shared-memory limit to `bytes`, once per (kernel, device).
atlaskv_status akv_smem_limit(const void *kernel, size_t bytes);

// The sequence part over a paged cache (cache.cu): normalised output oseq
// [B H_kv][G N][D] and log-sum-exp lse_seq [B H_kv][G N] (natural log), float32.
atlaskv_status akv_cache_matches(const atlaskv_cache *cache, int n_kv_heads, int head_dim);
// akv_cache_check: the refusals that akv_cache_part would give with enough workspace.
atlaskv_status akv_cache_check(const atlaskv_cache *cache, const atlaskv_seqs *seqs, int dtype, int H, const void *q,
                               float scale);
atlaskv_status akv_cache_part(atlaskv_cache *cache, const atlaskv_seqs *seqs, int dtype, int H, const void *q, float scale,
                              float *oseq, float *lse_seq, void *workspace, size_t workspace_bytes, void *stream);
