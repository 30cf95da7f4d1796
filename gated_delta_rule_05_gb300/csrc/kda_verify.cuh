// kda_verify.cuh -- the launches of the calls that verify a tree of drafted
// tokens (the attention's are in kda_tree.cuh).
#pragma once

#include "kda_internal.cuh"

namespace kda {

// kda_decode_multi over a tree of drafted tokens (parent [N, Ts], not null).
cudaError_t launch_decode_tree(const void* q, const void* k, const void* v,
                               const float* log_alpha, const float* beta, const float* S_in,
                               const int32_t* parent, float* states, int32_t N, int32_t Ts,
                               int32_t H, int32_t d, kda_dtype_t dtype, void* o,
                               cudaStream_t stream);

// Per logits row: log probabilities of J given tokens, entropy, the K largest.
constexpr int kMaxAlternatives = 32;
cudaError_t launch_token_logprobs(const void* logits, long long row_stride, const int32_t* tokens,
                                  int32_t T, int32_t V, int32_t J, int32_t K, bool bf16,
                                  float* logprobs, float* entropy, int32_t* top_ids,
                                  float* top_logprobs, cudaStream_t stream);

// Rows of k and v into cache pages (kda_cache_commit, kda_cache_append).
struct CacheArgs {
    const uint8_t *k, *v;             // [layers, rows, row_bytes]
    uint8_t *k_cache, *v_cache;       // [layers][num_pages][page_size][row_bytes]
    long long rows;                   // N * Ts, or the packed token count
    long long page_bytes, layer_bytes;
    int32_t layers, N, Ts, row_bytes, num_pages, page_size, max_pages;
    const int32_t *path, *count;      // commit: [N, Ts] or null, [N]
    const int32_t* cu_seqlens;        // append: [N + 1]
    const int32_t *page_table, *lengths;
    int32_t* new_lengths;             // [N] or null
};
cudaError_t launch_cache_rows(const CacheArgs& args, cudaStream_t stream);

}  // namespace kda
