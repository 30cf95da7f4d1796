// kda_prompt.cuh -- what the calls that take a prompt and its answer through the
// softmax attention layers share: arguments and launches.
#pragma once

#include "kda_tree.cuh"

namespace kda {

// ------------------------------------------------------------ prompt attention
struct PromptArgs {
    const void *q, *k, *v;            // tokens of q_stride, k_stride, v_stride elements
    long long q_stride, k_stride, v_stride;
    const int32_t *cu_q, *cu_k;       // [N + 1]; null: one sequence of all rows
    int32_t N, T, Tk;
    int32_t Hq, Hkv, G;               // G = Hq / Hkv
    float scale_log2;                 // scale * log2(e)
    void* o;                          // [T, Hq, d]
    int32_t* status;                  // tensor-core kernel: words of the workspace
    uint32_t* counter;
    bool starve;                      // test of the waits that give up
};

// The rows of sequence n: from q0, lq of them, and k0, lk; whatever the offsets
// hold, rows that exist.
struct PromptSeq {
    int q0, lq, k0, lk;
};
__device__ __forceinline__ void prompt_rows(const int32_t* cu, int n, int rows, int& first, int& count)
{
    first = 0;
    int end = rows;
    if (cu) {
        first = max(__ldg(cu + n), 0);
        end = min(__ldg(cu + n + 1), rows);
    }
    count = end > first ? end - first : 0;     // (their difference may not fit)
}
__device__ __forceinline__ PromptSeq prompt_seq(const PromptArgs& a, int n)
{
    PromptSeq s;
    prompt_rows(a.cu_q, n, a.T, s.q0, s.lq);
    prompt_rows(a.cu_k, n, a.Tk, s.k0, s.lk);
    return s;
}

// All three take every length and layout.  On the CUDA cores in fp32 (KDA_FORCE_SIMT in the
// environment): every type, head size and scale.
cudaError_t launch_prompt_attention(const PromptArgs& args, int32_t d, kda_dtype_t dtype, cudaStream_t stream);

// Products of fp16 pairs: the same, to 22 bits for fp32 inputs or outputs.
cudaError_t launch_prompt_attention_split(const PromptArgs& args, int32_t d, kda_dtype_t dtype, cudaStream_t stream);

// The tcgen05 kernel: bf16 in and out, d = 64 or 128, a positive scale (it finds a
// row's maximum before it applies the scale), at most 128 heads to a key head.
bool prompt_tc_supported(const PromptArgs& args, int32_t d, kda_dtype_t dtype);
cudaError_t launch_prompt_attention_tc(PromptArgs args, int32_t d, int sms, cudaStream_t stream);

// --------------------------------------------------- rotated rows into a cache
struct RotaryArgs {
    const uint8_t *q, *k, *v;         // q may be null
    uint8_t *q_out, *k_out;           // null: not wanted
    long long q_row, k_row, v_row, q_out_row, k_out_row;   // bytes from token to token
    uint8_t *k_cache, *v_cache;       // [num_pages][page_size][Hkv][d]
    float *k_scales, *v_scales;       // [num_pages][page_size / block][Hkv]
    long long page_bytes;
    const int32_t *cu_seqlens, *page_table, *lengths;
    int32_t* new_lengths;             // [N] or null
    const float* inv_freq;            // [rot / 2]
    int32_t T, N, Hq, Hkv, rot, num_pages, page_size, max_pages;
    int32_t block;                    // rows per scale; 0: the cache is in k's type
    bool interleaved;
    // of the launch: blocks of 8-bit units, rows of their windows, parts of a window's heads, warps
    // of a team; parts of a row's heads and heads of a part
    int32_t unit_blocks, window, splits, team, chunks, chunk_heads;
};
constexpr int kMaxScaleBlock = 128;
cudaError_t launch_cache_append_rotary(RotaryArgs args, int32_t d, bool bf16, int sms, cudaStream_t stream);

// ------------------------------------------------ attention to a cache of 8 bits
struct E4m3Args {
    // N, lengths, page_table, page_size, max_pages, groups, row_tiles of the call, Hkv
    // >> heads_log heads, and Ts = 1: the split of the work (kda_tree.cuh) over an item's
    // rows and one more, so that an item without any has a tile
    TreeArgs split;
    int32_t heads_log;                // log2 of the cache heads of an item
    const void* q;                    // [N, Ts, Hq, d]
    const uint8_t *k_cache, *v_cache;
    const float *k_scales, *v_scales; // [num_pages][page_size / block][Hkv]
    int32_t Ts, Hq, Hkv, G, R;        // R = Ts G rows per (sequence, cache head)
    int32_t num_pages, block, blocks; // blocks: of a page
    uint32_t block_magic;             // ceil(2^32 / block): a row's block by a multiplication
    int32_t tile_pages, tile_rows;    // a tile's keys as whole pages and rows
    long long page_stride;            // bytes
    float scale_log2;
    void* o;
    float* part;                      // 2 slots per CTA, per head: [16][d] o, [16] m, [16] m of the values, [16] l
    int32_t* status;                  // the workspace's timeout word
    bool starve;                      // test of the waits that give up
};
constexpr int kMaxE4m3Page = 65536;   // rows of a page (block_magic is exact up to there)
size_t e4m3_workspace_bytes(int32_t Ts, int32_t Hq, int32_t Hkv, int32_t d, int sms);
cudaError_t launch_cache_attention_e4m3(E4m3Args args, int32_t d, kda_dtype_t dtype, int sms, cudaStream_t stream);

}  // namespace kda
