// kda_verify_api.cu -- the C ABI of the calls that verify a tree of drafted
// tokens (include/kda.h): argument validation and dispatch.
#include <limits.h>
#include <stdint.h>

#include "kda_tree.cuh"
#include "kda_verify.cuh"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool supported_d(int32_t d) { return d == 16 || d == 32 || d == 64 || d == 128; }

bool overlaps(const void* a, size_t na, const void* b, size_t nb)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

bool valid_dtype(kda_dtype_t t) { return t == KDA_BF16 || t == KDA_FP32 || t == KDA_BF16_F32OUT; }

size_t in_bytes(kda_dtype_t t) { return t == KDA_FP32 ? 4 : 2; }
size_t out_bytes(kda_dtype_t t) { return t == KDA_BF16 ? 2 : 4; }

// The sizes that the attention and its workspace take: a row tile is a block index.
bool attention_sizes(int32_t N, int32_t Ts, int32_t Hq, int32_t Hkv, int32_t d)
{
    return N >= 1 && Ts >= 1 && Hkv >= 1 && Hq >= Hkv && Hq % Hkv == 0 && (int64_t)Ts * Hq <= (1 << 20) &&
           (int64_t)Hkv * d <= INT32_MAX;
}

// Bytes from the first to the last element of a layer's pages, and whether the
// strides are ones that the kernels take.
bool cache_shape(int32_t num_pages, int32_t page_size, int32_t Hkv, int32_t d, int64_t page_stride,
                 size_t elem, size_t* bytes)
{
    const int64_t page_elems = (int64_t)page_size * Hkv * d;
    if (num_pages > 1 && (page_stride < page_elems || (page_stride * (int64_t)elem) % 16 != 0)) return false;
    *bytes = ((size_t)(num_pages - 1) * (size_t)(num_pages > 1 ? page_stride : 0) + (size_t)page_elems) * elem;
    return true;
}

}  // namespace

extern "C" {

size_t kda_tree_attention_workspace_bytes(int32_t N, int32_t Ts, int32_t Hq, int32_t Hkv, int32_t d,
                                          kda_dtype_t dtype)
{
    if (!valid_dtype(dtype) || !supported_d(d) || Ts > kda::kTreeMaxNodes ||
        !attention_sizes(N, Ts, Hq, Hkv, d))
        return 0;
    return kda::tree_workspace_bytes(Ts, Hq, Hkv, d, dtype, kda::device_sm_count());
}

kda_status_t kda_tree_attention(const void* q, const void* k, const void* v, const int32_t* parent,
                                const void* k_cache, const void* v_cache, const int32_t* page_table,
                                const int32_t* lengths, int32_t N, int32_t Ts, int32_t Hq,
                                int32_t Hkv, int32_t d, int32_t num_pages, int32_t page_size,
                                int32_t max_pages, int64_t page_stride, kda_dtype_t dtype,
                                float scale, void* o, void* workspace, size_t workspace_bytes,
                                cudaStream_t stream)
{
    if (!valid_dtype(dtype) || !supported_d(d)) return KDA_ERR_UNSUPPORTED;
    if (Ts > kda::kTreeMaxNodes) return KDA_ERR_UNSUPPORTED;
    if (!attention_sizes(N, Ts, Hq, Hkv, d)) return KDA_ERR_INVALID_ARG;
    if (num_pages < 0 || page_size < 1 || max_pages < 0) return KDA_ERR_INVALID_ARG;
    // Positions (of the drafted rows too) are 32-bit.
    if ((int64_t)max_pages * page_size > INT32_MAX - 1024) return KDA_ERR_INVALID_ARG;
    if (!q || !k || !v || !lengths || !o) return KDA_ERR_INVALID_ARG;
    const bool cached = num_pages > 0 && max_pages > 0;
    if (cached && (!k_cache || !v_cache || !page_table)) return KDA_ERR_INVALID_ARG;
    const void* ptrs16[] = {q, k, v, k_cache, v_cache, o};
    for (const void* p : ptrs16)
        if (p && !aligned(p, 16)) return KDA_ERR_INVALID_ARG;
    const void* ptrs4[] = {parent, page_table, lengths};
    for (const void* p : ptrs4)
        if (p && !aligned(p, 4)) return KDA_ERR_INVALID_ARG;
    size_t cache_bytes = 0;
    if (cached && !cache_shape(num_pages, page_size, Hkv, d, page_stride, in_bytes(dtype), &cache_bytes))
        return KDA_ERR_INVALID_ARG;
    const size_t o_bytes = (size_t)N * Ts * Hq * d * out_bytes(dtype);
    const size_t q_bytes = (size_t)N * Ts * Hq * d * in_bytes(dtype);
    const size_t kv_bytes = (size_t)N * Ts * Hkv * d * in_bytes(dtype);
    if (overlaps(o, o_bytes, q, q_bytes) || overlaps(o, o_bytes, k, kv_bytes) ||
        overlaps(o, o_bytes, v, kv_bytes))
        return KDA_ERR_INVALID_ARG;
    if (cached && (overlaps(o, o_bytes, k_cache, cache_bytes) || overlaps(o, o_bytes, v_cache, cache_bytes)))
        return KDA_ERR_INVALID_ARG;
    const int sms = kda::device_sm_count();
    if (!workspace || workspace_bytes < kda::tree_workspace_bytes(Ts, Hq, Hkv, d, dtype, sms) ||
        !aligned(workspace, 256)) return KDA_ERR_WORKSPACE;

    kda::TreeArgs a = {};
    a.q = q;
    a.k = k;
    a.v = v;
    a.parent = parent;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.page_table = page_table;
    a.lengths = lengths;
    a.N = N;
    a.Ts = Ts;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = Hq / Hkv;
    a.R = Ts * a.G;
    a.num_pages = cached ? num_pages : 0;
    a.page_size = page_size;
    a.max_pages = cached ? max_pages : 0;
    a.page_stride = page_stride;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.o = o;
    a.status = static_cast<int32_t*>(workspace);
    a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kda::kWsHeaderBytes);
    const cudaError_t err = kda::launch_tree_attention(a, d, dtype, sms, stream);
    return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status_t kda_decode_tree(const void* q, const void* k, const void* v, const float* log_alpha,
                             const float* beta, const float* S_in, const int32_t* parent, int32_t N,
                             int32_t Ts, int32_t H, int32_t d_k, int32_t d_v, kda_dtype_t dtype,
                             void* o, float* states, cudaStream_t stream)
{
    if (!valid_dtype(dtype)) return KDA_ERR_UNSUPPORTED;
    if (d_k != d_v || !supported_d(d_k) || (parent && Ts > kda::kTreeMaxNodes)) return KDA_ERR_UNSUPPORTED;
    if (N < 1 || Ts < 1 || H < 1) return KDA_ERR_INVALID_ARG;
    if (!q || !k || !v || !log_alpha || !beta || !S_in || !o || !states) return KDA_ERR_INVALID_ARG;
    const void* ptrs16[] = {q, k, v, log_alpha, o, S_in, states};
    for (const void* p : ptrs16)
        if (!aligned(p, 16)) return KDA_ERR_INVALID_ARG;
    if (!aligned(beta, 4) || !aligned(parent, 4)) return KDA_ERR_INVALID_ARG;
    const size_t state_bytes = (size_t)N * H * d_k * d_v * sizeof(float);
    const size_t states_bytes = state_bytes * Ts;
    const size_t tokens = (size_t)N * Ts * H;
    const size_t o_bytes = tokens * d_v * out_bytes(dtype), qkv_bytes = tokens * d_k * in_bytes(dtype);
    if (overlaps(states, states_bytes, o, o_bytes)) return KDA_ERR_INVALID_ARG;
    // Read by the CTAs of other value columns, and ahead, while one writes its results.
    const struct { const void* p; size_t n; } reads[] = {
        {S_in, state_bytes}, {q, qkv_bytes}, {k, qkv_bytes}, {v, qkv_bytes}, {log_alpha, tokens * d_k * 4},
        {beta, tokens * 4}, {parent, (size_t)N * Ts * 4}};
    for (const auto& r : reads)
        if (r.p && (overlaps(o, o_bytes, r.p, r.n) || overlaps(states, states_bytes, r.p, r.n)))
            return KDA_ERR_INVALID_ARG;
    if (!parent)
        return kda_decode_multi(q, k, v, log_alpha, beta, S_in, N, Ts, H, d_k, d_v, dtype, o, states,
                                stream);
    const cudaError_t err = kda::launch_decode_tree(q, k, v, log_alpha, beta, S_in, parent, states, N,
                                                    Ts, H, d_k, dtype, o, stream);
    return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status_t kda_token_logprobs(const void* logits, int64_t row_stride, const int32_t* tokens,
                                int32_t T, int32_t V, int32_t J, int32_t K, kda_dtype_t dtype,
                                float* logprobs, float* entropy, int32_t* top_ids,
                                float* top_logprobs, cudaStream_t stream)
{
    if (dtype != KDA_BF16_F32OUT && dtype != KDA_FP32) return KDA_ERR_UNSUPPORTED;
    if (K > kda::kMaxAlternatives) return KDA_ERR_UNSUPPORTED;
    if (T < 1 || V < 1 || J < 0 || K < 0 || K > V || row_stride < V) return KDA_ERR_INVALID_ARG;
    if (!logits || (J > 0 && (!tokens || !logprobs)) || (K > 0 && (!top_ids || !top_logprobs)))
        return KDA_ERR_INVALID_ARG;
    if (J == 0 && K == 0 && !entropy) return KDA_ERR_INVALID_ARG;
    if (!aligned(logits, 16)) return KDA_ERR_INVALID_ARG;
    const void* ptrs4[] = {tokens, logprobs, entropy, top_ids, top_logprobs};
    for (const void* p : ptrs4)
        if (p && !aligned(p, 4)) return KDA_ERR_INVALID_ARG;
    const cudaError_t err =
        kda::launch_token_logprobs(logits, row_stride, tokens, T, V, J, K, dtype != KDA_FP32, logprobs,
                                   entropy, top_ids, top_logprobs, stream);
    return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"

namespace {

kda_status_t cache_rows(const void* k, const void* v, const int32_t* path, const int32_t* count,
                        const int32_t* cu_seqlens, int64_t rows, const int32_t* page_table,
                        const int32_t* lengths, int32_t layers, int32_t N, int32_t Ts, int32_t Hkv,
                        int32_t d, int32_t num_pages, int32_t page_size, int32_t max_pages,
                        int64_t page_stride, int64_t layer_stride, kda_dtype_t dtype, void* k_cache,
                        void* v_cache, int32_t* new_lengths, cudaStream_t stream)
{
    if (!valid_dtype(dtype) || !supported_d(d)) return KDA_ERR_UNSUPPORTED;
    if (layers < 1 || N < 1 || Hkv < 1 || rows < 0) return KDA_ERR_INVALID_ARG;
    if (num_pages < 1 || page_size < 1 || max_pages < 1) return KDA_ERR_INVALID_ARG;
    if ((int64_t)max_pages * page_size > INT32_MAX || rows > INT32_MAX ||
        (int64_t)Hkv * d * 4 > INT32_MAX || layers > 65535)
        return KDA_ERR_INVALID_ARG;
    if ((rows > 0 && (!k || !v)) || !k_cache || !v_cache || !page_table || !lengths)
        return KDA_ERR_INVALID_ARG;
    const void* ptrs16[] = {k, v, k_cache, v_cache};
    for (const void* p : ptrs16)
        if (p && !aligned(p, 16)) return KDA_ERR_INVALID_ARG;
    const void* ptrs4[] = {path, count, cu_seqlens, page_table, lengths, new_lengths};
    for (const void* p : ptrs4)
        if (p && !aligned(p, 4)) return KDA_ERR_INVALID_ARG;
    const size_t elem = in_bytes(dtype);
    size_t layer_bytes = 0;
    if (!cache_shape(num_pages, page_size, Hkv, d, page_stride, elem, &layer_bytes))
        return KDA_ERR_INVALID_ARG;
    if (layers > 1 && ((layer_stride * (int64_t)elem) % 16 != 0 || layer_stride < (int64_t)page_size * Hkv * d))
        return KDA_ERR_INVALID_ARG;
    const size_t cache_bytes = (size_t)(layers - 1) * (size_t)(layers > 1 ? layer_stride : 0) * elem + layer_bytes;
    const size_t in = (size_t)layers * (size_t)rows * Hkv * d * elem;
    const void* ins[] = {k, v};
    const void* outs[] = {k_cache, v_cache};
    for (const void* x : ins)
        for (const void* y : outs)
            if (rows > 0 && overlaps(x, in, y, cache_bytes)) return KDA_ERR_INVALID_ARG;
    // Written by some CTAs while others still read theirs.
    if (new_lengths) {
        const struct { const void* p; size_t n; } reads[] = {
            {lengths, (size_t)N}, {count, (size_t)N}, {path, (size_t)rows}, {cu_seqlens, (size_t)N + 1},
            {page_table, (size_t)N * max_pages}};
        for (const auto& r : reads)
            if (r.p && overlaps(new_lengths, 4 * (size_t)N, r.p, 4 * r.n)) return KDA_ERR_INVALID_ARG;
    }

    kda::CacheArgs a = {};
    a.k = static_cast<const uint8_t*>(k);
    a.v = static_cast<const uint8_t*>(v);
    a.k_cache = static_cast<uint8_t*>(k_cache);
    a.v_cache = static_cast<uint8_t*>(v_cache);
    a.rows = rows;
    a.row_bytes = Hkv * d * (int32_t)elem;
    a.page_bytes = page_stride * (int64_t)elem;
    a.layer_bytes = layer_stride * (int64_t)elem;
    a.layers = layers;
    a.N = N;
    a.Ts = Ts;
    a.num_pages = num_pages;
    a.page_size = page_size;
    a.max_pages = max_pages;
    a.path = path;
    a.count = count;
    a.cu_seqlens = cu_seqlens;
    a.page_table = page_table;
    a.lengths = lengths;
    a.new_lengths = new_lengths;
    const cudaError_t err = kda::launch_cache_rows(a, stream);
    return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace

extern "C" {

kda_status_t kda_cache_commit(const void* k, const void* v, const int32_t* path, const int32_t* count,
                              const int32_t* page_table, const int32_t* lengths, int32_t layers,
                              int32_t N, int32_t Ts, int32_t Hkv, int32_t d, int32_t num_pages,
                              int32_t page_size, int32_t max_pages, int64_t page_stride,
                              int64_t layer_stride, kda_dtype_t dtype, void* k_cache, void* v_cache,
                              int32_t* new_lengths, cudaStream_t stream)
{
    if (Ts < 1) return KDA_ERR_INVALID_ARG;
    return cache_rows(k, v, path, count, nullptr, (int64_t)N * Ts, page_table, lengths, layers, N, Ts,
                      Hkv, d, num_pages, page_size, max_pages, page_stride, layer_stride, dtype,
                      k_cache, v_cache, new_lengths, stream);
}

kda_status_t kda_cache_append(const void* k, const void* v, const int32_t* cu_seqlens,
                              int64_t total_tokens, const int32_t* page_table, const int32_t* lengths,
                              int32_t layers, int32_t N, int32_t Hkv, int32_t d, int32_t num_pages,
                              int32_t page_size, int32_t max_pages, int64_t page_stride,
                              int64_t layer_stride, kda_dtype_t dtype, void* k_cache, void* v_cache,
                              int32_t* new_lengths, cudaStream_t stream)
{
    if (!cu_seqlens) return KDA_ERR_INVALID_ARG;
    return cache_rows(k, v, nullptr, nullptr, cu_seqlens, total_tokens, page_table, lengths, layers, N,
                      1, Hkv, d, num_pages, page_size, max_pages, page_stride, layer_stride, dtype,
                      k_cache, v_cache, new_lengths, stream);
}

}  // extern "C"
