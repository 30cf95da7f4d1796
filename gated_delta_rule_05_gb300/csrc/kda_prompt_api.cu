// kda_prompt_api.cu -- the C ABI of the calls that take a prompt and its answer
// through the softmax layers (include/kda.h): argument validation and dispatch.
#include <limits.h>
#include <stdint.h>

#include "kda_args.cuh"
#include "kda_prompt.cuh"

using namespace kda::args;

namespace {

// T rows of `width` bytes, `step` bytes apart.
struct RowSpan {
    const void* p;
    int64_t step, width, rows;
};

RowSpan row_span(const void* p, int64_t stride, int64_t elems, int64_t rows, size_t elem)
{
    return {p, (rows > 1 ? stride : elems) * (int64_t)elem, elems * (int64_t)elem, rows};
}

bool row_stride_ok(int64_t stride, int64_t elems, int64_t rows, size_t elem)
{
    return rows <= 1 || (stride >= elems && stride <= (INT64_MAX >> 34) && (stride * (int64_t)elem) % 16 == 0);
}

size_t span_bytes(const RowSpan& s) { return s.rows < 1 ? 0 : (size_t)((s.rows - 1) * s.step + s.width); }

// Whether rows of the two meet; views of one buffer's tokens lie between each other's
// rows.
bool rows_meet(const RowSpan& a, const RowSpan& b)
{
    if (!a.p || !b.p || a.rows < 1 || b.rows < 1) return false;
    if (!overlaps(a.p, span_bytes(a), b.p, span_bytes(b))) return false;
    if (a.step != b.step || a.rows < 2 || b.rows < 2) return true;
    const int64_t x = static_cast<int64_t>(reinterpret_cast<uintptr_t>(a.p) % (uintptr_t)a.step);
    const int64_t y = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.p) % (uintptr_t)a.step);
    const int64_t apart = (y - x + a.step) % a.step;
    return apart < a.width || apart + b.width > a.step;
}

bool meets(const RowSpan& a, const void* p, size_t bytes)
{
    return a.p && p && a.rows > 0 && bytes > 0 && overlaps(a.p, span_bytes(a), p, bytes);
}

bool head_sizes(int32_t Hq, int32_t Hkv, int32_t d)
{
    return Hkv >= 1 && Hq >= Hkv && Hq % Hkv == 0 && Hq <= (1 << 20) && (int64_t)Hq * d * 4 <= INT32_MAX;
}

bool prompt_sizes(int32_t num_seqs, int32_t Hq, int32_t Hkv, int32_t d)
{
    return num_seqs >= 1 && head_sizes(Hq, Hkv, d) && Hkv <= 65535;
}

bool newest_sizes(int32_t N, int32_t Ts, int32_t Hq, int32_t Hkv, int32_t d)
{
    return N >= 1 && Ts >= 1 && head_sizes(Hq, Hkv, d) && (int64_t)Ts * Hq <= (1 << 20);
}

}  // namespace

extern "C" {

size_t kda_prompt_attention_workspace_bytes(int32_t num_seqs, int32_t Hq, int32_t Hkv, int32_t d, kda_dtype_t dtype)
{
    return valid_dtype(dtype) && supported_d(d) && prompt_sizes(num_seqs, Hq, Hkv, d) ? kda::kWsHeaderBytes : 0;
}

kda_status_t kda_prompt_attention(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                                  int64_t v_stride, const int32_t* cu_seqlens, const int32_t* cu_seqlens_k,
                                  int32_t num_seqs, int64_t total_tokens, int64_t total_keys, int32_t Hq, int32_t Hkv,
                                  int32_t d, kda_dtype_t dtype, float scale, void* o, void* workspace,
                                  size_t workspace_bytes, cudaStream_t stream)
{
    if (!valid_dtype(dtype) || !supported_d(d)) return KDA_ERR_UNSUPPORTED;
    if (!prompt_sizes(num_seqs, Hq, Hkv, d)) return KDA_ERR_INVALID_ARG;
    if (total_tokens < 0 || total_keys < 0 || total_tokens > INT32_MAX - 65536 || total_keys > INT32_MAX - 65536)
        return KDA_ERR_INVALID_ARG;
    if (num_seqs > 1 && !cu_seqlens) return KDA_ERR_INVALID_ARG;
    if (cu_seqlens_k ? !cu_seqlens : total_keys != total_tokens) return KDA_ERR_INVALID_ARG;
    const size_t elem = in_bytes(dtype);
    if ((total_tokens > 0 && (!q || !o)) || (total_keys > 0 && (!k || !v))) return KDA_ERR_INVALID_ARG;
    const void* ptrs16[] = {q, k, v, o};
    for (const void* p : ptrs16)
        if (p && !aligned(p, 16)) return KDA_ERR_INVALID_ARG;
    const void* ptrs4[] = {cu_seqlens, cu_seqlens_k};
    for (const void* p : ptrs4)
        if (p && !aligned(p, 4)) return KDA_ERR_INVALID_ARG;
    const int64_t qw = (int64_t)Hq * d, kw = (int64_t)Hkv * d;
    if (!row_stride_ok(q_stride, qw, total_tokens, elem) || !row_stride_ok(k_stride, kw, total_keys, elem) ||
        !row_stride_ok(v_stride, kw, total_keys, elem))
        return KDA_ERR_INVALID_ARG;
    if (total_tokens == 0) return KDA_OK;
    // a row tile of a key head is a block index
    if (((total_tokens * (Hq / Hkv)) / 64 + num_seqs) * Hkv > INT32_MAX) return KDA_ERR_INVALID_ARG;
    const size_t o_bytes = (size_t)total_tokens * qw * out_bytes(dtype);
    const size_t cu_bytes = 4 * ((size_t)num_seqs + 1);
    if (meets(row_span(q, q_stride, qw, total_tokens, elem), o, o_bytes) ||
        meets(row_span(k, k_stride, kw, total_keys, elem), o, o_bytes) ||
        meets(row_span(v, v_stride, kw, total_keys, elem), o, o_bytes) ||
        (cu_seqlens && overlaps(cu_seqlens, cu_bytes, o, o_bytes)) ||
        (cu_seqlens_k && overlaps(cu_seqlens_k, cu_bytes, o, o_bytes)))
        return KDA_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < kda::kWsHeaderBytes || !aligned(workspace, 256)) return KDA_ERR_WORKSPACE;
    if (overlaps(workspace, kda::kWsHeaderBytes, o, o_bytes) ||
        (cu_seqlens && overlaps(cu_seqlens, cu_bytes, workspace, kda::kWsHeaderBytes)) ||
        (cu_seqlens_k && overlaps(cu_seqlens_k, cu_bytes, workspace, kda::kWsHeaderBytes)) ||
        meets(row_span(q, q_stride, qw, total_tokens, elem), workspace, kda::kWsHeaderBytes) ||
        meets(row_span(k, k_stride, kw, total_keys, elem), workspace, kda::kWsHeaderBytes) ||
        meets(row_span(v, v_stride, kw, total_keys, elem), workspace, kda::kWsHeaderBytes))
        return KDA_ERR_INVALID_ARG;

    kda::PromptArgs a = {};
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = total_tokens > 1 ? q_stride : qw;
    a.k_stride = total_keys > 1 ? k_stride : kw;
    a.v_stride = total_keys > 1 ? v_stride : kw;
    a.cu_q = cu_seqlens;
    a.cu_k = cu_seqlens_k ? cu_seqlens_k : cu_seqlens;
    a.N = num_seqs;
    a.T = (int32_t)total_tokens;
    a.Tk = (int32_t)total_keys;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = Hq / Hkv;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.o = o;
    a.status = static_cast<int32_t*>(workspace) + kda::kWsTimeoutWord;
    a.counter = static_cast<uint32_t*>(workspace) + kda::kWsCounterWord;
    const int sms = kda::device_sm_count();
    const cudaError_t err = getenv("KDA_FORCE_SIMT") != nullptr ? kda::launch_prompt_attention(a, d, dtype, stream)
                            : kda::prompt_tc_supported(a, d, dtype)
                                ? kda::launch_prompt_attention_tc(a, d, sms > 0 ? sms : 1, stream)
                                : kda::launch_prompt_attention_split(a, d, dtype, stream);
    return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status_t kda_cache_append_rotary(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                                     int64_t v_stride, const int32_t* cu_seqlens, int64_t total_tokens,
                                     const float* inv_freq, int32_t rot_dim, int32_t interleaved,
                                     const int32_t* page_table, const int32_t* lengths, int32_t N, int32_t Hq,
                                     int32_t Hkv, int32_t d, int32_t num_pages, int32_t page_size, int32_t max_pages,
                                     int64_t page_stride, int32_t block, kda_dtype_t dtype, void* q_out,
                                     int64_t q_out_stride, void* k_out, int64_t k_out_stride, void* k_cache,
                                     void* v_cache, float* k_scales, float* v_scales, int32_t* new_lengths,
                                     cudaStream_t stream)
{
    if (!valid_dtype(dtype) || !supported_d(d) || block > kda::kMaxScaleBlock) return KDA_ERR_UNSUPPORTED;
    if (N < 1 || Hkv < 1 || Hq < 0 || (Hq > 0 && Hq % Hkv != 0)) return KDA_ERR_INVALID_ARG;
    if ((int64_t)Hq * d * 4 > INT32_MAX || (int64_t)Hkv * d * 4 > INT32_MAX) return KDA_ERR_INVALID_ARG;
    if (total_tokens < 0 || total_tokens > INT32_MAX - 65536) return KDA_ERR_INVALID_ARG;
    if (rot_dim < 16 || rot_dim > d || rot_dim % 16 != 0 || !inv_freq) return KDA_ERR_INVALID_ARG;
    if (num_pages < 1 || page_size < 1 || max_pages < 1 || (int64_t)max_pages * page_size > INT32_MAX)
        return KDA_ERR_INVALID_ARG;
    if (block < 0 || (block > 0 && page_size % block != 0)) return KDA_ERR_INVALID_ARG;
    if (!cu_seqlens || !lengths || !page_table || !k_cache || !v_cache || (block > 0 && (!k_scales || !v_scales)))
        return KDA_ERR_INVALID_ARG;
    if (total_tokens > 0 && (!k || !v || (Hq > 0 && (!q || !q_out)))) return KDA_ERR_INVALID_ARG;
    if (Hq == 0 && (q || q_out)) return KDA_ERR_INVALID_ARG;
    const void* ptrs16[] = {q, k, v, q_out, k_out, k_cache, v_cache};
    for (const void* p : ptrs16)
        if (p && !aligned(p, 16)) return KDA_ERR_INVALID_ARG;
    const void* ptrs4[] = {cu_seqlens, lengths, page_table, inv_freq, k_scales, v_scales, new_lengths};
    for (const void* p : ptrs4)
        if (p && !aligned(p, 4)) return KDA_ERR_INVALID_ARG;
    const size_t elem = in_bytes(dtype), held = block > 0 ? 1 : elem;
    const int64_t T = total_tokens, qw = (int64_t)Hq * d, kw = (int64_t)Hkv * d;
    if (!row_stride_ok(k_stride, kw, T, elem) || !row_stride_ok(v_stride, kw, T, elem) ||
        (Hq > 0 && (!row_stride_ok(q_stride, qw, T, elem) || !row_stride_ok(q_out_stride, qw, T, elem))) ||
        (k_out && !row_stride_ok(k_out_stride, kw, T, elem)))
        return KDA_ERR_INVALID_ARG;
    size_t cache_bytes = 0;
    if (!cache_shape(num_pages, page_size, Hkv, d, page_stride, held, &cache_bytes)) return KDA_ERR_INVALID_ARG;
    const RowSpan qi = row_span(Hq ? q : nullptr, q_stride, qw, T, elem), ki = row_span(k, k_stride, kw, T, elem);
    const RowSpan vi = row_span(v, v_stride, kw, T, elem), qo = row_span(q_out, q_out_stride, qw, T, elem);
    const RowSpan ko = row_span(k_out, k_out_stride, kw, T, elem);
    const auto same = [](const RowSpan& a, const RowSpan& b) { return a.p == b.p && a.step == b.step; };
    if ((!same(qo, qi) && rows_meet(qo, qi)) || rows_meet(qo, ki) || rows_meet(qo, vi) || rows_meet(qo, ko) ||
        (!same(ko, ki) && rows_meet(ko, ki)) || rows_meet(ko, qi) || rows_meet(ko, vi))
        return KDA_ERR_INVALID_ARG;
    const size_t scale_bytes = block > 0 ? 4 * (size_t)num_pages * (page_size / block) * Hkv : 0;
    const size_t len_bytes = 4 * (size_t)N;
    const struct { const void* p; size_t n; } writes[] = {
        {k_cache, cache_bytes}, {v_cache, cache_bytes}, {block ? k_scales : nullptr, scale_bytes},
        {block ? v_scales : nullptr, scale_bytes}, {new_lengths, len_bytes}};
    const struct { const void* p; size_t n; } reads[] = {
        {cu_seqlens, len_bytes + 4}, {lengths, len_bytes}, {page_table, len_bytes * max_pages},
        {inv_freq, 2 * (size_t)rot_dim}};
    for (const auto& w : writes) {
        if (!w.p) continue;
        for (const RowSpan& x : {qi, ki, vi, qo, ko})
            if (meets(x, w.p, w.n)) return KDA_ERR_INVALID_ARG;
        for (const auto& r : reads)
            if (overlaps(w.p, w.n, r.p, r.n)) return KDA_ERR_INVALID_ARG;
    }
    for (const auto& r : reads)
        if (meets(qo, r.p, r.n) || meets(ko, r.p, r.n)) return KDA_ERR_INVALID_ARG;
    // (the pages of keys and values may lie between each other's)
    for (int i = 2; i < 5; ++i)
        for (int j = 0; j < i; ++j)
            if (writes[i].p && writes[j].p && overlaps(writes[i].p, writes[i].n, writes[j].p, writes[j].n))
                return KDA_ERR_INVALID_ARG;

    kda::RotaryArgs a = {};
    a.q = static_cast<const uint8_t*>(Hq ? q : nullptr);
    a.k = static_cast<const uint8_t*>(k);
    a.v = static_cast<const uint8_t*>(v);
    a.q_out = static_cast<uint8_t*>(q_out);
    a.k_out = static_cast<uint8_t*>(k_out);
    a.q_row = qi.step;
    a.k_row = ki.step;
    a.v_row = vi.step;
    a.q_out_row = qo.step;
    a.k_out_row = ko.step;
    a.k_cache = static_cast<uint8_t*>(k_cache);
    a.v_cache = static_cast<uint8_t*>(v_cache);
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.page_bytes = page_stride * (int64_t)held;
    a.cu_seqlens = cu_seqlens;
    a.page_table = page_table;
    a.lengths = lengths;
    a.new_lengths = new_lengths;
    a.inv_freq = inv_freq;
    a.T = (int32_t)T;
    a.N = N;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.rot = rot_dim;
    a.num_pages = num_pages;
    a.page_size = page_size;
    a.max_pages = max_pages;
    a.block = block;
    a.interleaved = interleaved != 0;
    const int sms = kda::device_sm_count();
    const cudaError_t err = kda::launch_cache_append_rotary(a, d, dtype != KDA_FP32, sms > 0 ? sms : 1, stream);
    return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

size_t kda_cache_attention_e4m3_workspace_bytes(int32_t N, int32_t Ts, int32_t Hq, int32_t Hkv, int32_t d,
                                                kda_dtype_t dtype)
{
    if (!valid_dtype(dtype) || !supported_d(d) || !newest_sizes(N, Ts, Hq, Hkv, d)) return 0;
    return kda::e4m3_workspace_bytes(Ts, Hq, Hkv, d, kda::device_sm_count());
}

kda_status_t kda_cache_attention_e4m3(const void* q, const void* k_cache, const void* v_cache, const float* k_scales,
                                      const float* v_scales, const int32_t* page_table, const int32_t* lengths,
                                      int32_t N, int32_t Ts, int32_t Hq, int32_t Hkv, int32_t d, int32_t num_pages,
                                      int32_t page_size, int32_t max_pages, int64_t page_stride, int32_t block,
                                      kda_dtype_t dtype, float scale, void* o, void* workspace, size_t workspace_bytes,
                                      cudaStream_t stream)
{
    if (!valid_dtype(dtype) || !supported_d(d) || page_size > kda::kMaxE4m3Page) return KDA_ERR_UNSUPPORTED;
    if (!newest_sizes(N, Ts, Hq, Hkv, d)) return KDA_ERR_INVALID_ARG;
    if (num_pages < 1 || page_size < 1 || max_pages < 1 || block < 1 || page_size % block != 0)
        return KDA_ERR_INVALID_ARG;
    if ((int64_t)max_pages * page_size > INT32_MAX - 1024) return KDA_ERR_INVALID_ARG;
    if (!q || !k_cache || !v_cache || !k_scales || !v_scales || !page_table || !lengths || !o) return KDA_ERR_INVALID_ARG;
    const void* ptrs16[] = {q, k_cache, v_cache, o};
    for (const void* p : ptrs16)
        if (!aligned(p, 16)) return KDA_ERR_INVALID_ARG;
    const void* ptrs4[] = {k_scales, v_scales, page_table, lengths};
    for (const void* p : ptrs4)
        if (!aligned(p, 4)) return KDA_ERR_INVALID_ARG;
    size_t cache_bytes = 0;
    if (!cache_shape(num_pages, page_size, Hkv, d, page_stride, 1, &cache_bytes)) return KDA_ERR_INVALID_ARG;
    const size_t rows = (size_t)N * Ts * Hq * d, o_bytes = rows * out_bytes(dtype);
    const size_t scale_bytes = 4 * (size_t)num_pages * (page_size / block) * Hkv;
    const int sms = kda::device_sm_count();
    const size_t need = kda::e4m3_workspace_bytes(Ts, Hq, Hkv, d, sms);
    if (!workspace || workspace_bytes < need || !aligned(workspace, 256)) return KDA_ERR_WORKSPACE;
    const struct { const void* p; size_t n; } reads[] = {
        {q, rows * in_bytes(dtype)}, {k_cache, cache_bytes}, {v_cache, cache_bytes}, {k_scales, scale_bytes},
        {v_scales, scale_bytes}, {page_table, 4 * (size_t)N * max_pages}, {lengths, 4 * (size_t)N}};
    for (const auto& r : reads)
        if (overlaps(o, o_bytes, r.p, r.n) || overlaps(workspace, need, r.p, r.n)) return KDA_ERR_INVALID_ARG;
    if (overlaps(o, o_bytes, workspace, need)) return KDA_ERR_INVALID_ARG;

    kda::E4m3Args a = {};
    a.split.N = N;
    a.split.Ts = 1;
    a.Hkv = Hkv;
    a.split.lengths = lengths;
    a.split.page_table = page_table;
    a.split.page_size = page_size;
    a.split.max_pages = max_pages;
    a.q = q;
    a.k_cache = static_cast<const uint8_t*>(k_cache);
    a.v_cache = static_cast<const uint8_t*>(v_cache);
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.Ts = Ts;
    a.Hq = Hq;
    a.G = Hq / Hkv;
    a.R = Ts * a.G;
    a.num_pages = num_pages;
    a.block = block;
    a.blocks = page_size / block;
    a.block_magic = block > 1 ? (uint32_t)(((1ull << 32) + block - 1) / block) : 0;
    a.page_stride = page_stride;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.o = o;
    a.status = static_cast<int32_t*>(workspace) + kda::kWsTimeoutWord;
    a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kda::kWsHeaderBytes);
    const cudaError_t err = kda::launch_cache_attention_e4m3(a, d, dtype, sms, stream);
    return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
