// pa_api_weights.cu — C ABI of the caches that evict tokens: rotary positions
// and their paged write, attention that accumulates each key's weight, the
// eviction.  Like pa_api.cu, every entry point validates on the host and
// launches nothing when a check fails.
#include <algorithm>
#include <climits>
#include <cstdint>

#include "pa_internal.cuh"

namespace pa {
namespace {

bool aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
size_t round_up(size_t n) { return (n + 255) / 256 * 256; }

// Longest contexts: the decode's second launch has a CTA for every 1024 tokens, and 65535 rows of CTAs; elsewhere indices are
// 32-bit integers that pass a context's end by less than 2^30.
constexpr int kMaxDecodeContext = 65534 * 1024, kMaxContext = 1 << 30;

// Shapes of the rotary calls.
int rope_ok(int num_tokens, int num_q_heads, int num_kv_heads, int head_dim, int dtype, int num_axes, int rot_dim) {
    if (num_tokens < 0 || num_q_heads < 0 || num_kv_heads < 0 || head_dim < 1 || rot_dim < 0 || rot_dim > head_dim ||
        rot_dim % 2 != 0 || (rot_dim > 0 && num_axes < 1))
        return PA_ERR_INVALID_ARG;
    if (dtype != PA_F32 && dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
    if (head_dim > 1024 || (long long)(num_q_heads + (long long)num_kv_heads) * head_dim > (1 << 20))
        return PA_ERR_UNSUPPORTED;
    return PA_OK;
}

// Partial rows ((sequence, kv head, partition)) that pa_decode's plan of any call of up to num_seqs sequences and
// max_context_len tokens has, so that one workspace serves a batch that shrinks: a smaller batch is cut finer.  For each
// batch size and each partition of the plan's halvings the most rows are those of the longest context for which the plan
// stops there: the next longer partition must give fewer than two items per SM.
long long most_partials(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int max_context_len, int num_sms) {
    long long most = std::max(1LL, (long long)num_seqs * num_kv_heads);  // one each, with no token too
    for (long long n = 1; n <= num_seqs; ++n) {
        // the plan at these lengths, where its partition changes: the longest context that has it
        long long ctx = max_context_len;
        while (ctx > 0) {
            const DecodePlan plan = plan_decode((int)n, num_q_heads, num_kv_heads, head_dim, (int)ctx, num_sms, SIZE_MAX);
            const long long small = std::max(64, (plan.partition / 4) & ~63);
            most = std::max(most, n * num_kv_heads * std::min(128LL, (ctx + small - 1) / small));
            if (plan.partition <= 64) break;
            // the longest shorter context with a shorter partition
            long long lo = 0, hi = ctx;  // plan(lo) shorter (or lo == 0), plan(hi) this long
            while (hi - lo > 1) {
                const long long mid = (lo + hi) / 2;
                (plan_decode((int)n, num_q_heads, num_kv_heads, head_dim, (int)mid, num_sms, SIZE_MAX).partition <
                 plan.partition ? lo : hi) = mid;
            }
            ctx = lo;
        }
    }
    return most;
}

// Spans that the keys of pa_prefill_chunk_weights's query tiles are cut into: as many as places for CTAs that the tiles leave
// idle can take; one where the tiles fill the GPU.  On the tensor cores (tiles of 128 rows and 128 keys, a CTA an SM) a span
// has three key tiles at least: 37 queries over 3000 keys, 16 tiles, 54.4 us with one span, 35.5 with spans of two key tiles,
// 34.0 of three, 36.1 of four.  On the CUDA cores (tiles of 64, two CTAs an SM) a key tile takes so long that each may be a
// span: 20 fp32 queries over 235 keys, 32/8 heads, 99 us with spans of three tiles or more, 66 of two, 57 of one.
int spans_of(int num_chunks, int total_q, int max_q_len, int group, int num_kv_heads, int max_context_len, int num_sms,
             bool tc) {
    const int tile = tc ? 128 : 64, ctas = tc ? num_sms : 2 * num_sms, least = tc ? 3 : 1, per_tile = tile / group;
    const long long tiles = (long long)num_chunks * num_kv_heads * ((max_q_len + per_tile - 1) / per_tile);
    const long long key_tiles = ((long long)max_context_len + tile - 1) / tile;
    // (q may have rows behind its chunks; the workspace holds 128 rows for each SM)
    const long long fit = 128LL * num_sms / ((long long)total_q * group * num_kv_heads);
    return (int)std::max(1LL, std::min({(long long)kMaxSpans, ctas / std::max(1LL, tiles), key_tiles / least, fit}));
}

// Workspace of pa_prefill_chunk_weights: the rows' lse, what comes before each chunk, the keys' partial sums (rows of 256
// keys, one for each (chunk, kv head, 256 keys) and one more for each SM, in kKeyParts parts), and the spans' partial rows:
// tiles of 128 rows of which there are no more than SMs, and no more than kMaxSpans of a row.
struct PrefillWeightsWorkspace {
    size_t lse, runs, partial, ml, o, total;
};
PrefillWeightsWorkspace prefill_weights_layout(int num_chunks, int total_q, int num_q_heads, int num_kv_heads,
                                               int max_context_len, int num_sms) {
    PrefillWeightsWorkspace w;
    const size_t rows = (size_t)num_chunks * num_kv_heads * (((size_t)max_context_len + 255) / 256) + num_sms;
    const size_t q_rows = (size_t)total_q * num_q_heads;
    const size_t span_rows = std::min(q_rows * kMaxSpans, (size_t)num_sms * 128);
    w.lse = 0;
    w.runs = round_up(q_rows * 4);
    w.partial = w.runs + round_up(((size_t)num_chunks + 1) * sizeof(KeyRuns));
    w.ml = w.partial + rows * 256 * kKeyParts * 4;
    w.o = w.ml + round_up(span_rows * sizeof(float2));
    w.total = w.o + span_rows * 128 * 4;
    return w;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

int pa_rope(void* q_out, void* k_out, const void* q, const void* k, int num_tokens, int num_q_heads, int num_kv_heads,
            int head_dim, int dtype, long long q_stride, long long k_stride, const int32_t* rope_pos, int num_axes,
            const float* inv_freq, const int32_t* axis, int rot_dim, int interleaved, int32_t* error_count,
            void* stream) {
    int rc = rope_ok(num_tokens, num_q_heads, num_kv_heads, head_dim, dtype, num_axes, rot_dim);
    if (rc != PA_OK) return rc;
    if (num_tokens == 0 || num_q_heads + num_kv_heads == 0) return PA_OK;
    if ((num_q_heads > 0 && (!q || !q_out)) || (num_kv_heads > 0 && (!k || !k_out)) ||
        (rot_dim > 0 && (!rope_pos || !inv_freq)))
        return PA_ERR_INVALID_ARG;
    int num_sms = 0;
    if ((rc = check_device(&num_sms)) != PA_OK) return rc;
    RopeParams p;
    p.q = q;
    p.k = k;
    p.v = nullptr;
    p.q_out = q_out;
    p.k_out = k_out;
    p.v_out = nullptr;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = 0;
    p.rope_pos = rope_pos;
    p.inv_freq = inv_freq;
    p.axis = axis;
    p.num_tokens = num_tokens;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.head_dim = head_dim;
    p.rot_dim = rot_dim;
    p.num_axes = num_axes;
    p.interleaved = interleaved != 0;
    p.error_count = error_count;
    return launch_rope(p, dtype, num_sms, static_cast<cudaStream_t>(stream));
}

int pa_rope_write_kv_paged(void* q_out, const void* q, const void* k_new, const void* v_new, int num_tokens,
                           int num_q_heads, int num_kv_heads, int head_dim, int dtype, long long q_stride,
                           long long k_stride, long long v_stride, const int32_t* rope_pos, int num_axes,
                           const float* inv_freq, const int32_t* axis, int rot_dim, int interleaved, void* k_cache,
                           void* v_cache, int num_blocks, int block_size, const int32_t* block_tables, int num_seqs,
                           int max_blocks_per_seq, const int32_t* seq_idx, const int32_t* pos, float* key_weights,
                           int32_t* key_pos, int key_width, const int32_t* token_pos, int64_t* slot_mapping,
                           int32_t* error_count, void* stream) {
    int rc = rope_ok(num_tokens, num_q_heads, num_kv_heads, head_dim, dtype, num_axes, rot_dim);
    if (rc != PA_OK) return rc;
    if (num_kv_heads < 1 || num_blocks < 0 || block_size < 1 || num_seqs < 0 || max_blocks_per_seq < 0 || key_width < 0 ||
        (key_weights == nullptr) != (key_pos == nullptr) || (key_weights != nullptr && key_width < 1))
        return PA_ERR_INVALID_ARG;
    if (block_size > (1 << 30)) return PA_ERR_UNSUPPORTED;
    if (num_tokens == 0) return PA_OK;
    if ((num_q_heads > 0 && (!q || !q_out)) || !k_new || !v_new || !k_cache || !v_cache || !seq_idx || !pos ||
        (num_seqs > 0 && max_blocks_per_seq > 0 && !block_tables) || (rot_dim > 0 && (!rope_pos || !inv_freq)))
        return PA_ERR_INVALID_ARG;
    int num_sms = 0;
    if ((rc = check_device(&num_sms)) != PA_OK) return rc;
    RopeParams p;
    p.q = q;
    p.k = k_new;
    p.v = v_new;
    p.q_out = q_out;
    p.k_out = k_cache;
    p.v_out = v_cache;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.rope_pos = rope_pos;
    p.inv_freq = inv_freq;
    p.axis = axis;
    p.num_tokens = num_tokens;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.head_dim = head_dim;
    p.rot_dim = rot_dim;
    p.num_axes = num_axes;
    p.interleaved = interleaved != 0;
    p.block_tables = block_tables;
    p.seq_idx = seq_idx;
    p.pos = pos;
    p.token_pos = token_pos;
    p.num_blocks = num_blocks;
    p.block_size = block_size;
    p.num_seqs = num_seqs;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.key_weights = key_weights;
    p.key_pos = key_pos;
    p.key_width = key_weights ? key_width : 0;
    p.slot_mapping = slot_mapping;
    p.error_count = error_count;
    return launch_rope(p, dtype, num_sms, static_cast<cudaStream_t>(stream));
}

size_t pa_decode_weights_workspace_size(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                        int max_context_len) {
    if (num_seqs < 0 || max_context_len < 0 || max_context_len > kMaxDecodeContext ||
        decode_shape_ok(num_q_heads, num_kv_heads, head_dim, block_size))
        return 0;
    int num_sms = 0;
    if (check_device(&num_sms) != PA_OK) return 0;
    const long long partials = most_partials(num_seqs, num_q_heads, num_kv_heads, head_dim, max_context_len, num_sms);
    if (partials > INT_MAX) return 0;
    // (as many sequences of one kv head and one partial each)
    const int group = num_q_heads / num_kv_heads;
    return decode_workspace_layout((int)partials, group, 1, head_dim, 1).total +
           round_up((size_t)num_seqs * num_q_heads * max_context_len * 4);
}

int pa_decode_weights(void* out, const void* q, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                      int dtype, const void* k_cache, const void* v_cache, int num_blocks, int block_size,
                      const int32_t* block_tables, int max_blocks_per_seq, const int32_t* context_lens,
                      int max_context_len, float scale, float* key_weights, int key_width, void* workspace,
                      size_t workspace_bytes, int32_t* error_count, void* stream) {
    if (num_seqs < 0 || num_blocks < 0 || max_blocks_per_seq < 0 || max_context_len < 0 || key_width < max_context_len)
        return PA_ERR_INVALID_ARG;
    int rc = decode_shape_ok(num_q_heads, num_kv_heads, head_dim, block_size);
    if (rc != PA_OK) return rc;
    if ((dtype != PA_F32 && dtype != PA_BF16) || max_context_len > kMaxDecodeContext) return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !context_lens || (key_width > 0 && !key_weights) ||
        (max_blocks_per_seq > 0 && !block_tables))
        return PA_ERR_INVALID_ARG;
    int num_sms = 0;
    if ((rc = check_device(&num_sms)) != PA_OK) return rc;
    const DecodePlan plan =
        plan_decode(num_seqs, num_q_heads, num_kv_heads, head_dim, max_context_len, num_sms, SIZE_MAX);
    const DecodeWorkspace lay =
        decode_workspace_layout(num_seqs, num_q_heads, num_kv_heads, head_dim, plan.max_splits);
    const size_t scores = (size_t)num_seqs * num_q_heads * max_context_len * 4;
    if (!workspace || workspace_bytes < lay.total + scores || !aligned(workspace, 256)) return PA_ERR_WORKSPACE;
    char* ws = static_cast<char*>(workspace);
    DecodeParams p;
    p.out = out;
    p.q = q;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.error_count = error_count;
    p.work = reinterpret_cast<int*>(ws + lay.work);
    p.ws_ml = reinterpret_cast<float2*>(ws + lay.ml);
    p.ws_o = reinterpret_cast<float*>(ws + lay.o);
    p.ws_scores = reinterpret_cast<float*>(ws + lay.total);
    p.score_width = max_context_len;
    p.key_weights = key_weights;
    p.key_width = key_width;
    p.num_seqs = num_seqs;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.head_dim = head_dim;
    p.group = num_q_heads / num_kv_heads;
    p.num_blocks = num_blocks;
    p.block_size = block_size;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.max_context_len = max_context_len;
    p.partition = plan.partition;
    p.small_partition = plan.small_partition;
    p.small_from = plan.small_from;
    p.max_splits = plan.max_splits;
    p.scale_log2 = scale * 1.4426950408889634f;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (decode_tc_supported(p, dtype)) {
        rc = launch_decode_tc(p, num_sms, st);
    } else {
        p.small_from = 1 << 30;  // one CTA for each partition: uniform ones
        rc = launch_decode_weights_fma(p, dtype, st);
    }
    return rc != PA_OK ? rc : launch_decode_weights(p, dtype, st);
}

size_t pa_prefill_weights_workspace_size(int num_chunks, int total_q, int max_q_len, int num_q_heads, int num_kv_heads,
                                         int head_dim, int block_size, int max_context_len) {
    if (num_chunks < 0 || total_q < 0 || max_q_len < 0 || max_context_len < 0 || max_context_len > kMaxContext ||
        decode_shape_ok(num_q_heads, num_kv_heads, head_dim, block_size))
        return 0;
    int num_sms = 0;
    if (check_device(&num_sms) != PA_OK) return 0;
    return prefill_weights_layout(num_chunks, total_q, num_q_heads, num_kv_heads, max_context_len, num_sms).total;
}

int pa_prefill_chunk_weights(void* out, const void* q, const int32_t* cu_q_lens, const int32_t* q_start_pos,
                             const int32_t* seq_of_chunk, int num_chunks, int total_q, int max_q_len, int num_seqs,
                             int num_q_heads, int num_kv_heads, int head_dim, int dtype, const void* k_cache,
                             const void* v_cache, int num_blocks, int block_size, const int32_t* block_tables,
                             int max_blocks_per_seq, const int32_t* context_lens, int max_context_len, float scale,
                             float* key_weights, int key_width, void* workspace, size_t workspace_bytes,
                             int32_t* error_count, void* stream) {
    if (num_chunks < 0 || total_q < 0 || max_q_len < 0 || num_seqs < 0 || num_blocks < 0 || max_blocks_per_seq < 0 ||
        max_context_len < 0 || key_width < max_context_len)
        return PA_ERR_INVALID_ARG;
    int rc = decode_shape_ok(num_q_heads, num_kv_heads, head_dim, block_size);
    if (rc != PA_OK) return rc;
    if ((dtype != PA_F32 && dtype != PA_BF16) || max_context_len > kMaxContext) return PA_ERR_UNSUPPORTED;
    if (num_chunks == 0 || total_q == 0 || max_q_len == 0) return PA_OK;
    if (!out || !q || !cu_q_lens || !q_start_pos || !seq_of_chunk || !k_cache || !v_cache || !context_lens ||
        !block_tables || num_seqs == 0 || (key_width > 0 && !key_weights))
        return PA_ERR_INVALID_ARG;
    int num_sms = 0;
    if ((rc = check_device(&num_sms)) != PA_OK) return rc;
    PrefillParams p;
    p.out = out;
    p.q = q;
    p.cu_q_lens = cu_q_lens;
    p.q_start_pos = q_start_pos;
    p.seq_of_chunk = seq_of_chunk;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.error_count = error_count;
    p.num_chunks = num_chunks;
    p.total_q = total_q;
    p.max_q_len = max_q_len = std::min(max_q_len, total_q);  // (no usable chunk is longer)
    p.num_seqs = num_seqs;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.head_dim = head_dim;
    p.group = num_q_heads / num_kv_heads;
    p.num_blocks = num_blocks;
    p.block_size = block_size;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.max_context_len = max_context_len;
    p.scale_log2 = scale * 1.4426950408889634f;
    const PrefillWeightsWorkspace lay =
        prefill_weights_layout(num_chunks, total_q, num_q_heads, num_kv_heads, max_context_len, num_sms);
    if (!workspace || workspace_bytes < lay.total || !aligned(workspace, 256)) return PA_ERR_WORKSPACE;
    char* ws = static_cast<char*>(workspace);
    p.lse = reinterpret_cast<float*>(ws + lay.lse);
    p.partial = reinterpret_cast<float*>(ws + lay.partial);
    p.key_weights = key_weights;
    p.key_width = key_width;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    // (the second kernel keeps 8 bytes for each chunk in its 128 KB of key buffers at first)
    const bool tc = prefill_tc_supported(p, dtype) && num_chunks <= 16384 && max_context_len > 0;
    p.spans = spans_of(num_chunks, total_q, max_q_len, p.group, num_kv_heads, max_context_len, num_sms, tc);
    p.part_ml = reinterpret_cast<float2*>(ws + lay.ml);
    p.part_o = reinterpret_cast<float*>(ws + lay.o);
    if (tc) {
        p.runs = reinterpret_cast<KeyRuns*>(ws + lay.runs);
        rc = launch_prefill_tc(p, st);
        if (rc == PA_OK) rc = launch_prefill_weights_tc(p, num_sms, st);
    } else {
        rc = launch_prefill_weights_fma(p, dtype, st);
    }
    return rc != PA_OK ? rc : launch_prefill_weights_add(p, st);
}

size_t pa_evict_workspace_size(int num_seqs, int num_kv_heads, int max_context_len, int budget) {
    if (num_seqs < 0 || num_kv_heads < 1 || max_context_len < 0 || max_context_len > kMaxContext || budget < 1) return 0;
    const EvictWorkspace lay = evict_workspace_layout(num_seqs, num_kv_heads, max_context_len, budget);
    return lay.max_moves > kMaxMoves ? 0 : lay.total;
}

int pa_evict_tokens(void* k_cache, void* v_cache, int num_blocks, int block_size, int num_kv_heads, int head_dim,
                    int dtype, const int32_t* block_tables, int num_seqs, int max_blocks_per_seq,
                    const int32_t* context_lens, int max_context_len, float* key_weights, int32_t* key_pos,
                    int key_width, const int32_t* next_pos, int budget, int keep_first, int keep_recent,
                    int32_t* new_lens, void* workspace, size_t workspace_bytes, int32_t* error_count, void* stream) {
    if (num_blocks < 0 || block_size < 1 || num_kv_heads < 1 || head_dim < 1 || num_seqs < 0 || max_blocks_per_seq < 0 ||
        max_context_len < 0 || key_width < max_context_len || budget < 1 || keep_first < 0 || keep_recent < 0 ||
        (long long)keep_first + keep_recent > budget)
        return PA_ERR_INVALID_ARG;
    if ((dtype != PA_F32 && dtype != PA_BF16) || max_context_len > kMaxContext) return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PA_OK;
    if (!k_cache || !v_cache || !context_lens || !next_pos || !new_lens || (key_width > 0 && (!key_weights || !key_pos)) ||
        (max_blocks_per_seq > 0 && !block_tables))
        return PA_ERR_INVALID_ARG;
    const long long row_bytes = (long long)head_dim * elem_size(dtype);
    if (row_bytes % 16 != 0 || row_bytes > (1 << 20) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        (long long)num_seqs * num_kv_heads > INT_MAX)
        return PA_ERR_UNSUPPORTED;
    const EvictWorkspace lay = evict_workspace_layout(num_seqs, num_kv_heads, max_context_len, budget);
    if (lay.max_moves > kMaxMoves) return PA_ERR_UNSUPPORTED;
    int rc = check_device(nullptr);
    if (rc != PA_OK) return rc;
    if (!workspace || workspace_bytes < lay.total || !aligned(workspace, 256)) return PA_ERR_WORKSPACE;
    char* ws = static_cast<char*>(workspace);
    EvictParams p;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.num_blocks = num_blocks;
    p.block_size = block_size;
    p.num_kv_heads = num_kv_heads;
    p.block_tables = block_tables;
    p.num_seqs = num_seqs;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.context_lens = context_lens;
    p.max_context_len = max_context_len;
    p.key_weights = key_weights;
    p.key_pos = key_pos;
    p.key_width = key_width;
    p.next_pos = next_pos;
    p.budget = budget;
    p.keep_first = keep_first;
    p.keep_recent = keep_recent;
    p.new_lens = new_lens;
    p.counts = reinterpret_cast<int*>(ws + lay.counts);
    p.lens = reinterpret_cast<int*>(ws + lay.lens);
    p.src = reinterpret_cast<int*>(ws + lay.src);
    p.dst = reinterpret_cast<int*>(ws + lay.dst);
    p.max_moves = lay.max_moves;
    p.error_count = error_count;
    return launch_evict(p, (int)row_bytes, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
