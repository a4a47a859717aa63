// pa_api_fp8_block.cu — C ABI of the e4m3 pools with a scale per (block, kv
// head): argument checks and dispatch.  Like pa_api.cu, every entry point
// validates on the host and launches nothing when a check fails.
#include <algorithm>
#include <climits>
#include <cstdint>

#include "pa_internal.cuh"

namespace pa {
namespace {
bool aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// The split of pa_decode_fp8_block's contexts: partitions of whole 128-token stages (powers of two), long enough that a
// partition's partial result is small beside the codes it reads, short enough that the batch (at its longest context: the
// lengths live on the device) gives every SM six items; at most 128 partials per (sequence, head).  The last fifth of the
// sequences is split in half partitions, so that the ends are less uneven.  Measured, us (64 sequences, 65,500 tokens,
// 32/8 heads; 16 long contexts, 189,395 tokens, 64/8 heads; 16 other long contexts, 32/8 heads; 64 contexts of 1000; 8 of
// 2000 to 4000 tokens):
//   a tenth in quarter partitions, eight items per SM   32.5   74.7   62.7   36.1   21.4
//   a tenth in quarter partitions, six                  32.2   74.3   62.1   33.9   19.3
//   15 % in halves, six                                 32.6   73.2   59.7   32.4   19.2
//   a fifth in halves, six                              31.9   74.0   59.4   32.4   19.1
//   a quarter in halves, six                            32.3   73.8   59.5   32.7   20.2
//   a fifth in quarters, eight                          32.2   79.3   60.9   36.4   21.4
//   partitions of 512 / 2048 (a tenth in quarters / eighths, eight)  34.0 / 32.6   80.0 / 78.1   63.0 / 66.6
constexpr int kPartition = 1024, kItemsPerSm = 6, kTailPercent = 20, kTailDivisor = 2;

DecodePlan plan_decode_fp8_block(int num_seqs, int num_kv_heads, int max_context_len, int num_sms) {
    auto splits = [&](long long part) { return max_context_len <= part ? 1LL : (max_context_len + part - 1) / part; };
    long long part = kPartition;
    while (part > 128 && splits(part) * num_seqs * num_kv_heads < (long long)kItemsPerSm * num_sms)
        part /= 2;
    while (splits(part) > 128) part *= 2;
    long long small = part / kTailDivisor < 128 ? 128 : part / kTailDivisor;
    while (splits(small) > 128) small *= 2;
    const int tail = small < part ? (int)((long long)num_seqs * kTailPercent / 100) : 0;
    return DecodePlan{(int)part, (int)splits(tail ? small : part), (int)small, num_seqs - tail};
}

// The most partial rows of a kv head that the plan of any call of up to num_seqs sequences and max_context_len tokens has,
// so that one workspace serves a batch that shrinks (a smaller one is cut finer, and may have more of them than a larger).
// With kPartition tokens a partition, sequences of half ones have the most.  Where the plan halved its
// partitions, twice as long ones gave fewer than kItemsPerSm items per SM: halving them doubles the items at
// most, and the tail's shorter ones do so kTailDivisor-fold; no partition is below 128 tokens.
long long most_partials(int num_seqs, int num_kv_heads, int max_context_len, int num_sms) {
    auto splits = [&](long long part) {
        const long long n = max_context_len <= part ? 1LL : (max_context_len + part - 1) / part;
        return n < 128 ? n : 128LL;
    };
    const long long halved = (2LL * kTailDivisor * kItemsPerSm * num_sms - 1) / num_kv_heads;
    return std::max(num_seqs * splits(kPartition / kTailDivisor),
                    std::min(num_seqs * splits(128), halved));
}

// Row shape of the write and the read back: 16-byte pieces of codes, blocks of at most 1024 slots.
int rows_ok(int num_kv_heads, int head_dim, int block_size) {
    if (num_kv_heads < 1 || head_dim < 1 || block_size < 1) return PA_ERR_INVALID_ARG;
    if (head_dim % 16 != 0 || (long long)num_kv_heads * head_dim > (1 << 20) || block_size > 1024)
        return PA_ERR_UNSUPPORTED;
    return PA_OK;
}
}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

size_t pa_write_fp8_block_workspace_size(int num_tokens, int num_blocks, int block_size) {
    if (num_tokens < 0 || num_blocks < 0 || block_size < 1 || block_size > 1024) return 0;
    return write_fp8_block_workspace(num_tokens, num_blocks, block_size);
}

int pa_write_kv_paged_fp8_block(const void* k_new, const void* v_new, int num_tokens, int num_kv_heads, int head_dim,
                                void* k_cache, void* v_cache, float* k_scales, float* v_scales, int num_blocks,
                                int block_size, const int32_t* block_tables, int num_seqs, int max_blocks_per_seq,
                                const int32_t* seq_idx, const int32_t* pos, int64_t* slot_mapping, void* workspace,
                                size_t workspace_bytes, int32_t* error_count, void* stream) {
    if (num_tokens < 0 || num_blocks < 0 || num_seqs < 0 || max_blocks_per_seq < 0) return PA_ERR_INVALID_ARG;
    int rc = rows_ok(num_kv_heads, head_dim, block_size);
    if (rc != PA_OK) return rc;
    if (num_tokens == 0) return PA_OK;
    if (!k_new || !v_new || !k_cache || !v_cache || !k_scales || !v_scales || !seq_idx || !pos ||
        (num_seqs > 0 && max_blocks_per_seq > 0 && !block_tables))
        return PA_ERR_INVALID_ARG;
    if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16))
        return PA_ERR_UNSUPPORTED;
    int num_sms = 0;
    if ((rc = check_device(&num_sms)) != PA_OK) return rc;
    const size_t need = write_fp8_block_workspace(num_tokens, num_blocks, block_size);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256))) return PA_ERR_WORKSPACE;
    return launch_write_fp8_block(k_new, v_new, num_tokens, num_kv_heads, head_dim, k_cache, v_cache, k_scales,
                                  v_scales, num_blocks, block_size, block_tables, num_seqs, max_blocks_per_seq,
                                  seq_idx, pos, slot_mapping, workspace, num_sms, error_count,
                                  static_cast<cudaStream_t>(stream));
}

int pa_read_kv_paged_fp8_block(void* k_out, void* v_out, int num_tokens, int num_kv_heads, int head_dim, int dtype,
                               const void* k_cache, const void* v_cache, const float* k_scales, const float* v_scales,
                               int num_blocks, int block_size, const int32_t* block_tables, int num_seqs,
                               int max_blocks_per_seq, const int32_t* seq_idx, const int32_t* pos,
                               int32_t* error_count, void* stream) {
    if (num_tokens < 0 || num_blocks < 0 || num_seqs < 0 || max_blocks_per_seq < 0) return PA_ERR_INVALID_ARG;
    int rc = rows_ok(num_kv_heads, head_dim, block_size);
    if (rc != PA_OK) return rc;
    if (dtype != PA_F32 && dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
    if (num_tokens == 0) return PA_OK;
    if (!k_out || !v_out || !k_cache || !v_cache || !k_scales || !v_scales || !seq_idx || !pos ||
        (num_seqs > 0 && max_blocks_per_seq > 0 && !block_tables))
        return PA_ERR_INVALID_ARG;
    if (!aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16))
        return PA_ERR_UNSUPPORTED;
    if ((rc = check_device(nullptr)) != PA_OK) return rc;
    return launch_read_fp8_block(k_out, v_out, num_tokens, num_kv_heads, head_dim, dtype, k_cache, v_cache, k_scales,
                                 v_scales, num_blocks, block_size, block_tables, num_seqs, max_blocks_per_seq, seq_idx,
                                 pos, error_count, static_cast<cudaStream_t>(stream));
}

size_t pa_decode_fp8_block_workspace_size(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                          int block_size, int max_context_len) {
    if (num_seqs < 0 || max_context_len < 0 || decode_shape_ok(num_q_heads, num_kv_heads, head_dim, block_size))
        return 0;
    int num_sms = 0;
    if (check_device(&num_sms) != PA_OK) return 0;
    // (as many sequences of one partial each)
    const long long partials = most_partials(num_seqs, num_kv_heads, max_context_len, num_sms);
    if (partials > INT_MAX) return 0;
    return decode_workspace_layout((int)partials, num_q_heads, num_kv_heads, head_dim, 1).total;
}

int pa_decode_fp8_block(void* out, const void* q, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                        const void* k_cache, const void* v_cache, const float* k_scales, const float* v_scales,
                        int num_blocks, int block_size, const int32_t* block_tables, int max_blocks_per_seq,
                        const int32_t* context_lens, int max_context_len, float scale, void* workspace,
                        size_t workspace_bytes, int32_t* error_count, void* stream) {
    if (num_seqs < 0 || num_blocks < 0 || max_blocks_per_seq < 0 || max_context_len < 0) return PA_ERR_INVALID_ARG;
    int rc = decode_shape_ok(num_q_heads, num_kv_heads, head_dim, block_size);
    if (rc != PA_OK) return rc;
    if (num_seqs == 0) return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !k_scales || !v_scales || !context_lens ||
        (max_blocks_per_seq > 0 && !block_tables))
        return PA_ERR_INVALID_ARG;
    int num_sms = 0;
    if ((rc = check_device(&num_sms)) != PA_OK) return rc;
    const DecodePlan plan = plan_decode_fp8_block(num_seqs, num_kv_heads, max_context_len, num_sms);
    const DecodeWorkspace lay =
        decode_workspace_layout(num_seqs, num_q_heads, num_kv_heads, head_dim, plan.max_splits);
    if (!workspace || workspace_bytes < lay.total || !aligned(workspace, 256)) return PA_ERR_WORKSPACE;
    char* ws = static_cast<char*>(workspace);
    DecodeParams p;
    p.out = out;
    p.q = q;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.error_count = error_count;
    p.work = reinterpret_cast<int*>(ws + lay.work);
    p.ws_ml = reinterpret_cast<float2*>(ws + lay.ml);
    p.ws_o = reinterpret_cast<float*>(ws + lay.o);
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
    rc = decode_fp8_block_tc_supported(p) ? launch_decode_fp8_block_tc(p, num_sms, st)
                                          : launch_decode_fp8_block_fma(p, st);
    if (rc != PA_OK) return rc;
    return launch_decode_fp8_block_join(p, st);
}

size_t pa_prefill_fp8_block_workspace_size(int num_chunks, int total_q, int max_q_len, int num_q_heads,
                                           int num_kv_heads, int head_dim, int block_size, int max_context_len) {
    int num_sms = 0;
    if (num_chunks <= 0 || total_q <= 0 || max_q_len <= 0 || max_context_len < 0 ||
        decode_shape_ok(num_q_heads, num_kv_heads, head_dim, block_size) != PA_OK || head_dim != 128 ||
        num_q_heads / num_kv_heads > 8 || check_device(&num_sms) != PA_OK)
        return 0;
    return prefill_fp8_block_workspace(num_chunks, total_q, max_q_len, num_q_heads, num_kv_heads, max_context_len,
                                       num_sms);
}

int pa_prefill_chunk_fp8_block(void* out, const void* q, const int32_t* cu_q_lens, const int32_t* q_start_pos,
                               const int32_t* seq_of_chunk, int num_chunks, int total_q, int max_q_len, int num_seqs,
                               int num_q_heads, int num_kv_heads, int head_dim, const void* k_cache,
                               const void* v_cache, const float* k_scales, const float* v_scales, int num_blocks,
                               int block_size, const int32_t* block_tables, int max_blocks_per_seq,
                               const int32_t* context_lens, int max_context_len, float scale, void* workspace,
                               size_t workspace_bytes, int32_t* error_count, void* stream) {
    if (num_chunks < 0 || total_q < 0 || max_q_len < 0 || num_seqs < 0 || num_blocks < 0 || max_blocks_per_seq < 0 ||
        max_context_len < 0)
        return PA_ERR_INVALID_ARG;
    int rc = decode_shape_ok(num_q_heads, num_kv_heads, head_dim, block_size);
    if (rc != PA_OK) return rc;
    if (num_chunks == 0 || total_q == 0 || max_q_len == 0) return PA_OK;
    if (!out || !q || !cu_q_lens || !q_start_pos || !seq_of_chunk || !k_cache || !v_cache || !k_scales || !v_scales ||
        !context_lens || !block_tables || num_seqs == 0)
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
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.error_count = error_count;
    p.num_chunks = num_chunks;
    p.total_q = total_q;
    p.max_q_len = max_q_len;
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
    if (!prefill_fp8_block_tc_supported(p)) return launch_prefill_fp8_block_fma(p, static_cast<cudaStream_t>(stream));
    const size_t need = prefill_fp8_block_need(p, num_sms);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256))) return PA_ERR_WORKSPACE;
    return launch_prefill_fp8_block_tc(p, workspace, need > 0 ? workspace_bytes : 0, num_sms,
                                       static_cast<cudaStream_t>(stream));
}

}  // extern "C"
