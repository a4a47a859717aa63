// attend_fp8_block_fma.cu — decode and causal chunked prefill over e4m3 pools
// with a scale per (block, kv head) on the CUDA cores: the path for shapes the
// tensor-core kernels do not take (head_dim 64, groups over 8 query heads,
// block sizes that are no power of two from 8 to 128).
//
// The loop is fma_attend.cuh's; codes are widened as they are read from the
// staged rows.  Decode: one CTA per (sequence, kv head, partition), joined as in
// decode_fp8_block_tc.cu.  Prefill: one CTA per (query, kv head).  Bound by
// instructions, far from HBM (64 sequences, 32/8 heads of 128, 65,500 tokens:
// 750 us, 0.027 of the copy bandwidth, where the tensor-core kernel takes 31;
// four chunks of 512 queries at short offsets: 4.9 ms, where it takes 33 us).
#include "decode_common.cuh"
#include "fma_attend.cuh"

namespace pa {
namespace {

using Bf16 = __nv_bfloat16;

template <int D>
__global__ void __launch_bounds__(kFmaThreads) decode_fp8_block_fma_kernel(DecodeParams p) {
    using S = FmaShape<D>;
    pdl_trigger();
    pdl_wait();
    const int s = blockIdx.x, kvh = blockIdx.y, split = blockIdx.z, G = p.group;
    const int L = decode_context(p, s, split == 0 && kvh == 0 && threadIdx.x == 0);
    const int part = partition_of(p, s), nsplit = num_partitions(L, part);
    if (split >= nsplit) return;
    const int j0 = split * part, j1 = min(L, j0 + part);
    extern __shared__ float smem[];
    __shared__ float m_s[kFmaMaxGroup], l_s[kFmaMaxGroup], alpha_s[kFmaMaxGroup];
    float acc[S::kItems];
    const size_t row = ((size_t)s * p.num_q_heads + (size_t)kvh * G) * D;
    fma_attend<Bf16, D, e4m3_t>(static_cast<const Bf16*>(p.q) + row, G, static_cast<const e4m3_t*>(p.k_cache),
                                static_cast<const e4m3_t*>(p.v_cache),
                                p.block_tables + (size_t)s * p.max_blocks_per_seq, p.block_size, p.num_kv_heads, kvh,
                                p.num_blocks, j0, j1, p.scale_log2, p.error_count, smem, acc, m_s, l_s, alpha_s,
                                p.k_scales, p.v_scales);
    const size_t slot = decode_unit(p, s, kvh) * p.max_splits + split;
#pragma unroll
    for (int it = 0; it < S::kItems; ++it) {
        const int idx = threadIdx.x + it * kFmaThreads;
        if (idx >= G * D) continue;
        const float l = l_s[idx / D], o = l == 0.f ? 0.f : acc[it] / l;
        if (nsplit == 1) static_cast<Bf16*>(p.out)[row + idx] = from_float<Bf16>(o);
        else p.ws_o[slot * G * D + idx] = o;
    }
    if (nsplit > 1 && threadIdx.x < G)
        p.ws_ml[slot * G + threadIdx.x] = make_float2(m_s[threadIdx.x], l_s[threadIdx.x]);
}

template <int D>
__global__ void __launch_bounds__(kFmaThreads) prefill_fp8_block_fma_kernel(PrefillParams p) {
    using S = FmaShape<D>;
    pdl_trigger();
    pdl_wait();
    const int i = blockIdx.x, c = blockIdx.y, kvh = blockIdx.z, G = p.group;
    const int r0 = p.cu_q_lens[c], n = p.cu_q_lens[c + 1] - r0, s = p.seq_of_chunk[c], start = p.q_start_pos[c];
    if (n < 0 || r0 < 0 || r0 + n > p.total_q || n > p.max_q_len || s < 0 || s >= p.num_seqs || start < 0) {
        if (i == 0 && kvh == 0 && threadIdx.x == 0) count_error(p.error_count);
        return;
    }
    if (i >= n) return;
    const int cap = (int)min(min((long long)p.context_lens[s], (long long)p.max_context_len),
                             (long long)p.max_blocks_per_seq * p.block_size);
    if ((long long)start + i + 1 > cap && threadIdx.x == 0 && kvh == 0) count_error(p.error_count);
    const int L = (int)min((long long)start + i + 1, (long long)cap);  // causal: keys 0..start+i
    extern __shared__ float smem[];
    __shared__ float m_s[kFmaMaxGroup], l_s[kFmaMaxGroup], alpha_s[kFmaMaxGroup];
    float acc[S::kItems];
    const size_t row = ((size_t)(r0 + i) * p.num_q_heads + (size_t)kvh * G) * D;
    fma_attend<Bf16, D, e4m3_t>(static_cast<const Bf16*>(p.q) + row, G, static_cast<const e4m3_t*>(p.k_cache),
                                static_cast<const e4m3_t*>(p.v_cache),
                                p.block_tables + (size_t)s * p.max_blocks_per_seq, p.block_size, p.num_kv_heads, kvh,
                                p.num_blocks, 0, L, p.scale_log2, p.error_count, smem, acc, m_s, l_s, alpha_s,
                                p.k_scales, p.v_scales);
#pragma unroll
    for (int it = 0; it < S::kItems; ++it) {
        const int idx = threadIdx.x + it * kFmaThreads;
        if (idx >= G * D) continue;
        const float l = l_s[idx / D];
        static_cast<Bf16*>(p.out)[row + idx] = from_float<Bf16>(l == 0.f ? 0.f : acc[it] / l);
    }
}

template <int D>
int decode(const DecodeParams& p, cudaStream_t stream) {
    const size_t smem = FmaShape<D>::kSmemBytes;
    const int rc = ensure_dynamic_smem(reinterpret_cast<const void*>(decode_fp8_block_fma_kernel<D>), smem);
    if (rc != PA_OK) return rc;
    return launch_kernel(decode_fp8_block_fma_kernel<D>, dim3(p.num_seqs, p.num_kv_heads, p.max_splits),
                         dim3(kFmaThreads), smem, stream, p);
}

template <int D>
int prefill(const PrefillParams& p, cudaStream_t stream) {
    const size_t smem = FmaShape<D>::kSmemBytes;
    const int rc = ensure_dynamic_smem(reinterpret_cast<const void*>(prefill_fp8_block_fma_kernel<D>), smem);
    if (rc != PA_OK) return rc;
    return launch_kernel(prefill_fp8_block_fma_kernel<D>, dim3(p.max_q_len, p.num_chunks, p.num_kv_heads),
                         dim3(kFmaThreads), smem, stream, p);
}

}  // namespace

int launch_decode_fp8_block_fma(const DecodeParams& p, cudaStream_t stream) {
    if (p.group > kFmaMaxGroup || p.num_kv_heads > 65535 || p.max_splits > 128) return PA_ERR_UNSUPPORTED;
    return p.head_dim == 64 ? decode<64>(p, stream) : decode<128>(p, stream);
}

int launch_prefill_fp8_block_fma(const PrefillParams& p, cudaStream_t stream) {
    if (p.group > kFmaMaxGroup || p.num_chunks > 65535 || p.num_kv_heads > 65535) return PA_ERR_UNSUPPORTED;
    return p.head_dim == 64 ? prefill<64>(p, stream) : prefill<128>(p, stream);
}

}  // namespace pa
