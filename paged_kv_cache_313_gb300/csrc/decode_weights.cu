// decode_weights.cu — the second launch of pa_decode_weights: the split-KV
// combine, and the softmax weight of every key added to its accumulated weight.
//
// The decode kernel (decode_tc.cu, decode_fma.cu) has left each score x (base-2
// units, -inf for a masked token) and each partition's (m, l) in the workspace.
// With lse_g = m* + log2(sum_i l_i 2^(m_i - m*)) over a head's partitions,
//     key_weights[s][kv head][j] += sum over the group's heads g of 2^(x_jg - lse_g)
// and, where a context has several partitions, out = sum_i 2^(m_i - lse) l_i o_i.
//
// A CTA takes kTokens tokens of one (sequence, kv head); the CTA of the first
// ones combines the partial outputs too.  An element of key_weights has one
// owner: no atomics, and the sums' order is fixed.
#include "decode_common.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 1024;
constexpr int kMaxGroup = 16, kMaxSplits = 128;

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) decode_weights_kernel(const DecodeParams p) {
    __shared__ float lse_s[kMaxGroup];
    __shared__ float share[kMaxSplits][kMaxGroup];  // a partition's part of the output
    pdl_trigger();
    pdl_wait();
    const int unit = blockIdx.x, s = unit / p.num_kv_heads, kvh = unit - s * p.num_kv_heads;
    const int G = p.group, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int L = decode_context(p, s, false);
    const int first = blockIdx.y * kTokens;
    if (first >= max(L, 1)) return;
    const int nsplit = num_partitions(L, partition_of(p, s));
    const bool merge = blockIdx.y == 0 && nsplit > 1;
    const float2* ml = p.ws_ml + (size_t)unit * p.max_splits * G;
    for (int g = warp; g < G; g += kThreads / 32) {
        float2 v[kMaxSplits / 32];
        float m = -INFINITY;
#pragma unroll
        for (int k = 0; k < kMaxSplits / 32; ++k) {
            const int i = lane + 32 * k;
            v[k] = i < nsplit ? __ldcg(ml + (size_t)i * G + g) : make_float2(-INFINITY, 0.f);
            if (v[k].y != 0.f) m = fmaxf(m, v[k].x);
        }
        m = warp_max(m);
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < kMaxSplits / 32; ++k)
            if (v[k].y != 0.f) sum += v[k].y * exp2f(v[k].x - m);  // (a NaN counts: it is not 0)
        sum = warp_sum(sum);
        const float lse = sum == 0.f ? INFINITY : m + log2f(sum);  // no key: every weight is 0
        if (lane == 0) lse_s[g] = lse;
        if (merge)
#pragma unroll
            for (int k = 0; k < kMaxSplits / 32; ++k)
                if (lane + 32 * k < nsplit)
                    share[lane + 32 * k][g] = v[k].y == 0.f ? 0.f : v[k].y * exp2f(v[k].x - m) / sum;
    }
    __syncthreads();
    if (merge) {
        constexpr int kAhead = 16;
        const float4* o = reinterpret_cast<const float4*>(p.ws_o + (size_t)unit * p.max_splits * G * D);
        for (int i = threadIdx.x; i < G * (D / 4); i += kThreads) {
            const int g = i / (D / 4);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k0 = 0; k0 < nsplit; k0 += kAhead) {
                float4 x[kAhead];
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
                    if (k0 + k < nsplit) x[k] = __ldcg(o + (size_t)(k0 + k) * G * (D / 4) + i);
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
                    if (k0 + k < nsplit) {
                        const float w = share[k0 + k][g];
                        acc.x = fmaf(w, x[k].x, acc.x);
                        acc.y = fmaf(w, x[k].y, acc.y);
                        acc.z = fmaf(w, x[k].z, acc.z);
                        acc.w = fmaf(w, x[k].w, acc.w);
                    }
            }
            T* out = static_cast<T*>(p.out) + ((size_t)s * p.num_q_heads + (size_t)kvh * G) * D + 4 * i;
            out[0] = from_float<T>(acc.x);
            out[1] = from_float<T>(acc.y);
            out[2] = from_float<T>(acc.z);
            out[3] = from_float<T>(acc.w);
        }
    }
    const float* scores = p.ws_scores + (size_t)unit * p.score_width * G;
    float* weights = p.key_weights + (size_t)unit * p.key_width;
    const int last = min(L, first + kTokens);
#pragma unroll 4
    for (int j = first + threadIdx.x; j < last; j += kThreads) {
        const float* x = scores + (size_t)j * G;
        float sum = 0.f;
        if ((G & 3) == 0) {
            for (int g = 0; g < G; g += 4) {
                const float4 v = __ldcg(reinterpret_cast<const float4*>(x + g));
                sum += (exp2f(v.x - lse_s[g]) + exp2f(v.y - lse_s[g + 1])) +
                       (exp2f(v.z - lse_s[g + 2]) + exp2f(v.w - lse_s[g + 3]));
            }
        } else {
            for (int g = 0; g < G; ++g) sum += exp2f(__ldcg(x + g) - lse_s[g]);
        }
        weights[j] += sum;
    }
}

}  // namespace

int launch_decode_weights(const DecodeParams& p, int dtype, cudaStream_t stream) {
    if (p.group > kMaxGroup || p.max_splits > kMaxSplits) return PA_ERR_UNSUPPORTED;
    const int pieces = p.max_context_len > kTokens ? (p.max_context_len + kTokens - 1) / kTokens : 1;
    if (pieces > 65535) return PA_ERR_UNSUPPORTED;
    const dim3 grid(p.num_seqs * p.num_kv_heads, pieces), block(kThreads);
    if (dtype == PA_F32)
        return p.head_dim == 64 ? launch_kernel(decode_weights_kernel<float, 64>, grid, block, 0, stream, p)
                                : launch_kernel(decode_weights_kernel<float, 128>, grid, block, 0, stream, p);
    return p.head_dim == 64 ? launch_kernel(decode_weights_kernel<__nv_bfloat16, 64>, grid, block, 0, stream, p)
                            : launch_kernel(decode_weights_kernel<__nv_bfloat16, 128>, grid, block, 0, stream, p);
}

}  // namespace pa
