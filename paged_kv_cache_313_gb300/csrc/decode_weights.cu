// decode_weights.cu — the second launch of pa_decode_weights: the split-KV
// combine, and the softmax weight of every key added to its accumulated weight.
//
// The decode kernel (decode_tc.cu, decode_weights_fma.cu) has left each score x (base-2
// units, -inf for a masked token) and each partition's (m, l) in the workspace.
// With lse_g = m* + log2(sum_i l_i 2^(m_i - m*)) over a head's partitions,
//     key_weights[s][kv head][j] += sum over the group's heads g of 2^(x_jg - lse_g)
// and, where a context has several partitions, out = sum_i 2^(m_i - lse) l_i o_i.
//
// A CTA takes kTokens tokens of one (sequence, kv head), and one more CTA the
// partial outputs.  What a CTA reads (scores, weights, the partitions' states) is
// loaded all at once, before the first of it is used: bound by the latency of the
// scores, which lie in L2.  An element of key_weights has one owner: no atomics, and
// the sums' order is fixed.
//
// 64 sequences (60,000 tokens, 32/8 heads): 52.4 us with the decode kernel, 46.6 without
// the scores and this launch; 16 contexts of 1k to 32k (190,000 tokens, 64/8 heads): 155 us,
// 126 without (48 MB of scores written and read).  Loading scores as they are used took
// 60.1 and 170; 2048 tokens a CTA 165, 512 tokens 160; persistent CTAs that pass over the
// items of shorter contexts 168 to 233 (two to six an SM; their registers spilled).
#include "decode_common.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 1024;
constexpr int kEach = kTokens / kThreads;
constexpr int kMaxGroup = 16, kMaxSplits = 128;

// G consecutive scores.
template <int G>
__device__ __forceinline__ void load_scores(const float* x, float (&v)[G]) {
    if constexpr (G % 4 == 0) {
#pragma unroll
        for (int g = 0; g < G; g += 4) {
            const float4 t = __ldcg(reinterpret_cast<const float4*>(x + g));
            v[g] = t.x;
            v[g + 1] = t.y;
            v[g + 2] = t.z;
            v[g + 3] = t.w;
        }
    } else if constexpr (G == 2) {
        const float2 t = __ldcg(reinterpret_cast<const float2*>(x));
        v[0] = t.x;
        v[1] = t.y;
    } else {
#pragma unroll
        for (int g = 0; g < G; ++g) v[g] = __ldcg(x + g);
    }
}

// kG: the group's heads, 0 for a number without an instance of its own.
template <typename T, int D, int kG>
__global__ void __launch_bounds__(kThreads, 4) decode_weights_kernel(const DecodeParams p) {
    __shared__ float lse_s[kMaxGroup];
    __shared__ float share[kMaxSplits][kMaxGroup];  // a partition's part of the output
    pdl_trigger();
    pdl_wait();
    const int unit = blockIdx.x, s = unit / p.num_kv_heads, kvh = unit - s * p.num_kv_heads;
    const int G = kG ? kG : p.group, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int L = decode_context(p, s, false);
    const int nsplit = num_partitions(L, partition_of(p, s));
    const bool merge = blockIdx.y == 0;  // the CTA of the partial outputs
    const int first = ((int)blockIdx.y - 1) * kTokens;
    if (merge ? nsplit <= 1 : first >= L) return;
    const float* scores = p.ws_scores + (size_t)unit * p.score_width * G;
    float* weights = p.key_weights + (size_t)unit * p.key_width;
    float x[kEach][kG ? kG : 1], w[kEach];
    if (!merge) {
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int j = first + e * kThreads + threadIdx.x;
            if (j >= L) continue;
            w[e] = weights[j];
            if constexpr (kG != 0) load_scores<kG>(scores + (size_t)j * kG, x[e]);
        }
    }
    const float2* ml = p.ws_ml + (size_t)unit * p.max_splits * G;
    bool nan = false;
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
        nan |= isnan(lse);
        if (lane == 0) lse_s[g] = lse;
        if (merge)
#pragma unroll
            for (int k = 0; k < kMaxSplits / 32; ++k)
                if (lane + 32 * k < nsplit)
                    share[lane + 32 * k][g] = v[k].y == 0.f ? 0.f : v[k].y * exp2f(v[k].x - m) / sum;
    }
    nan = __syncthreads_or(nan);
    if (merge) {
        constexpr int kAhead = 8;
        const float4* o = reinterpret_cast<const float4*>(p.ws_o + (size_t)unit * p.max_splits * G * D);
        for (int i = threadIdx.x; i < G * (D / 4); i += kThreads) {
            const int g = i / (D / 4);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k0 = 0; k0 < nsplit; k0 += kAhead) {
                float4 y[kAhead];
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
                    if (k0 + k < nsplit) y[k] = __ldcg(o + (size_t)(k0 + k) * G * (D / 4) + i);
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
                    if (k0 + k < nsplit) {
                        const float f = share[k0 + k][g];
                        acc.x = fmaf(f, y[k].x, acc.x);
                        acc.y = fmaf(f, y[k].y, acc.y);
                        acc.z = fmaf(f, y[k].z, acc.z);
                        acc.w = fmaf(f, y[k].w, acc.w);
                    }
            }
            T* out = static_cast<T*>(p.out) + ((size_t)s * p.num_q_heads + (size_t)kvh * G) * D + 4 * i;
            out[0] = from_float<T>(acc.x);
            out[1] = from_float<T>(acc.y);
            out[2] = from_float<T>(acc.z);
            out[3] = from_float<T>(acc.w);
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        const int j = first + e * kThreads + threadIdx.x;
        if (j >= L) continue;
        float sum = 0.f;
        bool masked = true;  // -inf for every head
        if constexpr (kG != 0) {
#pragma unroll
            for (int g = 0; g < kG; ++g) sum += exp2f(x[e][g] - lse_s[g]);
            if (nan)
#pragma unroll
                for (int g = 0; g < kG; ++g) masked = masked && x[e][g] == -INFINITY;
        } else {
            for (int g = 0; g < G; ++g) {
                const float y = __ldcg(scores + (size_t)j * G + g);
                sum += exp2f(y - lse_s[g]);
                masked = masked && y == -INFINITY;
            }
        }
        // (-inf - NaN would reach masked tokens.  A look at each score, instead of where a sum is NaN: 156 -> 161 us for 16
        // long contexts.)
        if (nan && masked) sum = 0.f;
        weights[j] = w[e] + sum;
    }
}

template <typename T, int D>
int launch(const DecodeParams& p, dim3 grid, cudaStream_t stream) {
    const dim3 block(kThreads);
    switch (p.group) {
        case 1: return launch_kernel(decode_weights_kernel<T, D, 1>, grid, block, 0, stream, p);
        case 2: return launch_kernel(decode_weights_kernel<T, D, 2>, grid, block, 0, stream, p);
        case 4: return launch_kernel(decode_weights_kernel<T, D, 4>, grid, block, 0, stream, p);
        case 8: return launch_kernel(decode_weights_kernel<T, D, 8>, grid, block, 0, stream, p);
        default: return launch_kernel(decode_weights_kernel<T, D, 0>, grid, block, 0, stream, p);
    }
}

}  // namespace

int launch_decode_weights(const DecodeParams& p, int dtype, cudaStream_t stream) {
    if (p.group > kMaxGroup || p.max_splits > kMaxSplits) return PA_ERR_UNSUPPORTED;
    const int pieces = (p.max_context_len + kTokens - 1) / kTokens;
    const dim3 grid(p.num_seqs * p.num_kv_heads, 1 + pieces);
    if (dtype == PA_F32)
        return p.head_dim == 64 ? launch<float, 64>(p, grid, stream) : launch<float, 128>(p, grid, stream);
    return p.head_dim == 64 ? launch<__nv_bfloat16, 64>(p, grid, stream) : launch<__nv_bfloat16, 128>(p, grid, stream);
}

}  // namespace pa
