// decode_weights_fma.cu — the attention of pa_decode_weights on the CUDA cores:
// fp32 pools, and the shapes that the tensor-core decode kernel does not take.
//
// One CTA per (sequence, kv head, partition of the context).  Tiles of 32 tokens
// come in through a ring of two (cp.async, 16 bytes a thread, rows of tokens without a
// valid block filled with zeros), so that a tile is on its way while one is worked on.  Scores: eight lanes a token, each on every eighth 16-byte piece of
// its row against all G query heads.  Softmax: a warp a head, a lane a token, online.
// P V: a thread four columns and a share of the tile's tokens, its share of the output
// in registers until the partition ends.  Scores go to the workspace and every
// partition's (m, l) too; decode_weights.cu does the rest.
//
// Bound by latency, not by memory: 64 fp32 sequences (12,500 tokens, 32/8 heads), 79 us under the
// profiler, have DRAM at 17% and issue in 45% of the cycles with 16 warps an SM, whose wait is for
// shared memory (2.1 cycles an instruction), instructions' own latency (2.0) and the blocks'
// look-ups (1.2).  With 16 bf16 heads a kv head one CTA fits an SM: issue in 27%, 3.5 cycles an
// instruction for shared memory.
//
// 64 fp32 sequences (18,000 tokens, 32/8 heads): 96 us, 1.5 TB/s = 0.22 of the copy bandwidth; four
// of 1 to 40 tokens 7.1 us with both launches.  The CUDA-core decode kernel with the scores added (a warp a token, 64-token
// pieces one after the other) took 498 and 19.0, and 1054 instead of 166 with 16 bf16 heads a kv
// head.
#include "decode_common.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kTile = 32;
constexpr int kLanes = 8;  // lanes that share a token's scores

// kG: query heads a kv head, rounded up to a power of two.
template <typename T, int D, int kG>
struct Shape {
    static constexpr int kVec = 16 / (int)sizeof(T);           // elements of a 16-byte piece
    static constexpr int kPieces = D / kVec;                   // pieces of a row
    static constexpr int kRow = D + kVec;                      // elements from one staged row to the next
    static constexpr int kColumns = D / 4, kShares = kThreads / kColumns, kPerShare = kTile / kShares;
    static constexpr size_t kTileBytes = (size_t)kTile * kRow * sizeof(T);
    static constexpr size_t kStage = 2 * kTileBytes;           // K and V
    static constexpr size_t kQ = 2 * kStage;                   // float [kG][D], scaled
    static constexpr size_t kP = kQ + sizeof(float) * kG * D;  // float [kG][kTile]
    static constexpr size_t kScale = kP + sizeof(float) * kG * kTile;  // float [kG]: the tile's rescale; then m, l
    static constexpr size_t kSmem = kScale + sizeof(float) * 3 * kG;
    // the shares' outputs are added in the tiles' place, as many heads at a time as fit there
    static constexpr int kFit = (int)(kQ / (sizeof(float) * kShares * D)), kHeads = kG < kFit ? kG : kFit;
    static_assert(kHeads >= 1, "room for a head's shares");
};

__device__ __forceinline__ void copy16(void* dst, const void* src, bool have) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src), "r"(have ? 16 : 0)
                 : "memory");
}

// 4 elements from shared memory as floats.
__device__ __forceinline__ float4 four(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 four(const __nv_bfloat16* p) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                       __uint_as_float(v.y & 0xFFFF0000u));
}

template <typename T, int D, int kG>
__global__ void __launch_bounds__(kThreads) decode_weights_fma_kernel(const DecodeParams p) {
    using S = Shape<T, D, kG>;
    extern __shared__ __align__(16) uint8_t smem[];
    pdl_trigger();
    pdl_wait();
    const int s = blockIdx.x, kvh = blockIdx.y, split = blockIdx.z, G = p.group, B = p.block_size, Hkv = p.num_kv_heads;
    const int L = decode_context(p, s, split == 0 && kvh == 0 && threadIdx.x == 0);
    const int nsplit = num_partitions(L, p.partition);
    if (split >= nsplit) return;
    const int j0 = split * p.partition, j1 = min(L, j0 + p.partition);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* q_s = reinterpret_cast<float*>(smem + S::kQ);
    float* p_s = reinterpret_cast<float*>(smem + S::kP);
    float* alpha_s = reinterpret_cast<float*>(smem + S::kScale);
    float *m_s = alpha_s + kG, *l_s = m_s + kG;
    const int32_t* table = p.block_tables + (size_t)s * p.max_blocks_per_seq;
    const T* kc = static_cast<const T*>(p.k_cache);
    const T* vc = static_cast<const T*>(p.v_cache);

    // tile t's rows; thread i copies pieces i, i + kThreads, ... of K and of V.  Errors are counted with the copies.
    auto load_tile = [&](int t) {
        uint8_t* dst = smem + (t & 1) * S::kStage;
        for (int i = threadIdx.x; i < kTile * S::kPieces; i += kThreads) {
            const int r = i / S::kPieces, c = i - r * S::kPieces, j = j0 + t * kTile + r;
            int pb = -1;
            if (j < j1) {
                pb = table[j / B];
                if (pb < 0 || pb >= p.num_blocks) {
                    if (c == 0 && (j % B == 0 || j == j0)) count_error(p.error_count);
                    pb = -1;
                }
            }
            const size_t at = pb >= 0 ? (((size_t)pb * B + j % B) * Hkv + kvh) * D + (size_t)c * S::kVec : 0;
            const size_t to = ((size_t)r * S::kRow + (size_t)c * S::kVec) * sizeof(T);
            copy16(dst + to, kc + at, pb >= 0);
            copy16(dst + S::kTileBytes + to, vc + at, pb >= 0);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const int tiles = (j1 - j0 + kTile - 1) / kTile;
    if (tiles > 0) load_tile(0);
    const T* q = static_cast<const T*>(p.q) + ((size_t)s * p.num_q_heads + (size_t)kvh * G) * D;
    for (int i = threadIdx.x; i < kG * D; i += kThreads) q_s[i] = i < G * D ? to_float(q[i]) : 0.f;
    if ((int)threadIdx.x < kG) {
        m_s[threadIdx.x] = -INFINITY;
        l_s[threadIdx.x] = 0.f;
    }
    // this thread's columns and tokens of P V
    const int column = threadIdx.x % S::kColumns * 4, share = threadIdx.x / S::kColumns;
    float acc[kG][4];
#pragma unroll
    for (int g = 0; g < kG; ++g) acc[g][0] = acc[g][1] = acc[g][2] = acc[g][3] = 0.f;
    float* scores = p.ws_scores + decode_unit(p, s, kvh) * p.score_width * G;
    for (int t = 0; t < tiles; ++t) {
        if (t + 1 < tiles) {
            load_tile(t + 1);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        __syncthreads();
        const T* ks = reinterpret_cast<const T*>(smem + (t & 1) * S::kStage);
        const T* vs = reinterpret_cast<const T*>(smem + (t & 1) * S::kStage + S::kTileBytes);
        {  // scores: token `r`, this lane's pieces `part`, part + 8, ...
            const int r = threadIdx.x / kLanes, part = threadIdx.x % kLanes, j = j0 + t * kTile + r;
            float dot[kG];
#pragma unroll
            for (int g = 0; g < kG; ++g) dot[g] = 0.f;
#pragma unroll
            for (int c = part; c < S::kPieces; c += kLanes) {
#pragma unroll
                for (int e = 0; e < S::kVec; e += 4) {
                    const float4 k = four(ks + r * S::kRow + c * S::kVec + e);
#pragma unroll
                    for (int g = 0; g < kG; ++g) {
                        const float4 x = four(q_s + g * D + c * S::kVec + e);
                        dot[g] = fmaf(x.x, k.x, fmaf(x.y, k.y, fmaf(x.z, k.z, fmaf(x.w, k.w, dot[g]))));
                    }
                }
            }
#pragma unroll
            for (int g = 0; g < kG; ++g)
#pragma unroll
                for (int off = 1; off < kLanes; off <<= 1) dot[g] += __shfl_xor_sync(0xffffffffu, dot[g], off);
            bool valid = false;
            if (j < j1) {
                const int pb = table[j / B];
                valid = pb >= 0 && pb < p.num_blocks;
            }
#pragma unroll
            for (int g = 0; g < kG; ++g)
                if (g % kLanes == part && g < G) {
                    const float x = valid ? dot[g] * p.scale_log2 : -INFINITY;
                    p_s[g * kTile + r] = x;
                    if (j < j1) scores[(size_t)j * G + g] = x;
                }
        }
        __syncthreads();
        for (int g = warp; g < G; g += kWarps) {  // softmax: lane = token
            const float x = p_s[g * kTile + lane], m_old = m_s[g];
            const float m = fmaxf(m_old, warp_max(x));
            // (all scores -inf: nothing; NaN scores leave the maximum and make the sum NaN)
            const float e = x == -INFINITY ? 0.f : exp2f(x - m);
            p_s[g * kTile + lane] = e;
            const float sum = warp_sum(e);
            if (lane == 0) {
                const float a = m_old == -INFINITY ? (l_s[g] == 0.f ? 0.f : 1.f) : exp2f(m_old - m);
                alpha_s[g] = a;
                l_s[g] = l_s[g] * a + sum;
                m_s[g] = m;
            }
        }
        __syncthreads();
        // (tokens at or beyond j1 have zero rows and zero weights)
        float4 v[S::kPerShare];
#pragma unroll
        for (int i = 0; i < S::kPerShare; ++i) v[i] = four(vs + (share * S::kPerShare + i) * S::kRow + column);
#pragma unroll
        for (int g = 0; g < kG; ++g) {
            if (g >= G) break;
            const float a = alpha_s[g];
            float o[4] = {acc[g][0] * a, acc[g][1] * a, acc[g][2] * a, acc[g][3] * a};
#pragma unroll
            for (int i = 0; i < S::kPerShare; ++i) {
                const float w = p_s[g * kTile + share * S::kPerShare + i];
                o[0] = fmaf(w, v[i].x, o[0]);
                o[1] = fmaf(w, v[i].y, o[1]);
                o[2] = fmaf(w, v[i].z, o[2]);
                o[3] = fmaf(w, v[i].w, o[3]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[g][e] = o[e];
        }
        __syncthreads();  // the tile's buffer and p_s go to the next tiles
    }
    // the shares' outputs, a few heads at a time, in the tiles' place
    constexpr int kHeads = S::kHeads;
    float* sums = reinterpret_cast<float*>(smem);  // [kShares][kHeads][D]
    const size_t part = decode_unit(p, s, kvh) * p.max_splits + split;
    for (int g0 = 0; g0 < G; g0 += kHeads) {
#pragma unroll
        for (int g = 0; g < kG; ++g)
            if (g >= g0 && g < g0 + kHeads && g < G)
                *reinterpret_cast<float4*>(sums + ((size_t)share * kHeads + (g - g0)) * D + column) =
                    make_float4(acc[g][0], acc[g][1], acc[g][2], acc[g][3]);
        __syncthreads();
        for (int i = threadIdx.x; i < min(kHeads, G - g0) * D; i += kThreads) {
            float o = 0.f;
#pragma unroll
            for (int k = 0; k < S::kShares; ++k) o += sums[(size_t)k * kHeads * D + i];
            const float l = l_s[g0 + i / D];
            o = l == 0.f ? 0.f : o / l;
            const size_t at = (size_t)g0 * D + i;
            if (nsplit == 1)
                static_cast<T*>(p.out)[((size_t)s * p.num_q_heads + (size_t)kvh * G) * D + at] = from_float<T>(o);
            else
                p.ws_o[part * G * D + at] = o;
        }
        __syncthreads();
    }
    if ((int)threadIdx.x < G) p.ws_ml[part * G + threadIdx.x] = make_float2(m_s[threadIdx.x], l_s[threadIdx.x]);
}

template <typename T, int D, int kG>
int launch_heads(const DecodeParams& p, cudaStream_t stream) {
    using S = Shape<T, D, kG>;
    const int rc = ensure_dynamic_smem(reinterpret_cast<const void*>(decode_weights_fma_kernel<T, D, kG>), S::kSmem);
    if (rc != PA_OK) return rc;
    return launch_kernel(decode_weights_fma_kernel<T, D, kG>, dim3(p.num_seqs, p.num_kv_heads, p.max_splits), dim3(kThreads),
                         S::kSmem, stream, p);
}

template <typename T, int D>
int launch(const DecodeParams& p, cudaStream_t stream) {
    if (p.group <= 1) return launch_heads<T, D, 1>(p, stream);
    if (p.group <= 2) return launch_heads<T, D, 2>(p, stream);
    if (p.group <= 4) return launch_heads<T, D, 4>(p, stream);
    if (p.group <= 8) return launch_heads<T, D, 8>(p, stream);
    return launch_heads<T, D, 16>(p, stream);
}

}  // namespace

int launch_decode_weights_fma(const DecodeParams& p, int dtype, cudaStream_t stream) {
    if (p.group > 16 || p.max_splits > 128 || p.num_kv_heads > 65535) return PA_ERR_UNSUPPORTED;
    if (((uintptr_t)p.k_cache & 15) || ((uintptr_t)p.v_cache & 15)) return PA_ERR_UNSUPPORTED;
    if (dtype == PA_F32) return p.head_dim == 64 ? launch<float, 64>(p, stream) : launch<float, 128>(p, stream);
    return p.head_dim == 64 ? launch<__nv_bfloat16, 64>(p, stream) : launch<__nv_bfloat16, 128>(p, stream);
}

}  // namespace pa
