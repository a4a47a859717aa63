// prefill_weights_fma.cu — pa_prefill_chunk_weights on the CUDA cores: fp32
// pools, and the shapes that the tensor-core kernels do not take; and the
// addition of the keys' partial sums, for both.
//
// A key's weight needs the final softmax sum of every row that sees it, so
// there are two passes over Q K^T.  attend_kernel: a tile of 64 query rows
// (positions times the G heads of a kv head) against tiles of 64 keys, with an
// online softmax; it leaves the output and each row's lse = m + log2(l).
// Few tiles share their keys' tiles out to several CTAs (spans), whose rows another launch joins.
// column_kernel: a tile of 64 keys against the row tiles that see it, summing
// 2^(x - lse) down the rows in registers.  Both hold their tiles in shared
// memory in 32 bits and compute 4 x 4 scores a thread.  Under the profiler, four 512-query fp32
// chunks, the attention and the columns issue in 67 and 59% of the cycles, with shared memory's
// pipe at 55 and 45% and the FMA pipe at 49 and 43%: two CTAs an SM (registers and shared memory)
// do not hide the latency of the reads between them.  Four 512-query fp32 chunks at 26 to 587, 32/8 heads: 0.99 ms (1.34
// with a tile's loads one after the other, a check of each row against each key of V and the
// probabilities read one by one; with 8 x 4 scores a thread 1.11, but three 100-query bf16
// chunks of head_dim 64 45 us instead of 33: half as many warps); two 60-query fp32 chunks
// over 238 and 522 keys, 8/2 heads, 49 us (196 without the spans).
#include <type_traits>

#include "prefill_weights.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 64;

template <int D>
struct Shape {
    static constexpr int kPad = D + 4;  // floats in a staged row: 16-byte accesses of 8 rows touch all banks
    static constexpr int kPRow = kTile + 4;  // 16-byte aligned
    static constexpr size_t kSmem = sizeof(float) * (2 * kTile * kPad + kTile * kPRow);
};

// 4 elements as they lie in memory, and as floats.
template <typename T> struct Four;
template <> struct Four<float> { using type = float4; };
template <> struct Four<__nv_bfloat16> { using type = uint2; };
__device__ __forceinline__ float4 widen(float4 v) { return v; }
__device__ __forceinline__ float4 widen(uint2 v) {
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                       __uint_as_float(v.y & 0xFFFF0000u));
}

// kTile rows into shared memory; row_of(r) gives the row's first element or nullptr (zeros).  A thread's loads are all on
// their way before the first of them is stored.
template <typename T, int D, typename F>
__device__ __forceinline__ void stage(float* dst, F row_of) {
    using V = typename Four<T>::type;
    constexpr int kPieces = D / 4, kEach = kTile * kPieces / kThreads;
    V v[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const int i = threadIdx.x + k * kThreads, r = i / kPieces, c = i - r * kPieces;
        const T* src = row_of(r);
        v[k] = src ? *reinterpret_cast<const V*>(src + 4 * c) : V{};
    }
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const int i = threadIdx.x + k * kThreads, r = i / kPieces, c = i - r * kPieces;
        *reinterpret_cast<float4*>(dst + r * Shape<D>::kPad + 4 * c) = widen(v[k]);
    }
}

// acc[i][j] = a row (ty + 16 i) . b row (tx + 16 j)
template <int D>
__device__ __forceinline__ void scores(const float* a, const float* b, int ty, int tx, float (&acc)[4][4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll 8
    for (int d = 0; d < D; d += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(a + (ty + 16 * i) * Shape<D>::kPad + d);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(b + (tx + 16 * j) * Shape<D>::kPad + d);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[i][j] = fmaf(x[i].x, y[j].x, fmaf(x[i].y, y[j].y, fmaf(x[i].z, y[j].z, fmaf(x[i].w, y[j].w, acc[i][j]))));
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) attend_kernel(const PrefillParams p) {
    constexpr int kPad = Shape<D>::kPad, kPRow = Shape<D>::kPRow, kCols = D / 64;  // float4 columns a thread holds of each output row
    extern __shared__ float smem[];
    float *qs = smem, *ks = smem + kTile * kPad, *ps = ks + kTile * kPad;  // ps: [kTile][kPRow]
    __shared__ int block_s[kTile];
    pdl_trigger();
    pdl_wait();
    // a tile's keys are cut into spans where there are few tiles
    const int c = blockIdx.y, kvh = blockIdx.z / p.spans, span = blockIdx.z - kvh * p.spans, G = p.group, B = p.block_size;
    WeightChunk d;
    if (!weight_chunk(p, c, d)) {
        if (blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0) count_error(p.error_count);
        return;
    }
    const int per_tile = kTile / G, i0 = blockIdx.x * per_tile;
    if (i0 >= d.n) return;
    const int nq = min(per_tile, d.n - i0);
    const int want = d.start + i0 + nq, nkeys = max(0, min(want, d.cap));  // keys [0, nkeys) for the tile's last row
    if (want > d.cap && blockIdx.z == 0 && threadIdx.x == 0) count_error(p.error_count);
    const int span_keys = ((nkeys + kTile - 1) / kTile + p.spans - 1) / p.spans * kTile;
    const int key0 = (int)min((long long)nkeys, (long long)span * span_keys);
    const int key1 = (int)min((long long)nkeys, (long long)key0 + span_keys);
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    const int32_t* table = p.block_tables + (size_t)d.s * p.max_blocks_per_seq;
    const T* q = static_cast<const T*>(p.q) + ((size_t)(d.r0 + i0) * p.num_q_heads + (size_t)kvh * G) * D;
    stage<T, D>(qs, [&](int r) { return r < nq * G ? q + ((size_t)(r / G) * p.num_q_heads + r % G) * D : nullptr; });

    float m[4], l[4], o[4][kCols][4];
    int limit[4];  // keys that the row sees
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty + 16 * i;
        m[i] = -INFINITY;
        l[i] = 0.f;
        limit[i] = r < nq * G ? min(d.start + i0 + r / G + 1, d.cap) : 0;
#pragma unroll
        for (int k = 0; k < kCols; ++k) o[i][k][0] = o[i][k][1] = o[i][k][2] = o[i][k][3] = 0.f;
    }
    for (int j0 = key0; j0 < key1; j0 += kTile) {
        __syncthreads();
        if ((int)threadIdx.x < kTile) {
            const int j = j0 + threadIdx.x;
            int pb = -1;
            if (j < key1) {
                pb = table[j / B];
                if (pb < 0 || pb >= p.num_blocks) {
                    if (i0 + nq == d.n && (j % B == 0 || threadIdx.x == 0)) count_error(p.error_count);
                    pb = -1;
                }
            }
            block_s[threadIdx.x] = pb;
        }
        __syncthreads();
        auto row_of = [&](const void* pool) {
            return [&, pool](int r) {
                const int pb = block_s[r];
                return pb < 0 ? nullptr
                              : static_cast<const T*>(pool) + (((size_t)pb * B + (j0 + r) % B) * p.num_kv_heads + kvh) * D;
            };
        };
        stage<T, D>(ks, row_of(p.k_cache));
        __syncthreads();
        float x[4][4];
        scores<D>(qs, ks, ty, tx, x);
        float alpha[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = tx + 16 * j;
                x[i][j] = j0 + k < limit[i] && block_s[k] >= 0 ? x[i][j] * p.scale_log2 : -INFINITY;
                mx = fmaxf(mx, x[i][j]);
            }
#pragma unroll
            for (int off = 1; off < 16; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            const float now = fmaxf(m[i], mx);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // (all scores -inf: nothing; NaN scores leave the maximum and make the sum NaN)
                const float e = x[i][j] == -INFINITY ? 0.f : exp2f(x[i][j] - now);
                ps[(ty + 16 * i) * kPRow + tx + 16 * j] = e;
                sum += e;
            }
#pragma unroll
            for (int off = 1; off < 16; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            alpha[i] = m[i] == -INFINITY ? (l[i] == 0.f ? 0.f : 1.f) : exp2f(m[i] - now);
            l[i] = l[i] * alpha[i] + sum;
            m[i] = now;
        }
        __syncthreads();
        stage<T, D>(ks, row_of(p.v_cache));
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < kCols; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][k][e] *= alpha[i];
        auto add_values = [&](auto all_see) {
#pragma unroll 2
        for (int j = 0; j < kTile; j += 4) {
            float4 w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(ps + (ty + 16 * i) * kPRow + j);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float4 v[kCols];
#pragma unroll
                for (int k = 0; k < kCols; ++k) v[k] = *reinterpret_cast<const float4*>(ks + (j + e) * kPad + 64 * k + 4 * tx);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float f = e == 0 ? w[i].x : e == 1 ? w[i].y : e == 2 ? w[i].z : w[i].w;
                    // a row does not see the keys behind it, whatever they hold
                    if (!all_see && j0 + j + e >= limit[i]) continue;
#pragma unroll
                    for (int k = 0; k < kCols; ++k) {
                        o[i][k][0] = fmaf(f, v[k].x, o[i][k][0]);
                        o[i][k][1] = fmaf(f, v[k].y, o[i][k][1]);
                        o[i][k][2] = fmaf(f, v[k].z, o[i][k][2]);
                        o[i][k][3] = fmaf(f, v[k].w, o[i][k][3]);
                    }
                }
            }
        }
        };
        // (rows behind the tile's last one are not stored)
        if (j0 + kTile <= min(d.start + i0 + 1, d.cap)) add_values(std::true_type{});
        else add_values(std::false_type{});
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty + 16 * i;
        if (r >= nq * G) continue;
        const size_t row = (size_t)(d.r0 + i0) * G + r;
        const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
        if (p.spans > 1) {
            const size_t at = ((size_t)span * p.num_kv_heads + kvh) * p.total_q * G + row;
            if (tx == 0) p.part_ml[at] = make_float2(m[i], l[i]);
#pragma unroll
            for (int k = 0; k < kCols; ++k)
                *reinterpret_cast<float4*>(p.part_o + at * D + 64 * k + 4 * tx) =
                    make_float4(o[i][k][0] * inv, o[i][k][1] * inv, o[i][k][2] * inv, o[i][k][3] * inv);
            continue;
        }
        if (tx == 0) p.lse[(size_t)kvh * p.total_q * G + row] = l[i] == 0.f ? INFINITY : m[i] + log2f(l[i]);
        T* out = static_cast<T*>(p.out) + ((size_t)(d.r0 + i0 + r / G) * p.num_q_heads + (size_t)kvh * G + r % G) * D;
#pragma unroll
        for (int k = 0; k < kCols; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) out[64 * k + 4 * tx + e] = from_float<T>(o[i][k][e] * inv);
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) column_kernel(const PrefillParams p) {
    constexpr int kPad = Shape<D>::kPad;
    extern __shared__ float smem[];
    float *ks = smem, *qs = smem + kTile * kPad, *sums = qs + kTile * kPad;  // sums: [16][kTile]
    __shared__ float lse_s[kTile];
    pdl_trigger();
    pdl_wait();
    const int c = blockIdx.y, kvh = blockIdx.z, G = p.group, B = p.block_size;
    const int j0 = blockIdx.x * kTile;
    WeightChunk d;
    if (!weight_chunk(p, c, d) || j0 >= d.nkeys) return;
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    const int32_t* table = p.block_tables + (size_t)d.s * p.max_blocks_per_seq;
    auto block_of = [&](int r) {
        const int j = j0 + r;
        if (j >= d.nkeys) return -1;
        const int pb = table[j / B];
        return pb >= 0 && pb < p.num_blocks ? pb : -1;
    };
    stage<T, D>(ks, [&](int r) {
        const int pb = block_of(r);
        return pb < 0 ? nullptr
                      : static_cast<const T*>(p.k_cache) + (((size_t)pb * B + (j0 + r) % B) * p.num_kv_heads + kvh) * D;
    });
    const int per_tile = kTile / G;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    bool valid[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) valid[j] = block_of(tx + 16 * j) >= 0;
    // the first tile of rows that sees a key of this tile
    for (int i0 = max(0, j0 - d.start) / per_tile * per_tile; i0 < d.n; i0 += per_tile) {
        const int nq = min(per_tile, d.n - i0);
        const T* q = static_cast<const T*>(p.q) + ((size_t)(d.r0 + i0) * p.num_q_heads + (size_t)kvh * G) * D;
        __syncthreads();
        stage<T, D>(qs, [&](int r) { return r < nq * G ? q + ((size_t)(r / G) * p.num_q_heads + r % G) * D : nullptr; });
        if ((int)threadIdx.x < kTile)
            lse_s[threadIdx.x] = (int)threadIdx.x < nq * G
                                     ? p.lse[(size_t)kvh * p.total_q * G + (size_t)(d.r0 + i0) * G + threadIdx.x]
                                     : INFINITY;
        __syncthreads();
        float x[4][4];
        scores<D>(qs, ks, ty, tx, x);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty + 16 * i, limit = min(d.start + i0 + r / G + 1, d.cap);
            if (r >= nq * G) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (valid[j] && j0 + tx + 16 * j < limit) sum[j] += exp2f(x[i][j] * p.scale_log2 - lse_s[r]);
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) sums[ty * kTile + tx + 16 * j] = sum[j];
    __syncthreads();
    if ((int)threadIdx.x < kTile && j0 + (int)threadIdx.x < d.nkeys) {
        float total = 0.f;
        for (int i = 0; i < 16; ++i) total += sums[i * kTile + threadIdx.x];
        p.partial[((size_t)c * p.num_kv_heads + kvh) * p.max_context_len + j0 + threadIdx.x] = total;
    }
}

template <typename T, int D>
int launch(const PrefillParams& p, cudaStream_t stream) {
    int rc = ensure_dynamic_smem(reinterpret_cast<const void*>(attend_kernel<T, D>), Shape<D>::kSmem);
    if (rc == PA_OK) rc = ensure_dynamic_smem(reinterpret_cast<const void*>(column_kernel<T, D>), Shape<D>::kSmem);
    if (rc != PA_OK) return rc;
    const int per_tile = kTile / p.group;
    rc = launch_kernel(attend_kernel<T, D>,
                       dim3((p.max_q_len + per_tile - 1) / per_tile, p.num_chunks, p.num_kv_heads * p.spans), dim3(kThreads),
                       Shape<D>::kSmem, stream, p);
    if (rc == PA_OK && p.spans > 1) rc = launch_prefill_spans_join(p, sizeof(T) == 4 ? PA_F32 : PA_BF16, stream);
    if (rc != PA_OK || p.max_context_len == 0) return rc;
    return launch_kernel(column_kernel<T, D>, dim3((p.max_context_len + kTile - 1) / kTile, p.num_chunks, p.num_kv_heads),
                         dim3(kThreads), Shape<D>::kSmem, stream, p);
}

// The spans' partial rows joined, and their lse: a warp a (query, head).  Row = chunk row, the heads of a row together.
template <typename T, int D>
__global__ void __launch_bounds__(256) spans_join_kernel(const PrefillParams p) {
    pdl_trigger();
    pdl_wait();
    WeightChunk d;
    if (!weight_chunk(p, blockIdx.y, d)) return;
    const int G = p.group, Hq = p.num_q_heads, lane = threadIdx.x & 31;
    const long long rows = (long long)d.n * Hq, row0 = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row0 >= rows) return;
    const int i = (int)(row0 / Hq), h = (int)(row0 - (long long)i * Hq), kvh = h / G;
    const size_t stride = (size_t)p.num_kv_heads * p.total_q * G;
    const size_t row = ((size_t)kvh * p.total_q + d.r0 + i) * G + (h - kvh * G);
    float2 v[kMaxSpans / 32];
    float m = -INFINITY;
#pragma unroll
    for (int k = 0; k < kMaxSpans / 32; ++k) {
        const int e = lane + 32 * k;
        v[k] = e < p.spans ? __ldcg(p.part_ml + e * stride + row) : make_float2(-INFINITY, 0.f);
        if (v[k].y != 0.f) m = fmaxf(m, v[k].x);
    }
    m = warp_max(m);
    float w[kMaxSpans / 32], sum = 0.f;
#pragma unroll
    for (int k = 0; k < kMaxSpans / 32; ++k) {
        w[k] = v[k].y != 0.f ? v[k].y * exp2f(v[k].x - m) : 0.f;  // (a NaN counts)
        sum += w[k];
    }
    sum = warp_sum(sum);
    if (lane == 0) p.lse[row] = sum == 0.f ? INFINITY : m + log2f(sum);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    constexpr int kPairs = D / 64, kAhead = 8;  // pairs of columns a lane has, 64 columns apart
    const float2* o = reinterpret_cast<const float2*>(p.part_o + row * D) + lane;
    float2 acc[kPairs];
#pragma unroll
    for (int c = 0; c < kPairs; ++c) acc[c] = make_float2(0.f, 0.f);
    for (int e0 = 0; e0 < p.spans; e0 += kAhead) {
        float2 x[kAhead][kPairs];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
#pragma unroll
            for (int c = 0; c < kPairs; ++c)
                if (e0 + k < p.spans) x[k][c] = __ldcg(o + (e0 + k) * stride * (D / 2) + 32 * c);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int e = e0 + k;
            const float f = __shfl_sync(0xffffffffu, e < 32 ? w[0] : w[1], e & 31) * inv;
            if (e < p.spans)
#pragma unroll
                for (int c = 0; c < kPairs; ++c) {
                    acc[c].x = fmaf(f, x[k][c].x, acc[c].x);
                    acc[c].y = fmaf(f, x[k][c].y, acc[c].y);
                }
        }
    }
    T* out = static_cast<T*>(p.out) + ((size_t)(d.r0 + i) * Hq + h) * D + 2 * lane;
#pragma unroll
    for (int c = 0; c < kPairs; ++c) {
        out[64 * c] = from_float<T>(acc[c].x);
        out[64 * c + 1] = from_float<T>(acc[c].y);
    }
}

template <typename T, int D>
int launch_join(const PrefillParams& p, cudaStream_t stream) {
    const long long rows = (long long)p.max_q_len * p.num_q_heads;
    return launch_kernel(spans_join_kernel<T, D>, dim3((unsigned)((rows + 7) / 8), p.num_chunks), dim3(256), 0, stream, p);
}

// The chunks' partial sums added to their sequences' weights.  The first usable chunk of a sequence adds those of all its
// chunks, in the order of the chunks and of the pieces: one owner for each element, and one order.
constexpr int kAddThreads = 256;
__global__ void __launch_bounds__(kAddThreads) add_kernel(const PrefillParams p) {
    pdl_trigger();
    pdl_wait();
    const int c = blockIdx.y, kvh = blockIdx.z, j = blockIdx.x * kAddThreads + threadIdx.x;
    WeightChunk d;
    if (!weight_chunk(p, c, d)) return;
    bool mine = true;
    for (int e = threadIdx.x; e < c && mine; e += kAddThreads) {
        WeightChunk o;
        if (p.seq_of_chunk[e] == d.s && weight_chunk(p, e, o)) mine = false;
    }
    if (!__syncthreads_and(mine)) return;
    float sum = 0.f;
    bool any = false;
    __shared__ int later[kAddThreads];
    for (int e0 = c; e0 < p.num_chunks; e0 += kAddThreads) {  // this sequence's chunks among the next kAddThreads
        __syncthreads();
        const int e = e0 + threadIdx.x;
        const bool same = e < p.num_chunks && p.seq_of_chunk[e] == d.s;
        later[threadIdx.x] = same;
        if (!__syncthreads_or(same)) continue;
        for (int k = 0; k < kAddThreads && e0 + k < p.num_chunks; ++k) {
            WeightChunk o;
            if (!later[k] || !weight_chunk(p, e0 + k, o) || j >= o.nkeys) continue;
            any = true;
            if (!p.runs) {
                sum += p.partial[((size_t)(e0 + k) * p.num_kv_heads + kvh) * p.max_context_len + j];
                continue;
            }
            // the run of key j's pair: its units, and the CTAs that took them
            const int per_tile = 128 / p.group, pair = j / kKeys;
            const unsigned long long per = p.runs[p.num_chunks].units;
            const KeyRuns at = p.runs[e0 + k];
            const unsigned long long first =
                at.units + (unsigned long long)kvh * key_units(o, per_tile) + key_units(o, per_tile, pair);
            const unsigned long long last =
                first + key_tiles(o, per_tile) - key_first_tile(o, pair, per_tile) - 1;
            const int run = at.runs + kvh * key_pairs(o) + pair;
            for (unsigned long long b = first / per; b <= last / per; ++b)
                for (int h = 0; h < kKeyParts; ++h)
                    sum += p.partial[((size_t)(run + b) * kKeyParts + h) * kKeys + j % kKeys];
        }
    }
    if (any) p.key_weights[((size_t)d.s * p.num_kv_heads + kvh) * p.key_width + j] += sum;
}

}  // namespace

int launch_prefill_weights_fma(const PrefillParams& p, int dtype, cudaStream_t stream) {
    if (p.group > 16 || p.num_chunks > 65535 || (long long)p.num_kv_heads * p.spans > 65535) return PA_ERR_UNSUPPORTED;
    if (((uintptr_t)p.q & 15) || ((uintptr_t)p.k_cache & 15) || ((uintptr_t)p.v_cache & 15)) return PA_ERR_UNSUPPORTED;
    if (dtype == PA_F32) return p.head_dim == 64 ? launch<float, 64>(p, stream) : launch<float, 128>(p, stream);
    return p.head_dim == 64 ? launch<__nv_bfloat16, 64>(p, stream) : launch<__nv_bfloat16, 128>(p, stream);
}

int launch_prefill_spans_join(const PrefillParams& p, int dtype, cudaStream_t stream) {
    if (dtype == PA_F32) return p.head_dim == 64 ? launch_join<float, 64>(p, stream) : launch_join<float, 128>(p, stream);
    return p.head_dim == 64 ? launch_join<__nv_bfloat16, 64>(p, stream) : launch_join<__nv_bfloat16, 128>(p, stream);
}

int launch_prefill_weights_add(const PrefillParams& p, cudaStream_t stream) {
    if (p.max_context_len == 0) return PA_OK;
    return launch_kernel(add_kernel, dim3((p.max_context_len + kAddThreads - 1) / kAddThreads, p.num_chunks, p.num_kv_heads),
                         dim3(kAddThreads), 0, stream, p);
}

}  // namespace pa
