// rope.cu — rotary positions with several axes on a step's queries and keys,
// alone (pa_rope) or with the paged write (pa_rope_write_kv_paged).
//
// Pair i of a head (elements i and R/2 + i, or 2i and 2i + 1 where pairs are
// interleaved) is the complex number a + ib; at position pos[axis[i]] it is
// multiplied by e^(i angle), angle = pos[axis[i]] * inv_freq[i].  Elements from
// R on stay as they are.
//
// The angle is wanted modulo a turn.  A float product loses that for far
// positions (10^5 rad is known to 2^-7 in 24 bits), and 64-bit floats are slow
// here, so it is counted in whole numbers: inv_freq = m 2^e with a 24-bit m, and
//     turns per position * 2^64 = m K 2^(e-2),  K = round(2^66 / (2 pi)),
// kept modulo 2^64; times the position, modulo 2^64, is the fraction of a turn,
// exact to 2^-32 for every 32-bit position.  Its upper half as a signed number
// is the angle in half turns for sincospi.
//
// Bound by memory: q, k and v are read once and written once.  One CTA per
// token: its first loads go out before the angles are worked out (once per
// token and pair, shared by all heads through shared memory).
#include "pa_internal.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 2;  // items whose loads a thread issues before the angles

template <typename T, int VEC> struct Chunk;  // VEC elements moved by one access
template <> struct Chunk<__nv_bfloat16, 8> { using type = uint4; };
template <> struct Chunk<float, 4> { using type = uint4; };
template <> struct Chunk<__nv_bfloat16, 1> { using type = uint16_t; };
template <> struct Chunk<float, 1> { using type = uint32_t; };

// inv_freq as turns per position, 2^-64 turns, modulo a turn (see above); *finite false for an infinity or NaN.
__device__ __forceinline__ uint64_t turns_of(float inv_freq, bool* finite) {
    constexpr uint64_t kInvTau = 0xA2F9836E4E44152Aull;  // 2^66 / (2 pi), rounded
    const uint32_t u = __float_as_uint(inv_freq), ex = (u >> 23) & 255u;
    *finite = ex != 255u;
    const uint64_t m = (u & 0x7FFFFFu) | (ex ? 0x800000u : 0u);
    const uint64_t lo = m * kInvTau, hi = __umul64hi(m, kInvTau);
    const int right = 2 - ((int)(ex ? ex : 1u) - 150);  // inv_freq = m 2^(ex - 150)
    uint64_t t;
    if (right <= 0) t = -right < 64 ? lo << -right : 0;
    else if (right < 64) t = (lo >> right) | (hi << (64 - right));
    else t = right < 128 ? hi >> (right - 64) : 0;
    return (u >> 31) ? 0 - t : t;
}

template <typename T, int VEC, bool kWrite>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p) {
    using C = typename Chunk<T, VEC>::type;
    extern __shared__ float2 turn[];  // cos and sin of each pair
    pdl_trigger();
    pdl_wait();
    const long long t = blockIdx.x;
    const int D = p.head_dim, half = p.rot_dim / 2;
    const int per_head = half / VEC + (D - p.rot_dim) / VEC;  // pair items, then pass-through items
    const int items = (p.num_q_heads + p.num_kv_heads) * per_head + (kWrite ? p.num_kv_heads * (D / VEC) : 0);

    // Item i of the token: a chunk and, where it is turned, its partner's chunk, `b` chunks further on (0: copied); the first
    // of its pairs; its element's offset within a row of q (row 0), k (1) or v (2).
    struct Item {
        int row, offset, b, pair;
    };
    auto item_of = [&](int i) {
        Item it{};
        const int rotated = (p.num_q_heads + p.num_kv_heads) * per_head;
        if (kWrite && i >= rotated) {
            it.row = 2;
            it.offset = (i - rotated) * VEC;
        } else {
            const int h = p.by_head.div(i), c = i - h * per_head;
            it.row = h >= p.num_q_heads;
            it.offset = (h - (it.row ? p.num_q_heads : 0)) * D;
            if (c < half / VEC) {
                it.offset += p.interleaved ? 2 * c * VEC : c * VEC;
                it.b = p.interleaved ? 1 : half / VEC;
                it.pair = c * VEC;
            } else {
                it.offset += p.rot_dim + (c - half / VEC) * VEC;
            }
        }
        return it;
    };
    Item it[kAhead];
    C a[kAhead], b[kAhead];
    auto load = [&](int k, int i) {
        it[k] = item_of(i);
        const void* base = it[k].row == 0 ? p.q : it[k].row == 1 ? p.k : p.v;
        const long long stride = it[k].row == 0 ? p.q_stride : it[k].row == 1 ? p.k_stride : p.v_stride;
        const C* src = reinterpret_cast<const C*>(static_cast<const T*>(base) + t * stride + it[k].offset);
        a[k] = *src;
        if (it[k].b) b[k] = src[it[k].b];
    };
    auto store = [&](int k, long long slot) {
        if (it[k].b) {
            T* x = reinterpret_cast<T*>(&a[k]);
            T* y = reinterpret_cast<T*>(&b[k]);
            auto pair = [&](T& re, T& im, int i) {
                const float2 cs = turn[it[k].pair + i];
                const float r = to_float(re), m = to_float(im);
                re = from_float<T>(r * cs.x - m * cs.y);
                im = from_float<T>(m * cs.x + r * cs.y);
            };
            if (p.interleaved) {
                if constexpr (VEC == 1) {
                    pair(x[0], y[0], 0);
                } else {
#pragma unroll
                    for (int i = 0; i < VEC / 2; ++i) {
                        pair(x[2 * i], x[2 * i + 1], i);
                        pair(y[2 * i], y[2 * i + 1], VEC / 2 + i);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) pair(x[i], y[i], i);
            }
        }
        if (it[k].row && slot < 0) return;
        void* base = it[k].row == 0 ? p.q_out : it[k].row == 1 ? p.k_out : p.v_out;
        const long long row = it[k].row == 0 ? t * p.num_q_heads : slot * p.num_kv_heads;
        C* dst = reinterpret_cast<C*>(static_cast<T*>(base) + row * D + it[k].offset);
        *dst = a[k];
        if (it[k].b) dst[it[k].b] = b[k];
    };

    // the rows' loads first: nothing that they wait for is behind the look-ups below
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
        if ((int)threadIdx.x + k * kThreads < items) load(k, threadIdx.x + k * kThreads);
    // then what the look-ups begin with, all at once: index and sequence, and this thread's first pair
    int s = 0, at = 0;
    if (kWrite) {
        at = p.pos[t];
        s = p.seq_idx[t];
    }
    auto axis_of = [&](int i) { return i < half && p.axis ? p.axis[i] : 0; };
    auto freq_of = [&](int i) { return i < half ? p.inv_freq[i] : 0.f; };
    int axis = axis_of(threadIdx.x);
    float freq = freq_of(threadIdx.x);
    long long slot = t;  // the row of K and V that is written, -1 for none
    if (kWrite) {
        slot = -1;
        const int block = p.by_block.div(max(at, 0) & 0x3FFFFFFF);
        if (at >= 0 && at < (1 << 30) && s >= 0 && s < p.num_seqs && block < p.max_blocks_per_seq &&
            (!p.key_width || at < p.key_width)) {
            const int physical = p.block_tables[(long long)s * p.max_blocks_per_seq + block];
            if (physical >= 0 && physical < p.num_blocks)
                slot = (long long)physical * p.block_size + (at - block * p.block_size);
        }
    }
    for (int i = threadIdx.x; i < half; i += kThreads) {
        const bool known = axis >= 0 && axis < p.num_axes;
        const int where = known ? p.rope_pos[(long long)axis * p.num_tokens + t] : 0;
        if (!known) count_error(p.error_count);
        bool finite;
        const uint64_t per = turns_of(freq, &finite);
        const int32_t turns = (int32_t)((per * (uint64_t)(int64_t)where) >> 32);  // fraction of a turn, 2^-32
        float2 cs;
        sincospif((float)turns * 0x1p-31f, &cs.y, &cs.x);
        if (!finite) cs = make_float2(NAN, NAN);
        turn[i] = cs;
        axis = axis_of(i + kThreads);
        freq = freq_of(i + kThreads);
    }
    if (kWrite) {
        if (threadIdx.x == 0) {
            if (at >= 0 && slot < 0) count_error(p.error_count);
            if (p.slot_mapping) p.slot_mapping[t] = slot;
        }
        if (at < 0) return;  // padding: nothing of the token is written
    }
    if (kWrite && p.key_width && slot >= 0)
        for (int h = threadIdx.x; h < p.num_kv_heads; h += kThreads) {
            const long long e = ((long long)s * p.num_kv_heads + h) * p.key_width + at;
            p.key_weights[e] = 0.f;
            p.key_pos[e] = p.token_pos ? p.token_pos[t] : at;
        }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
        if ((int)threadIdx.x + k * kThreads < items) store(k, slot);
    for (int i = threadIdx.x + kAhead * kThreads; i < items; i += kThreads) {
        load(0, i);
        store(0, slot);
    }
}

template <typename T, int VEC>
int launch(const RopeParams& p, cudaStream_t stream) {
    const int half = p.rot_dim / 2;
    RopeParams r = p;
    r.by_block = Divisor((uint32_t)p.block_size);
    r.by_head = Divisor((uint32_t)(half / VEC + (p.head_dim - p.rot_dim) / VEC));
    const size_t smem = sizeof(float2) * half;
    return p.block_tables || p.pos
               ? launch_kernel(rope_kernel<T, VEC, true>, dim3(p.num_tokens), dim3(kThreads), smem, stream, r)
               : launch_kernel(rope_kernel<T, VEC, false>, dim3(p.num_tokens), dim3(kThreads), smem, stream, r);
}

}  // namespace

int launch_rope(const RopeParams& p, int dtype, cudaStream_t stream) {
    // 16-byte accesses where every chunk that they touch starts on 16 bytes, single elements otherwise
    const int es = elem_size(dtype);
    const uintptr_t mix = (uintptr_t)p.q | (uintptr_t)p.k | (uintptr_t)p.v | (uintptr_t)p.q_out | (uintptr_t)p.k_out |
                          (uintptr_t)p.v_out | (uintptr_t)(p.q_stride * es) | (uintptr_t)(p.k_stride * es) |
                          (uintptr_t)(p.v_stride * es) | (uintptr_t)(p.head_dim * es) | (uintptr_t)(p.rot_dim / 2 * es);
    const bool wide = (mix & 15u) == 0;
    if (dtype == PA_F32) return wide ? launch<float, 4>(p, stream) : launch<float, 1>(p, stream);
    return wide ? launch<__nv_bfloat16, 8>(p, stream) : launch<__nv_bfloat16, 1>(p, stream);
}

}  // namespace pa
