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
// Bound by memory: q, k and v are read once and written once.
//
// rope_kernel, where a head's pairs are 2, 4, 8 or 16 pieces of 16 bytes: a warp
// per token (or per part of its heads, where tokens are few), a lane always on the
// same pairs, so that their angles stay in its registers: each is worked out by one
// lane and handed round once, and a head costs a lane two loads, its products and two
// stores.  (A CTA a token with the angles in shared memory spent about 3200 warp
// instructions a token, and took 66.9 us for the write of 8448 tokens of 32/8 heads; this
// takes 41.4, and 35.8 to 36.1 = 5.8 TB/s = 0.86 of the copy bandwidth with streaming loads and stores.  Four
// prompts of 2047 tokens without the write: 28.3 us = 5.9 TB/s; a step of 64 tokens: 2.6
// and 3.7 us in a stream of such calls, the launch's time.)  rope_any_kernel, for the other
// shapes: a CTA per token, the angles in shared memory.
#include <algorithm>

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

// cos and sin of pair i of a token, of `axis` and `freq`; *known false where there is no such axis (the pair stays).
__device__ __forceinline__ float2 turn_of(const RopeParams& p, long long t, int axis, float freq, bool* known) {
    *known = axis >= 0 && axis < p.num_axes;
    const int where = *known ? p.rope_pos[(long long)axis * p.num_tokens + t] : 0;
    bool finite;
    const uint64_t per = turns_of(freq, &finite);
    const int32_t turns = (int32_t)((per * (uint64_t)(int64_t)where) >> 32);  // fraction of a turn, 2^-32
    float2 cs;
    sincospif((float)turns * 0x1p-31f, &cs.y, &cs.x);
    return finite ? cs : make_float2(NAN, NAN);
}

// The slot of index `at` of sequence s, -1 where there is none.
__device__ __forceinline__ long long slot_of(const RopeParams& p, int s, int at) {
    const int block = p.by_block.div(max(at, 0) & 0x3FFFFFFF);
    if (at < 0 || at >= (1 << 30) || s < 0 || s >= p.num_seqs || block >= p.max_blocks_per_seq ||
        (p.key_width && at >= p.key_width))
        return -1;
    const int physical = p.block_tables[(long long)s * p.max_blocks_per_seq + block];
    return physical >= 0 && physical < p.num_blocks ? (long long)physical * p.block_size + (at - block * p.block_size) : -1;
}

__device__ __forceinline__ void reset_key(const RopeParams& p, long long t, int s, int at, int h) {
    const long long e = ((long long)s * p.num_kv_heads + h) * p.key_width + at;
    p.key_weights[e] = 0.f;
    p.key_pos[e] = p.token_pos ? p.token_pos[t] : at;
}

// kPieces pieces of VEC pairs a head: lane l is on piece l % kPieces of every (32 / kPieces)-th head.
constexpr int kWarps = 4;
template <typename T, int kPieces, bool kWrite>
__global__ void __launch_bounds__(kWarps * 32) rope_kernel(const RopeParams p, const int vecs_after) {
    constexpr int VEC = 16 / (int)sizeof(T), kGroups = 32 / kPieces;
    constexpr int kOwn = VEC > kGroups ? VEC / kGroups : 1;  // of its VEC pairs, those whose angles a lane works out
    constexpr int kBatch = 4;                                // heads whose loads are on their way together
    pdl_trigger();
    pdl_wait();
    const long long t = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (t >= p.num_tokens) return;
    const int lane = threadIdx.x & 31, piece = lane % kPieces, group = lane / kPieces;
    const int D = p.head_dim, Hq = p.num_q_heads, Hkv = p.num_kv_heads, heads = Hq + Hkv;
    const int part = blockIdx.y, parts = gridDim.y;
    const int step = kGroups * parts;  // from a lane's head to its next one
    // a pair's elements lie `apart` chunks from one another
    const int chunk0 = p.interleaved ? 2 * piece : piece, apart = p.interleaved ? 1 : kPieces;
    auto load = [&](int h, uint4& a, uint4& b) {
        const T* row = h < Hq ? static_cast<const T*>(p.q) + t * p.q_stride + (long long)h * D
                              : static_cast<const T*>(p.k) + t * p.k_stride + (long long)(h - Hq) * D;
        const uint4* src = reinterpret_cast<const uint4*>(row) + chunk0;
        a = __ldcs(src);
        b = __ldcs(src + apart);
    };
    // the first heads' loads, then the look-ups' first loads, then what follows from those
    uint4 a[kBatch], b[kBatch];
    const int h0 = part * kGroups + group;
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
        if (h0 + k * step < heads) load(h0 + k * step, a[k], b[k]);
    int s = 0, at = 0;
    if (kWrite) {
        at = p.pos[t];
        s = p.seq_idx[t];
    }
    // pairs piece * VEC + e, e from mine * kOwn on
    const int mine = group % (VEC / kOwn);
    int axis[kOwn];
    float freq[kOwn];
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        axis[i] = p.axis ? p.axis[piece * VEC + mine * kOwn + i] : 0;
        freq[i] = p.inv_freq[piece * VEC + mine * kOwn + i];
    }
    const long long slot = kWrite ? slot_of(p, s, at) : t;
    float2 own[kOwn], cs[VEC];
    int unknown = 0;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        bool known;
        own[i] = turn_of(p, t, axis[i], freq[i], &known);
        unknown += !known;
    }
    if (unknown && part == 0 && group < VEC / kOwn) count_error(p.error_count, unknown);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        const int from = (e / kOwn) * kPieces + piece;
        cs[e] = make_float2(__shfl_sync(0xffffffffu, own[e % kOwn].x, from), __shfl_sync(0xffffffffu, own[e % kOwn].y, from));
    }
    if (kWrite) {
        if (part == 0 && lane == 0) {
            if (at >= 0 && slot < 0) count_error(p.error_count);
            if (p.slot_mapping) p.slot_mapping[t] = slot;
        }
        if (at < 0) return;  // padding: nothing of the token is written
        if (part == 0 && slot >= 0 && p.key_width)
            for (int h = lane; h < Hkv; h += 32) reset_key(p, t, s, at, h);
    }
    auto store = [&](int h, uint4& a, uint4& b) {
        T* x = reinterpret_cast<T*>(&a);
        T* y = reinterpret_cast<T*>(&b);
        auto pair = [&](T& re, T& im, float2 c) {
            const float r = to_float(re), m = to_float(im);
            re = from_float<T>(r * c.x - m * c.y);
            im = from_float<T>(m * c.x + r * c.y);
        };
        if (p.interleaved) {
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) {
                pair(x[2 * i], x[2 * i + 1], cs[i]);
                pair(y[2 * i], y[2 * i + 1], cs[VEC / 2 + i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) pair(x[i], y[i], cs[i]);
        }
        if (h >= Hq && slot < 0) return;
        T* row = h < Hq ? static_cast<T*>(p.q_out) + (t * Hq + h) * D
                        : static_cast<T*>(p.k_out) + (slot * Hkv + (h - Hq)) * D;
        uint4* dst = reinterpret_cast<uint4*>(row) + chunk0;
        __stcs(dst, a);
        __stcs(dst + apart, b);
    };
    for (int h = h0; h < heads; h += kBatch * step) {
        if (h != h0)
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (h + k * step < heads) load(h + k * step, a[k], b[k]);
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (h + k * step < heads) store(h + k * step, a[k], b[k]);
    }
    // copies, 16 bytes a lane: what lies behind the pairs of every head, then V
    auto copy = [&](int n, auto src_of, auto dst_of) {
        for (int i0 = part * 32 + lane; i0 < n; i0 += kBatch * 32 * parts) {
            uint4 v[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (i0 + k * 32 * parts < n) v[k] = __ldcs(src_of(i0 + k * 32 * parts));
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (i0 + k * 32 * parts < n) {
                    uint4* dst = dst_of(i0 + k * 32 * parts);
                    if (dst) __stcs(dst, v[k]);
                }
        }
    };
    if (vecs_after > 0)
        copy(
            heads * vecs_after,
            [&](int i) {
                const int h = p.by_head.div(i), c = i - h * vecs_after;
                const T* row = h < Hq ? static_cast<const T*>(p.q) + t * p.q_stride + (long long)h * D
                                      : static_cast<const T*>(p.k) + t * p.k_stride + (long long)(h - Hq) * D;
                return reinterpret_cast<const uint4*>(row + p.rot_dim) + c;
            },
            [&](int i) -> uint4* {
                const int h = p.by_head.div(i), c = i - h * vecs_after;
                if (h >= Hq && slot < 0) return nullptr;
                T* row = h < Hq ? static_cast<T*>(p.q_out) + (t * Hq + h) * D
                                : static_cast<T*>(p.k_out) + (slot * Hkv + (h - Hq)) * D;
                return reinterpret_cast<uint4*>(row + p.rot_dim) + c;
            });
    if (kWrite && slot >= 0)
        copy(
            Hkv * (D / VEC),
            [&](int i) { return reinterpret_cast<const uint4*>(static_cast<const T*>(p.v) + t * p.v_stride) + i; },
            [&](int i) { return reinterpret_cast<uint4*>(static_cast<T*>(p.v_out) + slot * Hkv * D) + i; });
}

template <typename T, int VEC, bool kWrite>
__global__ void __launch_bounds__(kThreads) rope_any_kernel(const RopeParams p) {
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
    const long long slot = kWrite ? slot_of(p, s, at) : t;  // the row of K and V that is written, -1 for none
    for (int i = threadIdx.x; i < half; i += kThreads) {
        bool known;
        turn[i] = turn_of(p, t, axis, freq, &known);
        if (!known) count_error(p.error_count);
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
        for (int h = threadIdx.x; h < p.num_kv_heads; h += kThreads) reset_key(p, t, s, at, h);
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
int launch_any(const RopeParams& p, cudaStream_t stream) {
    const int half = p.rot_dim / 2;
    RopeParams r = p;
    r.by_head = Divisor((uint32_t)(half / VEC + (p.head_dim - p.rot_dim) / VEC));
    const size_t smem = sizeof(float2) * half;
    return p.pos ? launch_kernel(rope_any_kernel<T, VEC, true>, dim3(p.num_tokens), dim3(kThreads), smem, stream, r)
                 : launch_kernel(rope_any_kernel<T, VEC, false>, dim3(p.num_tokens), dim3(kThreads), smem, stream, r);
}

template <typename T, int kPieces>
int launch(const RopeParams& p, int num_sms, cudaStream_t stream) {
    constexpr int VEC = 16 / (int)sizeof(T);
    RopeParams r = p;
    const int after = (p.head_dim - p.rot_dim) / VEC;
    r.by_head = Divisor((uint32_t)(after > 0 ? after : 1));
    // few tokens: their heads are dealt out to several warps, until a warp has one head a lane or every SM 16 warps
    const int most = (p.num_q_heads + p.num_kv_heads + 32 / kPieces - 1) / (32 / kPieces);
    const int parts = std::max(1, std::min({most, 16 * num_sms / p.num_tokens, 65535}));
    const dim3 grid((p.num_tokens + kWarps - 1) / kWarps, parts);
    return p.pos ? launch_kernel(rope_kernel<T, kPieces, true>, grid, dim3(kWarps * 32), 0, stream, r, after)
                 : launch_kernel(rope_kernel<T, kPieces, false>, grid, dim3(kWarps * 32), 0, stream, r, after);
}

template <typename T>
int launch_wide(const RopeParams& p, int num_sms, cudaStream_t stream) {
    constexpr int VEC = 16 / (int)sizeof(T);
    switch (p.rot_dim / 2 % VEC == 0 ? p.rot_dim / 2 / VEC : 0) {
        case 2: return launch<T, 2>(p, num_sms, stream);
        case 4: return launch<T, 4>(p, num_sms, stream);
        case 8: return launch<T, 8>(p, num_sms, stream);
        case 16: return launch<T, 16>(p, num_sms, stream);
        default: return launch_any<T, VEC>(p, stream);
    }
}

}  // namespace

int launch_rope(const RopeParams& params, int dtype, int num_sms, cudaStream_t stream) {
    // 16-byte accesses where every chunk that they touch starts on 16 bytes, single elements otherwise
    RopeParams p = params;
    p.by_block = Divisor((uint32_t)p.block_size);
    const int es = elem_size(dtype);
    const uintptr_t mix = (uintptr_t)p.q | (uintptr_t)p.k | (uintptr_t)p.v | (uintptr_t)p.q_out | (uintptr_t)p.k_out |
                          (uintptr_t)p.v_out | (uintptr_t)(p.q_stride * es) | (uintptr_t)(p.k_stride * es) |
                          (uintptr_t)(p.v_stride * es) | (uintptr_t)(p.head_dim * es) | (uintptr_t)(p.rot_dim / 2 * es);
    const bool wide = (mix & 15u) == 0;
    if (dtype == PA_F32) return wide ? launch_wide<float>(p, num_sms, stream) : launch_any<float, 1>(p, stream);
    return wide ? launch_wide<__nv_bfloat16>(p, num_sms, stream) : launch_any<__nv_bfloat16, 1>(p, stream);
}

}  // namespace pa
