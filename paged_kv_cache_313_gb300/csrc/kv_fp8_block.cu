// kv_fp8_block.cu — e4m3 pools with one scale for each (block, kv head): the
// quantising write and the read back.
//
// A block's values are code * scale[block][head].  The write takes, for the
// rows a call stores into a block, the smallest power of two s with
// max|x| <= 448 s and never goes below the block's scale from before, unless
// the call stores the block's first slot, which starts the block anew.  Where
// the scale grows the block's other codes are stored again under the new one.
// Powers of two make both steps exact in float: x / s shifts an exponent, and
// so does a code's move to a larger scale (only e4m3's subnormals round), so
// a block that grows token by token loses nothing by being stored again.
//
// The work unit is a physical block with all of the call's tokens that fall
// into it (whatever their order in the arrays), so the maximum needs no atomics
// and every code is written once.  A warp takes one (head, K or V) of the block:
// it loads the rows into registers (256 16-byte
// pieces at a time, a 16-token block of head_dim 128; of larger blocks all but
// the last 256 are loaded twice, the second time from L1/L2), takes the maximum
// with one warp reduction and stores the codes.
//
// Finding a block's tokens:
//   * up to kScanTokens tokens (decode steps): one launch, a CTA per token;
//     every CTA resolves all tokens itself and only the first token of each
//     block goes on.  No workspace, no second launch.  (8 heads of 128, blocks
//     of 16, this form / the other: 64 tokens of as many sequences 4.3 / 7.0 us,
//     512 8.5 / 11.2, 1024 14.9 / 17.3, 2048 34.0 / 27.7; one chunk of 512
//     tokens 7.3 / 7.5, of 1024 10.5 / 8.3.)
//   * more tokens: a first launch resolves each token once, records it as its
//     slot's writer (atomicMax, so of several tokens naming one slot the last
//     is stored, as in the one-launch form) and lists each block once; a second
//     launch walks the list, a warp per (block, head, side) without a barrier
//     among them.  It leaves the workspace zeroed again.
//
// Bound: a decode step by its launch and the latency of its dependent loads.
// Longer calls by the second launch, and there not by HBM (26 % of the DRAM
// peak): each warp walks list, writers, rows and stores alone, with nothing of
// its next unit under way, and the 256 pieces that it keeps spill (68 bytes of
// stores and 104 of loads a thread; 36 and 76 in the one-launch form).
// Measured (8 heads of 128, blocks of 16): four prompts of 2048 tokens 18.1 us
// (50.5 MB: 0.41 of the copy bandwidth; about 14 us of it the second launch);
// 256 decode tokens and 4 x 512 over blocks of 32 13.5 us.  Read back of 89,556
// tokens to bf16 87.0 us, 551 MB: 0.94; to fp32 202 us, 917 MB: 0.67.
#include "pa_internal.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kScanTokens = 1024;  // largest call of the one-launch form
constexpr int kMaxBlock = 1024;    // slots per block
constexpr int kCached = 8;         // 16-byte pieces of a (block, head, side) that a lane keeps in registers
constexpr int kMinExponent = -100; // scale of an all-zero block: 2^-100

struct BlockWriteParams {
    const uint4* k_new;  // [num_tokens][num_kv_heads][head_dim] bf16
    const uint4* v_new;
    uint8_t* k_cache;
    uint8_t* v_cache;
    float* k_scales;
    float* v_scales;
    const int32_t* block_tables;
    const int32_t* seq_idx;
    const int32_t* pos;
    int64_t* slots;
    int32_t* error_count;
    int num_tokens, num_kv_heads, head_dim, num_blocks, block_size, num_seqs, max_blocks_per_seq;
    Divisor per_pairs;  // by 2 num_kv_heads
    // two-launch form (workspace)
    int32_t* counters;  // [0] blocks listed, [1] CTAs done
    int32_t* listed;    // [num_blocks] 1: the block is on the list
    int32_t* finished;  // [num_blocks] warps that are through with the block's writers
    int32_t* writer;    // [num_blocks][block_size] token + 1 of the slot's writer, 0: none
    int32_t* list;      // [min(num_tokens, num_blocks)] the listed blocks
};

// Physical block and offset of token t; -1 when it is not stored (pos < 0), -2 when an index is invalid.
__device__ __forceinline__ int resolve(const BlockWriteParams& p, int t, int& off) {
    const int pos = p.pos[t], s = p.seq_idx[t];
    off = 0;
    if (pos < 0) return -1;
    const int lb = pos / p.block_size;
    off = pos - lb * p.block_size;
    if (s < 0 || s >= p.num_seqs || lb >= p.max_blocks_per_seq) return -2;
    const int pb = p.block_tables[(long long)s * p.max_blocks_per_seq + lb];
    return pb >= 0 && pb < p.num_blocks ? pb : -2;
}

// Magnitudes of eight bf16, the larger of each pair of halves, as two 16-bit maxima in one word.
__device__ __forceinline__ uint32_t amax_bits8(const uint4& x, uint32_t m) {
    m = __vmaxu2(m, __vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu));
    return __vmaxu2(m, __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
}
// The same with infinities and NaN left out: they take no part in the scale.
__device__ __forceinline__ uint32_t amax_finite8(const uint4& x, uint32_t m) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t v = (w[i >> 1] >> (16 * (i & 1))) & 0x7FFFu;
        m = __vmaxu2(m, v >= 0x7F80u ? 0u : v);
    }
    return m;
}

// 2^e with e the smallest integer such that amax <= 448 * 2^e = 1.75 * 2^(e + 8), at least kMinExponent.
__device__ __forceinline__ float scale_of_amax(uint32_t bf16_bits) {
    const int e = (int)(bf16_bits >> 7) - 127 - 8 + ((bf16_bits & 0x7Fu) > 0x60u ? 1 : 0);
    return __uint_as_float((uint32_t)((bf16_bits == 0 ? kMinExponent : max(e, kMinExponent)) + 127) << 23);
}

// Eight bf16 to eight e4m3 codes of x / s for an s that is no power of two (one that the caller put there).
__device__ __forceinline__ uint2 codes8_div(const uint4& x, float s) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c[i] = pack_e4m3x2(__fdiv_rn(__uint_as_float(w[i] << 16), s), __fdiv_rn(__uint_as_float(w[i] & 0xFFFF0000u), s));
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// Two codes moved to a scale 1 / f times as large (f <= 1).
__device__ __forceinline__ uint16_t recode2(uint16_t c, float f) {
    const float2 v = e4m3x2_to_float2(c);
    return pack_e4m3x2(__fmul_rn(v.x, f), __fmul_rn(v.y, f));
}

// One warp stores the call's rows of (block pb, head h, K or V); writer[off] is the token + 1 that the call stores in
// slot off, 0 for none.  kPieces: 16-byte pieces of a row's head (head_dim / 8), 0 for a head_dim that is no 64 or
// 128, whose pieces take a division each.
template <int kPieces>
__device__ __forceinline__ void store_rows(const BlockWriteParams& p, int pb, int pair, const int32_t* writer,
                                           int lane) {
    const int h = pair >> 1, D = p.head_dim, pieces = kPieces ? kPieces : D / 8, row_pieces = p.num_kv_heads * pieces;
    const uint4* src = ((pair & 1) ? p.v_new : p.k_new) + h * pieces;
    const size_t row_bytes = (size_t)p.num_kv_heads * D;
    uint8_t* cache = ((pair & 1) ? p.v_cache : p.k_cache) + (size_t)pb * p.block_size * row_bytes + (size_t)h * D;
    float* scale_ptr = ((pair & 1) ? p.v_scales : p.k_scales) + (size_t)pb * p.num_kv_heads + h;
    const int total = p.block_size * pieces;
    const float old = *scale_ptr;
    const bool fresh = writer[0] != 0;
    // the block's pieces in batches of kCached a lane, whose loads go out together; the last batch of the first pass
    // stays in registers for the second, which walks them the other way
    constexpr int kBatch = 32 * kCached;
    const int last = (total - 1) / kBatch * kBatch;
    uint4 x[kCached];
    int tok[kCached];
    auto load_batch = [&](int i0) {
#pragma unroll
        for (int k = 0; k < kCached; ++k) {
            const int i = i0 + lane + 32 * k;
            tok[k] = i < total ? writer[i / pieces] : 0;
        }
#pragma unroll
        for (int k = 0; k < kCached; ++k) {
            const int i = i0 + lane + 32 * k;
            x[k] = make_uint4(0u, 0u, 0u, 0u);
            if (tok[k] != 0) x[k] = __ldg(src + (size_t)(tok[k] - 1) * row_pieces + i % pieces);
        }
    };
    uint32_t am = 0;
#pragma unroll 1
    for (int i0 = 0; i0 <= last; i0 += kBatch) {
        load_batch(i0);
#pragma unroll
        for (int k = 0; k < kCached; ++k) am = amax_bits8(x[k], am);
    }
    am = __reduce_max_sync(0xffffffffu, max(am & 0xFFFFu, am >> 16));
    if (am >= 0x7F80u) {  // an infinity or a NaN among them: once more, without
        am = 0;
#pragma unroll 1
        for (int i = lane; i < total; i += 32) {
            const int t = writer[i / pieces];
            if (t != 0) am = amax_finite8(__ldg(src + (size_t)(t - 1) * row_pieces + i % pieces), am);
        }
        am = __reduce_max_sync(0xffffffffu, max(am & 0xFFFFu, am >> 16));
    }
    const float base = !fresh && old > 0.f ? old : 0.f;
    const float s = fmaxf(base, scale_of_amax(am));
    const float inv = 1.0f / s;  // exact for a power of two
    const bool pow2 = (__float_as_uint(s) & 0x7FFFFFu) == 0;
    auto slot = [&](int i) {  // the eight codes of piece i
        const int off = i / pieces;
        return reinterpret_cast<uint2*>(cache + off * row_bytes + (i - off * pieces) * 8);
    };
#pragma unroll 1
    for (int i0 = last; i0 >= 0; i0 -= kBatch) {
        if (i0 != last) load_batch(i0);
#pragma unroll
        for (int k = 0; k < kCached; ++k)
            if (tok[k] != 0)
                *slot(i0 + lane + 32 * k) = make_uint2(e4m3x4_of_bf16x4(make_uint2(x[k].x, x[k].y), inv),
                                                       e4m3x4_of_bf16x4(make_uint2(x[k].z, x[k].w), inv));
    }
    if (!pow2) {  // under a scale that the caller put there: the quotients, not the products with a rounded reciprocal
#pragma unroll 1
        for (int i = lane; i < total; i += 32) {
            const int t = writer[i / pieces];
            if (t != 0) *slot(i) = codes8_div(__ldg(src + (size_t)(t - 1) * row_pieces + i % pieces), s);
        }
    }
    if (!fresh && s > base) {  // the block's other codes keep their values under the larger scale
        const float f = __fdiv_rn(base, s);
#pragma unroll 1
        for (int i0 = lane; i0 < total; i0 += 32 * 4) {
            uint2 v[4];
            bool keep[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = i0 + 32 * k;
                keep[k] = i < total && writer[i / pieces] == 0;
                if (keep[k]) v[k] = *slot(i);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (keep[k])
                    *slot(i0 + 32 * k) = make_uint2(
                        (uint32_t)recode2((uint16_t)v[k].x, f) | ((uint32_t)recode2((uint16_t)(v[k].x >> 16), f) << 16),
                        (uint32_t)recode2((uint16_t)v[k].y, f) | ((uint32_t)recode2((uint16_t)(v[k].y >> 16), f) << 16));
        }
    }
    __syncwarp();  // every lane has read the old scale
    if (lane == 0) *scale_ptr = s;
}

// One launch: CTA (token, slice of the (head, side) pairs).  The first token of each block stores the block.
template <int kPieces>
__global__ void __launch_bounds__(kThreads, 4) write_scan_kernel(const BlockWriteParams p) {
    pdl_trigger();
    pdl_wait();
    __shared__ int32_t writer[kMaxBlock];
    const int t = blockIdx.x, B = p.block_size;
    for (int i = threadIdx.x; i < B; i += kThreads) writer[i] = 0;
    int my_off;
    const int mine = resolve(p, t, my_off);
    if (blockIdx.y == 0 && threadIdx.x == 0) {
        if (p.slots) p.slots[t] = mine < 0 ? -1 : (long long)mine * B + my_off;
        if (mine == -2) count_error(p.error_count);
    }
    if (mine < 0) return;
    __syncthreads();
    bool earlier = false;
    for (int i = threadIdx.x; i < p.num_tokens; i += kThreads) {
        int off;
        if (resolve(p, i, off) != mine) continue;
        earlier |= i < t;
        atomicMax(&writer[off], i + 1);
    }
    if (__syncthreads_or(earlier)) return;
    for (int pair = blockIdx.y * kWarps + (threadIdx.x >> 5); pair < 2 * p.num_kv_heads; pair += gridDim.y * kWarps)
        store_rows<kPieces>(p, mine, pair, writer, threadIdx.x & 31);
}

// Two launches, first: each token becomes its slot's writer and lists its block.
__global__ void __launch_bounds__(kThreads) write_list_kernel(const BlockWriteParams p) {
    pdl_trigger();
    pdl_wait();
    const int t = blockIdx.x * kThreads + threadIdx.x;
    if (t >= p.num_tokens) return;
    int off;
    const int pb = resolve(p, t, off);
    if (p.slots) p.slots[t] = pb < 0 ? -1 : (long long)pb * p.block_size + off;
    if (pb == -2) count_error(p.error_count);
    if (pb < 0) return;
    atomicMax(&p.writer[(size_t)pb * p.block_size + off], t + 1);
    if (atomicExch(&p.listed[pb], 1) == 0) p.list[atomicAdd(&p.counters[0], 1)] = pb;
}

// Second: a warp per (block of the list, pair), each on its own.
template <int kPieces>
__global__ void __launch_bounds__(kThreads, 4) write_listed_kernel(const BlockWriteParams p) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, pairs = 2 * p.num_kv_heads, B = p.block_size;
    // (unit = b * pairs + pair; below 2^30 warps, so the first unit and the stride are)
    const int first = blockIdx.x * kWarps + (threadIdx.x >> 5), stride = gridDim.x * kWarps, listed = p.counters[0];
    const int step_b = p.per_pairs.div(stride), step_pair = stride - step_b * pairs;
    int b = p.per_pairs.div(first), pair = first - b * pairs;
    for (; b < listed; b += step_b, pair += step_pair) {
        if (pair >= pairs) {
            pair -= pairs;
            if (++b >= listed) break;
        }
        const int pb = p.list[b];
        int32_t* writer = p.writer + (size_t)pb * B;
        store_rows<kPieces>(p, pb, pair, writer, lane);
        // the last of the block's warps to have read its writers clears them for the next call
        int done = 0;
        if (lane == 0) done = atomicAdd(&p.finished[pb], 1);
        if (__shfl_sync(0xffffffffu, done, 0) == pairs - 1) {
            for (int i = lane; i < B; i += 32) writer[i] = 0;
            if (lane == 0) {
                p.finished[pb] = 0;
                p.listed[pb] = 0;
                p.list[b] = 0;
            }
        }
    }
    // (every warp has read the count before its CTA adds its tick)
    __syncthreads();
    if (threadIdx.x == 0 && atomicAdd(&p.counters[1], 1) == (int)gridDim.x - 1) {
        p.counters[0] = 0;
        p.counters[1] = 0;
    }
}

// Read back: a CTA takes kReadTokens tokens, resolves them once, and its threads turn 16 codes at a time into
// values (the product with the scale in float, rounded once to T).
constexpr int kReadTokens = 8;

template <typename T>
__global__ void __launch_bounds__(kThreads)
    read_kernel(T* __restrict__ k_out, T* __restrict__ v_out, int num_tokens, int num_kv_heads,
                const uint4* __restrict__ k_cache, const uint4* __restrict__ v_cache,
                const float* __restrict__ k_scales, const float* __restrict__ v_scales, int num_blocks, int block_size,
                const int32_t* __restrict__ block_tables, int num_seqs, int max_blocks_per_seq,
                const int32_t* __restrict__ seq_idx, const int32_t* __restrict__ pos, int32_t* error_count,
                const Divisor per_row, const Divisor per_head) {
    pdl_trigger();
    pdl_wait();
    __shared__ int s_block[kReadTokens], s_off[kReadTokens];
    const int t0 = blockIdx.x * kReadTokens, nt = min(kReadTokens, num_tokens - t0);
    if (threadIdx.x < nt) {
        BlockWriteParams q = {};
        q.block_tables = block_tables;
        q.seq_idx = seq_idx;
        q.pos = pos;
        q.num_blocks = num_blocks;
        q.block_size = block_size;
        q.num_seqs = num_seqs;
        q.max_blocks_per_seq = max_blocks_per_seq;
        int off;
        const int pb = resolve(q, t0 + threadIdx.x, off);
        if (pb == -2) count_error(error_count);
        s_block[threadIdx.x] = pb;
        s_off[threadIdx.x] = off;
    }
    __syncthreads();
    const int pieces = (int)per_row.d, total = 2 * nt * pieces;  // 16-code pieces of a token's row; below 2^21
#pragma unroll 4
    for (int i = threadIdx.x; i < total; i += kThreads) {
        const int row = per_row.div(i), c = i - row * pieces, t = row >> 1;
        const bool v_side = row & 1;
        const int pb = s_block[t];
        if (pb < 0) continue;
        const uint4 x = __ldg((v_side ? v_cache : k_cache) + ((size_t)pb * block_size + s_off[t]) * pieces + c);
        const float s = __ldg((v_side ? v_scales : k_scales) + (size_t)pb * num_kv_heads + per_head.div(c));
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        __align__(16) T y[16];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float2 f = e4m3x2_to_float2((uint16_t)(w[k >> 1] >> (16 * (k & 1))));
            y[2 * k] = from_float<T>(__fmul_rn(f.x, s));
            y[2 * k + 1] = from_float<T>(__fmul_rn(f.y, s));
        }
        uint4* dst = reinterpret_cast<uint4*>((v_side ? v_out : k_out) + ((size_t)(t0 + t) * pieces + c) * 16);
#pragma unroll
        for (int k = 0; k < (int)sizeof(T); ++k) dst[k] = reinterpret_cast<const uint4*>(y)[k];
    }
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

struct WriteWorkspace {
    size_t listed, finished, writer, list, total;
};
WriteWorkspace write_workspace(int num_tokens, int num_blocks, int block_size) {
    WriteWorkspace w;
    w.listed = 256;
    w.finished = w.listed + up256((size_t)num_blocks * 4);
    w.writer = w.finished + up256((size_t)num_blocks * 4);
    w.list = w.writer + up256((size_t)num_blocks * block_size * 4);
    w.total = w.list + up256((size_t)(num_tokens < num_blocks ? num_tokens : num_blocks) * 4);
    return w;
}

}  // namespace

size_t write_fp8_block_workspace(int num_tokens, int num_blocks, int block_size) {
    return num_tokens <= kScanTokens ? 0 : write_workspace(num_tokens, num_blocks, block_size).total;
}

int launch_write_fp8_block(const void* k_new, const void* v_new, int num_tokens, int num_kv_heads, int head_dim,
                           void* k_cache, void* v_cache, float* k_scales, float* v_scales, int num_blocks,
                           int block_size, const int32_t* block_tables, int num_seqs, int max_blocks_per_seq,
                           const int32_t* seq_idx, const int32_t* pos, int64_t* slot_mapping, void* workspace,
                           int num_sms, int32_t* error_count, cudaStream_t stream) {
    BlockWriteParams p = {};
    p.k_new = static_cast<const uint4*>(k_new);
    p.v_new = static_cast<const uint4*>(v_new);
    p.k_cache = static_cast<uint8_t*>(k_cache);
    p.v_cache = static_cast<uint8_t*>(v_cache);
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    p.block_tables = block_tables;
    p.seq_idx = seq_idx;
    p.pos = pos;
    p.slots = slot_mapping;
    p.error_count = error_count;
    p.num_tokens = num_tokens;
    p.num_kv_heads = num_kv_heads;
    p.head_dim = head_dim;
    p.num_blocks = num_blocks;
    p.block_size = block_size;
    p.num_seqs = num_seqs;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.per_pairs = Divisor((uint32_t)(2 * num_kv_heads));
    const int slices = (2 * num_kv_heads + kWarps - 1) / kWarps, gy = slices < 64 ? slices : 64;
    if (num_tokens <= kScanTokens) {
        auto kernel = head_dim == 128 ? write_scan_kernel<16> : head_dim == 64 ? write_scan_kernel<8> : write_scan_kernel<0>;
        // every slice scans the tokens again: worth it while the tokens alone leave SMs idle (in slices / in one: 64
        // tokens 4.3 / 5.2 us, 256 5.4 / 7.4, 512 9.5 / 8.4, 1024 18.6 / 14.9)
        return launch_kernel(kernel, dim3(num_tokens, num_tokens < 2 * num_sms ? gy : 1), dim3(kThreads), 0, stream, p);
    }
    const WriteWorkspace w = write_workspace(num_tokens, num_blocks, block_size);
    char* ws = static_cast<char*>(workspace);
    p.counters = reinterpret_cast<int32_t*>(ws);
    p.listed = reinterpret_cast<int32_t*>(ws + w.listed);
    p.finished = reinterpret_cast<int32_t*>(ws + w.finished);
    p.writer = reinterpret_cast<int32_t*>(ws + w.writer);
    p.list = reinterpret_cast<int32_t*>(ws + w.list);
    const int rc = launch_kernel(write_list_kernel, dim3((num_tokens + kThreads - 1) / kThreads), dim3(kThreads), 0,
                                 stream, p);
    if (rc != PA_OK) return rc;
    const long long most = ((long long)(num_tokens < num_blocks ? num_tokens : num_blocks) * 2 * num_kv_heads + kWarps - 1) / kWarps;
    // CTAs that fit the GPU, and up to three times as many behind them, which start as those end: with one round only, some
    // warps had two units where most had one (256 decode tokens and 4 x 512 over blocks of 32: 15.2 us, so 13.8)
    const long long fill = 4LL * num_sms, ctas = most < 1 ? 1 : most < 4 * fill ? most : 4 * fill;
    auto kernel =
        head_dim == 128 ? write_listed_kernel<16> : head_dim == 64 ? write_listed_kernel<8> : write_listed_kernel<0>;
    return launch_kernel(kernel, dim3((unsigned)ctas), dim3(kThreads), 0, stream, p);
}

int launch_read_fp8_block(void* k_out, void* v_out, int num_tokens, int num_kv_heads, int head_dim, int dtype,
                          const void* k_cache, const void* v_cache, const float* k_scales, const float* v_scales,
                          int num_blocks, int block_size, const int32_t* block_tables, int num_seqs,
                          int max_blocks_per_seq, const int32_t* seq_idx, const int32_t* pos, int32_t* error_count,
                          cudaStream_t stream) {
    const dim3 grid((num_tokens + kReadTokens - 1) / kReadTokens), block(kThreads);
    const uint4 *kc = static_cast<const uint4*>(k_cache), *vc = static_cast<const uint4*>(v_cache);
    const Divisor per_row((uint32_t)(num_kv_heads * (head_dim / 16))), per_head((uint32_t)(head_dim / 16));
    if (dtype == PA_F32)
        return launch_kernel(read_kernel<float>, grid, block, 0, stream, static_cast<float*>(k_out),
                             static_cast<float*>(v_out), num_tokens, num_kv_heads, kc, vc, k_scales,
                             v_scales, num_blocks, block_size, block_tables, num_seqs, max_blocks_per_seq, seq_idx, pos,
                             error_count, per_row, per_head);
    return launch_kernel(read_kernel<__nv_bfloat16>, grid, block, 0, stream, static_cast<__nv_bfloat16*>(k_out),
                         static_cast<__nv_bfloat16*>(v_out), num_tokens, num_kv_heads, kc, vc, k_scales,
                         v_scales, num_blocks, block_size, block_tables, num_seqs, max_blocks_per_seq, seq_idx, pos,
                         error_count, per_row, per_head);
}

}  // namespace pa
