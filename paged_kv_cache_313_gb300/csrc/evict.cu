// evict.cu — eviction of a cache's tokens by accumulated attention weight.
//
// A (sequence, kv head) of more than `budget` tokens keeps the `budget` best:
// its protected tokens (the sequence's first and most recent ones) before all
// others, the others by weight, ties by the lowest index.  Kept tokens at or
// beyond the budget move, in order, into the places below it that are free, so
// no row is both read and written and the moves run in any order.
//
// Two launches.  select_kernel, one CTA per (sequence, kv head): the weights
// become 32-bit keys whose order is that of the ranks, the budget-th largest
// key is found digit by digit (histograms in shared memory), and the moves are
// listed.  move_kernel: CTAs of kMoves moves each copy the rows of K and V and
// the tokens' weights and places.
#include "pa_internal.cuh"

namespace pa {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kDigit = 11, kBins = 1 << kDigit;  // 32 bits in digits of 11, 11 and 10
constexpr int kPerThread = kBins / kThreads;
constexpr int kKeysMax = 40 * 1024;  // keys held in shared memory; those of longer contexts are made again when needed
constexpr int kMoves = 64, kMoveThreads = 256;

// Larger keys rank first: protected tokens, then weights from +inf down to -inf, -0 as 0, NaN as -inf.
__device__ __forceinline__ uint32_t key_of(float weight, int place, int keep_first, long long recent_from) {
    if (place < keep_first || (long long)place >= recent_from) return 0xFFFFFFFFu;
    if (isnan(weight)) weight = -INFINITY;
    const uint32_t u = __float_as_uint(weight + 0.f);
    return (u >> 31) ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kThreads) select_kernel(const EvictParams p, int keys_held) {
    extern __shared__ uint32_t keys[];
    __shared__ int hist[kBins], warp_sum_s[kWarps], found[2];
    pdl_trigger();
    pdl_wait();
    const int pair = blockIdx.x, s = pair / p.num_kv_heads;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int L = p.context_lens[s];
    const int cap = (int)min((long long)p.max_context_len, (long long)p.max_blocks_per_seq * p.block_size);
    if (L < 0 || L > cap) {
        if (threadIdx.x == 0 && pair == s * p.num_kv_heads) count_error(p.error_count);
        L = L < 0 ? 0 : cap;
    }
    const int budget = p.budget;
    if (threadIdx.x == 0) {
        if (pair == s * p.num_kv_heads) p.lens[s] = min(L, budget);
        if (L <= budget) p.counts[pair] = 0;
    }
    if (L <= budget) return;

    const float* weights = p.key_weights + (size_t)pair * p.key_width;
    const int32_t* places = p.key_pos + (size_t)pair * p.key_width;
    const long long recent_from = (long long)p.next_pos[s] - p.keep_recent;
    for (int j = threadIdx.x; j < min(L, keys_held); j += kThreads)
        keys[j] = key_of(weights[j], places[j], p.keep_first, recent_from);
    auto key = [&](int j) {
        return j < keys_held ? keys[j] : key_of(weights[j], places[j], p.keep_first, recent_from);
    };

    // the budget-th largest key, from its highest digit down: among the keys that share the digits found so far,
    // `want` is the rank still looked for
    uint32_t prefix = 0, mask = 0;
    int want = budget;
    for (int shift = 32 - kDigit; ; shift = shift > kDigit ? shift - kDigit : 0) {
        const int width = mask ? (shift == 0 ? 32 - 2 * kDigit : kDigit) : kDigit;
        const uint32_t digit_mask = (1u << width) - 1u;
        for (int i = threadIdx.x; i < kBins; i += kThreads) hist[i] = 0;
        __syncthreads();
        for (int j = threadIdx.x; j < L; j += kThreads) {
            const uint32_t k = key(j);
            if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & digit_mask], 1);
        }
        __syncthreads();
        // thread t sums bins [top - 3, top] downwards from the highest: the bin where the running count reaches `want`
        const int top = kBins - 1 - threadIdx.x * kPerThread;
        int local = 0;
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) local += hist[top - i];
        int incl = local;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += v;
        }
        if (lane == 31) warp_sum_s[warp] = incl;
        __syncthreads();
        int before = incl - local;
        for (int w = 0; w < warp; ++w) before += warp_sum_s[w];
        if (before < want && want <= before + local) {
            int b = top;
            while (before + hist[b] < want) before += hist[b--];
            found[0] = b;
            found[1] = want - before;
        }
        __syncthreads();
        prefix |= (uint32_t)found[0] << shift;
        mask |= digit_mask << shift;
        want = found[1];
        if (shift == 0) break;
    }
    // kept: keys above `prefix`, and the first `want` of those equal to it.  Each warp takes a run of tokens: the equal
    // keys before its run, then the free places and the moved tokens before it, then the lists.
    const int run = (L + kWarps * 32 - 1) / (kWarps * 32) * 32;
    const int j0 = warp * run, j1 = min(L, j0 + run);
    auto scan_warps = [&](int mine) {  // the sum over the warps before this one
        __syncthreads();
        if (lane == 0) warp_sum_s[warp] = mine;
        __syncthreads();
        int sum = 0;
        for (int w = 0; w < warp; ++w) sum += warp_sum_s[w];
        return sum;
    };
    int equal = 0;
    for (int j = j0 + lane; j - lane < j1; j += 32)
        equal += __popc(__ballot_sync(0xffffffffu, j < j1 && key(j) == prefix));
    const int equal_before = scan_warps(equal);
    const uint32_t below = (1u << lane) - 1u;
    auto walk = [&](auto visit) {  // visit(j, is a free place, is moved, mask of each)
        int eq = equal_before;
        for (int j = j0 + lane; j - lane < j1; j += 32) {
            const uint32_t k = j < j1 ? key(j) : 0u;
            const bool tie = j < j1 && k == prefix;
            const uint32_t ties = __ballot_sync(0xffffffffu, tie);
            const bool kept = j < j1 && (k > prefix || (tie && eq + __popc(ties & below) < want));
            eq += __popc(ties);
            visit(j, __ballot_sync(0xffffffffu, j < min(j1, budget) && !kept),
                  __ballot_sync(0xffffffffu, j >= budget && kept));
        }
    };
    int free_places = 0, moved = 0;
    walk([&](int, uint32_t f, uint32_t m) {
        free_places += __popc(f);
        moved += __popc(m);
    });
    int f_at = scan_warps(free_places), m_at = scan_warps(moved);
    int* src = p.src + (size_t)pair * p.max_moves;
    int* dst = p.dst + (size_t)pair * p.max_moves;
    walk([&](int j, uint32_t f, uint32_t m) {
        if ((f >> lane) & 1u) dst[f_at + __popc(f & below)] = j;
        if ((m >> lane) & 1u) src[m_at + __popc(m & below)] = j;
        f_at += __popc(f);
        m_at += __popc(m);
    });
    if (threadIdx.x == kThreads - 1) p.counts[pair] = m_at;
}

// VECS 16-byte pieces in a row of one kv head.
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const EvictParams p, int vecs, Divisor by_vecs) {
    __shared__ long long from[kMoves], to[kMoves];
    pdl_trigger();
    pdl_wait();
    const int pair = blockIdx.x, first = blockIdx.y * kMoves;
    const int s = pair / p.num_kv_heads, h = pair - s * p.num_kv_heads;
    if (blockIdx.y == 0 && h == 0 && threadIdx.x == 0) p.new_lens[s] = p.lens[s];
    const int n = min(kMoves, p.counts[pair] - first);
    if (n <= 0) return;
    if ((int)threadIdx.x < n) {
        const size_t at = (size_t)pair * p.max_moves + first + threadIdx.x;
        const int a = p.src[at], b = p.dst[at];
        const int32_t* table = p.block_tables + (size_t)s * p.max_blocks_per_seq;
        const int pa_ = table[a / p.block_size], pb = table[b / p.block_size];
        const bool ok = pa_ >= 0 && pa_ < p.num_blocks && pb >= 0 && pb < p.num_blocks;
        if (!ok) count_error(p.error_count);
        from[threadIdx.x] = ok ? ((long long)pa_ * p.block_size + a % p.block_size) * p.num_kv_heads + h : -1;
        to[threadIdx.x] = ((long long)pb * p.block_size + b % p.block_size) * p.num_kv_heads + h;
        const size_t row = (size_t)pair * p.key_width;
        p.key_weights[row + b] = p.key_weights[row + a];
        p.key_pos[row + b] = p.key_pos[row + a];
    }
    __syncthreads();
    const uint4* kc = static_cast<const uint4*>(p.k_cache);
    const uint4* vc = static_cast<const uint4*>(p.v_cache);
    constexpr int kUnroll = 4;
    const int total = n * vecs;
    for (int i0 = threadIdx.x; i0 < total; i0 += kMoveThreads * kUnroll) {
        uint4 k[kUnroll], v[kUnroll];
        long long at[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = i0 + u * kMoveThreads;
            at[u] = -1;
            if (i >= total) continue;
            const int m = by_vecs.div(i), c = i - m * vecs;
            if (from[m] < 0) continue;
            at[u] = to[m] * vecs + c;
            k[u] = kc[from[m] * vecs + c];
            v[u] = vc[from[m] * vecs + c];
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (at[u] >= 0) {
                static_cast<uint4*>(p.k_cache)[at[u]] = k[u];
                static_cast<uint4*>(p.v_cache)[at[u]] = v[u];
            }
    }
}

}  // namespace

EvictWorkspace evict_workspace_layout(int num_seqs, int num_kv_heads, int max_context_len, int budget) {
    EvictWorkspace w;
    const size_t pairs = (size_t)num_seqs * num_kv_heads;
    w.max_moves = max_context_len > budget ? (max_context_len - budget < budget ? max_context_len - budget : budget) : 0;
    w.counts = 0;
    w.lens = w.counts + pairs * 4;
    w.src = (w.lens + (size_t)num_seqs * 4 + 255) / 256 * 256;
    w.dst = w.src + pairs * w.max_moves * 4;
    w.total = (w.dst + pairs * w.max_moves * 4 + 256) / 256 * 256;
    return w;
}

int launch_evict(const EvictParams& p, int row_bytes, cudaStream_t stream) {
    const int held = p.max_context_len < kKeysMax ? p.max_context_len : kKeysMax;
    const size_t smem = (size_t)held * 4;
    int rc = ensure_dynamic_smem(reinterpret_cast<const void*>(select_kernel), (size_t)kKeysMax * 4);
    if (rc != PA_OK) return rc;
    const int pairs = p.num_seqs * p.num_kv_heads;
    if ((rc = launch_kernel(select_kernel, dim3(pairs), dim3(kThreads), smem, stream, p, held)) != PA_OK) return rc;
    const int pieces = p.max_moves > 0 ? (p.max_moves + kMoves - 1) / kMoves : 1;
    return launch_kernel(move_kernel, dim3(pairs, pieces), dim3(kMoveThreads), 0, stream, p, row_bytes / 16,
                         Divisor((uint32_t)(row_bytes / 16)));
}

}  // namespace pa
