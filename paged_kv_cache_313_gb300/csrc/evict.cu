// evict.cu — eviction of a cache's tokens by accumulated attention weight.
//
// A (sequence, kv head) of more than `budget` tokens keeps the `budget` best:
// its protected tokens (the sequence's first and most recent ones) before all
// others, the others by weight, ties by the lowest index.  Kept tokens at or
// beyond the budget move, in order, into the places below it that are free, so
// no row is both read and written and the moves run in any order.
//
// select_kernel, one CTA per (sequence, kv head): the weights become 32-bit keys
// whose order is that of the ranks, and the budget-th largest is found 12, 12 and 8 bits
// at a time by histograms in shared memory.  (12 bits are sign, exponent and three more:
// they spread weights of any scale over many counters.  With eight, a handful of counters
// took most of the time; a list of the keys in the first bin, searched bit by bit, took
// 8600 cycles where the second and third histogram take 3000.)  Then each warp lists the
// moves of its run of tokens.  A thread meets the same tokens every time, so its keys are
// its own.  move_kernel: CTAs of kMoves moves each copy the rows of K and V and the tokens'
// weights and places.  Where there can be few moves (a cache kept near its budget),
// select_kernel makes them itself.
//
// 64 sequences of 2064 tokens, 8 heads, cut to 2048: 14.3 us (one launch; bound by the chain of
// its barriers and look-ups, 17 MB would take 2.5).  16 prompts of 1k to 32k tokens cut to 4096:
// 47 to 52 us (with cold caches 25 the selection, which the longest context bounds, and 25 the moves).
#include "pa_internal.cuh"

namespace pa {
namespace {

constexpr int kMaxWarps = 32;
constexpr int kBins = 4096, kLastBins = 256;
constexpr int kKeysMax = 40 * 1024;  // keys held in shared memory; those of longer contexts are made again when needed
constexpr int kEarly = 8;  // tokens of a lane that are loaded before the length is known
constexpr int kMoves = kMaxMoves / 65535, kMoveThreads = 256;
constexpr int kOwnMoves = 128;  // the most moves that select_kernel makes itself

// Larger keys rank first: protected tokens, then weights from +inf down to -inf, -0 as 0, NaN as -inf.
__device__ __forceinline__ uint32_t key_of(float weight, int place, int keep_first, long long recent_from) {
    if (place < keep_first || (long long)place >= recent_from) return 0xFFFFFFFFu;
    if (isnan(weight)) weight = -INFINITY;
    const uint32_t u = __float_as_uint(weight + 0.f);
    return (u >> 31) ? ~u : u | 0x80000000u;
}

// The moves list[0 .. n) of a (sequence, kv head): rows of `vecs` 16-byte pieces, by the CTA's `threads` threads.
struct Move {
    long long from, to;  // rows of the pools, from < 0: a block is invalid, no rows
};
__device__ __forceinline__ Move move_of(const EvictParams& p, int s, int h, int a, int b) {
    const int32_t* table = p.block_tables + (size_t)s * p.max_blocks_per_seq;
    const int ba = a / p.block_size, bb = b / p.block_size;
    const int from = table[ba], to = table[bb];
    const bool ok = from >= 0 && from < p.num_blocks && to >= 0 && to < p.num_blocks;
    if (!ok) count_error(p.error_count);
    return Move{ok ? ((long long)from * p.block_size + (a - ba * p.block_size)) * p.num_kv_heads + h : -1,
                ((long long)to * p.block_size + (b - bb * p.block_size)) * p.num_kv_heads + h};
}
__device__ __forceinline__ void move_rows(const EvictParams& p, const Move* list, int n, int threads) {
    const int vecs = p.vecs;
    const uint4* kc = static_cast<const uint4*>(p.k_cache);
    const uint4* vc = static_cast<const uint4*>(p.v_cache);
    constexpr int kUnroll = 4;
    const int total = n * vecs;
    for (int i0 = threadIdx.x; i0 < total; i0 += threads * kUnroll) {
        uint4 k[kUnroll], v[kUnroll];
        long long at[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = i0 + u * threads;
            at[u] = -1;
            if (i >= total) continue;
            const int m = p.by_vecs.div(i), c = i - m * vecs;
            const Move mv = list[m];
            if (mv.from < 0) continue;
            at[u] = mv.to * vecs + c;
            k[u] = kc[mv.from * vecs + c];
            v[u] = vc[mv.from * vecs + c];
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (at[u] >= 0) {
                static_cast<uint4*>(p.k_cache)[at[u]] = k[u];
                static_cast<uint4*>(p.v_cache)[at[u]] = v[u];
            }
    }
}

template <bool kOwn>
__global__ void __launch_bounds__(1024) select_kernel(const EvictParams p, int keys_held) {
    extern __shared__ uint32_t keys[];
    __shared__ int hist[2 * kBins + kLastBins], sums[kMaxWarps], found[2];
    // of each warp's run: kept for certain and tied, below the budget and from it on
    __shared__ int4 runs[kMaxWarps];
    __shared__ int2 own[kOwn ? kOwnMoves : 1];     // (from, to) as cache indices
    __shared__ Move own_rows[kOwn ? kOwnMoves : 1];
    __shared__ int own_moves;  // (not in `runs`: other warps may still be reading it when the last one knows the number)
    pdl_trigger();
    pdl_wait();
    const int pair = blockIdx.x, s = pair / p.num_kv_heads, threads = blockDim.x, warps = threads >> 5;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // this warp's run of tokens, by the longest context, so that its first weights and places can be on their way while the
    // length is; a lane has every 32nd of them
    const int run = (p.max_context_len + threads - 1) / threads * 32;
    float* weights = p.key_weights + (size_t)pair * p.key_width;
    int32_t* places = p.key_pos + (size_t)pair * p.key_width;
    float w_early[kEarly];
    int place_early[kEarly];
#pragma unroll
    for (int i = 0; i < kEarly; ++i) {
        const int j = warp * run + lane + 32 * i;
        if (32 * i < run && j < p.max_context_len) {  // (key_width is no less)
            w_early[i] = weights[j];
            place_early[i] = places[j];
        }
    }
    int L = p.context_lens[s];
    const int cap = (int)min((long long)p.max_context_len, (long long)p.max_blocks_per_seq * p.block_size);
    if (L < 0 || L > cap) {
        if (threadIdx.x == 0 && pair == s * p.num_kv_heads) count_error(p.error_count);
        L = L < 0 ? 0 : cap;
    }
    const int budget = p.budget;
    if (threadIdx.x == 0) {
        if (pair == s * p.num_kv_heads) p.lens[s] = min(L, budget);
        if (!kOwn && L <= budget) p.counts[pair] = 0;
    }
    if (L <= budget) return;
    for (int i = threadIdx.x; i < 2 * kBins + kLastBins; i += threads) hist[i] = 0;

    const int j0 = min(L, warp * run), j1 = min(L, j0 + run);
    const long long recent_from = (long long)p.next_pos[s] - p.keep_recent;
#pragma unroll
    for (int i = 0; i < kEarly; ++i) {
        const int j = j0 + lane + 32 * i;
        if (j < min(j1, keys_held)) keys[j] = key_of(w_early[i], place_early[i], p.keep_first, recent_from);
    }
#pragma unroll 4
    for (int j = j0 + lane + 32 * kEarly; j < min(j1, keys_held); j += 32)
        keys[j] = key_of(weights[j], places[j], p.keep_first, recent_from);
    auto key = [&](int j) {
        return j < keys_held ? keys[j] : key_of(weights[j], places[j], p.keep_first, recent_from);
    };
    __syncthreads();

    // the budget-th largest key: among the keys that share the digits found so far, `want` is the rank still looked for
    uint32_t prefix = 0;
    int want = budget;
    // (one body for the three digits, and few unrolled loops: every instruction is fetched anew by each launch, and a body
    // for each digit took longer)
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int bins = pass < 2 ? kBins : kLastBins, shift = pass == 0 ? 20 : pass == 1 ? 8 : 0;
        int* counts = hist + pass * kBins;
        const uint32_t known = pass == 0 ? 0u : ~0u << (shift + (pass == 1 ? 12 : 8)), match = pass == 0 ? 0u : prefix << (32 - 12 * pass);
#pragma unroll 2
        for (int j = j0 + lane; j < j1; j += 32) {
            const uint32_t k = key(j);
            if ((k & known) == match) atomicAdd(&counts[(k >> shift) & (uint32_t)(bins - 1)], 1);
        }
        __syncthreads();
        // each warp sums its bins from the top (a warp's worth at least); the one that meets `want` looks closer
        const int each = max(32, bins / warps), top = bins - 1 - warp * each - lane;
        int local = 0;
        if (warp * each < bins) {
#pragma unroll 4
            for (int i = 0; i < each; i += 32) local += counts[top - i];
        }
        local = __reduce_add_sync(0xffffffffu, local);
        if (lane == 0) sums[warp] = local;
        __syncthreads();
        int before = __reduce_add_sync(0xffffffffu, lane < warp ? sums[lane] : 0);
        if (before < want && want <= before + local) {
            constexpr int kRows = 4;  // rows of 32 bins looked at together
            for (int i = 0; i < each; i += 32 * kRows) {
                int mine[kRows], row[kRows], at = before, n = 0;
#pragma unroll
                for (int k = 0; k < kRows; ++k) mine[k] = i + 32 * k < each ? counts[top - i - 32 * k] : 0;
#pragma unroll
                for (int k = 0; k < kRows; ++k) row[k] = __reduce_add_sync(0xffffffffu, mine[k]);
#pragma unroll
                for (int k = 0; k < kRows; ++k)
                    if (n == k && at + row[k] < want) {
                        at += row[k];
                        ++n;
                    }
                before = at;
                if (n == kRows) continue;
                const int count = n == 0 ? mine[0] : n == 1 ? mine[1] : n == 2 ? mine[2] : mine[3];
                int incl = count;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, incl, off);
                    if (lane >= off) incl += v;
                }
                if (before + incl - count < want && want <= before + incl) {
                    found[0] = top - i - 32 * n;
                    found[1] = want - (before + incl - count);
                }
                break;
            }
        }
        __syncthreads();
        prefix = prefix * (uint32_t)bins + (uint32_t)found[0];
        want = found[1];
    }
    // kept: keys above `prefix`, and the first `want` of those equal to it.  Lane l holds the l-th group of 32 tokens of the
    // run, as bits (longer runs: one chunk of 32 groups after the other).
    uint32_t above = 0, tied = 0;
    const int chunks = (run + 1023) / 1024;
    auto groups = [&](int chunk) {
        const int from = j0 + chunk * 1024, groups_here = min(32, (j1 - from + 31) / 32);
        above = tied = 0;
#pragma unroll 2
        for (int i = 0; i < groups_here; ++i) {
            const int j = from + 32 * i + lane;
            const uint32_t k = j < j1 ? key(j) : 0u;  // (no key is 0)
            const uint32_t a = __ballot_sync(0xffffffffu, k > prefix), t = __ballot_sync(0xffffffffu, k == prefix);
            if (lane == i) {
                above = a;
                tied = t;
            }
        }
    };
    auto bits_below = [](int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; };
    int4 mine = make_int4(0, 0, 0, 0);  // above and tied below the budget, above and tied from it on
#pragma unroll 1
    for (int chunk = 0; chunk < chunks; ++chunk) {
        groups(chunk);
        const uint32_t low = bits_below(budget - (j0 + chunk * 1024 + 32 * lane));
        mine.x += __popc(above & low);
        mine.y += __popc(tied & low);
        mine.z += __popc(above & ~low);
        mine.w += __popc(tied & ~low);
    }
    mine.x = __reduce_add_sync(0xffffffffu, mine.x);
    mine.y = __reduce_add_sync(0xffffffffu, mine.y);
    mine.z = __reduce_add_sync(0xffffffffu, mine.z);
    mine.w = __reduce_add_sync(0xffffffffu, mine.w);
    if (lane == 0) runs[warp] = mine;
    __syncthreads();
    auto sums_before = [&](int x) {  // over the lanes before this one
        int incl = x;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += v;
        }
        return incl - x;
    };
    // what lies in the runs before this one (lane w looks at run w): ties, places that get free, tokens that move
    const int4 theirs = lane < warps ? runs[lane] : make_int4(0, 0, 0, 0);
    const int ties_before = sums_before(theirs.y + theirs.w);
    const int kept_low = max(0, min(want - ties_before, theirs.y));
    const int kept_high = max(0, min(want - ties_before - theirs.y, theirs.w));
    const int tokens = min(budget, (lane + 1) * run) - min(budget, lane * run);
    int free_at = __reduce_add_sync(0xffffffffu, lane < warp ? tokens - theirs.x - kept_low : 0);
    int move_at = __reduce_add_sync(0xffffffffu, lane < warp ? theirs.z + kept_high : 0);
    int ties = __shfl_sync(0xffffffffu, ties_before, warp);
    int* src = p.src + (size_t)pair * p.max_moves;
    int* dst = p.dst + (size_t)pair * p.max_moves;
    for (int chunk = 0; chunk < chunks; ++chunk) {
        if (chunks > 1) groups(chunk);
        const int from = j0 + chunk * 1024 + 32 * lane;  // this lane's group
        const uint32_t low = bits_below(budget - from), live = bits_below(j1 - from);
        const int my_ties = __popc(tied), my_before = ties + sums_before(my_ties);
        ties += __reduce_add_sync(0xffffffffu, my_ties);
        uint32_t kept = above;
        const int keep_ties = min(want - my_before, my_ties);
        if (keep_ties == my_ties) kept |= tied;
        else
            for (uint32_t t = tied, n = 0; (int)n < keep_ties; ++n, t &= t - 1) kept |= t & (0u - t);
        uint32_t f = ~kept & low & live, m = kept & ~low;
        const int nf = __popc(f), nm = __popc(m);
        int fa = free_at + sums_before(nf), ma = move_at + sums_before(nm);
        free_at += __reduce_add_sync(0xffffffffu, nf);
        move_at += __reduce_add_sync(0xffffffffu, nm);
        for (; f; f &= f - 1, ++fa) {  // (there are as many free places as moves)
            if (kOwn) own[fa].y = from + __ffs(f) - 1;
            else dst[fa] = from + __ffs(f) - 1;
        }
        for (; m; m &= m - 1, ++ma) {
            if (kOwn) own[ma].x = from + __ffs(m) - 1;
            else src[ma] = from + __ffs(m) - 1;
        }
    }
    if (!kOwn) {
        if (warp == warps - 1 && lane == 0) p.counts[pair] = move_at;
        return;
    }
    if (warp == warps - 1 && lane == 0) own_moves = move_at;
    __syncthreads();
    const int n = own_moves;
    if ((int)threadIdx.x < n) {
        const int2 m = own[threadIdx.x];
        own_rows[threadIdx.x] = move_of(p, s, pair - s * p.num_kv_heads, m.x, m.y);
        weights[m.y] = weights[m.x];
        places[m.y] = places[m.x];
    }
    __syncthreads();
    move_rows(p, own_rows, n, threads);
}

__global__ void __launch_bounds__(kMoveThreads) move_kernel(const EvictParams p) {
    __shared__ Move list[kMoves];
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
        list[threadIdx.x] = move_of(p, s, h, a, b);
        const size_t row = (size_t)pair * p.key_width;
        p.key_weights[row + b] = p.key_weights[row + a];
        p.key_pos[row + b] = p.key_pos[row + a];
    }
    __syncthreads();
    move_rows(p, list, n, kMoveThreads);
}

// new_lens after select_kernel, where it lies in context_lens or next_pos, which every CTA of that kernel reads.
__global__ void lens_kernel(const EvictParams p) {
    pdl_trigger();
    pdl_wait();
    const int s = blockIdx.x * blockDim.x + threadIdx.x;
    if (s < p.num_seqs) p.new_lens[s] = p.lens[s];
}

bool overlap(const int32_t* a, const int32_t* b, int n) {
    return (uintptr_t)a < (uintptr_t)(b + n) && (uintptr_t)b < (uintptr_t)(a + n);
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

int launch_evict(const EvictParams& params, int row_bytes, cudaStream_t stream) {
    EvictParams p = params;
    p.vecs = row_bytes / 16;
    p.by_vecs = Divisor((uint32_t)p.vecs);
    const int held = p.max_context_len < kKeysMax ? p.max_context_len : kKeysMax;
    const size_t smem = (size_t)held * 4;
    // (the kernel reads no length before it has its own: the limit of one launch is that of all)
    int rc = ensure_dynamic_smem(reinterpret_cast<const void*>(select_kernel<true>), (size_t)kKeysMax * 4);
    if (rc == PA_OK) rc = ensure_dynamic_smem(reinterpret_cast<const void*>(select_kernel<false>), (size_t)kKeysMax * 4);
    if (rc != PA_OK) return rc;
    const int pairs = p.num_seqs * p.num_kv_heads;
    // Threads of a CTA by the longest context: fewer pass a barrier sooner and leave an SM room for more CTAs, more scan a
    // context sooner.  Measured with 256, 512 and 1024 threads, us: 512 pairs of 2064 cut by 16 12.5, 17.9, 31.9, of 4096
    // 16.4, 21.0, 35.1; of 8192 cut by 92 48, 39, 54, of 16384 86, 56, 71; 64 pairs of 16384 34, 20, 16, of 32768 62, 36, 24,
    // cut to 4096 109, 82, 71.
    const dim3 block(p.max_context_len > 16384 ? 1024 : p.max_context_len > 4096 ? 512 : 256);
    const bool own = p.max_moves <= kOwnMoves;
    const bool aliased = overlap(p.new_lens, p.context_lens, p.num_seqs) || overlap(p.new_lens, p.next_pos, p.num_seqs);
    if (own && !aliased) p.lens = p.new_lens;
    rc = own ? launch_kernel(select_kernel<true>, dim3(pairs), block, smem, stream, p, held)
             : launch_kernel(select_kernel<false>, dim3(pairs), block, smem, stream, p, held);
    if (rc != PA_OK) return rc;
    if (own) {
        if (!aliased) return PA_OK;
        return launch_kernel(lens_kernel, dim3((p.num_seqs + 255) / 256), dim3(256), 0, stream, p);
    }
    return launch_kernel(move_kernel, dim3(pairs, (p.max_moves + kMoves - 1) / kMoves), dim3(kMoveThreads), 0, stream, p);
}

}  // namespace pa
