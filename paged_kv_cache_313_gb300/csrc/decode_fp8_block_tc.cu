// decode_fp8_block_tc.cu — paged decode over e4m3 pools with a scale per
// (block, kv head), on the 5th-generation tensor cores.
//
// What it computes: for sequence s, kv head h and its G query heads,
//     out = sum_j softmax_j(scale q.K_j) V_j,  K_j = code ks[block(j)], V_j = code vs[block(j)].
//
// The codes go from HBM to the tensor cores without passing through a
// register.  Keys are the M side of both products, so the few query heads make
// a narrow N of 16 columns and a whole stage of 128 tokens is four MMAs each:
//     S^T[128 tokens x 16] = K[128 x 128] . Qp^T            (K-major, as the TMA box left it)
//     O^T[128 dims x 16]   = V^T[128 dims x 128 tokens] . Pp (V MN-major, as the box left it)
// Both operands of a kind::f8f6f4 MMA are e4m3, so the queries and the
// probabilities are split into two e4m3 terms x = hi + lo / 16, whose products
// are separate columns:
//   * queries: scaled by a power of two that puts the row's largest magnitude
//     in [128, 256); two terms hold a bf16's 8 bits exactly (an element below
//     2^-14 of the row's largest is off by 2^-20 of that largest at most);
//   * weights: 256 p', two terms off by 2^-8 relative, a bf16's rounding, and at
//     least 2^-14 (2^-22 of the stage's largest p').
// ks multiplies a token's scores; vs is part of the exponent, p' = 2^(x + log2(vs) - m)
// with m the stage's maximum of x + log2(vs): the terms' floor is relative to the
// stage's largest p vs.  The sum of the softmax takes p' / vs in float, unrounded.
// A stage's output and sum are brought to the running maximum in float.
//
// Work.  An item is (sequence, partition, kv head); items are numbered as in
// decode_tc.cu (partition 0 of every (sequence, head) directly, later
// partitions through a prefix sum) and handed out by a queue.  Two CTAs per
// SM, each with a ring of three stages of 32 KB:
//   warp 4  producer: per stage one TMA box per block of K and of V (a block of
//           one kv head: block_size rows of 128 bytes), the blocks' scales
//           (loaded a 32-entry table chunk ahead), and on an item's first stage
//           the query rows.
//   warp 5  splits the queries on an item's first stage; issues S^T of a stage
//           when it lands and O^T of the stage before when its P is written.
//   warps 0-3  a thread per token of the stage: scores from tensor memory, the
//           maximum over the warp with one reduction per head, over the four
//           warps through shared memory, p, its two terms as one 16-byte row of
//           the P operand; and a thread per head dim for the output: O^T of the
//           stage before, 8 or 16 values, added to float registers.
// Tokens beyond the context or in a block without a valid table entry are
// masked, and their V rows zeroed in shared memory, so that whatever the pool
// holds there (NaN codes too) never reaches a sum.  Waits, drains and the
// queue's reset follow decode_tc.cu.
//
// Bound: HBM.  A stage is 32 KB, 0.74 us of an SM's share of the measured copy
// bandwidth; the softmax of a stage is about 250 warp instructions.  Measured: 64
// sequences, 32/8 heads, 65,500 tokens 31.2 us (135 MB: 0.64 of the copy
// bandwidth, start, uneven ends and join included); 16 long contexts, 64/8 heads,
// 189,395 tokens 73.1 us (0.79; CTAs take a stage every 3.0k cycles, 0.93); four
// sequences of up to 40 tokens 6.6 us.  On the CUDA cores the first two take 750
// and 2953 us.
#include <climits>

#include "decode_common.cuh"
#include "sm100_ptx.cuh"

namespace pa {
namespace {

constexpr int kD = 128;
constexpr int kTok = 128;  // tokens per stage
constexpr int kStages = 3;
constexpr int kTile = kTok * kD;  // bytes of a stage's K (or V)
constexpr int kThreads = 192;
constexpr int kProducer = 4, kMma = 5;
constexpr int kMaxSeqs = 512;  // per launch (the prefix sum lives in shared memory)
constexpr int kMaxBlocks = kTok / 8;  // blocks of a stage
constexpr uint32_t kTmemCols = 64;    // S0 | S1 | O0 | O1, 16 columns each
// A V scale below 2^-80 of the stage's largest or 2^-100 (the smallest that the write makes) counts as 0.
constexpr float kHold = 8.271806125530277e-25f, kLeastScale = 7.888609052210118e-31f;

// num_partitions for this file's partitions, which are powers of two.
__device__ __forceinline__ int partitions(int L, int part) {
    return L <= part ? 1 : ((L - 1) >> (31 - __clz(part))) + 1;
}

struct Stage {
    int s, kvh, split, flags;  // flags: 1 first stage of the item, 2 last, 4 the item writes the output, 8 no more
    int ntok;                  // tokens of the stage
    uint32_t blocks;           // bit b: block b of the stage has a valid table entry
    float vmax;                // the largest V scale of its blocks
    int pad;
};

// shared memory, offsets from a 1024-aligned base
constexpr int kRing = 0;
constexpr int kQp = kRing + kStages * 2 * kTile;     // e4m3 [16][128]: the query terms, 128-byte swizzled
constexpr int kP = kQp + 16 * kD;                    // e4m3 [2][128 tokens][16]
constexpr int kQ = kP + 2 * kTok * 16;               // bf16 [kStages][8][128]: raw query rows
constexpr int kKs = kQ + kStages * 8 * kD * 2;       // float [kStages][kMaxBlocks]
constexpr int kVs = kKs + kStages * kMaxBlocks * 4;
constexpr int kCum = kVs + kStages * kMaxBlocks * 4;  // int [kMaxSeqs + 1], padded to 16 bytes
constexpr int kRed = kCum + (kMaxSeqs + 4) * 4;       // float [2][4][8]: the warps' maxima
constexpr int kRedL = kRed + 2 * 4 * 8 * 4;           // float [4][8]: the warps' sums
constexpr int kQf = kRedL + 4 * 8 * 4;                // float [2][8]: what a query row's terms are multiplied with
constexpr int kScan = kQf + 2 * 8 * 4;                // int [8]
constexpr int kStage = kScan + 32;                    // Stage [kStages]
constexpr int kBars = kStage + kStages * (int)sizeof(Stage);
// full[kStages], empty[kStages], s_full[2], p_full[2], o_full[2], q_ready[2], softmax barrier, cum, drain
constexpr int kNumBars = 2 * kStages + 11;
constexpr int kTmemSlot = kBars + kNumBars * 8;
constexpr int kEnd = kTmemSlot + 16;
constexpr size_t kSmemBytes = 1024 + kEnd;
static_assert(kQp % 1024 == 0 && kP % 16 == 0 && kQ % 16 == 0 && kRed % 16 == 0 && kStage % 16 == 0 && kBars % 8 == 0,
              "alignment");
// an SM holds 228 KiB, of which 1 KiB is taken by each resident CTA
static_assert(kSmemBytes <= 228 * 1024 / 2 - 1024, "two CTAs per SM");

// kHeads: columns kept for query heads, 4 (groups up to 4) or 8; hi terms are columns 0..kHeads-1, lo terms the next.
// (Groups of 4 with 4 columns / with 8: 64 sequences 30.9 / 32.9 us, 16 long contexts 67.5 / 70.1, one 8000-token
// context 15.3 / 15.7.)
template <int kHeads>
__global__ void __launch_bounds__(kThreads, 2)
    decode_fp8_block_tc_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                               const DecodeParams p, const Divisor per_heads) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    int* cum = reinterpret_cast<int*>(smem + kCum);
    int* scan = reinterpret_cast<int*>(smem + kScan);  // [0..3] warp totals, [4] items of partitions >= 1
    Stage* stages = reinterpret_cast<Stage*>(smem + kStage);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kBars);
    uint64_t *empty = full + kStages, *s_full = empty + kStages, *p_full = s_full + 2, *o_full = p_full + 2;
    uint64_t *q_ready = o_full + 2, *warp_bar = q_ready + 2, *cum_bar = warp_bar + 1, *drain_bar = cum_bar + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kTmemSlot);
    const int N = p.num_seqs, Hkv = p.num_kv_heads, G = p.group, B = p.block_size;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 2);  // the copies' arming and the scales
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&o_full[i], 1);
            mbar_init(&q_ready[i], 1);
        }
        mbar_init(warp_bar, 4);
        mbar_init(cum_bar, 1);
        mbar_init(drain_bar, 1);
        fence_mbar_init();
    }
    // query rows without a head stay zero
    for (int i = threadIdx.x; i < 16 * kD / 16; i += kThreads)
        reinterpret_cast<uint4*>(smem + kQp)[i] = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
    pdl_trigger();
    pdl_wait();
    // the first item of most CTAs begins its sequence: its length and table entries are asked for before the set-up ends
    const int n_first = N * Hkv;  // partition-0 items
    int early = -1, early_len = 0;
    if (warp == kProducer && (int)blockIdx.x < n_first) {
        const int s0 = per_heads.div(blockIdx.x);
        early_len = p.context_lens[s0];
        if (lane < p.max_blocks_per_seq) early = p.block_tables[(size_t)s0 * p.max_blocks_per_seq + lane];
    }
    if (warp == kMma) {  // after the wait: a kernel before this one may still be about to take its tensor memory
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    auto later_items = [&](int s) {
        return (partitions(decode_context(p, s, false), partition_of(p, s)) - 1) * Hkv;
    };
    if (warp < 4) {  // prefix sum of the later partitions' counts, while the producer starts its first item
        const int per = (N + 127) / 128, first = threadIdx.x * per;
        int local = 0;
        for (int i = first; i < min(first + per, N); ++i) {
            if (blockIdx.x == 0) decode_context(p, i, true);
            local += later_items(i);
        }
        int incl = local;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += v;
        }
        if (lane == 31) scan[warp] = incl;
        asm volatile("bar.sync 1, 128;" ::: "memory");
        int run = incl - local;
        for (int w = 0; w < warp; ++w) run += scan[w];
        for (int i = first; i < min(first + per, N); ++i) {
            cum[i] = run;
            run += later_items(i);
        }
        if (threadIdx.x == 0) scan[4] = scan[0] + scan[1] + scan[2] + scan[3];
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (threadIdx.x == 0) mbar_arrive(cum_bar);
    }

    if (warp == kProducer) {
        // ================================================================ producer
        if (lane == 0) {
            tma_prefetch_desc(&tmk);
            tma_prefetch_desc(&tmv);
        }
        struct Item {
            int s, split, kvh, nsplit, j0, ntok, nblk;
        };
        const int log2b = 31 - __clz(B);
        auto describe = [&](int it, int known_len) {  // known_len: the item's context_lens entry, or INT_MIN
            Item d;
            if (it < n_first) {
                d.s = per_heads.div(it);
                d.split = 0;
                d.kvh = it - d.s * Hkv;
            } else {
                it -= n_first;
                int lo = 0, hi = N - 1;
                while (lo < hi) {  // the last sequence with cum <= it
                    const int mid = (lo + hi + 1) >> 1;
                    if (cum[mid] <= it) lo = mid; else hi = mid - 1;
                }
                d.s = lo;
                const int r = it - cum[lo];
                d.split = per_heads.div(r) + 1;
                d.kvh = r - (d.split - 1) * Hkv;
            }
            const int L = known_len == INT_MIN ? decode_context(p, d.s, false) : clamp_context(p, known_len);
            const int part = partition_of(p, d.s);
            d.nsplit = partitions(L, part);
            d.j0 = d.split * part;
            d.ntok = max(0, min(L - d.j0, part));
            d.nblk = (d.ntok + B - 1) >> log2b;
            return d;
        };
        // this lane's entry of a 32-block chunk of an item's table, and its scales (0 without a valid block)
        auto load_raw = [&](const Item& d, int chunk) {
            const int i = chunk * 32 + lane;
            return i < d.nblk ? p.block_tables[(size_t)d.s * p.max_blocks_per_seq + (d.j0 >> log2b) + i] : -1;
        };
        auto load_scales = [&](const Item& d, int pb) {
            if (pb < 0 || pb >= p.num_blocks) return make_float2(0.f, 0.f);
            const size_t i = (size_t)pb * Hkv + d.kvh;
            return make_float2(__ldg(p.k_scales + i), __ldg(p.v_scales + i));
        };
        const int bps = kTok >> log2b, log2spc = log2b - 2;  // blocks per stage; 32-block chunks are 2^log2spc stages
        const uint64_t policy = l2_policy_evict_first();  // K and V are read once
        bool ok = true;
        int total = -1;
        auto is_item = [&](int it) {
            if (it < n_first) return true;
            if (total < 0) {
                total = 0;
                if (mbar_wait_warp(cum_bar, 0)) total = n_first + scan[4];
                else ok = false;
            }
            return it < total;
        };
        int item = blockIdx.x, nxt = 0;
        Item d{};
        int raw = -1;
        float2 sc = make_float2(0.f, 0.f);
        if (is_item(item)) {
            d = describe(item, item < n_first ? early_len : INT_MIN);
            raw = item < n_first ? (lane < d.nblk ? early : -1) : load_raw(d, 0);
            sc = load_scales(d, raw);
        }
        uint32_t n = 0;  // stages issued
        while (ok && is_item(item)) {
            const int nst = max(1, (d.ntok + kTok - 1) / kTok);
            // the next item is claimed three stages before the last, described a stage later, its scales loaded last
            const int claim_at = max(0, nst - 3), describe_at = min(nst - 1, claim_at + 1);
            const int scales_at = min(nst - 1, describe_at + 1);
            int item2 = INT_MAX, raw2 = -1, raw_next = -1;
            float2 sc2 = make_float2(0.f, 0.f), sc_next = make_float2(0.f, 0.f);
            Item d2{};
            int pb = -1;
            for (int st = 0; st < nst; ++st, ++n) {
                const int slot = n % kStages, chunk = st >> log2spc, l = st - (chunk << log2spc);
                if (l == 0) {
                    if (chunk > 0) {
                        raw = raw_next;
                        sc = sc_next;
                    }
                    pb = raw;
                    if (chunk * 32 + lane < d.nblk && (raw < 0 || raw >= p.num_blocks)) {
                        count_error(p.error_count);
                        pb = -1;
                    }
                }
                if (n >= kStages && !mbar_wait_warp(&empty[slot], ((n / kStages) - 1) & 1)) {
                    ok = false;
                    break;
                }
                const uint32_t valid = __ballot_sync(0xffffffffu, pb >= 0);
                const uint32_t mine = (valid >> (l * bps)) & (bps == 32 ? ~0u : (1u << bps) - 1u);
                if (lane == 0) {
                    uint32_t bytes = (uint32_t)__popc(mine) * 2u * B * kD;
                    if (st == 0) bytes += (uint32_t)(G * kD * 2);
                    mbar_arrive_expect_tx(&full[slot], bytes);
                    if (st == 0)
                        bulk_load(smem + kQ + slot * 8 * kD * 2,
                                  static_cast<const __nv_bfloat16*>(p.q) +
                                      ((size_t)d.s * p.num_q_heads + (size_t)d.kvh * G) * kD,
                                  (uint32_t)(G * kD * 2), &full[slot]);
                }
                __syncwarp();  // armed before any copy is issued
                // lanes [0, bps) copy the stage's K blocks, lanes [bps, 2 bps) its V blocks
                const bool v_side = lane >= bps;
                const int b = v_side ? lane - bps : lane;
                const int src = l * bps + (lane < 2 * bps ? b : 0);
                const int my_pb = __shfl_sync(0xffffffffu, pb, src);
                if (lane < 2 * bps && my_pb >= 0)
                    tma_load_3d_hint(smem + kRing + slot * 2 * kTile + v_side * kTile + b * B * kD,
                                     v_side ? &tmv : &tmk, 0, my_pb * B, d.kvh, &full[slot], policy);
                const float ks = __shfl_sync(0xffffffffu, sc.x, src), vs = __shfl_sync(0xffffffffu, sc.y, src);
                const float vm = redux_max(lane < bps ? vs : 0.f);
                if (lane < bps) {
                    reinterpret_cast<float*>(smem + kKs)[slot * kMaxBlocks + lane] = ks;
                    reinterpret_cast<float*>(smem + kVs)[slot * kMaxBlocks + lane] = vs;
                }
                if (lane == 0) {
                    Stage& g = stages[slot];
                    g.s = d.s;
                    g.kvh = d.kvh;
                    g.split = d.split;
                    g.flags = (st == 0 ? 1 : 0) | (st == nst - 1 ? 2 : 0) | (d.nsplit == 1 ? 4 : 0);
                    g.ntok = min(kTok, d.ntok - st * kTok);
                    g.blocks = mine;
                    g.vmax = vm;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[slot]);
                // loads for later stages, used a stage or more from now
                if (l == 0) raw_next = load_raw(d, chunk + 1);
                if (l == 1) sc_next = load_scales(d, raw_next);
                if (st == claim_at && lane == 0) nxt = (int)gridDim.x + atomicAdd(&p.work[0], 1);
                if (st == describe_at) {
                    item2 = __shfl_sync(0xffffffffu, nxt, 0);
                    if (is_item(item2)) {
                        d2 = describe(item2, INT_MIN);
                        raw2 = load_raw(d2, 0);
                    }
                }
                if (st == scales_at) sc2 = load_scales(d2, raw2);
            }
            item = item2;
            d = d2;
            raw = raw2;
            sc = sc2;
        }
        // the stage that ends the other warps' loops
        const int slot = n % kStages;
        const bool free_slot = n < kStages || mbar_wait_warp(&empty[slot], ((n / kStages) - 1) & 1);
        if (lane == 0) {
            if (!ok || !free_slot) count_error(p.error_count);
            if (free_slot) {
                stages[slot].flags = 8;
                mbar_arrive_expect_tx(&full[slot], 0);
                mbar_arrive(&full[slot]);
            }
            // every copy has landed before the CTA exits
            if (!drain_ring(full, kStages, n + (free_slot ? 1 : 0))) count_error(p.error_count);
        }
        __syncwarp();
    } else if (warp == kMma) {
        // ================================================================ MMA issuer
        constexpr uint32_t idesc_s = umma_idesc_e4m3(128, 16, false, false);
        constexpr uint32_t idesc_o = umma_idesc_e4m3(128, 16, true, true);
        const uint32_t ring = smem_u32(smem + kRing);
        const uint64_t dq = umma_desc_sw128(smem_u32(smem + kQp), 16, 1024);
        const uint64_t dk0 = umma_desc_sw128(ring, 16, 1024), dv0 = umma_desc_sw128(ring + kTile, 16, 1024);
        const uint64_t dp0 = umma_desc_plain(smem_u32(smem + kP), 128, 128);
        bool ok = true;
        // O^T of stage i: V^T P, when its P is written
        auto issue_pv = [&](uint32_t i) {
            const int slot = i % kStages, b = i & 1;
            if (!mbar_wait_warp(&p_full[b], (i >> 1) & 1)) {
                ok = false;
                return;
            }
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < kTok / 32; ++k)
                umma_e4m3_warp(tmem + 32 + b * 16, dv0 + (uint64_t)((slot * 2 * kTile + k * 32 * kD) >> 4),
                               dp0 + (uint64_t)((b * kTok * 16 + k * 32 * 16) >> 4), idesc_o, k > 0);
            umma_commit_warp(&o_full[b]);
            umma_commit_warp(&empty[slot]);
        };
        int items = 0;
        for (uint32_t i = 0; ok; ++i) {
            const int slot = i % kStages;
            // the stage before goes first unless this one has landed already
            const bool landed = __all_sync(0xffffffffu, mbar_test_wait(&full[slot], (i / kStages) & 1));
            if (!landed) {
                if (i > 0) issue_pv(i - 1);
                if (!ok || !mbar_wait_warp(&full[slot], (i / kStages) & 1)) {
                    ok = false;
                    break;
                }
            }
            const int flags = stages[slot].flags;
            if (!(flags & 8)) {
                if (flags & 1) {
                    // the item's query terms; their buffer is free once the last S^T is done
                    if (i > 0 && !mbar_wait_warp(&s_full[(i - 1) & 1], ((i - 1) >> 1) & 1)) {
                        ok = false;
                        break;
                    }
                    for (int h = 0; h < G; ++h) {
                        const uint2 x = reinterpret_cast<const uint2*>(smem + kQ + (slot * 8 + h) * kD * 2)[lane];
                        const uint32_t m2 = __vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu);
                        const uint32_t am = __reduce_max_sync(0xffffffffu, max(m2 & 0xFFFFu, m2 >> 16));
                        const int e = min(134 - (int)(am >> 7), 126);  // |x| 2^e in [128, 256)
                        // (a row with an infinity or a NaN becomes NaN: the conversion would hold an infinity at 448)
                        const float f = am >= 0x7F80u ? NAN : __uint_as_float((uint32_t)(e + 127) << 23);
                        float v[4] = {__uint_as_float(x.x << 16) * f, __uint_as_float(x.x & 0xFFFF0000u) * f,
                                      __uint_as_float(x.y << 16) * f, __uint_as_float(x.y & 0xFFFF0000u) * f};
                        uint32_t hi = 0, lo = 0;
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint16_t c = pack_e4m3x2(v[2 * j], v[2 * j + 1]);
                            const float2 r = e4m3x2_to_float2(c);
                            hi |= (uint32_t)c << (16 * j);
                            lo |= (uint32_t)pack_e4m3x2((v[2 * j] - r.x) * 16.f, (v[2 * j + 1] - r.y) * 16.f) << (16 * j);
                        }
                        // row r of the tile: its 16-byte pieces are swizzled by r mod 8
                        auto at = [&](int r) {
                            return reinterpret_cast<uint32_t*>(smem + kQp + r * kD + (((lane >> 2) ^ (r & 7)) << 4) +
                                                               (lane & 3) * 4);
                        };
                        *at(h) = hi;
                        *at(kHeads + h) = lo;
                        if (lane == 0)
                            reinterpret_cast<float*>(smem + kQf)[(items & 1) * 8 + h] =
                                __uint_as_float((uint32_t)(127 - e) << 23);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&q_ready[items & 1]);
                    ++items;
                }
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < kD / 32; ++k)
                    umma_e4m3_warp(tmem + (i & 1) * 16, dk0 + (uint64_t)((slot * 2 * kTile + k * 32) >> 4),
                                   dq + (uint64_t)((k * 32) >> 4), idesc_s, k > 0);
                umma_commit_warp(&s_full[i & 1]);
            }
            if (landed && i > 0) issue_pv(i - 1);
            if (flags & 8) break;
        }
        if (!ok && lane == 0) count_error(p.error_count);
        // no MMA is running when the tensor memory is freed
        umma_commit_warp(drain_bar);
        if (!mbar_wait_warp(drain_bar, 0) && lane == 0) count_error(p.error_count);
        __syncwarp();
    } else {
        // ================================================================ softmax and output
        const int t = threadIdx.x;  // token of the stage, and head dim of the output
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        const int log2b = 31 - __clz(B);
        float(*red)[4][8] = reinterpret_cast<float(*)[4][8]>(smem + kRed);
        float(*red_l)[8] = reinterpret_cast<float(*)[8]>(smem + kRedL);
        BoundedWarpBarrier sync{warp_bar, 0};
        float m[kHeads], l[kHeads], acc[kHeads], bring[kHeads], qf[kHeads];
        bool ok = true;
        int items = 0;
        auto load_cols = [&](uint32_t col, float (&hi)[kHeads], float (&lo)[kHeads]) {
            if constexpr (kHeads == 8) {
                float v[16];
                tmem_ld16(tmem + lanes + col, v);
                tmem_wait_ld();
#pragma unroll
                for (int h = 0; h < 8; ++h) hi[h] = v[h], lo[h] = v[8 + h];
            } else {
                float v[8];
                tmem_ld8(tmem + lanes + col, v);
                tmem_wait_ld();
#pragma unroll
                for (int h = 0; h < 4; ++h) hi[h] = v[h], lo[h] = v[4 + h];
            }
        };
        auto add_output = [&](uint32_t i) {  // acc += O^T of stage i, this thread's head dim
            if (!mbar_wait_warp(&o_full[i & 1], (i >> 1) & 1)) {
                ok = false;
                return;
            }
            tc_fence_after();
            float hi[kHeads], lo[kHeads];
            load_cols(32 + (i & 1) * 16, hi, lo);
#pragma unroll
            for (int h = 0; h < kHeads; ++h) acc[h] = fmaf(fmaf(lo[h], 1.f / 16, hi[h]), bring[h], acc[h]);
        };
        for (uint32_t i = 0; ok; ++i) {
            const int slot = i % kStages, b = i & 1;
            if (!mbar_wait_warp(&full[slot], (i / kStages) & 1)) {
                ok = false;
                break;
            }
            const Stage g = stages[slot];
            if (g.flags & 8) break;
            const bool valid = t < g.ntok && ((g.blocks >> (t >> log2b)) & 1u);
            const float ks = reinterpret_cast<const float*>(smem + kKs)[slot * kMaxBlocks + (t >> log2b)];
            const float vs = reinterpret_cast<const float*>(smem + kVs)[slot * kMaxBlocks + (t >> log2b)];
            // (a V below `hold` adds nothing, its key's weight still counts in the sum)
            const float hold = fmaxf(g.vmax * kHold, kLeastScale);
            const float off = __log2f(fmaxf(vs, hold)), unit = vs >= hold ? 256.f : 0.f;
            const float inv_vs = exp2f(-off);  // (a subnormal beyond a scale of 2^126, where fast_exp2 gives 0)
            if (g.flags & 1) {
                if (!mbar_wait_warp(&q_ready[items & 1], (items >> 1) & 1)) {
                    ok = false;
                    break;
                }
#pragma unroll
                for (int h = 0; h < kHeads; ++h) {
                    m[h] = -INFINITY;
                    l[h] = acc[h] = 0.f;
                    qf[h] = h < G ? reinterpret_cast<const float*>(smem + kQf)[(items & 1) * 8 + h] : 0.f;
                }
                ++items;
            }
            if (!mbar_wait_warp(&s_full[b], (i >> 1) & 1)) {
                ok = false;
                break;
            }
            tc_fence_after();
            float x[kHeads];
            {
                float hi[kHeads], lo[kHeads], wm[8];
                load_cols(b * 16, hi, lo);
                const float c = ks * p.scale_log2;
#pragma unroll
                for (int h = 0; h < 8; ++h) wm[h] = -INFINITY;
#pragma unroll
                for (int h = 0; h < kHeads; ++h) {
                    x[h] = valid ? fmaf(fmaf(lo[h], 1.f / 16, hi[h]) * qf[h], c, off) : -INFINITY;
                    wm[h] = redux_max(x[h]);
                }
                if (lane == 0) {
                    *reinterpret_cast<float4*>(&red[b][warp][0]) = make_float4(wm[0], wm[1], wm[2], wm[3]);
                    if (kHeads == 8)
                        *reinterpret_cast<float4*>(&red[b][warp][4]) = make_float4(wm[4], wm[5], wm[6], wm[7]);
                }
            }
            if (!sync.sync()) {
                ok = false;
                break;
            }
            // the stage's maxima mx, the running ones, and what the state so far (where the stage's are larger: grow) or this
            // stage's sums (where not) are multiplied with to come to the running maxima, as a factor that applies twice:
            // the maxima have the V scales in them, so that they may be 2^220 apart between stages whose keys weigh the
            // same, and the sums, which are divided by the scales, keep what one factor would flush to 0 (an output's
            // part from so small a V is nothing, its product may flush)
            float mx[kHeads], root[kHeads];
            bool grow[kHeads];
#pragma unroll
            for (int h4 = 0; h4 < kHeads / 4; ++h4) {
                *reinterpret_cast<float4*>(mx + 4 * h4) = *reinterpret_cast<const float4*>(&red[b][0][4 * h4]);
#pragma unroll
                for (int w = 1; w < 4; ++w) {
                    const float4 o = *reinterpret_cast<const float4*>(&red[b][w][4 * h4]);
                    mx[4 * h4] = fmaxf(mx[4 * h4], o.x);
                    mx[4 * h4 + 1] = fmaxf(mx[4 * h4 + 1], o.y);
                    mx[4 * h4 + 2] = fmaxf(mx[4 * h4 + 2], o.z);
                    mx[4 * h4 + 3] = fmaxf(mx[4 * h4 + 3], o.w);
                }
            }
#pragma unroll
            for (int h = 0; h < kHeads; ++h) {
                grow[h] = mx[h] > m[h];
                // (0 at the first finite maximum, and for a stage without one)
                root[h] = mx[h] == -INFINITY ? 0.f : fast_exp2(0.5f * (fminf(m[h], mx[h]) - fmaxf(m[h], mx[h])));
                m[h] = fmaxf(m[h], mx[h]);
            }
            uint32_t row[4] = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int h2 = 0; h2 < kHeads / 2; ++h2) {
                float w[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int h = 2 * h2 + j;
                    const float e = valid ? fast_exp2(x[h] - mx[h]) : 0.f;
                    const float add = e * inv_vs;
                    l[h] = fmaf((grow[h] ? l[h] : add) * root[h], root[h], grow[h] ? add : l[h]);
                    w[j] = e * unit;
                }
                const uint16_t hi = pack_e4m3x2(w[0], w[1]);
                const float2 r = e4m3x2_to_float2(hi);
                const uint16_t lo = pack_e4m3x2((w[0] - r.x) * 16.f, (w[1] - r.y) * 16.f);
                row[h2 >> 1] |= (uint32_t)hi << (16 * (h2 & 1));
                row[kHeads / 4 + (h2 >> 1)] |= (uint32_t)lo << (16 * (h2 & 1));
            }
            if (!valid) row[0] = row[1] = row[2] = row[3] = 0u;
            reinterpret_cast<uint4*>(smem + kP + b * kTok * 16)[t] = make_uint4(row[0], row[1], row[2], row[3]);
            if (!valid) {  // whatever the pool holds for this token must not meet even a zero
                uint4* vrow = reinterpret_cast<uint4*>(smem + kRing + slot * 2 * kTile + kTile + t * kD);
#pragma unroll
                for (int k = 0; k < kD / 16; ++k) vrow[k] = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            tc_fence_before();  // S of this stage and O of the stage before the last have been read
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[b]);
            // the output of the stage before, brought to the maxima as of that stage by `bring`, then to this one's
            if (!(g.flags & 1)) add_output(i - 1);
            if (!ok) break;
#pragma unroll
            for (int h = 0; h < kHeads; ++h) {
                const float f = root[h] * root[h];
                if (grow[h]) acc[h] *= f;
                bring[h] = grow[h] ? 1.f / 256 : f * (1.f / 256);
            }
            if (!(g.flags & 2)) continue;
            // ---- end of the item: the sums over all tokens, then this thread's head dim of every head
            add_output(i);
            if (!ok) break;
#pragma unroll
            for (int h = 0; h < kHeads; ++h) {
                const float s = warp_sum(l[h]);
                if (lane == 0) red_l[warp][h] = s;
            }
            if (!sync.sync()) {
                ok = false;
                break;
            }
            const size_t slot_ws = decode_unit(p, g.s, g.kvh) * p.max_splits + g.split;
#pragma unroll
            for (int h = 0; h < kHeads; ++h) {
                if (h >= G) break;
                const float L = (red_l[0][h] + red_l[1][h]) + (red_l[2][h] + red_l[3][h]);
                // (a NaN sum, of a NaN that the sequence holds, stays one)
                const float o = L == 0.f ? 0.f : acc[h] / L;
                if (g.flags & 4) {
                    static_cast<__nv_bfloat16*>(p.out)[((size_t)g.s * p.num_q_heads + (size_t)g.kvh * G + h) * kD + t] =
                        __float2bfloat16_rn(o);
                } else {
                    p.ws_o[(slot_ws * G + h) * kD + t] = o;
                    if (t == 0) p.ws_ml[slot_ws * G + h] = make_float2(m[h], L);
                }
            }
        }
        if (!ok && lane == 0) count_error(p.error_count);
    }
    // ---- the last CTA to finish resets the queue for the next call
    tc_fence_before();
    __syncthreads();
    if (warp == kMma) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
    if (threadIdx.x == 0) {
        __threadfence();
        if (atomicAdd(&p.work[1], 1) == (int)gridDim.x - 1) {
            atomicExch(&p.work[0], 0);
            atomicExch(&p.work[1], 0);
        }
    }
}

template <int kHeads>
int launch(const DecodeParams& p, int num_sms, cudaStream_t stream) {
    CUtensorMap tmk, tmv;
    int rc = pool_tensor_map_rows(&tmk, p.k_cache, p.num_blocks, p.block_size, p.num_kv_heads, kD, true);
    if (rc != PA_OK) return rc;
    if ((rc = pool_tensor_map_rows(&tmv, p.v_cache, p.num_blocks, p.block_size, p.num_kv_heads, kD, true)) != PA_OK)
        return rc;
    auto kernel = decode_fp8_block_tc_kernel<kHeads>;
    if ((rc = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), kSmemBytes)) != PA_OK) return rc;
    const long long most = (long long)p.num_seqs * p.num_kv_heads * p.max_splits, slots = 2LL * num_sms;
    return launch_kernel(kernel, dim3((unsigned)(most < slots ? most : slots)), dim3(kThreads), kSmemBytes, stream,
                         tmk, tmv, p, Divisor((uint32_t)p.num_kv_heads));
}

// The join of a split context's partials (m_i, l_i, o_i): out = sum_i w_i o_i / sum_i w_i, w_i = l_i 2^(m_i - max m).
// A CTA of four warps per (sequence, query head): a thread per split for the weights, then every fourth split to each
// warp, eight of its rows in flight, summed in split order and the warps' sums in warp order.  (One warp per (sequence,
// head) took 12.4 us for 16 sequences of up to 64 splits and 64 heads, its loads one round of eight after another.)
template <int D>
__global__ void __launch_bounds__(128) decode_fp8_block_join_kernel(const DecodeParams p) {
    constexpr int kCols = D / 4;  // float4 columns of a row
    pdl_trigger();
    pdl_wait();
    __shared__ float weight[128], warp_m[4], warp_w[4];
    __shared__ float4 sums[4][kCols];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = p.group, Hq = p.num_q_heads;
    const uint32_t u = blockIdx.x;
    const int s = (int)(u / (uint32_t)Hq), h = (int)(u - (uint32_t)s * (uint32_t)Hq);
    const int n = partitions(decode_context(p, s, false), partition_of(p, s));
    if (n <= 1) return;  // stored by the decode kernel
    const int kvh = h / G;
    const size_t base = decode_unit(p, s, kvh) * p.max_splits * G + (h - kvh * G);  // (split 0, this head)
    const float4* o = reinterpret_cast<const float4*>(p.ws_o + base * D) + (lane < kCols ? lane : 0);
    const size_t row = (size_t)G * D / 4;
    float4 x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (warp + 4 * k < n) x[k] = __ldcg(o + (size_t)(warp + 4 * k) * row);
    const float2 ml = (int)threadIdx.x < n ? __ldcg(p.ws_ml + base + (size_t)threadIdx.x * G) : make_float2(-INFINITY, 0.f);
    const float mw = warp_max(ml.y != 0.f ? ml.x : -INFINITY);  // (a NaN sum stays in, and makes NaN of the output)
    if (lane == 0) warp_m[warp] = mw;
    __syncthreads();
    const float m = fmaxf(fmaxf(warp_m[0], warp_m[1]), fmaxf(warp_m[2], warp_m[3]));
    const float e = exp2f(0.5f * (ml.x - m));  // (twice, as in the kernel above)
    const float w = ml.y != 0.f ? ml.y * e * e : 0.f;
    weight[threadIdx.x] = w;
    const float ws = warp_sum(w);
    if (lane == 0) warp_w[warp] = ws;
    __syncthreads();
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = warp; i0 < n; i0 += 32) {
        if (i0 != warp) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (i0 + 4 * k < n) x[k] = __ldcg(o + (size_t)(i0 + 4 * k) * row);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (i0 + 4 * k >= n) break;
            const float wi = weight[i0 + 4 * k];
            acc.x = fmaf(wi, x[k].x, acc.x);
            acc.y = fmaf(wi, x[k].y, acc.y);
            acc.z = fmaf(wi, x[k].z, acc.z);
            acc.w = fmaf(wi, x[k].w, acc.w);
        }
    }
    if (lane < kCols) sums[warp][lane] = acc;
    __syncthreads();
    if (warp != 0 || lane >= kCols) return;
    const float total = (warp_w[0] + warp_w[1]) + (warp_w[2] + warp_w[3]);
    const float inv = total == 0.f ? 0.f : 1.f / total;
#pragma unroll
    for (int k = 1; k < 4; ++k) {
        const float4 v = sums[k][lane];
        acc.x += v.x;
        acc.y += v.y;
        acc.z += v.z;
        acc.w += v.w;
    }
    // (two-byte stores: `out` has no alignment to keep)
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + (size_t)u * D + lane * 4;
    out[0] = __float2bfloat16_rn(acc.x * inv);
    out[1] = __float2bfloat16_rn(acc.y * inv);
    out[2] = __float2bfloat16_rn(acc.z * inv);
    out[3] = __float2bfloat16_rn(acc.w * inv);
}

}  // namespace

int launch_decode_fp8_block_join(const DecodeParams& p, cudaStream_t stream) {
    if (p.max_splits <= 1) return PA_OK;
    const long long units = (long long)p.num_seqs * p.num_q_heads;
    if (p.max_splits > 128 || units > 0x7FFFFFFF) return PA_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)units), block(128);
    return p.head_dim == 64 ? launch_kernel(decode_fp8_block_join_kernel<64>, grid, block, 0, stream, p)
                            : launch_kernel(decode_fp8_block_join_kernel<128>, grid, block, 0, stream, p);
}

bool decode_fp8_block_tc_supported(const DecodeParams& p) {
    const int B = p.block_size;
    if (p.head_dim != kD || p.group > 8 || B < 8 || B > 128 || (B & (B - 1)) != 0) return false;
    if (((uintptr_t)p.k_cache & 15) || ((uintptr_t)p.v_cache & 15) || ((uintptr_t)p.q & 15)) return false;
    // (item numbers of a launch stay below 2^30)
    return (long long)p.num_blocks * B < (1LL << 31) && p.num_blocks > 0 && p.partition % kTok == 0 &&
           (long long)kMaxSeqs * p.num_kv_heads * p.max_splits < (1LL << 30);
}

int launch_decode_fp8_block_tc(const DecodeParams& p, int num_sms, cudaStream_t stream) {
    // up to kMaxSeqs sequences a launch; launches of one call follow one another on the stream and share the queue
    for (int s0 = 0; s0 < p.num_seqs; s0 += kMaxSeqs) {
        DecodeParams c = p;
        const size_t row = (size_t)s0 * p.num_q_heads * kD, unit = (size_t)s0 * p.num_kv_heads * p.max_splits * p.group;
        c.num_seqs = p.num_seqs - s0 < kMaxSeqs ? p.num_seqs - s0 : kMaxSeqs;
        c.out = static_cast<__nv_bfloat16*>(p.out) + row;
        c.q = static_cast<const __nv_bfloat16*>(p.q) + row;
        c.block_tables = p.block_tables + (size_t)s0 * p.max_blocks_per_seq;
        c.context_lens = p.context_lens + s0;
        c.small_from = p.small_from - s0;  // (negative: all of them)
        c.ws_ml = p.ws_ml + unit;
        c.ws_o = p.ws_o + unit * kD;
        const int rc = p.group <= 4 ? launch<4>(c, num_sms, stream) : launch<8>(c, num_sms, stream);
        if (rc != PA_OK) return rc;
    }
    return PA_OK;
}

}  // namespace pa
