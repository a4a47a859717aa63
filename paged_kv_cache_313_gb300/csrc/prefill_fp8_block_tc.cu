// prefill_fp8_block_tc.cu — causal chunked prefill over e4m3 pools with a scale
// per (block, kv head), on the 5th-generation tensor cores.
//
// What it computes: query i of chunk c, at position q_start_pos[c] + i, attends
// the keys up to its own position, K_j = code ks[block(j)], V_j = code vs[block(j)].
//
// A work item is (query tile, kv head, chunk, span of keys).  A tile is 128
// rows: 128 / G positions times the G query heads of the kv head.  Keys come
// in tiles of 128, one TMA box per block.
//
// Products.
//   S = Q K^T   kind::f8f6f4, 128 x 128 x 128: K as the box left it.  The
//               queries, scaled by a power of two that puts a row's largest
//               magnitude in [128, 256), are two e4m3 terms hi + lo that both
//               accumulate into S: a bf16's 8 bits exactly, but for elements
//               below 2^-10 of the row's largest (off by 2^-17 of it at most).
//   O += P V    kind::f16: V's codes widened to f16 (exact) in shared memory by
//               four converter warps, P in f16 in tensor memory, over the S it
//               came from.  (P as two e4m3 terms would spare the widening, but
//               its floor, 2^-17 of the largest weight, is too coarse for long
//               diffuse contexts, and the split costs twice the widening.)
// ks multiplies a key's scores; vs is part of the exponent, P' = 2^(x + log2(vs) - m)
// with m the running maximum of x + log2(vs), so it costs nothing per element and
// a row's largest P' is about 1 whatever the scales: f16's floor, 2^-25, is relative
// to the row's own largest p vs, not to blocks that it gives no weight or does not
// see.  The softmax's sum takes the float P' of 8 keys of one block (of 32 where
// blocks have 32 keys) times 1 / vs.
//
// Two softmax groups of four warps, a thread per row, take alternate pieces of
// 64 keys (a half of every key tile each), with their own running maximum, sum
// and O, joined once per item.  S is a ring of three pieces in tensor memory:
// while a group is at one, its next is there already, so that neither waits for
// the chain P -> P V -> Q K^T.  The query terms are in tensor memory too: as
// shared-memory operands they were read again by every product, and shared
// memory bandwidth set the pace (2.65k cycles per key tile against 1.0k of
// tensor work).  The maximum is lazy: it is looked for, and O rescaled, only
// when a piece's weights under the old one come to more than 2^9.
//
// Few rows: the plan cuts the keys of a tile into spans, whose partial results
// (float, in the workspace) a second kernel joins.
//
//   warps 0-7   softmax, group w / 4            warp 13  K tiles, masks, scales
//   warps 8-11  V widening, query terms         warp 14  V tiles
//   warp 12     tensor memory, issue of P V     warp 15  issue of Q K^T
// Waits are bounded, copies and MMAs drained, as in prefill_tc.cu.
//
// Bound: the softmax warps' issue and the hand-overs between the warps (the two
// products are 1.05k cycles of a key tile's 2.0k).  Measured: 2048 queries at
// position 5,916, 64/8 heads, 391 us over 64-token blocks (466 GFLOP: 1.19
// PFLOP/s, 0.61 of cuBLAS bf16; 407 among other calls) and 401 over 16-token
// blocks, whose copies are four times as many; four chunks of 512 queries at
// short offsets, 32/8 heads, 33.0 us; 37 queries at 2,955 16.5 us.  On the CUDA
// cores the last two take 4.9 and 1.2 ms.
#include <algorithm>
#include <climits>

#include "pa_internal.cuh"
#include "sm100_ptx.cuh"

namespace pa {
namespace {

constexpr int kD = 128;
constexpr int kTile = 128;             // rows of a query tile, keys of a key tile
constexpr int kCodes = kTile * kD;     // bytes of a tile of codes
constexpr int kHalfBytes = kTile * 128;  // bytes of a 64-column half of a widened tile
constexpr int kThreads = 512;
constexpr int kConverters = 4, kConvWarp = 8, kMmaWarp = 12, kKWarp = 13, kVWarp = 14, kSWarp = 15;
constexpr int kKStages = 4, kVStages = 3, kVhStages = 2, kInfo = 8;
// The converters may be two items ahead of the softmax (items of one key tile), never four: four slots keep an item's
// query factors, and the phase of its barrier, until the softmax has come to it.
constexpr int kQSlots = 4;
constexpr int kPieces = 3;  // ring of S pieces
constexpr int kNanSlots = 8;  // a slot is reset two items before its own, when the softmax is past its last use
constexpr int kItems = 8;   // ring of item descriptions
// tensor memory columns: O of group 0 and 1, the query terms (hi, lo; four codes a column), the S pieces
constexpr uint32_t kTO = 0, kTQ = 256, kTS = 320;
constexpr float kMost = 512.f;  // largest sum of a piece's weights before a row's maximum is looked for again
constexpr float kTiny = 1e-37f;  // the least factor of a score: 0 would make NaN of a masked key's -inf
// A V scale counts as at least 2^-80 of the item's largest so far and 2^-100 (the smallest that the write makes), so
// that the weights of its keys stay in float's range; what such a V adds is below 2^-71 of that largest scale.
constexpr float kHold = 8.271806125530277e-25f, kLeastScale = 7.888609052210118e-31f;

// shared memory, offsets from a 1024-aligned base
constexpr int kQ = 0;  // [hi, lo][128 rows][128], 16-byte pieces swizzled by row: staged for tensor memory
constexpr int kK = kQ + 2 * kCodes;
constexpr int kV = kK + kKStages * kCodes;
constexpr int kVh = kV + kVStages * kCodes;
constexpr int kConsts = kVh + kVhStages * 2 * kHalfBytes;  // float4 [kInfo][16]: per 8 keys ks', log2(vs), 1/vs
constexpr int kMask = kConsts + kInfo * 16 * 16;           // uint32 [kInfo][4]
constexpr int kVMask = kMask + kInfo * 16;                 // uint32 [kVStages][4]: the same for the converters
constexpr int kQf = kVMask + kVStages * 16;                // float [kQSlots][128]
constexpr int kState = kQf + kQSlots * kTile * 4;          // float2 [2 items][2 groups][128]: m, l
constexpr int kNan = kState + 2 * 2 * kTile * 8;           // int [kNanSlots][kD + 1]: see clear_nans
constexpr int kItem = (kNan + kNanSlots * (kD + 1) * 4 + 15) / 16 * 16;  // Item [kItems]
constexpr int kBars = kItem + kItems * 48;
constexpr int kNumBars = 2 * kKStages + 2 * kVStages + kVhStages + 3 * kPieces + kQSlots + 1 + kInfo + 2 * kItems + 3;
constexpr int kTmemSlot = kBars + kNumBars * 8;
constexpr size_t kSmemBytes = 1024 + kTmemSlot + 16;
static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");

// A work item as the warps pass it on; nt key tiles from tile t0 on, nt < 0: no more items.
struct Item {
    int kvh, row, nq, pos;  // kv head; first query (row of q) and their number; position of the first
    int last_key, t0, nt;   // the tile's last visible key
    int s, span, spans, pad[2];
};

struct Bars {
    uint64_t* base;
    __device__ uint64_t* k_full(int i) const { return base + i; }
    __device__ uint64_t* k_empty(int i) const { return base + kKStages + i; }
    __device__ uint64_t* v_full(int i) const { return base + 2 * kKStages + i; }
    __device__ uint64_t* v_empty(int i) const { return v_full(kVStages + i); }
    __device__ uint64_t* vh_full(int i) const { return v_full(2 * kVStages + i); }
    __device__ uint64_t* s_full(int i) const { return vh_full(kVhStages + i); }
    __device__ uint64_t* p_full(int i) const { return s_full(kPieces + i); }
    __device__ uint64_t* pv_done(int i) const { return s_full(2 * kPieces + i); }
    __device__ uint64_t* q_full(int i) const { return pv_done(kPieces + i); }
    __device__ uint64_t* q_empty() const { return q_full(kQSlots); }
    __device__ uint64_t* info(int i) const { return q_full(kQSlots + 1 + i); }
    __device__ uint64_t* item_full(int i) const { return info(kInfo + i); }
    __device__ uint64_t* item_empty(int i) const { return item_full(kItems + i); }
    __device__ uint64_t* o_free() const { return item_full(2 * kItems); }
    __device__ uint64_t* joined() const { return item_full(2 * kItems + 2); }  // the softmax warps' barrier
    __device__ uint64_t* drain() const { return item_full(2 * kItems + 1); }  // by both issuing warps
};

// The kernel's own parameters: the plan's key tiles per span and spans per tile, and what items are numbered by.
struct Spans {
    int tiles, count;
    int items;  // query tiles x chunks x kv heads x spans
    Divisor per_rank, per_count, per_heads, per_tiles, per_ppt;
    float* o;    // [count][total_q][num_q_heads][kD]
    float2* ml;  // [count][total_q][num_q_heads]
};

// A 32-byte global store (the address 32-byte aligned).
__device__ __forceinline__ void store32(void* ptr, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(ptr), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// One piece's S (64 keys): two query terms in tensor memory (32 columns each from `a`), four steps of 32 dims, K
// rows described by (lo, hi); `bar`, and `bar2` if given, complete with it.  And one piece's P V: four steps of 16 keys.
// Each is one election, its MMAs and commits: the issuing warp shares its scheduler with three busy ones, so its
// instructions are counted.
__device__ __forceinline__ void issue_s(uint32_t d, uint32_t a, uint32_t lo, uint32_t hi, uint32_t idesc, uint64_t* bar,
                                        uint64_t* bar2) {
#define PA_STEP(A, B, ACC)                                                                     \
    "add.u32 t, %1, " A ";\n\tadd.u32 l, %2, " B ";\n\tmov.b64 b, {l, %3};\n\t"               \
    "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [t], b, %4, " ACC ";\n\t"
    asm volatile(
        "{\n\t.reg .pred e, y, n;\n\t.reg .b32 t, l;\n\t.reg .b64 b;\n\t"
        "setp.eq.u32 y, 0, 0;\n\tsetp.ne.u32 n, 0, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
        PA_STEP("0", "0", "n") PA_STEP("8", "2", "y") PA_STEP("16", "4", "y") PA_STEP("24", "6", "y")
        PA_STEP("32", "0", "y") PA_STEP("40", "2", "y") PA_STEP("48", "4", "y") PA_STEP("56", "6", "y")
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n\t"
        "setp.ne.u32 y, %6, 0;\n\tand.pred e, e, y;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%6];\n\t"
        "}" ::"r"(d), "r"(a), "r"(lo), "r"(hi), "r"(idesc), "r"(smem_u32(bar)), "r"(bar2 ? smem_u32(bar2) : 0u)
        : "memory");
#undef PA_STEP
}
__device__ __forceinline__ void issue_o(uint32_t d, uint32_t a, uint32_t lo, uint32_t hi, uint32_t idesc,
                                        uint32_t accumulate, uint64_t* bar) {
#define PA_STEP(A, B, ACC)                                                                     \
    "add.u32 t, %1, " A ";\n\tadd.u32 l, %2, " B ";\n\tmov.b64 b, {l, %3};\n\t"               \
    "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [t], b, %4, " ACC ";\n\t"
    asm volatile(
        "{\n\t.reg .pred e, y, f;\n\t.reg .b32 t, l;\n\t.reg .b64 b;\n\t"
        "setp.eq.u32 y, 0, 0;\n\tsetp.ne.u32 f, %5, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
        PA_STEP("0", "0", "f") PA_STEP("8", "128", "y") PA_STEP("16", "256", "y") PA_STEP("24", "384", "y")
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%6];\n\t"
        "}" ::"r"(d), "r"(a), "r"(lo), "r"(hi), "r"(idesc), "r"(accumulate), "r"(smem_u32(bar)) : "memory");
#undef PA_STEP
}

// The queries of a chunk: first row, count, sequence and start; false when they make no sense.
__device__ __forceinline__ bool chunk_of(const PrefillParams& p, int c, int& r0, int& n, int& s, int& start) {
    r0 = p.cu_q_lens[c];
    n = p.cu_q_lens[c + 1] - r0;
    s = p.seq_of_chunk[c];
    start = p.q_start_pos[c];
    return n >= 0 && r0 >= 0 && r0 + n <= p.total_q && n <= p.max_q_len && s >= 0 && s < p.num_seqs && start >= 0;
}
// Keys that sequence s may be asked for.
__device__ __forceinline__ int key_cap(const PrefillParams& p, int s) {
    const long long table = (long long)p.max_blocks_per_seq * p.block_size;
    return (int)min(min((long long)p.context_lens[s], (long long)p.max_context_len), table);
}

// kKeys: keys that share a block, and so their factors, as far as the softmax goes by it: 8, 16 or 32 (the block size up
// to 32).  (2048 queries at 5,916 over 64-token blocks with 32 / 8: 391 / 433 us; over 16-token blocks with 16 / 8: 401 /
// 445.)
template <int kKeys>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_fp8_block_tc_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                                const PrefillParams p, const Spans spans) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const Bars bars{reinterpret_cast<uint64_t*>(smem + kBars)};
    uint32_t* mask = reinterpret_cast<uint32_t*>(smem + kMask);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kTmemSlot);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = p.group, B = p.block_size, Hkv = p.num_kv_heads;
    const int ppt = kTile / G;  // positions per tile; rows from ppt * G on are unused
    const int log2b = 31 - __clz(B);
    const uint32_t inv_g = (65536 + G - 1) / G;  // r / G = r * inv_g >> 16 for r < 128 and G <= 8 (checked for all)

    if (warp == 0) {  // the barriers, a lane each: in this order in memory, with these numbers of arrivals
        for (int i = lane; i < kNumBars; i += 32) {
            uint64_t* bar = bars.base + i;
            const bool conv = (bar >= bars.v_empty(0) && bar < bars.vh_full(kVhStages)) ||
                              (bar >= bars.q_full(0) && bar < bars.q_full(kQSlots));
            const int n = conv                                                        ? kConverters
                          : bar >= bars.p_full(0) && bar < bars.p_full(kPieces)       ? 4
                          : bar >= bars.item_empty(0) && bar < bars.item_empty(kItems) ? 8 + kConverters + 3  // every other warp
                          : bar == bars.o_free() || bar == bars.joined()              ? 8
                          : bar == bars.drain()                                       ? 2
                                                                                      : 1;
            mbar_init(bar, n);
        }
        fence_mbar_init();
    }
    for (int i = threadIdx.x; i < kNanSlots * (kD + 1); i += kThreads) reinterpret_cast<int*>(smem + kNan)[i] = INT_MAX;
    pdl_trigger();
    pdl_wait();
    if (warp == kMmaWarp) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    bool ok = true;
    // Item n, from the warp that describes them (every lane gets it; false at the end, or after a wait that gave up).
    auto take_item = [&](uint32_t n, Item& d) {
        if (!mbar_wait_warp(bars.item_full(n % kItems), (n / kItems) & 1)) {
            ok = false;
            return false;
        }
        d = *reinterpret_cast<const Item*>(smem + kItem + n % kItems * sizeof(Item));
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.item_empty(n % kItems));
        return d.nt >= 0;
    };

    // Registers: 128 a thread at launch (512 threads take all of the SM's).  The softmax warps get 152 of them, for 64
    // scores and what becomes of them, the others 104: 2 * 152 + 104 + 104 = 4 * 128.  No role may spill: eight bytes
    // spilled in the softmax took the long chunk from 387 to 416 us.
    if (warp >= kMmaWarp) asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == kKWarp || warp == kVWarp) {
        // ============================================================ producers
        const int bpt = kTile >> log2b, tpc = 32 / bpt;  // blocks per tile, tiles per 32-entry chunk of the table
        if (lane == 0) tma_prefetch_desc(warp == kVWarp ? &tmv : &tmk);
        // The V warp describes the items.  (query tile rank, chunk, kv head, span), the latest tile of every chunk
        // first; CTA b takes one of every pass of gridDim.x items, in serpentine order, so that heavy and light ones
        // pair up.  It stays an item ahead of its own copies: when every warp described its items itself, that took
        // each of them 3.3k cycles an item, between the epilogue of one and the first score of the next.
        const int num_items = spans.items;  // below 2^30
        const int passes = (num_items - 1) / (int)gridDim.x + 1;
        int pass = 0;
        uint32_t published = 0;
        auto describe = [&](Item& d) {  // the item of this pass; false for an empty one
            const int g = gridDim.x, b = blockIdx.x, k = pass * g + ((pass & 1) ? g - 1 - b : b);
            if (k >= num_items) return false;
            const int rank = spans.per_rank.div(k);
            int rem = k - rank * (int)spans.per_rank.d;
            const int unit = spans.per_count.div(rem), ch = spans.per_heads.div(unit);
            d.span = rem - unit * spans.count;
            d.kvh = unit - ch * Hkv;
            int r0, n, start;
            if (!chunk_of(p, ch, r0, n, d.s, start)) {
                if (rank == 0 && d.kvh == 0 && d.span == 0 && lane == 0) count_error(p.error_count);
                return false;
            }
            const int tiles = n > (1 << 29) ? (n + ppt - 1) / ppt : spans.per_ppt.div(n + ppt - 1);
            if (rank >= tiles) return false;
            const int i0 = (tiles - 1 - rank) * ppt;
            d.row = r0 + i0;
            d.nq = min(ppt, n - i0);
            d.pos = (int)min((long long)start + i0, 0x7FFFFFFELL - kTile);
            const int cap = key_cap(p, d.s);
            d.last_key = d.pos + d.nq - 1;
            if (d.last_key >= cap) {
                if (d.span == 0 && lane == 0) count_error(p.error_count);
                d.last_key = cap - 1;
            }
            const int all = d.last_key >= 0 ? d.last_key / kTile + 1 : 0;
            d.spans = spans.per_tiles.div(all + spans.tiles - 1);  // (tiles of 128 keys: below 2^25)
            d.t0 = d.span * spans.tiles;
            d.nt = min(spans.tiles, all - d.t0);
            if (all == 0 && d.span == 0) {
                // Without any key the output is zeros, stored here: every item that is passed on has keys.  (Passed on like
                // the others, such an item behind one of more tiles than the ring of V holds stopped the kernel: the
                // converters looked past it for their next one, this warp waited for them before it passed that on.)
#pragma unroll 1
                for (int r = 0; r < d.nq * G; ++r) {
                    const int pos = r * inv_g >> 16;
                    const size_t row = (size_t)(d.row + pos) * p.num_q_heads + d.kvh * G + (r - pos * G);
                    reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + row * kD)[lane] = make_uint2(0u, 0u);
                }
            }
            return d.span < d.spans;
        };
        auto publish = [&](Item& d) {  // the next item, or the end
            d.nt = -1;
            for (; pass < passes; ++pass)
                if (describe(d)) break;
                else d.nt = -1;
            ++pass;
            const int i = published % kItems;
            if (published >= kItems && !mbar_wait_warp(bars.item_empty(i), ((published / kItems) - 1) & 1)) {
                ok = false;
                d.nt = -1;
                return;
            }
            if (lane == 0) {
                *reinterpret_cast<Item*>(smem + kItem + i * sizeof(Item)) = d;
                mbar_arrive(bars.item_full(i));
            }
            __syncwarp();
            ++published;
        };
        // A tile of 16-token blocks is eight copies of about 75 cycles each to issue, so what else a warp does for it
        // counts (factors and ring indices worked out for every tile anew took 2.9k cycles a tile, longer than the
        // products).  One body for both sides: the warps share an instruction cache, and a body each, shorter as it was,
        // cost 4 %.
        {
            const bool v_side = warp == kVWarp;
            const uint32_t stages = v_side ? kVStages : kKStages;
            const CUtensorMap* map = v_side ? &tmv : &tmk;
            const uint32_t all = (1u << bpt) - 1u;
            uint64_t *const fulls = v_side ? bars.v_full(0) : bars.k_full(0), *const empties = v_side ? bars.v_empty(0) : bars.k_empty(0);
            uint32_t* const masks = v_side ? reinterpret_cast<uint32_t*>(smem + kVMask) : mask;
            const int my_blk = ((lane & 15) * 8) >> log2b;  // block, in its tile, of this lane's group of 8 keys
            uint8_t* my_dst = smem + (v_side ? kV : kK) + (lane << log2b) * kD;
            uint32_t g = 0, items = 0, st = 0, round = 0;  // key tiles and items so far; the ring's stage and its round
            Item d{}, ahead{};  // (the V warp's first has no tiles, so that there is one place to publish from)
            for (; ok; ++items) {
                if (v_side) {
                    d = ahead;
                    if (d.nt < 0) break;
                    publish(ahead);
                } else if (!take_item(items, d)) {
                    break;
                }
                const int first = d.t0 * bpt;  // first block
                const int nblk = min((d.last_key + B) >> log2b, (d.t0 + d.nt) * bpt) - first;
                const int32_t* table = p.block_tables + (size_t)d.s * p.max_blocks_per_seq + first;
                auto load_raw = [&](int chunk) {
                    const int i = chunk * 32 + lane;
                    return i < nblk ? table[i] : -1;
                };
                auto load_scales = [&](int pb) {
                    if (v_side || pb < 0 || pb >= p.num_blocks) return make_float2(0.f, 0.f);
                    const size_t i = (size_t)pb * Hkv + d.kvh;
                    return make_float2(__ldg(p.k_scales + i), __ldg(p.v_scales + i));
                };
                int raw = d.nt > 0 ? load_raw(0) : -1, token = -1;  // table entry of this lane's block, its first token
                float2 sc = load_scales(raw);
                uint32_t valid = 0;                       // the chunk's blocks with a valid table entry
                float ks = 0.f, off = 0.f, inv_vs = 0.f;  // of this lane's block: what the softmax needs of it
                float top = 0.f;                          // the largest V scale of the item so far
                int keys = d.last_key + 1 - d.t0 * kTile;  // visible from this tile on
                for (int j = 0, chunk = 0, l = 0; j < d.nt; ++j, ++g, keys -= kTile) {
                    if (l == 0) {
                        const bool valid_raw = raw >= 0 && raw < p.num_blocks;
                        if (!v_side && !valid_raw && chunk * 32 + lane < nblk) count_error(p.error_count);
                        token = valid_raw ? raw << log2b : -1;
                        valid = __ballot_sync(0xffffffffu, valid_raw);
                        if (!v_side) {
                            top = fmaxf(top, redux_max(sc.y));
                            ks = sc.x * fabsf(p.scale_log2);
                            off = __log2f(fmaxf(sc.y, fmaxf(top * kHold, kLeastScale)));
                            inv_vs = exp2f(-off);  // (a subnormal beyond a scale of 2^126, where fast_exp2 gives 0)
                        }
                    }
                    const uint32_t mine = (valid >> (l * bpt)) & all;
                    uint64_t* full = fulls + st;
                    if (round > 0 && !mbar_wait_warp(empties + st, (round - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    const int slot = g % kInfo;
                    if (lane < 4) {  // key-validity mask: 32 keys a word
                        uint32_t m = ~0u;
                        if (mine != all || keys < kTile) {
                            const int left = keys - 32 * lane;
                            m = left >= 32 ? ~0u : left > 0 ? (1u << left) - 1u : 0u;
                            if (B >= 32) {
                                if (!((mine >> ((32 * lane) >> log2b)) & 1u)) m = 0u;
                            } else {
                                const int per = 32 >> log2b;
                                for (int b = 0; b < per; ++b)
                                    if (!((mine >> (lane * per + b)) & 1u)) m &= ~(((1u << B) - 1u) << (b * B));
                            }
                        }
                        masks[(v_side ? st : slot) * 4 + lane] = m;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)__popc(mine) << (log2b + 7));
                    const int my_token = __shfl_sync(0xffffffffu, token, l * bpt + lane);
                    __syncwarp();  // armed before any copy is issued
                    if (lane < bpt && my_token >= 0) tma_load_3d(my_dst + st * kCodes, map, 0, my_token, d.kvh, full);
                    if (!v_side) {
                        // what the softmax needs of this tile's 16 groups of 8 keys
                        const int blk = l * bpt + my_blk;
                        const float a = __shfl_sync(0xffffffffu, ks, blk), o = __shfl_sync(0xffffffffu, off, blk);
                        const float z = __shfl_sync(0xffffffffu, inv_vs, blk);
                        if (lane < 16) reinterpret_cast<float4*>(smem + kConsts)[slot * 16 + lane] = make_float4(a, o, z, 0.f);
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bars.info(slot));
                    }
                    if (++st == stages) st = 0, ++round;
                    // the next chunk's entries, at the end of this one's first tile, and their scales a tile later
                    if (l == 0) raw = load_raw(chunk + 1);
                    if (l == 1) sc = load_scales(raw);  // (a chunk has two tiles at least)
                    if (++l == tpc) l = 0, ++chunk;
                }
            }
            if (lane == 0) {
                if (!ok) count_error(p.error_count);
                if (!drain_ring(fulls, stages, g)) count_error(p.error_count);
            }
            __syncwarp();
        }
    } else if (warp == kMmaWarp || warp == kSWarp) {
        // ============================================================ MMA issuers
        // Warp kSWarp issues every piece's S = Q K^T, warp kMmaWarp every piece's O += P V: one warp doing both in
        // turn took 1.55k cycles a piece, most of it in waking up and in queueing behind its own last product.
        const bool s_side = warp == kSWarp;
        constexpr uint32_t idesc_s = umma_idesc_e4m3(128, 64, false, false);
        // kind::f16 with f16 operands (format 0), V MN-major
        constexpr uint32_t idesc_o = (1u << 4) | (1u << 16) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
        const uint64_t dk0 = umma_desc_sw128(smem_u32(smem + kK), 16, 1024);
        const uint64_t dv0 = umma_desc_sw128(smem_u32(smem + kVh), kHalfBytes, 1024);
        // (the same in every lane; said so, it goes to the uniform registers that an MMA's operands need)
        auto uniform = [](uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); };
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            if (ok && !mbar_wait_warp(bar, parity)) ok = false;
            return ok;
        };
        uint32_t g = 0, items = 0, sb = 0, round = 0;  // key tiles, items; the piece's buffer and its round
        Item d;
        for (uint32_t n = 0; ok && take_item(n, d); ++n) {
            const uint32_t nt = uniform(d.nt);
            // an item's first S waits for its query terms, its first product until the last item's epilogue has read O
            if (s_side) wait(bars.q_full(items % kQSlots), (items / kQSlots) & 1);
            else if (items > 0) wait(bars.o_free(), (items - 1) & 1);
            for (uint32_t j = 0; j < nt && ok; ++j, ++g) {
                const uint32_t st = g % kKStages, vh = g % kVhStages;
                if (s_side) wait(bars.k_full(st), (g / kKStages) & 1);
                else wait(bars.vh_full(vh), (g / kVhStages) & 1);
#pragma unroll
                for (uint32_t x = 0; x < 2; ++x) {
                    if (s_side) {
                        if (round > 0 && !wait(bars.pv_done(sb), (round - 1) & 1)) break;
                        tc_fence_after();
                        issue_s(tmem + kTS + sb * 64, tmem + kTQ,
                                (uint32_t)dk0 + ((st * kCodes + x * 64 * kD) >> 4), (uint32_t)(dk0 >> 32), idesc_s,
                                bars.s_full(sb), x ? bars.k_empty(st) : nullptr);
                        if (x && j == nt - 1) umma_commit_warp(bars.q_empty());
                    } else {
                        if (!wait(bars.p_full(sb), round & 1)) break;
                        tc_fence_after();
                        issue_o(tmem + kTO + x * 128, tmem + kTS + sb * 64,
                                (uint32_t)dv0 + ((vh * 2 * kHalfBytes + x * 64 * 128) >> 4), (uint32_t)(dv0 >> 32),
                                idesc_o, j, bars.pv_done(sb));  // which frees the piece, and with its second the widened V
                    }
                    if (++sb == kPieces) sb = 0, ++round;
                }
            }
            ++items;
        }
        if (!ok && lane == 0) count_error(p.error_count);
        umma_commit_warp(bars.drain());  // no MMA is running when the tensor memory is freed
        if (!mbar_wait_warp(bars.drain(), 0) && lane == 0) count_error(p.error_count);
        __syncwarp();
    } else if (warp >= kConvWarp && warp < kMmaWarp) {
        // ============================================================ converters
        asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        const int w = warp - kConvWarp;
        uint32_t g = 0, items = 0;
        // an item's query rows, half a row a lane and 16 rows at a time (a whole row a lane takes 64 registers for the row
        // alone): two e4m3 terms staged in shared memory, and the factor that undoes their scaling.  In f16, which holds a
        // scaled bf16 exactly down to 2^-24.
        auto stage_q = [&](const Item& d, uint32_t item) {
            // (a converter is less than two key tiles, so two items, ahead of another: no one has written there yet)
            int* nan = reinterpret_cast<int*>(smem + kNan) + (item + 2) % kNanSlots * (kD + 1);
            nan[w * 32 + lane] = INT_MAX;
            if (w == 0 && lane == 0) nan[kD] = INT_MAX;
            const int half = lane & 1;
#pragma unroll 1
            for (int r = w * 32 + (lane >> 1), end = r + 32; r < end; r += 16) {
                const int pos = r * inv_g >> 16;
                const uint4* src = reinterpret_cast<const uint4*>(
                    static_cast<const __nv_bfloat16*>(p.q) +
                    ((size_t)(d.row + pos) * p.num_q_heads + d.kvh * G + (r - pos * G)) * kD) + half * (kD / 16);
                uint4 x[kD / 16];
#pragma unroll
                for (int k = 0; k < kD / 16; ++k) x[k] = pos < d.nq ? __ldg(src + k) : make_uint4(0u, 0u, 0u, 0u);
                uint32_t m2 = 0;
#pragma unroll
                for (int k = 0; k < kD / 16; ++k)
                    m2 = __vmaxu2(m2, __vmaxu2(__vmaxu2(x[k].x & 0x7FFF7FFFu, x[k].y & 0x7FFF7FFFu),
                                               __vmaxu2(x[k].z & 0x7FFF7FFFu, x[k].w & 0x7FFF7FFFu)));
                m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, 1));
                const uint32_t am = max(m2 & 0xFFFFu, m2 >> 16);
                const int e = min(134 - (int)(am >> 7), 126);  // |x| 2^e in [128, 256)
                // a negative softmax scale negates the queries, so that scores only meet positive factors; a row with an
                // infinity or a NaN becomes NaN (the conversion would hold an infinity at 448)
                const float f = am >= 0x7F80u ? NAN : copysignf(__uint_as_float((uint32_t)(e + 127) << 23), p.scale_log2);
                uint8_t* row = smem + kQ + r * kD;
#pragma unroll
                for (int k = 0; k < kD / 32; ++k) {
                    const uint32_t in[8] = {x[2 * k].x,     x[2 * k].y,     x[2 * k].z,     x[2 * k].w,
                                            x[2 * k + 1].x, x[2 * k + 1].y, x[2 * k + 1].z, x[2 * k + 1].w};
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t c[2], b[2];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint32_t v = in[2 * i + j];
                            const uint32_t h =
                                pack_f16x2(__uint_as_float(v << 16) * f, __uint_as_float(v & 0xFFFF0000u) * f);
                            c[j] = e4m3x2_of_f16x2(h);
                            b[j] = e4m3x2_of_f16x2(sub_f16x2(h, e4m3x2_to_f16x2(c[j])));
                        }
                        hi[i] = c[0] | (c[1] << 16);
                        lo[i] = b[0] | (b[1] << 16);
                    }
                    const int at = ((half * 4 + k) ^ (r & 7)) << 4;
                    *reinterpret_cast<uint4*>(row + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4*>(row + kCodes + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                if (half == 0)
                    reinterpret_cast<float*>(smem + kQf)[item % kQSlots * kTile + r] = __uint_as_float((uint32_t)(127 - e) << 23);
            }
        };
        // the staged rows into tensor memory (a lane's row is its tensor-memory lane), once the item before is through
        // its last S
        auto finish_q = [&](uint32_t item) {
            __syncwarp();
            if (item > 0 && !mbar_wait_warp(bars.q_empty(), (item - 1) & 1)) {
                ok = false;
                return;
            }
            tc_fence_after();
            const int r = w * 32 + lane;
#pragma unroll
            for (int term = 0; term < 2; ++term) {
                uint32_t v[32];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint4 x = *reinterpret_cast<const uint4*>(smem + kQ + term * kCodes + r * kD + ((k ^ (r & 7)) << 4));
                    v[4 * k] = x.x;
                    v[4 * k + 1] = x.y;
                    v[4 * k + 2] = x.z;
                    v[4 * k + 3] = x.w;
                }
                tmem_st32u(tmem + ((uint32_t)(w * 32) << 16) + kTQ + term * 32, v);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.q_full(item % kQSlots));
        };
        // NaN codes in a tile whose keys not every row sees would reach every row through P = 0.  They are cleared, and
        // the first key with one is noted for its column (and for all columns, at kD): the output of the rows that see
        // it becomes NaN there.  This lane's codes are 16 bytes of every 16th key.
        auto clear_nans = [&](uint8_t* src, int column, int key0, int first_key, const uint32_t* valid, uint32_t item) {
            int* nan = reinterpret_cast<int*>(smem + kNan) + item % kNanSlots * (kD + 1);
#pragma unroll 1
            for (int i = 0; i < kTile / 16; ++i) {
                const int key = key0 + 16 * i;
#pragma unroll 1
                for (int b = 0; b < 16; ++b) {
                    uint8_t* code = src + i * 16 * kD + b;
                    if ((*code & 0x7f) != 0x7f) continue;
                    *code = 0;
                    if (!((valid[key >> 5] >> (key & 31)) & 1u)) continue;
                    atomicMin(nan + column + b, first_key + key);
                    atomicMin(nan + kD, first_key + key);
                }
            }
            fence_proxy_async_smem();  // before the buffer is copied to again
        };
        Item d, nx;
        bool have = take_item(0, d);
        if (have) {
            stage_q(d, 0);
            finish_q(0);
        }
        while (have && ok) {
            const bool have_next = take_item(items + 1, nx);
            if (!ok) break;
            for (int j = 0; j < d.nt; ++j, ++g) {
                const uint32_t vs = g % kVStages, vh = g % kVhStages;
                const uint32_t last = 2 * (g - kVhStages) + 1;  // the piece that read this buffer last
                // a lane widens 16 codes of a key, 8 lanes a key; a warp takes keys 16 i + 4 w .. + 3, whose swizzle is
                // the same for every i.  The codes are loaded while the buffer is still being read.
                const uint32_t key0 = 4 * w + (lane >> 3), ch = lane & 7, sw = key0 & 7;
                uint8_t* src = smem + kV + vs * kCodes + key0 * kD + ((ch ^ sw) << 4);
                uint8_t* dst = smem + kVh + vh * 2 * kHalfBytes + (ch >> 2) * kHalfBytes + key0 * 128;
                uint8_t *dst0 = dst + ((((ch & 3) * 2) ^ sw) << 4), *dst1 = dst + ((((ch & 3) * 2 + 1) ^ sw) << 4);
                if (!mbar_wait_warp(bars.v_full(vs), (g / kVStages) & 1)) {
                    ok = false;
                    break;
                }
                const int first_key = (d.t0 + j) * kTile;
                if (first_key + kTile - 1 > d.pos) {
                    uint32_t bad = 0;
#pragma unroll 2
                    for (int i = 0; i < kTile / 16; ++i) {
                        const uint4 c = *reinterpret_cast<const uint4*>(src + i * 16 * kD);
                        bad |= ((c.x & 0x7F7F7F7Fu) + 0x01010101u) | ((c.y & 0x7F7F7F7Fu) + 0x01010101u) |
                               ((c.z & 0x7F7F7F7Fu) + 0x01010101u) | ((c.w & 0x7F7F7F7Fu) + 0x01010101u);
                    }
                    if (bad & 0x80808080u)
                        clear_nans(src, ch * 16, key0, first_key, reinterpret_cast<const uint32_t*>(smem + kVMask + vs * 16),
                                   items);
                    __syncwarp();
                }
                uint4 x[kTile / 16];
#pragma unroll
                for (int i = 0; i < kTile / 16; ++i) x[i] = *reinterpret_cast<const uint4*>(src + i * 16 * kD);
                const uint4 m = *reinterpret_cast<const uint4*>(smem + kVMask + vs * 16);
                if ((m.x & m.y & m.z & m.w) != ~0u) {
#pragma unroll
                    for (int i = 0; i < kTile / 16; ++i) {
                        const uint32_t word = i < 2 ? m.x : i < 4 ? m.y : i < 6 ? m.z : m.w;
                        if (!((word >> ((i & 1) * 16 + key0)) & 1u)) x[i] = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bars.v_empty(vs));
                if (g >= kVhStages && !mbar_wait_warp(bars.pv_done(last % kPieces), (last / kPieces) & 1)) {
                    ok = false;
                    break;
                }
#pragma unroll
                for (int i = 0; i < kTile / 16; ++i) {
                    const uint32_t in[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                    uint32_t out[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        out[2 * k] = e4m3x2_to_f16x2(in[k] & 0xFFFFu);
                        out[2 * k + 1] = e4m3x2_to_f16x2(in[k] >> 16);
                    }
                    *reinterpret_cast<uint4*>(dst0 + i * 16 * 128) = make_uint4(out[0], out[1], out[2], out[3]);
                    *reinterpret_cast<uint4*>(dst1 + i * 16 * 128) = make_uint4(out[4], out[5], out[6], out[7]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bars.vh_full(vh));
                if (j == 0 && have_next) stage_q(nx, items + 1);  // early, while the softmax is at this item's first keys
            }
            if (!ok) break;
            if (have_next) finish_q(items + 1);
            ++items;
            have = have_next;
            d = nx;
        }
        if (!ok && lane == 0) count_error(p.error_count);
    } else if (warp < kConvWarp) {
        // ============================================================ softmax and output
        asm volatile("setmaxnreg.inc.sync.aligned.u32 152;");
        const int x = warp >> 2;                       // group
        const int r = (warp & 3) * 32 + lane;          // row = tensor-memory lane
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t t_o = tmem + lanes + kTO + x * 128;
        float2* state = reinterpret_cast<float2*>(smem + kState);
        uint32_t g = 0;  // key tiles (pieces of this group)
        BoundedWarpBarrier joined{bars.joined(), 0};
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            if (ok && !mbar_wait_warp(bar, parity)) ok = false;
        };
        const bool out_al32 = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
        const int my_pos = r * inv_g >> 16;  // the row's position in a tile, and its head of the group
        for (uint32_t n = 0;; ++n) {
            // (the item's description stays in shared memory until the end of its epilogue, for the registers' sake)
            wait(bars.item_full(n % kItems), (n / kItems) & 1);
            if (!ok) break;
            const Item& d = *reinterpret_cast<const Item*>(smem + kItem + n % kItems * sizeof(Item));
            if (d.nt < 0) break;
            const uint32_t end = g + d.nt;
            const int my_last = min(d.pos + min(my_pos, d.nq - 1), d.last_key);  // (unused rows mask as the last used one)
            const int least_last = __reduce_min_sync(0xffffffffu, my_last);
            float m = -INFINITY, l = 0.f, qf = 0.f;
            int key0 = d.t0 * kTile + x * 64;  // the piece's first key
            wait(bars.q_full(n % kQSlots), (n / kQSlots) & 1);
            qf = reinterpret_cast<const float*>(smem + kQf)[n % kQSlots * kTile + r];
            bool first = true, open = true;  // nothing in O yet; there are rows without a key so far
            for (; g != end; ++g, key0 += kTile, first = false) {
                const uint32_t piece = 2 * g + x, sb = piece % kPieces, t_s = tmem + lanes + kTS + sb * 64;
                const int slot = g % kInfo;
                wait(bars.info(slot), (g / kInfo) & 1);
                const float4* kc = reinterpret_cast<const float4*>(smem + kConsts) + slot * 16 + x * 8;
                // (all of this before the wait for S, which it does not need)
                const uint2 vm = *reinterpret_cast<const uint2*>(mask + slot * 4 + x * 2);
                const bool dense = key0 + 63 <= least_last && (vm.x & vm.y) == ~0u;  // every key, for every row of the warp
                // The weights are taken with the maximum so far.  Only when a row's 64 of them come to more than 2^9
                // (which is how a larger one shows, without a pass for the maximum) or a row has seen no key yet, the
                // maximum is looked for, O brought to it, and the weights taken again.
                bool look = open;
                constexpr bool kAhead = kKeys >= 16;  // up to four blocks' factors are read ahead, eight blocks' where they are used
                float4 k4[kAhead ? 64 / kKeys : 1];
                auto factors = [&](int b) {
                    float4 f = kc[b * kKeys / 8];
                    f.x = fmaxf(f.x * qf, kTiny);
                    return f;
                };
                if constexpr (kAhead) {
#pragma unroll
                    for (int b = 0; b < 64 / kKeys; ++b) k4[b] = factors(b);
                }
                uint32_t pk[32];
                float sum, most;
                wait(bars.s_full(sb), (piece / kPieces) & 1);
                if (!ok) break;
                tc_fence_after();
                while (true) {
                    float s[64];
                    {
                        float a[32], b[32];
                        tmem_ld32(t_s, a);
                        tmem_ld32(t_s + 32, b);
#pragma unroll
                        for (int i = 0; i < 32; ++i) s[i] = a[i], s[32 + i] = b[i];
                    }
                    tmem_wait_ld();
                    if (!dense) {  // the row's visible and valid keys as 64 bits
                        const uint2 v = *reinterpret_cast<const uint2*>(mask + slot * 4 + x * 2);
                        const int vis = my_last - key0 + 1;
                        const uint32_t w0 = v.x & (vis >= 32 ? ~0u : vis > 0 ? (1u << vis) - 1u : 0u);
                        const uint32_t w1 = v.y & (vis >= 64 ? ~0u : vis > 32 ? (1u << (vis - 32)) - 1u : 0u);
#pragma unroll
                        for (int k = 0; k < 64; ++k)
                            if (!((k < 32 ? w0 : w1) & (1u << (k & 31)))) s[k] = -INFINITY;
                    }
                    if (look) {
                        float mt = m;
#pragma unroll
                        for (int b = 0; b < 64; b += kKeys) {
                            float u[2] = {s[b], s[b + 1]};
#pragma unroll
                            for (int i = 2; i < kKeys; i += 2) u[i / 2 & 1] = fmax3(u[i / 2 & 1], s[b + i], s[b + i + 1]);
                            const float4 f = kAhead ? k4[kAhead ? b / kKeys : 0] : factors(b / kKeys);
                            mt = fmaxf(mt, fmaf(fmaxf(u[0], u[1]), f.x, f.y));
                        }
                        if (!first) {
                            // the products issued so far have to be done before O changes
                            wait(bars.pv_done((piece - 2) % kPieces), ((piece - 2) / kPieces) & 1);
                            tc_fence_after();
                            // (the factor's square root, twice for the sum: the maxima have the V scales in them and may
                            // be 2^220 apart between keys of the same weight, and the sum, divided by the scales, keeps
                            // what one factor would flush to 0)
                            const float root = mt == m ? 1.f : fast_exp2(0.5f * (m - mt)), alpha = root * root;
#pragma unroll 1
                            for (int q = 0; q < 8; ++q) {
                                float o[16];
                                tmem_ld16(t_o + q * 16, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 16; ++i) o[i] *= alpha;
                                tmem_st16(t_o + q * 16, o);
                            }
                            tmem_wait_st();
                            l = l * root * root;
                        }
                        m = mt;
                        open = __any_sync(0xffffffffu, m == -INFINITY);
                    }
                    sum = most = 0.f;
                    const float m_fin = m == -INFINITY ? 0.f : m;  // no key yet: every P' is 2^-inf
#pragma unroll
                    for (int b = 0; b < 64; b += kKeys) {
                        const float4 f = kAhead ? k4[kAhead ? b / kKeys : 0] : factors(b / kKeys);
                        const float a = f.x, o = f.y - m_fin;
                        const unsigned long long a2 = f32x2_pack(a, a), o2 = f32x2_pack(o, o);
                        unsigned long long part[2];  // the keys' weights, in pairs and two chains
#pragma unroll
                        for (int i = 0; i < kKeys / 2; ++i) {
                            float y0, y1;
                            f32x2_unpack(fma_f32x2(f32x2_pack(s[b + 2 * i], s[b + 2 * i + 1]), a2, o2), y0, y1);
                            const float e0 = fast_exp2(y0), e1 = fast_exp2(y1);
                            pk[b / 2 + i] = pack_f16x2(e0, e1);
                            part[i & 1] = i < 2 ? f32x2_pack(e0, e1) : add_f32x2(part[i & 1], f32x2_pack(e0, e1));
                        }
                        float u, v;
                        f32x2_unpack(add_f32x2(part[0], part[1]), u, v);
                        most += u + v;
                        sum = fmaf(u + v, f.z, sum);
                    }
                    if (look || !__any_sync(0xffffffffu, most > kMost)) break;
                    look = true;
                }
                {
                    l += sum;
                    tmem_st32u(t_s, pk);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0 && ok) mbar_arrive(bars.p_full(sb));
                }
            }
            // ---- the item's output: both groups' states joined, each group stores 64 columns of the row
            if (!ok) break;
            float mo, lo;
            {
                const uint32_t last = 2 * (g - 1) + x;  // this group's last piece
                wait(bars.pv_done(last % kPieces), (last / kPieces) & 1);
                // (two copies by item: the other group may be an item behind)
                float2* st = state + (n & 1) * 2 * kTile;
                st[x * kTile + r] = make_float2(m, l);
                tc_fence_before();
                if (!ok || !joined.sync()) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const float2 o = st[(x ^ 1) * kTile + r];
                mo = o.x;
                lo = o.y;
            }
            const float M = fmaxf(m, mo);
            // (the weight of a state without a valid key is 0, and its O is not looked at; that of a state of NaN scores,
            // which no maximum takes up, is NaN)
            const bool use_own = !(m == -INFINITY && l == 0.f), use_oth = !(mo == -INFINITY && lo == 0.f);
            const float w_own = use_own ? fast_exp2(0.5f * (m - M)) : 0.f, w_oth = use_oth ? fast_exp2(0.5f * (mo - M)) : 0.f;
            const float L = w_own * l * w_own + w_oth * lo * w_oth, inv = L == 0.f ? 0.f : 1.f / L;
            const float f_own = w_own * w_own * inv, f_oth = w_oth * w_oth * inv;
            const bool row_ok = my_pos < d.nq;
            const size_t row = (size_t)(d.row + my_pos) * p.num_q_heads + d.kvh * G + (r - my_pos * G);
            const bool direct = d.spans == 1;
            const size_t part = (size_t)d.span * p.total_q * p.num_q_heads + row;
            const uint32_t t_oth = tmem + lanes + kTO + (x ^ 1) * 128;
            if (!direct && row_ok && x == 0) spans.ml[part] = make_float2(M, L);
#pragma unroll 1
            for (int col = x * 64; col < x * 64 + 64; col += 32) {
                float o[32];
                {
                    float b[32];
                    tmem_ld32(t_o + col, o);
                    tmem_ld32(t_oth + col, b);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = (use_own ? o[i] * f_own : 0.f) + (use_oth ? b[i] * f_oth : 0.f);
                }
                if (!row_ok) continue;
                if (direct) {
                    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + row * kD + col;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t w[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(o[16 * k + 2 * i], o[16 * k + 2 * i + 1]);
                        if (out_al32) {
                            store32(out + 16 * k, w);
                        } else {
                            reinterpret_cast<uint4*>(out + 16 * k)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                            reinterpret_cast<uint4*>(out + 16 * k)[1] = make_uint4(w[4], w[5], w[6], w[7]);
                        }
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t w[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(o[8 * k + i]);
                        store32(spans.o + part * kD + col + 8 * k, w);
                    }
                }
            }
            // NaN among the V of the tile's own keys (see clear_nans), where this row sees them
            const int* nan = reinterpret_cast<const int*>(smem + kNan) + n % kNanSlots * (kD + 1);
            if (nan[kD] != INT_MAX && row_ok) {
                const int my_last = min(d.pos + my_pos, d.last_key);
#pragma unroll 1
                for (int col = x * 64; col < x * 64 + 64; ++col) {
                    if (nan[col] > my_last) continue;
                    if (direct) static_cast<__nv_bfloat16*>(p.out)[row * kD + col] = __float2bfloat16_rn(NAN);
                    else spans.o[part * kD + col] = NAN;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0 && ok) mbar_arrive(bars.o_free());
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.item_empty(n % kItems));
        }
        if (!ok && lane == 0) count_error(p.error_count);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the spans of a tile's rows: a warp per (row, query head), a float4 of columns per lane, in span order.  The
// first kAhead spans' rows are asked for before it is known how many there are (their addresses hold for every row),
// and the row's chunk is found by all lanes at once, so that two loads follow one another instead of six.
__global__ void __launch_bounds__(128) prefill_fp8_block_join_kernel(const PrefillParams p, const Spans spans) {
    constexpr int kAhead = 8;
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, G = p.group, ppt = kTile / G;
    const long long rows = (long long)p.total_q * p.num_q_heads, stride = (long long)gridDim.x * 4;
    for (long long u = (long long)blockIdx.x * 4 + (threadIdx.x >> 5); u < rows; u += stride) {
        const int q = (int)(u / p.num_q_heads);
        float4 o[kAhead];
        float2 ml[kAhead];
        auto load = [&](int i0) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (i0 + k < spans.count) {
                    ml[k] = __ldcg(spans.ml + (size_t)(i0 + k) * rows + u);
                    o[k] = __ldcg(reinterpret_cast<const float4*>(spans.o + ((size_t)(i0 + k) * rows + u) * kD) + lane);
                }
        };
        load(0);
        // the chunk of row q: the largest c with cu_q_lens[c] <= q
        int c = -1;
        for (int c0 = 0; c0 < p.num_chunks; c0 += 32) {
            const uint32_t le = __ballot_sync(0xffffffffu, c0 + lane < p.num_chunks && p.cu_q_lens[c0 + lane] <= q);
            if (le != 0) c = c0 + 31 - __clz(le);
        }
        int r0, n, s, start;
        if (c < 0 || !chunk_of(p, c, r0, n, s, start) || q >= r0 + n) continue;
        const int tile_end = min((q - r0) / ppt * ppt + ppt, n);  // as the kernel above cuts the chunk
        const int last = min((int)min((long long)start + tile_end - 1, 0x7FFFFFFELL), key_cap(p, s) - 1);
        const int all = last >= 0 ? last / kTile + 1 : 0, count = max(1, (all + spans.tiles - 1) / spans.tiles);
        if (count == 1) continue;  // stored directly
        float m = -INFINITY, wsum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i0 = 0; i0 < count; i0 += kAhead) {
            if (i0 > 0) load(i0);
            float mx = m;
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (i0 + k < count && ml[k].y != 0.f) mx = fmaxf(mx, ml[k].x);
            const float r = m == mx ? 1.f : exp2f(0.5f * (m - mx));  // (twice, as in the kernel above)
            m = mx;
            wsum = wsum * r * r;
            acc = make_float4(acc.x * r * r, acc.y * r * r, acc.z * r * r, acc.w * r * r);
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (i0 + k >= count || ml[k].y == 0.f) continue;
                const float e = exp2f(0.5f * (ml[k].x - m)), w = ml[k].y * e * e;
                wsum += w;
                acc.x = fmaf(w, o[k].x, acc.x);
                acc.y = fmaf(w, o[k].y, acc.y);
                acc.z = fmaf(w, o[k].z, acc.z);
                acc.w = fmaf(w, o[k].w, acc.w);
            }
        }
        const float inv = wsum == 0.f ? 0.f : 1.f / wsum;
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + u * kD + lane * 4) =
            make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    }
}

// Query tiles times kv heads.
long long work_items(int num_chunks, int max_q_len, int num_kv_heads, int group) {
    const int ppt = kTile / group;
    return (long long)((max_q_len + ppt - 1) / ppt) * num_chunks * num_kv_heads;
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }
size_t partial_bytes(size_t rows) { return rows == 0 ? 0 : up256(rows * kD * sizeof(float)) + up256(rows * sizeof(float2)); }

// Key tiles per span and spans per query tile.  Where the tiles alone leave half of the SMs idle their keys are cut so
// that the items make up one round of the GPU, into spans of at least two key tiles (a span's partial rows cost about
// one key tile's time to store and join): 37 queries at 2,955, 8 kv heads, 16.5 us, uncut 35.5; but 160 query tiles of
// 21 key tiles cut in two 62.7, uncut 53.4.  The count comes from the largest context, the lengths live on the device.
// No more spans than `workspace_bytes` holds the partial rows of, for all `total_rows` (query, head) rows of q.
Spans plan_spans(int num_chunks, int max_q_len, int num_kv_heads, int group, int max_context_len, int num_sms,
                 size_t total_rows, size_t workspace_bytes) {
    const int tiles = max_context_len > 0 ? (max_context_len - 1) / kTile + 1 : 1;
    const long long items = work_items(num_chunks, max_q_len, num_kv_heads, group);
    long long want = items > 0 && items < num_sms ? num_sms / items : 1;
    if (want > tiles / 2) want = tiles / 2;
    Spans s;
    s.o = nullptr;
    s.ml = nullptr;
    do {
        s.tiles = want > 1 ? (int)((tiles + want - 1) / want) : tiles;
        s.count = (tiles + s.tiles - 1) / s.tiles;
    } while (s.count > 1 && partial_bytes(s.count * total_rows) > workspace_bytes && --want > 0);
    return s;
}

// The rows of q that a call's chunks can have: there may be others behind the last one.
size_t chunk_rows(int num_chunks, int total_q, int max_q_len, int num_q_heads) {
    return (size_t)std::min<long long>(total_q, (long long)num_chunks * max_q_len) * num_q_heads;
}

}  // namespace

// What the calls of these sizes need, with room for the rows behind the chunks; and at least what every call of no more
// chunks, queries and context needs: such a call has more spans where it has fewer tiles, at most one item a SM.
size_t prefill_fp8_block_workspace(int num_chunks, int total_q, int max_q_len, int num_q_heads, int num_kv_heads,
                                   int max_context_len, int num_sms) {
    const int group = num_q_heads / num_kv_heads;
    const size_t all = (size_t)total_q * num_q_heads;
    const Spans s = plan_spans(num_chunks, max_q_len, num_kv_heads, group, max_context_len, num_sms, all, SIZE_MAX);
    const size_t these = s.count > 1 ? partial_bytes(s.count * all) : 0;
    const size_t tiles = max_context_len > 0 ? (max_context_len - 1) / kTile + 1 : 1;
    const size_t count = std::min<size_t>(num_sms / num_kv_heads, tiles / 2);
    if (count < 2) return these;
    const size_t rows = std::min(count * chunk_rows(num_chunks, total_q, max_q_len, num_q_heads),
                                 (size_t)num_sms * (kTile / group) / num_kv_heads * num_q_heads);
    return std::max(these, partial_bytes(rows));
}

size_t prefill_fp8_block_need(const PrefillParams& p, int num_sms) {
    const size_t rows = chunk_rows(p.num_chunks, p.total_q, p.max_q_len, p.num_q_heads);
    const Spans s =
        plan_spans(p.num_chunks, p.max_q_len, p.num_kv_heads, p.group, p.max_context_len, num_sms, rows, SIZE_MAX);
    return s.count > 1 ? partial_bytes(s.count * rows) : 0;
}

bool prefill_fp8_block_tc_supported(const PrefillParams& p) {
    const int B = p.block_size;
    if (p.head_dim != kD || p.group > 8 || B < 8 || B > 128 || (B & (B - 1)) != 0) return false;
    if (((uintptr_t)p.k_cache & 15) || ((uintptr_t)p.v_cache & 15) || ((uintptr_t)p.q & 15) || ((uintptr_t)p.out & 15))
        return false;
    // (items: the tiles of every chunk and kv head, or, cut into spans, at most one a SM)
    return (long long)p.num_blocks * B < (1LL << 31) && p.num_blocks > 0 &&
           work_items(p.num_chunks, p.max_q_len, p.num_kv_heads, p.group) < (1LL << 29);
}

int launch_prefill_fp8_block_tc(const PrefillParams& p, void* workspace, size_t workspace_bytes, int num_sms,
                                cudaStream_t stream) {
    CUtensorMap tmk, tmv;
    int rc = pool_tensor_map_rows(&tmk, p.k_cache, p.num_blocks, p.block_size, p.num_kv_heads, kD, true);
    if (rc != PA_OK) return rc;
    if ((rc = pool_tensor_map_rows(&tmv, p.v_cache, p.num_blocks, p.block_size, p.num_kv_heads, kD, true)) != PA_OK)
        return rc;
    auto kernel = p.block_size == 8    ? prefill_fp8_block_tc_kernel<8>
                  : p.block_size == 16 ? prefill_fp8_block_tc_kernel<16>
                                       : prefill_fp8_block_tc_kernel<32>;
    if ((rc = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), kSmemBytes)) != PA_OK) return rc;
    const size_t total_rows = (size_t)p.total_q * p.num_q_heads;
    Spans s = plan_spans(p.num_chunks, p.max_q_len, p.num_kv_heads, p.group, p.max_context_len, num_sms, total_rows,
                         workspace_bytes);
    if (s.count > 1) {
        s.o = static_cast<float*>(workspace);
        s.ml = reinterpret_cast<float2*>(static_cast<char*>(workspace) + up256(s.count * total_rows * kD * sizeof(float)));
    }
    const long long items = work_items(p.num_chunks, p.max_q_len, p.num_kv_heads, p.group) * s.count;
    s.items = (int)items;
    s.per_rank = Divisor((uint32_t)(p.num_chunks * p.num_kv_heads * s.count));
    s.per_count = Divisor((uint32_t)s.count);
    s.per_heads = Divisor((uint32_t)p.num_kv_heads);
    s.per_tiles = Divisor((uint32_t)s.tiles);
    s.per_ppt = Divisor((uint32_t)(kTile / p.group));
    rc = launch_kernel(kernel, dim3((unsigned)(items < num_sms ? items : num_sms)),
                       dim3(kThreads), kSmemBytes, stream, tmk, tmv, p, s);
    if (rc != PA_OK || s.count <= 1) return rc;
    const long long warps = (long long)p.total_q * p.num_q_heads, ctas = (warps + 3) / 4;
    return launch_kernel(prefill_fp8_block_join_kernel, dim3((unsigned)(ctas < 16LL * num_sms ? ctas : 16LL * num_sms)),
                         dim3(128), 0, stream, p, s);
}

}  // namespace pa
