// prefill_weights_tc.cu — the keys' weights of pa_prefill_chunk_weights on the
// 5th-gen tensor cores (tcgen05, accumulators in TMEM), bf16, head_dim 128.
//
// The attention kernel (prefill_tc.cu) has left every row's lse.  Here
//     sum over the rows r that see key j of 2^(x_rj - lse_r),  x = scale log2(e) Q K^T
// for every key.  A row of tensor memory is a query row, so its lse is one register of
// one thread; a thread keeps a sum for each of 128 keys over all its rows, and the 32
// lanes' sums are added only when the keys change.  (With a key a row, each score's lse
// came from shared memory, whose bandwidth the products' operands take up: 2.3 times
// the time of the products.)  Bound by the tensor cores (half the attention's products),
// shared memory (a 128 x 256 x 16 product reads 12 KB in 128 cycles, and the query tiles'
// copies write) and the exponentials alike: 2048 queries at 5900, 64/8 heads, 235 GFLOP,
// 192 us = 1.23 PFLOP/s = 0.63 of the bf16 peak (without the exponentials and sums 127).
// A key a row took 276, this layout 253 at first, 223 with the rows' lse loaded a tile ahead
// and not touched before its use, 201 with dense and masked tiles in loops apart, 195 with the
// choice between them made without a vote.
//
// A run is a pair of 128-key tiles of one (chunk, kv head) against the 128-row query
// tiles (positions times the G heads of the kv head) that see a key of it, in order.
// The 256 keys stay in shared memory while the query tiles stream through a ring, so
// that a query tile's 32 KB feed two products.  The kernel is persistent, one CTA per
// SM: all runs in order, (chunk, kv head, pair), are one sequence of (pair, query tile)
// units, and CTA b takes units [b per, (b + 1) per) of it, wherever they begin and end.
// Each part of a run leaves a row of 256 sums: run number + CTA number is a row of its
// own.  The next run's keys are loaded into the other of two buffers meanwhile.
//
// Warp roles (384 threads):
//   warp 0      producer: keys (one TMA box per block and 64-column half) and query
//               tiles (one box per half)
//   warp 1      owner of the tensor memory and issuer of the products
//   warps 4-11  the sums: a thread a query row and 128 of the 256 keys; they take the
//               registers that warps 0-3 give up
// Every wait is bounded, tensor memory is always freed, and copies and products
// in flight are waited for before a CTA exits, as in prefill_tc.cu.
#include "prefill_weights.cuh"
#include "sm100_ptx.cuh"

namespace pa {
namespace {

constexpr int kTile = 128;
constexpr int kD = 128;
static_assert(kKeys == 2 * kTile, "keys of a run");
constexpr int kMinUnits = 2;
constexpr int kHalf = 128 * 128;           // bytes of a 64-column half of a 128-row tile
constexpr int kTileBytes = 2 * kHalf;
constexpr int kSumWarps = 8;
constexpr int kThreads = (kSumWarps + 4) * 32;
// registers a thread: 4 warps of 56 and 8 of 224 are the 12 of 168 that the block is launched with
#define PA_OTHER_REGS "56"
#define PA_SUM_REGS "224"
constexpr int kKeyHalf = kKeys * 128;      // bytes of a 64-column half of the run's keys
constexpr uint32_t kTmemCols = 512;        // two buffers of two key tiles' scores
constexpr int kQStages = 3;
constexpr int kK = 0;                      // [2 buffers][2 halves][256 keys]
constexpr int kQ = kK + 4 * kTileBytes;
constexpr int kBars = kQ + kQStages * kTileBytes;
// k_full[2], k_empty[2], q_full[3], q_empty[3], s_full[2], s_empty[2], d_empty[2], drain
constexpr int kNumBars = 4 + 2 * kQStages + 6 + 1;
constexpr int kTmemSlot = kBars + kNumBars * 8;
constexpr int kStart = (kTmemSlot + 4 + 7) / 8 * 8;
struct Start {  // where a CTA's units begin
    int c, kvh, pair, tile;
    long long units;
};
struct Run {  // as the producer describes it to the other warps; nt == 0: no more
    int s, kvh, r0, n, start, nkeys, j0, t0, nt, row;
};
constexpr int kRuns = kStart + sizeof(Start);  // Run [2]
constexpr size_t kSmemBytes = 1024 + kRuns + 2 * sizeof(Run);
static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");

struct Bars {
    uint64_t* base;
    __device__ uint64_t* k_full(int i) const { return base + i; }
    __device__ uint64_t* k_empty(int i) const { return base + 2 + i; }
    __device__ uint64_t* q_full(int i) const { return base + 4 + i; }
    __device__ uint64_t* q_empty(int i) const { return base + 4 + kQStages + i; }
    __device__ uint64_t* s_full(int i) const { return base + 4 + 2 * kQStages + i; }
    __device__ uint64_t* s_empty(int i) const { return base + 6 + 2 * kQStages + i; }
    __device__ uint64_t* d_empty(int i) const { return base + 8 + 2 * kQStages + i; }
    __device__ uint64_t* drain() const { return base + 10 + 2 * kQStages; }
};

__global__ void __launch_bounds__(kThreads, 1)
    key_weights_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                       const PrefillParams p) {
    pdl_trigger();
    pdl_wait();
    const int G = p.group, B = p.block_size, Hkv = p.num_kv_heads;
    const int per_tile = kTile / G;  // positions of a query tile
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const Bars bars{reinterpret_cast<uint64_t*>(smem + kBars)};
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kTmemSlot);
    Start* start = reinterpret_cast<Start*>(smem + kStart);
    Run* runs = reinterpret_cast<Run*>(smem + kRuns);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bars.k_full(i), 1);
            mbar_init(bars.k_empty(i), 1);
            mbar_init(bars.s_full(i), 1);
            mbar_init(bars.s_empty(i), kSumWarps);
            mbar_init(bars.d_empty(i), kSumWarps + 1);
        }
        for (int i = 0; i < kQStages; ++i) {
            mbar_init(bars.q_full(i), 1);
            mbar_init(bars.q_empty(i), 1);
        }
        mbar_init(bars.drain(), 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // ---- this CTA's units.  The chunks' units, then the sums before each chunk, in the key buffers (not yet in use); CTA 0
    // leaves what the addition needs to find a key's rows.
    unsigned long long* before = reinterpret_cast<unsigned long long*>(smem + kK);
    for (int c = threadIdx.x; c < p.num_chunks; c += kThreads) {
        WeightChunk d;
        before[c] = weight_chunk(p, c, d) ? (unsigned long long)key_units(d, per_tile) * Hkv : 0ull;
    }
    __syncthreads();
    if (warp == 0) {
        unsigned long long units = 0;
        int runs = 0;
        const int n32 = (p.num_chunks + 31) / 32 * 32;
        for (int c = lane; c < n32; c += 32) {
            WeightChunk d;
            const bool have = c < p.num_chunks && weight_chunk(p, c, d);
            unsigned long long u = have ? before[c] : 0ull;
            int r = have ? key_pairs(d) * Hkv : 0;
            const unsigned long long mine = u;
            const int mine_r = r;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const unsigned long long v = __shfl_up_sync(0xffffffffu, u, off);
                const int w = __shfl_up_sync(0xffffffffu, r, off);
                if (lane >= off) {
                    u += v;
                    r += w;
                }
            }
            if (c < p.num_chunks) {
                before[c] = units + u - mine;
                if (blockIdx.x == 0) p.runs[c] = KeyRuns{units + u - mine, runs + r - mine_r};
            }
            units += __shfl_sync(0xffffffffu, u, 31);
            runs += __shfl_sync(0xffffffffu, r, 31);
        }
        const unsigned long long per = max((units + gridDim.x - 1) / gridDim.x, (unsigned long long)kMinUnits);
        if (blockIdx.x == 0 && lane == 0) p.runs[p.num_chunks] = KeyRuns{per, 0};
        __syncwarp();
        const unsigned long long first = blockIdx.x * per;
        if (lane == 0) {
            *start = Start{0, 0, 0, 0, first < units ? (long long)min(per, units - first) : 0LL};
            if (first < units) {
                int lo = 0, hi = p.num_chunks - 1;  // the last chunk that begins at or before `first` (empty ones before it)
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if (before[mid] <= first) lo = mid; else hi = mid - 1;
                }
                WeightChunk d;
                weight_chunk(p, lo, d);
                const unsigned long long in_chunk = first - before[lo], each = key_units(d, per_tile);
                start->c = lo;
                start->kvh = (int)(in_chunk / each);
                long long left = (long long)(in_chunk - start->kvh * each);
                int pair = 0;
                // the pairs that every query sees, all of one length, then the others
                const int tiles = key_tiles(d, per_tile), whole = min(key_pairs(d), d.start / kKeys + 1);
                pair = (int)min((long long)whole, left / tiles);
                left -= (long long)pair * tiles;
                while (left >= tiles - key_first_tile(d, pair, per_tile)) left -= tiles - key_first_tile(d, pair++, per_tile);
                start->pair = pair;
                start->tile = key_first_tile(d, pair, per_tile) + (int)left;
            }
        }
    }
    // rows of a query tile that no copy fills (groups that do not divide 128): zeros, whose scores are finite for finite keys
    if (per_tile * G < kTile)
        for (int i = threadIdx.x; i < kQStages * kTileBytes / 16; i += kThreads)
            reinterpret_cast<uint4*>(smem + kQ)[i] = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();  // the key buffers (and these) go to the copies
    __syncthreads();
    if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 " PA_OTHER_REGS ";");

    bool ok = true;
    int ni = 0;           // runs taken
    uint32_t g = 0;       // query tiles taken
    // waits until use number n of a ring of `stages` may overwrite what use n - stages left
    auto free_slot = [&](uint64_t* bar, uint32_t n, uint32_t stages) {
        return n < stages || mbar_wait_warp(bar, (n / stages - 1) & 1);
    };

    // the next run, once its keys have landed; false when there is none
    auto next_run = [&](Run& run) {
        if (!mbar_wait_warp(bars.k_full(ni & 1), (ni >> 1) & 1)) ok = false;
        if (!ok) return false;
        run = runs[ni & 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.d_empty(ni & 1));
        ++ni;
        return run.nt > 0;
    };

    if (warp == 0) {
        // ============================================================ producer
        if (lane == 0) {
            tma_prefetch_desc(&tmq);
            tma_prefetch_desc(&tmk);
        }
        WeightChunk d;
        int c = start->c, kvh = start->kvh, pair = start->pair, tile = start->tile, row = 0;
        long long left = start->units;
        if (left > 0) {
            for (int e = lane; e < c; e += 32)  // runs before this CTA's first one
                if (weight_chunk(p, e, d)) row += key_pairs(d) * Hkv;
            row = __reduce_add_sync(0xffffffffu, row);
            weight_chunk(p, c, d);
            row += kvh * key_pairs(d) + pair + blockIdx.x;
        }
        const int bpi = kKeys / B;  // blocks of a run
        while (ok) {
            const int kb = ni & 1;
            const int j0 = pair * kKeys;
            const int nt = left > 0 ? (int)min((long long)(key_tiles(d, per_tile) - tile), left) : 0;
            int pb = -1;
            if (nt > 0) {
                const int first = j0 / B, nblk = (d.nkeys + B - 1) / B - first;
                if (lane < bpi && lane < nblk) {
                    pb = p.block_tables[(size_t)d.s * p.max_blocks_per_seq + first + lane];
                    if (pb >= p.num_blocks) pb = -1;  // (the attention kernel has counted it)
                }
            }
            const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, pb >= 0)) * 2u * B * 128u;
            if (!free_slot(bars.k_empty(kb), ni, 2) || !free_slot(bars.d_empty(kb), ni, 2)) {
                ok = false;
                break;
            }
            if (lane == 0) {
                runs[kb] = Run{d.s, kvh, d.r0, d.n, d.start, d.nkeys, j0, tile, nt, row};
                mbar_arrive_expect_tx(bars.k_full(kb), bytes);
            }
            __syncwarp();
            ++ni;
            if (nt == 0) break;
            if (pb >= 0) {
                uint8_t* dst = smem + kK + 2 * kb * kKeyHalf + lane * B * 128;  // block `lane` of the run
                for (int h = 0; h < 2; ++h)
                    tma_load_2d(dst + h * kKeyHalf, &tmk, kvh * kD + h * 64, pb * B, bars.k_full(kb));
            }
            for (int t = 0; t < nt; ++t, ++g) {
                const int st = g % kQStages;
                if (!free_slot(bars.q_empty(st), g, kQStages)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    mbar_arrive_expect_tx(bars.q_full(st), 2 * per_tile * G * 128);
                    for (int h = 0; h < 2; ++h)
                        tma_load_3d(smem + kQ + st * kTileBytes + h * kHalf, &tmq, h * 64, kvh * G,
                                    d.r0 + (tile + t) * per_tile, bars.q_full(st));
                }
                __syncwarp();
            }
            // the next run in order: (chunk, kv head, pair), chunks without keys passed over
            left -= nt;
            ++row;
            if (left > 0) {
                if (++pair == key_pairs(d)) {
                    pair = 0;
                    if (++kvh == Hkv) {
                        kvh = 0;
                        do ++c;
                        while (!(weight_chunk(p, c, d) && key_pairs(d) > 0));
                    }
                }
                tile = key_first_tile(d, pair, per_tile);
            }
        }
        if (!ok && lane == 0) count_error(p.error_count);
        if (lane == 0 && !(drain_ring(bars.k_full(0), 2, ni) && drain_ring(bars.q_full(0), kQStages, g)))
            count_error(p.error_count);
        __syncwarp();
    } else if (warp == 1) {
        // ============================================================ products
        constexpr uint32_t idesc = umma_idesc_bf16(kTile, kKeys, false, false);
        const uint64_t dk0 = umma_desc_sw128(smem_u32(smem + kK), 16, 1024);
        const uint64_t dq0 = umma_desc_sw128(smem_u32(smem + kQ), 16, 1024);
        for (Run it; next_run(it);) {
            const int kb = (ni - 1) & 1;
            for (int t = 0; t < it.nt && ok; ++t, ++g) {
                const int st = g % kQStages, sb = g & 1;
                if (!mbar_wait_warp(bars.q_full(st), (g / kQStages) & 1)) {
                    ok = false;
                    break;
                }
                if (!free_slot(bars.s_empty(sb), g, 2)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t dk = dk0 + (uint64_t)((2 * kb * kKeyHalf) >> 4);
                const uint64_t dq = dq0 + (uint64_t)((st * kTileBytes) >> 4);
#pragma unroll
                for (int kk = 0; kk < kD / 16; ++kk)
                    umma_bf16_warp(tmem + sb * kKeys, dq + (uint64_t)(((kk >> 2) * kHalf + (kk & 3) * 32) >> 4),
                                   dk + (uint64_t)(((kk >> 2) * kKeyHalf + (kk & 3) * 32) >> 4), idesc, kk > 0);
                umma_commit_warp(bars.s_full(sb));
                umma_commit_warp(bars.q_empty(st));
            }
            umma_commit_warp(bars.k_empty(kb));
        }
        if (!ok && lane == 0) count_error(p.error_count);
        umma_commit_warp(bars.drain());
        if (!mbar_wait_warp(bars.drain(), 0) && lane == 0) count_error(p.error_count);
        __syncwarp();
    } else if (warp >= 4) {
        // ============================================================ sums
        asm volatile("setmaxnreg.inc.sync.aligned.u32 " PA_SUM_REGS ";");
        const int quarter = warp & 3, col0 = ((warp - 4) >> 2) * 128;
        const int r = quarter * 32 + lane;  // this thread's row of a query tile
        const uint32_t at0 = tmem + ((uint32_t)(quarter * 32) << 16) + col0;
        const int r_pos = r / G;            // and its position
        const float sl2 = p.scale_log2;
        const unsigned long long s2 = f32x2_pack(sl2, sl2);
        for (Run it; next_run(it);) {
            // the lse of this thread's row in query tile t of the run; loaded a tile ahead, and not touched before it is needed
            const float* lse = p.lse + ((size_t)it.kvh * p.total_q + it.r0) * G + r;
            auto has_row = [&](int t) { return t < it.nt && r < min(per_tile, it.n - (it.t0 + t) * per_tile) * G; };
            auto load_lse = [&](int t) { return has_row(t) ? __ldg(lse + (size_t)(it.t0 + t) * per_tile * G) : 0.f; };
            unsigned long long sum2[64];  // sums of keys col0 + 2 i and col0 + 2 i + 1
#pragma unroll
            for (int i = 0; i < 64; ++i) sum2[i] = f32x2_pack(0.f, 0.f);
            const int see0 = it.start + r_pos + 1 - it.j0 - col0;
            float lse_next = load_lse(0);
            for (int t = 0; t < it.nt; ++t, ++g) {
                const int sb = g & 1, i0 = (it.t0 + t) * per_tile;
                const float nl = has_row(t) ? -lse_next : -INFINITY;
                lse_next = load_lse(t + 1);
                // this row sees the first `see` of the thread's keys
                int see = see0 + i0;
                const bool dense = it.n - i0 >= per_tile && see - r_pos >= 128;  // every row, the first one's position too
                if (nl == -INFINITY) see = 0;  // (no such row; or one without keys, or with an infinite lse: weights of 0)
                if (ok && !mbar_wait(bars.s_full(sb), (g >> 1) & 1)) ok = false;
                __syncwarp();
                tc_fence_after();
                const unsigned long long nl2 = f32x2_pack(nl, nl);
                // 32 keys at a time, the next ones on their way.  (Dense tiles have a loop of their own: their instructions lie
                // together.)
                auto add_tile = [&](auto add) {
                    float xs[2][32];
                    tmem_ld32(at0 + sb * kKeys, xs[0]);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float(&x)[32] = xs[q & 1];
                        tmem_wait_ld32(x);
                        if (q < 3) tmem_ld32(at0 + sb * kKeys + (q + 1) * 32, xs[(q + 1) & 1]);
                        if (q == 3) {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0 && ok) mbar_arrive(bars.s_empty(sb));
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float y0, y1;
                            add(q * 32 + 2 * i, x[2 * i], x[2 * i + 1], y0, y1);
                            sum2[q * 16 + i] = add_f32x2(sum2[q * 16 + i], f32x2_pack(fast_exp2(y0), fast_exp2(y1)));
                        }
                    }
                };
                if (dense)
                    add_tile([&](int, float x0, float x1, float& y0, float& y1) {
                        f32x2_unpack(fma_f32x2(f32x2_pack(x0, x1), s2, nl2), y0, y1);
                    });
                else
                    add_tile([&](int key, float x0, float x1, float& y0, float& y1) {
                        y0 = key < see ? fmaf(x0, sl2, nl) : -INFINITY;
                        y1 = key + 1 < see ? fmaf(x1, sl2, nl) : -INFINITY;
                    });
            }
            // the lanes' sums added, halving what a lane holds each time: 4 keys are left to each
            float v[128];
#pragma unroll
            for (int i = 0; i < 64; ++i) f32x2_unpack(sum2[i], v[2 * i], v[2 * i + 1]);
            if (r >= per_tile * G) {  // a row that no query fills: 0 times an infinity among the keys is NaN
#pragma unroll
                for (int i = 0; i < 128; ++i) v[i] = 0.f;
            }
            int first = 0;
#pragma unroll
            for (int n = 64; n >= 4; n >>= 1) {
                const int bit = n >> 2;
                const bool upper = lane & bit;
                first += upper ? n : 0;
#pragma unroll
                for (int i = 0; i < n; ++i) {
                    const float give = upper ? v[i] : v[i + n], keep = upper ? v[i + n] : v[i];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, give, bit);
                }
            }
            // keys of an invalid block draw nothing (4 keys from a multiple of 4 are of one block)
            const int j = it.j0 + col0 + first;
            bool valid = j < it.nkeys;
            if (valid) {
                const int pb = p.block_tables[(size_t)it.s * p.max_blocks_per_seq + j / B];
                valid = pb >= 0 && pb < p.num_blocks;
            }
            *reinterpret_cast<float4*>(p.partial + ((size_t)it.row * kKeyParts + quarter) * kKeys + col0 + first) =
                valid ? make_float4(v[0], v[1], v[2], v[3]) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if (!ok && lane == 0) count_error(p.error_count);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

}  // namespace

int launch_prefill_weights_tc(const PrefillParams& p, int num_sms, cudaStream_t stream) {
    CUtensorMap tmq, tmk;
    auto enc = tensor_map_encoder();
    if (!enc) return PA_ERR_CUDA;
    const int G = p.group;
    cuuint64_t dims[3] = {(cuuint64_t)kD, (cuuint64_t)p.num_q_heads, (cuuint64_t)p.total_q};
    cuuint64_t strides[2] = {(cuuint64_t)kD * 2, (cuuint64_t)p.num_q_heads * kD * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)(kTile / G)};
    cuuint32_t estr[3] = {1, 1, 1};
    if (enc(&tmq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p.q), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return PA_ERR_UNSUPPORTED;
    int rc = pool_tensor_map(&tmk, p.k_cache, p.num_blocks, p.block_size, p.num_kv_heads, kD);
    if (rc != PA_OK) return rc;
    if ((rc = ensure_dynamic_smem(reinterpret_cast<const void*>(key_weights_kernel), kSmemBytes)) != PA_OK) return rc;
    return launch_kernel(key_weights_kernel, dim3((unsigned)num_sms), dim3(kThreads), kSmemBytes, stream, tmq, tmk, p);
}

}  // namespace pa
