// prefill_weights_tc.cu — the keys' weights of pa_prefill_chunk_weights on the
// 5th-gen tensor cores (tcgen05, accumulators in TMEM), bf16, head_dim 128.
//
// The attention kernel (prefill_tc.cu) has left every row's lse.  Here
//     partial[chunk][kv head][piece][j] = sum over the piece's rows r of 2^(x_rj - lse_r)
// with x = scale log2(e) Q K^T.  The product is taken transposed, K Q^T: a row of
// tensor memory is a key, so a thread sums its key's weights in a register and
// nothing crosses threads.  Bound by the tensor cores (half the attention's
// products) and the exponentials alike.
//
// A work item is (chunk, kv head, piece of the chunk's query tiles, pair of
// 128-key tiles).  Its 256 keys stay in shared memory while the piece's 128-row
// query tiles (positions times the G heads of the kv head) stream through a
// ring, so that a query tile's 32 KB feed two products.  The kernel is
// persistent, one CTA per SM; the next item's keys are loaded into the other of
// two buffers meanwhile.
//
// Warp roles (352 threads):
//   warp 0     producer: key tiles (one TMA box per block and 64-column half) and
//              query tiles (one box per half)
//   warp 1     owner of the tensor memory and issuer of the products
//   warps 2-9  the sums: four warps for each of the two key tiles, a thread a key
//   warp 10    the query tiles' lse, to shared memory
// Every wait is bounded, tensor memory is always freed, and copies and products
// in flight are waited for before a CTA exits, as in prefill_tc.cu.
#include "prefill_weights.cuh"
#include "sm100_ptx.cuh"

namespace pa {
namespace {

constexpr int kTile = 128;
constexpr int kD = 128;
constexpr int kKeys = 2 * kTile;           // keys of an item
constexpr int kHalf = 128 * 128;           // bytes of a 64-column half of a 128-row tile
constexpr int kTileBytes = 2 * kHalf;
constexpr int kThreads = 352;
constexpr int kLseWarp = 10;
constexpr uint32_t kTmemCols = 512;        // two buffers of two key tiles' scores
constexpr int kQStages = 3;
constexpr int kK = 0;                      // [2 buffers][2 tiles]
constexpr int kQ = kK + 4 * kTileBytes;
constexpr int kLse = kQ + kQStages * kTileBytes;  // float [kQStages][128]
constexpr int kBars = kLse + kQStages * kTile * 4;
// k_full[2], k_empty[2], q_full[3], q_empty[3], l_full[3], l_empty[3], s_full[2][2], s_empty[2][2], drain
constexpr int kNumBars = 4 + 4 * kQStages + 8 + 1;
constexpr int kTmemSlot = kBars + kNumBars * 8;
constexpr size_t kSmemBytes = 1024 + kTmemSlot + 16;
static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");

struct Bars {
    uint64_t* base;
    __device__ uint64_t* k_full(int i) const { return base + i; }
    __device__ uint64_t* k_empty(int i) const { return base + 2 + i; }
    __device__ uint64_t* q_full(int i) const { return base + 4 + i; }
    __device__ uint64_t* q_empty(int i) const { return base + 4 + kQStages + i; }
    __device__ uint64_t* l_full(int i) const { return base + 4 + 2 * kQStages + i; }
    __device__ uint64_t* l_empty(int i) const { return base + 4 + 3 * kQStages + i; }
    __device__ uint64_t* s_full(int b, int t) const { return base + 4 + 4 * kQStages + 2 * b + t; }
    __device__ uint64_t* s_empty(int b, int t) const { return base + 8 + 4 * kQStages + 2 * b + t; }
    __device__ uint64_t* drain() const { return base + 12 + 4 * kQStages; }
};

__global__ void __launch_bounds__(kThreads, 1)
    key_weights_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                       const PrefillParams p, const int piece_tiles) {
    pdl_trigger();
    pdl_wait();
    const int G = p.group, B = p.block_size, Hkv = p.num_kv_heads;
    const int per_tile = kTile / G;  // positions of a query tile
    const int pairs_max = (p.max_context_len + kKeys - 1) / kKeys;
    const int num_items = p.num_chunks * Hkv * p.pieces * pairs_max;

    struct Item {
        WeightChunk d;
        int c, kvh, piece, j0, t0, nt;  // first key, first query tile, query tiles
    };
    // item k: neighbours differ in the keys and share the queries; false for one without a key that a query of it sees
    auto describe = [&](int k, Item& it) {
        const int pair = k % pairs_max;
        k /= pairs_max;
        it.piece = k % p.pieces;
        k /= p.pieces;
        it.kvh = k % Hkv;
        it.c = k / Hkv;
        if (!weight_chunk(p, it.c, it.d)) return false;
        it.j0 = pair * kKeys;
        if (it.j0 >= it.d.nkeys) return false;
        const int tiles = (it.d.n + per_tile - 1) / per_tile;
        it.t0 = max(it.piece * piece_tiles, max(0, it.j0 - it.d.start) / per_tile);
        it.nt = min(tiles, (it.piece + 1) * piece_tiles) - it.t0;
        return it.nt > 0;
    };

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const Bars bars{reinterpret_cast<uint64_t*>(smem + kBars)};
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kTmemSlot);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bars.k_full(i), 1);
            mbar_init(bars.k_empty(i), 1);
            for (int t = 0; t < 2; ++t) {
                mbar_init(bars.s_full(i, t), 1);
                mbar_init(bars.s_empty(i, t), 4);
            }
        }
        for (int i = 0; i < kQStages; ++i) {
            mbar_init(bars.q_full(i), 1);
            mbar_init(bars.q_empty(i), 1);
            mbar_init(bars.l_full(i), 1);
            mbar_init(bars.l_empty(i), 8);
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
    bool ok = true;
    int ni = 0;           // items taken
    uint32_t g = 0;       // query tiles taken
    // waits until use number n of a ring of `stages` may overwrite what use n - stages left
    auto free_slot = [&](uint64_t* bar, uint32_t n, uint32_t stages) {
        return n < stages || mbar_wait_warp(bar, (n / stages - 1) & 1);
    };

    if (warp == 0) {
        // ============================================================ producer
        if (lane == 0) {
            tma_prefetch_desc(&tmq);
            tma_prefetch_desc(&tmk);
        }
        for (int k = blockIdx.x; k < num_items && ok; k += gridDim.x) {
            Item it;
            if (!describe(k, it)) continue;
            const int kb = ni & 1, bpi = kKeys / B;  // blocks of an item
            const int first = it.j0 / B, nblk = (it.d.nkeys + B - 1) / B - first;
            int pb = -1;
            if (lane < bpi && lane < nblk) {
                pb = p.block_tables[(size_t)it.d.s * p.max_blocks_per_seq + first + lane];
                if (pb >= p.num_blocks) pb = -1;  // (the attention kernel has counted it)
            }
            const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, pb >= 0)) * 2u * B * 128u;
            if (!free_slot(bars.k_empty(kb), ni, 2)) {
                ok = false;
                break;
            }
            if (lane == 0) mbar_arrive_expect_tx(bars.k_full(kb), bytes);
            __syncwarp();
            if (pb >= 0) {
                // block `lane` of the item: rows lane * B on of tile (lane * B) / 128
                const int row = lane * B, tile = row / kTile;
                uint8_t* dst = smem + kK + (2 * kb + tile) * kTileBytes + (row - tile * kTile) * 128;
                for (int h = 0; h < 2; ++h)
                    tma_load_2d(dst + h * kHalf, &tmk, it.kvh * kD + h * 64, pb * B, bars.k_full(kb));
            }
            ++ni;
            for (int t = 0; t < it.nt; ++t, ++g) {
                const int st = g % kQStages;
                if (!free_slot(bars.q_empty(st), g, kQStages)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    mbar_arrive_expect_tx(bars.q_full(st), 2 * per_tile * G * 128);
                    for (int h = 0; h < 2; ++h)
                        tma_load_3d(smem + kQ + st * kTileBytes + h * kHalf, &tmq, h * 64, it.kvh * G,
                                    it.d.r0 + (it.t0 + t) * per_tile, bars.q_full(st));
                }
                __syncwarp();
            }
        }
        if (!ok && lane == 0) count_error(p.error_count);
        if (lane == 0 && !(drain_ring(bars.k_full(0), 2, ni) && drain_ring(bars.q_full(0), kQStages, g)))
            count_error(p.error_count);
        __syncwarp();
    } else if (warp == 1) {
        // ============================================================ products
        constexpr uint32_t idesc = umma_idesc_bf16(128, 128, false, false);
        const uint64_t dk0 = umma_desc_sw128(smem_u32(smem + kK), 16, 1024);
        const uint64_t dq0 = umma_desc_sw128(smem_u32(smem + kQ), 16, 1024);
        for (int k = blockIdx.x; k < num_items && ok; k += gridDim.x) {
            Item it;
            if (!describe(k, it)) continue;
            const int kb = ni & 1;
            if (!mbar_wait_warp(bars.k_full(kb), (ni >> 1) & 1)) {
                ok = false;
                break;
            }
            for (int t = 0; t < it.nt && ok; ++t, ++g) {
                const int st = g % kQStages, sb = g & 1;
                if (!mbar_wait_warp(bars.q_full(st), (g / kQStages) & 1)) {
                    ok = false;
                    break;
                }
                for (int tile = 0; tile < 2; ++tile) {
                    if (!free_slot(bars.s_empty(sb, tile), g, 2)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t dk = dk0 + (uint64_t)(((2 * kb + tile) * kTileBytes) >> 4);
                    const uint64_t dq = dq0 + (uint64_t)((st * kTileBytes) >> 4);
#pragma unroll
                    for (int kk = 0; kk < kD / 16; ++kk) {
                        const uint64_t off = (uint64_t)(((kk >> 2) * kHalf + (kk & 3) * 32) >> 4);
                        umma_bf16_warp(tmem + sb * 256 + tile * 128, dk + off, dq + off, idesc, kk > 0);
                    }
                    umma_commit_warp(bars.s_full(sb, tile));
                }
                if (!ok) break;
                umma_commit_warp(bars.q_empty(st));
            }
            umma_commit_warp(bars.k_empty(kb));
            ++ni;
        }
        if (!ok && lane == 0) count_error(p.error_count);
        umma_commit_warp(bars.drain());
        if (!mbar_wait_warp(bars.drain(), 0) && lane == 0) count_error(p.error_count);
        __syncwarp();
    } else if (warp == kLseWarp) {
        // ============================================================ lse
        for (int k = blockIdx.x; k < num_items && ok; k += gridDim.x) {
            Item it;
            if (!describe(k, it)) continue;
            const float* lse = p.lse + ((size_t)it.kvh * p.total_q + it.d.r0) * G;
            for (int t = 0; t < it.nt; ++t, ++g) {
                const int st = g % kQStages, i0 = (it.t0 + t) * per_tile;
                const int rows = min(per_tile, it.d.n - i0) * G;
                float v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[i] = lane + 32 * i < rows ? -lse[(size_t)i0 * G + lane + 32 * i] : -INFINITY;
                if (!free_slot(bars.l_empty(st), g, kQStages)) {
                    ok = false;
                    break;
                }
                float* to = reinterpret_cast<float*>(smem + kLse) + st * kTile;
#pragma unroll
                for (int i = 0; i < 4; ++i) to[lane + 32 * i] = v[i];
                __syncwarp();
                if (lane == 0) mbar_arrive(bars.l_full(st));
            }
        }
        if (!ok && lane == 0) count_error(p.error_count);
    } else {
        // ============================================================ sums
        const int quarter = warp & 3, tile = (warp - 2) >> 2;
        const int r = quarter * 32 + lane;  // this thread's key of the tile
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const float sl2 = p.scale_log2;
        const unsigned long long s2 = f32x2_pack(sl2, sl2);
        for (int k = blockIdx.x; k < num_items; k += gridDim.x) {
            Item it;
            if (!describe(k, it)) continue;
            const int j = it.j0 + tile * kTile + r;
            bool valid = j < it.d.nkeys;
            if (valid) {
                const int pb = p.block_tables[(size_t)it.d.s * p.max_blocks_per_seq + j / B];
                valid = pb >= 0 && pb < p.num_blocks;
            }
            unsigned long long sum2[2] = {f32x2_pack(0.f, 0.f), f32x2_pack(0.f, 0.f)};
            for (int t = 0; t < it.nt; ++t, ++g) {
                const int st = g % kQStages, sb = g & 1, i0 = (it.t0 + t) * per_tile;
                // rows [lo, hi) of the tile see key j
                const int hi = valid ? min(per_tile, it.d.n - i0) * G : 0;
                const int lo = max(0, j - it.d.start - i0) * G;
                if (ok && !mbar_wait(bars.l_full(st), (g / kQStages) & 1)) ok = false;
                if (ok && !mbar_wait(bars.s_full(sb, tile), (g >> 1) & 1)) ok = false;
                __syncwarp();
                tc_fence_after();
                const float4* lse = reinterpret_cast<const float4*>(smem + kLse) + st * (kTile / 4);
                const uint32_t at = tmem + lane_off + sb * 256 + tile * 128;
                const bool dense = __all_sync(0xffffffffu, lo == 0 && hi == kTile);
                float x[2][32];
                tmem_ld32(at, x[0]);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    tmem_wait_ld32(x[q & 1]);
                    if (q < 3) tmem_ld32(at + (q + 1) * 32, x[(q + 1) & 1]);
                    float(&v)[32] = x[q & 1];
                    if (dense) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float4 l = lse[q * 8 + i];
                            float y0, y1, y2, y3;
                            f32x2_unpack(fma_f32x2(f32x2_pack(v[4 * i], v[4 * i + 1]), s2, f32x2_pack(l.x, l.y)), y0, y1);
                            f32x2_unpack(fma_f32x2(f32x2_pack(v[4 * i + 2], v[4 * i + 3]), s2, f32x2_pack(l.z, l.w)), y2, y3);
                            sum2[0] = add_f32x2(sum2[0], f32x2_pack(fast_exp2(y0), fast_exp2(y1)));
                            sum2[1] = add_f32x2(sum2[1], f32x2_pack(fast_exp2(y2), fast_exp2(y3)));
                        }
                    } else {
                        const float* l1 = reinterpret_cast<const float*>(lse) + q * 32;
                        float a = 0.f;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (q * 32 + i >= lo && q * 32 + i < hi) a += fast_exp2(fmaf(v[i], sl2, l1[i]));
                        sum2[0] = add_f32x2(sum2[0], f32x2_pack(a, 0.f));
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0 && ok) {
                    mbar_arrive(bars.s_empty(sb, tile));
                    mbar_arrive(bars.l_empty(st));
                }
            }
            float a, b, c, d;
            f32x2_unpack(sum2[0], a, b);
            f32x2_unpack(sum2[1], c, d);
            if (j < it.d.nkeys)
                p.partial[(((size_t)it.c * Hkv + it.kvh) * p.pieces + it.piece) * p.partial_width + j] = (a + b) + (c + d);
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

int launch_prefill_weights_tc(const PrefillParams& p, int piece_tiles, int num_sms, cudaStream_t stream) {
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
    const long long items = (long long)p.num_chunks * p.num_kv_heads * p.pieces * ((p.max_context_len + kKeys - 1) / kKeys);
    if (items == 0) return PA_OK;
    return launch_kernel(key_weights_kernel, dim3((unsigned)(items < num_sms ? items : num_sms)), dim3(kThreads), kSmemBytes,
                         stream, tmq, tmk, p, piece_tiles);
}

}  // namespace pa
