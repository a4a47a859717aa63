// prefill_weights.cuh — a chunk of pa_prefill_chunk_weights as its kernels see it.
#pragma once

#include "pa_internal.cuh"

namespace pa {

struct WeightChunk {
    int r0, n, s, start;
    int cap;    // tokens of the sequence that may be read
    int nkeys;  // keys that the chunk's queries see: [0, nkeys)
};

// false for a chunk that cannot be used (the attention kernel counts it).
__device__ __forceinline__ bool weight_chunk(const PrefillParams& p, int c, WeightChunk& d) {
    d.r0 = p.cu_q_lens[c];
    d.n = p.cu_q_lens[c + 1] - d.r0;
    d.s = p.seq_of_chunk[c];
    d.start = p.q_start_pos[c];
    if (d.n < 0 || d.r0 < 0 || d.r0 + d.n > p.total_q || d.n > p.max_q_len || d.s < 0 || d.s >= p.num_seqs ||
        d.start < 0 || d.start > 0x7FFFFFFF - d.n)
        return false;
    d.cap = min(min(p.context_lens[d.s], p.max_context_len),
                (int)min((long long)p.max_blocks_per_seq * p.block_size, 0x7FFFFFFFLL));
    d.nkeys = max(0, (int)min((long long)d.start + d.n, (long long)d.cap));
    if (d.n == 0) d.nkeys = 0;
    return true;
}

// The tensor-core path (prefill_weights_tc.cu): pairs of 128-key tiles, tiles of 128 query rows (128 / G positions).
constexpr int kKeys = 256;
__device__ __forceinline__ int key_pairs(const WeightChunk& d) { return (d.nkeys + kKeys - 1) / kKeys; }
__device__ __forceinline__ int key_tiles(const WeightChunk& d, int per_tile) { return (d.n + per_tile - 1) / per_tile; }
// The first query tile that sees a key of the pair (there is one: its first key is below nkeys).
__device__ __forceinline__ int key_first_tile(const WeightChunk& d, int pair, int per_tile) {
    return max(0, pair * kKeys - d.start) / per_tile;
}
// (pair, query tile) units of one kv head, those of pairs below `pairs`.
__device__ __forceinline__ long long key_units(const WeightChunk& d, int per_tile, int pairs) {
    long long units = (long long)pairs * key_tiles(d, per_tile);
    for (int pair = d.start / kKeys + 1; pair < pairs; ++pair) units -= key_first_tile(d, pair, per_tile);
    return units;
}
__device__ __forceinline__ long long key_units(const WeightChunk& d, int per_tile) {
    return key_units(d, per_tile, key_pairs(d));
}

}  // namespace pa
