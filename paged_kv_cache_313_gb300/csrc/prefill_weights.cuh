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
        d.start < 0)
        return false;
    d.cap = min(min(p.context_lens[d.s], p.max_context_len),
                (int)min((long long)p.max_blocks_per_seq * p.block_size, 0x7FFFFFFFLL));
    d.nkeys = max(0, (int)min((long long)d.start + d.n, (long long)d.cap));
    if (d.n == 0) d.nkeys = 0;
    return true;
}

}  // namespace pa
