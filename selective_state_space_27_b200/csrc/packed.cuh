// Packed sequences and their cache slots, as every serving kernel reads them.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace ms {

// Rows [begin, end) of sequence s: the values of cu_seqlens clamped to [0,
// tokens], so that no malformed value reaches memory outside the tensors.
struct SeqRange {
    int begin, end;
};

__device__ __forceinline__ SeqRange seq_range(const int32_t *cu, int64_t s, int64_t tokens) {
    if (!cu) return {static_cast<int>(s), static_cast<int>(s) + 1};
    const int t = static_cast<int>(tokens);
    const int a = min(max(__ldg(cu + s), 0), t);
    const int b = min(max(__ldg(cu + s + 1), a), t);
    return {a, b};
}

// The cache slot of sequence s, or -1 when the sequence is skipped: its index
// lies outside the cache, or an earlier sequence has the same one (two writers
// of one entry would race). Called by all threads of the block with the same
// s; the earlier indices are compared by all of them together. Without an
// index table sequence s has slot s.
__device__ __forceinline__ int block_slot(const int32_t *idx, int64_t s, int64_t slots) {
    if (!idx) return s < slots ? static_cast<int>(s) : -1;
    const int v = __ldg(idx + s);
    const bool in = v >= 0 && v < slots;
    bool twin = false;
    if (in)
        for (int64_t j = threadIdx.x; j < s; j += blockDim.x) twin |= __ldg(idx + j) == v;
    return __syncthreads_or(twin) || !in ? -1 : v;
}

// First sequence whose end lies behind token t (nseq if none does). Called by
// whole warps, whose lanes look at 32 sequences in one round of loads.
__device__ __forceinline__ int seq_of_token(const int32_t *cu, int nseq, int t) {
    const int lane = threadIdx.x & 31;
    int lo = 0;
    for (int n = nseq; n > 0;) {
        const int step = (n + 31) / 32, c = lane * step;
        const bool ended = c < n && __ldg(cu + lo + c + 1) <= t;
        const int k = __popc(__ballot_sync(0xffffffffu, ended));   // (the first k probes, the offsets never fall)
        if (k == 0) break;
        lo += (k - 1) * step + 1;
        n = min(step - 1, n - (k - 1) * step - 1);
    }
    return lo;
}

}  // namespace ms
