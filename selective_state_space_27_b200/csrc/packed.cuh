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

// First sequence whose end lies behind token t (nseq if none does).
__device__ __forceinline__ int seq_of_token(const int32_t *cu, int nseq, int t) {
    int lo = 0, hi = nseq;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(cu + mid + 1) > t) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

}  // namespace ms
