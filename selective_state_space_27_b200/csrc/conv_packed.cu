// Short causal depthwise convolution over packed sequences (channels
// contiguous), for prompts and for single tokens:
//   y[t, c] = act(bias[c] + sum_k w[c, k] x[t - W + 1 + k, c])
// ("Notas sobre Mamba", section "O bloco Mamba": the short convolution and
// SiLU in front of the SSM; the Mamba-2 block runs it over x, B and C.)
//
// Every input is read once and every output written once, with W + 4 or so
// float32 operations per element: bound by HBM bandwidth. A thread owns four
// channels and slides a window of W inputs down the tokens in registers, so an
// input is loaded once per tile of tokens plus W - 1 look-back rows per tile.
// Measured on B200 for 24000 tokens x 4352 channels, bf16, W = 4: 83 us (77% of
// the measured copy bandwidth). The next rows of a thread wait in shared memory
// (with the next four in registers 85 us). Four rows at a time, three times: 84
// us with two times or with two rows, 88 us with eight rows twice; 88 us with 1280
// threads per SM (48 registers: spills), 89 us with blocks of 256 threads instead
// of 64 (28 warps per SM fit instead of 32). Measured before the rows waited in
// shared memory: eight channels per thread 117 us (too few warps), two 89 us,
// eight tiles per thread instead of one stretch of rows 104 us. The special
// function unit is 64% busy (exponential and reciprocal of the SiLU). float32: 154
// us (83%). 4353 channels, one per thread without rows ahead in shared
// memory: 156 us in bf16, 208 in float32.
//
// Two kinds of work. A tile is a stretch of consecutive rows of the packed
// stream, whatever sequences they belong to, except each sequence's first
// W - 1 tokens. Those, which read the state, are the sequence's own work,
// which then also replaces the state by the last W - 1 inputs: the state is
// read and written by the same thread, so updating it in place needs no
// ordering between blocks. Single tokens are the sequences' work alone.
#include "launch.h"
#include "packed.cuh"
#include "vec.cuh"

namespace ms {
namespace {

constexpr int S = 3, U = 4;                // batches in shared memory, rows of a batch
constexpr int kMaxThreads = 64;
constexpr int kThreadsPerSm = 1024;        // threads that run together on an SM

template <typename T, int VEC, int W>
struct Taps {
    float w[W][VEC], b[VEC];
    int silu;
    __device__ __forceinline__ void load(const ConvPackedParams &p, int64_t c) {
        // the VEC x W weights of the thread are consecutive; 16 bytes at a time where they are aligned
        float t[VEC * W];
        const float *src = p.weight + c * W;
        if (VEC * W % 4 == 0 && p.w_vec) {
#pragma unroll
            for (int i = 0; i < VEC * W / 4; ++i) {
                const float4 q = __ldg(reinterpret_cast<const float4 *>(src) + i);
                t[4 * i] = q.x; t[4 * i + 1] = q.y; t[4 * i + 2] = q.z; t[4 * i + 3] = q.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < VEC * W; ++i) t[i] = __ldg(src + i);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
#pragma unroll
            for (int k = 0; k < W; ++k) w[k][e] = t[e * W + k];
            b[e] = p.bias ? __ldg(p.bias + c + e) : 0.f;
        }
        silu = p.silu;
    }
    // window: the W inputs that end at this token, oldest first
    __device__ __forceinline__ Raw<T, VEC> apply(const float (&win)[W][VEC]) const {
        float o[VEC];
        if constexpr (VEC == 1) {
            float acc = b[0];
#pragma unroll
            for (int k = 0; k < W; ++k) acc = fmaf(w[k][0], win[k][0], acc);
            o[0] = silu ? acc * sigmoid(acc) : acc;
        } else {
#pragma unroll
            for (int e = 0; e < VEC; e += 2) {
                float2 acc = f2(b[e], b[e + 1]);
#pragma unroll
                for (int k = 0; k < W; ++k) acc = fma2(f2(w[k][e], w[k][e + 1]), f2(win[k][e], win[k][e + 1]), acc);
                if (silu) acc = mul2(acc, sigmoid2(acc));
                o[e] = acc.x;
                o[e + 1] = acc.y;
            }
        }
        return narrow<T, VEC>(o);
    }
};

template <int W, int VEC>
__device__ __forceinline__ void shift(float (&win)[W][VEC]) {
#pragma unroll
    for (int k = 0; k + 1 < W; ++k)
#pragma unroll
        for (int e = 0; e < VEC; ++e) win[k][e] = win[k + 1][e];
}

// The first W - 1 tokens of sequence s and its state.
template <typename T, int VEC, int W>
__device__ __forceinline__ void sequence_start(const ConvPackedParams &p, const Taps<T, VEC, W> &f, int64_t s,
                                               int64_t c, bool on) {
    const SeqRange q = seq_range(p.cu, s, p.tokens);
    const int slot = p.state || p.idx ? block_slot(p.idx, s, p.slots) : 0;
    if (slot < 0 || !on) return;
    const T *x = static_cast<const T *>(p.x) + c;
    T *y = static_cast<T *>(p.y) + c;
    const int len = q.end - q.begin;
    const bool resumed = p.state && (!p.cu || (p.has_init && p.has_init[s]));
    T *st = static_cast<T *>(p.state) + slot * p.st_slot + c;
    constexpr int H = W > 1 ? W - 1 : 1;
    Raw<T, VEC> hist[H] = {}, in[H] = {};
    if (W > 1 && resumed) {
#pragma unroll
        for (int j = 0; j + 1 < W; ++j) hist[j] = *reinterpret_cast<const Raw<T, VEC> *>(st + j * p.st_row);
    }
#pragma unroll
    for (int j = 0; j + 1 < W; ++j)
        if (j < len) in[j] = load_raw<T, VEC>(x + (q.begin + static_cast<int64_t>(j)) * p.x_st);
    float win[W][VEC] = {};
#pragma unroll
    for (int j = 0; j + 1 < W; ++j) widen<T, VEC>(hist[j], win[j + 1]);
#pragma unroll
    for (int j = 0; j + 1 < W; ++j) {
        if (j < len) {
            shift<W, VEC>(win);
            widen<T, VEC>(in[j], win[W - 1]);
            store_raw<T, VEC>(y + (q.begin + static_cast<int64_t>(j)) * p.y_st, f.apply(win));
        }
    }
    if constexpr (W == 1) {
        // no history: the tiles take every token, except in the single-token form, which has none
        if (!p.cu) {
            widen<T, VEC>(load_raw<T, VEC>(x + q.begin * p.x_st), win[0]);
            store_raw<T, VEC>(y + q.begin * p.y_st, f.apply(win));
        }
        return;
    }
    if (!p.state) return;
    // the last W - 1 of (history, inputs)
#pragma unroll
    for (int j = 0; j + 1 < W; ++j) {
        Raw<T, VEC> r{};
        if (len >= W - 1) {
            r = load_raw<T, VEC>(x + (q.end - static_cast<int64_t>(W - 1) + j) * p.x_st);
        } else {
#pragma unroll
            for (int l = 0; l + 1 < W; ++l)
                if (l == len) {
                    if (j + l < W - 1) r = hist[j + l < H ? j + l : 0];
                    else r = in[j + l - (W - 1) >= 0 ? j + l - (W - 1) : 0];
                }
        }
        store_raw<T, VEC>(st + j * p.st_row, r);
    }
}

// One value of the ring (8 or 16 bytes).
template <typename R>
__device__ __forceinline__ R load_ring(uint32_t at) {
    union { R r; uint32_t w[sizeof(R) / 4]; } v;
    if constexpr (sizeof(R) == 8)
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.w[0]), "=r"(v.w[1]) : "r"(at) : "memory");
    else
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]) : "r"(at) : "memory");
    return v.r;
}

// Rows [t0, t1) of the packed stream, without the first W - 1 of each sequence.
template <typename T, int VEC, int W>
__device__ __forceinline__ void tile_rows(const ConvPackedParams &p, const Taps<T, VEC, W> &f, int t0, int t1,
                                          int64_t c, bool on, uint32_t ring) {
    const T *x = static_cast<const T *>(p.x) + c;
    T *y = static_cast<T *>(p.y) + c;
    const int nseq = static_cast<int>(p.nseq);
    int t = t0;
    for (int s = seq_of_token(p.cu, nseq, t0); s < nseq && t < t1; ++s) {
        const SeqRange q = seq_range(p.cu, s, p.tokens);
        if (q.begin >= t1) break;
        int from = max(t, min(q.begin + (W - 1), q.end));
        const int to = min(t1, q.end);
        t = max(t, to);
        if (from >= to) continue;
        if ((p.state || p.idx) && block_slot(p.idx, s, p.slots) < 0) continue;
        if (!on) continue;
        float win[W][VEC] = {};
#pragma unroll
        for (int j = 0; j + 1 < W; ++j)
            widen<T, VEC>(load_raw<T, VEC>(x + (from - (W - 1) + static_cast<int64_t>(j)) * p.x_st), win[j + 1]);
        const T *xp = x + from * p.x_st;
        T *yp = y + from * p.y_st;
        constexpr int B = sizeof(Raw<T, VEC>);
        if constexpr (B >= 8) {
            // batches of U rows on their way in shared memory (each thread its own values)
            const int batches = (to - from) / U;
            auto place = [&](int b, int u) {
                return ring + (static_cast<uint32_t>(b % S * U + u) * blockDim.x + threadIdx.x) * B;
            };
            const T *ahead = xp;
            auto issue = [&](int b) {
                if (b < batches) {
#pragma unroll
                    for (int u = 0; u < U; ++u) cp_async_full<B>(place(b, u), ahead + u * p.x_st);
                    ahead += U * p.x_st;
                }
                cp_async_commit();
            };
#pragma unroll
            for (int b = 0; b + 1 < S; ++b) issue(b);
            for (int b = 0; b < batches; ++b) {
                issue(b + S - 1);
                cp_async_wait<S - 1>();
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    shift<W, VEC>(win);
                    widen<T, VEC>(load_ring<Raw<T, VEC>>(place(b, u)), win[W - 1]);
                    store_raw<T, VEC>(yp + u * p.y_st, f.apply(win));
                }
                yp += U * p.y_st;
            }
            from += batches * U;
            xp += static_cast<int64_t>(batches) * U * p.x_st;
        }
        for (; from < to; ++from) {
            shift<W, VEC>(win);
            widen<T, VEC>(load_raw<T, VEC>(xp), win[W - 1]);
            store_raw<T, VEC>(yp, f.apply(win));
            xp += p.x_st;
            yp += p.y_st;
        }
    }
}

// A block keeps the filters of its channels and takes the sequences and the
// tiles blockIdx.x, blockIdx.x + gridDim.x, ...
template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kMaxThreads, kThreadsPerSm / kMaxThreads) conv_packed_kernel(const ConvPackedParams p) {
    extern __shared__ __align__(16) uint8_t rows_ahead[];
    const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(rows_ahead));
    const int64_t c = (static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x) * VEC;
    const bool on = c < p.channels;
    Taps<T, VEC, W> f;
    if (on) f.load(p, c);
    for (int64_t i = blockIdx.x; i < p.nseq; i += gridDim.x) sequence_start<T, VEC, W>(p, f, i, c, on);
    // (the first tile of a block: where its count of sequences left off)
    const int64_t skip = p.nseq % gridDim.x, b = blockIdx.x;
    for (int64_t i = b >= skip ? b - skip : b + gridDim.x - skip; i < p.tiles; i += gridDim.x)
        tile_rows<T, VEC, W>(p, f, static_cast<int>(i * p.tile), static_cast<int>(min64((i + 1) * p.tile, p.tokens)), c,
                             on, ring);
}

template <typename T, int VEC>
cudaError_t launch_w(const ConvPackedParams &p0, int num_sms, cudaStream_t stream) {
    ConvPackedParams p = p0;
    const int64_t nvec = (p.channels + VEC - 1) / VEC;
    // warps of channels, spread evenly over blocks of at most kMaxThreads threads
    const int64_t warps = (nvec + 31) / 32, nb = (warps * 32 + kMaxThreads - 1) / kMaxThreads;
    const int threads = static_cast<int>((warps + nb - 1) / nb) * 32;
    // As many blocks as run together, each with one stretch of rows (at least 8:
    // every stretch reads W - 1 look-back rows again) and its share of the sequences.
    const int64_t most = max64(1, static_cast<int64_t>(kThreadsPerSm / threads) * num_sms / nb);
    p.tile = max64(8, ((p.tokens + most - 1) / most + 3) / 4 * 4);
    p.tiles = p.cu ? (p.tokens + p.tile - 1) / p.tile : 0;
    p.w_vec = reinterpret_cast<uintptr_t>(p.weight) % 16 == 0;
    const dim3 grid(static_cast<unsigned>(min64(p.nseq + p.tiles, most)), static_cast<unsigned>(nb));
    const size_t smem = p.tiles && sizeof(Raw<T, VEC>) >= 8 ? sizeof(Raw<T, VEC>) * S * U * threads : 0;
    switch (p.width) {
    case 1: conv_packed_kernel<T, VEC, 1><<<grid, threads, smem, stream>>>(p); break;
    case 2: conv_packed_kernel<T, VEC, 2><<<grid, threads, smem, stream>>>(p); break;
    case 3: conv_packed_kernel<T, VEC, 3><<<grid, threads, smem, stream>>>(p); break;
    default: conv_packed_kernel<T, VEC, 4><<<grid, threads, smem, stream>>>(p); break;
    }
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const ConvPackedParams &p, int num_sms, cudaStream_t stream) {
    const int eb = sizeof(T);
    auto ok = [&](int vec) {
        return p.channels % vec == 0 && vec_ok(p.x, p.x_st, eb, vec) && vec_ok(p.y, p.y_st, eb, vec) &&
               vec_ok(p.state, p.st_slot, eb, vec) && vec_ok(p.state, p.st_row, eb, vec);
    };
    // Four channels per thread where sizes, strides and pointers allow it, else one.
    if (ok(4)) return launch_w<T, 4>(p, num_sms, stream);
    // One channel each: at most as many at a time as a grid's 65535 blocks in y hold.
    constexpr int64_t kMost = static_cast<int64_t>(65535) * kMaxThreads;
    for (int64_t c = 0; c < p.channels; c += kMost) {
        ConvPackedParams q = p;
        q.channels = min64(p.channels - c, kMost);
        q.x = static_cast<const T *>(p.x) + c;
        q.y = static_cast<T *>(p.y) + c;
        if (p.state) q.state = static_cast<T *>(p.state) + c;
        q.weight = p.weight + c * p.width;
        if (p.bias) q.bias = p.bias + c;
        const cudaError_t e = launch_w<T, 1>(q, num_sms, stream);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_conv_packed(const ConvPackedParams &p, int in_dtype, int num_sms, cudaStream_t stream) {
    return in_dtype == 0 ? launch_t<float>(p, num_sms, stream) : launch_t<__nv_bfloat16>(p, num_sms, stream);
}

}  // namespace ms
