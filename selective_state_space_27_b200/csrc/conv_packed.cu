// Short causal depthwise convolution over packed sequences (channels
// contiguous), for prompts and for single tokens:
//   y[t, c] = act(bias[c] + sum_k w[c, k] x[t - W + 1 + k, c])
// ("Notas sobre Mamba", section "O bloco Mamba": the short convolution and
// SiLU in front of the SSM; the Mamba-2 block runs it over x, B and C.)
//
// Every input is read once and every output written once, with W + 4 or so
// float32 operations per element: the kernel is bound by HBM bandwidth. A
// thread owns VEC channels (16 bytes) and slides a window of W inputs down the
// tokens in registers, so an input is loaded once per tile of tokens plus W - 1
// look-back rows per tile.
//
// Two kinds of blocks. A tile block takes `tile` consecutive rows of the packed
// stream, whatever sequences they belong to, except each sequence's first
// W - 1 tokens. Those, which read the state, belong to the sequence's own
// block, which then also replaces the state by the last W - 1 inputs: the
// state is read and written by the same thread, so updating it in place needs
// no ordering between blocks. Single tokens are the sequence blocks alone.
#include "launch.h"
#include "packed.cuh"
#include "vec.cuh"

namespace ms {
namespace {

constexpr int kMaxThreads = 256;

template <typename T, int VEC, int W>
struct Taps {
    float w[W][VEC], b[VEC];
    int silu;
    __device__ __forceinline__ void load(const ConvPackedParams &p, int64_t c) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
#pragma unroll
            for (int k = 0; k < W; ++k) w[k][e] = __ldg(p.weight + (c + e) * W + k);
            b[e] = p.bias ? __ldg(p.bias + c + e) : 0.f;
        }
        silu = p.silu;
    }
    // window: the W inputs that end at this token, oldest first
    __device__ __forceinline__ Raw<T, VEC> apply(const float (&win)[W][VEC]) const {
        float o[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float acc = b[e];
#pragma unroll
            for (int k = 0; k < W; ++k) acc = fmaf(w[k][e], win[k][e], acc);
            o[e] = silu ? acc * sigmoid(acc) : acc;
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

template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kMaxThreads) conv_packed_kernel(const ConvPackedParams p) {
    const int64_t c = (static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x) * VEC;
    const bool on = c < p.channels;
    const T *x = static_cast<const T *>(p.x) + c;
    T *y = static_cast<T *>(p.y) + c;

    if (blockIdx.x < p.nseq) {
        const int64_t s = blockIdx.x;
        const SeqRange q = seq_range(p.cu, s, p.tokens);
        const int slot = p.state || p.idx ? block_slot(p.idx, s, p.slots) : 0;
        if (slot < 0 || !on) return;
        const int len = q.end - q.begin;
        const bool resumed = p.state && (!p.cu || (p.has_init && p.has_init[s]));
        T *st = static_cast<T *>(p.state) + slot * p.st_slot + c;
        Taps<T, VEC, W> f;
        f.load(p, c);
        constexpr int H = W > 1 ? W - 1 : 1;
        Raw<T, VEC> hist[H] = {}, in[H] = {};
        if (W > 1 && resumed) {
#pragma unroll
            for (int j = 0; j < W - 1; ++j) hist[j] = *reinterpret_cast<const Raw<T, VEC> *>(st + j * p.st_row);
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            if (j < len) in[j] = load_raw<T, VEC>(x + (q.begin + static_cast<int64_t>(j)) * p.x_st);
        float win[W][VEC] = {};
#pragma unroll
        for (int j = 0; j < W - 1; ++j) widen<T, VEC>(hist[j], win[j + 1]);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            if (j < len) {
                shift<W, VEC>(win);
                widen<T, VEC>(in[j], win[W - 1]);
                store_raw<T, VEC>(y + (q.begin + static_cast<int64_t>(j)) * p.y_st, f.apply(win));
            }
        }
        if (W == 1 || !p.state) return;
        // the last W - 1 of (history, inputs)
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            Raw<T, VEC> r{};
            if (len >= W - 1) {
                r = load_raw<T, VEC>(x + (q.end - static_cast<int64_t>(W - 1) + j) * p.x_st);
            } else {
#pragma unroll
                for (int l = 0; l < W - 1; ++l)
                    if (l == len) r = j + l < W - 1 ? hist[j + l < W - 1 ? j + l : 0] : in[j + l - (W - 1) >= 0 ? j + l - (W - 1) : 0];
            }
            store_raw<T, VEC>(st + j * p.st_row, r);
        }
        return;
    }

    // rows [t0, t1) of the packed stream
    const int64_t t0 = (static_cast<int64_t>(blockIdx.x) - p.nseq) * p.tile;
    const int t1 = static_cast<int>(min64(t0 + p.tile, p.tokens));
    const int nseq = static_cast<int>(p.nseq);
    int t = static_cast<int>(t0);
    int s = seq_of_token(p.cu, nseq, t);
    Taps<T, VEC, W> f;
    if (on) f.load(p, c);
    for (; s < nseq && t < t1; ++s) {
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
        for (int j = 0; j < W - 1; ++j)
            widen<T, VEC>(load_raw<T, VEC>(x + (from - (W - 1) + static_cast<int64_t>(j)) * p.x_st), win[j + 1]);
        constexpr int U = 8;   // loads in flight per thread
        const T *xp = x + from * p.x_st;
        T *yp = y + from * p.y_st;
        for (; from + U <= to; from += U) {
            Raw<T, VEC> r[U];
#pragma unroll
            for (int u = 0; u < U; ++u) r[u] = load_raw<T, VEC>(xp + u * p.x_st);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                shift<W, VEC>(win);
                widen<T, VEC>(r[u], win[W - 1]);
                store_raw<T, VEC>(yp + u * p.y_st, f.apply(win));
            }
            xp += U * p.x_st;
            yp += U * p.y_st;
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

template <typename T, int VEC>
cudaError_t launch_w(const ConvPackedParams &p0, int num_sms, cudaStream_t stream) {
    ConvPackedParams p = p0;
    const int64_t nvec = (p.channels + VEC - 1) / VEC;
    // warps of channels, spread evenly over blocks of at most kMaxThreads threads
    const int64_t warps = (nvec + 31) / 32, nb = (warps * 32 + kMaxThreads - 1) / kMaxThreads;
    const int threads = static_cast<int>((warps + nb - 1) / nb) * 32;
    // Longer tiles re-read fewer look-back rows (W - 1 per tile); short ones
    // give a small call enough blocks to fill the SMs.
    p.tile = 32;
    while (p.tile > 8 && (p.tokens + p.tile - 1) / p.tile * nb < 4 * num_sms) p.tile /= 2;
    const int64_t tiles = p.cu ? (p.tokens + p.tile - 1) / p.tile : 0;
    const dim3 grid(static_cast<unsigned>(p.nseq + tiles), static_cast<unsigned>(nb));
    switch (p.width) {
    case 1: conv_packed_kernel<T, VEC, 1><<<grid, threads, 0, stream>>>(p); break;
    case 2: conv_packed_kernel<T, VEC, 2><<<grid, threads, 0, stream>>>(p); break;
    case 3: conv_packed_kernel<T, VEC, 3><<<grid, threads, 0, stream>>>(p); break;
    default: conv_packed_kernel<T, VEC, 4><<<grid, threads, 0, stream>>>(p); break;
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
    // 16-byte vectors where sizes, strides and pointers allow them, else single elements
    if (ok(16 / eb)) return launch_w<T, 16 / eb>(p, num_sms, stream);
    return launch_w<T, 1>(p, num_sms, stream);
}

}  // namespace

cudaError_t launch_conv_packed(const ConvPackedParams &p, int in_dtype, int num_sms, cudaStream_t stream) {
    return in_dtype == 0 ? launch_t<float>(p, num_sms, stream) : launch_t<__nv_bfloat16>(p, num_sms, stream);
}

}  // namespace ms
