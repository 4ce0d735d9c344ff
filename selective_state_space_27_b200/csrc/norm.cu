// RMS norm fused with the residual sum (before a block) or the SiLU gate
// (after it), by groups of channels, forward and backward, in float32:
//   v = x [silu(z)];  v = residual + scale v;  y = v r w [silu(z)],
//   r = 1 / sqrt(mean(v^2) + eps)
// Backward, with n = v r, u = dy w (dy silu(z) w for the gate behind the norm):
//   dv = (u - n mean(u n)) r + dsum,  dresidual = dv,
//   dx = scale dv [silu(z)],  dz = scale dv x silu'(z)  or  dy n w silu'(z),
//   dw = sum over rows of dy n  (the sums over rows in a fixed order)
//
// A row's values are read once, kept in registers between the reduction and
// the result, and written once: both directions are bound by HBM bandwidth. A
// team of threads owns one (row, group): up to a warp for small groups
// (several teams per warp for very small ones), a block for long ones. In the
// backward a team stays on one group of channels and walks down the rows of
// its slab, so that its share of dw stays in registers; the slabs' shares are
// added by a second kernel.
#include "launch.h"
#include "vec.cuh"

namespace ms {
namespace {

constexpr int kWarps = 4;                // warps per block of the warp-team kernels
constexpr int kMaxBlock = 512;           // threads of a block team

// Sum over a team: `ts` lanes of a warp (a power of two), or the whole block.
template <bool BLOCK, int K>
__device__ __forceinline__ void team_sum(float (&v)[K], int ts, float *smem) {
    for (int o = (BLOCK ? 32 : ts) >> 1; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if constexpr (BLOCK) {
        const int warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
        __syncthreads();   // the previous sum's values have been read
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int k = 0; k < K; ++k) smem[k * 32 + warp] = v[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float t = 0.f;
            for (int w = 0; w < nw; ++w) t += smem[k * 32 + w];
            v[k] = t;
        }
    }
}

// The value that is normed, of VEC channels at element i of the row; `sum` is
// what residual_out stores.
template <typename T, typename R, int VEC>
struct FwdRow {
    const T *x, *z;
    const R *res;
    R *ro;
    T *y;
    const float *w;
    __device__ __forceinline__ FwdRow(const NormParams &p, int64_t row, int64_t c0)
        : x(static_cast<const T *>(p.x) + row * p.x_sr + c0),
          z(p.z ? static_cast<const T *>(p.z) + row * p.z_sr + c0 : nullptr),
          res(p.res ? static_cast<const R *>(p.res) + row * p.res_sr + c0 : nullptr),
          ro(p.res ? static_cast<R *>(p.ro) + row * p.ro_sr + c0 : nullptr),
          y(static_cast<T *>(p.y) + row * p.y_sr + c0), w(p.w ? p.w + c0 : nullptr) {}
};

template <typename T, typename R, int VEC>
__device__ __forceinline__ void norm_value(const NormParams &p, const Raw<T, VEC> &xr, const Raw<T, VEC> &zr,
                                           const Raw<R, VEC> &rr, float (&v)[VEC]) {
    widen<T, VEC>(xr, v);
    if (p.z && p.gate_first) {
        float z[VEC];
        widen<T, VEC>(zr, z);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] *= z[e] * sigmoid(z[e]);
    }
    if (p.res) {
        float r[VEC];
        widen<R, VEC>(rr, r);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = fmaf(p.scale, v[e], r[e]);
    }
}

template <typename T, typename R, int VEC>
__device__ __forceinline__ void norm_store(const NormParams &p, const FwdRow<T, R, VEC> &row, int64_t i, float r,
                                           const float (&v)[VEC], const Raw<T, VEC> &zr) {
    float w[VEC], o[VEC];
    if (row.w) load_f32<VEC>(row.w + i, w);
#pragma unroll
    for (int e = 0; e < VEC; ++e) o[e] = row.w ? v[e] * r * w[e] : v[e] * r;
    if (p.z && !p.gate_first) {
        float z[VEC];
        widen<T, VEC>(zr, z);
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] *= z[e] * sigmoid(z[e]);
    }
    store_raw<T, VEC>(row.y + i, narrow<T, VEC>(o));
}

// One (row, group) per team; NV vectors per thread in registers.
template <typename T, typename R, int VEC, int NV, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? kMaxBlock : kWarps * 32) norm_fwd_kernel(const NormParams p) {
    __shared__ float smem[32];
    const int ts = BLOCK ? (int)blockDim.x : p.team;
    const int lane = BLOCK ? (int)threadIdx.x : (int)(threadIdx.x & (ts - 1));
    const int64_t item = BLOCK ? blockIdx.x
                               : static_cast<int64_t>(blockIdx.x) * (blockDim.x / ts) + threadIdx.x / ts;
    const bool on = item < p.rows * p.groups;   // (false only in the last block of warp teams)
    const int64_t row = on ? item / p.groups : 0, c0 = on ? (item % p.groups) * p.gs : 0;
    const FwdRow<T, R, VEC> q(p, row, c0);
    const int nvec = on ? static_cast<int>(p.gs / VEC) : 0;
    Raw<T, VEC> xr[NV], zr[NV];
    Raw<R, VEC> rr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = lane + i * ts;
        xr[i] = {};
        zr[i] = {};
        rr[i] = {};
        if (j < nvec) {
            xr[i] = load_raw<T, VEC>(q.x + j * VEC);
            if (q.z) zr[i] = load_raw<T, VEC>(q.z + j * VEC);
            if (q.res) rr[i] = load_raw<R, VEC>(q.res + j * VEC);
        }
    }
    float v[NV][VEC], ss[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        norm_value<T, R, VEC>(p, xr[i], zr[i], rr[i], v[i]);
        const int j = lane + i * ts;
        if (j < nvec) {
            if (q.ro) store_raw<R, VEC>(q.ro + j * VEC, narrow<R, VEC>(v[i]));
#pragma unroll
            for (int e = 0; e < VEC; ++e) ss[0] = fmaf(v[i][e], v[i][e], ss[0]);
        }
    }
    team_sum<BLOCK, 1>(ss, ts, smem);
    const float r = rsqrtf(ss[0] * p.inv_gs + p.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = lane + i * ts;
        if (j < nvec) norm_store<T, R, VEC>(p, q, j * VEC, r, v[i], zr[i]);
    }
}

// Groups too long for the registers of a block: two passes over the row.
template <typename T, typename R, int VEC>
__global__ void __launch_bounds__(kMaxBlock) norm_fwd_long_kernel(const NormParams p) {
    __shared__ float smem[32];
    const int64_t row = blockIdx.x / p.groups, c0 = (blockIdx.x % p.groups) * p.gs;
    const FwdRow<T, R, VEC> q(p, row, c0);
    const int64_t nvec = p.gs / VEC;
    float ss[1] = {0.f};
    auto value = [&](int64_t j, Raw<T, VEC> &zr, float(&v)[VEC]) {
        Raw<R, VEC> rr{};
        zr = {};
        if (q.z) zr = load_raw<T, VEC>(q.z + j * VEC);
        if (q.res) rr = load_raw<R, VEC>(q.res + j * VEC);
        norm_value<T, R, VEC>(p, load_raw<T, VEC>(q.x + j * VEC), zr, rr, v);
    };
    for (int64_t j = threadIdx.x; j < nvec; j += blockDim.x) {
        Raw<T, VEC> zr;
        float v[VEC];
        value(j, zr, v);
        if (q.ro) store_raw<R, VEC>(q.ro + j * VEC, narrow<R, VEC>(v));
#pragma unroll
        for (int e = 0; e < VEC; ++e) ss[0] = fmaf(v[e], v[e], ss[0]);
    }
    team_sum<true, 1>(ss, 0, smem);
    const float r = rsqrtf(ss[0] * p.inv_gs + p.eps);
    for (int64_t j = threadIdx.x; j < nvec; j += blockDim.x) {
        Raw<T, VEC> zr;
        float v[VEC];
        value(j, zr, v);
        norm_store<T, R, VEC>(p, q, j * VEC, r, v, zr);
    }
}

// ---- backward ----------------------------------------------------------------

template <typename T, typename R, int VEC>
struct BwdRow {
    const T *dy, *x, *z;
    const R *sum, *ds;
    T *dx, *dz;
    R *dres;
    __device__ __forceinline__ BwdRow(const NormParams &p, const NormBwdParams &g, int64_t row, int64_t c0)
        : dy(static_cast<const T *>(g.dy) + row * g.dy_sr + c0),
          x(g.need_x ? static_cast<const T *>(p.x) + row * p.x_sr + c0 : nullptr),
          z(p.z ? static_cast<const T *>(p.z) + row * p.z_sr + c0 : nullptr),
          sum(p.ro ? static_cast<const R *>(p.ro) + row * p.ro_sr + c0 : nullptr),
          ds(g.dro ? static_cast<const R *>(g.dro) + row * g.dro_sr + c0 : nullptr),
          dx(static_cast<T *>(g.dx) + row * g.dx_sr + c0),
          dz(p.z ? static_cast<T *>(g.dz) + row * g.dz_sr + c0 : nullptr),
          dres(p.ro ? static_cast<R *>(g.dres) + row * g.dres_sr + c0 : nullptr) {}
};

// What one thread knows of VEC channels of a row before the reductions.
template <typename T, typename R, int VEC>
struct BwdVec {
    Raw<T, VEC> dy, x, z;
    Raw<R, VEC> sum, ds;
    __device__ __forceinline__ void load(const BwdRow<T, R, VEC> &q, int64_t i) {
        dy = load_raw<T, VEC>(q.dy + i);
        if (q.x) x = load_raw<T, VEC>(q.x + i);
        if (q.z) z = load_raw<T, VEC>(q.z + i);
        if (q.sum) sum = load_raw<R, VEC>(q.sum + i);
        if (q.ds) ds = load_raw<R, VEC>(q.ds + i);
    }
    // v, and dy as it reaches the norm's output (before the weight)
    __device__ __forceinline__ void values(const NormParams &p, float (&v)[VEC], float (&d)[VEC]) const {
        widen<T, VEC>(dy, d);
        if (p.ro) widen<R, VEC>(sum, v);
        else widen<T, VEC>(x, v);
        if (p.z && (!p.ro || !p.gate_first)) {
            float zf[VEC];
            widen<T, VEC>(z, zf);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float s = zf[e] * sigmoid(zf[e]);
                if (p.gate_first) v[e] *= s;
                else d[e] *= s;
            }
        }
    }
    // the gradients, from r and m = mean(u v) r^3 (u = d w)
    __device__ __forceinline__ void store(const NormParams &p, const BwdRow<T, R, VEC> &q, int64_t i, float r, float m,
                                          const float (&v)[VEC], const float (&d)[VEC], const float (&w)[VEC]) const {
        float dv[VEC], zf[VEC], sg[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) dv[e] = fmaf(r, d[e] * w[e], -m * v[e]);
        if (q.sum) {
            if (q.ds) {
                float t[VEC];
                widen<R, VEC>(ds, t);
#pragma unroll
                for (int e = 0; e < VEC; ++e) dv[e] += t[e];
            }
            store_raw<R, VEC>(q.dres + i, narrow<R, VEC>(dv));
#pragma unroll
            for (int e = 0; e < VEC; ++e) dv[e] *= p.scale;
        }
        if (q.z) {
            float dz[VEC], f[VEC];
            widen<T, VEC>(z, zf);
            if (p.gate_first) widen<T, VEC>(x, f);
            else widen<T, VEC>(dy, f);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                sg[e] = sigmoid(zf[e]);
                const float slope = sg[e] * fmaf(zf[e], 1.f - sg[e], 1.f);
                dz[e] = (p.gate_first ? dv[e] : v[e] * r * w[e]) * f[e] * slope;
                if (p.gate_first) dv[e] *= zf[e] * sg[e];
            }
            store_raw<T, VEC>(q.dz + i, narrow<T, VEC>(dz));
        }
        store_raw<T, VEC>(q.dx + i, narrow<T, VEC>(dv));
    }
};

// Block (slab, group): teams walk rows slab * teams + team, + slabs * teams, ...
template <typename T, typename R, int VEC, int NV, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? kMaxBlock : kWarps * 32) norm_bwd_kernel(const NormParams p,
                                                                                   const NormBwdParams g) {
    extern __shared__ float dwsum[];   // warp teams: the group's share of dw
    __shared__ float smem[64];
    const int ts = BLOCK ? (int)blockDim.x : p.team;
    const int teams = blockDim.x / ts, team = threadIdx.x / ts;
    const int lane = threadIdx.x - team * ts;
    const int64_t slab = blockIdx.x / p.groups, c0 = (blockIdx.x % p.groups) * p.gs;
    const int nvec = static_cast<int>(p.gs / VEC);
    float dw[NV][VEC] = {};
    // every team of a block makes the same number of rounds (the last ones on row 0, without effect)
    for (int64_t r0 = slab * teams; r0 < p.rows; r0 += g.slabs * teams) {
        const int64_t row = r0 + team;
        const bool on = row < p.rows;
        const BwdRow<T, R, VEC> q(p, g, on ? row : 0, c0);
        BwdVec<T, R, VEC> in[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = lane + i * ts;
            in[i] = {};
            if (on && j < nvec) in[i].load(q, j * VEC);
        }
        float v[NV][VEC], d[NV][VEC], s[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = lane + i * ts;
            in[i].values(p, v[i], d[i]);
            float w[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) w[e] = 1.f;
            if (p.w && j < nvec) load_f32<VEC>(p.w + c0 + j * VEC, w);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                s[0] = fmaf(v[i][e], v[i][e], s[0]);
                s[1] = fmaf(d[i][e] * w[e], v[i][e], s[1]);
            }
        }
        team_sum<BLOCK, 2>(s, ts, smem);
        const float r = rsqrtf(s[0] * p.inv_gs + p.eps);
        const float m = s[1] * p.inv_gs * r * r * r;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = lane + i * ts;
            if (on && j < nvec) {
                float w[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) w[e] = 1.f;
                if (p.w) load_f32<VEC>(p.w + c0 + j * VEC, w);
                in[i].store(p, q, j * VEC, r, m, v[i], d[i], w);
#pragma unroll
                for (int e = 0; e < VEC; ++e) dw[i][e] = fmaf(d[i][e], v[i][e] * r, dw[i][e]);
            }
        }
    }
    if (!g.partial) return;
    float *out = g.partial + slab * p.dim + c0;
    if constexpr (BLOCK) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = lane + i * ts;
            if (j < nvec)
#pragma unroll
                for (int e = 0; e < VEC; ++e) out[j * VEC + e] = dw[i][e];
        }
    } else {
        // teams of a warp by shuffles, then the warps one behind the other
        for (int o = ts; o < 32; o <<= 1)
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < VEC; ++e) dw[i][e] += __shfl_xor_sync(0xffffffffu, dw[i][e], o);
        const int warp = threadIdx.x >> 5, wl = threadIdx.x & 31;
        for (int k = 0; k < (int)(blockDim.x >> 5); ++k) {
            if (warp == k && wl < ts)
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int j = lane + i * ts;
                    if (j < nvec)
#pragma unroll
                        for (int e = 0; e < VEC; ++e)
                            dwsum[j * VEC + e] = k == 0 ? dw[i][e] : dwsum[j * VEC + e] + dw[i][e];
                }
            __syncthreads();
        }
        for (int64_t j = threadIdx.x; j < p.gs; j += blockDim.x) out[j] = dwsum[j];
    }
}

// Groups too long for the registers of a block: two passes over each row, the
// slab's share of dw kept in memory.
template <typename T, typename R, int VEC>
__global__ void __launch_bounds__(kMaxBlock) norm_bwd_long_kernel(const NormParams p, const NormBwdParams g) {
    __shared__ float smem[64];
    const int64_t slab = blockIdx.x / p.groups, c0 = (blockIdx.x % p.groups) * p.gs;
    const int64_t nvec = p.gs / VEC;
    float *out = g.partial ? g.partial + slab * p.dim + c0 : nullptr;
    auto weight = [&](int64_t j, float(&w)[VEC]) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) w[e] = 1.f;
        if (p.w) load_f32<VEC>(p.w + c0 + j * VEC, w);
    };
    bool first = true;
    for (int64_t row = slab; row < p.rows; row += g.slabs, first = false) {
        const BwdRow<T, R, VEC> q(p, g, row, c0);
        float s[2] = {0.f, 0.f};
        for (int64_t j = threadIdx.x; j < nvec; j += blockDim.x) {
            BwdVec<T, R, VEC> in{};
            float v[VEC], d[VEC], w[VEC];
            in.load(q, j * VEC);
            in.values(p, v, d);
            weight(j, w);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                s[0] = fmaf(v[e], v[e], s[0]);
                s[1] = fmaf(d[e] * w[e], v[e], s[1]);
            }
        }
        team_sum<true, 2>(s, 0, smem);
        const float r = rsqrtf(s[0] * p.inv_gs + p.eps);
        const float m = s[1] * p.inv_gs * r * r * r;
        for (int64_t j = threadIdx.x; j < nvec; j += blockDim.x) {
            BwdVec<T, R, VEC> in{};
            float v[VEC], d[VEC], w[VEC];
            in.load(q, j * VEC);
            in.values(p, v, d);
            weight(j, w);
            in.store(p, q, j * VEC, r, m, v, d, w);
            if (out)
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    out[j * VEC + e] = fmaf(d[e], v[e] * r, first ? 0.f : out[j * VEC + e]);
        }
    }
}

// dw[c] = sum over slabs of partial[slab][c], in slab order within 16 strided
// sums that are then added in order.
__global__ void __launch_bounds__(512) norm_dw_kernel(const float *partial, float *dw, int64_t slabs, int64_t dim) {
    __shared__ float acc[16][33];
    const int cx = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + cx;
    float s = 0.f;
    if (c < dim)
        for (int64_t i = k; i < slabs; i += 16) s += partial[i * dim + c];
    acc[k][cx] = s;
    __syncthreads();
    if (k == 0 && c < dim) {
#pragma unroll
        for (int i = 1; i < 16; ++i) s += acc[i][cx];
        dw[c] = s;
    }
}

// How a (row, group) is shared out: team of `ts` threads with nv vectors each;
// nv 0: two passes by a block.
struct Teams {
    bool block;
    int ts, nv;
};

Teams teams_of(int64_t nvec) {
    if (nvec <= 32 * 4) {
        int ts = 1;
        while (ts < 32 && ts < nvec) ts *= 2;
        const int64_t n = (nvec + ts - 1) / ts;
        return {false, ts, n <= 1 ? 1 : n <= 2 ? 2 : 4};
    }
    // a block: one vector per thread up to 256 threads, then two, then up to four
    const int nv = nvec <= 256 ? 1 : nvec <= 2 * kMaxBlock ? 2 : 4;
    if (nvec > nv * kMaxBlock) return {true, kMaxBlock, 0};
    const int64_t t = (nvec + nv - 1) / nv;
    return {true, static_cast<int>((t + 31) / 32 * 32), nv};
}

template <typename T, typename R, int VEC>
cudaError_t fwd_vec(const NormParams &p0, cudaStream_t stream) {
    NormParams p = p0;
    const Teams t = teams_of(p.gs / VEC);
    const int64_t items = p.rows * p.groups;
    p.team = t.ts;
    if (!t.block) {
        const int per = kWarps * 32 / t.ts;
        const unsigned grid = static_cast<unsigned>((items + per - 1) / per);
        if (t.nv == 1) norm_fwd_kernel<T, R, VEC, 1, false><<<grid, kWarps * 32, 0, stream>>>(p);
        else if (t.nv == 2) norm_fwd_kernel<T, R, VEC, 2, false><<<grid, kWarps * 32, 0, stream>>>(p);
        else norm_fwd_kernel<T, R, VEC, 4, false><<<grid, kWarps * 32, 0, stream>>>(p);
    } else {
        const unsigned grid = static_cast<unsigned>(items);
        if (t.nv == 0) norm_fwd_long_kernel<T, R, VEC><<<grid, t.ts, 0, stream>>>(p);
        else if (t.nv == 1) norm_fwd_kernel<T, R, VEC, 1, true><<<grid, t.ts, 0, stream>>>(p);
        else if (t.nv == 2) norm_fwd_kernel<T, R, VEC, 2, true><<<grid, t.ts, 0, stream>>>(p);
        else norm_fwd_kernel<T, R, VEC, 4, true><<<grid, t.ts, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

template <typename T, typename R, int VEC>
cudaError_t bwd_vec(const NormParams &p0, const NormBwdParams &g, cudaStream_t stream) {
    NormParams p = p0;
    const Teams t = teams_of(p.gs / VEC);
    p.team = t.ts;
    const unsigned grid = static_cast<unsigned>(g.slabs * p.groups);
    const size_t sm = static_cast<size_t>(p.gs) * sizeof(float);
    if (!t.block) {
        if (t.nv == 1) norm_bwd_kernel<T, R, VEC, 1, false><<<grid, kWarps * 32, sm, stream>>>(p, g);
        else if (t.nv == 2) norm_bwd_kernel<T, R, VEC, 2, false><<<grid, kWarps * 32, sm, stream>>>(p, g);
        else norm_bwd_kernel<T, R, VEC, 4, false><<<grid, kWarps * 32, sm, stream>>>(p, g);
    } else if (t.nv == 0) {
        norm_bwd_long_kernel<T, R, VEC><<<grid, t.ts, 0, stream>>>(p, g);
    } else if (t.nv == 1) {
        norm_bwd_kernel<T, R, VEC, 1, true><<<grid, t.ts, 0, stream>>>(p, g);
    } else if (t.nv == 2) {
        norm_bwd_kernel<T, R, VEC, 2, true><<<grid, t.ts, 0, stream>>>(p, g);
    } else {
        norm_bwd_kernel<T, R, VEC, 4, true><<<grid, t.ts, 0, stream>>>(p, g);
    }
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !g.dw || g.partial == g.dw) return e;
    norm_dw_kernel<<<static_cast<unsigned>((p.dim + 31) / 32), 512, 0, stream>>>(g.partial, g.dw, g.slabs, p.dim);
    return cudaGetLastError();
}

// Widest vectors (16 bytes of the input type, 8 of a float32 row, or single
// elements) that every tensor of the call allows.
int vector_width(const NormParams &p, const NormBwdParams *g, int eb, int rb) {
    for (int vec : {16 / eb, 2, 1}) {
        bool ok = p.gs % vec == 0 && vec_ok(p.x, p.x_sr, eb, vec) && vec_ok(p.z, p.z_sr, eb, vec) &&
                  vec_ok(p.res, p.res_sr, rb, vec) && vec_ok(p.ro, p.ro_sr, rb, vec) && vec_ok(p.w, 0, 4, vec);
        if (!g) ok = ok && vec_ok(p.y, p.y_sr, eb, vec);
        else
            ok = ok && vec_ok(g->dy, g->dy_sr, eb, vec) && vec_ok(g->dro, g->dro_sr, rb, vec) &&
                 vec_ok(g->dx, g->dx_sr, eb, vec) && vec_ok(g->dz, g->dz_sr, eb, vec) &&
                 vec_ok(g->dres, g->dres_sr, rb, vec);
        if (ok) return vec;
    }
    return 1;
}

}  // namespace

int64_t norm_bwd_slabs(int64_t rows, int64_t dim, int64_t gs, int num_sms) {
    // about 16 warps per SM over all groups, at least 4 rows per slab
    const int64_t groups = dim / gs;
    const int64_t blocks = static_cast<int64_t>(num_sms) * (gs <= 1024 ? 8 : 3);
    const int64_t want = (blocks + groups - 1) / groups;
    const int64_t most = (rows + 3) / 4;
    return max64(1, min64(want, most));
}

cudaError_t launch_norm_fwd(const NormParams &p, int in_dtype, int res_dtype, cudaStream_t stream) {
    const int eb = in_dtype == 0 ? 4 : 2, rb = res_dtype == 0 ? 4 : 2;
    const int vec = vector_width(p, nullptr, eb, rb);
    if (in_dtype == 0) {
        if (vec == 4) return fwd_vec<float, float, 4>(p, stream);
        if (vec == 2) return fwd_vec<float, float, 2>(p, stream);
        return fwd_vec<float, float, 1>(p, stream);
    }
    using B = __nv_bfloat16;
    if (res_dtype == 0) {
        if (vec == 8) return fwd_vec<B, float, 8>(p, stream);
        if (vec == 2) return fwd_vec<B, float, 2>(p, stream);
        return fwd_vec<B, float, 1>(p, stream);
    }
    if (vec == 8) return fwd_vec<B, B, 8>(p, stream);
    if (vec == 2) return fwd_vec<B, B, 2>(p, stream);
    return fwd_vec<B, B, 1>(p, stream);
}

cudaError_t launch_norm_bwd(const NormParams &p, const NormBwdParams &g, int in_dtype, int res_dtype,
                            cudaStream_t stream) {
    const int eb = in_dtype == 0 ? 4 : 2, rb = res_dtype == 0 ? 4 : 2;
    const int vec = vector_width(p, &g, eb, rb);
    if (in_dtype == 0) {
        if (vec == 4) return bwd_vec<float, float, 4>(p, g, stream);
        if (vec == 2) return bwd_vec<float, float, 2>(p, g, stream);
        return bwd_vec<float, float, 1>(p, g, stream);
    }
    using B = __nv_bfloat16;
    if (res_dtype == 0) {
        if (vec == 8) return bwd_vec<B, float, 8>(p, g, stream);
        if (vec == 2) return bwd_vec<B, float, 2>(p, g, stream);
        return bwd_vec<B, float, 1>(p, g, stream);
    }
    if (vec == 8) return bwd_vec<B, B, 8>(p, g, stream);
    if (vec == 2) return bwd_vec<B, B, 2>(p, g, stream);
    return bwd_vec<B, B, 1>(p, g, stream);
}

}  // namespace ms
