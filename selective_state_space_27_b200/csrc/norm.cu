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
// Measured on B200 for 16384 rows x 8 groups of 512, bf16, gated: forward 73 us
// (84% of the measured copy bandwidth), backward 125 us (82%; 130 to 135 over
// seconds, where the clock falls under the power limit). 116 registers leave
// the backward 16 warps per SM: with a row's loads in registers they came in bursts
// between the reductions (137 us), so the next rows wait in shared memory, and the
// row in work is read from there twice (once, held over the reduction: 130 us).
// 4099 rows x 1530, float32, with a residual: backward 31 us (62%, 5 us of it the
// second kernel's). 16384 x 2048, bf16, float32 residual: 66 us (93%), backward 130
// us (63%). bf16 groups that are no multiple of 8 take vectors of two or one element
// without the usual modes: 16384 x 8 groups of 500, gated, 119 and 267 us; 16384 x
// 5001, two passes by single elements, 316 us and 1.01 ms. The same for the forward (teams walk rows, the next ones in
// shared memory) gave 72 to 76 us against 73. Taking the gate's two reciprocals of a pair from one of their
// product, to relieve the special function unit (56% busy in the forward), made
// all of them slower: 86 and 158 us.
#include <type_traits>

#include "dependent.cuh"
#include "launch.h"
#include "vec.cuh"

namespace ms {
namespace {

constexpr int kWarps = 4;                // warps per block of the warp-team kernels
constexpr int kMaxBlock = 512;           // threads of a block team
constexpr int kBwdThreads = 512;         // threads of the backward that run together on an SM

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

// What the call combines, known at compile time for the usual calls (their
// kernels then have no branches per vector); kAny looks at the arguments.
enum Mode { kPlain, kGateFirst, kGateLast, kResidual, kAny };

template <int MODE>
struct Has {
    static __device__ __forceinline__ bool z(const NormParams &p) {
        return MODE == kAny ? p.z != nullptr : MODE == kGateFirst || MODE == kGateLast;
    }
    static __device__ __forceinline__ bool first(const NormParams &p) {
        return MODE == kAny ? p.gate_first != 0 : MODE == kGateFirst;
    }
    // residual_out is given exactly when there is a residual
    static __device__ __forceinline__ bool res(const NormParams &p) {
        return MODE == kAny ? p.ro != nullptr : MODE == kResidual;
    }
};

inline Mode mode_of(const NormParams &p) {
    if (p.ro) return p.z ? kAny : kResidual;
    return !p.z ? kPlain : p.gate_first ? kGateFirst : kGateLast;
}

// f[e] silu(z[e]) in place.
template <int VEC>
__device__ __forceinline__ void silu_times(float (&f)[VEC], const float (&z)[VEC]) {
    if constexpr (VEC == 1) {
        f[0] *= z[0] * sigmoid(z[0]);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {
            const float2 zz = f2(z[e], z[e + 1]);
            const float2 t = mul2(f2(f[e], f[e + 1]), mul2(zz, sigmoid2(zz)));
            f[e] = t.x;
            f[e + 1] = t.y;
        }
    }
}

template <int VEC>
__device__ __forceinline__ void sigmoids(const float (&z)[VEC], float (&g)[VEC]) {
    if constexpr (VEC == 1) {
        g[0] = sigmoid(z[0]);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {
            const float2 t = sigmoid2(f2(z[e], z[e + 1]));
            g[e] = t.x;
            g[e + 1] = t.y;
        }
    }
}

// The value that is normed, of VEC channels at element i of the row; `sum` is
// what residual_out stores.
template <typename T, typename R, int VEC, int MODE>
struct FwdRow {
    using H = Has<MODE>;
    const T *x, *z;
    const R *res;
    R *ro;
    T *y;
    const float *w;
    __device__ __forceinline__ FwdRow(const NormParams &p, int64_t row, int64_t c0)
        : x(static_cast<const T *>(p.x) + row * p.x_sr + c0),
          z(H::z(p) ? static_cast<const T *>(p.z) + row * p.z_sr + c0 : nullptr),
          res(H::res(p) ? static_cast<const R *>(p.res) + row * p.res_sr + c0 : nullptr),
          ro(H::res(p) ? static_cast<R *>(p.ro) + row * p.ro_sr + c0 : nullptr),
          y(static_cast<T *>(p.y) + row * p.y_sr + c0), w(p.w ? p.w + c0 : nullptr) {}
};

template <typename T, typename R, int VEC, int MODE>
__device__ __forceinline__ void norm_value(const NormParams &p, const Raw<T, VEC> &xr, const Raw<T, VEC> &zr,
                                           const Raw<R, VEC> &rr, float (&v)[VEC]) {
    widen<T, VEC>(xr, v);
    if (Has<MODE>::z(p) && Has<MODE>::first(p)) {
        float z[VEC];
        widen<T, VEC>(zr, z);
        silu_times<VEC>(v, z);
    }
    if (Has<MODE>::res(p)) {
        float r[VEC];
        widen<R, VEC>(rr, r);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = fmaf(p.scale, v[e], r[e]);
    }
}

template <typename T, typename R, int VEC, int MODE>
__device__ __forceinline__ void norm_store(const NormParams &p, const FwdRow<T, R, VEC, MODE> &row, int64_t i, float r,
                                           const float (&v)[VEC], const Raw<T, VEC> &zr) {
    float w[VEC], o[VEC];
    if (row.w) load_f32<VEC>(row.w + i, w);
#pragma unroll
    for (int e = 0; e < VEC; ++e) o[e] = row.w ? v[e] * r * w[e] : v[e] * r;
    if (Has<MODE>::z(p) && !Has<MODE>::first(p)) {
        float z[VEC];
        widen<T, VEC>(zr, z);
        silu_times<VEC>(o, z);
    }
    store_raw<T, VEC>(row.y + i, narrow<T, VEC>(o));
}

// One (row, group) per team; NV vectors per thread in registers.
template <typename T, typename R, int VEC, int NV, bool BLOCK, int MODE>
__global__ void __launch_bounds__(BLOCK ? kMaxBlock : kWarps * 32) norm_fwd_kernel(const NormParams p) {
    __shared__ float smem[32];
    const int ts = BLOCK ? (int)blockDim.x : p.team;
    const int lane = BLOCK ? (int)threadIdx.x : (int)(threadIdx.x & (ts - 1));
    const int64_t item = BLOCK ? blockIdx.x
                               : static_cast<int64_t>(blockIdx.x) * (blockDim.x / ts) + threadIdx.x / ts;
    const bool on = item < p.rows * p.groups;   // (false only in the last block of warp teams)
    const int64_t row = on ? item / p.groups : 0, c0 = on ? (item % p.groups) * p.gs : 0;
    const FwdRow<T, R, VEC, MODE> q(p, row, c0);
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
            if (Has<MODE>::z(p)) zr[i] = load_raw<T, VEC>(q.z + j * VEC);
            if (Has<MODE>::res(p)) rr[i] = load_raw<R, VEC>(q.res + j * VEC);
        }
    }
    float v[NV][VEC], ss[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        norm_value<T, R, VEC, MODE>(p, xr[i], zr[i], rr[i], v[i]);
        const int j = lane + i * ts;
        if (j < nvec) {
            if (Has<MODE>::res(p)) store_raw<R, VEC>(q.ro + j * VEC, narrow<R, VEC>(v[i]));
#pragma unroll
            for (int e = 0; e < VEC; ++e) ss[0] = fmaf(v[i][e], v[i][e], ss[0]);
        }
    }
    team_sum<BLOCK, 1>(ss, ts, smem);
    const float r = rsqrtf(ss[0] * p.inv_gs + p.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = lane + i * ts;
        if (j < nvec) norm_store<T, R, VEC, MODE>(p, q, j * VEC, r, v[i], zr[i]);
    }
}

// Groups too long for the registers of a block: two passes over the row.
template <typename T, typename R, int VEC>
__global__ void __launch_bounds__(kMaxBlock) norm_fwd_long_kernel(const NormParams p) {
    __shared__ float smem[32];
    const int64_t row = blockIdx.x / p.groups, c0 = (blockIdx.x % p.groups) * p.gs;
    const FwdRow<T, R, VEC, kAny> q(p, row, c0);
    const int64_t nvec = p.gs / VEC;
    float ss[1] = {0.f};
    auto value = [&](int64_t j, Raw<T, VEC> &zr, float(&v)[VEC]) {
        Raw<R, VEC> rr{};
        zr = {};
        if (q.z) zr = load_raw<T, VEC>(q.z + j * VEC);
        if (q.res) rr = load_raw<R, VEC>(q.res + j * VEC);
        norm_value<T, R, VEC, kAny>(p, load_raw<T, VEC>(q.x + j * VEC), zr, rr, v);
    };
    for (int64_t j = threadIdx.x; j < nvec; j += blockDim.x) {
        Raw<T, VEC> zr;
        float v[VEC];
        value(j, zr, v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) ss[0] = fmaf(v[e], v[e], ss[0]);
    }
    team_sum<true, 1>(ss, 0, smem);
    const float r = rsqrtf(ss[0] * p.inv_gs + p.eps);
    for (int64_t j = threadIdx.x; j < nvec; j += blockDim.x) {
        Raw<T, VEC> zr;
        float v[VEC];
        value(j, zr, v);
        if (q.ro) store_raw<R, VEC>(q.ro + j * VEC, narrow<R, VEC>(v));
        norm_store<T, R, VEC, kAny>(p, q, j * VEC, r, v, zr);
    }
}

// ---- backward ----------------------------------------------------------------

template <typename T, typename R, int VEC, int MODE>
struct BwdRow {
    using H = Has<MODE>;
    const T *dy, *x, *z;
    const R *sum, *ds;
    T *dx, *dz;
    R *dres;
    __device__ __forceinline__ BwdRow(const NormParams &p, const NormBwdParams &g, int64_t row, int64_t c0)
        : dy(static_cast<const T *>(g.dy) + row * g.dy_sr + c0),
          x(!H::res(p) || (H::z(p) && H::first(p)) ? static_cast<const T *>(p.x) + row * p.x_sr + c0 : nullptr),
          z(H::z(p) ? static_cast<const T *>(p.z) + row * p.z_sr + c0 : nullptr),
          sum(H::res(p) ? static_cast<const R *>(p.ro) + row * p.ro_sr + c0 : nullptr),
          ds(H::res(p) && g.dro ? static_cast<const R *>(g.dro) + row * g.dro_sr + c0 : nullptr),
          dx(static_cast<T *>(g.dx) + row * g.dx_sr + c0),
          dz(H::z(p) ? static_cast<T *>(g.dz) + row * g.dz_sr + c0 : nullptr),
          dres(H::res(p) ? static_cast<R *>(g.dres) + row * g.dres_sr + c0 : nullptr) {}
};

// What one thread knows of VEC channels of a row before the reductions.
template <typename T, typename R, int VEC, int MODE>
struct BwdVec {
    using H = Has<MODE>;
    Raw<T, VEC> dy, x, z;
    Raw<R, VEC> sum, ds;
    __device__ __forceinline__ void load(const NormParams &p, const BwdRow<T, R, VEC, MODE> &q, int64_t i) {
        dy = load_raw<T, VEC>(q.dy + i);
        if (!H::res(p) || (H::z(p) && H::first(p))) x = load_raw<T, VEC>(q.x + i);
        if (H::z(p)) z = load_raw<T, VEC>(q.z + i);
        if (H::res(p)) sum = load_raw<R, VEC>(q.sum + i);
        if (H::res(p) && q.ds) ds = load_raw<R, VEC>(q.ds + i);
    }
    // The same by way of shared memory, where the loads of the next rows wait without
    // holding registers: a thread's pieces lie blockDim.x apart, it alone writes
    // and reads them.
    static constexpr int kT = VEC * (int)sizeof(T), kR = VEC * (int)sizeof(R);
    static constexpr int kBytes = MODE == kResidual ? kT + 2 * kR : MODE == kPlain ? 2 * kT : 3 * kT;
    static __device__ __forceinline__ void stage(uint32_t at, const BwdRow<T, R, VEC, MODE> &q, int64_t i) {
        put<kT>(at, 0, q.dy + i);
        if constexpr (MODE == kResidual) {
            put<kR>(at, kT, q.sum + i);
            if (q.ds) put<kR>(at, kT + kR, q.ds + i);
        } else {
            put<kT>(at, kT, q.x + i);
            if constexpr (MODE != kPlain) put<kT>(at, 2 * kT, q.z + i);
        }
    }
    __device__ __forceinline__ void fetch(uint32_t at, const BwdRow<T, R, VEC, MODE> &q) {
        get<kT>(at, 0, &dy);
        if constexpr (MODE == kResidual) {
            get<kR>(at, kT, &sum);
            if (q.ds) get<kR>(at, kT + kR, &ds);
        } else {
            get<kT>(at, kT, &x);
            if constexpr (MODE != kPlain) get<kT>(at, 2 * kT, &z);
        }
    }
    template <int N> static __device__ __forceinline__ void put(uint32_t at, int off, const void *src) {
        constexpr int P = N < 16 ? N : 16;
#pragma unroll
        for (int o = 0; o < N; o += P)
            cp_async_full<P>(at + (uint32_t)(off + o) * blockDim.x + threadIdx.x * P, static_cast<const char *>(src) + o);
    }
    template <int N> static __device__ __forceinline__ void get(uint32_t at, int off, void *dst) {
        uint32_t *d = static_cast<uint32_t *>(dst);
        if constexpr (N == 8) {
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(d[0]), "=r"(d[1])
                         : "r"(at + (uint32_t)off * blockDim.x + threadIdx.x * 8u) : "memory");
        } else {
#pragma unroll
            for (int o = 0; o < N; o += 16)
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(d[o / 4]), "=r"(d[o / 4 + 1]), "=r"(d[o / 4 + 2]), "=r"(d[o / 4 + 3])
                             : "r"(at + (uint32_t)(off + o) * blockDim.x + threadIdx.x * 16u) : "memory");
        }
    }
    // v, and dy as it reaches the norm's output (before the weight)
    __device__ __forceinline__ void values(const NormParams &p, float (&v)[VEC], float (&d)[VEC]) const {
        widen<T, VEC>(dy, d);
        if (H::res(p)) widen<R, VEC>(sum, v);
        else widen<T, VEC>(x, v);
        if (H::z(p) && (!H::res(p) || !H::first(p))) {
            float zf[VEC];
            widen<T, VEC>(z, zf);
            if (H::first(p)) silu_times<VEC>(v, zf);
            else silu_times<VEC>(d, zf);
        }
    }
    // the gradients, from r and m = mean(u v) r^3 (u = d w)
    __device__ __forceinline__ void store(const NormParams &p, const BwdRow<T, R, VEC, MODE> &q, int64_t i, float r, float m,
                                          const float (&v)[VEC], const float (&d)[VEC], const float (&w)[VEC]) const {
        float dv[VEC], zf[VEC], sg[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) dv[e] = fmaf(r, d[e] * w[e], -m * v[e]);
        if (H::res(p)) {
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
        if (H::z(p)) {
            float dz[VEC], f[VEC];
            widen<T, VEC>(z, zf);
            if (H::first(p)) widen<T, VEC>(x, f);
            else widen<T, VEC>(dy, f);
            sigmoids<VEC>(zf, sg);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float slope = sg[e] * fmaf(zf[e], 1.f - sg[e], 1.f);
                dz[e] = (H::first(p) ? dv[e] : v[e] * r * w[e]) * f[e] * slope;
                if (H::first(p)) dv[e] *= zf[e] * sg[e];
            }
            store_raw<T, VEC>(q.dz + i, narrow<T, VEC>(dz));
        }
        store_raw<T, VEC>(q.dx + i, narrow<T, VEC>(dv));
    }
};

// Rows in shared memory per thread: the one in work and those on their way (0: the
// rows are loaded into registers, for vectors below 8 bytes and for the threads
// with the most bytes, whose rows would not fit twice). Gated bf16 groups of 512
// have 96 bytes: 127 us with three rows, 129 with two, 127 with four; 192 bytes
// (float32 with a residual): 34 us with two rows, 49 with three.
template <typename T, typename R, int VEC, int NV, int MODE>
constexpr int stages_of() {
    constexpr int bytes = NV * BwdVec<T, R, VEC, MODE>::kBytes;
    return MODE == kAny || bytes > 192 ? 0 : bytes > 96 ? 2 : 3;
}

// Block (slab, group): teams walk rows slab * teams + team, + slabs * teams, ...
template <typename T, typename R, int VEC, int NV, bool BLOCK, int MODE>
__global__ void __launch_bounds__(BLOCK ? kMaxBlock : kWarps * 32, BLOCK ? 1 : kBwdThreads / (kWarps * 32))
    norm_bwd_kernel(const NormParams p, const NormBwdParams g) {
    extern __shared__ __align__(16) float dwsum[];   // warp teams: the group's share of dw
    __shared__ float smem[64];
    const int ts = BLOCK ? (int)blockDim.x : p.team;
    const int teams = blockDim.x / ts, team = threadIdx.x / ts;
    const int lane = threadIdx.x - team * ts;
    const int64_t slab = blockIdx.x / p.groups, c0 = (blockIdx.x % p.groups) * p.gs;
    const int nvec = static_cast<int>(p.gs / VEC);
    float dw[NV][VEC] = {}, w[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) w[i][e] = 1.f;
        if (p.w && lane + i * ts < nvec) load_f32<VEC>(p.w + c0 + (lane + i * ts) * VEC, w[i]);
    }
    constexpr int S = stages_of<T, R, VEC, NV, MODE>();
    using Vec = BwdVec<T, R, VEC, MODE>;
    // (behind the share of dw)
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(dwsum) + (BLOCK ? 0u : (uint32_t)(p.gs + 3) / 4u * 16u);
    auto slot = [&](int st, int i) { return ring + (uint32_t)((st * NV + i) * Vec::kBytes) * blockDim.x; };
    auto stage_row = [&](int64_t r0, int st) {
        if constexpr (S > 0) {
            const int64_t row = r0 + team;
            if (row < p.rows) {
                const BwdRow<T, R, VEC, MODE> q(p, g, row, c0);
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (lane + i * ts < nvec) Vec::stage(slot(st, i), q, (lane + i * ts) * VEC);
            }
            cp_async_commit();
        }
    };
    const int64_t stride = g.slabs * teams;
    int now = 0;   // the row's place in the ring
    if constexpr (S > 0)
#pragma unroll
        for (int k = 0; k + 1 < S; ++k) stage_row(slab * teams + k * stride, k);
    // every team of a block makes the same number of rounds (the last ones on row 0, without effect)
    for (int64_t r0 = slab * teams; r0 < p.rows; r0 += stride) {
        const int64_t row = r0 + team;
        const bool on = row < p.rows;
        const BwdRow<T, R, VEC, MODE> q(p, g, on ? row : 0, c0);
        Vec in[NV];
        if constexpr (S > 0) {
            stage_row(r0 + (S - 1) * stride, now == 0 ? S - 1 : now - 1);
            cp_async_wait<S - 1>();
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = lane + i * ts;
            in[i] = {};
            if (on && j < nvec) {
                if constexpr (S > 0) in[i].fetch(slot(now, i), q);
                else in[i].load(p, q, j * VEC);
            }
        }
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float v[VEC], d[VEC];
            in[i].values(p, v, d);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                s[0] = fmaf(v[e], v[e], s[0]);
                s[1] = fmaf(d[e] * w[i][e], v[e], s[1]);
            }
        }
        team_sum<BLOCK, 2>(s, ts, smem);
        const float r = rsqrtf(s[0] * p.inv_gs + p.eps);
        const float m = s[1] * p.inv_gs * r * r * r;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = lane + i * ts;
            if (on && j < nvec) {
                float v[VEC], d[VEC];
                if constexpr (S > 0) in[i].fetch(slot(now, i), q);   // (once more: not held over the reduction)
                in[i].values(p, v, d);
                in[i].store(p, q, j * VEC, r, m, v, d, w[i]);
#pragma unroll
                for (int e = 0; e < VEC; ++e) dw[i][e] = fmaf(d[e], v[e] * r, dw[i][e]);
            }
        }
        if constexpr (S > 0) now = now + 1 == S ? 0 : now + 1;
    }
    if (!g.partial) return;
    dependents_may_start();
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
        const BwdRow<T, R, VEC, kAny> q(p, g, row, c0);
        float s[2] = {0.f, 0.f};
        for (int64_t j = threadIdx.x; j < nvec; j += blockDim.x) {
            BwdVec<T, R, VEC, kAny> in{};
            float v[VEC], d[VEC], w[VEC];
            in.load(p, q, j * VEC);
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
            BwdVec<T, R, VEC, kAny> in{};
            float v[VEC], d[VEC], w[VEC];
            in.load(p, q, j * VEC);
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

// dw[c] = sum over slabs of partial[slab][c], in a fixed order: 8 columns per
// block (32 bytes of a row), 128 strided sums each, those by shuffles and warps.
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float *partial, float *dw, int64_t slabs, int64_t dim) {
    __shared__ float acc[32][8];
    wait_for_previous();
    const int cx = threadIdx.x & 7, k = threadIdx.x >> 3;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 8 + cx;
    float s = 0.f;
    if (c < dim) {
#pragma unroll 4
        for (int64_t i = k; i < slabs; i += 128) s += __ldcg(partial + i * dim + c);   // (written while this kernel runs)
    }
    s += __shfl_xor_sync(0xffffffffu, s, 8);
    s += __shfl_xor_sync(0xffffffffu, s, 16);
    if ((threadIdx.x & 31) < 8) acc[threadIdx.x >> 5][cx] = s;
    __syncthreads();
    if (threadIdx.x < 8 && c < dim) {
        s = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) s += acc[i][cx];
        dw[c] = s;
    }
}

// How a (row, group) is shared out: team of `ts` threads with nv vectors each;
// nv 0: two passes by a block.
struct Teams {
    bool block;
    int ts, nv;
};

// nvec vectors of vec elements: sixteen elements per thread, up to thirty-two for
// the longest rows. (The backward with 8 per thread, twice the threads on a row:
// 176 us against 135 us for 16384 x 8 groups of 512.)
Teams teams_of(int64_t nvec, int vec) {
    const int full = 16 / vec < 8 ? 16 / vec : 8;   // vectors per thread
    if (nvec <= 32 * full) {
        int ts = 1;
        while (ts < 32 && ts < nvec) ts *= 2;
        int nv = 1;
        while (static_cast<int64_t>(nv) * ts < nvec) nv *= 2;
        return {false, ts, nv};
    }
    for (int nv = full; nv <= 8 && nv * vec <= 32; nv *= 2)
        if (nvec <= static_cast<int64_t>(nv) * kMaxBlock) {
            const int64_t t = (nvec + nv - 1) / nv;
            return {true, static_cast<int>((t + 31) / 32 * 32), nv};
        }
    return {true, kMaxBlock, 0};
}

// f(NV) with the plan's vectors per thread as a compile-time value (those that
// a vector width can have: up to twice 16 elements, at most 8 vectors).
template <int VEC, typename F>
cudaError_t with_nv(int nv, F f) {
    constexpr int kMost = 32 / VEC < 8 ? 32 / VEC : 8;
    if constexpr (kMost >= 8)
        if (nv == 8) return f(std::integral_constant<int, 8>());
    if constexpr (kMost >= 4)
        if (nv == 4) return f(std::integral_constant<int, 4>());
    if (nv == 2) return f(std::integral_constant<int, 2>());
    return f(std::integral_constant<int, 1>());
}

// f(MODE) with the call's mode as a compile-time value: the usual ones for the
// vectors of 8 bytes and more, kAny for everything else.
template <typename T, typename R, int VEC, typename F>
cudaError_t with_mode(const NormParams &p, F f) {
    if constexpr (VEC * sizeof(T) >= 8) {
        const Mode m = mode_of(p);
        if (m == kResidual) return f(std::integral_constant<int, kResidual>());
        if constexpr (std::is_same<T, R>::value) {   // (without a residual R is T)
            if (m == kPlain) return f(std::integral_constant<int, kPlain>());
            if (m == kGateFirst) return f(std::integral_constant<int, kGateFirst>());
            if (m == kGateLast) return f(std::integral_constant<int, kGateLast>());
        }
    }
    return f(std::integral_constant<int, kAny>());
}

template <typename T, typename R, int VEC>
cudaError_t fwd_vec(const NormParams &p0, cudaStream_t stream) {
    NormParams p = p0;
    const Teams t = teams_of(p.gs / VEC, VEC);
    const int64_t items = p.rows * p.groups;
    p.team = t.ts;
    if (t.nv == 0) {
        norm_fwd_long_kernel<T, R, VEC><<<static_cast<unsigned>(items), t.ts, 0, stream>>>(p);
        return cudaGetLastError();
    }
    return with_mode<T, R, VEC>(p, [&](auto mode) {
        return with_nv<VEC>(t.nv, [&](auto nv) {
            constexpr int NV = decltype(nv)::value, MODE = decltype(mode)::value;
            if (t.block) {
                norm_fwd_kernel<T, R, VEC, NV, true, MODE><<<static_cast<unsigned>(items), t.ts, 0, stream>>>(p);
            } else {
                const int per = kWarps * 32 / t.ts;
                norm_fwd_kernel<T, R, VEC, NV, false, MODE>
                    <<<static_cast<unsigned>((items + per - 1) / per), kWarps * 32, 0, stream>>>(p);
            }
            return cudaGetLastError();
        });
    });
}

template <typename T, typename R, int VEC>
cudaError_t bwd_vec(const NormParams &p0, const NormBwdParams &g, cudaStream_t stream) {
    NormParams p = p0;
    const Teams t = teams_of(p.gs / VEC, VEC);
    p.team = t.ts;
    const unsigned grid = static_cast<unsigned>(g.slabs * p.groups);
    cudaError_t e;
    if (t.nv == 0) {
        norm_bwd_long_kernel<T, R, VEC><<<grid, t.ts, 0, stream>>>(p, g);
        e = cudaGetLastError();
    } else {
        e = with_mode<T, R, VEC>(p, [&](auto mode) {
            return with_nv<VEC>(t.nv, [&](auto nv) {
                constexpr int NV = decltype(nv)::value, MODE = decltype(mode)::value;
                constexpr int row = stages_of<T, R, VEC, NV, MODE>() * NV * BwdVec<T, R, VEC, MODE>::kBytes;
                const auto launch = [&](auto kernel, int threads, int64_t share) {
                    const size_t smem = static_cast<size_t>(row) * threads + static_cast<size_t>(share + 3) / 4 * 16;
                    if (smem > 47 * 1024) {   // (the kernel's own 256 bytes count, too)
                        const cudaError_t a = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                                   static_cast<int>(smem));
                        if (a != cudaSuccess) return a;
                    }
                    kernel<<<grid, threads, smem, stream>>>(p, g);
                    return cudaGetLastError();
                };
                if (t.block) return launch(norm_bwd_kernel<T, R, VEC, NV, true, MODE>, t.ts, 0);
                return launch(norm_bwd_kernel<T, R, VEC, NV, false, MODE>, kWarps * 32, p.gs);
            });
        });
    }
    if (e != cudaSuccess || !g.dw || g.partial == g.dw) return e;
    return launch_dependent(norm_dw_kernel, dim3(static_cast<unsigned>((p.dim + 7) / 8)), 1024, 0, stream,
                            static_cast<const float *>(g.partial), g.dw, g.slabs, p.dim);
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
    // As many blocks as run together (512 threads of 128 registers per SM; twice as
    // many blocks, in two rounds: 143 us against 135 us), at least 4 rows per slab.
    const int64_t groups = dim / gs;
    const int64_t threads = gs <= 512 ? kWarps * 32 : min64((gs + 511) / 512 * 32, kMaxBlock);
    const int64_t blocks = num_sms * (kBwdThreads / threads);
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
