// One token per request through the Mamba-2 scalar-decay recurrence, states in
// cache slots ("Mamba-2 e State Space Duality (SSD)", the decode step with one
// decay per head):
//   delta = softplus(dt + dt_bias),  H = exp(delta A) H + (delta x) B^T
//   y = (H C + D x) silu(z)
// per request and head, H of headdim x dstate float32 values.
//
// A step reads and writes every live state once (8 bytes per value) against
// 5 operations: bound by HBM bandwidth. A block owns rows of one (request,
// head); the lanes of a warp (fewer for a small dstate) cover a row of the
// state with 16-byte accesses, all rows of a warp are loaded before any
// arithmetic, and the rows' readouts are summed together in a transposed
// shuffle reduction.
// Measured on B200, bf16, headdim 64, dstate 128: 256 requests x 64 heads
// 174 us (93% of the measured copy bandwidth), 2 requests x 80 heads 6.2 us on
// the device.
#include "launch.h"
#include "packed.cuh"
#include "vec.cuh"

namespace ms {
namespace {

constexpr int kWarps = 8;

// Vector path: dstate a multiple of 4, LPR lanes per row with V float4 pieces
// each (piece q + LPR v of the row), R rows per lane.
template <typename T, int LPR, int V, int R>
__global__ void __launch_bounds__(kWarps * 32) ssd_update_vec_kernel(const SsdUpdateParams p) {
    constexpr int kRowsPerPass = 32 / LPR;           // rows a warp covers at once
    constexpr int kRows = kWarps * kRowsPerPass * R;
    const int64_t b = blockIdx.y;
    const int h = blockIdx.x / p.row_blocks, rb = blockIdx.x - h * p.row_blocks;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int q = lane % LPR;
    const int nq = p.dstate / 4;
    const int row0 = rb * kRows + warp * (kRowsPerPass * R) + lane / LPR;

    // the state is read before its slot is known to be this request's own: the
    // earlier requests' indices are compared while the loads are in flight
    const int v0 = p.idx ? __ldg(p.idx + b) : static_cast<int>(b);
    const bool in = v0 >= 0 && v0 < p.slots;
    float *st = p.state + static_cast<int64_t>(in ? v0 : 0) * p.s_slot + static_cast<int64_t>(h) * p.headdim * p.dstate;
    float4 H[R][V];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int row = row0 + r * kRowsPerPass, j = q + v * LPR;
            H[r][v] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (in && row < p.headdim && j < nq)
                H[r][v] = __ldcs(reinterpret_cast<const float4 *>(st + static_cast<int64_t>(row) * p.dstate) + j);
        }
    if (block_slot(p.idx, b, p.slots) < 0) return;

    const int g = h / p.hpg;
    const T *Bp = static_cast<const T *>(p.B) + b * p.B_sb + static_cast<int64_t>(g) * p.dstate;
    const T *Cp = static_cast<const T *>(p.C) + b * p.C_sb + static_cast<int64_t>(g) * p.dstate;
    float Bv[V][4], Cv[V][4];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int j = q + v * LPR;
#pragma unroll
        for (int e = 0; e < 4; ++e) Bv[v][e] = Cv[v][e] = 0.f;
        if (j < nq) {
            widen<T, 4>(load_raw<T, 4>(Bp + 4 * j), Bv[v]);
            widen<T, 4>(load_raw<T, 4>(Cp + 4 * j), Cv[v]);
        }
    }
    float delta = to_f32<T>(__ldg(static_cast<const T *>(p.dt) + b * p.dt_sb + h));
    if (p.dt_bias) delta += __ldg(p.dt_bias + h);
    if (p.softplus) delta = softplus_fine(delta);
    const float a = ex2_approx(delta * __ldg(p.A + h) * kLog2e);
    const float Dh = p.D ? __ldg(p.D + h) : 0.f;
    const T *xp = static_cast<const T *>(p.x) + b * p.x_sb + static_cast<int64_t>(h) * p.headdim;

    float acc[R], xs[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int row = row0 + r * kRowsPerPass;
        xs[r] = row < p.headdim ? to_f32<T>(__ldg(xp + row)) : 0.f;
        const float dx = delta * xs[r];
        acc[r] = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float4 &f = H[r][v];
            f.x = fmaf(a, f.x, dx * Bv[v][0]);
            f.y = fmaf(a, f.y, dx * Bv[v][1]);
            f.z = fmaf(a, f.z, dx * Bv[v][2]);
            f.w = fmaf(a, f.w, dx * Bv[v][3]);
            acc[r] = fmaf(Cv[v][0], f.x, fmaf(Cv[v][1], f.y, fmaf(Cv[v][2], f.z, fmaf(Cv[v][3], f.w, acc[r]))));
            const int j = q + v * LPR;
            if (row < p.headdim && j < nq)
                __stcs(reinterpret_cast<float4 *>(st + static_cast<int64_t>(row) * p.dstate) + j, f);
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) acc[r] += __shfl_xor_sync(0xffffffffu, acc[r], o);
    // lane q of a row's lanes stores row r = q (q + LPR, ... when there are more rows than lanes)
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int row = row0 + r * kRowsPerPass;
        if (q == r % LPR && row < p.headdim) {
            float y = fmaf(Dh, xs[r], acc[r]);
            const int64_t at = static_cast<int64_t>(h) * p.headdim + row;
            if (p.z) {
                const float z = to_f32<T>(__ldg(static_cast<const T *>(p.z) + b * p.z_sb + at));
                y *= z * sigmoid(z);
            }
            static_cast<T *>(p.y)[b * p.y_sb + at] = from_f32<T>(y);
        }
    }
}

// Any dstate up to 256 and any alignment: a warp per row, single elements.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) ssd_update_kernel(const SsdUpdateParams p) {
    const int64_t b = blockIdx.y;
    const int h = blockIdx.x / p.row_blocks, rb = blockIdx.x - h * p.row_blocks;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slot = block_slot(p.idx, b, p.slots);
    const int row = rb * kWarps + warp;
    if (slot < 0 || row >= p.headdim) return;
    const int g = h / p.hpg;
    const T *Bp = static_cast<const T *>(p.B) + b * p.B_sb + static_cast<int64_t>(g) * p.dstate;
    const T *Cp = static_cast<const T *>(p.C) + b * p.C_sb + static_cast<int64_t>(g) * p.dstate;
    float delta = to_f32<T>(__ldg(static_cast<const T *>(p.dt) + b * p.dt_sb + h));
    if (p.dt_bias) delta += __ldg(p.dt_bias + h);
    if (p.softplus) delta = softplus_fine(delta);
    const float a = ex2_approx(delta * __ldg(p.A + h) * kLog2e);
    const int64_t at = static_cast<int64_t>(h) * p.headdim + row;
    const float x = to_f32<T>(__ldg(static_cast<const T *>(p.x) + b * p.x_sb + at));
    float *st = p.state + slot * p.s_slot + at * p.dstate;
    float acc = 0.f;
    for (int n = lane; n < p.dstate; n += 32) {
        const float f = fmaf(a, st[n], delta * x * to_f32<T>(__ldg(Bp + n)));
        st[n] = f;
        acc = fmaf(to_f32<T>(__ldg(Cp + n)), f, acc);
    }
    for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (lane == 0) {
        float y = fmaf(p.D ? __ldg(p.D + h) : 0.f, x, acc);
        if (p.z) {
            const float z = to_f32<T>(__ldg(static_cast<const T *>(p.z) + b * p.z_sb + at));
            y *= z * sigmoid(z);
        }
        static_cast<T *>(p.y)[b * p.y_sb + at] = from_f32<T>(y);
    }
}

template <typename T, int LPR, int V, int R>
cudaError_t launch_vec(SsdUpdateParams p, cudaStream_t stream) {
    constexpr int kRows = kWarps * (32 / LPR) * R;
    p.row_blocks = (p.headdim + kRows - 1) / kRows;
    const dim3 grid(static_cast<unsigned>(p.nheads * p.row_blocks), static_cast<unsigned>(p.batch));
    ssd_update_vec_kernel<T, LPR, V, R><<<grid, kWarps * 32, 0, stream>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(SsdUpdateParams p, cudaStream_t stream) {
    const int eb = sizeof(T);
    // 16-byte pieces of the state, 4 elements of B and C at a time
    const bool vec = p.dstate % 4 == 0 && vec_ok(p.state, p.s_slot, 4, 4) && vec_ok(p.B, p.B_sb, eb, 4) &&
                     vec_ok(p.C, p.C_sb, eb, 4);
    if (!vec) {
        p.row_blocks = (p.headdim + kWarps - 1) / kWarps;
        const dim3 grid(static_cast<unsigned>(p.nheads * p.row_blocks), static_cast<unsigned>(p.batch));
        ssd_update_kernel<T><<<grid, kWarps * 32, 0, stream>>>(p);
        return cudaGetLastError();
    }
    if (p.dstate <= 16) return launch_vec<T, 4, 1, 2>(p, stream);
    if (p.dstate <= 32) return launch_vec<T, 8, 1, 2>(p, stream);
    if (p.dstate <= 64) return launch_vec<T, 16, 1, 4>(p, stream);
    if (p.dstate <= 128) return launch_vec<T, 32, 1, 8>(p, stream);
    return launch_vec<T, 32, 2, 4>(p, stream);
}

}  // namespace

cudaError_t launch_ssd_update(const SsdUpdateParams &p, int in_dtype, cudaStream_t stream) {
    return in_dtype == 0 ? launch_t<float>(p, stream) : launch_t<__nv_bfloat16>(p, stream);
}

}  // namespace ms
