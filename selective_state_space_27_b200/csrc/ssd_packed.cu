// Mamba-2 scalar-decay SSM (SSD) over packed sequences on the sm_100a tensor
// cores: headdim P = 64, dstate N = 128, bf16 inputs, float32 states in cache
// slots. The recurrence and the pages it follows are those of ssd_fwd.cu.
//
// Mathematics. A sequence is walked in chunks of Q = 128 tokens. With s_r the
// running sum of delta A inside the chunk (log2 units, s_end its last value):
//   G     = C B^T                                     (Q x Q)
//   M'_ri = [i <= r] 2^(s_r - s_i) delta_i G_ri
//   Y     = M' X + 2^(s_r) (C H^T) + D X              H: state before the chunk
//   H     = 2^(s_end) H + B^T (w X),  w_i = 2^(s_end - s_i) delta_i
// Rounding: M' and the copy of H that C multiplies are rounded to bf16 once
// each (Y itself is bf16). The state is float32 and stays exact to float32
// rounding of its inputs: w X is split into two bf16 terms (hi + lo, 2^-17
// relative), the products accumulate on the state in float32, and w comes from
// sums that end at the chunk's last token, so that large running sums do not
// cancel. A token's decay is taken as at least 2^-160, which is 0 in float32
// either way; it keeps the running sums small.
//
// Layout. One CTA walks one segment (see below) of one (sequence, head) with
// two CTAs per SM, so that one's loads and tensor work overlap the other's
// arithmetic: 98 KB of shared memory (X, B, C, the state's bf16 copy; the
// split w X takes C's place, which is done with by then) and 256 columns of
// tensor memory (G, overwritten in place by M' as the A operand of M' X; Y;
// the state). The decayed state and the decayed inter-chunk term with the skip
// are written into the accumulators, so the products add onto them.
// Roles (320 threads): warps 0-7 arithmetic (warp w: rows 32 (w % 4) .. + 31
// of the tile, column half w / 4), warp 8 TMA loads and step sizes, warp 9
// tensor memory and MMA issue.
//
// Long sequences with few heads are cut into segments that run side by side
// (ssd_packed_segment): a first kernel computes what every segment but a
// sequence's last adds to the state from zero (the state product alone), a
// second one forms each segment's initial state from those of the segments
// before it and does the rest. Two launches on one stream: no CTA waits for
// another.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "device_math.cuh"
#include "launch.h"
#include "mambascan.h"
#include "packed.cuh"
#include "tensor_map.h"
#include "umma.cuh"
#include "vec.cuh"

namespace ms {
namespace {

using namespace umma;

constexpr int kQ = 128, kP = 64, kN = 128;
constexpr int kWarpsC = 8;                        // arithmetic warps
constexpr int kThreads = kWarpsC * 32 + 64;
constexpr int kTmaWarp = kWarpsC, kMmaWarp = kWarpsC + 1;
constexpr float kMinStep = -160.f;                // smallest log2 decay of one token

// Shared memory from a 1024-byte aligned base; tiles of 128-byte-swizzled atoms.
constexpr uint32_t kAtom = kQ * 128;              // 128 rows of 128 bytes
constexpr uint32_t kOffX = 0;                     // X: 128 tokens x 64
constexpr uint32_t kOffB = kAtom;                 // B: 128 tokens x 128, two atoms
constexpr uint32_t kOffC = kOffB + 2 * kAtom;     // C, then the hi and lo terms of w X
constexpr uint32_t kOffH = kOffC + 2 * kAtom;     // H (128 rows n x 64 bf16 along p)
constexpr uint32_t kOffStep = kOffH + kAtom;      // two buffers of StepData
struct StepData {
    float s[kQ];      // running sum of delta A (log2)
    float cf[kQ];     // 2^(s at the end of the token's 32-token block - s_i) delta_i
    float dl[kQ];     // delta_i
    float w[kQ];      // 2^(s_end - s_i) delta_i
};
constexpr uint32_t kOffBar = kOffStep + 2 * sizeof(StepData);
// Barriers; chunk k completes phase k of each, step[k % 2] its phase k / 2:
//   full    X, B, C of chunk k landed                        <- TMA bytes
//   gfull   G(k) and C H^T(k) done: C is free                <- tcgen05.commit
//   pready  M', Y start, w X of chunk k written              <- arithmetic warps
//   sfull   the state after chunk k                          <- tcgen05.commit
//   yfull   Y(k) done: X, B and w X are free, loads of k + 1 go out  <- tcgen05.commit
//   hready  state tile and accumulator for chunk k written, Y(k - 1) read  <- arithmetic warps
//   step    step data of chunk k written                     <- 32 producer lanes
// No waiter falls two phases behind: the next phase of full, gfull, sfull and
// yfull needs pready(k + 1), which every arithmetic warp gives after its waits
// for chunk k; the producer's next load follows its wait for yfull(k); step
// data of chunk k + 2 follows yfull(k).
enum Bar { kFull, kGFull, kPReady, kSFull, kYFull, kHReady, kStep0, kStep1, kDrain, kNumBars };
constexpr uint32_t kOffMisc = kOffBar + kNumBars * 8;   // tensor memory address, abort flag, segment
constexpr uint32_t kSmemBytes = kOffMisc + 32;
static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two CTAs per SM");

constexpr uint32_t kTmemCols = 256;
constexpr uint32_t kColG = 0, kColY = 128, kColS = 192;

// What a CTA works on: chunks of 128 tokens from row `row`, `len` tokens, of
// sequence `seq`; segment `seg` of `nseg`, whose first place is `base`.
struct Segment {
    int seq, row, len, seg, nseg;
    int64_t base;
};

// Place -> (sequence, segment). Without segments a sequence has one place. With
// segments of Qs tokens, sequence s starts at place cu[s] / Qs + s: since
// ceil(len / Qs) <= floor((cu + len) / Qs) - floor(cu / Qs) + 1 its segments end
// before the next one's first place; places in between have nothing to do.
// Searched by one warp, 32 sequences at a time.
__device__ __forceinline__ bool find_segment(const SsdPackedParams &p, int64_t place, int lane, Segment &g)
{
    const int T = (int)p.tokens;
    if (p.seg_chunks == 0) {
        const SeqRange q = seq_range(p.cu, place, p.tokens);
        g = {(int)place, q.begin, q.end - q.begin, 0, 1, place};
        return true;
    }
    const int Qs = p.seg_chunks * kQ;
    int lo = 0, n = (int)p.nseq;
    while (n > 1) {
        const int step = (n + 31) / 32, c = lane * step;
        bool le = false;
        if (c < n) le = (int64_t)(min(max(__ldg(p.cu + lo + c), 0), T) / Qs) + lo + c <= place;
        const int k = max(__popc(__ballot_sync(0xffffffffu, le)) - 1, 0);
        lo += k * step;
        n = min(step, n - k * step);
    }
    const SeqRange q = seq_range(p.cu, lo, p.tokens);
    const int64_t base = (int64_t)(q.begin / Qs) + lo;
    const int len = q.end - q.begin;
    const int64_t seg = place - base;
    const int nseg = len > 0 ? (len + Qs - 1) / Qs : 1;
    if (seg < 0 || seg >= nseg) return false;
    g = {lo, q.begin + (int)seg * Qs, min(len - (int)seg * Qs, Qs), (int)seg, nseg, base};
    return true;
}

__device__ __forceinline__ float delta_of(const SsdPackedParams &p, float dt, float bias)
{
    const float v = dt + bias;
    return p.softplus ? softplus_precise(v) : v;
}

__device__ __forceinline__ float log2_decay(float delta, float A2) { return fmaxf(delta * A2, kMinStep); }

// Inclusive prefix and exclusive suffix sums over 128 tokens, four per lane.
__device__ __forceinline__ void token_sums(const float (&a)[4], int lane, float (&pre)[4], float (&suf)[4], float &all)
{
    pre[0] = a[0];
#pragma unroll
    for (int k = 1; k < 4; ++k) pre[k] = pre[k - 1] + a[k];
    suf[3] = 0.f;
#pragma unroll
    for (int k = 2; k >= 0; --k) suf[k] = suf[k + 1] + a[k + 1];
    float up = pre[3], dn = pre[3];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float u = __shfl_up_sync(0xffffffffu, up, o), d = __shfl_down_sync(0xffffffffu, dn, o);
        if (lane >= o) up += u;
        if (lane + o < 32) dn += d;
    }
    all = __shfl_sync(0xffffffffu, up, 31);
    float before = __shfl_up_sync(0xffffffffu, up, 1), after = __shfl_down_sync(0xffffffffu, dn, 1);
    if (lane == 0) before = 0.f;
    if (lane == 31) after = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        pre[k] += before;
        suf[k] += after;
    }
}

// Split w x into bf16 hi + lo for one row's 32 columns (half hq of row r) and
// store both into the operand tiles at `tile` (lo one atom further).
__device__ __forceinline__ void store_split(uint32_t tile, int r, int q, const uint4 &x, float w)
{
    const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float a = bf16_lo(xw[e]) * w, b = bf16_hi(xw[e]) * w;
        hi[e] = pack_bf16(a, b);
        lo[e] = pack_bf16(a - bf16_lo(hi[e]), b - bf16_hi(hi[e]));
    }
    const uint32_t at = tile + sw128((uint32_t)r, (uint32_t)q);
    st_shared_v4(at, hi[0], hi[1], hi[2], hi[3]);
    st_shared_v4(at + kAtom, lo[0], lo[1], lo[2], lo[3]);
}

// The tensor core's descriptors of the state product B^T (w X), hi then lo.
__device__ __forceinline__ void issue_state_product(uint32_t tmem, uint32_t base)
{
    constexpr uint32_t id_s = bf16_idesc(128, 64, true, true);
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int k = 0; k < 8; ++k)
            mma_bf16(tmem + kColS, sw128_desc(base + kOffB + (uint32_t)k * 2048u, kAtom, 1024),
                     sw128_desc(base + kOffC + (uint32_t)t * kAtom + (uint32_t)k * 2048u, kAtom, 1024), id_s, 1);
}

// State values of this thread: n = 32 sub + lane, p = 32 hq .. + 31; global
// layout (p, n), so a warp's lanes are consecutive.
__device__ __forceinline__ void load_state(const float *src, int r, int hq, float (&v)[32])
{
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = src ? __ldcg(src + (32 * hq + j) * kN + r) : 0.f;
}

__device__ __forceinline__ void store_state(float *dst, int r, int hq, const float (&v)[32])
{
#pragma unroll
    for (int j = 0; j < 32; ++j) __stcg(dst + (32 * hq + j) * kN + r, v[j]);
}

__device__ __forceinline__ void tmem_load32(uint32_t taddr, float (&v)[32])
{
    float a[16], b[16];
    tmem_load16(taddr, a);
    tmem_load16(taddr + 16, b);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        v[j] = a[j];
        v[16 + j] = b[j];
    }
}

__device__ __forceinline__ void tmem_store32_scaled(uint32_t taddr, const float (&v)[32], float f)
{
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        float a[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) a[j] = v[16 * q + j] * f;
        tmem_store16(taddr + 16u * q, a);
    }
}

__device__ __forceinline__ void state_tile(uint32_t tile, int r, int hq, const float (&v)[32])
{
#pragma unroll
    for (int q = 0; q < 4; ++q)
        st_shared_v4(tile + sw128((uint32_t)r, (uint32_t)(4 * hq + q)), pack_bf16(v[8 * q], v[8 * q + 1]),
                     pack_bf16(v[8 * q + 2], v[8 * q + 3]), pack_bf16(v[8 * q + 4], v[8 * q + 5]),
                     pack_bf16(v[8 * q + 6], v[8 * q + 7]));
}

// Where a sequence's state of head h lies: its segments' zero-start states by
// place, the copy of its initial state in its last segment's place.
__device__ __forceinline__ float *seg_state(const SsdPackedParams &p, int64_t place, int h)
{
    return p.seg_states + (place * p.nheads + h) * (int64_t)(kP * kN);
}

// Set up by all threads: barriers, tensor memory, the segment; false when the
// CTA has nothing to do (then nothing is allocated).
__device__ __forceinline__ bool setup(const SsdPackedParams &p, uint8_t *smem, uint32_t base, int64_t place,
                                      Segment &g, int &slot, uint32_t &tmem, bool last_too)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (base & 1023u) {
        if (threadIdx.x == 0) atomicExch(p.status, (int)MS_ERR_ALIGNMENT);
        return false;
    }
    bool have = find_segment(p, place, lane, g);
    have = have && (last_too || g.seg + 1 < g.nseg);
    if (!have) return false;   // (the same for every thread)
    slot = p.state || p.idx ? block_slot(p.idx, g.seq, p.slots) : 0;
    if (slot < 0) return false;
    auto bar = [&](int i) { return base + kOffBar + 8u * (uint32_t)i; };
    if (threadIdx.x == 0) {
        mbar_init(bar(kFull), 1);
        mbar_init(bar(kGFull), 1);
        mbar_init(bar(kPReady), kWarpsC);
        mbar_init(bar(kSFull), 1);
        mbar_init(bar(kYFull), 1);
        mbar_init(bar(kHReady), kWarpsC);
        mbar_init(bar(kStep0), 32);
        mbar_init(bar(kStep1), 32);
        mbar_init(bar(kDrain), 1);
        *reinterpret_cast<volatile int *>(smem + kOffMisc + 8) = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) tmem_alloc(base + kOffMisc, kTmemCols);
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    tmem = *reinterpret_cast<volatile uint32_t *>(smem + kOffMisc);
    return true;
}

__device__ __forceinline__ void teardown(uint32_t tmem)
{
    tc_before_sync();
    __syncthreads();
    if ((threadIdx.x >> 5) == kMmaWarp) {
        tc_after_sync();
        tmem_free(tmem, kTmemCols);
    }
}

// ---- first kernel: what a segment adds to the state ---------------------------
// Every segment but a sequence's last (so all its chunks are full): the state
// at its end, from the sequence's initial state for the first segment and from
// zero for the others, and its decay. The weights count to the segment's end,
// so the chunks' products add up without rescaling.
__global__ void __launch_bounds__(kThreads, 2)
ssd_packed_states_kernel(const __grid_constant__ CUtensorMap x_map, const __grid_constant__ CUtensorMap b_map,
                         const SsdPackedParams p)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = smem_addr(smem);
    const int64_t place = blockIdx.x / p.nheads;
    const int h = (int)(blockIdx.x - place * p.nheads);
    Segment g;
    int slot;
    uint32_t tmem;
    if (!setup(p, smem, base, place, g, slot, tmem, false)) return;
    auto bar = [&](int i) { return base + kOffBar + 8u * (uint32_t)i; };
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + kOffMisc + 8);
    const uint64_t wlim = p.wait_limit_ns;
    StepData *step = reinterpret_cast<StepData *>(smem + kOffStep);
    const int K = (g.len + kQ - 1) / kQ;
    const int hg = h / (int)(p.nheads / p.ngroups);
    const float A2 = p.A[h] * kLog2e, bias = p.dt_bias ? p.dt_bias[h] : 0.f;

    if (warp == kTmaWarp) {
        const uint16_t *dtp = reinterpret_cast<const uint16_t *>(p.dt) + (int64_t)g.row * p.dt_st + h;
        auto deltas = [&](int k, float (&d)[4], float (&a)[4]) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = k * kQ + 4 * lane + j;
                d[j] = t < g.len ? delta_of(p, load_bf16(dtp, (int64_t)t * p.dt_st), bias) : 0.f;
                a[j] = t < g.len ? log2_decay(d[j], A2) : 0.f;
            }
        };
        // decay of the whole segment, then of what follows each chunk
        float total = 0.f;
        for (int k = K - 1; k >= 0; --k) {
            float d[4], a[4];
            deltas(k, d, a);
            total += (a[0] + a[1]) + (a[2] + a[3]);
        }
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        if (lane == 0) p.seg_decay[place * p.nheads + h] = total;
        // chunks run from the segment's end to its start, so that the decay of
        // what follows a chunk is a sum that ends at the segment's end
        float after = 0.f;
        int issued = 0;
        for (int i = 0; i < K; ++i) {
            const int k = K - 1 - i;
            if (i > 0 && !__all_sync(0xffffffffu, role_wait(bar(kYFull), (i - 1) & 1, abort_flag, wlim))) {
                if (lane == 0) give_up(p.status, abort_flag);
                break;
            }
            if (lane == 0) {
                const int row = g.row + k * kQ;
                mbar_arrive_tx(bar(kFull), 3 * kAtom);
                tma_load_2d(base + kOffX, &x_map, bar(kFull), h * kP, row);
                tma_load_2d(base + kOffB, &b_map, bar(kFull), hg * kN, row);
                tma_load_2d(base + kOffB + kAtom, &b_map, bar(kFull), hg * kN + 64, row);
                if (k > 0) tma_prefetch_2d(&x_map, h * kP, row - kQ);
            }
            issued = i + 1;
            float d[4], a[4], pre[4], suf[4], all;
            deltas(k, d, a);
            token_sums(a, lane, pre, suf, all);
            float w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = ex2(suf[j] + after) * d[j];
            after += all;
            *reinterpret_cast<float4 *>(step[i & 1].w + 4 * lane) = make_float4(w[0], w[1], w[2], w[3]);
            if (lane == 0) step[i & 1].s[0] = total;
            mbar_arrive(bar(kStep0 + (i & 1)));
        }
        if (lane == 0 && issued) mbar_wait(bar(kFull), (issued - 1) & 1);   // loads in flight must land
        __syncwarp();
    } else if (warp == kMmaWarp) {
        if (lane == 0) {
            for (int i = 0; i < K; ++i) {
                if (!role_wait(bar(kPReady), i & 1, abort_flag, wlim)) {
                    give_up(p.status, abort_flag);
                    break;
                }
                tc_after_sync();
                issue_state_product(tmem, base);
                mma_commit(bar(kYFull));
            }
            mma_commit(bar(kDrain));
            mbar_wait(bar(kDrain), 0);
        }
        __syncwarp();
    } else {
        const int sub = warp & 3, hq = warp >> 2, r = sub * 32 + lane;
        const uint32_t tl = tmem + ((uint32_t)(sub * 32) << 16);
        bool ok = true;
        auto wait = [&](uint32_t b, uint32_t parity) {
            if (ok) ok = __all_sync(0xffffffffu, role_wait(b, parity, abort_flag, wlim));
            if (!ok && lane == 0) give_up(p.status, abort_flag);
        };
        float v[32];
        const bool resumed = g.seg == 0 && p.state && p.has_init && p.has_init[g.seq];
        load_state(resumed ? p.state + slot * p.s_slot + (int64_t)h * (kP * kN) : nullptr, r, hq, v);
        // the second kernel's first segment reads the initial state from here: its
        // last segment replaces the one in the cache
        if (resumed) store_state(seg_state(p, g.base + g.nseg - 1, h), r, hq, v);
        for (int i = 0; i < K; ++i) {
            wait(bar(kStep0 + (i & 1)), (i >> 1) & 1);
            if (i == 0 && ok) {
                tmem_store32_scaled(tl + kColS + 32u * hq, v, ex2(step[0].s[0]));
                tmem_store_wait();
            }
            wait(bar(kFull), i & 1);
            if (i > 0) wait(bar(kYFull), (i - 1) & 1);
            if (ok) {
                const float w = step[i & 1].w[r];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    store_split(base + kOffC, r, 4 * hq + q,
                                ld_shared_v4(base + kOffX + sw128((uint32_t)r, (uint32_t)(4 * hq + q))), w);
            }
            async_proxy_fence();
            tc_before_sync();
            __syncwarp();
            if (lane == 0 && ok) mbar_arrive(bar(kPReady));
        }
        wait(bar(kYFull), (K - 1) & 1);
        if (ok) {
            tc_after_sync();
            tmem_load32(tl + kColS + 32u * hq, v);
            store_state(seg_state(p, place, h), r, hq, v);
        }
    }
    teardown(tmem);
}

// ---- second kernel: outputs and final states ------------------------------------

// M' of row r in its 32-row block SUB: columns 32 j + 16 hq .. + 15, j = 0 .. 3,
// in place of G as packed pairs (8 columns from where the 16 started). Below
// the diagonal block the decay is split at the end of the column's block, both
// factors at most 1 for a decaying state; above it M' is zero.
template <int SUB>
__device__ __forceinline__ void build_mask(uint32_t tg, const StepData &st, int r, int hq)
{
    const float sr = st.s[r];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int i0 = 32 * j + 16 * hq;
        uint32_t m[8];
        if (j <= SUB) {
            float gv[16];
            tmem_load16(tg + (uint32_t)i0, gv);
            if (j < SUB) {
                const float rf = ex2(sr - st.s[32 * j + 31]);
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float4 c = *reinterpret_cast<const float4 *>(st.cf + i0 + 2 * e);
                    m[e] = pack_bf16(gv[2 * e] * (rf * c.x), gv[2 * e + 1] * (rf * c.y));
                    m[e + 1] = pack_bf16(gv[2 * e + 2] * (rf * c.z), gv[2 * e + 3] * (rf * c.w));
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float4 s = *reinterpret_cast<const float4 *>(st.s + i0 + 2 * e);
                    const float4 d = *reinterpret_cast<const float4 *>(st.dl + i0 + 2 * e);
                    const int i = i0 + 2 * e;
                    m[e] = pack_bf16(i <= r ? gv[2 * e] * (ex2(sr - s.x) * d.x) : 0.f,
                                     i + 1 <= r ? gv[2 * e + 1] * (ex2(sr - s.y) * d.y) : 0.f);
                    m[e + 1] = pack_bf16(i + 2 <= r ? gv[2 * e + 2] * (ex2(sr - s.z) * d.z) : 0.f,
                                         i + 3 <= r ? gv[2 * e + 3] * (ex2(sr - s.w) * d.w) : 0.f);
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) m[e] = 0u;
        }
        tmem_store8(tg + (uint32_t)i0, m);
    }
}

__global__ void __launch_bounds__(kThreads, 2)
ssd_packed_kernel(const __grid_constant__ CUtensorMap x_map, const __grid_constant__ CUtensorMap b_map,
                  const __grid_constant__ CUtensorMap c_map, const SsdPackedParams p)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = smem_addr(smem);
    const int64_t place = blockIdx.x / p.nheads;
    const int h = (int)(blockIdx.x - place * p.nheads);
    Segment g;
    int slot;
    uint32_t tmem;
    if (!setup(p, smem, base, place, g, slot, tmem, true)) return;
    auto bar = [&](int i) { return base + kOffBar + 8u * (uint32_t)i; };
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + kOffMisc + 8);
    const uint64_t wlim = p.wait_limit_ns;
    StepData *step = reinterpret_cast<StepData *>(smem + kOffStep);
    const int K = (g.len + kQ - 1) / kQ;
    const int hg = h / (int)(p.nheads / p.ngroups);

    if (warp == kTmaWarp) {
        // ---- loads of chunk k, then the step data of chunk k + 1 ----
        const float A2 = p.A[h] * kLog2e, bias = p.dt_bias ? p.dt_bias[h] : 0.f;
        const uint16_t *dtp = reinterpret_cast<const uint16_t *>(p.dt) + (int64_t)g.row * p.dt_st + h;
        auto write_step = [&](int k) {
            float d[4], a[4], pre[4], suf[4], all;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = k * kQ + 4 * lane + j;
                d[j] = t < g.len ? delta_of(p, load_bf16(dtp, (int64_t)t * p.dt_st), bias) : 0.f;
                a[j] = t < g.len ? log2_decay(d[j], A2) : 0.f;
            }
            token_sums(a, lane, pre, suf, all);
            // running sum at the end of the 32-token block (lanes 8 b .. 8 b + 7 hold block b)
            const float send = __shfl_sync(0xffffffffu, pre[3], lane | 7);
            float cf[4], w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                cf[j] = ex2(send - pre[j]) * d[j];
                w[j] = ex2(suf[j]) * d[j];
            }
            StepData &st = step[k & 1];
            *reinterpret_cast<float4 *>(st.s + 4 * lane) = make_float4(pre[0], pre[1], pre[2], pre[3]);
            *reinterpret_cast<float4 *>(st.cf + 4 * lane) = make_float4(cf[0], cf[1], cf[2], cf[3]);
            *reinterpret_cast<float4 *>(st.dl + 4 * lane) = make_float4(d[0], d[1], d[2], d[3]);
            *reinterpret_cast<float4 *>(st.w + 4 * lane) = make_float4(w[0], w[1], w[2], w[3]);
            mbar_arrive(bar(kStep0 + (k & 1)));
        };
        int issued = 0;
        for (int k = 0; k < K; ++k) {
            if (k > 0 && !__all_sync(0xffffffffu, role_wait(bar(kYFull), (k - 1) & 1, abort_flag, wlim))) {
                if (lane == 0) give_up(p.status, abort_flag);
                break;
            }
            if (lane == 0) {
                const int row = g.row + k * kQ;
                mbar_arrive_tx(bar(kFull), 5 * kAtom);
                tma_load_2d(base + kOffC, &c_map, bar(kFull), hg * kN, row);
                tma_load_2d(base + kOffC + kAtom, &c_map, bar(kFull), hg * kN + 64, row);
                tma_load_2d(base + kOffB, &b_map, bar(kFull), hg * kN, row);
                tma_load_2d(base + kOffB + kAtom, &b_map, bar(kFull), hg * kN + 64, row);
                tma_load_2d(base + kOffX, &x_map, bar(kFull), h * kP, row);
                if (k + 1 < K) tma_prefetch_2d(&x_map, h * kP, row + kQ);
            }
            issued = k + 1;
            if (k == 0) write_step(0);
            if (k + 1 < K) write_step(k + 1);
        }
        if (lane == 0 && issued) mbar_wait(bar(kFull), (issued - 1) & 1);   // loads in flight must land
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ---- MMA issue (one thread) ----
        if (lane == 0) {
            constexpr uint32_t id_g = bf16_idesc(128, 128, false, false);   // G = C B^T
            constexpr uint32_t id_y = bf16_idesc(128, 64, false, true);     // C H^T and M' X
            for (int k = 0; k < K; ++k) {
                if (!role_wait(bar(kFull), k & 1, abort_flag, wlim)) {
                    give_up(p.status, abort_flag);
                    break;
                }
                tc_after_sync();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t off = (uint32_t)(i >> 2) * kAtom + (uint32_t)(i & 3) * 32u;
                    mma_bf16(tmem + kColG, sw128_desc(base + kOffC + off, 16, 1024),
                             sw128_desc(base + kOffB + off, 16, 1024), id_g, i > 0);
                }
                if (!role_wait(bar(kHReady), k & 1, abort_flag, wlim)) {
                    give_up(p.status, abort_flag);
                    break;
                }
                tc_after_sync();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t off = (uint32_t)(i >> 2) * kAtom + (uint32_t)(i & 3) * 32u;
                    mma_bf16(tmem + kColY, sw128_desc(base + kOffC + off, 16, 1024),
                             sw128_desc(base + kOffH + (uint32_t)i * 2048u, kAtom, 1024), id_y, i > 0);
                }
                mma_commit(bar(kGFull));
                if (!role_wait(bar(kPReady), k & 1, abort_flag, wlim)) {
                    give_up(p.status, abort_flag);
                    break;
                }
                tc_after_sync();
                issue_state_product(tmem, base);
                mma_commit(bar(kSFull));
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    mma_bf16_ta(tmem + kColY, tmem + kColG + 16u * (uint32_t)i,
                                sw128_desc(base + kOffX + (uint32_t)i * 2048u, kAtom, 1024), id_y, 1);
                mma_commit(bar(kYFull));
            }
            mma_commit(bar(kDrain));   // every MMA must finish before the tensor memory is freed
            mbar_wait(bar(kDrain), 0);
        }
        __syncwarp();
    } else {
        const int sub = warp & 3, hq = warp >> 2, r = sub * 32 + lane;
        const uint32_t tl = tmem + ((uint32_t)(sub * 32) << 16);
        bool ok = true;
        auto wait = [&](uint32_t b, uint32_t parity) {
            if (ok) ok = __all_sync(0xffffffffu, role_wait(b, parity, abort_flag, wlim));
            if (!ok && lane == 0) give_up(p.status, abort_flag);
        };
        float *cache = p.state ? p.state + slot * p.s_slot + (int64_t)h * (kP * kN) : nullptr;
        const bool resumed = cache && p.has_init && p.has_init[g.seq];
        // the state before the segment
        float v0[32];
        if (g.nseg == 1) {
            load_state(resumed ? cache : nullptr, r, hq, v0);
        } else if (g.seg == 0) {
            load_state(resumed ? seg_state(p, g.base + g.nseg - 1, h) : nullptr, r, hq, v0);
        } else {
            load_state(seg_state(p, g.base, h), r, hq, v0);
            for (int i = 1; i < g.seg; ++i) {
                const float f = ex2(__ldg(p.seg_decay + (g.base + i) * p.nheads + h));
                const float *src = seg_state(p, g.base + i, h);
#pragma unroll
                for (int j = 0; j < 32; ++j) v0[j] = fmaf(f, v0[j], __ldcg(src + (32 * hq + j) * kN + r));
            }
        }
        // what chunk k starts from: the state's bf16 tile, and its decayed value in the accumulator
        auto advance = [&](int k, const float (&v)[32]) {
            wait(bar(kStep0 + (k & 1)), (k >> 1) & 1);
            if (ok) {
                state_tile(base + kOffH, r, hq, v);
                tmem_store32_scaled(tl + kColS + 32u * hq, v, ex2(step[k & 1].s[kQ - 1]));
                tmem_store_wait();
            }
        };
        auto give = [&](int b) {
            async_proxy_fence();
            tc_before_sync();
            __syncwarp();
            if (lane == 0 && ok) mbar_arrive(bar(b));
        };
        const bool last = cache && g.seg + 1 == g.nseg;
        if (K > 0) {
            advance(0, v0);
            give(kHReady);
        } else if (last && !resumed) {   // an empty sequence leaves the state it starts from
            store_state(cache, r, hq, v0);
        }
        const float Dh = p.D ? p.D[h] : 0.f;
        const int64_t col = (int64_t)h * kP + 32 * hq;
        for (int k = 0; k < K; ++k) {
            const int left = g.len - k * kQ;   // live rows of this chunk
            const bool live = r < left;
            const StepData &st = step[k & 1];
            wait(bar(kFull), k & 1);
            wait(bar(kGFull), k & 1);
            if (ok) {
                tc_after_sync();
                const uint32_t tg = tl + kColG;
                switch (sub) {
                case 0: build_mask<0>(tg, st, r, hq); break;
                case 1: build_mask<1>(tg, st, r, hq); break;
                case 2: build_mask<2>(tg, st, r, hq); break;
                default: build_mask<3>(tg, st, r, hq); break;
                }
                const float er = ex2(st.s[r]), w = st.w[r];
#pragma unroll
                for (int q2 = 0; q2 < 2; ++q2) {
                    float y[16];
                    tmem_load16(tl + kColY + 32u * hq + 16u * q2, y);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const uint32_t at = sw128((uint32_t)r, (uint32_t)(4 * hq + 2 * q2 + q));
                        uint4 x = ld_shared_v4(base + kOffX + at);
                        if (!live) {
                            // rows behind the sequence hold other data (any bits): zero where products sum over them
                            x = make_uint4(0u, 0u, 0u, 0u);
                            st_shared_v4(base + kOffX + at, 0u, 0u, 0u, 0u);
                        }
                        const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int j = 8 * q + 2 * e;
                            y[j] = fmaf(er, y[j], Dh * bf16_lo(xw[e]));
                            y[j + 1] = fmaf(er, y[j + 1], Dh * bf16_hi(xw[e]));
                        }
                        store_split(base + kOffC, r, 4 * hq + 2 * q2 + q, x, w);
                    }
                    tmem_store16(tl + kColY + 32u * hq + 16u * q2, y);
                }
                if (!live) {
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        st_shared_v4(base + kOffB + (uint32_t)hq * kAtom + sw128((uint32_t)r, (uint32_t)q), 0u, 0u, 0u,
                                     0u);
                }
                tmem_store_wait();
            }
            give(kPReady);

            // the gate of this thread's outputs, on its way while the products run
            const int64_t row = (int64_t)g.row + k * kQ + r;
            uint4 zq[4];
            if (p.z && live) {
                const uint4 *zp = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.z) + row * p.z_st +
                                                                  col);
#pragma unroll
                for (int q = 0; q < 4; ++q) zq[q] = __ldg(zp + q);
            }
            wait(bar(kSFull), k & 1);
            {
                float v[32];
                if (ok) {
                    tc_after_sync();
                    tmem_load32(tl + kColS + 32u * hq, v);
                }
                if (k + 1 < K) advance(k + 1, v);
                else if (ok && last) store_state(cache, r, hq, v);   // the state after the sequence
            }
            wait(bar(kYFull), k & 1);
            float y[32];
            if (ok) {
                tc_after_sync();
                tmem_load32(tl + kColY + 32u * hq, y);
            }
            if (k + 1 < K) give(kHReady);
            if (ok && live) {
                uint4 *yp = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.y) + row * p.y_st + col);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t ow[4];
                    const uint32_t zw[4] = {zq[q].x, zq[q].y, zq[q].z, zq[q].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float a = y[8 * q + 2 * e], b = y[8 * q + 2 * e + 1];
                        if (p.z) {
                            const float za = bf16_lo(zw[e]), zb = bf16_hi(zw[e]);
                            a *= za * sigmoid(za);
                            b *= zb * sigmoid(zb);
                        }
                        ow[e] = pack_bf16(a, b);
                    }
                    yp[q] = make_uint4(ow[0], ow[1], ow[2], ow[3]);
                }
            }
        }
    }
    teardown(tmem);
}

// A bf16 map over (inner, rows) delivering 64 x 128 boxes into
// 128-byte-swizzled shared memory; rows past the last read as zero.
bool encode_rows(CUtensorMap *m, const void *ptr, int64_t inner, int64_t rows, int64_t row_stride)
{
    const EncodeTiled fn = encoder();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)row_stride * 2u};
    const cuuint32_t box[2] = {64u, (cuuint32_t)kQ};
    const cuuint32_t elem[2] = {1u, 1u};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(ptr), dims, strides, box, elem,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// Chunks per segment: the choice among powers of two (and no cut) with the
// smallest estimate of the time, in chunk times of one of the 2 x num_sms CTAs
// that run together. Cut into segments of c chunks the work is that of all
// chunks plus 0.6 of a chunk for each chunk in a segment that is not its
// sequence's last, spread over the CTAs, plus the last segment's own length
// and a second launch.
int ssd_packed_segment(int64_t tokens, int64_t nseq, int64_t nheads, int64_t max_seqlen, int num_sms)
{
    const int64_t slots = 2 * (int64_t)(num_sms > 0 ? num_sms : 1);
    const int64_t longest = ((max_seqlen > 0 ? min64(max_seqlen, tokens) : tokens) + kQ - 1) / kQ;
    const int64_t chunks = tokens / kQ + nseq;
    const double all = (double)chunks * (double)nheads / (double)slots;
    double best = all > (double)longest ? all + 0.5 * (double)longest : (double)longest;
    int pick = 0;
    for (int c = 4; c <= 64 && c < longest; c *= 2) {
        const double cut = all * 1.6 + 1.5 * c + 4.0;
        if (cut < best) {
            best = cut;
            pick = c;
        }
    }
    return pick;
}

int64_t ssd_packed_places(int64_t tokens, int64_t nseq, int seg_chunks)
{
    return seg_chunks ? tokens / (seg_chunks * kQ) + nseq : nseq;
}

namespace {
size_t decay_offset() { return 256; }
size_t states_offset(int64_t places, int64_t nheads)
{
    return 256 + (((size_t)places * (size_t)nheads * sizeof(float) + 255) / 256) * 256;
}
}  // namespace

size_t ssd_packed_ws_bytes(int64_t tokens, int64_t nseq, int64_t nheads, int seg_chunks)
{
    if (!seg_chunks) return 256;
    const int64_t places = ssd_packed_places(tokens, nseq, seg_chunks);
    return states_offset(places, nheads) + (size_t)places * (size_t)nheads * kP * kN * sizeof(float);
}

void ssd_packed_bind(SsdPackedParams &p, void *ws)
{
    p.status = static_cast<int *>(ws);
    if (!p.seg_chunks) return;
    const int64_t places = ssd_packed_places(p.tokens, p.nseq, p.seg_chunks);
    p.seg_decay = reinterpret_cast<float *>(static_cast<char *>(ws) + decay_offset());
    p.seg_states = reinterpret_cast<float *>(static_cast<char *>(ws) + states_offset(places, p.nheads));
}

cudaError_t launch_ssd_packed(const SsdPackedParams &p, cudaStream_t stream)
{
    CUtensorMap xm, bm, cm;
    // (without tokens nothing is loaded; the maps then only need a valid address)
    const int64_t rows = max64(p.tokens, 1);
    const void *none = p.status;
    const int64_t xi = p.nheads * kP, bi = p.ngroups * kN;
    if (!encode_rows(&xm, p.tokens ? p.x : none, xi, rows, p.tokens ? p.x_st : xi) ||
        !encode_rows(&bm, p.tokens ? p.B : none, bi, rows, p.tokens ? p.B_st : bi) ||
        !encode_rows(&cm, p.tokens ? p.C : none, bi, rows, p.tokens ? p.C_st : bi))
        return cudaErrorNotSupported;
    cudaError_t e =
        cudaFuncSetAttribute(ssd_packed_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(ssd_packed_states_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)kSmemBytes);
    if (e == cudaSuccess) e = cudaMemsetAsync(p.status, 0, sizeof(int), stream);
    if (e != cudaSuccess) return e;
    const unsigned grid = static_cast<unsigned>(ssd_packed_places(p.tokens, p.nseq, p.seg_chunks) * p.nheads);
    if (p.seg_chunks) {
        ssd_packed_states_kernel<<<grid, kThreads, kSmemBytes, stream>>>(xm, bm, p);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    ssd_packed_kernel<<<grid, kThreads, kSmemBytes, stream>>>(xm, bm, cm, p);
    return cudaGetLastError();
}

}  // namespace ms
