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
// arithmetic: 100 KB of shared memory (X, B, C, the state's bf16 copy; the
// split w X takes C's place, which is done with by then) and 256 columns of
// tensor memory (G, overwritten in place by M' as the A operand of M' X; Y;
// the state). The decayed state and the decayed inter-chunk term with the skip
// are written into the accumulators, so the products add onto them.
// Roles (320 threads): warps 0-7 arithmetic (warp w: rows 32 (w % 4) .. + 31
// of the tile, column half w / 4, sixteen columns at a time: nothing may spill,
// the L1 that shared memory leaves is far too small for it), warp 8 TMA loads
// and step sizes, warp 9 tensor memory and MMA issue.
// Order within a chunk: G and C H^T; w X and the start of Y; the state product
// runs while the warps build M'; M' X runs while they pass the state on; B and C
// of the next chunk are on their way since the state product ended.
//
// Long sequences with few heads are cut into segments that run side by side
// (ssd_packed_segment): a first kernel computes what every segment but a
// sequence's last adds to the state from zero (the state product alone), a
// second one adds these up along each sequence, a third one does the rest from
// the state that its segment starts from. Three launches on one stream: no CTA
// waits for another.
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
constexpr int kParts = kWarpsC / 4;               // column parts of an arithmetic warp group
constexpr int kCQ = 4 / kParts;                   // column quarters (16 columns) per warp
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
//   full    B and C of chunk k landed                        <- TMA bytes
//   xfull   X of chunk k landed                              <- TMA bytes
//   gfull   G(k) and C H^T(k) done: C is free                <- tcgen05.commit
//   wready  w X and the start of Y of chunk k written        <- arithmetic warps
//   mready  M' of chunk k written                            <- arithmetic warps
//   sfull   the state after chunk k; B and w X are free, B and C of k + 1 go out  <- tcgen05.commit
//   yfull   Y(k) done: X is free, X of k + 1 goes out        <- tcgen05.commit
//   hready  state tile and accumulator for chunk k written, Y(k - 1) read  <- arithmetic warps
//   step    step data of chunk k written                     <- 32 producer lanes
// No waiter falls two phases behind: the next phase of full, xfull, gfull,
// sfull and yfull needs wready(k + 1), which every arithmetic warp gives after
// its waits for chunk k; the producer's loads follow its own waits for sfull(k)
// and yfull(k), and sfull(k + 1) needs those loads; the issuer waits for
// yfull(k) before G(k + 1); step data of chunk k + 2 follows yfull(k).
enum Bar { kFull, kXFull, kGFull, kWReady, kMReady, kSFull, kYFull, kHReady, kStep0, kStep1, kDrain, kNumBars };
constexpr uint32_t kOffMisc = kOffBar + kNumBars * 8;   // tensor memory address, abort flag, segment
constexpr uint32_t kSmemBytes = kOffMisc + 32;
static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two CTAs per SM");

constexpr uint32_t kTmemCols = 256;
constexpr uint32_t kColG = 0, kColY = 128, kColS = 192;

// A bounded wait whose slow path is a call: the loop below waits in many places
// and its code has to stay small for the instruction cache.
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int *abort_flag, uint64_t limit_ns)
{
    return role_wait(bar, parity, abort_flag, limit_ns);
}

__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int *abort_flag, uint64_t limit_ns)
{
    return mbar_test(bar, parity) || wait_slow(bar, parity, abort_flag, limit_ns);
}

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
        // up to 32 sequences: the longest first, so that the last CTAs to start are short
        int s = (int)place;
        if (p.nseq <= 32) {
            int len = -1, rank = 0;
            if (lane < p.nseq) {
                const SeqRange q = seq_range(p.cu, lane, p.tokens);
                len = q.end - q.begin;
            }
            for (int j = 0; j < (int)p.nseq; ++j) {
                const int other = __shfl_sync(0xffffffffu, len, j);
                rank += other > len || (other == len && j < lane);
            }
            s = __ffs(__ballot_sync(0xffffffffu, lane < p.nseq && rank == (int)place)) - 1;
        }
        const SeqRange q = seq_range(p.cu, s, p.tokens);
        g = {s, q.begin, q.end - q.begin, 0, 1, place};
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

// The step inputs of tokens t .. t + 3 of a segment of len tokens (0 behind its end).
__device__ __forceinline__ void load_steps(const uint16_t *dt, int64_t stride, int t, int len, float (&v)[4])
{
    const uint16_t *at = dt + t * stride;
#pragma unroll
    for (int j = 0; j < 4; ++j, at += stride) v[j] = t + j < len ? __uint_as_float((uint32_t)__ldg(at) << 16) : 0.f;
}

__device__ __forceinline__ float delta_of(const SsdPackedParams &p, float dt, float bias)
{
    const float v = dt + bias;
    return p.softplus ? softplus_fine(v) : v;
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

// Split w x (eight values of row r, 16-byte piece q) into bf16 hi + lo and
// store both into the operand tiles at `tile` (lo one atom further).
__device__ __forceinline__ void store_split(uint32_t tile, int r, int q, const float2 (&x)[4], float w)
{
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 a = mul2(x[e], f2(w, w));
        hi[e] = pack_bf16(a.x, a.y);
        const float2 d = add2(a, f2(-bf16_lo(hi[e]), -bf16_hi(hi[e])));
        lo[e] = pack_bf16(d.x, d.y);
    }
    const uint32_t at = tile + sw128((uint32_t)r, (uint32_t)q);
    st_shared_v4(at, hi[0], hi[1], hi[2], hi[3]);
    st_shared_v4(at + kAtom, lo[0], lo[1], lo[2], lo[3]);
}

__device__ __forceinline__ void widen8(const uint4 &x, float2 (&v)[4])
{
    v[0] = f2(bf16_lo(x.x), bf16_hi(x.x));
    v[1] = f2(bf16_lo(x.y), bf16_hi(x.y));
    v[2] = f2(bf16_lo(x.z), bf16_hi(x.z));
    v[3] = f2(bf16_lo(x.w), bf16_hi(x.w));
}

// The state product B^T (w X), hi then lo, onto what the accumulator holds or in its place.
__device__ __forceinline__ void issue_state_product(uint32_t tmem, uint32_t base, bool onto)
{
    constexpr uint32_t id_s = bf16_idesc(128, 64, true, true);
    const uint64_t b = sw128_desc(base + kOffB, kAtom, 1024), x = sw128_desc(base + kOffC, kAtom, 1024);
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int k = 0; k < 8; ++k)
            mma_bf16(tmem + kColS, b + (uint32_t)k * (2048u >> 4), x + (uint32_t)(t * kAtom + k * 2048u) / 16u, id_s,
                     onto || t > 0 || k > 0);
}

// State values of this thread: n = 32 sub + lane, p = 16 cq .. + 15 for the column quarter cq; global
// layout (p, n), so a warp's lanes are consecutive.
__device__ __forceinline__ void load_state(const float *src, int r, int cq, float (&v)[16])
{
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = src ? __ldcg(src + (16 * cq + j) * kN + r) : 0.f;
}

__device__ __forceinline__ void store_state(float *dst, int r, int cq, const float (&v)[16])
{
#pragma unroll
    for (int j = 0; j < 16; ++j) __stcg(dst + (16 * cq + j) * kN + r, v[j]);
}

__device__ __forceinline__ void tmem_store16_scaled(uint32_t taddr, const float (&v)[16], float f)
{
    float a[16];
#pragma unroll
    for (int j = 0; j < 16; j += 2) {
        const float2 t = mul2(f2(v[j], v[j + 1]), f2(f, f));
        a[j] = t.x;
        a[j + 1] = t.y;
    }
    tmem_store16(taddr, a);
}

__device__ __forceinline__ void state_tile(uint32_t tile, int r, int cq, const float (&v)[16])
{
#pragma unroll
    for (int q = 0; q < 2; ++q)
        st_shared_v4(tile + sw128((uint32_t)r, (uint32_t)(2 * cq + q)), pack_bf16(v[8 * q], v[8 * q + 1]),
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
        mbar_init(bar(kXFull), 1);
        mbar_init(bar(kWReady), kWarpsC);
        mbar_init(bar(kMReady), kWarpsC);
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
        float dtv[4];   // the step inputs of the next chunk (all its tokens are the segment's)
        load_steps(dtp, p.dt_st, (K - 1) * kQ + 4 * lane, g.len, dtv);
        // Chunks run from the segment's end to its start: the decay of what follows a
        // chunk is then a sum that ends at the segment's end.
        bool ok = true;
        auto wait = [&](uint32_t b, uint32_t parity) {
            if (ok) ok = __all_sync(0xffffffffu, wait_for(b, parity, abort_flag, wlim));
            if (!ok && lane == 0) give_up(p.status, abort_flag);
            return ok;
        };
        auto load_x = [&](int i) {
            if (lane == 0) {
                mbar_arrive_tx(bar(kXFull), kAtom);
                tma_load_2d(base + kOffX, &x_map, bar(kXFull), h * kP, g.row + (K - 1 - i) * kQ);
            }
        };
        auto load_b = [&](int i) {
            if (lane == 0) {
                const int row = g.row + (K - 1 - i) * kQ;
                mbar_arrive_tx(bar(kFull), 2 * kAtom);
                tma_load_2d(base + kOffB, &b_map, bar(kFull), hg * kN, row);
                tma_load_2d(base + kOffB + kAtom, &b_map, bar(kFull), hg * kN + 64, row);
                if (i + 1 < K) tma_prefetch_2d(&x_map, h * kP, row - kQ);
            }
        };
        float after = 0.f;
        int xs = 1, bs = 1;   // chunks on their way
        load_x(0);
        load_b(0);
        for (int i = 0; i < K; ++i) {
            float d[4], a[4], pre[4], suf[4], all;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                d[j] = delta_of(p, dtv[j], bias);
                a[j] = log2_decay(d[j], A2);
            }
            if (i + 1 < K) load_steps(dtp, p.dt_st, (K - 2 - i) * kQ + 4 * lane, g.len, dtv);
            token_sums(a, lane, pre, suf, all);
            float w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = ex2(suf[j] + after) * d[j];
            after += all;
            // (the buffer's last reader was chunk i - 2, behind yfull(i - 2))
            *reinterpret_cast<float4 *>(step[i & 1].w + 4 * lane) = make_float4(w[0], w[1], w[2], w[3]);
            if (lane == 0) step[i & 1].s[0] = after;
            mbar_arrive(bar(kStep0 + (i & 1)));
            if (i + 1 == K) break;
            if (!wait(bar(kWReady), i & 1)) break;
            load_x(i + 1);
            xs = i + 2;
            if (!wait(bar(kYFull), i & 1)) break;
            load_b(i + 1);
            bs = i + 2;
        }
        if (lane == 0) {
            p.seg_decay[place * p.nheads + h] = after;
            mbar_wait(bar(kFull), (bs - 1) & 1);   // loads in flight must land
            mbar_wait(bar(kXFull), (xs - 1) & 1);
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        if (lane == 0) {
            for (int i = 0; i < K; ++i) {
                if (!wait_for(bar(kWReady), i & 1, abort_flag, wlim)) {
                    give_up(p.status, abort_flag);
                    break;
                }
                if (!wait_for(bar(kFull), i & 1, abort_flag, wlim)) {
                    give_up(p.status, abort_flag);
                    break;
                }
                tc_after_sync();
                issue_state_product(tmem, base, i > 0);
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
            if (ok) ok = __all_sync(0xffffffffu, wait_for(b, parity, abort_flag, wlim));
            if (!ok && lane == 0) give_up(p.status, abort_flag);
        };
        const bool resumed = g.seg == 0 && p.state && p.has_init && p.has_init[g.seq];
        const float *cache = resumed ? p.state + slot * p.s_slot + (int64_t)h * (kP * kN) : nullptr;
        for (int i = 0; i < K; ++i) {
            wait(bar(kStep0 + (i & 1)), (i >> 1) & 1);
            wait(bar(kXFull), i & 1);
            if (i > 0) wait(bar(kYFull), (i - 1) & 1);
            if (ok) {
                const float w = step[i & 1].w[r];
#pragma unroll
                for (int q = 2 * kCQ * hq; q < 2 * kCQ * (hq + 1); ++q) {
                    float2 x[4];
                    widen8(ld_shared_v4(base + kOffX + sw128((uint32_t)r, (uint32_t)q)), x);
                    store_split(base + kOffC, r, q, x, w);
                }
            }
            async_proxy_fence();
            __syncwarp();
            if (lane == 0 && ok) mbar_arrive(bar(kWReady));
        }
        wait(bar(kYFull), (K - 1) & 1);
        if (ok) {
            tc_after_sync();
            const float f = ex2(step[(K - 1) & 1].s[0]);
#pragma unroll 1
            for (int c = kCQ * hq; c < kCQ * (hq + 1); ++c) {
                float v[16];
                tmem_load16(tl + kColS + 16u * c, v);
                if (cache) {
                    float v0[16];
                    load_state(cache, r, c, v0);
                    // the third kernel's first segment reads the initial state from here: its
                    // last segment replaces the one in the cache
                    store_state(seg_state(p, g.base + g.nseg - 1, h), r, c, v0);
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = fmaf(f, v0[j], v[j]);
                }
                store_state(seg_state(p, place, h), r, c, v);
            }
        }
    }
    teardown(tmem);
}

// ---- second kernel: the state at the end of each segment ------------------------
// A thread takes four values of the state of one (sequence, head) through the
// sequence's segments: place m then holds the state after segment m.
__global__ void __launch_bounds__(256) ssd_packed_pass_kernel(const SsdPackedParams p)
{
    constexpr int kBlocks = kP * kN / 4 / 256;   // blocks per (sequence, head)
    const int64_t pair = blockIdx.x / kBlocks;
    const int part = (int)(blockIdx.x - pair * kBlocks);
    const int64_t s = pair / p.nheads;
    const int h = (int)(pair - s * p.nheads);
    const SeqRange q = seq_range(p.cu, s, p.tokens);
    const int Qs = p.seg_chunks * kQ, nseg = (q.end - q.begin + Qs - 1) / Qs;
    if (nseg < 3) return;   // (the state after the first segment is complete as it is)
    if ((p.state || p.idx) && block_slot(p.idx, s, p.slots) < 0) return;
    const int64_t base = q.begin / Qs + s;
    const int64_t step = p.nheads * (int64_t)(kP * kN / 4);
    float4 *at = reinterpret_cast<float4 *>(seg_state(p, base, h)) + part * 256 + threadIdx.x;
    float4 v = __ldcg(at);
    for (int m = 1; m + 1 < nseg; ++m) {
        at += step;
        const float4 a = __ldcg(at);
        const float f = ex2(__ldcg(p.seg_decay + (base + m) * p.nheads + h));
        v.x = fmaf(f, v.x, a.x);
        v.y = fmaf(f, v.y, a.y);
        v.z = fmaf(f, v.z, a.z);
        v.w = fmaf(f, v.w, a.w);
        __stcg(at, v);
    }
}

// ---- third kernel: outputs and final states ------------------------------------

// M' of row r of the 32-row block `sub`, in place of G: the 16 columns from 16 kk
// become 8 columns of packed pairs from where they started. In
// the blocks before the diagonal one the decay is split at the end of the
// column's block, both factors at most 1 for a decaying state; behind it M' is
// zero.
__device__ __forceinline__ void build_mask(uint32_t tg, const StepData &st, int r, int sub, int kk)
{
    const int i0 = 16 * kk, j = kk >> 1;
    uint32_t m[8];
    if (j > sub) {
#pragma unroll
        for (int e = 0; e < 8; ++e) m[e] = 0u;
    } else {
        const float sr = st.s[r];
        float gv[16];
        tmem_load16(tg + (uint32_t)i0, gv);
        if (j < sub) {
            const float rf = ex2(sr - st.s[32 * j + 31]);
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const float4 c = *reinterpret_cast<const float4 *>(st.cf + i0 + 2 * e);
                const float2 a = mul2(f2(gv[2 * e], gv[2 * e + 1]), mul2(f2(rf, rf), f2(c.x, c.y)));
                const float2 b = mul2(f2(gv[2 * e + 2], gv[2 * e + 3]), mul2(f2(rf, rf), f2(c.z, c.w)));
                m[e] = pack_bf16(a.x, a.y);
                m[e + 1] = pack_bf16(b.x, b.y);
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
    }
    tmem_store8(tg + (uint32_t)i0, m);
}

// GATE: y is multiplied by silu(z) (its own kernel: the code of the loop has to
// stay small for the instruction cache).
template <bool GATE>
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
        float dtv[4];   // the step inputs of the chunk whose step data comes next
        auto load_dt = [&](int k) { load_steps(dtp, p.dt_st, k * kQ + 4 * lane, g.len, dtv); };
        auto write_step = [&](int k) {
            float d[4], a[4], pre[4], suf[4], all;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = k * kQ + 4 * lane + j;
                d[j] = t < g.len ? delta_of(p, dtv[j], bias) : 0.f;
                a[j] = t < g.len ? log2_decay(d[j], A2) : 0.f;
            }
            load_dt(k + 1);
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
        bool ok = true;
        auto wait = [&](uint32_t b, uint32_t parity) {
            if (ok) ok = __all_sync(0xffffffffu, wait_for(b, parity, abort_flag, wlim));
            if (!ok && lane == 0) give_up(p.status, abort_flag);
            return ok;
        };
        int bc = 0, xs = 0;   // chunks whose B and C, and whose X, are on their way
        auto load_bc = [&](int k) {
            if (lane == 0) {
                const int row = g.row + k * kQ;
                mbar_arrive_tx(bar(kFull), 4 * kAtom);
                tma_load_2d(base + kOffC, &c_map, bar(kFull), hg * kN, row);
                tma_load_2d(base + kOffB, &b_map, bar(kFull), hg * kN, row);
                tma_load_2d(base + kOffC + kAtom, &c_map, bar(kFull), hg * kN + 64, row);
                tma_load_2d(base + kOffB + kAtom, &b_map, bar(kFull), hg * kN + 64, row);
            }
            bc = k + 1;
        };
        auto load_x = [&](int k) {
            if (lane == 0) {
                const int row = g.row + k * kQ;
                mbar_arrive_tx(bar(kXFull), kAtom);
                tma_load_2d(base + kOffX, &x_map, bar(kXFull), h * kP, row);
                if (k + 1 < K) tma_prefetch_2d(&x_map, h * kP, row + kQ);
            }
            xs = k + 1;
        };
        if (K > 0) {
            load_bc(0);
            load_x(0);
            load_dt(0);
            write_step(0);
        }
        for (int k = 0; k + 1 < K; ++k) {
            write_step(k + 1);   // (its buffer's last reader was chunk k - 1, behind yfull(k - 1))
            if (!wait(bar(kSFull), k & 1)) break;
            load_bc(k + 1);
            if (!wait(bar(kYFull), k & 1)) break;
            load_x(k + 1);
        }
        if (lane == 0) {   // loads in flight must land
            if (bc) mbar_wait(bar(kFull), (bc - 1) & 1);
            if (xs) mbar_wait(bar(kXFull), (xs - 1) & 1);
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ---- MMA issue (one thread) ----
        if (lane == 0) {
            constexpr uint32_t id_g = bf16_idesc(128, 128, false, false);   // G = C B^T
            constexpr uint32_t id_y = bf16_idesc(128, 64, false, true);     // C H^T and M' X
            const uint64_t dc = sw128_desc(base + kOffC, 16, 1024), db = sw128_desc(base + kOffB, 16, 1024);
            const uint64_t dh = sw128_desc(base + kOffH, kAtom, 1024), dx = sw128_desc(base + kOffX, kAtom, 1024);
            auto wait = [&](int b, int k) {
                if (wait_for(bar(b), k & 1, abort_flag, wlim)) return true;
                give_up(p.status, abort_flag);
                return false;
            };
            for (int k = 0; k < K; ++k) {
                if (!wait(kFull, k) || (k > 0 && !wait(kYFull, k - 1))) break;   // (M' X(k - 1) reads G's columns)
                tc_after_sync();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t off = ((uint32_t)(i >> 2) * kAtom + (uint32_t)(i & 3) * 32u) >> 4;
                    mma_bf16(tmem + kColG, dc + off, db + off, id_g, i > 0);
                }
                if (!wait(kHReady, k)) break;
                tc_after_sync();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t off = ((uint32_t)(i >> 2) * kAtom + (uint32_t)(i & 3) * 32u) >> 4;
                    mma_bf16(tmem + kColY, dc + off, dh + (uint32_t)i * (2048u >> 4), id_y, i > 0);
                }
                mma_commit(bar(kGFull));
                if (!wait(kWReady, k)) break;
                tc_after_sync();
                issue_state_product(tmem, base, true);
                mma_commit(bar(kSFull));
                if (!wait(kMReady, k)) break;
                tc_after_sync();
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    mma_bf16_ta(tmem + kColY, tmem + kColG + 16u * (uint32_t)i, dx + (uint32_t)i * (2048u >> 4), id_y,
                                1);
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
            if (ok) ok = __all_sync(0xffffffffu, wait_for(b, parity, abort_flag, wlim));
            if (!ok && lane == 0) give_up(p.status, abort_flag);
        };
        float *cache = p.state ? p.state + slot * p.s_slot + (int64_t)h * (kP * kN) : nullptr;
        const bool resumed = cache && p.has_init && p.has_init[g.seq];
        // the state before the segment
        const bool last = cache && g.seg + 1 == g.nseg;
        auto give = [&](int b) {
            async_proxy_fence();
            tc_before_sync();
            __syncwarp();
            if (lane == 0 && ok) mbar_arrive(bar(b));
        };
        // what a chunk starts from: the state's bf16 tile, and its decayed value in the accumulator
        auto start = [&](int c, const float (&v)[16], float decay) {
            state_tile(base + kOffH, r, c, v);
            tmem_store16_scaled(tl + kColS + 16u * c, v, decay);
        };
        if (K > 0) wait(bar(kStep0), 0);
        const float decay0 = ex2(step[0].s[kQ - 1]);
#pragma unroll 1
        for (int c = kCQ * hq; c < kCQ * (hq + 1); ++c) {
            float v[16];
            if (g.nseg == 1) {
                load_state(resumed ? cache : nullptr, r, c, v);
            } else if (g.seg == 0) {
                load_state(resumed ? seg_state(p, g.base + g.nseg - 1, h) : nullptr, r, c, v);
            } else {
                load_state(seg_state(p, place - 1, h), r, c, v);
            }
            if (K > 0) {
                if (ok) start(c, v, decay0);
            } else if (last && !resumed) {   // an empty sequence leaves the state it starts from
                store_state(cache, r, c, v);
            }
        }
        if (K > 0) {
            tmem_store_wait();
            give(kHReady);
        }
        const float Dh = p.D ? p.D[h] : 0.f;
        const int64_t col = (int64_t)h * kP + 16 * kCQ * hq;
        for (int k = 0; k < K; ++k) {
            const bool live = r < g.len - k * kQ;
            const StepData &st = step[k & 1];
            wait(bar(kXFull), k & 1);
            wait(bar(kGFull), k & 1);
            if (ok) {
                tc_after_sync();
                const float er = ex2(st.s[r]), w = st.w[r];
#pragma unroll 1
                for (int c = kCQ * hq; c < kCQ * (hq + 1); ++c) {
                    float y[16];
                    tmem_load16(tl + kColY + 16u * c, y);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const uint32_t at = base + kOffX + sw128((uint32_t)r, (uint32_t)(2 * c + q));
                        uint4 xr = ld_shared_v4(at);
                        if (!live) {
                            // rows behind the sequence hold other data (any bits): zero where products sum over them
                            xr = make_uint4(0u, 0u, 0u, 0u);
                            st_shared_v4(at, 0u, 0u, 0u, 0u);
                        }
                        float2 x[4];
                        widen8(xr, x);
                        store_split(base + kOffC, r, 2 * c + q, x, w);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int j = 8 * q + 2 * e;
                            const float2 t = fma2(f2(er, er), f2(y[j], y[j + 1]), mul2(f2(Dh, Dh), x[e]));
                            y[j] = t.x;
                            y[j + 1] = t.y;
                        }
                    }
                    tmem_store16(tl + kColY + 16u * c, y);
                }
                if (!live) {
#pragma unroll
                    for (int i = 0; i < 4 * kCQ; ++i) {
                        const uint32_t q = (uint32_t)(4 * kCQ * hq + i);
                        st_shared_v4(base + kOffB + (q >> 3) * kAtom + sw128((uint32_t)r, q & 7u), 0u, 0u, 0u, 0u);
                    }
                }
                tmem_store_wait();
            }
            give(kWReady);
            if (ok) {
#pragma unroll 1
                for (int kk = hq; kk < 8; kk += kParts) build_mask(tl + kColG, st, r, sub, kk);
                tmem_store_wait();
            }
            give(kMReady);

            wait(bar(kSFull), k & 1);
            if (k + 1 < K) wait(bar(kStep0 + ((k + 1) & 1)), ((k + 1) >> 1) & 1);
            if (ok) {
                tc_after_sync();
                const float decay = ex2(step[(k + 1) & 1].s[kQ - 1]);
#pragma unroll 1
                for (int c = kCQ * hq; c < kCQ * (hq + 1); ++c) {
                    float v[16];
                    tmem_load16(tl + kColS + 16u * c, v);
                    if (k + 1 < K) start(c, v, decay);
                    else if (last) store_state(cache, r, c, v);   // the state after the sequence
                }
                tmem_store_wait();
            }
            wait(bar(kYFull), k & 1);
            uint32_t o[8 * kCQ];
            if (ok) {
                tc_after_sync();
                const int64_t row = (int64_t)g.row + k * kQ + r;
                const uint4 *zp = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.z) + row * p.z_st + col);
#pragma unroll
                for (int c = 0; c < kCQ; ++c) {
                    float y[16];
                    tmem_load16(tl + kColY + 16u * (kCQ * hq + c), y);
                    if (GATE && live) {
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            float2 z[4];
                            widen8(__ldg(zp + 2 * c + q), z);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                y[8 * q + 2 * e] *= z[e].x * sigmoid(z[e].x);
                                y[8 * q + 2 * e + 1] *= z[e].y * sigmoid(z[e].y);
                            }
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[8 * c + e] = pack_bf16(y[2 * e], y[2 * e + 1]);
                }
            }
            if (k + 1 < K) give(kHReady);
            if (ok && live) {
                uint16_t *yp = static_cast<uint16_t *>(p.y) + ((int64_t)g.row + k * kQ + r) * p.y_st + col;
#pragma unroll
                for (int c = 0; c < kCQ; ++c) {
                    if (p.y_wide) {
                        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(yp + 16 * c),
                                     "r"(o[8 * c]), "r"(o[8 * c + 1]), "r"(o[8 * c + 2]), "r"(o[8 * c + 3]),
                                     "r"(o[8 * c + 4]), "r"(o[8 * c + 5]), "r"(o[8 * c + 6]), "r"(o[8 * c + 7])
                                     : "memory");
                    } else {
                        reinterpret_cast<uint4 *>(yp)[2 * c] = make_uint4(o[8 * c], o[8 * c + 1], o[8 * c + 2], o[8 * c + 3]);
                        reinterpret_cast<uint4 *>(yp)[2 * c + 1] = 
                            make_uint4(o[8 * c + 4], o[8 * c + 5], o[8 * c + 6], o[8 * c + 7]);
                    }
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

// Chunks per segment (0: sequences are not cut): the smallest estimate of the
// time, in chunk times of the 2 x num_sms CTAs that run together. n CTAs of at
// most c chunks take c when they all run at once, else their work spread over
// the places plus half a CTA at the end. A CTA's start costs about 0.7 of a
// chunk; a chunk of the first kernel costs half as much as one of the third,
// and the additional launches and the pass along the segments about 1 and one
// thousandth of a chunk for each segment and head.
int ssd_packed_segment(int64_t tokens, int64_t nseq, int64_t nheads, int64_t max_seqlen, int num_sms)
{
    const double slots = 2.0 * (num_sms > 0 ? num_sms : 1);
    const int64_t longest = ((max_seqlen > 0 ? min64(max_seqlen, tokens) : tokens) + kQ - 1) / kQ;
    const double chunks = (double)tokens / kQ + 0.5 * (double)nseq, h = (double)nheads;
    const auto spread = [&](double n, double mean, double most) {
        return n <= slots ? most : n * mean / slots + 0.5 * most;
    };
    double best = spread((double)nseq * h, chunks / (double)nseq + 0.7, (double)longest + 0.7);
    int pick = 0;
    for (int c = 2; c < longest && c <= 128; ++c) {
        const double segs = chunks / c + 0.5 * (double)nseq, mean = chunks / segs;
        const double early = max64(0, (int64_t)(segs - (double)nseq));   // not their sequence's last
        const double t = spread(segs * h, mean + 0.7, c + 0.7) + 0.5 * spread(early * h, c + 1.4, c + 1.4) + 1.0 +
                         0.001 * early * h;
        if (t < best) {
            best = t;
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

cudaError_t launch_ssd_packed(const SsdPackedParams &p0, cudaStream_t stream)
{
    SsdPackedParams p = p0;
    p.y_wide = reinterpret_cast<uintptr_t>(p.y) % 32 == 0 && p.y_st % 16 == 0;
    CUtensorMap xm, bm, cm;
    // (without tokens nothing is loaded; the maps then only need a valid address)
    const int64_t rows = max64(p.tokens, 1);
    const void *none = p.status;
    const int64_t xi = p.nheads * kP, bi = p.ngroups * kN;
    if (!encode_rows(&xm, p.tokens ? p.x : none, xi, rows, p.tokens ? p.x_st : xi) ||
        !encode_rows(&bm, p.tokens ? p.B : none, bi, rows, p.tokens ? p.B_st : bi) ||
        !encode_rows(&cm, p.tokens ? p.C : none, bi, rows, p.tokens ? p.C_st : bi))
        return cudaErrorNotSupported;
    const auto kernel = p.z ? ssd_packed_kernel<true> : ssd_packed_kernel<false>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
    if (e == cudaSuccess && p.seg_chunks)
        e = cudaFuncSetAttribute(ssd_packed_states_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)kSmemBytes);
    if (e == cudaSuccess) e = cudaMemsetAsync(p.status, 0, sizeof(int), stream);
    if (e != cudaSuccess) return e;
    const unsigned grid = static_cast<unsigned>(ssd_packed_places(p.tokens, p.nseq, p.seg_chunks) * p.nheads);
    if (p.seg_chunks) {
        ssd_packed_states_kernel<<<grid, kThreads, kSmemBytes, stream>>>(xm, bm, p);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        ssd_packed_pass_kernel<<<static_cast<unsigned>(p.nseq * p.nheads * (kP * kN / 4 / 256)), 256, 0, stream>>>(p);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    kernel<<<grid, kThreads, kSmemBytes, stream>>>(xm, bm, cm, p);
    return cudaGetLastError();
}

}  // namespace ms
