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
// Layout. On sm_100a an MMA of 128 rows takes 64 clocks for any N up to 128
// (measured), so a product with N = 64, one head, wastes half of the tensor
// core. One CTA per SM therefore walks one segment (see below) of TWO heads of
// one group: they share B, C and G, and C H^T and B^T (w X) are products with
// N = 128. Per chunk and pair of heads 48 MMAs of 64 clocks, against 80 one by
// one. Where the SMs have room for a CTA per head, each takes ONE head: its chunk
// still takes 0.7 of the time, with half the arithmetic and shared-memory traffic
// (measured; ssd_packed_plan). 512 columns of tensor memory: G; M' of both heads (the A operand of
// M' X); Y and the states of both. 208 KB of shared memory: X twice (the next
// chunk's loads while this one is worked on), B, C, the split w X and the
// states' bf16 copies, whose place the lo term of w X takes between C H^T and
// the next state. The decayed state and the decayed inter-chunk term with the
// skip are written into the accumulators, so the products add onto them.
// Roles (640 threads): warps 0-15 arithmetic (head w / 8; rows 32 (w % 4) ..
// + 31 of the tile; columns by half, sixteen at a time: next to nothing may spill
// (three registers of the gated kernel do), the L1 that shared memory leaves is too
// small for it), warps 16-17 the heads' step
// sizes, warp 18 TMA loads, warp 19 tensor memory and MMA issue.
// Order within a chunk: w X while G and C H^T run; the start of Y; M' while the
// state product runs; the next state while M' X runs. Loads go out as soon as
// their buffer was read for the last time.
//
// Long sequences with few heads are cut into segments that run side by side
// (ssd_packed_plan): a first kernel computes what every segment but a
// sequence's last adds to the state from zero (the state product alone), a
// second one adds these up along each sequence, a third one does the rest from
// the state that its segment starts from. The kernels of a call follow each other
// on the stream, each starting while the one in front of it ends; no CTA waits
// for another one of its kernel.
//
// Measured on B200, bf16, in runs of a few milliseconds: 16 ragged prompts of 24000
// tokens, 64 heads, half of them resumed, 183 us (2.6 times what its bytes take; the
// longest prompts first, so the SMs end within 3% of each other); 4 x 8192 tokens x
// 64 heads 239 us (the dense kernel, one head per CTA: 385 us); one prompt of 32768
// tokens x 24 heads 136 to 142 us in segments, 41 + 8 + 99 us one by one. Over
// seconds the clock falls under the power limit: 203, 260 and 142 us. Three prompts
// of 378 tokens x 24 heads take 13 us on the device in a chain of calls.
// A chunk of a pair of heads takes about 6800 clocks, of
// which the tensor core works 45%. What bounds it is the chain w X - state
// product - next state - C H^T together with shared memory, which is about 75%
// busy with the products' operands (2304 clocks), TMA (1024) and the arithmetic
// warps' own accesses (1800), so that arithmetic beside the products slows both.
// Measured and not kept (4 x 8192 x 64 heads, against 240 us at the time): C H^T
// issued before G 259 us; w X made while M' X runs 249 us; X kept in registers 241 us (spills);
// one head per CTA and two CTAs per SM 298 us; w X shared out unevenly 271 us; M'
// made while C H^T runs and the next hi term beside M' X (X then read twice) 255 us.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "dependent.cuh"
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
constexpr int kWarpsC = 16;                       // arithmetic warps, eight per head
constexpr int kStepWarp = kWarpsC, kTmaWarp = kWarpsC + 2, kMmaWarp = kWarpsC + 3;
constexpr int kThreads = (kWarpsC + 4) * 32;
constexpr float kMinStep = -160.f;                // smallest log2 decay of one token

// Shared memory from a 1024-byte aligned base; tiles of 128-byte-swizzled atoms.
constexpr uint32_t kAtom = kQ * 128;              // 128 rows of 128 bytes
constexpr uint32_t kOffX = 0;                     // X: two buffers x two heads x (128 tokens x 64)
constexpr uint32_t kOffB = 4 * kAtom;             // B: 128 tokens x 128, two atoms
constexpr uint32_t kOffC = 6 * kAtom;             // C
constexpr uint32_t kOffW = 8 * kAtom;             // the hi terms of w X of both heads
constexpr uint32_t kOffH = 10 * kAtom;            // H of both heads (128 rows n x 64 bf16 along p each), or the lo terms
constexpr uint32_t kOffStep = 12 * kAtom;         // StepData[kSteps][2 heads]
struct StepData {
    float s[kQ];      // running sum of delta A (log2)
    float cf[kQ];     // 2^(s at the end of the token's 32-token block - s_i) delta_i
    float dl[kQ];     // delta_i
    float w[kQ];      // 2^(s_end - s_i) delta_i
};
constexpr int kSteps = 4;                         // chunks of step data, made ahead of their use
constexpr uint32_t kOffBar = kOffStep + kSteps * 2 * sizeof(StepData);
// Barriers; chunk k completes phase k of each, xfull[k % 2] its phase k / 2 and
// step[head][k % 4] its phase k / 4 (ystore, sfree alike). "Heads" are the live ones (the last pair of a
// group with an odd number of heads has one):
//   full    B and C of chunk k landed                        <- TMA bytes
//   xfull   X of chunk k landed                              <- TMA bytes
//   gfull   G(k) and C H^T(k) done: C and the state tile are free  <- tcgen05.commit
//   wready  w X of chunk k written                           <- arithmetic warps of the heads
//   mready  the start of Y and M' of chunk k written, G(k) read  <- arithmetic warps of the heads
//   sfull   the states after chunk k; B, w X and the state tile are free  <- tcgen05.commit
//   yfull   Y(k) done                                        <- tcgen05.commit
//   ystore  y of chunk k in X's place, to be stored from there  <- arithmetic warps of the heads, of buffer k % 2
//   sfree   the same: the step data of chunk k are free      <- tcgen05.commit, of buffer k % 4
//   hready  state tile and accumulator for chunk k written   <- arithmetic warps of the heads
//   yfree   Y(k) read                                        <- arithmetic warps of the heads
//   step    step data of chunk k written                     <- 32 lanes of a step warp
// No waiter falls two phases behind (a parity wait would then miss its phase):
// the next phase of gfull, sfull and yfull needs wready or hready of chunk k + 1,
// which every arithmetic warp gives after its waits for chunk k; that of full
// needs the loading warp, behind its wait for sfull(k); those of ystore, sfree,
// xfull and step of a buffer need that buffer filled again by the warp that waits
// for it; and what the issuing warp waits for follows from what it issues later.
enum Bar { kFull, kXFull0, kXFull1, kGFull, kWReady, kMReady, kSFull, kYFull, kYStore0, kYStore1,
           kHReady, kYFree, kDrain, kStep0, kSFree0 = kStep0 + 2 * kSteps, kNumBars = kSFree0 + kSteps };
constexpr uint32_t kOffTmem = kNumBars * 8;             // behind the barriers: tensor memory address, abort flag
constexpr uint32_t kSmemBytes = kOffBar + kOffTmem + 16;
static_assert(kSmemBytes <= 232448, "shared memory per CTA");
// The states kernel: X three times, where the hi term of w X takes its place, B and
// the lo term twice (the products of one chunk run while the next one's w X is made
// and the one after that is loaded).
constexpr uint32_t kStB = 6 * kAtom, kStL = 10 * kAtom, kStStep = 14 * kAtom;
struct alignas(16) StateStep {
    float w[kQ], decay;   // 2^(s to the segment's end) delta_i; decay from this chunk to the segment's end
};
constexpr uint32_t kStBar = kStStep + 4 * sizeof(StateStep);   // StateStep[2 buffers][2 heads]
constexpr uint32_t kStSmemBytes = kStBar + kOffTmem + 16;
static_assert(kStSmemBytes <= 232448, "shared memory per CTA");

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColG = 0, kColM = 128, kColY = 256, kColS = 384;   // M', Y and S: 64 columns per head

// Index of step data and its barrier's phase.
__device__ __forceinline__ int step_of(int k) { return k & (kSteps - 1); }
__device__ __forceinline__ uint32_t step_phase(int k) { return (uint32_t)(k / kSteps) & 1u; }

// Failures on this device since the library was loaded, for callers that keep no
// workspace and so no status word. Nothing reads it but ssd_packed_failures.
__device__ unsigned long long failures;

// A bounded wait. When its limit runs out it records that in the status word and
// raises the CTA's abort flag; from then on every wait of the CTA returns at once,
// no more loads are issued and the other roles run to their end on what is there:
// all addresses stay in bounds, and the loads and MMAs in flight are still waited
// for before the CTA leaves.
// The slow path is a call: the loops wait in many places and their code has to
// stay small for the instruction cache.
__device__ __noinline__ void wait_slow(uint32_t bar, uint32_t parity, volatile int *abort_flag, int *status,
                                       uint64_t limit_ns)
{
    const uint64_t t0 = global_ns();
    while (!*abort_flag && !mbar_test(bar, parity))
        if (global_ns() - t0 > limit_ns) {
            wait_for_previous();   // (the status word was cleared, or a kernel's failure is in it)
            give_up(status, abort_flag);
            atomicAdd(&failures, 1ull);
        }
}

struct Waiter {
    uint32_t bars;
    volatile int *abort_flag;
    int *status;
    uint64_t limit_ns;
    // one thread
    __device__ __forceinline__ void one(int b, uint32_t parity) const
    {
        const uint32_t at = bars + 8u * (uint32_t)b;
        if (!mbar_test(at, parity)) wait_slow(at, parity, abort_flag, status, limit_ns);
    }
    // all lanes of a warp, together afterwards
    __device__ __forceinline__ void operator()(int b, uint32_t parity) const
    {
        one(b, parity);
        __syncwarp();
    }
    // for the loading warp: false when the CTA has given up. It then issues nothing
    // more: a load is announced only on a barrier whose last phase has completed.
    __device__ __forceinline__ bool go(int b, uint32_t parity) const
    {
        one(b, parity);
        return __all_sync(0xffffffffu, !*abort_flag);
    }
};

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
// Up to 32 sequences are looked up together, one per lane, with their slots and
// in one round of loads (a CTA starts with it); more are searched 32 at a time.
// Whole sequences run longest first up to 32, else in the caller's order (39 of 300
// tokens and one of 1500, 64 heads: 153 us with the long one first, 174 us last).
// slot: the sequence's cache slot, -1 when it is skipped. Called by whole blocks.
__device__ __forceinline__ bool find_segment(const SsdPackedParams &p, int64_t place, int lane, Segment &g, int &slot)
{
    const int T = (int)p.tokens, n = (int)p.nseq;
    const int Qs = p.seg_chunks * kQ;
    if (n <= 32) {
        SeqRange q{0, 0};
        int idx = lane;
        if (lane < n) {
            q = seq_range(p.cu, lane, p.tokens);
            if (p.idx) idx = __ldg(p.idx + lane);
        }
        int s, len = q.end - q.begin;
        if (Qs == 0) {
            // the longest first, so that the last CTAs to start are short
            int rank = 0;
            for (int j = 0; j < n; ++j) {
                const int other = __shfl_sync(0xffffffffu, len, j);
                rank += other > len || (other == len && j < lane);
            }
            s = __ffs(__ballot_sync(0xffffffffu, lane < n && rank == (int)place)) - 1;
        } else {
            s = __popc(__ballot_sync(0xffffffffu, lane < n && (int64_t)(q.begin / Qs) + lane <= place)) - 1;
        }
        s = max(s, 0);
        const int begin = __shfl_sync(0xffffffffu, q.begin, s);
        len = __shfl_sync(0xffffffffu, len, s);
        slot = __shfl_sync(0xffffffffu, idx, s);
        const bool twin = __any_sync(0xffffffffu, lane < s && idx == slot);   // (an earlier sequence's)
        if (!p.state && !p.idx) slot = 0;
        else if (slot < 0 || slot >= p.slots || twin) slot = -1;
        g = {s, begin, len, 0, 1, place};
    } else {
        int lo = (int)place;
        if (Qs > 0) {
            lo = 0;
            for (int m = n; m > 1;) {
                const int step = (m + 31) / 32, c = lane * step;
                bool le = false;
                if (c < m) le = (int64_t)(min(max(__ldg(p.cu + lo + c), 0), T) / Qs) + lo + c <= place;
                const int k = max(__popc(__ballot_sync(0xffffffffu, le)) - 1, 0);
                lo += k * step;
                m = min(step, m - k * step);
            }
        }
        const SeqRange q = seq_range(p.cu, lo, p.tokens);
        g = {lo, q.begin, q.end - q.begin, 0, 1, place};
        slot = p.state || p.idx ? block_slot(p.idx, lo, p.slots) : 0;
    }
    if (Qs == 0) return true;
    g.base = (int64_t)(g.row / Qs) + g.seq;
    const int64_t seg = place - g.base;
    g.nseg = g.len > 0 ? (g.len + Qs - 1) / Qs : 1;
    if (seg < 0 || seg >= g.nseg) return false;
    g.seg = (int)seg;
    g.row += g.seg * Qs;
    g.len = min(g.len - g.seg * Qs, Qs);
    return true;
}

// The step inputs (bf16 bits) of tokens t .. t + 3 of a segment of len tokens, 0
// behind its end. Kept as loaded: widening them here would wait for the loads.
__device__ __forceinline__ void load_steps(const uint16_t *dt, int64_t stride, int t, int len, uint16_t (&v)[4])
{
    const uint16_t *at = dt + t * stride;
#pragma unroll
    for (int j = 0; j < 4; ++j, at += stride) {
        v[j] = 0;
        if (t + j < len) v[j] = __ldg(at);
    }
}

__device__ __forceinline__ float delta_of(const SsdPackedParams &p, uint16_t dt, float bias)
{
    const float v = __uint_as_float((uint32_t)dt << 16) + bias;
    return p.softplus ? softplus_fine(v) : v;
}

// (max.NaN: a decay that is NaN stays NaN, which fmaxf would replace by the bound)
__device__ __forceinline__ float log2_decay(float delta, float A2)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(delta * A2), "f"(kMinStep));
    return r;
}

// Exclusive suffix sums over 128 tokens, four per lane, and the sum of all, of two chunks.
__device__ __forceinline__ void suffix_sums2(const float (&a)[2][4], int lane, float (&suf)[2][4], float (&all)[2])
{
    float dn[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        suf[u][3] = 0.f;
#pragma unroll
        for (int k = 2; k >= 0; --k) suf[u][k] = suf[u][k + 1] + a[u][k + 1];
        dn[u] = suf[u][0] + a[u][0];
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float d0 = __shfl_down_sync(0xffffffffu, dn[0], o), d1 = __shfl_down_sync(0xffffffffu, dn[1], o);
        if (lane + o < 32) {
            dn[0] += d0;
            dn[1] += d1;
        }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        all[u] = __shfl_sync(0xffffffffu, dn[u], 0);
        float after = __shfl_down_sync(0xffffffffu, dn[u], 1);
        if (lane == 31) after = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) suf[u][k] += after;
    }
}

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

__device__ __forceinline__ void widen8(const uint4 &x, float2 (&v)[4])
{
    v[0] = f2(bf16_lo(x.x), bf16_hi(x.x));
    v[1] = f2(bf16_lo(x.y), bf16_hi(x.y));
    v[2] = f2(bf16_lo(x.z), bf16_hi(x.z));
    v[3] = f2(bf16_lo(x.w), bf16_hi(x.w));
}

// Split w x (eight values) into bf16 hi + lo.
__device__ __forceinline__ void split(const uint4 &xr, float w, uint32_t (&hi)[4], uint32_t (&lo)[4])
{
    float2 x[4];
    widen8(xr, x);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 a = mul2(x[e], f2(w, w));
        hi[e] = pack_bf16(a.x, a.y);
        const float2 d = add2(a, f2(-bf16_lo(hi[e]), -bf16_hi(hi[e])));
        lo[e] = pack_bf16(d.x, d.y);
    }
}

// The state product B^T (w X) of both heads, hi then lo, onto what the accumulator holds or in its place.
__device__ __forceinline__ void issue_state_product(uint32_t tmem, uint32_t b_tile, uint32_t hi_tile, uint32_t lo_tile,
                                                    bool onto, int nh)
{
    const uint32_t id_s = bf16_idesc(128, 64 * nh, true, true);
    const uint64_t b = sw128_desc(b_tile, kAtom, 1024);
    const uint64_t hi = sw128_desc(hi_tile, kAtom, 1024), lo = sw128_desc(lo_tile, kAtom, 1024);
#pragma unroll
    for (int k = 0; k < 8; ++k)
        mma_bf16(tmem + kColS, b + (uint32_t)k * (2048u >> 4), hi + (uint32_t)k * (2048u >> 4), id_s, onto || k > 0);
#pragma unroll
    for (int k = 0; k < 8; ++k)
        mma_bf16(tmem + kColS, b + (uint32_t)k * (2048u >> 4), lo + (uint32_t)k * (2048u >> 4), id_s, 1);
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

// Heads h and (nh == 2) h + 1 of group `group`: up to `each` heads of a group per CTA.
struct Pair {
    int h, nh, group;
};

__host__ __device__ __forceinline__ int64_t pairs_of(int64_t nheads, int64_t ngroups, int each)
{
    return ngroups * ((nheads / ngroups + each - 1) / each);
}

__device__ __forceinline__ Pair pair_of(const SsdPackedParams &p, int i)
{
    const int hpg = (int)(p.nheads / p.ngroups), ppg = (hpg + p.each - 1) / p.each, group = i / ppg;
    const int first = p.each * (i - group * ppg);
    return {group * hpg + first, min(p.each, hpg - first), group};
}

// Set up by all threads: barriers, tensor memory, the segment; false when the
// CTA has nothing to do (then nothing is allocated).
__device__ __forceinline__ bool setup(const SsdPackedParams &p, uint8_t *smem, uint32_t base, uint32_t off_bar,
                                      int64_t place, int nh, Segment &g, int &slot, uint32_t &tmem, bool last_too)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (base & 1023u) {
        wait_for_previous();
        if (threadIdx.x == 0) {
            atomicExch(p.status, (int)MS_ERR_ALIGNMENT);
            atomicAdd(&failures, 1ull);
        }
        return false;
    }
    // (the same for every thread)
    if (!find_segment(p, place, lane, g, slot) || slot < 0 || !(last_too || g.seg + 1 < g.nseg)) return false;
    if (threadIdx.x == 0) {
        auto init = [&](int b, int count) { mbar_init(base + off_bar + 8u * (uint32_t)b, (uint32_t)count); };
        for (int b : {kXFull0, kXFull1, kGFull, kSFull, kYFull, kDrain}) init(b, 1);
        init(kFull, 2);   // B and C
        for (int b : {kWReady, kMReady, kHReady, kYFree, kYStore0, kYStore1}) init(b, 8 * nh);
        for (int i = 0; i < 2 * kSteps; ++i) init(kStep0 + i, 32);
        for (int i = 0; i < kSteps; ++i) init(kSFree0 + i, 1);
        *reinterpret_cast<volatile int *>(smem + off_bar + kOffTmem + 8) = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) tmem_alloc(base + off_bar + kOffTmem, kTmemCols);
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    tmem = *reinterpret_cast<volatile uint32_t *>(smem + off_bar + kOffTmem);
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
    wait_for_previous();   // a kernel does not end before the one in front of it has
}

// ---- first kernel: what a segment adds to the state ---------------------------
// Every segment but a sequence's last (so all its chunks are full): the state
// at its end, from the sequence's initial state for the first segment and from
// zero for the others, and its decay. Chunks run from the segment's end to its
// start: the decay of what follows a chunk is then a sum that ends at the
// segment's end, the weights count to there and the chunks' products add up
// without rescaling. Its barriers: xfull0 / xfull1 / sfull X (by
// place), gfull / yfull B, wready / hready w X, step and sfree (the products of the
// chunk are done), these by buffer. No waiter falls two phases behind: the next
// phase of each needs the products of its buffer's last chunk, which need every
// wait for that chunk (w X of chunk i + 1 may be ready before B of chunk i has
// come, so one barrier for both buffers would not do). X loaded into one place once
// it had been read took 44 us against 40 for 32768 tokens x 24 heads.
__global__ void __launch_bounds__(kThreads, 1)
ssd_packed_states_kernel(const __grid_constant__ CUtensorMap x_map, const __grid_constant__ CUtensorMap b_map,
                         const SsdPackedParams p)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = smem_addr(smem);
    const int pairs = (int)pairs_of(p.nheads, p.ngroups, p.each);
    const int64_t place = blockIdx.x / pairs;
    const Pair hp = pair_of(p, (int)(blockIdx.x - place * pairs));
    Segment g;
    int slot;
    uint32_t tmem;
    if (!setup(p, smem, base, kStBar, place, hp.nh, g, slot, tmem, false)) {
        wait_for_previous();
        return;
    }
    auto bar = [&](int i) { return base + kStBar + 8u * (uint32_t)i; };
    StateStep *step = reinterpret_cast<StateStep *>(smem + kStStep);
    const int K = (g.len + kQ - 1) / kQ;
    const Waiter wait{base + kStBar, reinterpret_cast<volatile int *>(smem + kStBar + kOffTmem + 8), p.status,
                      p.wait_limit_ns};
    auto phase = [](int i) { return (uint32_t)(i >> 1) & 1u; };   // of the barriers with two buffers
    auto bfull = [](int i) { return i & 1 ? kYFull : kGFull; };
    auto wready = [](int i) { return i & 1 ? kHReady : kWReady; };
    auto xfull = [](int i) { return i % 3 == 0 ? kXFull0 : i % 3 == 1 ? kXFull1 : kSFull; };
    auto xphase = [](int i) { return (uint32_t)(i / 3) & 1u; };
    auto xplace = [&](int i) { return base + (uint32_t)(2 * (i % 3)) * kAtom; };

    if (warp == kStepWarp || warp == kStepWarp + 1) {
        const int head = warp - kStepWarp, h = hp.h + head;
        if (head < hp.nh) {
            const float A2 = p.A[h] * kLog2e, bias = p.dt_bias ? p.dt_bias[h] : 0.f;
            const uint16_t *dtp = reinterpret_cast<const uint16_t *>(p.dt) + (int64_t)g.row * p.dt_st + h;
            // Two chunks at a time: the sums' shuffles wait for each other, and behind the
            // products' operand reads; those of two chunks overlap.
            uint16_t dtv[2][4];   // the step inputs of the next two chunks
            float after = 0.f;    // decay behind them
            auto fetch = [&](int i, uint16_t (&v)[4]) {
                if (i < K) load_steps(dtp, p.dt_st, (K - 1 - i) * kQ + 4 * lane, g.len, v);
            };
            fetch(0, dtv[0]);
            fetch(1, dtv[1]);
            for (int i0 = 0; i0 < K; i0 += 2) {
                float d[2][4], a[2][4], suf[2][4], all[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        d[u][j] = delta_of(p, dtv[u][j], bias);
                        a[u][j] = log2_decay(d[u][j], A2);
                    }
                    fetch(i0 + 2 + u, dtv[u]);
                }
                suffix_sums2(a, lane, suf, all);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int i = i0 + u;
                    if (i >= K) break;
                    float w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[j] = ex2(suf[u][j] + after) * d[u][j];
                    after += all[u];
                    if (i >= 2) wait(kSFree0 + (i & 1), phase(i - 2));
                    StateStep &st = step[2 * (i & 1) + head];
                    *reinterpret_cast<float4 *>(st.w + 4 * lane) = make_float4(w[0], w[1], w[2], w[3]);
                    if (lane == 0) st.decay = after;
                    mbar_arrive(bar(kStep0 + 2 * (i & 1) + head));
                }
            }
            if (lane == 0) p.seg_decay[place * p.nheads + h] = after;
        }
    } else if (warp == kTmaWarp) {
        int bs = 0, xs = 0;   // chunks whose B, and whose X, are on their way
        auto load_x = [&](int i) {
            if (lane == 0) {
                mbar_arrive_tx(bar(xfull(i)), (uint32_t)hp.nh * kAtom);
                for (int j = 0; j < hp.nh; ++j)
                    tma_load_2d(xplace(i) + (uint32_t)j * kAtom, &x_map, bar(xfull(i)), (hp.h + j) * kP,
                                g.row + (K - 1 - i) * kQ);
            }
            xs = i + 1;
        };
        if (K > 0) load_x(0);
        for (int i = 0; i < K; ++i) {
            const int row = g.row + (K - 1 - i) * kQ;
            if (i >= 2 && !wait.go(kSFree0 + (i & 1), phase(i - 2))) break;
            if (lane == 0) {
                const uint32_t full = bar(bfull(i)), b = base + kStB + (uint32_t)(2 * (i & 1)) * kAtom;
                mbar_arrive_tx(full, 2 * kAtom);
                tma_load_2d(b, &b_map, full, hp.group * kN, row);
                tma_load_2d(b + kAtom, &b_map, full, hp.group * kN + 64, row);
            }
            bs = i + 1;
            if (i + 1 < K) load_x(i + 1);   // (its place was free with chunk i - 2's products, too)
            __syncwarp();
        }
        if (lane == 0) {   // loads in flight must land
            for (int i = max(0, xs - 3); i < xs; ++i) mbar_wait(bar(xfull(i)), xphase(i));
            for (int i = max(0, bs - 2); i < bs; ++i) mbar_wait(bar(bfull(i)), phase(i));
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        if (lane == 0) {
            for (int i = 0; i < K; ++i) {
                wait.one(bfull(i), phase(i));
                wait.one(wready(i), phase(i));
                tc_after_sync();
                const uint32_t two = (uint32_t)(2 * (i & 1)) * kAtom;
                issue_state_product(tmem, base + kStB + two, xplace(i), base + kStL + two, i > 0, hp.nh);
                mma_commit(bar(kSFree0 + (i & 1)));
            }
            mma_commit(bar(kDrain));   // every MMA must finish before the tensor memory is freed
            mbar_wait(bar(kDrain), 0);
        }
        __syncwarp();
    } else if ((warp >> 3) < hp.nh) {
        const int head = warp >> 3, h = hp.h + head, sub = warp & 3, hq = (warp >> 2) & 1, r = sub * 32 + lane;
        const uint32_t tl = tmem + ((uint32_t)(sub * 32) << 16) + kColS + 64u * (uint32_t)head;
        const bool resumed = g.seg == 0 && p.state && p.has_init && p.has_init[g.seq];
        const float *cache = resumed ? p.state + slot * p.s_slot + (int64_t)h * (kP * kN) : nullptr;
        for (int i = 0; i < K; ++i) {
            wait(kStep0 + 2 * (i & 1) + head, phase(i));
            wait(xfull(i), xphase(i));
            const float w = step[2 * (i & 1) + head].w[r];
            const uint32_t xt = xplace(i) + (uint32_t)head * kAtom;
            const uint32_t lt = base + kStL + (uint32_t)(2 * (i & 1) + head) * kAtom;
            if (i >= 2) wait(kSFree0 + (i & 1), phase(i - 2));
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t at = sw128((uint32_t)r, (uint32_t)(4 * hq + q));
                uint32_t hi[4], lo[4];
                split(ld_shared_v4(xt + at), w, hi, lo);
                st_shared_v4(xt + at, hi[0], hi[1], hi[2], hi[3]);
                st_shared_v4(lt + at, lo[0], lo[1], lo[2], lo[3]);
            }
            async_proxy_fence();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(wready(i)));
        }
        wait(kSFree0 + ((K - 1) & 1), phase(K - 1));
        dependents_may_start();
        tc_after_sync();
        const float f = ex2(step[2 * ((K - 1) & 1) + head].decay);
        float v[32];
        if (cache) {
            // the third kernel's first segment reads the initial state from its copy: its
            // last segment replaces the one in the cache
            load_state(cache, r, hq, v);
            store_state(seg_state(p, g.base + g.nseg - 1, h), r, hq, v);
            float t[32];
            tmem_load32(tl + 32u * hq, t);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = fmaf(f, v[j], t[j]);
        } else {
            tmem_load32(tl + 32u * hq, v);
        }
        store_state(seg_state(p, place, h), r, hq, v);
    }
    teardown(tmem);
}

// ---- second kernel: the state at the end of each segment ------------------------
// A thread takes four values of the state of one (sequence, head) through the
// sequence's segments: place m then holds the state after segment m.
__global__ void __launch_bounds__(256) ssd_packed_pass_kernel(const SsdPackedParams p)
{
    wait_for_previous();
    dependents_may_start();
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
    constexpr int U = 8;   // segments loaded ahead
    for (int m = 1; m + 1 < nseg; m += U) {
        const int n = min(U, nseg - 1 - m);
        float4 a[U];
        float f[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (u < n) {
                a[u] = __ldcg(at + (u + 1) * step);
                f[u] = __ldcg(p.seg_decay + (base + m + u) * p.nheads + h);
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (u < n) {
                const float e = ex2(f[u]);
                v.x = fmaf(e, v.x, a[u].x);
                v.y = fmaf(e, v.y, a[u].y);
                v.z = fmaf(e, v.z, a[u].z);
                v.w = fmaf(e, v.w, a[u].w);
                __stcg(at + (u + 1) * step, v);
            }
        at += U * step;
    }
}

// ---- third kernel: outputs and final states ------------------------------------

// M' of row r of the 32-row block `sub`: the 32 columns of G of block j <= sub
// become 16 columns of packed pairs. The decay is split at the end of the
// column's block: 2^(s_r - s_e) 2^(s_e - s_i). Before the diagonal block both
// factors are at most 1 for a decaying state. In it the first one grows up to
// the block's whole decay, which fits a float32 (and its counterpart does not
// vanish) up to 2^100; stronger decays take the difference itself. (The blocks
// behind the diagonal are zero, written once.)
__device__ __forceinline__ void build_mask(uint32_t tg, uint32_t tm, const StepData &st, float sr, int r, int sub, int j)
{
    uint32_t m[16];
    float gv[32];
    tmem_load32(tg + 32u * (uint32_t)j, gv);
    const float se = st.s[32 * j + 31];
    if (j < sub || fabsf(st.s[32 * j] - se) <= 100.f) {
        const float rf = ex2(sr - se);
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
            const float4 c = *reinterpret_cast<const float4 *>(st.cf + 32 * j + 2 * e);
            const float2 a = mul2(f2(gv[2 * e], gv[2 * e + 1]), mul2(f2(rf, rf), f2(c.x, c.y)));
            const float2 b = mul2(f2(gv[2 * e + 2], gv[2 * e + 3]), mul2(f2(rf, rf), f2(c.z, c.w)));
            m[e] = pack_bf16(a.x, a.y);
            m[e + 1] = pack_bf16(b.x, b.y);
        }
        if (j == sub) {
            // row r sees the block's columns up to its own
            const int seen = r - 32 * j;
#pragma unroll
            for (int e = 0; e < 16; ++e)
                m[e] = 2 * e + 1 <= seen ? m[e] : 2 * e == seen ? m[e] & 0xFFFFu : 0u;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
            const float4 s = *reinterpret_cast<const float4 *>(st.s + 32 * j + 2 * e);
            const float4 d = *reinterpret_cast<const float4 *>(st.dl + 32 * j + 2 * e);
            const int i = 32 * j + 2 * e;
            m[e] = pack_bf16(i <= r ? gv[2 * e] * (ex2(sr - s.x) * d.x) : 0.f,
                             i + 1 <= r ? gv[2 * e + 1] * (ex2(sr - s.y) * d.y) : 0.f);
            m[e + 1] = pack_bf16(i + 2 <= r ? gv[2 * e + 2] * (ex2(sr - s.z) * d.z) : 0.f,
                                 i + 3 <= r ? gv[2 * e + 3] * (ex2(sr - s.w) * d.w) : 0.f);
        }
    }
    tmem_store16(tm + 16u * (uint32_t)j, m);
}

// The status word, cleared in front of a call's kernels: they start beside it.
__global__ void ssd_packed_clear_kernel(int *status)
{
    dependents_may_start();
    *status = 0;
}

// GATE: y is multiplied by silu(z) (its own kernel: the code of the loop has to
// stay small for the instruction cache).
template <bool GATE>
__global__ void __launch_bounds__(kThreads, 1)
ssd_packed_kernel(const __grid_constant__ CUtensorMap x_map, const __grid_constant__ CUtensorMap b_map,
                  const __grid_constant__ CUtensorMap c_map, const __grid_constant__ CUtensorMap y_map,
                  const SsdPackedParams p)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = smem_addr(smem);
    const int pairs = (int)pairs_of(p.nheads, p.ngroups, p.each);
    const int64_t place = blockIdx.x / pairs;
    const Pair hp = pair_of(p, (int)(blockIdx.x - place * pairs));
    Segment g;
    int slot;
    uint32_t tmem;
    if (!setup(p, smem, base, kOffBar, place, hp.nh, g, slot, tmem, true)) {
        wait_for_previous();
        return;
    }
    auto bar = [&](int i) { return base + kOffBar + 8u * (uint32_t)i; };
    StepData *step = reinterpret_cast<StepData *>(smem + kOffStep);
    const int K = (g.len + kQ - 1) / kQ;
    const Waiter wait{base + kOffBar, reinterpret_cast<volatile int *>(smem + kOffBar + kOffTmem + 8), p.status, p.wait_limit_ns};

    // (by every role in front of its first wait for another one that needs the segments'
    // states: the time until these are there must not count as its wait)
    auto after_states = [&] {
        if (p.seg_chunks) wait_for_previous();
    };

    if (warp == kStepWarp || warp == kStepWarp + 1) {
        // ---- step data of one head, up to kSteps chunks ahead ----
        const int head = warp - kStepWarp, h = hp.h + head;
        if (head < hp.nh) {
            const float A2 = p.A[h] * kLog2e, bias = p.dt_bias ? p.dt_bias[h] : 0.f;
            const uint16_t *dtp = reinterpret_cast<const uint16_t *>(p.dt) + (int64_t)g.row * p.dt_st + h;
            uint16_t dtv[4];   // the step inputs of the next chunk
            load_steps(dtp, p.dt_st, 4 * lane, g.len, dtv);
            for (int k = 0; k < K; ++k) {
                if (k == kSteps) after_states();
                if (k >= kSteps) wait(kSFree0 + step_of(k), step_phase(k - kSteps));
                float d[4], a[4], pre[4], suf[4], all, cf[4], w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool in = k * kQ + 4 * lane + j < g.len;
                    d[j] = in ? delta_of(p, dtv[j], bias) : 0.f;
                    a[j] = in ? log2_decay(d[j], A2) : 0.f;
                }
                load_steps(dtp, p.dt_st, (k + 1) * kQ + 4 * lane, g.len, dtv);
                token_sums(a, lane, pre, suf, all);
                // running sum at the end of the 32-token block (lanes 8 b .. 8 b + 7 hold block b)
                const float send = __shfl_sync(0xffffffffu, pre[3], lane | 7);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    cf[j] = ex2(send - pre[j]) * d[j];
                    w[j] = ex2(suf[j]) * d[j];
                }
                StepData &st = step[2 * step_of(k) + head];
                *reinterpret_cast<float4 *>(st.s + 4 * lane) = make_float4(pre[0], pre[1], pre[2], pre[3]);
                *reinterpret_cast<float4 *>(st.cf + 4 * lane) = make_float4(cf[0], cf[1], cf[2], cf[3]);
                *reinterpret_cast<float4 *>(st.dl + 4 * lane) = make_float4(d[0], d[1], d[2], d[3]);
                *reinterpret_cast<float4 *>(st.w + 4 * lane) = make_float4(w[0], w[1], w[2], w[3]);
                mbar_arrive(bar(kStep0 + 2 * step_of(k) + head));
            }
        }
    } else if (warp == kTmaWarp) {
        // ---- loads, each as soon as its buffer was read for the last time ----
        int cs = 0, bs = 0, xs = 0;   // chunks whose C, B and X are on their way
        auto load_bc = [&](const CUtensorMap *map, uint32_t tile, int k) {
            if (lane == 0) {
                const int row = g.row + k * kQ, col = hp.group * kN;
                mbar_arrive_tx(bar(kFull), 2 * kAtom);
                tma_load_2d(tile, map, bar(kFull), col, row);
                tma_load_2d(tile + kAtom, map, bar(kFull), col + 64, row);
            }
        };
        // (the wait: its source may be overwritten; the CTA also leaves only after that)
        auto store_y = [&](int k) {
            if (lane == 0) {
                for (int j = 0; j < hp.nh; ++j)
                    tma_store_2d(&y_map, base + kOffX + (uint32_t)(2 * (k & 1) + j) * kAtom, (hp.h + j) * kP,
                                 g.row + k * kQ);
                tma_store_read_wait();
            }
            __syncwarp();
        };
        auto load_x = [&](int k) {
            if (lane == 0) {
                const int row = g.row + k * kQ, st = k & 1;
                mbar_arrive_tx(bar(kXFull0 + st), (uint32_t)hp.nh * kAtom);
                for (int j = 0; j < hp.nh; ++j)
                    tma_load_2d(base + kOffX + (uint32_t)(2 * st + j) * kAtom, &x_map, bar(kXFull0 + st),
                                (hp.h + j) * kP, row);
            }
            xs = k + 1;
        };
        bool ok = true;
        for (int k = -1; k + 1 < K; ++k) {
            if (k == 0) after_states();
            if (k >= 0 && !(ok = wait.go(kGFull, k & 1))) break;
            load_bc(&c_map, base + kOffC, k + 1);
            cs = k + 2;
            if (k >= 0 && !(ok = wait.go(kSFull, k & 1))) break;
            load_bc(&b_map, base + kOffB, k + 1);
            bs = k + 2;
            if (k < 0) {
                load_x(0);
                if (K > 1) load_x(1);
            } else {
                // y of chunk k (a full one) from X's place, then X of chunk k + 2 there
                if (!(ok = wait.go(kYStore0 + (k & 1), (uint32_t)(k >> 1) & 1u))) break;
                store_y(k);
                if (k + 2 < K) load_x(k + 2);
            }
        }
        if (K == 1) after_states();
        if (ok && K > 0 && g.len >= K * kQ && wait.go(kYStore0 + ((K - 1) & 1), (uint32_t)((K - 1) >> 1) & 1u))
            store_y(K - 1);
        if (lane == 0) {   // loads in flight must land
            if (cs > bs) mbar_arrive(bar(kFull));   // (given up between the two: C's phase ends without B)
            if (cs) mbar_wait(bar(kFull), (uint32_t)(cs - 1) & 1u);
            for (int k = max(0, xs - 2); k < xs; ++k) mbar_wait(bar(kXFull0 + (k & 1)), (uint32_t)(k >> 1) & 1u);
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ---- MMA issue (one thread) ----
        if (lane == 0) {
            constexpr uint32_t id_g = bf16_idesc(128, 128, false, false);   // G = C B^T
            const uint32_t id_o = bf16_idesc(128, 64 * hp.nh, false, true); // C H^T of the heads
            constexpr uint32_t id_y = bf16_idesc(128, 64, false, true);     // M' X
            const uint64_t dc = sw128_desc(base + kOffC, 16, 1024), db = sw128_desc(base + kOffB, 16, 1024);
            const uint64_t dh = sw128_desc(base + kOffH, kAtom, 1024), dx = sw128_desc(base + kOffX, kAtom, 1024);
            for (int k = 0; k < K; ++k) {
                // (G(k - 1) was read before mready(k - 1), which the M' X products waited for)
                wait.one(kFull, k & 1);
                tc_after_sync();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t off = ((uint32_t)(i >> 2) * kAtom + (uint32_t)(i & 3) * 32u) >> 4;
                    mma_bf16(tmem + kColG, dc + off, db + off, id_g, i > 0);
                }
                if (k == 0) after_states();
                wait.one(kHReady, k & 1);
                if (k > 0) wait.one(kYFree, (k - 1) & 1);
                tc_after_sync();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t off = ((uint32_t)(i >> 2) * kAtom + (uint32_t)(i & 3) * 32u) >> 4;
                    mma_bf16(tmem + kColY, dc + off, dh + (uint32_t)i * (2048u >> 4), id_o, i > 0);
                }
                mma_commit(bar(kGFull));
                wait.one(kWReady, k & 1);
                tc_after_sync();
                issue_state_product(tmem, base + kOffB, base + kOffW, base + kOffH, true, hp.nh);
                mma_commit(bar(kSFull));
                wait.one(kMReady, k & 1);
                tc_after_sync();
                for (int j = 0; j < hp.nh; ++j) {
                    const uint64_t dxj = dx + (((uint32_t)(2 * (k & 1) + j) * kAtom) >> 4);
                    const uint32_t my = tmem + kColY + 64u * (uint32_t)j, mm = tmem + kColM + 64u * (uint32_t)j;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        mma_bf16_ta(my, mm + 8u * (uint32_t)i, dxj + (uint32_t)i * (2048u >> 4), id_y, 1);
                }
                mma_commit(bar(kYFull));
                mma_commit(bar(kSFree0 + step_of(k)));
            }
            mma_commit(bar(kDrain));   // every MMA must finish before the tensor memory is freed
            mbar_wait(bar(kDrain), 0);
        }
        __syncwarp();
    } else if ((warp >> 3) < hp.nh) {
        const int head = warp >> 3, h = hp.h + head, sub = warp & 3, hq = (warp >> 2) & 1, r = sub * 32 + lane;
        const uint32_t tl = tmem + ((uint32_t)(sub * 32) << 16);
        const uint32_t ty = tl + kColY + 64u * (uint32_t)head, ts = tl + kColS + 64u * (uint32_t)head;
        const uint32_t tm = tl + kColM + 64u * (uint32_t)head, htile = base + kOffH + (uint32_t)head * kAtom;
        float *cache = p.state ? p.state + slot * p.s_slot + (int64_t)h * (kP * kN) : nullptr;
        const bool resumed = cache && p.has_init && p.has_init[g.seq];
        const bool last = cache && g.seg + 1 == g.nseg;
        auto give = [&](int b) {
            async_proxy_fence();
            tc_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(b));
        };
        // what a chunk starts from: the state's bf16 tile, and its decayed value in the accumulator
        auto start = [&](float (&v)[32], float decay) {
            state_tile(htile, r, hq, v);
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
                const float2 t = mul2(f2(v[j], v[j + 1]), f2(decay, decay));
                v[j] = t.x;
                v[j + 1] = t.y;
            }
            tmem_store32(ts + 32u * hq, v);
        };
        if (K > 0) wait(kStep0 + head, 0);
        {
            // the state before the segment
            const float *from = g.nseg == 1 ? (resumed ? cache : nullptr)
                                : g.seg > 0 ? seg_state(p, place - 1, h)
                                            : (resumed ? seg_state(p, g.base + g.nseg - 1, h) : nullptr);
            float v[32];
            after_states();
            load_state(from, r, hq, v);
            if (K > 0) {
                start(v, ex2(step[head].s[kQ - 1]));
            } else if (last && !resumed) {   // an empty sequence leaves the state it starts from
                store_state(cache, r, hq, v);
            }
        }
        if (K > 0) {
            const uint32_t zero[16] = {};
            for (int j = sub + 1; j < 4; ++j)
                if ((j & 1) == hq) tmem_store16(tm + 16u * (uint32_t)j, zero);
            tmem_store_wait();
            give(kHReady);
        }
        const float Dh = p.D ? p.D[h] : 0.f;
        const int64_t col = (int64_t)h * kP + 32 * hq;
        for (int k = 0; k < K; ++k) {
            const bool live = r < g.len - k * kQ;
            const StepData &st = step[2 * step_of(k) + head];
            const uint32_t xt = base + kOffX + (uint32_t)(2 * (k & 1) + head) * kAtom;
            wait(kXFull0 + (k & 1), (uint32_t)(k >> 1) & 1u);
            const float sr = st.s[r];
            uint32_t lo[4][4] = {};
            {
                // w X: the hi term into its tile (free since the last state product), the lo term kept
                const float w = st.w[r];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t at = sw128((uint32_t)r, (uint32_t)(4 * hq + q));
                    uint4 xr = ld_shared_v4(xt + at);
                    if (!live) {
                        // rows behind the sequence hold other data (any bits): zero where products sum over them
                        xr = make_uint4(0u, 0u, 0u, 0u);
                        st_shared_v4(xt + at, 0u, 0u, 0u, 0u);
                    }
                    uint32_t hi[4];
                    split(xr, w, hi, lo[q]);
                    st_shared_v4(base + kOffW + (uint32_t)head * kAtom + at, hi[0], hi[1], hi[2], hi[3]);
                }
            }
            wait(kGFull, k & 1);
            {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    st_shared_v4(htile + sw128((uint32_t)r, (uint32_t)(4 * hq + q)), lo[q][0], lo[q][1], lo[q][2],
                                 lo[q][3]);
                if (!live && head == 0) {
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        st_shared_v4(base + kOffB + (uint32_t)hq * kAtom + sw128((uint32_t)r, (uint32_t)q), 0u, 0u, 0u,
                                     0u);
                }
            }
            give(kWReady);
            {
                tc_after_sync();
                const float er = ex2(sr);
                float y[32];
                tmem_load32(ty + 32u * hq, y);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float2 x[4];
                    widen8(ld_shared_v4(xt + sw128((uint32_t)r, (uint32_t)(4 * hq + q))), x);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = 8 * q + 2 * e;
                        const float2 t = fma2(f2(er, er), f2(y[j], y[j + 1]), mul2(f2(Dh, Dh), x[e]));
                        y[j] = t.x;
                        y[j + 1] = t.y;
                    }
                }
                tmem_store32(ty + 32u * hq, y);
#pragma unroll 1
                for (int j = hq; j <= sub; j += 2) build_mask(tl + kColG, tm, st, sr, r, sub, j);
                tmem_store_wait();
            }
            give(kMReady);

            const int64_t row = (int64_t)g.row + k * kQ + r;
            uint4 zq[GATE ? 4 : 1];   // the gate of this thread's outputs, on its way early
            if (GATE && live) {
                const uint4 *zp =
                    reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.z) + row * p.z_st + col);
#pragma unroll
                for (int q = 0; q < 4; ++q) zq[GATE ? q : 0] = __ldg(zp + q);
            }
            wait(kSFull, k & 1);
            if (k + 1 < K) wait(kStep0 + 2 * step_of(k + 1) + head, step_phase(k + 1));
            {
                tc_after_sync();
                float v[32];
                tmem_load32(ts + 32u * hq, v);
                if (k + 1 < K) start(v, ex2(step[2 * step_of(k + 1) + head].s[kQ - 1]));
                else if (last) store_state(cache, r, hq, v);   // the state after the sequence
                tmem_store_wait();
            }
            if (k + 1 < K) give(kHReady);
            wait(kYFull, k & 1);
            float y[32] = {};
            {
                tc_after_sync();
                tmem_load32(ty + 32u * hq, y);
            }
            tc_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kYFree));
            if (live) {
                uint32_t o[16];
                if (GATE) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float2 z[4];
                        widen8(zq[GATE ? q : 0], z);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 t = mul2(f2(y[8 * q + 2 * e], y[8 * q + 2 * e + 1]), mul2(z[e], sigmoid2(z[e])));
                            y[8 * q + 2 * e] = t.x;
                            y[8 * q + 2 * e + 1] = t.y;
                        }
                    }
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = pack_bf16(y[2 * e], y[2 * e + 1]);
                if (g.len >= (k + 1) * kQ) {
                    // a full chunk: into X's place, from where it is stored as a tile
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        st_shared_v4(xt + sw128((uint32_t)r, (uint32_t)(4 * hq + q)), o[4 * q], o[4 * q + 1],
                                     o[4 * q + 2], o[4 * q + 3]);
                } else {
                    // the sequence's last rows: other sequences' rows follow them
                    uint4 *yp = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.y) + row * p.y_st + col);
#pragma unroll
                    for (int q = 0; q < 4; ++q) yp[q] = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
                }
            }
            give(kYStore0 + (k & 1));
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

// A chunk of one head takes kOneHead of the time of a chunk of two (4096 tokens x
// 128 heads, a CTA per head against one per pair: 98 against 142 us; 512 tokens x
// 24 heads 16 against 20 us; where a CTA per head fills the SMs more than once the
// pairs win: 8192 tokens x 64 heads 105 against 186 us in segments).
constexpr double kOneHead = 0.7;

// Chunks per segment (0: sequences are not cut) and heads per CTA: the smallest
// estimate of the time, in chunk times of the num_sms CTAs that run together. n CTAs of at
// most c chunks take c when they all run at once, else their work spread over
// the places plus half a CTA at the end. A CTA's start costs about 0.7 of a
// chunk; a chunk of the first kernel costs half as much as one of the third,
// the additional launches about 1, and the pass along the segments one
// two-thousandth for each head and each segment but a sequence's last.
SsdPackedPlan ssd_packed_plan(int64_t tokens, int64_t nseq, int64_t nheads, int64_t ngroups, int64_t max_seqlen, int num_sms)
{
    const double slots = num_sms > 0 ? num_sms : 1;
    const int64_t longest = ((max_seqlen > 0 ? min64(max_seqlen, tokens) : tokens) + kQ - 1) / kQ;
    const double chunks = (double)tokens / kQ + 0.5 * (double)nseq;
    const auto spread = [&](double n, double mean, double most) {
        return n <= slots ? most : n * mean / slots + 0.5 * most;
    };
    SsdPackedPlan best{0, 2};
    double least = 0;
    for (int each = 2; each >= 1; --each) {
        const double h = (double)pairs_of(nheads, ngroups, each), unit = each == 2 ? 1.0 : kOneHead;
        const double whole = unit * spread((double)nseq * h, chunks / (double)nseq + 0.7, (double)longest + 0.7);
        if (each == 2 || whole < least) {
            least = whole;
            best = {0, each};
        }
        for (int c = 2; c < longest && c <= 128; ++c) {
            const double segs = chunks / c + 0.5 * (double)nseq, mean = chunks / segs;
            const double early = max64(0, (int64_t)(segs - (double)nseq));   // not their sequence's last
            const double t = unit * (spread(segs * h, mean + 0.7, c + 0.7) + 0.5 * spread(early * h, c + 1.4, c + 1.4)) +
                             1.0 + 0.001 * early * (double)nheads / 2;
            if (t < least) {
                least = t;
                best = {c, each};
            }
        }
    }
    return best;
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

cudaError_t ssd_packed_failures(unsigned long long *count, cudaStream_t stream)
{
    cudaError_t e = cudaMemcpyFromSymbolAsync(count, failures, sizeof(*count), 0, cudaMemcpyDeviceToHost, stream);
    return e == cudaSuccess ? cudaStreamSynchronize(stream) : e;
}

cudaError_t launch_ssd_packed(const SsdPackedParams &p, cudaStream_t stream)
{
    CUtensorMap xm, bm, cm, ym;
    // (without tokens nothing is loaded; the maps then only need a valid address)
    const int64_t rows = max64(p.tokens, 1);
    const void *none = p.status;
    const int64_t xi = p.nheads * kP, bi = p.ngroups * kN;
    if (!encode_rows(&xm, p.tokens ? p.x : none, xi, rows, p.tokens ? p.x_st : xi) ||
        !encode_rows(&bm, p.tokens ? p.B : none, bi, rows, p.tokens ? p.B_st : bi) ||
        !encode_rows(&cm, p.tokens ? p.C : none, bi, rows, p.tokens ? p.C_st : bi) ||
        !encode_rows(&ym, p.tokens ? p.y : none, xi, rows, p.tokens ? p.y_st : xi))
        return cudaErrorNotSupported;
    const auto kernel = p.z ? ssd_packed_kernel<true> : ssd_packed_kernel<false>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
    if (e == cudaSuccess && p.seg_chunks)
        e = cudaFuncSetAttribute(ssd_packed_states_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)kStSmemBytes);
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>(ssd_packed_places(p.tokens, p.nseq, p.seg_chunks) *
                                          pairs_of(p.nheads, p.ngroups, p.each)));
    ssd_packed_clear_kernel<<<1, 1, 0, stream>>>(p.status);
    e = cudaGetLastError();
    if (e == cudaSuccess && p.seg_chunks) {
        e = launch_dependent(ssd_packed_states_kernel, grid, kThreads, kStSmemBytes, stream, xm, bm, p);
        if (e == cudaSuccess)
            e = launch_dependent(ssd_packed_pass_kernel,
                                 dim3(static_cast<unsigned>(p.nseq * p.nheads * (kP * kN / 4 / 256))), 256, 0, stream, p);
    }
    return e == cudaSuccess ? launch_dependent(kernel, grid, kThreads, kSmemBytes, stream, xm, bm, cm, ym, p) : e;
}

}  // namespace ms
