// Decode attention over the quantised KV cache (one query token per sequence),
// for sm_103a: with g = h / (H_q / H_kv),
//   o_h = sum_{t < L} softmax_t(scale q_h . k_{g,t}) v_{g,t},
//   k_{t,d} = ck_{t,d} sk_{t,c} + bk_{t,c},  v likewise,  c = d / 64.
//
// Mathematics.  The codes themselves are the matrix operands, the affine part
// stays in fp32:
//   q . k_t  = sum_c ( sk_{t,c} sum_{d in c} q_d ck_{t,d}  +  bk_{t,c} sum_{d in c} q_d )
//   o_d      = sum_t (p_t sv_{t,c}) cv_{t,d}  +  sum_t p_t bv_{t,c}
// so no value is ever rebuilt, and nothing of K or V is rounded.  A code needs
// no conversion either: its bits at the bottom of a 16-bit word are the fp16
// subnormal c 2^-24 (at bits 4..7: c 2^-20), which the tensor cores multiply
// exactly; eight codes of 4 bits become four operand registers with one shift and
// four ANDs.  The factors 2^-24 / 2^-20 are undone in fp32.
// q is scaled per head by a power of two into fp16 (2^14..2^15 at its largest
// value, so a value keeps its 8 bits down to 2^-24 of that).  The weights
// p_t sv_{t,c} are rounded to fp16 (2^-11 relative) after a power of two f that
// keeps the largest scale seen in range: f follows the data as the running
// maximum of the softmax does.  One f does while the scales lie within 2^8 of each other,
// as a model's do; a warp that meets others (a token or a group of channels of very
// different size) goes on in a second loop with a factor for each head and group (131,072
// tokens 30.5 us where every V has a scale of 0, 23.5 else).  p is
// taken against a running maximum that moves only when a score passes it by 8 (in
// powers of two), which the vote that looks at the scales finds too; sums are fp32.
//
// Bound: the cache's bytes (36 per 64 values at 4 bits).  Work split: the cache
// blocks of all (sequence, KV head) segments form one list that the CTAs (one per
// SM) share evenly, so a batch of unlike lengths leaves no SM idle; a segment cut
// between CTAs leaves partials that a second kernel joins.  Short caches have a CTA for
// each segment and one launch.
// Inside a CTA:
//   last warps  producers of K and of V: one bulk copy per block for the codes and
//               one for the parameters (contiguous in the cache's layout) into a
//               ring of shared-memory stages;
//   the others  consumers, 16 or 32 tokens at a time each on its own, with their own
//               running maximum, sum and output: no barrier until the segment
//               ends, where the warps' results are joined through shared memory.
//               S^T = K q^T and O^T += V^T P on mma.sync m16n8k16 (fp16 in, fp32
//               out), the query heads of the KV head on the N = 8 side.  The order
//               of channels inside a matrix step is free, so each lane takes the
//               16 channels that one load gives it; P moves from the accumulator
//               layout to the operand layout by movmatrix.
// Every mbarrier wait is bounded; a wait that gives up records
// LILY_ERR_DEVICE_TIMEOUT, and the producers wait for their copies before they exit.
#include <cmath>
#include <cstdint>

#include "kvq_device.cuh"
#include "lily_internal.h"

namespace lily {
namespace {

// Consumer warps: 8 or 10 take 23.5 or 23.8 us for a sequence of 131,072 tokens (2 KV heads of
// 256), 13.7 or 14.1 for 24 short ones (4 heads of 128, 8 bits); eight long ones with 8 heads of
// 128 69.8 or 67.1.  6 are slower on long caches, 14 everywhere (registers).
constexpr int kNW = 8;
// + the producers of K and of V.  With D = 256 a consumer thread needs more than the 168 registers that ten or twelve
// warps have each: the producers' warpgroup (two of its warps idle) then gives registers up (168 x 12 warps =
// 224 x 8 + 56 x 4).  131,072 tokens of 2 heads take 23.2 us so, 24.4 without, at 8 bits 31.0 and 33.9;
// with D = 64 and 128, which fit in 168, the larger CTA costs 1 to 2.5%.
__host__ __device__ constexpr bool splits_registers(int D) { return D == 256; }
__host__ __device__ constexpr int threads_of(int D) { return (kNW + (splits_registers(D) ? 4 : 2)) * 32; }
constexpr int kProducerRegs = 56, kConsumerRegs = 224;
constexpr int kMaxThreads = threads_of(256);
constexpr int kMaxStages = 14;                // segments in flight <= stages < named barriers
constexpr int kSmemLimit = 227 * 1024;
constexpr int kBarriers = 15;                 // named barriers 1..15, by segment
constexpr float kNoMax = -1.7e38f;            // running maximum before any token (finite: -inf - kNoMax = -inf)
// Weights are taken against the running maximum plus kLift: they reach 2^(8 - kLift) at most, so that sums of
// 2^24 of them times values of any finite size stay finite.  (Small values end in fp32's smallest
// numbers instead: outputs below about 2^-100 lose bits.)
constexpr int kLift = 32;
// The factor f of the weights at most: before any token with a scale, and with scales below 2^-88.
constexpr int kMaxFactorLog = 126;
constexpr float kMaxFactor = 0x1p126f;
// f times the scales lies in [kLow, kHigh]: times a weight it is 2^15 at most, which fp16 holds, and times the largest
// weight 2^-1 at least (2^6 for the largest scales).  fp16 rounds the product by 2^-11 of itself, or by 2^-24
// (2^-31) of what the largest weight would have there.
constexpr float kHigh = 0x1p39f, kLow = 0x1p31f;

struct Fixed {
    uint64_t full[kMaxStages], empty[kMaxStages];
    int abort, b0, len0, pre, begin, total, used, sum[kMaxThreads / 32];
    alignas(8) float ml[kNW][8][2];
#ifdef LILY_TEST_STALL_T
    uint64_t never;  // test builds only: a barrier nothing arrives on
#endif
};
constexpr int kFixed = (sizeof(Fixed) + 127) / 128 * 128;

__host__ __device__ constexpr int merge_row(int D) { return D + 8; }  // floats of a head's row in the join buffer, padded
__host__ __device__ constexpr int merge_bytes(int D) { return kNW * 8 * merge_row(D) * 4; }
__host__ __device__ constexpr int stage_bytes(int D, int bs, int bits) { return 2 * (bs * D * bits / 8 + bs * (D / 64) * 4); }
__host__ __device__ constexpr int stages_for(int D, int bs, int bits)
{
    const int n = (kSmemLimit - kFixed - merge_bytes(D)) / stage_bytes(D, bs, bits);
    return n < kMaxStages ? n : kMaxStages;
}
// Tokens that a warp takes at a time: one or two halves of 16.
__host__ __device__ constexpr int unit_of(int D) { return D == 256 ? 16 : 32; }

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
// Registers of a thread from here on, for a warpgroup: more of them come from what another one has given back.
// The kernel is launched with 168 x 384, which the bounds above make it ask for.
template <int N, bool kMore>
__device__ __forceinline__ void set_max_registers()
{
    if constexpr (kMore)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
    else
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// d += a b: m16n8k16, fp16 inputs, fp32 accumulators
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Channel, within the 16 that lane t of a group holds, of slot r (low and high half
// of the first, of the second operand register) of K step j.
template <int BITS>
__device__ __forceinline__ constexpr int k_channel(int j, int r)
{
    return BITS == 4 ? 8 * (j >> 1) + (j & 1) + (r == 0 ? 0 : r == 1 ? 4 : r == 2 ? 2 : 6)
                     : 4 * j + (r == 0 ? 0 : r == 1 ? 2 : r == 2 ? 1 : 3);
}
// A token of the cache row that operand row / column k (0..7) of an 8-token half
// stands for: lanes t = 0..3 of one V load then read four consecutive rows.
__device__ __forceinline__ int token_of(int k) { return (k >> 1) | ((k & 1) << 2); }

__device__ __forceinline__ int length_of(const KvqAttnArgs &a, int L)
{
    const int cap = a.max_blocks * a.c.bs;
    if (L < 0 || L > cap) {
        record_error(&a.ctrl->status, kErrDeviceIndex);
        L = L < 0 ? 0 : cap;
    }
    return L;
}
// Cache blocks of a sequence in the work list (an empty one still has its zeros to write).
__device__ __forceinline__ int blocks_of(int L, int bs) { return L > 0 ? (L + bs - 1) / bs : 1; }

// This CTA's share of the work list: segments from (b, g, block j0) on, `left` blocks in all.
struct Walk {
    int b, g, j0, L, next, left;  // next: the length of sequence b + 1 as stored (loaded one sequence ahead)
};

template <int NT>  // threads of the CTA
__device__ __forceinline__ Walk first_segment(const KvqAttnArgs &a, Fixed &F)
{
    Walk w{};
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = blockIdx.x;
    if (a.whole) {
        w.b = c / a.c.H_kv;
        w.g = c % a.c.H_kv;
        w.L = length_of(a, a.seq_lens[w.b]);
        w.left = blocks_of(w.L, a.c.bs);
        return w;
    }
    if (a.B <= 32) {
        // every warp for itself, a sequence per lane: one load and no barrier
        const int stored = lane < a.B ? a.seq_lens[lane] : 0;
        const int len = lane < a.B ? length_of(a, stored) : 0, n = lane < a.B ? blocks_of(len, a.c.bs) * a.c.H_kv : 0;
        int inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += up;
        }
        const int total = __shfl_sync(0xffffffffu, inc, 31), used = min(total, static_cast<int>(gridDim.x));
        if (c >= used) return w;
        const int per = total / used, rest = total % used;
        const int begin = per * c + rest * c / used;
        w.left = per * (c + 1) + rest * (c + 1) / used - begin;
        w.b = __ffs(__ballot_sync(0xffffffffu, begin < inc)) - 1;
        w.L = __shfl_sync(0xffffffffu, len, w.b);
        w.next = __shfl_sync(0xffffffffu, stored, min(w.b + 1, 31));
        const int nblk = blocks_of(w.L, a.c.bs), off = begin - __shfl_sync(0xffffffffu, inc - n, w.b);
        w.g = off / nblk;
        w.j0 = off % nblk;
        if (lane == 0) {  // the same values from every warp; each reads its own
            F.begin = begin;
            F.total = total;
            F.used = used;
        }
        __syncwarp();
        return w;
    }
    // blocks of sequence s0 + tid: those of the threads before this one, and of all (fewer than 2^31 by the host's check)
    int len = 0, before, all;
    auto scan = [&](int s0) {
        int n = 0;
        if (s0 + tid < a.B) {
            len = length_of(a, a.seq_lens[s0 + tid]);
            n = blocks_of(len, a.c.bs) * a.c.H_kv;
        }
        int inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += up;
        }
        __syncthreads();
        if (lane == 31) F.sum[warp] = inc;
        __syncthreads();
        before = inc - n;
        all = 0;
#pragma unroll
        for (int i = 0; i < NT / 32; ++i) {
            if (i < warp) before += F.sum[i];
            all += F.sum[i];
        }
    };
    int total = 0;
    for (int s0 = 0; s0 < a.B; s0 += NT) {
        scan(s0);
        total += all;
    }
    // no more CTAs than blocks: every CTA between a segment's first and last has a part of it
    const int used = min(total, static_cast<int>(gridDim.x));
    if (c >= used) return w;
    const int per = total / used, rest = total % used;
    const int begin = per * c + rest * c / used;
    w.left = per * (c + 1) + rest * (c + 1) / used - begin;
    // the sequence that `begin` falls into (with no more sequences than threads, the scan above has it)
    int pre = 0;
    for (int s0 = 0; s0 < a.B; s0 += NT) {
        if (a.B > NT) scan(s0);
        const int lo = pre + before, n = s0 + tid < a.B ? blocks_of(len, a.c.bs) * a.c.H_kv : 0;
        if (begin >= lo && begin - lo < n) {
            F.b0 = s0 + tid;
            F.len0 = len;
            F.pre = lo;
            F.begin = begin;
            F.total = total;
            F.used = used;
        }
        pre += all;
        if (begin < pre) break;
    }
    __syncthreads();
    w.b = F.b0;
    w.L = F.len0;
    w.next = w.b + 1 < a.B ? a.seq_lens[w.b + 1] : 0;
    const int nblk = blocks_of(w.L, a.c.bs);
    w.g = (begin - F.pre) / nblk;
    w.j0 = (begin - F.pre) % nblk;
    return w;
}

// The next segment (after `done` blocks of this one).
__device__ __forceinline__ void advance(const KvqAttnArgs &a, Walk &w, int done)
{
    w.left -= done;
    w.j0 = 0;
    if (++w.g == a.c.H_kv) {
        w.g = 0;
        ++w.b;
        if (w.left > 0) {
            w.L = length_of(a, w.next);
            w.next = w.b + 1 < a.B ? a.seq_lens[w.b + 1] : 0;
        }
    }
}

// Four channels of head h of a segment: the warps' results on their common maximum,
// to the output (part < 0: the segment is whole) or to a part's slot.
template <int D>
__device__ __forceinline__ void join_column(const KvqAttnArgs &a, const Fixed &F, const float *merge, const Walk &w, int unit,
                                            int active, int part, int h, int d4)
{
    float M = kNoMax, den = 0.0f;
    float2 ml[kNW];
    const int w0 = unit % kNW;
    auto warp_of = [&](int j) { return w0 + j < kNW ? w0 + j : w0 + j - kNW; };
#pragma unroll
    for (int j = 0; j < kNW; ++j) {
        ml[j] = j < active ? *reinterpret_cast<const float2 *>(F.ml[warp_of(j)][h]) : make_float2(kNoMax, 0.0f);
        M = fmaxf(M, ml[j].x);
    }
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int j = 0; j < kNW; ++j) {
        const float4 x = j < active ? *reinterpret_cast<const float4 *>(merge + (warp_of(j) * 8 + h) * merge_row(D) + d4 * 4)
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
        const float e = ex2(ml[j].x - M);
        den = fmaf(e, ml[j].y, den);
        o.x = fmaf(e, x.x, o.x);
        o.y = fmaf(e, x.y, o.y);
        o.z = fmaf(e, x.z, o.z);
        o.w = fmaf(e, x.w, o.w);
    }
    if (part < 0) {
        const float r = den > 0.0f ? 1.0f / den : 0.0f;
        uint2 y;
        const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * r, o.y * r), hi = __floats2bfloat162_rn(o.z * r, o.w * r);
        y.x = *reinterpret_cast<const uint32_t *>(&lo);
        y.y = *reinterpret_cast<const uint32_t *>(&hi);
        reinterpret_cast<uint2 *>(a.out + (static_cast<size_t>(w.b) * a.H_q + w.g * a.group + h) * D)[d4] = y;
    } else {
        reinterpret_cast<float4 *>(a.part_acc + (static_cast<size_t>(part) * 8 + h) * D)[d4] = o;
        if (d4 == 0) *reinterpret_cast<float2 *>(a.part_ml + (static_cast<size_t>(part) * 8 + h) * 2) = make_float2(M, den);
    }
}

// The pieces of a consumer warp's work (lane = 4 gi + t), which both forms of it below share.
// q per head times a power of two in fp16: the operand registers of the K steps, and the sums per group.
template <int GR>
struct Query {
    uint32_t b[GR * 4][2];
    float sum[GR][2], mul[2];
};
template <int BITS, int GR>
__device__ __forceinline__ void load_query(const KvqAttnArgs &a, const Walk &w, int gi, int t, Query<GR> &q)
{
    constexpr int D = GR * 64;
    const uint16_t *qh = a.q + w.b * a.q_stride + static_cast<long long>(w.g * a.group + (gi < a.group ? gi : 0)) * D;
    uint32_t xs[GR][8];
    float big = 0.0f;
#pragma unroll
    for (int c = 0; c < GR; ++c) {
        const uint4 x0 = *reinterpret_cast<const uint4 *>(qh + c * 64 + t * 16);
        const uint4 x1 = *reinterpret_cast<const uint4 *>(qh + c * 64 + t * 16 + 8);
        xs[c][0] = x0.x; xs[c][1] = x0.y; xs[c][2] = x0.z; xs[c][3] = x0.w;
        xs[c][4] = x1.x; xs[c][5] = x1.y; xs[c][6] = x1.z; xs[c][7] = x1.w;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (gi >= a.group) xs[c][i] = 0u;
            big = fmaxf(big, fmaxf(fabsf(lo_bf16(xs[c][i])), fabsf(hi_bf16(xs[c][i]))));
        }
    }
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
    // 2^(14 - floor(log2 big)): its exponent field, within the normal numbers
    const int ef = big > 0.0f ? min(268 - max(static_cast<int>(__float_as_uint(big) >> 23), 1), 253) : 127;
    const float up = __uint_as_float(static_cast<uint32_t>(ef) << 23);
#pragma unroll
    for (int c = 0; c < GR; ++c) {
        float ones[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float u = BITS == 4 && (j & 1) ? up * 0.0625f : up;  // those codes carry 2^-20
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int i0 = k_channel<BITS>(j, 2 * r), i1 = k_channel<BITS>(j, 2 * r + 1);
                q.b[c * 4 + j][r] = pack_f16((i0 & 1 ? hi_bf16(xs[c][i0 / 2]) : lo_bf16(xs[c][i0 / 2])) * u,
                                            (i1 & 1 ? hi_bf16(xs[c][i1 / 2]) : lo_bf16(xs[c][i1 / 2])) * u);
            }
            // the sums over the group, heads 2t and 2t + 1, by a step against ones (16 where q has a sixteenth)
            const uint32_t one = BITS == 4 && (j & 1) ? 0x4C004C00u : 0x3C003C00u;
            mma_f16(ones, one, one, one, one, q.b[c * 4 + j][0], q.b[c * 4 + j][1]);
        }
        q.sum[c][0] = ones[0] * 0x1p-24f;
        q.sum[c][1] = ones[1] * 0x1p-24f;
    }
    const float m = a.scale_log2 * 0x1p24f * __uint_as_float(static_cast<uint32_t>(254 - ef) << 23);
    q.mul[0] = __shfl_sync(0xffffffffu, m, 8 * t);
    q.mul[1] = __shfl_sync(0xffffffffu, m, 8 * t + 4);
}

// Scores of a unit: sc[i][2h + x], tokens row + 16 i + 8 h, heads 2t + x.  One accumulator per (token half,
// group), four of them between dependent matrix steps.
template <int BITS, int GR, int bs, int IH>
__device__ __forceinline__ void score_unit(const uint8_t *kq, const uint8_t *kp, int row, int t, const Query<GR> &q, float (&sc)[IH][4])
{
    constexpr int GB = 8 * BITS;
    constexpr int KW = BITS / 2;
    uint32_t k0[IH][GR][KW], k1[IH][GR][KW];
    float d[IH][GR][4];
#pragma unroll
    for (int i = 0; i < IH; ++i)
#pragma unroll
        for (int c = 0; c < GR; ++c) {
            const uint8_t *p0 = kq + (c * bs + row + 16 * i) * GB + t * (GB / 4), *p1 = p0 + 8 * GB;
            if constexpr (BITS == 4) {
                const uint2 x0 = *reinterpret_cast<const uint2 *>(p0), x1 = *reinterpret_cast<const uint2 *>(p1);
                k0[i][c][0] = x0.x; k0[i][c][1] = x0.y;
                k1[i][c][0] = x1.x; k1[i][c][1] = x1.y;
            } else {
                const uint4 x0 = *reinterpret_cast<const uint4 *>(p0), x1 = *reinterpret_cast<const uint4 *>(p1);
                k0[i][c][0] = x0.x; k0[i][c][1] = x0.y; k0[i][c][2] = x0.z; k0[i][c][3] = x0.w;
                k1[i][c][0] = x1.x; k1[i][c][1] = x1.y; k1[i][c][2] = x1.z; k1[i][c][3] = x1.w;
            }
            d[i][c][0] = d[i][c][1] = d[i][c][2] = d[i][c][3] = 0.0f;
        }
#pragma unroll
    for (int x = 0; x < KW; ++x) {
#pragma unroll
        for (int odd = 0; odd < (BITS == 4 ? 2 : 1); ++odd) {
            const uint32_t M = BITS == 8 ? 0x00FF00FFu : odd ? 0x00F000F0u : 0x000F000Fu;
            const int j = BITS == 4 ? 2 * x + odd : x;
#pragma unroll
            for (int i = 0; i < IH; ++i)
#pragma unroll
                for (int c = 0; c < GR; ++c)
                    mma_f16(d[i][c], k0[i][c][x] & M, k1[i][c][x] & M, (k0[i][c][x] >> 8) & M, (k1[i][c][x] >> 8) & M,
                            q.b[c * 4 + j][0], q.b[c * 4 + j][1]);
        }
    }
#pragma unroll
    for (int i = 0; i < IH; ++i) {
        float *s4 = sc[i];
        s4[0] = s4[1] = s4[2] = s4[3] = 0.0f;
#pragma unroll
        for (int c = 0; c < GR; ++c) {
            const uint32_t w0 = *reinterpret_cast<const uint32_t *>(kp + (c * bs + row + 16 * i) * 4);
            const uint32_t w1 = *reinterpret_cast<const uint32_t *>(kp + (c * bs + row + 16 * i + 8) * 4);
            const float s0 = lo_bf16(w0), b0 = hi_bf16(w0), s1 = lo_bf16(w1), b1 = hi_bf16(w1);
            s4[0] = fmaf(b0, q.sum[c][0], fmaf(s0, d[i][c][0], s4[0]));
            s4[1] = fmaf(b0, q.sum[c][1], fmaf(s0, d[i][c][1], s4[1]));
            s4[2] = fmaf(b1, q.sum[c][0], fmaf(s1, d[i][c][2], s4[2]));
            s4[3] = fmaf(b1, q.sum[c][1], fmaf(s1, d[i][c][3], s4[3]));
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) s4[x] *= q.mul[x & 1];
    }
}

// Scale and bias of V, tokens row + 16 i + 8 h; `left` tokens of the unit exist (may be <= 0, or more than 32).  Rows
// behind the sequence have no weight, whatever they hold, and a scale (`idle`, or the one of the unit's first token) that moves no factor.
template <int GR, int bs, int IH>
__device__ __forceinline__ void load_scales(const uint8_t *vp, int row, int gi, int t, int left, uint32_t idle, uint32_t (&vw)[IH][GR][2], float (&sc)[IH][4])
{
#pragma unroll
    for (int i = 0; i < IH; ++i)
#pragma unroll
        for (int c = 0; c < GR; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                vw[i][c][h] = *reinterpret_cast<const uint32_t *>(vp + (c * bs + row + 16 * i + 8 * h) * 4);
    if (left < 16 * IH) {
        uint32_t first[GR];
#pragma unroll
        for (int c = 0; c < GR; ++c) first[c] = __shfl_sync(0xffffffffu, vw[0][c][0], t) & 0xFFFFu;
#pragma unroll
        for (int i = 0; i < IH; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (token_of(gi) + 16 * i + 8 * h >= left) {
                    sc[i][2 * h] = sc[i][2 * h + 1] = -INFINITY;
#pragma unroll
                    for (int c = 0; c < GR; ++c) vw[i][c][h] = left > 0 ? first[c] : idle;
                }
    }
}

// O^T += V^T P of 16 tokens (row0 the first one's, in the group's codes): the tokens on K, the weights in fp16, w0 the ones of the
// first eight tokens.
template <int BITS>
__device__ __forceinline__ void add_product(const uint8_t *vq, int row0, int gi, int t, uint32_t w0, uint32_t w1, float (&acc)[4][4])
{
    constexpr int GB = 8 * BITS;
    const uint32_t y0 = transpose8x8(w0), y1 = transpose8x8(w1);
    // lane: channels 8 gi .. 8 gi + 7 of the group, tokens t, t + 4, t + 8, t + 12
    const uint8_t *pv = vq + (row0 + t) * GB + gi * BITS;
    uint32_t v[4][2];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        if (BITS == 4) {
            v[r][0] = *reinterpret_cast<const uint32_t *>(pv + 4 * r * GB);
        } else {
            const uint2 x2 = *reinterpret_cast<const uint2 *>(pv + 4 * r * GB);
            v[r][0] = x2.x;
            v[r][1] = x2.y;
        }
    }
#pragma unroll
    for (int x = 0; x < BITS / 4; ++x) {
        const uint32_t za = __byte_perm(v[0][x], v[1][x], 0x5410), zb = __byte_perm(v[2][x], v[3][x], 0x5410);
        const uint32_t ya = __byte_perm(v[0][x], v[1][x], 0x7632), yb = __byte_perm(v[2][x], v[3][x], 0x7632);
        const uint32_t za8 = za >> 8, zb8 = zb >> 8, ya8 = ya >> 8, yb8 = yb >> 8;
        if (BITS == 4) {  // channels (0, 2), (1, 3), (4, 6), (5, 7)
            mma_f16(acc[0], za & 0x000F000Fu, za8 & 0x000F000Fu, zb & 0x000F000Fu, zb8 & 0x000F000Fu, y0, y1);
            mma_f16(acc[1], za & 0x00F000F0u, za8 & 0x00F000F0u, zb & 0x00F000F0u, zb8 & 0x00F000F0u, y0, y1);
            mma_f16(acc[2], ya & 0x000F000Fu, ya8 & 0x000F000Fu, yb & 0x000F000Fu, yb8 & 0x000F000Fu, y0, y1);
            mma_f16(acc[3], ya & 0x00F000F0u, ya8 & 0x00F000F0u, yb & 0x00F000F0u, yb8 & 0x00F000F0u, y0, y1);
        } else {          // channels (4x, 4x + 2), (4x + 1, 4x + 3)
            mma_f16(acc[2 * x], za & 0x00FF00FFu, ya & 0x00FF00FFu, zb & 0x00FF00FFu, yb & 0x00FF00FFu, y0, y1);
            mma_f16(acc[2 * x + 1], za8 & 0x00FF00FFu, ya8 & 0x00FF00FFu, zb8 & 0x00FF00FFu, yb8 & 0x00FF00FFu, y0, y1);
        }
    }
}

// (Without a split, one warp more in the launch bound than there are: the same 168 registers without 48 bytes of spills.)
template <int BITS, int GR, int bs>
__global__ void __launch_bounds__(threads_of(64 * GR) + (splits_registers(64 * GR) ? 0 : 32), 1) kvq_decode_kernel(const __grid_constant__ KvqAttnArgs a)
{
    constexpr int D = GR * 64, GB = 8 * BITS;  // bytes of a group's codes in one row
    extern __shared__ __align__(128) uint8_t base[];
    Fixed &F = *reinterpret_cast<Fixed *>(base);
    float *merge = reinterpret_cast<float *>(base + kFixed);  // [warp][head][merge_row]
    uint8_t *ring = base + kFixed + merge_bytes(D);
    constexpr int CB = GR * bs * GB, PB = GR * bs * 4, SB = 2 * (CB + PB);  // codes, parameters, stage
    constexpr int kUnit = unit_of(D), IH = kUnit / 16;
    // a warp's next unit is kNW units on: no further than the ring's length, so that when its stage has been issued, the
    // slot's last turn but one is over (the producers have waited for it)
    static_assert((kNW + bs / kUnit - 1) / (bs / kUnit) <= stages_for(D, bs, BITS), "ring too short");
    const int NS = a.stages, G = a.group;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gi = lane >> 2, t = lane & 3;
    int *status = &a.ctrl->status;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&F.full[i], 2);
            mbar_init(&F.empty[i], bs / kUnit);
        }
#ifdef LILY_TEST_STALL_T
        mbar_init(&F.never, 1);
#endif
        F.abort = 0;
        fence_mbar_init();
    }
    pdl_trigger();
    pdl_wait();
    __syncthreads();
    Walk w = first_segment<threads_of(D)>(a, F);

    if (warp >= kNW) {
        if constexpr (splits_registers(D)) {
            set_max_registers<kProducerRegs, false>();
            if (warp >= kNW + 2) return;
        }
        // ------------------------------------------------ producers: K, V (two, as issuing a copy takes ~130 cycles)
        const bool isv = warp > kNW;
        const uint8_t *codes = isv ? a.c.v_q : a.c.k_q;
        const uint16_t *params = isv ? a.c.v_sb : a.c.k_sb;
        uint8_t *dst0 = ring + (isv ? CB + PB : 0);
        int issued = 0, slot = 0;
        uint32_t turn = 0;  // of the ring, its parity
        bool ok = true, is_free = true;
        while (w.left > 0 && ok) {
            const int nblk = blocks_of(w.L, bs), n = min(nblk - w.j0, w.left);
            for (int i0 = 0; i0 < n && ok; i0 += 32) {
                int pb = 0;
                if (i0 + lane < n && w.L > 0) {
                    pb = a.block_table[static_cast<size_t>(w.b) * a.max_blocks + w.j0 + i0 + lane];
                    if (pb < 0 || pb >= a.c.n_blocks) {
                        record_error(status, kErrDeviceIndex);
                        pb = 0;
                    }
                }
                const long long row0 = (static_cast<long long>(pb) * a.c.H_kv + w.g) * (GR * bs);
                const int cnt = min(n - i0, 32);
                for (int i = 0; i < cnt; ++i) {
                    if (!__all_sync(0xffffffffu, is_free) && !(ok = warp_wait(&F.empty[slot], turn ^ 1u, &F.abort, status))) break;
                    const long long row = __shfl_sync(0xffffffffu, row0, i);
                    if (elect_one()) {
                        uint8_t *dst = dst0 + slot * SB;
                        mbar_arrive_expect_tx(&F.full[slot], static_cast<uint32_t>(CB + PB));
                        bulk_load(dst, codes + row * GB, CB, &F.full[slot]);
                        bulk_load(dst + CB, params + row * 2, PB, &F.full[slot]);
                    }
                    __syncwarp();
                    ++issued;
                    if (++slot == NS) {
                        slot = 0;
                        turn ^= 1u;
                    }
                    is_free = issued < NS || phase_done(&F.empty[slot], turn ^ 1u);  // looked at one stage ahead
                }
            }
            advance(a, w, n);
        }
        // no copy into this CTA's shared memory may still be in flight at exit
        const uint64_t t0 = global_timer_ns();
        for (int i = issued > NS ? issued - NS : 0; i < issued; ++i) {
            const uint32_t addr = smem_u32(&F.full[i % NS]);
            while (!mbar_try_wait(addr, (i / NS) & 1))
                if (global_timer_ns() - t0 > LILY_DRAIN_LIMIT_NS) {
                    record_error(status, kErrDeviceTimeout);
                    break;
                }
        }
        return;
    }

    // ---------------------------------------------------- consumers
    if constexpr (splits_registers(D)) set_max_registers<kConsumerRegs, true>();
    if (!a.whole && threadIdx.x == 0 && !a.key_by_segment && w.left == 0) a.meta[blockIdx.x] = make_int4(-1, 0, 0, 0);
    constexpr int ups = bs / kUnit;  // units per stage
    int unit = 0, stage0 = 0, bar = 0;  // units and stages of the segments before this one; named barrier
    bool ok = true;
    while (w.left > 0) {
        const int nblk = blocks_of(w.L, bs), n = min(nblk - w.j0, w.left);
        const int tok0 = w.j0 * bs, units = n * ups;
        // the units are dealt to the warps in turn; a warp that gets none of this segment goes on to the next one,
        // so short segments are worked on side by side
        const int first = (warp - unit % kNW + kNW) % kNW, active = min(units, kNW);
        if (first >= units) {
            unit += units;
            stage0 += n;
            bar = (bar + 1) % kBarriers;
            advance(a, w, n);
            continue;
        }

        Query<GR> q;
        load_query<BITS>(a, w, gi, t, q);
        float acc[GR][4][4], bsum[GR][2], m_run[2] = {kNoMax, kNoMax}, l_run[2] = {0.0f, 0.0f}, f = kMaxFactor;
#pragma unroll
        for (int c = 0; c < GR; ++c) {
            bsum[c][0] = bsum[c][1] = 0.0f;
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int x = 0; x < 4; ++x) acc[c][m][x] = 0.0f;
        }

#ifdef LILY_TEST_STALL_T
        // Test builds only: with that many sequences the first CTA's first unit waits for a barrier that nothing completes, so
        // that the wait runs out and every role gives up.
        if (a.N == LILY_TEST_STALL_T && blockIdx.x == 0 && unit + first == 0) ok = warp_wait(&F.never, 0, &F.abort, status);
#endif
        bool apart = false;
        // the second loop's factors, in the padding of the warp's rows: of head 2t + x and group c own[x * merge_row(D) + c]
        float *own = merge + (warp * 8 + 2 * t) * merge_row(D) + D;
        int u = first;
        for (; u < units; u += kNW) {
            const int st = stage0 + u / ups, turn = __umulhi(st, a.stages_inv), slot = st - turn * NS, r0 = (u % ups) * kUnit;
            // A warp meets a slot only in some of its turns, and copies land in any order: the slot's last turn has to be
            // over first, or `full` of the turn before, still open, has the parity of this one done.
            // Both are looked at in this order, without waiting in between.
            const uint32_t over = turn == 0 ? 1u : phase_done(&F.empty[slot], (turn - 1) & 1), here = phase_done(&F.full[slot], turn & 1);
            if (!ok || !__all_sync(0xffffffffu, over & here)) {
                ok = ok && (turn == 0 || mbar_wait(&F.empty[slot], (turn - 1) & 1, &F.abort, status)) &&
                     mbar_wait(&F.full[slot], turn & 1, &F.abort, status);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
            }
            const uint8_t *kq = ring + static_cast<size_t>(slot) * SB, *kp = kq + CB, *vq = kp + PB, *vp = vq + CB;
            const int left = w.L - (tok0 + u * kUnit);  // tokens of this unit that exist (may be <= 0, or more than 32)
            const int row = r0 + token_of(gi);          // + 16 i + 8 h: this lane's token rows of S^T

            float sc[IH][4];
            score_unit<BITS, GR, bs>(kq, kp, row, t, q, sc);
            uint32_t vw[IH][GR][2];
            load_scales<GR, bs>(vp, row, gi, t, left, ((254u + kLift) << 7) - (__float_as_uint(f) >> 16), vw, sc);

            // ---- running maximum, and the power of two of the value scales: both move rarely
            float top0 = fmaxf(sc[0][0], sc[0][2]), top1 = fmaxf(sc[0][1], sc[0][3]), smax = 0.0f, smin = INFINITY;
            if constexpr (IH == 2) {
                top0 = fmaxf(top0, fmaxf(sc[IH - 1][0], sc[IH - 1][2]));
                top1 = fmaxf(top1, fmaxf(sc[IH - 1][1], sc[IH - 1][3]));
            }
#pragma unroll
            for (int i = 0; i < IH; ++i)
#pragma unroll
                for (int c = 0; c < GR; ++c) {
                    const float s0 = fabsf(lo_bf16(vw[i][c][0])), s1 = fabsf(lo_bf16(vw[i][c][1]));
                    smax = fmaxf(smax, fmaxf(s0, s1));
                    smin = fminf(smin, fminf(s0, s1));
                }
            const bool grew = top0 > m_run[0] + (8.0f - kLift) || top1 > m_run[1] + (8.0f - kLift);
            if (__any_sync(0xffffffffu, grew || smax * f > kHigh || smin * f < kLow)) {
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    smax = fmaxf(smax, __shfl_xor_sync(0xffffffffu, smax, o));
                    smin = fminf(smin, __shfl_xor_sync(0xffffffffu, smin, o));
                }
                float to = f;
                if (smax * f > kHigh) {  // f smax back into [kHigh / 2, kHigh)
                    const int ex = min(max(260 + kLift - static_cast<int>(__float_as_uint(smax) >> 23), 1), 127 + kMaxFactorLog);
                    to = __uint_as_float(static_cast<uint32_t>(ex) << 23);
                }
                if (smin * to < kLow || (to < f * 0x1p-8f && f < kMaxFactor)) {
                    apart = true;
                    break;
                }
                float mn0 = top0, mn1 = top1;
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {
                    mn0 = fmaxf(mn0, __shfl_xor_sync(0xffffffffu, mn0, o));
                    mn1 = fmaxf(mn1, __shfl_xor_sync(0xffffffffu, mn1, o));
                }
                mn0 = fmaxf(mn0 + kLift, m_run[0]);
                mn1 = fmaxf(mn1 + kLift, m_run[1]);
                const float r = to < f ? to * (1.0f / f) : 1.0f, al0 = ex2(m_run[0] - mn0), al1 = ex2(m_run[1] - mn1);
                f = to;
                m_run[0] = mn0;
                m_run[1] = mn1;
                l_run[0] *= al0;
                l_run[1] *= al1;
#pragma unroll
                for (int c = 0; c < GR; ++c) {
                    bsum[c][0] *= al0;
                    bsum[c][1] *= al1;
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        acc[c][m][0] = acc[c][m][0] * al0 * r;
                        acc[c][m][1] = acc[c][m][1] * al1 * r;
                        acc[c][m][2] = acc[c][m][2] * al0 * r;
                        acc[c][m][3] = acc[c][m][3] * al1 * r;
                    }
                }
            }

            // ---- O^T += V^T P: weights p s f in fp16, tokens on K
#pragma unroll
            for (int i = 0; i < IH; ++i) {
                float p[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) p[x] = ex2(sc[i][x] - m_run[x & 1]);
                l_run[0] += p[0] + p[2];
                l_run[1] += p[1] + p[3];
                const float pf[4] = {p[0] * f, p[1] * f, p[2] * f, p[3] * f};
#pragma unroll
                for (int c = 0; c < GR; ++c) {
                    const uint32_t w0 = vw[i][c][0], w1 = vw[i][c][1];
                    const float s0 = lo_bf16(w0), b0 = hi_bf16(w0), s1 = lo_bf16(w1), b1 = hi_bf16(w1);
                    bsum[c][0] = fmaf(p[0], b0, fmaf(p[2], b1, bsum[c][0]));
                    bsum[c][1] = fmaf(p[1], b0, fmaf(p[3], b1, bsum[c][1]));
                    add_product<BITS>(vq, c * bs + r0 + 16 * i, gi, t, pack_f16(pf[0] * s0, pf[1] * s0), pack_f16(pf[2] * s1, pf[3] * s1), acc[c]);
                }
            }
            // the last one is given back after the join: no segment then meets another that has its named barrier
            __syncwarp();
            if (lane == 0 && u + kNW < units) mbar_arrive(&F.empty[slot]);
        }

        // ---- the units from u on, where scales do not lie within 2^8 of each other (or are 0): a factor for each head and group,
        // which follows the largest p s of that head and group, so that a token without weight in a head, and another
        // group, take no bits from it
        if (apart) {
            if (gi == 0) {
#pragma unroll
                for (int c = 0; c < GR; ++c) own[c] = own[merge_row(D) + c] = f;
            }
#pragma unroll 1
            for (; u < units; u += kNW) {
                const int st = stage0 + u / ups, turn = __umulhi(st, a.stages_inv), slot = st - turn * NS, r0 = (u % ups) * kUnit;
                ok = ok && (turn == 0 || mbar_wait(&F.empty[slot], (turn - 1) & 1, &F.abort, status)) &&
                     mbar_wait(&F.full[slot], turn & 1, &F.abort, status);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const uint8_t *kq = ring + static_cast<size_t>(slot) * SB, *kp = kq + CB, *vq = kp + PB, *vp = vq + CB;
                const int row = r0 + token_of(gi);
                float sc[IH][4], rise[2];
                uint32_t vw[IH][GR][2];
                score_unit<BITS, GR, bs>(kq, kp, row, t, q, sc);
                load_scales<GR, bs>(vp, row, gi, t, w.L - (tok0 + u * kUnit), 0u, vw, sc);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float mn = fmaxf(sc[0][x], sc[0][x + 2]);
                    if constexpr (IH == 2) mn = fmaxf(mn, fmaxf(sc[IH - 1][x], sc[IH - 1][x + 2]));
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
                    mn = fmaxf(mn + kLift, m_run[x]);
                    rise[x] = mn - m_run[x];
                    m_run[x] = mn;
                    l_run[x] *= ex2(-rise[x]);
                }
#pragma unroll
                for (int i = 0; i < IH; ++i)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        sc[i][x] = ex2(sc[i][x] - m_run[x & 1]);
                        l_run[x & 1] += sc[i][x];
                    }
#pragma unroll
                for (int c = 0; c < GR; ++c) {
                    float fc[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float al = ex2(-rise[x]);
                        float big = 0.0f;
                        bsum[c][x] *= al;
#pragma unroll
                        for (int i = 0; i < IH; ++i)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                bsum[c][x] = fmaf(sc[i][2 * h + x], hi_bf16(vw[i][c][h]), bsum[c][x]);
                                big = fmaxf(big, sc[i][2 * h + x] * fabsf(lo_bf16(vw[i][c][h])));
                            }
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
                        // What went in before weighs 2^-rise of what it did, and the factor goes up by as much; then it comes
                        // down to bring the largest p s f of this unit into [64, 128) where that would reach 2^15.
                        __syncwarp();
                        const int was = static_cast<int>(__float_as_uint(own[x * merge_row(D) + c]) >> 23), e = static_cast<int>(__float_as_uint(big) >> 23);
                        int now = min(was + static_cast<int>(fminf(rise[x], 256.0f)), 127 + kMaxFactorLog);
                        if (e + now >= 254 + 15) now = 254 + 6 - e;
                        fc[x] = __uint_as_float(static_cast<uint32_t>(now) << 23);
                        __syncwarp();
                        if (gi == 0) own[x * merge_row(D) + c] = fc[x];
                        // O times 2^(now - was - rise), in two steps as the power of two alone may be no number
                        const int half = (now - was) / 2;
                        const float r0 = __uint_as_float(static_cast<uint32_t>(127 + half) << 23);
                        const float r1 = __uint_as_float(static_cast<uint32_t>(127 + (now - was) - half) << 23) * al;
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            acc[c][m][x] = acc[c][m][x] * r0 * r1;
                            acc[c][m][x + 2] = acc[c][m][x + 2] * r0 * r1;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < IH; ++i) {
                        const float s0 = lo_bf16(vw[i][c][0]), s1 = lo_bf16(vw[i][c][1]);
                        add_product<BITS>(vq, c * bs + r0 + 16 * i, gi, t, pack_f16(sc[i][0] * s0 * fc[0], sc[i][1] * s0 * fc[1]),
                                          pack_f16(sc[i][2] * s1 * fc[0], sc[i][3] * s1 * fc[1]), acc[c]);
                    }
                }
                __syncwarp();
                if (lane == 0 && u + kNW < units) mbar_arrive(&F.empty[slot]);
            }
            __syncwarp();
        }

        // ---- the segment's end: this warp's sums over its lanes, then the warps through shared memory
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                l_run[x] += __shfl_xor_sync(0xffffffffu, l_run[x], o);
#pragma unroll
                for (int c = 0; c < GR; ++c) bsum[c][x] += __shfl_xor_sync(0xffffffffu, bsum[c][x], o);
            }
        }
        float rf[GR][2];  // 1 / f, a power of two
#pragma unroll
        for (int c = 0; c < GR; ++c)
#pragma unroll
            for (int x = 0; x < 2; ++x) rf[c][x] = __uint_as_float((254u << 23) - __float_as_uint(apart ? own[x * merge_row(D) + c] : f));
        const bool starts = w.j0 == 0, ends = w.j0 + n == nblk;
        const int part = 2 * blockIdx.x + (starts ? 1 : 0);
        auto join_sync = [&]() {
            if (active > 1)
                named_barrier_sync(1 + bar, active * 32);
            else
                __syncwarp();
        };
        if (gi == 0) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                F.ml[warp][2 * t + x][0] = m_run[x];
                F.ml[warp][2 * t + x][1] = l_run[x];
            }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            float *dst = merge + (warp * 8 + 2 * t + x) * merge_row(D) + gi * 8;
#pragma unroll
            for (int c = 0; c < GR; ++c) {
                auto out = [&](int m, int h) {
                    const float unit_scale = BITS == 4 && (m & 1) ? 0x1p20f : 0x1p24f;
                    return fmaf(acc[c][m][2 * h + x] * unit_scale, rf[c][x], bsum[c][x]);
                };
                *reinterpret_cast<float4 *>(dst + c * 64) = make_float4(out(0, 0), out(1, 0), out(0, 1), out(1, 1));
                *reinterpret_cast<float4 *>(dst + c * 64 + 4) = make_float4(out(2, 0), out(3, 0), out(2, 1), out(3, 1));
            }
        }
        join_sync();
        for (int i = first * 32 + lane; i < G * (D / 4); i += active * 32)
            join_column<D>(a, F, merge, w, unit, active, starts && ends ? -1 : part, i / (D / 4), i % (D / 4));
        if (!a.whole && first == 0 && lane == 0 && (a.key_by_segment ? starts : w.left == n)) {
            // who joins the parts: the CTAs from this one to the one that has the segment's last block
            const int bg = w.b * a.c.H_kv + w.g;
            const int last = static_cast<int>((static_cast<long long>(F.begin + stage0 - w.j0 + nblk) * F.used - 1) / F.total);
            a.meta[a.key_by_segment ? bg : blockIdx.x] = make_int4(starts && !ends ? bg : -1, blockIdx.x, last, 0);
        }
        unit += units;
        join_sync();
        if (lane == 0 && ok) mbar_arrive(&F.empty[(stage0 + (units - 1 - (units - 1 - first) % kNW) / ups) % NS]);
        stage0 += n;
        advance(a, w, n);
        bar = (bar + 1) % kBarriers;
    }
}

// Joins the parts of a segment that was cut: CTA (segment key x head, slice of kCols
// float4 columns of D), 256 threads: thread (e, sg) takes column e and parts sg,
// sg + kGroups, .. on a running maximum of its own; the part groups are joined by
// shuffles where a warp has several, then through shared memory, in a fixed order.  Parts
// of CTA c0 (the one the segment starts in) are in slot 2 c0 + 1, those of the following
// CTAs c in slot 2 c, up to the CTA it ends in.
template <int kCols>
__global__ void __launch_bounds__(256) kvq_combine_kernel(const __grid_constant__ KvqAttnArgs a)
{
    constexpr int kGroups = 256 / kCols, kBatch = 4, kRuns = kCols < 32 ? 8 : kGroups;  // kRuns: results in shared memory
    __shared__ float4 part[kRuns][kCols];
    __shared__ float part_m[kRuns], part_den[kRuns];
    const int key = blockIdx.x / a.group, h = blockIdx.x % a.group;
    const int tid = threadIdx.x, e = tid % kCols, sg = tid / kCols;
    pdl_trigger();
    pdl_wait();
    const int4 meta = a.meta[key];
    if (meta.x < 0) return;
    const int c0 = meta.y, S = meta.z - c0 + 1, q = blockIdx.y * kCols + e;
    auto slot = [&](int s) { return static_cast<size_t>(s == 0 ? 2 * c0 + 1 : 2 * (c0 + s)) * 8 + h; };
    float mt = kNoMax, den = 0.0f;
    float4 num = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto scale_by = [&](float c) {
        num.x *= c;
        num.y *= c;
        num.z *= c;
        num.w *= c;
        den *= c;
    };
    for (int s0 = sg; s0 < S; s0 += kBatch * kGroups) {
        float4 v[kBatch];
        float2 ml[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int s = s0 + k * kGroups;
            ml[k] = s < S ? *reinterpret_cast<const float2 *>(a.part_ml + slot(s) * 2) : make_float2(kNoMax, 0.0f);
            v[k] = s < S ? reinterpret_cast<const float4 *>(a.part_acc + slot(s) * a.D)[q] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float bm = mt;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) bm = fmaxf(bm, ml[k].x);
        scale_by(ex2(mt - bm));
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const float w = ex2(ml[k].x - bm);
            num.x = fmaf(w, v[k].x, num.x);
            num.y = fmaf(w, v[k].y, num.y);
            num.z = fmaf(w, v[k].z, num.z);
            num.w = fmaf(w, v[k].w, num.w);
            den = fmaf(w, ml[k].y, den);
        }
        mt = bm;
    }
    float mw = mt;
#pragma unroll
    for (int o = kCols; o < 32; o <<= 1) mw = fmaxf(mw, __shfl_xor_sync(0xffffffffu, mw, o));
    scale_by(ex2(mt - mw));
#pragma unroll
    for (int o = kCols; o < 32; o <<= 1) {
        num.x += __shfl_xor_sync(0xffffffffu, num.x, o);
        num.y += __shfl_xor_sync(0xffffffffu, num.y, o);
        num.z += __shfl_xor_sync(0xffffffffu, num.z, o);
        num.w += __shfl_xor_sync(0xffffffffu, num.w, o);
        den += __shfl_xor_sync(0xffffffffu, den, o);
    }
    const int run = kCols < 32 ? tid / 32 : sg;
    if (kCols >= 32 || (tid & 31) < kCols) part[run][e] = num;
    if (e == 0 && (kCols >= 32 || (tid & 31) == 0)) {
        part_m[run] = mw;
        part_den[run] = den;
    }
    __syncthreads();
    if (tid < kCols) {
        float mx = part_m[0];
#pragma unroll
        for (int w = 1; w < kRuns; ++w) mx = fmaxf(mx, part_m[w]);
        float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float dsum = 0.0f;
#pragma unroll
        for (int w = 0; w < kRuns; ++w) {
            const float f = ex2(part_m[w] - mx);
            const float4 x = part[w][tid];
            t.x = fmaf(f, x.x, t.x);
            t.y = fmaf(f, x.y, t.y);
            t.z = fmaf(f, x.z, t.z);
            t.w = fmaf(f, x.w, t.w);
            dsum = fmaf(f, part_den[w], dsum);
        }
        const float r = dsum > 0.0f ? 1.0f / dsum : 0.0f;
        uint2 y;
        const __nv_bfloat162 lo = __floats2bfloat162_rn(t.x * r, t.y * r), hi = __floats2bfloat162_rn(t.z * r, t.w * r);
        y.x = *reinterpret_cast<const uint32_t *>(&lo);
        y.y = *reinterpret_cast<const uint32_t *>(&hi);
        const int b = meta.x / a.c.H_kv, g = meta.x % a.c.H_kv;
        reinterpret_cast<uint2 *>(a.out + (static_cast<size_t>(b) * a.H_q + g * a.group + h) * a.D)[q] = y;
    }
}

template <int BITS, int GR, int bs>
cudaError_t launch(const KvqAttnArgs &a, int ctas, cudaStream_t stream)
{
    constexpr int NT = threads_of(64 * GR);
    const size_t smem = kFixed + merge_bytes(64 * GR) + static_cast<size_t>(a.stages) * stage_bytes(64 * GR, bs, BITS);
    const void *kernel = reinterpret_cast<const void *>(kvq_decode_kernel<BITS, GR, bs>);
    const cudaError_t e = set_max_dynamic_smem(kernel, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    if constexpr (splits_registers(64 * GR)) {
        // the consumers' share has to be there, or they would wait for it without end
        static const bool fits = [kernel] {
            cudaFuncAttributes at;
            return cudaFuncGetAttributes(&at, kernel) == cudaSuccess && at.numRegs * NT >= (kConsumerRegs * kNW + kProducerRegs * 4) * 32;
        }();
        if (!fits) return cudaErrorLaunchOutOfResources;
    }
    return launch_pdl(kvq_decode_kernel<BITS, GR, bs>, dim3(ctas), dim3(NT), smem, stream, a);
}
template <int BITS, int GR>
cudaError_t launch_bs(const KvqAttnArgs &a, int ctas, cudaStream_t stream)
{
    return a.c.bs == 32 ? launch<BITS, GR, 32>(a, ctas, stream) : a.c.bs == 64 ? launch<BITS, GR, 64>(a, ctas, stream) : launch<BITS, GR, 128>(a, ctas, stream);
}
template <int BITS>
cudaError_t launch_d(const KvqAttnArgs &a, int ctas, cudaStream_t stream)
{
    return a.D == 64 ? launch_bs<BITS, 1>(a, ctas, stream) : a.D == 128 ? launch_bs<BITS, 2>(a, ctas, stream) : launch_bs<BITS, 4>(a, ctas, stream);
}

}  // namespace

// A CTA for each segment, and no join, where no CTA then has much more than an even share
// of a full cache (by the table's width, as the lengths are on the device: short sequences under a wide
// table take the cut form): with n segments on 152 CTAs, where capacity (1 - n / 152) is at most 640
// tokens, which cost what cutting and joining does.  Measured, one CTA each against cut (2
// KV heads of 256): one sequence of 256 tokens 6.2 / 7.9 us, of 512 8.2 / 7.9, of 1,024
// 11.8 / 8.1; 64 sequences of 1,024 13.9 / 21.0.  (4 heads of 128: one of 512 tokens 5.6 /
// 6.6, 16 of 256 4.6 / 7.5.)  Above 1,024 tokens the lengths of a batch can differ too much
// from its capacity.
bool one_cta_each(long long segments, long long capacity)
{
    return segments <= kKvqDecodeCtas && capacity <= 1024 && capacity * (kKvqDecodeCtas - segments) <= 640LL * kKvqDecodeCtas;
}
// Segments from which the join takes all of D in a CTA.  Below, slices of 32 channels: a
// segment then has up to 152 parts (two segments of 32,768 tokens, slices 14.1 us, all of
// D 19.4); above, the slices are thousands of CTAs (128 segments of 1,024 tokens: 36 us,
// 22).  At 8 segments slices are ahead by 0.7 us, at 16 all of D is by 0.7.
constexpr int kJoinWhole = 16;

cudaError_t launch_kvq_decode(const KvqAttnArgs &args, cudaStream_t stream)
{
    KvqAttnArgs a = args;
    const long long segments = static_cast<long long>(a.B) * a.c.H_kv;
    a.whole = one_cta_each(segments, static_cast<long long>(a.max_blocks) * a.c.bs);
    a.key_by_segment = segments <= kKvqDecodeCtas;
    a.stages = stages_for(a.D, a.c.bs, a.c.bits);
    a.stages_inv = 0xFFFFFFFFu / a.stages + 1;  // x / stages = the high word of x stages_inv for x < 2^32 / stages
    const int ctas = a.whole ? static_cast<int>(segments) : kKvqDecodeCtas;
    const cudaError_t e = a.c.bits == 4 ? launch_d<4>(a, ctas, stream) : launch_d<8>(a, ctas, stream);
    if (e != cudaSuccess || a.whole) return e;
    const int keys = a.key_by_segment ? static_cast<int>(segments) : ctas;
    if (keys < kJoinWhole || a.D == 64) return launch_pdl(kvq_combine_kernel<8>, dim3(keys * a.group, a.D / 32), dim3(256), 0, stream, a);
    return a.D == 128 ? launch_pdl(kvq_combine_kernel<32>, dim3(keys * a.group), dim3(256), 0, stream, a)
                      : launch_pdl(kvq_combine_kernel<64>, dim3(keys * a.group), dim3(256), 0, stream, a);
}

}  // namespace lily
