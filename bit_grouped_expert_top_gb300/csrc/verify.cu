// Verification of drafted tokens against the target's probabilities, for sm_103a.
//
// Draft i of a sequence is accepted while u_i q_i(x_i) < p_i(x_i); after the first refusal
// one token is drawn from max(p - q, 0), after none from p: the smallest v with
//   sum_{w <= v} weight_w > r * sum_w weight_w.
// Sums over a vocabulary are taken in 64-bit fixed point (units of 2^-62, probabilities
// at most 1 and a row's sum below 4): integer sums are the same in any order, so the token
// does not depend on how a row is split, and u q < p is compared in fp64, where the
// product of two fp32 numbers is exact.
//
// Bound: latency (the acceptance is a chain of three dependent loads), then HBM: only the
// two rows that the next token is drawn from are read.  A cluster of up to eight CTAs takes one
// sequence; a warp sums one contiguous span of the row, the totals meet in distributed
// shared memory, and the CTA that holds the threshold looks through that one span again (from L2).
#include <cstdint>
#include <utility>

#include <cooperative_groups.h>

#include "lily_internal.h"

namespace lily {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxRanks = 8;
using u64 = unsigned long long;

// p in [0, 1] in units of 2^-62, rounded down (exact from 2^-38 on); 0 for NaN and below 0, 1 above 1.  With e
// the exponent's bits and m the 24-bit mantissa it is (m << 39) >> (127 - e): two words, by shifts that give 0 from 32 on.
__device__ __forceinline__ u64 fixed62(float p)
{
    const uint32_t bits = __float_as_uint(fminf(fmaxf(p, 0.0f), 1.0f));
    const uint32_t m = (bits & 0x7FFFFFu | 0x800000u) << 7, k = 127 - (bits >> 23);  // subnormals are far below 2^-62: 0 all the same
    uint32_t hi, lo, low;
    asm("shr.u32 %0, %1, %2;" : "=r"(hi) : "r"(m), "r"(k));
    asm("shl.b32 %0, %1, %2;" : "=r"(lo) : "r"(m), "r"(32 - k));
    asm("shr.u32 %0, %1, %2;" : "=r"(low) : "r"(m), "r"(k - 32));
    return static_cast<u64>(hi) << 32 | lo | low;
}

// r in [0, 1) in units of 2^-64 (values outside: the nearest).
__device__ __forceinline__ u64 fixed64(float r)
{
    if (!(r > 0.0f)) return 0;
    if (r >= 1.0f) return ~0ull;
    const uint32_t bits = __float_as_uint(r);
    const int e = static_cast<int>(bits >> 23);
    const u64 m = (bits & 0x7FFFFFu) | 0x800000u;
    return e >= 86 ? m << (e - 86) : e >= 62 ? m >> (86 - e) : 0;
}

__device__ __forceinline__ u64 warp_sum(u64 v)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum over the lanes up to this one.
__device__ __forceinline__ u64 warp_scan(u64 v, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 t = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += t;
    }
    return v;
}

// Weight of token v: max(p - q, 0), or p where there is no q; `gone` has none.
struct Row {
    const float *p, *q;
    int gone;
    static __device__ __forceinline__ u64 above(float pv, float qv)
    {
        const u64 a = fixed62(pv), b = fixed62(qv);
        return a > b ? a - b : 0;
    }
    __device__ __forceinline__ u64 operator()(int v) const
    {
        if (q) return above(p[v], q[v]);
        return v == gone ? 0 : fixed62(p[v]);
    }
};

// fixed62() by additions: p + 2, cut to the 2^-22 that its last bit is there, leaves 22 bits of p in the low bits of the pattern;
// the rest, times 2^22 and then 2^40, 22 and 18 more.  (Half as many cycles as the shifts: fp32 additions have twice the rate
// of integer shifts.)
struct Pieces {
    uint32_t a, b, c;
};

__device__ __forceinline__ Pieces pieces(float p)  // p in [0, 1]
{
    const float a = __fadd_rz(p, 2.0f), r = p - (a - 2.0f);
    const float b = __fmaf_rz(r, 0x1p22f, 2.0f), s = fmaf(b - 2.0f, -0x1p-22f, r);
    const float c = __fmaf_rz(s, 0x1p40f, 2.0f);
    return {__float_as_uint(a), __float_as_uint(b), __float_as_uint(c)};
}

// A 32-bit number, negative ones as they are modulo 2^64.
__device__ __forceinline__ u64 signed64(uint32_t v) { return static_cast<u64>(static_cast<long long>(static_cast<int>(v))); }

// A lane's part of the weights of [v0, v1): every 32nd, UNROLL loads of each row in flight.  (`gone` is taken off elsewhere.)
template <int UNROLL, bool Q>
__device__ __forceinline__ u64 lane_sum(const Row &row, int v0, int v1, int lane)
{
    // The patterns' own 2^30 vanishes where a multiple of four of them is added in 32 bits, zeros past the end among them.
    static_assert(Q || UNROLL % 4 == 0, "");
    u64 sum = 0;
    for (int v = v0 + lane; v < v1; v += 32 * UNROLL) {
        float pv[UNROLL], qv[UNROLL];
#pragma unroll
        for (int j = 0; j < UNROLL; ++j) {
            const bool on = v + 32 * j < v1;
            pv[j] = on ? row.p[v + 32 * j] : 0.0f;
            if (Q) qv[j] = on ? row.q[v + 32 * j] : 0.0f;
        }
        uint32_t a = 0, b = 0, c = 0;  // modulo 2^32: UNROLL numbers of at most 2^22, or differences of them
#pragma unroll
        for (int j = 0; j < UNROLL; ++j) {
            const float ps = __saturatef(pv[j]);  // 0 for NaN
            const Pieces p = pieces(ps);
            if (Q) {
                const float qs = __saturatef(qv[j]);
                const Pieces q = pieces(qs);
                if (ps > qs) {
                    a += p.a - q.a;
                    b += p.b - q.b;
                    c += p.c - q.c;
                }
            } else {
                a += p.a;
                b += p.b;
                c += p.c;
            }
        }
        sum += (signed64(a) << 40) + (signed64(b) << 18) + signed64(c);
    }
    return sum;
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS, 1)
    verify_kernel(const __grid_constant__ VerifyArgs a)
{
    constexpr int kWarps = THREADS / 32;
    __shared__ int first_refused;
    __shared__ u64 span_sum[32], scan_s[32], total_s[2];
    pdl_trigger();
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = a.ranks, rank = static_cast<int>(cluster.block_rank()), b = blockIdx.x / ranks, tid = threadIdx.x;
    const int warp = tid / 32, lane = tid % 32;
    if (tid == 0) first_refused = 0x7FFFFFFF;
    if (tid < 32) span_sum[tid] = scan_s[tid] = 0;
    __syncthreads();
    pdl_wait();

    const int c0 = a.cu[b], c1 = a.cu[b + 1], m = c1 - c0;
    const float r = a.r[b];
    if (c0 < 0 || c1 < c0 || c1 > a.N) {  // all CTAs of the cluster agree
        if (tid == 0) record_error(&a.ctrl->status, kErrDeviceIndex);
        return;
    }
    for (int i = tid; i < m; i += THREADS) {
        const int x = a.drafts[c0 + i];
        const float u = a.u[c0 + i];
        bool ok = false;
        if (x < 0 || x >= a.V) {
            record_error(&a.ctrl->status, kErrDeviceIndex);
        } else {
            const double px = __saturatef(a.p[(static_cast<long long>(c0) + b + i) * a.p_stride + x]);
            const double qx = a.q ? __saturatef(a.q[(static_cast<long long>(c0) + i) * a.q_stride + x]) : 1.0f;
            ok = static_cast<double>(u) * qx < px;
        }
        if (!ok) atomicMin(&first_refused, i);
    }
    __syncthreads();
    const int n = min(first_refused, m);
    const bool refused = n < m;
    if (rank == 0 && tid == 0) a.tokens[c0 + b + n] = -1;  // stays where no weight is; ahead of the cluster's barrier, behind which the token comes
    Row row;
    row.p = a.p + (static_cast<long long>(c0) + b + n) * a.p_stride;
    row.q = refused && a.q ? a.q + (static_cast<long long>(c0) + n) * a.q_stride : nullptr;
    row.gone = refused && !a.q ? a.drafts[c0 + n] : -1;
    // the warp's span: [V s / S, V (s + 1) / S) of S = ranks kWarps
    auto bound = [&](int i) { return static_cast<int>(static_cast<long long>(a.V) * i / (ranks * kWarps)); };
    const int s = rank * kWarps + warp, v0 = bound(s), v1 = bound(s + 1);
    u64 total = 0, before = 0;
    for (int pass = 0; pass < 2; ++pass) {
        u64 sum = warp_sum(row.q ? lane_sum<8, true>(row, v0, v1, lane) : lane_sum<16, false>(row, v0, v1, lane));
        if (row.gone >= v0 && row.gone < v1) sum -= fixed62(row.p[row.gone]);
        if (lane == 0) span_sum[warp] = sum;
        __syncthreads();
        if (warp == 0) {
            const u64 t = warp_sum(span_sum[lane]);
            if (lane == 0) total_s[pass] = t;
        }
        cluster.sync();
        total = before = 0;
#pragma unroll
        for (int k = 0; k < kMaxRanks; ++k) {
            if (k >= ranks) break;
            const u64 t = cluster.map_shared_rank(total_s, k)[pass];
            if (k < rank) before += t;
            total += t;
        }
        if (total || (!row.q && row.gone < 0)) break;
        // p nowhere above q (as sums that are rounded can give): the token comes from p itself
        row.q = nullptr;
        row.gone = -1;
    }
    auto done = cluster.barrier_arrive();  // nobody leaves while another reads
    if (rank == 0) {
        if (tid == 0) a.accepted[b] = n;
        for (int i = tid; i <= m; i += THREADS)
            if (i != n) a.tokens[c0 + b + i] = i < n ? a.drafts[c0 + i] : -1;
        if (total == 0 && tid == 0) record_error(&a.ctrl->status, kErrDeviceRange);
    }
    // the token is the first whose running sum passes `below`; the CTA that has it looks through its warp's span again, a
    // contiguous piece for each thread
    const u64 below = __umul64hi(total, fixed64(r));
    const u64 upto = warp_scan(span_sum[lane], lane);
    const unsigned passed = __ballot_sync(0xffffffffu, before <= below && below - before < upto);
    if (total && passed) {
        const int w = __ffs(passed) - 1;
        before += w ? __shfl_sync(0xffffffffu, upto, w - 1) : 0;
        const int u0 = bound(rank * kWarps + w), u1 = bound(rank * kWarps + w + 1);
        const int each = (u1 - u0 + THREADS - 1) / THREADS;
        const int a0 = min(u0 + tid * each, u1), a1 = min(a0 + each, u1);
        u64 mine = 0;
        for (int v = a0; v < a1; ++v) mine += row(v);
        const u64 in_warp = warp_scan(mine, lane);
        if (lane == 31) scan_s[warp] = in_warp;
        __syncthreads();
        before += warp_sum(lane < warp ? scan_s[lane] : 0) + in_warp - mine;
        if (below >= before && below - before < mine) {
            for (int v = a0; v < a1; ++v) {
                before += row(v);
                if (before > below) {
                    a.tokens[c0 + b + n] = v;
                    break;
                }
            }
        }
    }
    cluster.barrier_wait(std::move(done));
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs &args, int num_sms, cudaStream_t stream)
{
    VerifyArgs a = args;
    // One wave of CTAs (a CTA's time is a chain of loads and barriers, and clusters leave gaps between waves: 200 sequences of 20,000
    // tokens take 18.4 us with one CTA each, 25.1 with two, 75.4 with eight), in as many as that allows (64 of 131,072 13.7 with two, 16.7 with one).
    for (a.ranks = kMaxRanks; a.ranks > 1 && a.B * a.ranks > num_sms;) a.ranks /= 2;
    // twice the threads for a CTA's part of a long row (64 rows of 131,072 in two parts 13.7 us against 14.7; 200 of 20,000 in one
    // 19.2 against 18.4; eight of 100,003 in eight parts 10.1 against 10.3)
    const bool wide = a.V / a.ranks >= 32768;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(a.B * a.ranks);
    cfg.blockDim = dim3(wide ? 1024 : 512);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.ranks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.ranks > 1 ? 2 : 1;
    return wide ? cudaLaunchKernelEx(&cfg, verify_kernel<1024>, a) : cudaLaunchKernelEx(&cfg, verify_kernel<512>, a);
}

}  // namespace lily
