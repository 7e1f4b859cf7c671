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
// two rows that the next token is drawn from are read.  A cluster of kRanks CTAs takes one
// sequence; a warp sums one contiguous span of the row, the totals meet in distributed
// shared memory, and the CTA that holds the threshold looks through that one span again (from L2).
#include <cstdint>

#include <cooperative_groups.h>

#include "lily_internal.h"

namespace lily {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512, kWarps = kThreads / 32, kRanks = 8;
using u64 = unsigned long long;

// p in [0, 1] in units of 2^-62, rounded down (exact from 2^-38 on); 0 for NaN and below 0.
__device__ __forceinline__ u64 fixed62(float p)
{
    if (!(p > 0.0f)) return 0;
    p = fminf(p, 1.0f);
    const uint32_t bits = __float_as_uint(p);
    const int e = static_cast<int>(bits >> 23);          // value = mantissa * 2^(e - 150)
    const u64 m = (bits & 0x7FFFFFu) | 0x800000u;        // subnormals are far below 2^-62: 0 all the same
    return e >= 88 ? m << (e - 88) : e >= 64 ? m >> (88 - e) : 0;
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

// Weight of token v: max(p - q, 0), or p where there is no q; `gone` has none.
struct Row {
    const float *p, *q;
    int gone;
    __device__ __forceinline__ u64 weight(float pv, float qv, int v) const
    {
        const u64 a = fixed62(pv), b = q ? fixed62(qv) : 0;
        return a > b && v != gone ? a - b : 0;
    }
    __device__ __forceinline__ u64 operator()(int v) const { return weight(p[v], q ? q[v] : 0.0f, v); }
};

__global__ void __cluster_dims__(kRanks, 1, 1) __launch_bounds__(kThreads)
    verify_kernel(const __grid_constant__ VerifyArgs a)
{
    __shared__ int first_refused;
    __shared__ u64 span_sum[kWarps], total_s, scan_s[kWarps];
    pdl_trigger();
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank()), b = blockIdx.x / kRanks, tid = threadIdx.x;
    const int warp = tid / 32, lane = tid % 32;
    if (tid == 0) first_refused = 0x7FFFFFFF;
    __syncthreads();
    pdl_wait();

    const int c0 = a.cu[b], c1 = a.cu[b + 1], m = c1 - c0;
    if (c0 < 0 || c1 < c0 || c1 > a.N) {  // all CTAs of the cluster agree
        if (tid == 0) record_error(&a.ctrl->status, kErrDeviceIndex);
        return;
    }
    const float r = a.r[b];
    for (int i = tid; i < m; i += kThreads) {
        const int x = a.drafts[c0 + i];
        bool ok = false;
        if (x < 0 || x >= a.V) {
            record_error(&a.ctrl->status, kErrDeviceIndex);
        } else {
            const double px = a.p[(static_cast<long long>(c0) + b + i) * a.p_stride + x];
            const double qx = a.q ? a.q[(static_cast<long long>(c0) + i) * a.q_stride + x] : 1.0f;
            ok = static_cast<double>(a.u[c0 + i]) * qx < px;
        }
        if (!ok) atomicMin(&first_refused, i);
    }
    __syncthreads();
    const int n = min(first_refused, m);
    const bool refused = n < m;
    if (rank == 0) {
        if (tid == 0) a.accepted[b] = n;
        for (int i = tid; i <= m; i += kThreads)
            if (i != n) a.tokens[c0 + b + i] = i < n ? a.drafts[c0 + i] : -1;
    }

    Row row;
    row.p = a.p + (static_cast<long long>(c0) + b + n) * a.p_stride;
    row.q = refused && a.q ? a.q + (static_cast<long long>(c0) + n) * a.q_stride : nullptr;
    row.gone = refused && !a.q ? a.drafts[c0 + n] : -1;
    // the warp's span: [V s / S, V (s + 1) / S) of S = kRanks kWarps
    const int s = rank * kWarps + warp;
    auto bound = [&](int i) { return static_cast<int>(static_cast<long long>(a.V) * i / (kRanks * kWarps)); };
    const int v0 = bound(s), v1 = bound(s + 1);
    u64 total = 0, before = 0;
    for (int pass = 0; pass < 2; ++pass) {
        u64 sum = 0;
        constexpr int kUnroll = 8;
        int v = v0 + lane;
        for (; v + 32 * (kUnroll - 1) < v1; v += 32 * kUnroll) {
            float pv[kUnroll], qv[kUnroll];
#pragma unroll
            for (int j = 0; j < kUnroll; ++j) {
                pv[j] = row.p[v + 32 * j];
                qv[j] = row.q ? row.q[v + 32 * j] : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < kUnroll; ++j) sum += row.weight(pv[j], qv[j], v + 32 * j);
        }
        for (; v < v1; v += 32) sum += row(v);
        sum = warp_sum(sum);
        if (lane == 0) span_sum[warp] = sum;
        __syncthreads();
        if (warp == 0) {
            const u64 t = warp_sum(lane < kWarps ? span_sum[lane] : 0);
            if (lane == 0) total_s = t;
        }
        cluster.sync();
        total = before = 0;
        for (int k = 0; k < kRanks; ++k) {
            const u64 t = *cluster.map_shared_rank(&total_s, k);
            if (k < rank) before += t;
            total += t;
        }
        cluster.sync();  // nobody writes or leaves while another reads
        if (total || (!row.q && row.gone < 0)) break;
        // p nowhere above q (as sums that are rounded can give): the token comes from p itself
        row.q = nullptr;
        row.gone = -1;
    }
    if (total == 0) {
        if (rank == 0 && tid == 0) {
            a.tokens[c0 + b + n] = -1;
            record_error(&a.ctrl->status, kErrDeviceRange);
        }
        return;
    }
    // the token is the first whose running sum passes `below`
    const u64 below = __umul64hi(total, fixed64(r));
    if (below < before || below - before >= total_s) return;  // another CTA has it
    int w = 0;
    for (; w < kWarps - 1 && below - before >= span_sum[w]; ++w) before += span_sum[w];
    // that span again, a contiguous piece for each thread
    const int u0 = bound(rank * kWarps + w), u1 = bound(rank * kWarps + w + 1);
    const int each = (u1 - u0 + kThreads - 1) / kThreads;
    const int a0 = min(u0 + tid * each, u1), a1 = min(a0 + each, u1);
    u64 mine = 0;
    for (int v = a0; v < a1; ++v) mine += row(v);
    u64 upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 t = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += t;
    }
    if (lane == 31) scan_s[warp] = upto;
    __syncthreads();
    for (int k = 0; k < warp; ++k) before += scan_s[k];
    before += upto - mine;
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

}  // namespace

cudaError_t launch_verify(const VerifyArgs &a, cudaStream_t stream)
{
    return launch_pdl(verify_kernel, dim3(a.B * kRanks), dim3(kThreads), 0, stream, a);
}

}  // namespace lily
