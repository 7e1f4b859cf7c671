// Attention over the quantised KV cache, for sm_103a: per query token n of
// sequence b and query head h, with g = h / (H_q / H_kv),
//   o = sum_{t < limit} softmax_t(scale q . k_t) v_t,
// k_t and v_t the values code * scale + bias of row t of KV head g.
//
// One CTA per (query token, KV head) walks the cache in tiles of 32 tokens, the
// values rebuilt in fp32 in shared memory, with a running maximum and sum per
// query head.
#include <cmath>
#include <cstdint>

#include "lily_device.cuh"
#include "lily_internal.h"

namespace lily {
namespace {

constexpr int kThreads = 128;
constexpr int kTile = 32;  // tokens per tile

__global__ void __launch_bounds__(kThreads) kvq_prefill_kernel(const KvqAttnArgs a)
{
    extern __shared__ float sm[];
    const int D = a.D, G = a.group, n = blockIdx.x, g = blockIdx.y, tid = threadIdx.x;
    float *qs = sm, *kv = qs + kKvqMaxGroup * D, *p = kv + kTile * (D + 1), *al = p + kKvqMaxGroup * kTile;
    pdl_trigger();
    pdl_wait();
    int b = n, m = 1, i = 0;
    if (a.cu_q) {
        int lo = 0, hi = a.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.cu_q[mid] <= n)
                lo = mid;
            else
                hi = mid;
        }
        b = lo;
        i = n - a.cu_q[b];
        m = a.cu_q[b + 1] - a.cu_q[b];
        if (i < 0 || i >= m) return;  // padding
    }
    const long long cap = static_cast<long long>(a.max_blocks) * a.c.bs;
    long long L = a.seq_lens[b];
    if (L < 0 || L > cap) {
        if (tid == 0) record_error(&a.ctrl->status, kErrDeviceIndex);
        L = L < 0 ? 0 : cap;
    }
    const int limit = static_cast<int>(L - m + i + 1 > 0 ? L - m + i + 1 : 0);
    for (int j = tid; j < G * D; j += kThreads)
        qs[j] = __uint_as_float(static_cast<uint32_t>(a.q[n * a.q_stride + static_cast<long long>(g) * G * D + j]) << 16);
    float acc[kKvqMaxGroup][2], mx = -INFINITY, sum = 0.0f;
    for (int h = 0; h < kKvqMaxGroup; ++h) acc[h][0] = acc[h][1] = 0.0f;
    const int bits = a.c.bits, bs = a.c.bs, gb = 8 * bits;
    auto load = [&](const uint8_t *codes, const uint16_t *sb, int t0, int cnt) {
        for (int j = tid; j < cnt * D; j += kThreads) {
            const int t = j / D, d = j % D, pos = t0 + t;
            int pb = a.block_table[static_cast<size_t>(b) * a.max_blocks + pos / bs];
            if (pb < 0 || pb >= a.c.n_blocks) {
                record_error(&a.ctrl->status, kErrDeviceIndex);
                pb = 0;
            }
            const long long gi = ((static_cast<long long>(pb) * a.c.H_kv + g) * a.c.groups + d / 64) * bs + pos % bs;
            const uint32_t w = codes[gi * gb + (bits == 4 ? (d % 64) / 2 : d % 64)];
            const float c = static_cast<float>(bits == 4 ? (d % 2 ? w >> 4 : w & 15) : w);
            const uint32_t q = *reinterpret_cast<const uint32_t *>(sb + gi * 2);
            kv[t * (D + 1) + d] = fmaf(c, __uint_as_float(q << 16), __uint_as_float(q & 0xFFFF0000u));
        }
    };
    for (int t0 = 0; t0 < limit; t0 += kTile) {
        const int cnt = min(kTile, limit - t0);
        __syncthreads();
        load(a.c.k_q, a.c.k_sb, t0, cnt);
        __syncthreads();
        for (int j = tid; j < G * kTile; j += kThreads) {
            const int h = j / kTile, t = j % kTile;
            float s = -INFINITY;
            if (t < cnt) {
                s = 0.0f;
                for (int d = 0; d < D; ++d) s = fmaf(qs[h * D + d], kv[t * (D + 1) + d], s);
                s *= a.scale_log2;
            }
            p[j] = s;
        }
        __syncthreads();
        load(a.c.v_q, a.c.v_sb, t0, cnt);
        if (tid < G) {  // thread h: the running maximum and sum of head h
            float mn = mx;
            for (int t = 0; t < cnt; ++t) mn = fmaxf(mn, p[tid * kTile + t]);
            al[tid] = exp2f(mx - mn);
            sum *= al[tid];
            for (int t = 0; t < cnt; ++t) {
                const float w = exp2f(p[tid * kTile + t] - mn);
                p[tid * kTile + t] = w;
                sum += w;
            }
            mx = mn;
        }
        __syncthreads();
        for (int x = 0; x < 2; ++x) {
            const int d = tid + x * kThreads;
            if (d >= D) break;
            for (int h = 0; h < G; ++h) {
                float o = acc[h][x] * al[h];
                for (int t = 0; t < cnt; ++t) o = fmaf(p[h * kTile + t], kv[t * (D + 1) + d], o);
                acc[h][x] = o;
            }
        }
    }
    __syncthreads();
    if (tid < G) al[tid] = sum > 0.0f ? 1.0f / sum : 0.0f;
    __syncthreads();
    for (int x = 0; x < 2; ++x) {
        const int d = tid + x * kThreads;
        if (d >= D) break;
        for (int h = 0; h < G; ++h)
            a.out[(static_cast<size_t>(n) * a.H_q + g * G + h) * D + d] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[h][x] * al[h]));
    }
}

}  // namespace

cudaError_t launch_kvq_prefill(const KvqAttnArgs &a, cudaStream_t stream)
{
    const size_t smem = sizeof(float) * (kKvqMaxGroup * a.D + kTile * (a.D + 1) + kKvqMaxGroup * kTile + kKvqMaxGroup);
    const cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void *>(kvq_prefill_kernel), static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    return launch_pdl(kvq_prefill_kernel, dim3(a.N, a.c.H_kv), dim3(kThreads), smem, stream, a);
}

}  // namespace lily
