// The quantised KV cache: append (quantise new keys and values as they are
// written) and read back, for sm_103a.
//
// Method (page "Perplexity libera o Lily", noticiai.com.br): group-of-64 affine
// codes with a bf16 scale and bias, rebuilt by code * scale + bias (section
// "Prefill e decode: onde estao os ganhos"), applied to the fixed-block KV cache
// of the full-attention layers.  Per token, KV head and group of 64 channels,
// with lo / hi the group's extremes and L = 2^bits - 1:
//   scale = bf16((hi - lo) / L),  code = min(rint((x - lo) / scale), L),
//   value = code * scale + lo.
//
// Eight threads hold one group, eight channels each: the extremes are three
// butterfly shuffles.
#include <cstdint>

#include "lily_device.cuh"
#include "lily_internal.h"

namespace lily {
namespace {

constexpr int kThreads = 256;

// Cache row of the call's token n: physical block in .x, row in .y; .x < 0
// where there is none (padding, or an index out of range, which is recorded).
__device__ __forceinline__ int2 token_slot(const KvqCopyArgs &a, int n)
{
    int lo = 0, hi = a.B;  // the last b with cu[b] <= n
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.cu[mid] <= n)
            lo = mid;
        else
            hi = mid;
    }
    const int i = n - a.cu[lo];
    if (i < 0 || n >= a.cu[lo + 1]) return make_int2(-1, 0);
    const long long pos = static_cast<long long>(a.starts[lo]) + i;
    if (pos < 0 || pos >= static_cast<long long>(a.max_blocks) * a.c.bs) {
        record_error(&a.ctrl->status, kErrDeviceIndex);
        return make_int2(-1, 0);
    }
    const int p = static_cast<int>(pos);
    const int pb = a.block_table[static_cast<size_t>(lo) * a.max_blocks + p / a.c.bs];
    if (pb < 0 || pb >= a.c.n_blocks) {
        record_error(&a.ctrl->status, kErrDeviceIndex);
        return make_int2(-1, 0);
    }
    return make_int2(pb, p % a.c.bs);
}

// Index of (physical block, head, group, row) in the parameter arrays (pairs)
// and, times the bytes of a group's codes, in the code arrays.
__device__ __forceinline__ long long group_index(const KvqCache &c, int2 slot, int head, int group)
{
    return ((static_cast<long long>(slot.x) * c.H_kv + head) * c.groups + group) * c.bs + slot.y;
}

// The codes of eight channels x (fp32) of a group, packed low to high.
template <int BITS>
__device__ __forceinline__ uint2 quantise8(const float (&x)[8], float lo, float scale)
{
    constexpr float L = BITS == 4 ? 15.0f : 255.0f;
    uint32_t c[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float t = scale > 0.0f ? fminf(rintf((0.5f * x[j] - 0.5f * lo) / (0.5f * scale)), L) : 0.0f;
        c[j] = static_cast<uint32_t>(t);
    }
    uint2 w = make_uint2(0u, 0u);
    if (BITS == 4) {
#pragma unroll
        for (int j = 0; j < 8; ++j) w.x |= c[j] << (4 * j);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w.x |= c[j] << (8 * j);
            w.y |= c[j + 4] << (8 * j);
        }
    }
    return w;
}

template <int BITS>
__global__ void __launch_bounds__(kThreads) kvq_append_kernel(const KvqCopyArgs a)
{
    pdl_trigger();
    pdl_wait();
    const int n = blockIdx.x;
    const int2 slot = token_slot(a, n);
    if (slot.x < 0) return;
    const int units = 2 * a.c.H_kv * a.c.groups;  // K, then V
    for (int u0 = 0; u0 < units; u0 += kThreads / 8) {
        const int u = u0 + threadIdx.x / 8, e = threadIdx.x % 8;
        const bool act = u < units;
        const int uu = act ? u : 0;
        const int which = uu / (a.c.H_kv * a.c.groups), hg = uu % (a.c.H_kv * a.c.groups);
        const uint16_t *src = which ? a.v + n * a.v_stride : a.k + n * a.k_stride;
        const uint4 w = *reinterpret_cast<const uint4 *>(src + hg * 64 + e * 8);
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
        float x[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = __uint_as_float(ws[j] << 16);
            x[2 * j + 1] = __uint_as_float(ws[j] & 0xFFFF0000u);
        }
        float lo = x[0], hi = x[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) {
            lo = fminf(lo, x[j]);
            hi = fmaxf(hi, x[j]);
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
            lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        }
        // halves, so that the range of any two finite bf16 values is finite
        constexpr float L = BITS == 4 ? 15.0f : 255.0f;
        const __nv_bfloat16 sb = __float2bfloat16_rn((0.5f * hi - 0.5f * lo) / (0.5f * L));
        float scale = __bfloat162float(sb);
        if (!(scale >= 1.17549435e-38f)) scale = 0.0f;
        const uint2 c = quantise8<BITS>(x, lo, scale);
        if (!act) continue;
        const long long gi = group_index(a.c, slot, hg / a.c.groups, hg % a.c.groups);
        uint8_t *dq = (which ? a.c.v_q : a.c.k_q) + gi * (8 * BITS) + e * BITS;
        if (BITS == 4)
            *reinterpret_cast<uint32_t *>(dq) = c.x;
        else
            *reinterpret_cast<uint2 *>(dq) = c;
        if (e == 0)
            *reinterpret_cast<uint32_t *>((which ? a.c.v_sb : a.c.k_sb) + gi * 2) =
                (__float_as_uint(scale) >> 16) | (__float_as_uint(lo) & 0xFFFF0000u);
    }
}

template <int BITS>
__global__ void __launch_bounds__(kThreads) kvq_read_kernel(const KvqCopyArgs a)
{
    pdl_trigger();
    pdl_wait();
    const int n = blockIdx.x;
    const int2 slot = token_slot(a, n);
    if (slot.x < 0) return;
    const int units = 2 * a.c.H_kv * a.c.groups;
    for (int i = threadIdx.x; i < units * 8; i += kThreads) {
        const int u = i / 8, e = i % 8;
        const int which = u / (a.c.H_kv * a.c.groups), hg = u % (a.c.H_kv * a.c.groups);
        const long long gi = group_index(a.c, slot, hg / a.c.groups, hg % a.c.groups);
        const uint8_t *sq = (which ? a.c.v_q : a.c.k_q) + gi * (8 * BITS) + e * BITS;
        const uint32_t sb = *reinterpret_cast<const uint32_t *>((which ? a.c.v_sb : a.c.k_sb) + gi * 2);
        const float s = __uint_as_float(sb << 16), b = __uint_as_float(sb & 0xFFFF0000u);
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t w = BITS == 4 ? *reinterpret_cast<const uint32_t *>(sq) >> (8 * j)
                                         : static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(sq)[j]);
            const float c0 = static_cast<float>(w & ((1u << BITS) - 1)), c1 = static_cast<float>((w >> BITS) & ((1u << BITS) - 1));
            o[j] = static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(fmaf(c0, s, b)))) |
                   (static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(fmaf(c1, s, b)))) << 16);
        }
        uint16_t *dst = (which ? a.v + n * a.v_stride : a.k + n * a.k_stride) + hg * 64 + e * 8;
        *reinterpret_cast<uint4 *>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

}  // namespace

cudaError_t launch_kvq_append(const KvqCopyArgs &a, cudaStream_t stream)
{
    return launch_pdl(a.c.bits == 4 ? kvq_append_kernel<4> : kvq_append_kernel<8>, dim3(a.N), dim3(kThreads), 0, stream, a);
}

cudaError_t launch_kvq_read(const KvqCopyArgs &a, cudaStream_t stream)
{
    return launch_pdl(a.c.bits == 4 ? kvq_read_kernel<4> : kvq_read_kernel<8>, dim3(a.N), dim3(kThreads), 0, stream, a);
}

}  // namespace lily
