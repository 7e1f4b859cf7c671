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
// Bound: HBM (2 + 0.5625 bytes a value at 4 bits, 2 + 1.0625 at 8).  A warp takes
// four consecutive tokens of one (K or V, head, group): eight threads a token, eight
// channels each, so that it reads whole 128-byte lines of the bf16 side and touches
// one 128-byte run of codes; four such steps are in flight per thread.  The extremes
// are three butterfly shuffles of one packed register (lo, -hi).
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

// Scale and bias of a group, and what its codes are computed with: code =
// min(rint(q), L) with q = (x - lo) / scale, correctly rounded as in Markstein's
// division: q0 = d r with r = 1 / h, then q = q0 + r (d - q0 h) with fused
// multiply-adds, for d = (x - lo) m and h = scale m.  The factor m (a power of two)
// keeps every term within the normal numbers: x - lo of any two finite bf16 values is
// finite in halves, and below a scale of 2^-40 all of the group is below 2^-24, so 2^64
// lifts the remainder out of the subnormals.
struct GroupScale {
    float m, h, r, mlo;
    uint32_t sb;  // scale, bias as stored
};
template <int BITS>
__device__ __forceinline__ GroupScale group_scale(float lo, float hi)
{
    constexpr float L = BITS == 4 ? 15.0f : 255.0f;
    GroupScale g;
    float scale = __bfloat162float(__float2bfloat16_rn((0.5f * hi - 0.5f * lo) / (0.5f * L)));
    if (!(scale >= 1.17549435e-38f)) scale = 0.0f;  // 2^-126
    g.m = scale < 0x1p-40f ? 0x1p64f : 0.5f;
    g.h = scale * g.m;
    g.r = scale > 0.0f ? 1.0f / g.h : 0.0f;  // 0: every code is 0
    g.mlo = -lo * g.m;
    g.sb = (__float_as_uint(scale) >> 16) | (__float_as_uint(lo) & 0xFFFF0000u);
    return g;
}

// The codes of eight channels (bf16 pairs) packed low to high: n + 1.5 2^23 holds the
// integer n in its low bits, so the codes add up by multiply-adds on the bit patterns.
template <int BITS>
__device__ __forceinline__ uint2 quantise8(const uint4 &w, const GroupScale &g)
{
    constexpr float L = BITS == 4 ? 15.0f : 255.0f;
    constexpr uint32_t kMagic = 0x4B400000u, kStep = 1u << BITS;
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
    uint32_t c[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float x = j & 1 ? __uint_as_float(ws[j / 2] & 0xFFFF0000u) : __uint_as_float(ws[j / 2] << 16);
        const float d = fmaf(x, g.m, g.mlo);
        const float q0 = __fmul_rn(d, g.r);
        const float q = fmaf(g.r, fmaf(-q0, g.h, d), q0);
        c[j] = __float_as_uint(__fadd_rn(fminf(q, L), 12582912.0f));
    }
    if (BITS == 4) {
        uint32_t p = c[7], k = kMagic;
#pragma unroll
        for (int j = 6; j >= 0; --j) {
            p = p * kStep + c[j];
            k = k * kStep + kMagic;
        }
        return make_uint2(p - k, 0u);
    }
    uint32_t p = c[3], q = c[7], k = kMagic;
#pragma unroll
    for (int j = 2; j >= 0; --j) {
        p = p * kStep + c[j];
        q = q * kStep + c[j + 4];
        k = k * kStep + kMagic;
    }
    return make_uint2(p - k, q - k);
}

__device__ __forceinline__ uint32_t bf16x2_min(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t bf16x2_max(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

constexpr int kBatch = 4;  // groups of a warp's tokens in flight

// The CTA's 4 QUADS tokens from blockIdx.x 4 QUADS on: their cache rows, then
// fn(token within the call, slot, which, head * groups + group) for every quad and
// (K or V, head, group), in batches: `load` for all of a batch, then `use`.
template <int QUADS, typename T, typename Load, typename Use>
__device__ __forceinline__ void for_tokens(const KvqCopyArgs &a, const Load &load, const Use &use)
{
    __shared__ int2 slots[4 * QUADS];
    const int n0 = blockIdx.x * (4 * QUADS);
    if (threadIdx.x < 4 * QUADS)
        slots[threadIdx.x] = n0 + static_cast<int>(threadIdx.x) < a.N ? token_slot(a, n0 + threadIdx.x) : make_int2(-1, 0);
    __syncthreads();
    const int warp = threadIdx.x / 32, tok = (warp % QUADS) * 4 + (threadIdx.x % 32) / 8;
    const int2 slot = slots[tok];
    const long long n = n0 + tok;
    const int per = a.c.H_kv * a.c.groups, units = 2 * per;
    constexpr int kStride = kThreads / 32 / QUADS;
    for (int u0 = warp / QUADS; u0 < units; u0 += kStride * kBatch) {
        T v[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int u = u0 + i * kStride;
            if (slot.x >= 0 && u < units) v[i] = load(n, slot, u >= per, u >= per ? u - per : u);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int u = u0 + i * kStride;
            if (u < units) use(n, slot, u >= per, u >= per ? u - per : u, v[i]);  // the whole warp
        }
    }
}

template <int BITS, int QUADS>
__global__ void __launch_bounds__(kThreads) kvq_append_kernel(const __grid_constant__ KvqCopyArgs a)
{
    pdl_trigger();
    pdl_wait();
    const int e = threadIdx.x % 8;
    for_tokens<QUADS, uint4>(
        a,
        [&](long long n, int2, bool isv, int hg) {
            const uint16_t *src = isv ? a.v + n * a.v_stride : a.k + n * a.k_stride;
            return *reinterpret_cast<const uint4 *>(src + hg * 64 + e * 8);
        },
        [&](long long, int2 slot, bool isv, int hg, const uint4 &w) {
            const uint32_t lo2 = bf16x2_min(bf16x2_min(w.x, w.y), bf16x2_min(w.z, w.w));
            const uint32_t hi2 = bf16x2_max(bf16x2_max(w.x, w.y), bf16x2_max(w.z, w.w)) ^ 0x80008000u;  // -hi
            // (lo, -hi): the two halves of each, then the eight threads
            uint32_t x = bf16x2_min(__byte_perm(lo2, hi2, 0x5410), __byte_perm(lo2, hi2, 0x7632));
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) x = bf16x2_min(x, __shfl_xor_sync(0xffffffffu, x, o));
            if (slot.x < 0) return;
            const GroupScale g = group_scale<BITS>(__uint_as_float(x << 16), -__uint_as_float(x & 0xFFFF0000u));
            const uint2 c = quantise8<BITS>(w, g);
            const long long gi = group_index(a.c, slot, hg / a.c.groups, hg % a.c.groups);
            uint8_t *dq = (isv ? a.c.v_q : a.c.k_q) + gi * (8 * BITS) + e * BITS;
            if (BITS == 4)
                *reinterpret_cast<uint32_t *>(dq) = c.x;
            else
                *reinterpret_cast<uint2 *>(dq) = c;
            if (e == 0) *reinterpret_cast<uint32_t *>((isv ? a.c.v_sb : a.c.k_sb) + gi * 2) = g.sb;
        });
}

template <int BITS, int QUADS>
__global__ void __launch_bounds__(kThreads) kvq_read_kernel(const __grid_constant__ KvqCopyArgs a)
{
    pdl_trigger();
    pdl_wait();
    const int e = threadIdx.x % 8;
    struct Codes {
        uint32_t q0, q1, sb;
    };
    for_tokens<QUADS, Codes>(
        a,
        [&](long long, int2 slot, bool isv, int hg) {
            const long long gi = group_index(a.c, slot, hg / a.c.groups, hg % a.c.groups);
            const uint8_t *sq = (isv ? a.c.v_q : a.c.k_q) + gi * (8 * BITS) + e * BITS;
            Codes c;
            c.q0 = reinterpret_cast<const uint32_t *>(sq)[0];
            c.q1 = BITS == 8 ? reinterpret_cast<const uint32_t *>(sq)[BITS / 8] : 0u;
            c.sb = *reinterpret_cast<const uint32_t *>((isv ? a.c.v_sb : a.c.k_sb) + gi * 2);
            return c;
        },
        [&](long long n, int2 slot, bool isv, int hg, const Codes &c) {
            if (slot.x < 0) return;
            const float s = __uint_as_float(c.sb << 16), b = __uint_as_float(c.sb & 0xFFFF0000u);
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                // 2^23 + code is the code in the low bits of the pattern of 2^23
                const uint32_t w = BITS == 4 ? c.q0 >> (4 * j) : (j < 4 ? c.q0 : c.q1) >> (8 * (j & 3));
                const float code = __uint_as_float((w & ((1u << BITS) - 1)) | 0x4B000000u) - 8388608.0f;
                x[j] = fmaf(code, s, b);
            }
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __nv_bfloat162 y = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
                o[j] = *reinterpret_cast<const uint32_t *>(&y);
            }
            uint16_t *dst = (isv ? a.v + n * a.v_stride : a.k + n * a.k_stride) + hg * 64 + e * 8;
            *reinterpret_cast<uint4 *>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
        });
}

// 16 tokens a CTA; four where those would leave SMs idle (fewer than 16 x 304 tokens).
constexpr int kFewTokens = 16 * 304;
int ctas(int N, int quads) { return (N + 4 * quads - 1) / (4 * quads); }

template <int BITS>
cudaError_t append(const KvqCopyArgs &a, cudaStream_t stream)
{
    return a.N < kFewTokens ? launch_pdl(kvq_append_kernel<BITS, 1>, dim3(ctas(a.N, 1)), dim3(kThreads), 0, stream, a)
                            : launch_pdl(kvq_append_kernel<BITS, 4>, dim3(ctas(a.N, 4)), dim3(kThreads), 0, stream, a);
}
template <int BITS>
cudaError_t read(const KvqCopyArgs &a, cudaStream_t stream)
{
    return a.N < kFewTokens ? launch_pdl(kvq_read_kernel<BITS, 1>, dim3(ctas(a.N, 1)), dim3(kThreads), 0, stream, a)
                            : launch_pdl(kvq_read_kernel<BITS, 4>, dim3(ctas(a.N, 4)), dim3(kThreads), 0, stream, a);
}

}  // namespace

cudaError_t launch_kvq_append(const KvqCopyArgs &a, cudaStream_t stream)
{
    return a.c.bits == 4 ? append<4>(a, stream) : append<8>(a, stream);
}

cudaError_t launch_kvq_read(const KvqCopyArgs &a, cudaStream_t stream)
{
    return a.c.bits == 4 ? read<4>(a, stream) : read<8>(a, stream);
}

}  // namespace lily
