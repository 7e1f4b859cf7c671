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
// one 128-byte run of codes; several such steps are in flight per thread (append 3, read 8).
// The extremes are three butterfly shuffles of one packed register (lo, -hi).  Measured (2 KV
// heads of 256): 65,536 tokens at 4 bits read in 31.7 us (5.4 TB/s, 0.80 of the measured copy
// rate; writes are 78% of the bytes); with 4 heads of 128 at 8 bits, 63,251 tokens
// written and read back in 74.1 us (5.4 TB/s).  The append is near its issue limit, so its
// arithmetic takes two values an instruction (10,754 tokens written and read 17.3 us without,
// 16.5 with), and its first loads are issued before the tokens' rows are known (four tokens 4.4 ->
// 4.2 us).  Four groups in flight spill at five CTAs an SM (16.5 us, 17.9 at four) where
// three take 16.1 at four; the read with five CTAs takes 32.8 us, with six 48.4.
#include <cstdint>

#include "kvq_device.cuh"
#include "lily_internal.h"

namespace lily {
namespace {

constexpr int kThreads = 256;

constexpr int kMaxShared = kThreads - 1;  // sequences whose bounds a CTA takes into shared memory

// Cache row of the call's token n: physical block in .x, row in .y; .x < 0 where there
// is none (padding, or an index out of range, which is recorded).  cu, starts: the
// call's, or their copies in shared memory (a search in global memory is a chain of
// loads of ~0.6 us each).
__device__ __forceinline__ int2 token_slot(const KvqCopyArgs &a, const int *cu, const int *starts, int n)
{
    int lo = 0, hi = a.B;  // the last b with cu[b] <= n
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= n)
            lo = mid;
        else
            hi = mid;
    }
    const int i = n - cu[lo];
    if (i < 0 || n >= cu[lo + 1]) return make_int2(-1, 0);
    const long long pos = static_cast<long long>(starts[lo]) + i;
    if (pos < 0 || pos >= static_cast<long long>(a.max_blocks) * a.c.bs) {
        record_error(&a.ctrl->status, kErrDeviceIndex);
        return make_int2(-1, 0);
    }
    const int p = static_cast<int>(pos), bs_log = 31 - __clz(a.c.bs);
    const int pb = a.block_table[static_cast<size_t>(lo) * a.max_blocks + (p >> bs_log)];
    if (pb < 0 || pb >= a.c.n_blocks) {
        record_error(&a.ctrl->status, kErrDeviceIndex);
        return make_int2(-1, 0);
    }
    return make_int2(pb, p & (a.c.bs - 1));
}

// Scale and bias of a group, and what its codes are computed with.  Both quotients,
// (hi - lo) / L and q = (x - lo) / scale, are rounded correctly as in Markstein's
// division: q0 = d r with r about 1 / h, then q = q0 + r (d - q0 h) with fused
// multiply-adds; h has 8 bits, so no quotient of a 24-bit d comes nearer than 2^-33 to
// a rounding border, and r may be the hardware's approximation.  All of it is computed
// times m, a power of two that keeps every term within the normal numbers: the range of
// two finite bf16 values is finite in halves, and where it is below 2^-32 the group takes
// 2^64: then either all of it is below 2^-24, or (lo not below 1) its values are equal, at any
// size; those stay in halves, with a range and a scale of 0.
struct GroupScale {
    float m, h, r, mlo;
    uint32_t sb;  // scale, bias as stored
};
template <int BITS>
__device__ __forceinline__ GroupScale group_scale(float lo, float hi)
{
    constexpr float L = BITS == 4 ? 15.0f : 255.0f, rL = 1.0f / L;
    GroupScale g;
    const float half = 0.5f * hi - 0.5f * lo;
    const bool lift = half < 0x1p-33f && fabsf(lo) < 1.0f;
    g.m = lift ? 0x1p64f : 0.5f;
    g.mlo = -lo * g.m;
    const float range = fmaf(hi, g.m, g.mlo);
    const float q0 = __fmul_rn(range, rL);
    g.h = __bfloat162float(__float2bfloat16_rn(fmaf(fmaf(-q0, L, range), rL, q0)));
    if (g.h < (lift ? 0x1p-62f : 0x1p-127f)) g.h = 0.0f;  // a scale below 2^-126
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(g.r) : "f"(g.h));
    if (g.h == 0.0f) g.r = 0.0f;  // every code is 0
    g.sb = (__float_as_uint(g.h * (lift ? 0x1p-64f : 2.0f)) >> 16) | (__float_as_uint(lo) & 0xFFFF0000u);
    return g;
}

// The codes of eight channels (bf16 pairs) packed low to high: n + 1.5 2^23 holds the
// integer n in its low bits, so the codes add up by multiply-adds on the bit patterns.
template <int BITS>
__device__ __forceinline__ uint2 quantise8(const uint4 &w, const GroupScale &g)
{
    constexpr float L = 255.0f;
    constexpr uint32_t kMagic = 0x4B400000u, kStep = 1u << BITS;
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
    const unsigned long long m = pair(g.m, g.m), mlo = pair(g.mlo, g.mlo), h = pair(-g.h, -g.h), r = pair(g.r, g.r);
    uint32_t c[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // two values an instruction
        const unsigned long long d = fma2(pair(__uint_as_float(ws[j] << 16), __uint_as_float(ws[j] & 0xFFFF0000u)), m, mlo);
        const unsigned long long q0 = mul2(d, r);
        unsigned long long q = fma2(r, fma2(q0, h, d), q0);
        // the scale is rounded by 2^-8 at most, so at 4 bits q stays below 15.06 and needs no limit
        if constexpr (BITS == 8) {
            float a, b;
            unpair(q, a, b);
            q = pair(fminf(a, L), fminf(b, L));
        }
        float a, b;
        unpair(add2(q, pair(12582912.0f, 12582912.0f)), a, b);
        c[2 * j] = __float_as_uint(a);
        c[2 * j + 1] = __float_as_uint(b);
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

// One thread's place in a call: its token's row on the bf16 side (+ 64 per group), and
// in the codes and the parameters of K or of V (+ group_step bytes, + 2 bs elements).
struct Place {
    uint16_t *row;
    uint8_t *codes;
    uint16_t *params;
    int bs, groups;  // groups of a token: H_kv D / 64
    bool act;        // the token has a cache row
};

// The CTA's 4 QUADS tokens from blockIdx.x 4 QUADS on.  Half of the warps take K,
// half V; fn(place, group) runs for every group of the warp's four tokens, kBatch at a
// time: `load` for all of a batch, then `use` (by the whole warp).  kEarly: `load` needs
// only p.row, so the first batch is on its way while the tokens' cache rows are looked up.
template <int BITS, int QUADS, int kBatch, bool kEarly, typename T, typename Load, typename Use>
__device__ __forceinline__ void for_tokens(const KvqCopyArgs &a, const Load &load, const Use &use)
{
    __shared__ int2 slots[4 * QUADS];
    __shared__ int cu_s[kThreads], starts_s[kThreads];
    const int n0 = blockIdx.x * (4 * QUADS), t = threadIdx.x;
    const bool shared = a.B <= kMaxShared;
    if (shared) {
        if (t <= a.B) cu_s[t] = a.cu[t];
        if (t < a.B) starts_s[t] = a.starts[t];
    }
    constexpr int kStep = kThreads / 32 / QUADS / 2;
    const int warp = threadIdx.x / 32, e = threadIdx.x % 8, tok = (warp % QUADS) * 4 + (threadIdx.x % 32) / 8, first = warp / QUADS / 2;
    const long long n = n0 + tok;
    const bool isv = (warp / QUADS) & 1;
    Place p;
    p.bs = a.c.bs;
    p.groups = a.c.H_kv * a.c.groups;
    p.row = (isv ? a.v + n * a.v_stride : a.k + n * a.k_stride) + e * 8;
    T v[kBatch];
    auto load_batch = [&](int g0) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (p.act && g0 + i * kStep < p.groups) v[i] = load(p, g0 + i * kStep);
    };
    if (kEarly) {
        p.act = n < a.N;
        load_batch(first);
    }
    if (shared) __syncthreads();
    if (t < 4 * QUADS)
        slots[t] = n0 + t >= a.N ? make_int2(-1, 0) : shared ? token_slot(a, cu_s, starts_s, n0 + t) : token_slot(a, a.cu, a.starts, n0 + t);
    __syncthreads();
    const int2 slot = slots[tok];
    p.act = slot.x >= 0;
    const long long at = p.act ? static_cast<long long>(slot.x) * p.groups * p.bs + slot.y : 0;
    p.codes = (isv ? a.c.v_q : a.c.k_q) + at * (8 * BITS) + e * BITS;
    p.params = (isv ? a.c.v_sb : a.c.k_sb) + at * 2;
    for (int g0 = first; g0 < p.groups; g0 += kStep * kBatch) {
        if (!kEarly || g0 != first) load_batch(g0);
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (g0 + i * kStep < p.groups) use(p, g0 + i * kStep, v[i]);
    }
}

template <int BITS, int QUADS>
__global__ void __launch_bounds__(kThreads, 4) kvq_append_kernel(const __grid_constant__ KvqCopyArgs a)
{
    pdl_trigger();
    pdl_wait();
    for_tokens<BITS, QUADS, 3, true, uint4>(
        a, [](const Place &p, int g) { return *reinterpret_cast<const uint4 *>(p.row + g * 64); },
        [](const Place &p, int g, const uint4 &w) {
            const uint32_t lo2 = bf16x2_min(bf16x2_min(w.x, w.y), bf16x2_min(w.z, w.w));
            const uint32_t hi2 = bf16x2_max(bf16x2_max(w.x, w.y), bf16x2_max(w.z, w.w)) ^ 0x80008000u;  // -hi
            // (lo, -hi): the two halves of each, then the eight threads
            uint32_t x = bf16x2_min(__byte_perm(lo2, hi2, 0x5410), __byte_perm(lo2, hi2, 0x7632));
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) x = bf16x2_min(x, __shfl_xor_sync(0xffffffffu, x, o));
            if (!p.act) return;
            const GroupScale s = group_scale<BITS>(__uint_as_float(x << 16), -__uint_as_float(x & 0xFFFF0000u));
            const uint2 c = quantise8<BITS>(w, s);
            uint8_t *dst = p.codes + g * p.bs * (8 * BITS);
            if (BITS == 4)
                *reinterpret_cast<uint32_t *>(dst) = c.x;
            else
                *reinterpret_cast<uint2 *>(dst) = c;
            if (threadIdx.x % 8 == 0) *reinterpret_cast<uint32_t *>(p.params + g * p.bs * 2) = s.sb;
        });
}

template <int BITS, int QUADS>
__global__ void __launch_bounds__(kThreads, 4) kvq_read_kernel(const __grid_constant__ KvqCopyArgs a)
{
    pdl_trigger();
    pdl_wait();
    struct Codes {
        uint2 q;
        uint32_t sb;
    };
    for_tokens<BITS, QUADS, 8, false, Codes>(
        a,
        [](const Place &p, int g) {
            const uint8_t *src = p.codes + g * p.bs * (8 * BITS);
            Codes c;
            c.q = BITS == 8 ? *reinterpret_cast<const uint2 *>(src) : make_uint2(*reinterpret_cast<const uint32_t *>(src), 0u);
            c.sb = *reinterpret_cast<const uint32_t *>(p.params + g * p.bs * 2);
            return c;
        },
        [](const Place &p, int g, const Codes &c) {
            if (!p.act) return;
            const float s = __uint_as_float(c.sb << 16), b = __uint_as_float(c.sb & 0xFFFF0000u);
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // 2^23 + code is the code in the low bits of the pattern of 2^23
                const uint32_t w = BITS == 4 ? c.q.x >> (8 * j) : (j < 2 ? c.q.x : c.q.y) >> (16 * (j & 1));
                const float c0 = __uint_as_float((w & ((1u << BITS) - 1)) | 0x4B000000u) - 8388608.0f;
                const float c1 = __uint_as_float(((w >> BITS) & ((1u << BITS) - 1)) | 0x4B000000u) - 8388608.0f;
                const __nv_bfloat162 y = __floats2bfloat162_rn(fmaf(c0, s, b), fmaf(c1, s, b));
                o[j] = *reinterpret_cast<const uint32_t *>(&y);
            }
            *reinterpret_cast<uint4 *>(p.row + g * 64) = make_uint4(o[0], o[1], o[2], o[3]);
        });
}

// 16 tokens a CTA; four where 16 would leave half of the SMs without one (a CTA's first
// step waits for its tokens' rows, so more and smaller CTAs cost more otherwise: 4,385
// tokens of 64 channels and 3 heads read in 5.7 us with four a CTA, 3.1 us with 16).
constexpr int kFewTokens = 16 * 76;
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
