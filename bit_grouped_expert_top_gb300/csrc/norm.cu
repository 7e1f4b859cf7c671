// Root-mean-square norm with the residual's addition, for sm_103a; output in
// bf16, in e4m3 codes with a scale for each group of 64 channels, or both.
//
//   h = x + residual,  y = h / sqrt(mean_c h^2 + eps) * (weight + offset)
//   scale = max_group |y| / 448,  code = e4m3(y * (448 / max_group |y|))
//
// fp32 throughout; h and y are rounded once, as they are stored (the norm goes by the
// unrounded h, the codes by the unrounded y).
//
// Bound: HBM for a prompt, latency for a step.  One pass: a row stays in registers,
// TPR threads a row with PER vectors of eight channels each, so that the eight
// threads of a group of 64 are neighbours and its largest magnitude is three shuffles.
#include <cstdint>

#include <cuda_fp8.h>

#include "lily_internal.h"

namespace lily {
namespace {

// Threads of a CTA whose rows have TPR threads each: one row, where that is more than a warp, else 128 (with 256 the last CTAs end
// later: 60,000 rows of 128 13.5 us against 12.7, 32,784 of 256 14.8 against 13.9).
template <int TPR>
constexpr int kThreads = TPR > 32 ? TPR : 128;

__device__ __forceinline__ void unpack8(const uint4 &w, float (&v)[8])
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(u[j] << 16);
        v[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8])
{
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        u[j] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// Eight channels of an array of bf16 or fp32.
template <bool F32>
struct Vec {
    uint4 a[F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void *base, long long at)
    {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const char *>(base) + at * (F32 ? 4 : 2));
        a[0] = *p;
        if (F32) a[F32] = p[1];
    }
    __device__ __forceinline__ void values(float (&v)[8]) const
    {
        if (!F32) return unpack8(a[0], v);
        const uint32_t u[8] = {a[0].x, a[0].y, a[0].z, a[0].w, a[F32].x, a[F32].y, a[F32].z, a[F32].w};
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(u[j]);
    }
    static __device__ __forceinline__ void store(void *base, long long at, const float (&v)[8])
    {
        uint4 *p = reinterpret_cast<uint4 *>(static_cast<char *>(base) + at * (F32 ? 4 : 2));
        if (!F32) {
            *p = pack8(v);
        } else {
            p[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
            p[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
        }
    }
};

// Sum (or largest) over the TPR threads of a row; `part` holds a value of each warp.
template <int TPR, bool MAX>
__device__ __forceinline__ float over_row(float v, float *part)
{
    auto join = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
#pragma unroll
    for (int o = 1; o < (TPR < 32 ? TPR : 32); o <<= 1) v = join(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (TPR > 32) {
        constexpr int kWarps = TPR / 32;
        __syncthreads();
        if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
        __syncthreads();
        v = part[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) v = join(v, part[w]);
    }
    return v;
}

template <int TPR, int PER, bool XF32, int RES>  // RES: 0 none, 1 bf16, 2 fp32
__global__ void __launch_bounds__(kThreads<TPR>) norm_kernel(const __grid_constant__ NormArgs a)
{
    constexpr bool kWeightEarly = PER <= 2;
    __shared__ float part[kThreads<TPR> / 32];
    pdl_trigger();
    const int lane = threadIdx.x % TPR, vecs = a.d / 8;
    const long long row = static_cast<long long>(blockIdx.x) * (kThreads<TPR> / TPR) + threadIdx.x / TPR;
    const bool live = row < a.rows;
    const long long n = live ? row : 0;
    uint4 w[PER][2];
    auto load_weight = [&](int i) {
        const int c = lane + i * TPR;
        if (c < vecs && a.weight) {
            const char *p = static_cast<const char *>(a.weight) + static_cast<size_t>(c) * (a.w_f32 ? 32 : 16);
            w[i][0] = *reinterpret_cast<const uint4 *>(p);
            if (a.w_f32) w[i][1] = *reinterpret_cast<const uint4 *>(p + 16);
        }
    };
    pdl_wait();
    if (kWeightEarly) {
#pragma unroll
        for (int i = 0; i < PER; ++i) load_weight(i);
    }

    const long long x_at = n / a.H * a.x_stride + n % a.H * a.d, at = n * a.d;
    float h[PER][8];
    {
        Vec<XF32> x[PER];
        Vec<RES == 2> r[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int c = lane + i * TPR;
            if (c < vecs && live) {
                x[i].load(a.x, x_at + c * 8);
                if (RES) r[i].load(a.residual, at + c * 8);
            }
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int c = lane + i * TPR;
            if (c < vecs && live) {
                x[i].values(h[i]);
                if (RES) {
                    float v[8];
                    r[i].values(v);
#pragma unroll
                    for (int j = 0; j < 8; ++j) h[i][j] += v[j];
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) h[i][j] = 0.0f;
            }
        }
    }
    if (RES) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int c = lane + i * TPR;
            if (c < vecs && live) Vec<RES == 2>::store(a.h, at + c * 8, h[i]);
        }
    }
    auto squares = [&](float by) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float v = h[i][j] * by;
                s = fmaf(v, v, s);
            }
        return over_row<TPR, false>(s, part);
    };
    const float sum = squares(1.0f);
    float r = 1.0f / sqrtf(sum * a.inv_d + a.eps), by = 1.0f;
    // Squares that leave the fp32 range: the row is taken times a power of two that brings the larger
    // of its largest magnitude and sqrt(eps) to [1, 2).
    const bool far = !(sum < 0x1p120f) || (sum < 0x1p-80f && a.eps < 0x1p-80f);
    if (TPR < 32 ? __any_sync(0xffffffffu, far) : far) {
        float most = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) most = fmaxf(most, fabsf(h[i][j]));
        most = fmaxf(over_row<TPR, true>(most, part), sqrtf(a.eps));
        const int e = min(max(static_cast<int>(__float_as_uint(most) >> 23) - 127, -126), 126);
        const float pow2 = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        const float mean = squares(pow2) * a.inv_d + a.eps * pow2 * pow2;
        if (far) {
            by = pow2;
            r = mean == 0.0f ? 0.0f : 1.0f / sqrtf(mean);  // eps = 0 and a row of zeros: zeros (a NaN stays one)
        }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int c = lane + i * TPR;
        if (!kWeightEarly) load_weight(i);
        float y[8], f[8];
        if (!a.weight) {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = a.w_offset;
        } else {
            if (a.w_f32) {
                Vec<true> t;
                t.a[0] = w[i][0];
                t.a[1] = w[i][1];
                t.values(f);
            } else {
                unpack8(w[i][0], f);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] += a.w_offset;
        }
        float most = 0.0f;
        const bool on = c < vecs && live;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            y[j] = on ? h[i][j] * by * r * f[j] : 0.0f;
            most = fmaxf(most, fabsf(y[j]));
        }
        if (a.y && on) *reinterpret_cast<uint4 *>(a.y + at + c * 8) = pack8(y);
        if (a.y8) {  // d is a multiple of 64: a group's eight threads are all on or all off
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
            const bool some = most >= 0x1p-100f;
            const float inv = some ? 448.0f / most : 0.0f;
            uint32_t q[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * j] * inv, y[4 * j + 1] * inv), __NV_SATFINITE, __NV_E4M3);
                const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * j + 2] * inv, y[4 * j + 3] * inv), __NV_SATFINITE, __NV_E4M3);
                q[j] = lo | hi << 16;
            }
            if (on) {
                *reinterpret_cast<uint2 *>(a.y8 + at + c * 8) = make_uint2(q[0], q[1]);
                if (c % 8 == 0) a.y8_scale[n * (vecs / 8) + c / 8] = some ? most * (1.0f / 448.0f) : 0.0f;
            }
        }
    }
}

template <int TPR, int PER>
cudaError_t launch(const NormArgs &a, cudaStream_t stream)
{
    const dim3 grid(static_cast<unsigned>((a.rows + kThreads<TPR> / TPR - 1) / (kThreads<TPR> / TPR))), block(kThreads<TPR>);
    const int res = !a.residual ? 0 : a.h_f32 ? 2 : 1;
    if (a.x_f32)
        return res == 0   ? launch_pdl(norm_kernel<TPR, PER, true, 0>, grid, block, 0, stream, a)
               : res == 1 ? launch_pdl(norm_kernel<TPR, PER, true, 1>, grid, block, 0, stream, a)
                          : launch_pdl(norm_kernel<TPR, PER, true, 2>, grid, block, 0, stream, a);
    return res == 0   ? launch_pdl(norm_kernel<TPR, PER, false, 0>, grid, block, 0, stream, a)
           : res == 1 ? launch_pdl(norm_kernel<TPR, PER, false, 1>, grid, block, 0, stream, a)
                      : launch_pdl(norm_kernel<TPR, PER, false, 2>, grid, block, 0, stream, a);
}

}  // namespace

cudaError_t launch_norm(const NormArgs &a, cudaStream_t stream)
{
    const int vecs = a.d / 8;
    // Many rows: a few threads a row, with more vectors in flight each, up to 512 channels, then one vector a thread (32,784 rows
    // of 256 heads' channels: 8.3 us with 16 threads a row, 10.3 with 32; 16,384 rows of 512: 16.5 with 16, 17.6 with 64, 41.8 with
    // 256; 8,192 rows of 1,024: 14.1 with 128, 20.9 with 32; 4,096 of 4,096: 29.5 with 512, 31.3 with 256; 1,024 of 16,384: 34.4 with
    // 512, 38.3 with 1,024, 46.0 with 256).  Few rows: as many threads as a row has vectors (8 rows of 512: 1.6 us with 128, 3.3 with 16).
    // One border for three lengths: 2,047 rows of 128 take 3.6 us with 32 threads and 2.8 with 8, of 256 3.4 with 32 and 3.9 with 16, of
    // 512 4.1 with 128 and 6.8 with 16; 8,192 rows 5.3 and 4.3, 5.4 and 5.3, 11.4 and 9.4.
    const bool few = a.rows < 2048;
    if (vecs <= 8) return launch<8, 1>(a, stream);
    if (few && vecs <= 32) return launch<32, 1>(a, stream);
    if (few && vecs <= 128) return launch<128, 1>(a, stream);
    if (vecs <= 16) return launch<8, 2>(a, stream);
    if (vecs <= 32) return launch<16, 2>(a, stream);
    if (vecs <= 64) return launch<16, 4>(a, stream);
    if (vecs <= 128) return launch<128, 1>(a, stream);
    if (vecs <= 256) return launch<256, 1>(a, stream);
    if (vecs <= 512) return launch<512, 1>(a, stream);
    if (vecs <= 1024) return launch<256, 4>(a, stream);
    return launch<512, 4>(a, stream);
}

}  // namespace lily
