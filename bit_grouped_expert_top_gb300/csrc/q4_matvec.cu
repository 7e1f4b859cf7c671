// A few tokens times a matrix of 4-bit codes, for sm_103a:
//   out[t][n] = sum_k x[t][k] (q[n][k] scale[n][k/64] + bias[n][k/64]),   1 <= T <= 32.
//
// Per group g of 64 channels, with c = q[n][k]:
//   out[t][n] = sum_g scale[n][g] (sum_k c x[t][k]) + bias[n][g] (sum_k x[t][k])
// The inner products run on the tensor cores (mma.sync m16n8k16, the 16 rows a tile of the matrix,
// the 8 columns tokens), with nothing rebuilt: a code in the low bits of an fp16 pattern is
// the number code * 2^-24 (bits 0-3) or code * 2^-20 (bits 4-7), so eight codes are four
// masks and a shift.  x is brought to fp16 by a power of two for each token and group that puts
// the group's largest magnitude into [2^14, 2^15): its eight significant bits survive down to 2^-31 of
// that magnitude, and what is smaller is off by at most 2^-36 of it.  e4m3 tokens are fp16
// numbers already.  Sums are fp32, scaled and joined a group at a time.
//
// Bound: HBM (0.5625 bytes a weight).  The order of the channels within an mma is free as
// long as both sides agree: a thread takes 16 consecutive channels of a group (8 bytes), so the four
// threads of a row read 32 bytes, and the four groups that a warp takes at a time a whole line.
// The warps of a CTA share a row tile's K and join their sums in shared memory; a K whose x does
// not fit is cut over the CTAs of a cluster, joined through distributed shared memory.
#include <algorithm>
#include <cstdint>

#include <cooperative_groups.h>
#include <cuda_fp8.h>

#include "lily_internal.h"

namespace lily {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kPitch = 20;  // floats between tokens of a joined tile: the fragment's stores meet no bank twice

__device__ __forceinline__ uint2 ld_w2(const void *p)
{
    uint2 v;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}

__device__ __forceinline__ uint32_t ld_w1(const uint16_t *p)
{
    uint16_t v;
    asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(v) : "l"(p));
    return v;
}

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// What a lane holds of four groups of MT row tiles: rows g and g + 8 of each (g = lane / 4), channels
// [16 t, 16 t + 16) of each group (t = lane % 4); the scales and biases of the four groups.
template <int MT>
struct Quad {
    uint2 w[MT][2][4], s[MT][2], b[MT][2];
};

template <int MT, bool VEC>  // VEC: a row's scales of four groups are one aligned load
__device__ __forceinline__ void load_quad(Quad<MT> &f, const MatvecArgs &a, int row0, int g0, int g_end, int lane)
{
    const int groups = a.K / 64;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const long long row = min(row0 + 16 * m + 8 * h + lane / 4, a.rows - 1);
            const uint8_t *w = a.w + row * (a.K / 2) + g0 * 32 + lane % 4 * 8;
#pragma unroll
            for (int j = 0; j < 4; ++j) f.w[m][h][j] = g0 + j < g_end ? ld_w2(w + 32 * j) : make_uint2(0, 0);
            const uint16_t *s = a.s + row * groups + g0, *b = a.b + row * groups + g0;
            if (VEC) {
                const bool on = g0 < g_end;
                f.s[m][h] = on ? ld_w2(s) : make_uint2(0, 0);
                f.b[m][h] = on ? ld_w2(b) : make_uint2(0, 0);
            } else {
                uint32_t v[2][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[0][j] = g0 + j < g_end ? ld_w1(s + j) : 0;
                    v[1][j] = g0 + j < g_end ? ld_w1(b + j) : 0;
                }
                f.s[m][h] = make_uint2(v[0][0] | v[0][1] << 16, v[0][2] | v[0][3] << 16);
                f.b[m][h] = make_uint2(v[1][0] | v[1][1] << 16, v[1][2] | v[1][3] << 16);
            }
        }
}

__device__ __forceinline__ float bf16_of(const uint2 &v, int j)
{
    const uint32_t w = j < 2 ? v.x : v.y;
    return __uint_as_float(j & 1 ? w & 0xFFFF0000u : w << 16);
}

// x in shared memory, as the lanes take it: xf [NT][groups][2][32] of 16 bytes (word w of a group's channels
// 16 t + 8 w .. + 7 of token g, in the order 0 4 1 5 2 6 3 7, the odd ones of which are over 16), and
// xs [groups][8 NT] (the group's factor, sum of x times 2^-24).
template <int NT, bool CODES>
__device__ __forceinline__ void stage_x(const MatvecArgs &a, int g_first, int n_groups, uint4 *xf, float2 *xs)
{
    // eight threads a group of a token, eight channels each
    const int total = 8 * NT * n_groups * 8;
    for (int i = threadIdx.x; i < total; i += kThreads) {
        const int v = i % 8, g = i / 8 % n_groups, t = i / 8 / n_groups;
        const bool on = t < a.T;
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = 0.0f;
        float factor = 0.0f;
        const long long at = static_cast<long long>(t) * a.x_stride + (g_first + g) * 64 + v * 8;
        float by;
        if (CODES) {
            by = 64.0f;  // the largest code, 448, is 28,672
            if (on) {
                const uint2 c = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(a.x) + at);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t w = j < 2 ? c.x : c.y;
                    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> (16 * (j & 1))), __NV_E4M3);
                    const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&h));
                    x[2 * j] = p.x;
                    x[2 * j + 1] = p.y;
                }
                factor = a.x_scale[static_cast<long long>(t) * (a.K / 64) + g_first + g];
            }
        } else {
            float most = 0.0f;
            if (on) {
                const uint4 c = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.x) + at);
                const uint32_t u[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[2 * j] = __uint_as_float(u[j] << 16);
                    x[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) most = fmaxf(most, fabsf(x[j]));
            }
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
            // 2^(14 - floor(log2 most)), at most 2^127
            const int e = max(static_cast<int>(__float_as_uint(most) >> 23), 14);
            by = __uint_as_float(static_cast<uint32_t>(268 - min(e, 254)) << 23);
            factor = 1.0f;
        }
        float sum = ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float sixteenth = by * 0.0625f;
        uint32_t h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float f = j & 1 ? sixteenth : by;
            const __half2 p = __floats2half2_rn(x[j] * f, x[j + 4] * f);
            h[j] = *reinterpret_cast<const uint32_t *>(&p);
        }
        xf[((t / 8 * n_groups + g) * 2 + v % 2) * 32 + t % 8 * 4 + v / 2] = make_uint4(h[0], h[1], h[2], h[3]);
        if (v == 0) xs[g * 8 * NT + t] = make_float2(factor / by, sum * factor * 0x1p-24f);
    }
}

template <int NT, int MT>
__device__ __forceinline__ void use_quad(const Quad<MT> &f, float (&out)[NT][MT][4], int g0, int n_groups, const uint4 *xf,
                                         const float2 *xs, int lane)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (g0 + j >= n_groups) break;
        uint32_t w[MT][2][2][4];  // [tile][word][row half][pair]
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t v = k ? f.w[m][h][j].y : f.w[m][h][j].x, u = v >> 8;
                    w[m][k][h][0] = v & 0x000F000Fu;
                    w[m][k][h][1] = v & 0x00F000F0u;
                    w[m][k][h][2] = u & 0x000F000Fu;
                    w[m][k][h][3] = u & 0x00F000F0u;
                }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float acc[MT][4];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][i] = 0.0f;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint4 x = xf[((t * n_groups + g0 + j) * 2 + k) * 32 + lane];
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    mma(acc[m], w[m][k][0][0], w[m][k][1][0], w[m][k][0][1], w[m][k][1][1], x.x, x.y);
                    mma(acc[m], w[m][k][0][2], w[m][k][1][2], w[m][k][0][3], w[m][k][1][3], x.z, x.w);
                }
            }
            const float4 p = *reinterpret_cast<const float4 *>(xs + (g0 + j) * 8 * NT + t * 8 + lane % 4 * 2);
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float s = bf16_of(f.s[m][h], j), b = bf16_of(f.b[m][h], j);
                    out[t][m][2 * h] = fmaf(b, p.y, fmaf(s, acc[m][2 * h] * p.x, out[t][m][2 * h]));
                    out[t][m][2 * h + 1] = fmaf(b, p.w, fmaf(s, acc[m][2 * h + 1] * p.z, out[t][m][2 * h + 1]));
                }
        }
    }
}

template <int NT, int MT>
struct Layout {  // shared memory of a CTA that holds n_groups groups of x
    int n_groups;
    __host__ __device__ size_t xf() const { return static_cast<size_t>(NT) * n_groups * 2 * 32 * 16; }
    __host__ __device__ size_t xs() const { return static_cast<size_t>(n_groups) * 8 * NT * 8; }
    static constexpr size_t kJoin = static_cast<size_t>(kWarps) * MT * 8 * NT * kPitch * 4;
    __host__ __device__ size_t total() const { return xf() + xs() + kJoin; }
};

template <int NT, int MT, bool VEC, bool CODES>
__global__ void __launch_bounds__(kThreads) matvec_kernel(const __grid_constant__ MatvecArgs a)
{
    extern __shared__ __align__(16) unsigned char smem[];
    pdl_trigger();
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    // this CTA's groups, in whole quads of K's: [4 Q r / R, 4 Q (r + 1) / R)
    const int groups = a.K / 64, quads = (groups + 3) / 4;
    const int g_first = quads * rank / ranks * 4, g_last = min(quads * (rank + 1) / ranks * 4, groups);
    const int n_groups = g_last - g_first, my_quads = (n_groups + 3) / 4;
    const Layout<NT, MT> L{(quads + ranks - 1) / ranks * 4};
    uint4 *xf = reinterpret_cast<uint4 *>(smem);
    float2 *xs = reinterpret_cast<float2 *>(smem + L.xf());
    float *join = reinterpret_cast<float *>(smem + L.xf() + L.xs());

    const int wk = 1 << a.wk_log, wm = kWarps >> a.wk_log;        // warps along K, along rows
    const int k_warp = warp & (wk - 1), m_warp = warp >> a.wk_log;
    const int unit_rows = wm * MT * 16, units = (a.rows + unit_rows - 1) / unit_rows;
    const int stride = gridDim.x / ranks;
    int unit = blockIdx.x / ranks;
    Quad<MT> cur;
    auto load = [&](int u, int q) {
        load_quad<MT, VEC>(cur, a, u * unit_rows + m_warp * MT * 16, g_first + q * 4, q < my_quads ? g_last : 0, lane);
    };
    load(unit, k_warp);  // the matrix is never written by a kernel of the library: ahead of the wait
    pdl_wait();
    stage_x<NT, CODES>(a, g_first, n_groups, xf, xs);
    __syncthreads();
    for (; unit < units; unit += stride) {
        float out[NT][MT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) out[t][m][i] = 0.0f;
        for (int q = k_warp; q < my_quads; q += wk) {
            const Quad<MT> now = cur;
            if (q + wk < my_quads)
                load(unit, q + wk);
            else if (unit + stride < units)
                load(unit + stride, k_warp);
            use_quad<NT, MT>(now, out, q * 4, n_groups, xf, xs, lane);
        }
        // join: [warp][tile][token][row]
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    join[((warp * MT + m) * 8 * NT + t * 8 + lane % 4 * 2 + i % 2) * kPitch + i / 2 * 8 + lane / 4] = out[t][m][i];
        if (ranks > 1)
            cluster.sync();
        else
            __syncthreads();
        const int items = unit_rows * a.T;  // of (token, row of the unit), rows fastest; a rank takes every ranks-th block of 16
        for (int i = threadIdx.x; i < items; i += kThreads) {
            const int n = i % unit_rows, t = i / unit_rows;
            if (ranks > 1 && (i / 16) % ranks != rank) continue;
            const int mw = n / (16 * MT), m = n / 16 % MT;
            const int at = (((mw << a.wk_log) * MT + m) * 8 * NT + t) * kPitch + n % 16;
            float sum = 0.0f;
            for (int r = 0; r < ranks; ++r) {
                const float *from = ranks > 1 ? cluster.map_shared_rank(join, r) : join;
                for (int k = 0; k < wk; ++k) sum += from[at + k * MT * 8 * NT * kPitch];
            }
            const long long row = static_cast<long long>(unit) * unit_rows + n;
            if (row < a.rows) {
                sum *= 0x1p24f;
                const long long o = static_cast<long long>(t) * a.rows + row;
                if (a.out_f32)
                    static_cast<float *>(a.out)[o] = sum;
                else
                    static_cast<__nv_bfloat16 *>(a.out)[o] = __float2bfloat16_rn(sum);
            }
        }
        if (ranks > 1)
            cluster.sync();
        else
            __syncthreads();
    }
}

template <int NT, int MT, bool VEC, bool CODES>
cudaError_t launch(MatvecArgs a, int ranks, int num_sms, cudaStream_t stream)
{
    const int quads = (a.K / 64 + 3) / 4, per = (quads + ranks - 1) / ranks;
    a.wk_log = per >= 8 ? 3 : per >= 4 ? 2 : per >= 2 ? 1 : 0;
    const Layout<NT, MT> L{per * 4};
    const size_t smem = L.total();
    auto kernel = matvec_kernel<NT, MT, VEC, CODES>;
    cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void *>(kernel), static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    const int unit_rows = (kWarps >> a.wk_log) * MT * 16, units = (a.rows + unit_rows - 1) / unit_rows;
    const int per_sm = std::max(1, std::min<int>(3, 220 * 1024 / static_cast<int>(smem + 1024)));
    const int clusters = std::min(units, std::max(1, num_sms * per_sm / ranks));
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(clusters * ranks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ranks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ranks > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int NT, int MT>
cudaError_t launch(const MatvecArgs &a, int num_sms, cudaStream_t stream)
{
    // CTAs of a cluster along K: as many as x needs shared memory for
    int ranks = 1;
    while (ranks < 8 && NT * ((a.K + ranks - 1) / ranks) > 8192) ranks *= 2;
    const bool vec = a.K % 256 == 0;
    if (a.x_scale)
        return vec ? launch<NT, MT, true, true>(a, ranks, num_sms, stream) : launch<NT, MT, false, true>(a, ranks, num_sms, stream);
    return vec ? launch<NT, MT, true, false>(a, ranks, num_sms, stream) : launch<NT, MT, false, false>(a, ranks, num_sms, stream);
}

}  // namespace

cudaError_t launch_matvec(const MatvecArgs &a, int num_sms, cudaStream_t stream)
{
    if (a.T <= 8) return launch<1, 1>(a, num_sms, stream);
    if (a.T <= 16) return launch<2, 1>(a, num_sms, stream);
    return launch<4, 2>(a, num_sms, stream);
}

}  // namespace lily
