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
// numbers already.  Sums are fp32, scaled and joined a group at a time.  The biases of four groups are one more mma,
// on bf16: their 16 columns are the four sums of x, each as three bf16 numbers that add up to it exactly.
//
// Bound: HBM (0.5625 bytes a weight).  The order of the channels within an mma is free as
// long as both sides agree: a thread takes 16 consecutive channels of a group (8 bytes), so the four
// threads of a row read 32 bytes, and the four groups (a quad) that a warp takes at a time a whole line.  A quad stays in
// registers; as soon as a group of it is used, the same registers are loaded with the next quad's.
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

constexpr int kPitch = 20;      // floats between tokens of a joined tile: the fragment's stores meet no bank twice
constexpr int kTileBytes = 2560;  // a quad of 16 rows in the ring: 128 bytes of codes, 16 of scales, 16 of biases a row
static_assert(kTileBytes >= 4 * 8 * kPitch * 4, "a tile's sums of 32 tokens fit its slot");
constexpr int kMaxSmem = 226 * 1024;

// BYTES of which `n` are read, the rest zeros.
template <int BYTES>
__device__ __forceinline__ void copy(uint32_t to, const void *from, int n = BYTES)
{
    if (BYTES == 16)
        asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(to), "l"(from), "n"(BYTES), "r"(n) : "memory");
}

__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// All but the newest `stages - 2` groups of copies are there.
__device__ __forceinline__ void copy_wait(int stages)
{
    if (stages == 4)
        asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (stages == 3)
        asm volatile("cp.async.wait_group 1;" ::: "memory");
    else
        asm volatile("cp.async.wait_group 0;" ::: "memory");
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, const float (&c)[4])
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%4,%5}, {%6,%7}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(b0), "r"(b1));
}

// Two products at once: (a0, a1) * (b0, b1).
__device__ __forceinline__ void mul2(float &a0, float &a1, float b0, float b1)
{
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\tmul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "+f"(a0), "+f"(a1)
        : "f"(b0), "f"(b1));
}

__device__ __forceinline__ float bf16_of(const uint2 &v, int j)
{
    const uint32_t w = j < 2 ? v.x : v.y;
    return __uint_as_float(j & 1 ? w & 0xFFFF0000u : w << 16);
}

// Shared memory of a CTA that holds `quads` quads of x.
//   xf    [group][word w][token][t] of 16 bytes, the fragments: channels 16 t + 8 w .. + 7 of the group, in the order
//         0 4 1 5 2 6 3 7, the odd ones of which are over 16
//   xs    [quad][NT][t][j][2]: the factors of the quad's four groups for tokens 2 t and 2 t + 1
//   xb    [quad][NT][32 lanes] of 8 bytes: the fragment of the sums
//   part  two of a CTA's sums, [token][row], for its cluster
//   join  two of the warps' sums, where the ring's slots do not hold them
//   ring  [warp][stage][MT] tiles
struct Layout {
    int quads, T, nt, part_bytes, join_bytes, ring_bytes;
    __host__ __device__ int xs() const { return quads * T * 512; }
    __host__ __device__ int xb() const { return xs() + quads * nt * 128; }
    __host__ __device__ int part() const { return xb() + quads * nt * 256; }
    __host__ __device__ int join() const { return part() + 2 * part_bytes; }
    __host__ __device__ int ring() const { return join() + join_bytes; }
    __host__ __device__ int total() const { return ring() + ring_bytes; }
};

// Stages x of this CTA's quads (groups past g_last count as zeros).  Columns of tokens past T take the last token's
// fragments, and factors and sums that are left as they are: a column of an mma's product depends on
// its own token alone, and theirs is not stored.
template <int NT, int THREADS, bool CODES>
__device__ __forceinline__ void stage_x(const MatvecArgs &a, int g_first, int g_last, int quads, uint4 *xf, float *xs, uint16_t *xb)
{
    // eight threads a group of a token, eight channels each; kBatch loads in flight
    constexpr int kBatch = 4;
    const int per_token = quads * 32, total = a.T * per_token;
    for (int i0 = threadIdx.x; i0 - threadIdx.x % 32 < total; i0 += kBatch * THREADS) {
        uint4 raw[kBatch];
        float scale[kBatch];
#pragma unroll
        for (int r = 0; r < kBatch; ++r) {
            const int i = i0 + r * THREADS, t = i / per_token, g = g_first + i % per_token / 8;
            raw[r] = make_uint4(0, 0, 0, 0);
            scale[r] = 0.0f;
            if (i < total && g < g_last) {
                const long long at = t * a.x_stride + g * 64 + i % 8 * 8;
                if (CODES) {
                    const uint2 c = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(a.x) + at);
                    raw[r].x = c.x;
                    raw[r].y = c.y;
                    scale[r] = a.x_scale[static_cast<long long>(t) * (a.K / 64) + g];
                } else {
                    raw[r] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.x) + at);
                }
            }
        }
#pragma unroll
        for (int r = 0; r < kBatch; ++r) {
            const int i = i0 + r * THREADS, t = i / per_token, g = i % per_token / 8, v = i % 8;
            float x[8], by;
            if (CODES) {
                by = 64.0f;  // the largest code, 448, is 28,672
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t w = j < 2 ? raw[r].x : raw[r].y;
                    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> (16 * (j & 1))), __NV_E4M3);
                    const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&h));
                    x[2 * j] = p.x;
                    x[2 * j + 1] = p.y;
                }
            } else {
                const uint32_t u[4] = {raw[r].x, raw[r].y, raw[r].z, raw[r].w};
                float most = 0.0f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[2 * j] = __uint_as_float(u[j] << 16);
                    x[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
                    most = fmaxf(most, fmaxf(fabsf(x[2 * j]), fabsf(x[2 * j + 1])));
                }
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
                // 2^(14 - floor(log2 most)), at most 2^127
                const int e = max(static_cast<int>(__float_as_uint(most) >> 23), 14);
                by = __uint_as_float(static_cast<uint32_t>(268 - min(e, 254)) << 23);
                scale[r] = 1.0f;
            }
            float sum = ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (i >= total) continue;  // whole warps: a token has a multiple of 32 of them
            uint32_t h[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float f = j & 1 ? by * 0.0625f : by;
                const __half2 p = __floats2half2_rn(x[j] * f, x[j + 4] * f);
                h[j] = *reinterpret_cast<const uint32_t *>(&p);
            }
            xf[((g * 2 + v % 2) * a.T + t) * 4 + v / 2] = make_uint4(h[0], h[1], h[2], h[3]);
            if (v == 0) {
                const int q = g / 4, j = g % 4, tile = q * NT + t / 8;
                // the sums are held times 2^-12, the products with codes (2^-24 of them) times 2^12
                xs[tile * 32 + t % 8 / 2 * 8 + j * 2 + t % 2] = scale[r] * 0x1p12f / by;
                float rest = sum * scale[r] * 0x1p-12f;
                uint16_t part[3];
#pragma unroll
                for (int k = 0; k < 3; ++k) {  // what is left of 24 bits after eight more
                    const __nv_bfloat16 p = __float2bfloat16_rn(rest);
                    part[k] = __bfloat16_as_ushort(p);
                    rest -= __bfloat162float(p);
                }
                // columns: (first, second) of groups 0 1 | 2 3, then (third, nothing)
                uint16_t *to = xb + (tile * 32 + t % 8 * 4 + j / 2) * 4 + j % 2;
                to[0] = part[0];
                to[8] = part[1];
                to[2] = part[2];
                to[10] = 0;
            }
        }
    }
}

template <int NT, int MT, int WARPS, bool VEC, bool CODES>
__global__ void __launch_bounds__(WARPS * 32, 1) matvec_kernel(const __grid_constant__ MatvecArgs a)
{
    constexpr int kThreads = WARPS * 32, kStage = MT * kTileBytes;
    constexpr int kTokenFloats = 8 * NT * kPitch;        // a tile's sums
    constexpr bool kOwnJoin = NT == 1;                   // two buffers for the sums, else the slots of the ring
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ const float *joined[WARPS];
    pdl_trigger();
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = a.ranks, rank = ranks > 1 ? static_cast<int>(cluster.block_rank()) : 0;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    // this CTA's quads of K
    const int groups = a.K / 64, all_quads = (groups + 3) / 4;
    const int q_first = all_quads * rank / ranks, quads = all_quads * (rank + 1) / ranks - q_first;
    const int wk = 1 << a.wk_log, wm = WARPS >> a.wk_log;        // warps along K, along rows
    const int k_warp = warp & (wk - 1), m_warp = warp >> a.wk_log;
    const int unit_rows = wm * MT * 16, units = (a.rows + unit_rows - 1) / unit_rows;
    const Layout L{(all_quads + ranks - 1) / ranks, a.T, NT, ranks > 1 ? unit_rows * a.T * 4 : 0, kOwnJoin ? 2 * WARPS * MT * kTokenFloats * 4 : 0, 0};
    uint4 *xf = reinterpret_cast<uint4 *>(smem);
    float *xs = reinterpret_cast<float *>(smem + L.xs());
    uint2 *xb = reinterpret_cast<uint2 *>(smem + L.xb());
    unsigned char *ring = smem + L.ring() + warp * a.stages * kStage;
    const int stride = gridDim.x / ranks;
    int unit = blockIdx.x / ranks;

    // The copies of a quad.  Codes: lane l takes the 16-byte pieces l % 8 of rows l / 8 + 4 i, which go to the place
    // that keeps the reads below (rows 0-3, then 4-7, of a pair of pieces) off each other's banks.  Parameters: lanes 0-15 the
    // scales of a row, 16-31 the biases: one piece of eight bytes, or, where rows are not
    // aligned to that, the three words that hold them.
    const int piece = lane % 8, row_w = lane / 8;
    const long long half = a.K / 2, param_end = static_cast<long long>(a.rows) * groups;
    const uint16_t *params = lane < 16 ? a.s : a.b;
    const uint32_t ring_to = smem_u32(ring), to_w = row_w * 128 + ((piece >> 1 ^ row_w) * 2 + (piece & 1)) * 16, to_p = 2048 + lane * 16;
    int load_row = (unit * wm + m_warp) * (MT * 16), load_q = k_warp;
    uint32_t load_to = ring_to;
    const uint8_t *from_w = a.w + (load_row + row_w) * half + (q_first + load_q) * 128 + piece * 16;
    long long from_p = static_cast<long long>(load_row + lane % 16) * groups + (q_first + load_q) * 4;
    const int row_step = stride * unit_rows;
    const bool works = k_warp < quads;
    auto load = [&]() {
        if (works && load_row < a.rows) {
            const bool whole = load_row + MT * 16 <= a.rows && (VEC || q_first + load_q < all_quads - 1);
            if (whole) {
#pragma unroll
                for (int m = 0; m < MT; ++m) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) copy<16>(load_to + to_w + m * kTileBytes + i * 512, from_w + (16 * m + 4 * i) * half);
                    const uint16_t *p = params + from_p + 16 * m * groups;
                    if (VEC) {
                        copy<8>(load_to + to_p + m * kTileBytes, p);
                    } else {
                        const long long at = from_p + 16 * m * groups;
                        p = params + (at & ~1ll);
                        copy<4>(load_to + to_p + m * kTileBytes, p);
                        copy<4>(load_to + to_p + m * kTileBytes + 4, p + 2);
                        if (at & 1) copy<4>(load_to + to_p + m * kTileBytes + 8, p + 4, 2);  // the row's fourth
                    }
                }
            } else {  // rows past the end and, in the last quad, groups past the end are zeros
                const int pieces = (groups - (q_first + load_q) * 4) * 2;
#pragma unroll
                for (int m = 0; m < MT; ++m) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const bool on = load_row + 16 * m + 4 * i + row_w < a.rows && piece < pieces;
                        copy<16>(load_to + to_w + m * kTileBytes + i * 512, on ? from_w + (16 * m + 4 * i) * half : a.w, on ? 16 : 0);
                    }
                    const bool row_on = load_row + 16 * m + lane % 16 < a.rows;
                    const long long at = from_p + 16 * m * groups;
                    if (VEC) {
                        copy<8>(load_to + to_p + m * kTileBytes, row_on ? params + at : params, row_on ? 8 : 0);
                    } else {
#pragma unroll
                        for (int k = 0; k < 3; ++k) {
                            const long long word = (at & ~1ll) + 2 * k, left = row_on ? param_end - word : 0;
                            copy<4>(load_to + to_p + m * kTileBytes + 4 * k, left > 0 ? params + word : params, left <= 0 ? 0 : left < 2 ? 2 : 4);
                        }
                    }
                }
            }
            load_to += kStage;
            if (load_to == ring_to + a.stages * kStage) load_to = ring_to;
            load_q += wk;
            from_w += wk * 128;
            from_p += wk * 4;
            if (load_q >= quads) {
                from_w += row_step * half - (load_q - k_warp) * 128;
                from_p += static_cast<long long>(row_step) * groups - (load_q - k_warp) * 4;
                load_q = k_warp;
                load_row += row_step;
            }
        }
        copy_commit();
    };
    for (int i = 0; i < a.stages - 1; ++i) load();  // the matrix is never written by a kernel of the library: ahead of the wait
    pdl_wait();
    stage_x<NT, kThreads, CODES>(a, q_first * 4, min((q_first + quads) * 4, groups), quads, xf, xs, reinterpret_cast<uint16_t *>(xb));
    __syncthreads();
    // this lane's fragments of a group: token g of each eight, the last one for tokens past T
    const uint4 *x_lane = xf + g * 4 + t, *x_last = xf + (min(8 * NT - 8 + g, a.T - 1) * 4 + t);
    int slot = 0;
    for (int turn = 0; unit < units; unit += stride, turn ^= 1) {
        float out[NT][MT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) out[n][m][i] = 0.0f;
        unsigned char *tile = ring;
        for (int q = k_warp; q < quads; q += wk) {
            copy_wait(a.stages);
            __syncwarp();  // this quad is there for all lanes, and all are done with the one before
            load();
            tile = ring + slot * kStage;
            slot = slot + 1 == a.stages ? 0 : slot + 1;
            uint2 s[MT][2];
            uint32_t b[MT][2];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const unsigned char *p = tile + m * kTileBytes + 2048 + (g + 8 * h) * 16;
                    if (VEC) {
                        s[m][h] = *reinterpret_cast<const uint2 *>(p);
                        b[m][h] = *reinterpret_cast<const uint32_t *>(p + 256 + t % 2 * 4);
                    } else {
                        const int row = (unit * wm + m_warp) * (MT * 16) + m * 16 + g + 8 * h;
                        const int odd = (row & groups & 1) * 16;  // the first of the row's groups is in the upper half (a quad's first group is even)
                        const uint4 v = *reinterpret_cast<const uint4 *>(p);
                        const uint32_t *c = reinterpret_cast<const uint32_t *>(p + 256 + t % 2 * 4);
                        s[m][h] = make_uint2(__funnelshift_r(v.x, v.y, odd), __funnelshift_r(v.y, v.z, odd));
                        b[m][h] = __funnelshift_r(c[0], c[1], odd);
                        // groups past the row's end hold the next row's parameters, of any value: they count as zeros
                        const int left = groups - (q_first + q) * 4;
                        if (left < 4) {
                            s[m][h].y = left > 2 ? s[m][h].y & 0xFFFFu : 0;
                            s[m][h].x = left > 1 ? s[m][h].x : s[m][h].x & 0xFFFFu;
                            const int mine = left - t % 2 * 2;
                            b[m][h] = mine > 1 ? b[m][h] : mine > 0 ? b[m][h] & 0xFFFFu : 0;
                        }
                    }
                }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint2 x = xb[(q * NT + n) * 32 + lane];
#pragma unroll
                for (int m = 0; m < MT; ++m) mma_bf16(out[n][m], b[m][0], b[m][1], x.x, x.y);
            }
            const float *factors = xs + q * NT * 32 + t * 8;
            const int x_word = a.T * 4;
            int x_at = q * 8 * x_word;
#pragma unroll
            for (int j = 0; j < 4; ++j, x_at += 2 * x_word) {
                uint32_t c[MT][2][2][4];  // [tile][word][half of the word]: codes as a fragment
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint2 w = *reinterpret_cast<const uint2 *>(tile + m * kTileBytes + (g + 8 * h) * 128 + ((j ^ g & 3) * 32 + t * 8));
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint32_t v = k ? w.y : w.x, u = v >> 8;
                            c[m][k][0][h] = v & 0x000F000Fu;
                            c[m][k][0][2 + h] = v & 0x00F000F0u;
                            c[m][k][1][h] = u & 0x000F000Fu;
                            c[m][k][1][2 + h] = u & 0x00F000F0u;
                        }
                    }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint4 *x = (n == NT - 1 ? x_last : x_lane + n * 32) + x_at;
                    const uint4 x0 = x[0], x1 = x[x_word];
                    const float2 f = *reinterpret_cast<const float2 *>(factors + n * 32 + j * 2);
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                        float acc[4];
                        mma_f16(acc, c[m][0][0], x0.x, x0.y, zero);
                        mma_f16(acc, c[m][0][1], x0.z, x0.w, acc);
                        mma_f16(acc, c[m][1][0], x1.x, x1.y, acc);
                        mma_f16(acc, c[m][1][1], x1.z, x1.w, acc);
                        mul2(acc[0], acc[1], f.x, f.y);
                        mul2(acc[2], acc[3], f.x, f.y);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float by = bf16_of(s[m][h], j);
                            out[n][m][2 * h] = fmaf(by, acc[2 * h], out[n][m][2 * h]);
                            out[n][m][2 * h + 1] = fmaf(by, acc[2 * h + 1], out[n][m][2 * h + 1]);
                        }
                    }
                }
            }
        }
        // Join.  A warp's sums, [tile][token][row], go to a buffer, or to the slot that it used last (its first, if it has no part
        // of K).
        float *sums;
        if (kOwnJoin) {
            sums = reinterpret_cast<float *>(smem + L.join()) + (turn * WARPS + warp) * (MT * kTokenFloats);
        } else {
            __syncwarp();
            sums = reinterpret_cast<float *>(tile);
            if (lane == 0) joined[warp] = sums;
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) sums[m * kTokenFloats + (n * 8 + t * 2 + i % 2) * kPitch + i / 2 * 8 + g] = out[n][m][i];
        __syncthreads();
        // A thread takes four rows of a token: items of [token][row / 4].
        const int fours_log = 29 - __clz(unit_rows), items = a.T << fours_log;  // a unit's rows are a power of two
        auto local = [&](int i) {
            const int n = (i & (1 << fours_log) - 1) * 4, first = n / (16 * MT) << a.wk_log;
            const int at = n / 16 % MT * kTokenFloats + (i >> fours_log) * kPitch + n % 16;
            const float *own = reinterpret_cast<const float *>(smem + L.join()) + (turn * WARPS + first) * (MT * kTokenFloats) + at;
            float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
            for (int k = 0; k < wk; ++k) {
                const float4 v = *reinterpret_cast<const float4 *>(kOwnJoin ? own + k * (MT * kTokenFloats) : joined[first + k] + at);
                sum.x += v.x;
                sum.y += v.y;
                sum.z += v.z;
                sum.w += v.w;
            }
            return sum;
        };
        auto store = [&](int i, const float4 &sum) {
            const int row = unit * unit_rows + (i & (1 << fours_log) - 1) * 4;
            const float v[4] = {sum.x * 0x1p12f, sum.y * 0x1p12f, sum.z * 0x1p12f, sum.w * 0x1p12f};
            const long long o = static_cast<long long>(i >> fours_log) * a.rows + row;
            if (a.rows % 4 == 0) {
                if (row >= a.rows) return;
                if (a.out_f32) {
                    *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + o) = make_float4(v[0], v[1], v[2], v[3]);
                } else {
                    const __nv_bfloat162 p = __floats2bfloat162_rn(v[0], v[1]), r = __floats2bfloat162_rn(v[2], v[3]);
                    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + o) =
                        make_uint2(*reinterpret_cast<const uint32_t *>(&p), *reinterpret_cast<const uint32_t *>(&r));
                }
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (row + k < a.rows) {
                        if (a.out_f32)
                            static_cast<float *>(a.out)[o + k] = v[k];
                        else
                            static_cast<__nv_bfloat16 *>(a.out)[o + k] = __float2bfloat16_rn(v[k]);
                    }
            }
        };
        if (ranks == 1) {
            for (int i = threadIdx.x; i < items; i += kThreads) store(i, local(i));
        } else {
            // two buffers: the barrier of the next unit stands between a rank's reads of this one and its next writes
            float4 *part = reinterpret_cast<float4 *>(smem + L.part() + turn * L.part_bytes);
            for (int i = threadIdx.x; i < items; i += kThreads) part[i] = local(i);
            cluster.sync();
            for (int i = threadIdx.x + rank * kThreads; i < items; i += kThreads * ranks) {
                float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
                for (int r = 0; r < ranks; ++r) {
                    const float4 v = cluster.map_shared_rank(part, r)[i];
                    sum.x += v.x;
                    sum.y += v.y;
                    sum.z += v.z;
                    sum.w += v.w;
                }
                store(i, sum);
            }
        }
        if (!kOwnJoin) __syncthreads();  // the slots may be filled again
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (ranks > 1) cluster.sync();  // nobody leaves while another reads
}

template <int NT, int MT, int WARPS, bool VEC, bool CODES>
cudaError_t launch(MatvecArgs a, const Layout &L, int unit_rows, int num_sms, cudaStream_t stream)
{
    const int units = (a.rows + unit_rows - 1) / unit_rows;
    auto kernel = matvec_kernel<NT, MT, WARPS, VEC, CODES>;
    cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void *>(kernel), L.total());
    if (e != cudaSuccess) return e;
    const int clusters = std::min(units, std::max(1, num_sms / a.ranks));
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(clusters * a.ranks);
    cfg.blockDim = dim3(WARPS * 32);
    cfg.dynamicSmemBytes = L.total();
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.ranks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.ranks > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int NT, int MT, int WARPS>
cudaError_t launch(MatvecArgs a, int num_sms, cudaStream_t stream)
{
    const int quads = (a.K / 64 + 3) / 4;
    // CTAs of a cluster along K: as few as leave the ring enough stages beside x
    Layout L{};
    int unit_rows = 0;
    for (a.ranks = 1;; a.ranks *= 2) {
        const int per = (quads + a.ranks - 1) / a.ranks;
        a.wk_log = 0;
        while ((2 << a.wk_log) <= WARPS && (2 << a.wk_log) <= per) ++a.wk_log;
        unit_rows = (WARPS >> a.wk_log) * MT * 16;
        L = Layout{per, a.T, NT, a.ranks > 1 ? unit_rows * a.T * 4 : 0, NT == 1 ? 2 * WARPS * MT * 8 * NT * kPitch * 4 : 0, 0};
        a.stages = std::min(4, (kMaxSmem - L.total()) / (WARPS * MT * kTileBytes));
        if (a.stages >= (NT >= 3 ? 2 : 3)) break;
        if (a.ranks == 8) {  // the tokens do not fit: in two calls
            MatvecArgs b = a;
            b.T = a.T / 2;
            a.T -= b.T;
            a.x = static_cast<const char *>(a.x) + b.T * a.x_stride * (a.x_scale ? 1 : 2);
            if (a.x_scale) a.x_scale += b.T * (a.K / 64);
            a.out = static_cast<char *>(a.out) + b.T * static_cast<size_t>(a.rows) * (a.out_f32 ? 4 : 2);
            const cudaError_t e = launch_matvec(b, num_sms, stream);
            return e != cudaSuccess ? e : launch_matvec(a, num_sms, stream);
        }
    }
    L.ring_bytes = a.stages * WARPS * MT * kTileBytes;
    const bool vec = a.K % 256 == 0;
    if (a.x_scale)
        return vec ? launch<NT, MT, WARPS, true, true>(a, L, unit_rows, num_sms, stream) : launch<NT, MT, WARPS, false, true>(a, L, unit_rows, num_sms, stream);
    return vec ? launch<NT, MT, WARPS, true, false>(a, L, unit_rows, num_sms, stream) : launch<NT, MT, WARPS, false, false>(a, L, unit_rows, num_sms, stream);
}

}  // namespace

cudaError_t launch_matvec(const MatvecArgs &a, int num_sms, cudaStream_t stream)
{
    if (a.T <= 8) return launch<1, 1, 16>(a, num_sms, stream);
    if (a.T <= 16) return launch<2, 2, 8>(a, num_sms, stream);
    if (a.T <= 24) return launch<3, 2, 8>(a, num_sms, stream);
    return launch<4, 2, 8>(a, num_sms, stream);
}

}  // namespace lily
