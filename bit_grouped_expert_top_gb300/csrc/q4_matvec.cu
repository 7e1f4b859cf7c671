// A few tokens times a matrix of 4-bit codes, for sm_103a:
//   out[t][n] = sum_k x[t][k] (q[n][k] scale[n][k/64] + bias[n][k/64]),   1 <= T <= 32.
//
// Per group g of 64 channels, with c = q[n][k]:
//   out[t][n] = sum_g scale[n][g] (sum_k c x[t][k]) + bias[n][g] (sum_k x[t][k])
// The inner products run on the tensor cores (mma.sync m16n8k16 on fp16, the 16 rows a tile of the matrix, the 8
// columns tokens), with nothing rebuilt: a code in the low bits of an fp16 pattern is the number code * 2^-24 (bits 0-3) or
// code * 2^-20 (bits 4-7), so eight codes are four masks and a shift.  (The e4m3 form of mma.sync would take them with two
// masks, but here it is slower: 27 cycles a sub-core for twice the channels against 10, operands that change.)  bf16
// tokens are taken times a power of two that brings the largest of the 256 channels of a token that a warp holds into
// [2^14, 2^15): their eight significant bits survive down to 2^-31 of that largest magnitude, and what is smaller is off by at
// most 2^-36 of it.  The norm's e4m3 tokens are fp16 numbers already.  Sums are fp32, scaled and joined a group at a
// time.  The biases of four groups are one more mma, on bf16: their 16 columns are the four sums of x, each as three
// bf16 numbers that add up to it exactly.
//
// Bound: HBM (0.5625 bytes a weight).  The order of the channels within an mma is free as
// long as both sides agree: a thread takes 16 consecutive channels of a group.  A warp keeps the fragments of its four groups
// (a quad: 256 channels) of x in registers for the whole call and takes the rows' pieces of that quad past them, one tile
// of 16 rows after another, through a ring of asynchronous copies of its own; the warps of
// a CTA share a row's K and join their sums in shared memory.  A K of more quads than a CTA has warps for is cut over
// the CTAs of a cluster, which join through distributed shared memory.
#include <algorithm>
#include <cstdint>

#include <cooperative_groups.h>
#include <cuda_fp8.h>

#include "lily_internal.h"

namespace lily {
namespace {

namespace cg = cooperative_groups;

constexpr int kPitch = 20;        // floats between tokens of a joined tile: the fragment's stores meet no bank twice
constexpr int kTileBytes = 2560;  // a quad of 16 rows in the ring: 128 bytes of codes, 16 of scales, 16 of biases a row
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

// All but the newest `STAGES - 2` groups of copies are there.
template <int STAGES>
__device__ __forceinline__ void copy_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, const float (&c)[4])
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0, uint32_t b1, const float (&c)[4])
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%4,%5}, {%6,%7}, {%8,%9,%10,%11};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
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

__device__ __forceinline__ uint32_t f16x2(float a, float b)
{
    const __half2 p = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&p);
}

__device__ __forceinline__ float2 of_e4m3x2(uint32_t v)
{
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v), __NV_E4M3);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// A lane's part of a quad of x (lane 4 g + t): channels [16 t, 16 t + 16) of the quad's four groups of tokens 8 n + g, and
// the fragment of their sums.
template <int NT, bool CODES>
struct Tokens {
    uint32_t x[NT][4][8];             // [4 w + ..]: word w's channels 0 4, 1 5, 2 6, 3 7, the odd pairs over 16
    uint32_t sums[NT][2];
    float factor[CODES ? 1 : NT][2];  // bf16: of tokens 2 t and 2 t + 1
};

// Loads a quad of x (its groups from g_last on, and tokens past T, as zeros).  CODES: leaves the factors of its groups for
// tokens 2 t and 2 t + 1, [n][t][j][2], at `factors`.
template <int NT, bool CODES>
__device__ __forceinline__ void load_tokens(Tokens<NT, CODES> &to, const MatvecArgs &a, int g_first, int g_last, int lane, float *factors)
{
    const int t = lane % 4;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int token = 8 * n + lane / 4;
        uint4 raw[4][2];
        float scale[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            raw[j][0] = raw[j][1] = make_uint4(0, 0, 0, 0);
            scale[j] = 0.0f;
            if (token < a.T && g_first + j < g_last) {
                const long long at = token * a.x_stride + (g_first + j) * 64 + 16 * t;
                if (CODES) {
                    raw[j][0] = *reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(a.x) + at);
                    scale[j] = a.x_scale[static_cast<long long>(token) * (a.K / 64) + g_first + j];
                } else {
                    const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.x) + at);
                    raw[j][0] = p[0];
                    raw[j][1] = p[1];
                }
            }
        }
        float sum[4], by = 64.0f;  // the largest code, 448, is 28,672
        if (!CODES) {
            float most = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t u[8] = {raw[j][0].x, raw[j][0].y, raw[j][0].z, raw[j][0].w, raw[j][1].x, raw[j][1].y, raw[j][1].z, raw[j][1].w};
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    most = fmaxf(most, fmaxf(fabsf(__uint_as_float(u[i] << 16)), fabsf(__uint_as_float(u[i] & 0xFFFF0000u))));
            }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
            // x times 2^(14 - e), e = floor(log2 most) in [-113, 127]
            const int e = min(max(static_cast<int>(__float_as_uint(most) >> 23) - 127, -113), 127);
            const float factor = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
            by = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
#pragma unroll
            for (int i = 0; i < 2; ++i) to.factor[CODES ? 0 : n][i] = __shfl_sync(0xffffffffu, factor, (2 * t + i) * 4);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t u[8] = {raw[j][0].x, raw[j][0].y, raw[j][0].z, raw[j][0].w, raw[j][1].x, raw[j][1].y, raw[j][1].z, raw[j][1].w};
            float x[16];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 p = CODES ? of_e4m3x2(u[i / 2] >> (16 * (i & 1)) & 0xFFFFu)
                                       : make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u));
                x[2 * i] = p.x * by;
                x[2 * i + 1] = p.y * by;
            }
            sum[j] = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) sum[j] += x[i];
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float f = i & 1 ? 0.0625f : 1.0f;
                    to.x[n][j][4 * w + i] = f16x2(x[8 * w + i] * f, x[8 * w + i + 4] * f);
                }
            // products with codes are times 2^-24 and `by`
            if (CODES && t == 0) factors[((n * 4 + lane / 8) * 4 + j) * 2 + lane / 4 % 2] = scale[j] * 0x1p18f;
        }
        uint32_t part[4][3];  // the groups' sums as three bf16 numbers
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], o);
            float rest = sum[j] * (CODES ? scale[j] * 0.015625f : 0x1p-24f);
#pragma unroll
            for (int k = 0; k < 3; ++k) {  // what is left of 24 bits after eight more
                const __nv_bfloat16 p = __float2bfloat16_rn(rest);
                part[j][k] = __bfloat16_as_ushort(p);
                rest -= __bfloat162float(p);
            }
        }
        // columns 2 t, 2 t + 1: the first numbers of groups 0 1 | 2 3, then the second; columns 8 + 2 t: the third, nothing
        const int j = t % 2 * 2;
        uint32_t pair[3];
#pragma unroll
        for (int k = 0; k < 3; ++k) pair[k] = j ? part[2][k] | part[3][k] << 16 : part[0][k] | part[1][k] << 16;
        to.sums[n][0] = t < 2 ? pair[0] : pair[1];
        to.sums[n][1] = t < 2 ? pair[2] : 0;
    }
}

// Stages of a warp's ring: what shared memory leaves beside the joins, for two tiles a unit.
template <int NT, int WARPS>
constexpr int kStages = WARPS == 16 ? (NT == 1 ? 4 : 3) : 6;

// Shared memory: the factors [warp][QPW][NT][4][4][2]; for a cluster two of a CTA's sums, [token][row]; two of the warps' sums,
// [tile of the unit][warp][token][row]; the ring [warp][stage] of tiles.
struct Layout {
    int warps, quads_a_warp, nt, part_bytes, tiles_log, stages;
    __host__ __device__ int part() const { return warps * quads_a_warp * nt * 128; }
    __host__ __device__ int join() const { return part() + 2 * part_bytes; }
    __host__ __device__ int join_bytes() const { return (warps * 8 * nt * kPitch * 4) << tiles_log; }
    __host__ __device__ int ring() const { return join() + 2 * join_bytes(); }
    __host__ __device__ int total() const { return ring() + warps * stages * kTileBytes; }
};

template <int NT, int QPW, int WARPS, bool VEC, bool CODES>
__global__ void __launch_bounds__(WARPS * 32, 1) matvec_kernel(const __grid_constant__ MatvecArgs a)
{
    constexpr int kThreads = WARPS * 32, kSums = 8 * NT * kPitch, kS = kStages<NT, WARPS>;
    extern __shared__ __align__(128) unsigned char smem[];
    pdl_trigger();
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = a.ranks, rank = ranks > 1 ? static_cast<int>(cluster.block_rank()) : 0;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    // this CTA's quads of K; those of this warp are q_first + k_warp + i wk
    const int groups = a.K / 64, all_quads = (groups + 3) / 4;
    const int q_first = all_quads * rank / ranks, quads = all_quads * (rank + 1) / ranks - q_first;
    const int wk = 1 << a.wk_log, wm = WARPS >> a.wk_log, wm_log = 31 - __clz(wm);  // warps along K, along rows
    const int k_warp = warp & (wk - 1), m_warp = warp >> a.wk_log;
    const int my_quads = k_warp < quads ? (quads - k_warp + wk - 1) >> a.wk_log : 0;  // at most QPW
    // a step is a tile of each of the warps along rows; a unit, between joins, 2^tiles_log steps; a cluster takes steps that follow one another
    const int tiles_log = a.tiles_log, step_rows = wm * 16, unit_rows = step_rows << tiles_log;
    const int cluster_id = blockIdx.x / ranks;
    int step = cluster_id * a.steps_each + min(cluster_id, a.steps_more);
    const int last_step = step + a.steps_each + (cluster_id < a.steps_more ? 1 : 0);
    const Layout L{WARPS, QPW, NT, ranks > 1 ? unit_rows * a.T * 4 : 0, tiles_log, kS};
    float *factors = reinterpret_cast<float *>(smem) + warp * (QPW * NT * 32);
    unsigned char *ring = smem + L.ring() + warp * kS * kTileBytes;

    // The copies of a tile.  Codes: lane l takes the 16-byte pieces l % 8 of rows l / 8 + 4 i, which go to the place
    // that keeps the reads below (rows 0-3, then 4-7, of a pair of pieces) off each other's banks.  Parameters: lanes 0-15 the
    // scales of a row, 16-31 the biases: one piece of eight bytes, or, where rows are not
    // aligned to that, the three words that hold them.
    const int piece = lane % 8, row_w = lane / 8;
    const long long half = a.K / 2, param_end = static_cast<long long>(a.rows) * groups;
    const uint16_t *params = lane < 16 ? a.s : a.b;
    const uint32_t ring_to = smem_u32(ring), to_w = row_w * 128 + ((piece >> 1 ^ row_w) * 2 + (piece & 1)) * 16, to_p = 2048 + lane * 16;
    const long long w_step = step_rows * half;
    const int p_step = step_rows * groups, last_row = min(last_step * step_rows, a.rows);  // past this cluster's rows
    int load_row = step * step_rows + m_warp * 16, load_i = 0;
    uint32_t load_to = ring_to;
    const uint8_t *from_w = a.w + (load_row + row_w) * half + (q_first + k_warp) * 128 + piece * 16;
    long long from_p = static_cast<long long>(load_row + lane % 16) * groups + (q_first + k_warp) * 4;
    auto load = [&]() {
        if (my_quads > 0 && load_row < last_row) {
            const int q = q_first + k_warp + (load_i << a.wk_log);
            const uint8_t *w = from_w + load_i * (wk * 128);
            const long long at = from_p + load_i * (wk * 4);
            if (load_row + 16 <= a.rows && (VEC || q < all_quads - 1)) {
#pragma unroll
                for (int i = 0; i < 4; ++i) copy<16>(load_to + to_w + i * 512, w + 4 * i * half);
                if (VEC) {
                    copy<8>(load_to + to_p, params + at);
                } else {
                    const uint16_t *p = params + (at & ~1ll);
                    copy<4>(load_to + to_p, p);
                    copy<4>(load_to + to_p + 4, p + 2);
                    if (at & 1) copy<4>(load_to + to_p + 8, p + 4, 2);  // the row's fourth
                }
            } else {  // rows past the end and, in the last quad, groups past the end are zeros
                const int pieces = (groups - q * 4) * 2;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool on = load_row + 4 * i + row_w < a.rows && piece < pieces;
                    copy<16>(load_to + to_w + i * 512, on ? w + 4 * i * half : a.w, on ? 16 : 0);
                }
                const bool on = load_row + lane % 16 < a.rows;
                if (VEC) {
                    copy<8>(load_to + to_p, on ? params + at : params, on ? 8 : 0);
                } else {
#pragma unroll
                    for (int k = 0; k < 3; ++k) {
                        const long long word = (at & ~1ll) + 2 * k, left = on ? param_end - word : 0;
                        copy<4>(load_to + to_p + 4 * k, left > 0 ? params + word : params, left <= 0 ? 0 : left < 2 ? 2 : 4);
                    }
                }
            }
            load_to += kTileBytes;
            if (load_to == ring_to + kS * kTileBytes) load_to = ring_to;
            if (QPW == 1 || ++load_i == my_quads) {
                load_row += step_rows;
                from_w += w_step;
                from_p += p_step;
                load_i = 0;
            }
        }
        copy_commit();
    };
    for (int i = 0; i < kS - 1; ++i) load();  // the matrix is never written by a kernel of the library: ahead of the wait
    pdl_wait();
    Tokens<NT, CODES> x[QPW];
#pragma unroll
    for (int i = 0; i < QPW; ++i)
        if (i < my_quads)
            load_tokens<NT, CODES>(x[i], a, (q_first + k_warp + (i << a.wk_log)) * 4, groups, lane, factors + i * NT * 32);
    __syncwarp();
    const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const unsigned char *tile = ring;
    const unsigned char *const ring_end = ring + kS * kTileBytes;
    const int fours_log = 29 - __clz(unit_rows), items = a.T << fours_log;  // items of the join: [token][row / 4]
    for (int turn = 0; step < last_step; turn ^= 1) {
        float *sums = reinterpret_cast<float *>(smem + L.join() + turn * L.join_bytes()) + warp * kSums + t * (2 * kPitch) + g;
        const int first_row = step * step_rows, steps = min(1 << tiles_log, last_step - step);
        for (int r = 0; r < steps; ++r, ++step, sums += WARPS * kSums) {
            const int row0 = step * step_rows + m_warp * 16;
            float out[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) out[n][i] = 0.0f;
#pragma unroll
            for (int i = 0; i < QPW; ++i) {
                if (i >= my_quads || row0 >= a.rows) break;
                copy_wait<kS>();
                __syncwarp();  // this tile is there for all lanes, and all are done with the one before
                load();
                uint2 s[2];
                uint32_t b[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const unsigned char *p = tile + 2048 + (g + 8 * h) * 16;
                    if (VEC) {
                        s[h] = *reinterpret_cast<const uint2 *>(p);
                        b[h] = *reinterpret_cast<const uint32_t *>(p + 256 + t % 2 * 4);
                    } else {
                        // the first of the row's groups may be in the upper half of its word (a quad's first group is even)
                        const int odd = (row0 + g + 8 * h & groups & 1) * 16;
                        const uint4 v = *reinterpret_cast<const uint4 *>(p);
                        const uint32_t *c = reinterpret_cast<const uint32_t *>(p + 256 + t % 2 * 4);
                        s[h] = make_uint2(__funnelshift_r(v.x, v.y, odd), __funnelshift_r(v.y, v.z, odd));
                        b[h] = __funnelshift_r(c[0], c[1], odd);
                        // groups past the row's end hold the next row's parameters, of any value: they count as zeros
                        const int left = groups - (q_first + k_warp + (i << a.wk_log)) * 4;
                        if (left < 4) {
                            s[h].y = left > 2 ? s[h].y & 0xFFFFu : 0;
                            s[h].x = left > 1 ? s[h].x : s[h].x & 0xFFFFu;
                            const int mine = left - t % 2 * 2;
                            b[h] = mine > 1 ? b[h] : mine > 0 ? b[h] & 0xFFFFu : 0;
                        }
                    }
                }
                float part[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_bf16(part[n], b[0], b[1], x[i].sums[n][0], x[i].sums[n][1], zero);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t c[4][4];  // [word and half of it]: codes as a fragment
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint2 w = *reinterpret_cast<const uint2 *>(tile + (g + 8 * h) * 128 + ((j ^ g & 3) * 32 + t * 8));
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint32_t v = k ? w.y : w.x, u = v >> 8;
                            c[2 * k][h] = v & 0x000F000Fu;
                            c[2 * k][2 + h] = v & 0x00F000F0u;
                            c[2 * k + 1][h] = u & 0x000F000Fu;
                            c[2 * k + 1][2 + h] = u & 0x00F000F0u;
                        }
                    }
                    const float by[2] = {bf16_of(s[0], j), bf16_of(s[1], j)};
                    float acc[NT][4];  // the tokens' chains side by side: one alone waits 22 cycles for each mma
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma_f16(acc[n], c[0], x[i].x[n][j][0], x[i].x[n][j][1], zero);
#pragma unroll
                    for (int k = 1; k < 4; ++k)
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma_f16(acc[n], c[k], x[i].x[n][j][2 * k], x[i].x[n][j][2 * k + 1], acc[n]);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        if (CODES) {
                            const float2 f = *reinterpret_cast<const float2 *>(factors + ((i * NT + n) * 4 + t) * 8 + j * 2);
                            mul2(acc[n][0], acc[n][1], f.x, f.y);
                            mul2(acc[n][2], acc[n][3], f.x, f.y);
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k) part[n][k] = fmaf(by[k / 2], acc[n][k], part[n][k]);
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int k = 0; k < 4; ++k) out[n][k] = CODES ? out[n][k] + part[n][k] : fmaf(part[n][k], x[i].factor[CODES ? 0 : n][k % 2], out[n][k]);
                tile += kTileBytes;
                if (tile == ring_end) tile = ring;
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) sums[(n * 8 + i % 2) * kPitch + i / 2 * 8] = out[n][i];
        }
        // Join.  Two buffers: the barrier of the next unit stands between this one's reads and the next but one's writes.
        __syncthreads();
        const float *joined = reinterpret_cast<const float *>(smem + L.join() + turn * L.join_bytes());
        auto local = [&](int token, int n) {  // four rows of a token
            const int m = n >> 4 & wm - 1, r = n / 16 >> wm_log;
            const float *from = joined + (r * WARPS + (m << a.wk_log)) * kSums + token * kPitch + n % 16;
            float4 sum = *reinterpret_cast<const float4 *>(from);
#pragma unroll 8
            for (int k = 1; k < wk; ++k) {
                const float4 v = *reinterpret_cast<const float4 *>(from + k * kSums);
                sum.x += v.x;
                sum.y += v.y;
                sum.z += v.z;
                sum.w += v.w;
            }
            return sum;
        };
        const int end_row = min(first_row + steps * step_rows, a.rows);
        auto store = [&](int token, int n, const float4 &sum) {
            const int row = first_row + n;
            constexpr float kUnit = CODES ? 1.0f : 1024.0f;  // bf16: codes times 2^-24, x times 2^14 over its factor
            const float v[4] = {sum.x * kUnit, sum.y * kUnit, sum.z * kUnit, sum.w * kUnit};
            const long long o = static_cast<long long>(token) * a.rows + row;
            if (a.rows % 4 == 0) {
                if (row >= end_row) return;
                if (a.out_f32) {
                    *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + o) = make_float4(v[0], v[1], v[2], v[3]);
                } else {
                    const __nv_bfloat162 p = __floats2bfloat162_rn(v[0], v[1]), q = __floats2bfloat162_rn(v[2], v[3]);
                    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + o) =
                        make_uint2(*reinterpret_cast<const uint32_t *>(&p), *reinterpret_cast<const uint32_t *>(&q));
                }
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (row + k < end_row) {
                        if (a.out_f32)
                            static_cast<float *>(a.out)[o + k] = v[k];
                        else
                            static_cast<__nv_bfloat16 *>(a.out)[o + k] = __float2bfloat16_rn(v[k]);
                    }
            }
        };
        const int in_row = (1 << fours_log) - 1;
        if (ranks == 1) {
            for (int i = threadIdx.x; i < items; i += kThreads) store(i >> fours_log, (i & in_row) * 4, local(i >> fours_log, (i & in_row) * 4));
        } else {
            float4 *part = reinterpret_cast<float4 *>(smem + L.part() + turn * L.part_bytes);
            for (int i = threadIdx.x; i < items; i += kThreads) part[i] = local(i >> fours_log, (i & in_row) * 4);
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
                store(i >> fours_log, (i & in_row) * 4, sum);
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (ranks > 1) cluster.sync();  // nobody leaves while another reads
}

template <int NT, int QPW, int WARPS, bool VEC, bool CODES>
cudaError_t launch(MatvecArgs a, const Layout &L, int num_sms, cudaStream_t stream)
{
    const int step_rows = (WARPS >> a.wk_log) * 16, steps = (a.rows + step_rows - 1) / step_rows;
    auto kernel = matvec_kernel<NT, QPW, WARPS, VEC, CODES>;
    cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void *>(kernel), L.total());
    if (e != cudaSuccess) return e;
    const int clusters = std::min(steps, std::max(1, num_sms / a.ranks));
    a.steps_each = steps / clusters;
    a.steps_more = steps % clusters;
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

template <int NT, int QPW, int WARPS>
cudaError_t launch(const MatvecArgs &args, int num_sms, cudaStream_t stream)
{
    MatvecArgs a = args;
    const int quads = (a.K / 64 + 3) / 4;
    for (a.ranks = 1; (quads + a.ranks - 1) / a.ranks > QPW * WARPS;) a.ranks *= 2;  // at most 8: 64 quads
    const int per = (quads + a.ranks - 1) / a.ranks;
    a.wk_log = 0;
    while ((1 << a.wk_log) < WARPS && (1 << a.wk_log) * QPW < per) ++a.wk_log;
    // two tiles a unit halve the barriers, where there are units enough
    const int wm = WARPS >> a.wk_log;
    a.tiles_log = static_cast<long long>(a.rows) * a.ranks >= 4ll * 32 * wm * num_sms ? 1 : 0;
    const int unit_rows = wm * 16 << a.tiles_log;
    const Layout L{WARPS, QPW, NT, a.ranks > 1 ? unit_rows * a.T * 4 : 0, a.tiles_log, kStages<NT, WARPS>};
    if (L.total() > kMaxSmem) return cudaErrorInvalidConfiguration;
    const bool vec = a.K % 256 == 0;
    if (a.x_scale)
        return vec ? launch<NT, QPW, WARPS, true, true>(a, L, num_sms, stream) : launch<NT, QPW, WARPS, false, true>(a, L, num_sms, stream);
    return vec ? launch<NT, QPW, WARPS, true, false>(a, L, num_sms, stream) : launch<NT, QPW, WARPS, false, false>(a, L, num_sms, stream);
}

}  // namespace

cudaError_t launch_matvec(const MatvecArgs &a, int num_sms, cudaStream_t stream)
{
    if (a.T <= 8) return a.K <= 4096 ? launch<1, 1, 16>(a, num_sms, stream) : launch<1, 2, 16>(a, num_sms, stream);
    if (a.T <= 16) return launch<2, 1, 16>(a, num_sms, stream);
    if (a.T <= 24) return launch<3, 1, 8>(a, num_sms, stream);
    return launch<4, 1, 8>(a, num_sms, stream);
}

}  // namespace lily
