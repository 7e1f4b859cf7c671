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
// [2^14, 2^15): their eight significant bits survive down to 2^-27 of that largest magnitude, and what is smaller is off by at
// most 2^-35 of it.  The norm's e4m3 tokens are fp16 numbers already.  Sums are fp32, scaled and joined a group at a
// time.  The biases of four groups are one more mma, on bf16: their 16 columns are the four sums of x, each as three
// bf16 numbers that add up to it exactly.
//
// Bound: HBM (0.5625 bytes a weight) up to 8 tokens, then the tensor cores' and the warps' instructions: 65,536 more rows of 2,048
// cost 11.4 us for 1 token (6.6 TB/s), 12.1 for 8, 19.1 for 16, 30.9 for 32; launch, x and the last tiles 4 to 5 us (7 for 32
// tokens).  130,001 rows and 4 tokens: 28.1 us; 5,120 rows and 1 token: 4.0.  Warps along K are a power of two, and what K
// does not fill of them waits: 20,001 rows of 2,112 take 10.1 us for 1 token and 27.7 for 32, of 2,048 half as much a weight.  The order of the
// channels within an mma is free as long as both sides agree: a thread takes 16 consecutive channels of a group.  A warp keeps the
// fragments of its four groups (a quad: 256 channels) of x in registers and takes the rows' pieces of that quad past them, one
// tile of 16 rows after another, through a ring of asynchronous copies of its own; the warps of a CTA share a row's K and
// join their sums in shared memory.  A K of more quads than a CTA has warps for is taken in chunks: a block of rows has all its
// chunks one after another, with its sums so far in shared memory.  (A cluster of CTAs along K instead drains each warp's ring at
// every join, as the barrier's release waits for the copies: 16,384 rows of 8,192 and 32 tokens took 101 us.)
#include <algorithm>
#include <cstdint>

#include <cuda_fp8.h>

#include "lily_internal.h"

namespace lily {
namespace {

constexpr int kPitch = 20;        // floats between tokens of a joined tile: the fragment's stores meet no bank twice
constexpr int kSkew = 16;         // floats more between the two steps of a unit: the join reads both at once, off each other's banks
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

__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

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

// (c0, c1) += (a0, a1) * b.
__device__ __forceinline__ void fma2(float &c0, float &c1, float a0, float a1, float b)
{
    asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\tmov.b64 c, {%0, %1};\n\tfma.rn.f32x2 c, a, b, c;\n\tmov.b64 {%0, %1}, c;\n\t}"
        : "+f"(c0), "+f"(c1)
        : "f"(a0), "f"(a1), "f"(b));
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

__device__ __forceinline__ void load16(uint32_t *to, const char *p)
{
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(to[0]), "=r"(to[1]), "=r"(to[2]), "=r"(to[3]) : "l"(p) : "memory");
}

// Loads a quad of x (its groups from g_last on as zeros).  CODES: leaves the factors of its groups for
// tokens 2 t and 2 t + 1, [n][t][j][2], at `factors`.
template <int NT, bool VEC, bool CODES>
__device__ __forceinline__ void load_tokens(Tokens<NT, CODES> &to, const MatvecArgs &a, int g_first, int g_last, int lane, float *factors)
{
    const int t = lane % 4;
    // All loads first, to where their fp16 form goes: as asm, so that the compiler puts none off until others are converted (it did, for
    // another round trip; as the code stands it need not: 32 tokens on 65,536 rows of 2,048 38.1 us, 38.4 with plain loads, 24 on 2,048 of
    // 4,096 9.3 both ways).  Tokens past T are the last one again: their columns are not stored.
    float scale[CODES ? NT : 1];  // of group t
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const long long token = min(8 * n + lane / 4, a.T - 1);
        const char *p = static_cast<const char *>(a.x) + (token * a.x_stride + g_first * 64 + 16 * t) * (CODES ? 1 : 2);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t *x = to.x[n][j];
            if (VEC || g_first + j < g_last) {
                load16(x, p + j * (CODES ? 64 : 128));
                if (!CODES) load16(x + 4, p + j * 128 + 16);
            } else {
#pragma unroll
                for (int i = 0; i < (CODES ? 4 : 8); ++i) x[i] = 0;
            }
        }
        if (CODES) scale[CODES ? n : 0] = VEC || g_first + t < g_last ? a.x_scale[token * (a.K / 64) + g_first + t] : 0.0f;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float sum[4], by = 64.0f;  // the largest code, 448, is 28,672
        if (!CODES) {
            __nv_bfloat162 most2 = __floats2bfloat162_rn(0.0f, 0.0f);  // NaN leaves it
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) most2 = __hmax2(most2, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&to.x[n][j][i])));
            uint32_t most = max(static_cast<uint32_t>(__bfloat16_as_ushort(most2.x)), static_cast<uint32_t>(__bfloat16_as_ushort(most2.y)));
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
            // x times 2^(14 - e), e = floor(log2 most) in [-113, 127]
            const int e = min(max(static_cast<int>(most >> 7) - 127, -113), 127);
            const float factor = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
            by = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
#pragma unroll
            for (int i = 0; i < 2; ++i) to.factor[CODES ? 0 : n][i] = __shfl_sync(0xffffffffu, factor, (2 * t + i) * 4);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t *u = to.x[n][j];
            float x[16];
            const float sixteenth = by * 0.0625f;
            float even = 0.0f, odd = 0.0f;  // the sums, as the places are scaled
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 p = CODES ? of_e4m3x2(u[i / 2] >> (16 * (i & 1)) & 0xFFFFu)
                                       : make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u));
                x[2 * i] = p.x * by;
                x[2 * i + 1] = p.y * sixteenth;
                even += x[2 * i];
                odd += x[2 * i + 1];
            }
            sum[j] = fmaf(odd, 16.0f, even);
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
                for (int i = 0; i < 4; ++i) to.x[n][j][4 * w + i] = f16x2(x[8 * w + i], x[8 * w + i + 4]);
        }
        // the four lanes' sums of four groups: lane t gets the whole of group t's
        const float keep0 = (t & 1 ? sum[1] : sum[0]) + __shfl_xor_sync(0xffffffffu, t & 1 ? sum[0] : sum[1], 1);
        const float keep1 = (t & 1 ? sum[3] : sum[2]) + __shfl_xor_sync(0xffffffffu, t & 1 ? sum[2] : sum[3], 1);
        float rest = (t & 2 ? keep1 : keep0) + __shfl_xor_sync(0xffffffffu, t & 2 ? keep0 : keep1, 2);
        // Everything is 2^-10 of what it stands for until it is stored (kUnit), which leaves a factor of scale * 2^8 here: finite, and times a
        // group's largest sum of products too, for every scale that the norm gives (fp32's largest number over 448).  Products with
        // codes are times 2^-24 and `by`.
        rest *= CODES ? scale[CODES ? n : 0] * 0x1p-16f : 0x1p-24f;
        if (CODES) factors[((n * 4 + lane / 8) * 4 + t) * 2 + lane / 4 % 2] = scale[CODES ? n : 0] * 0x1p8f;
        // as three bf16 numbers: what is left of 24 bits after eight more
        const __nv_bfloat16 p0 = __float2bfloat16_rn(rest);
        rest -= __bfloat162float(p0);
        const __nv_bfloat16 p1 = __float2bfloat16_rn(rest);
        rest -= __bfloat162float(p1);
        const uint32_t first = __bfloat16_as_ushort(p0) | static_cast<uint32_t>(__bfloat16_as_ushort(p1)) << 16;
        const uint32_t last = __bfloat16_as_ushort(__float2bfloat16_rn(rest));
        // columns 2 t, 2 t + 1: the first numbers of groups 0 1 | 2 3, then the second; columns 8 + 2 t: the third, nothing
        const int from = lane & ~3 | t % 2 * 2;
        const uint32_t first0 = __shfl_sync(0xffffffffu, first, from), first1 = __shfl_sync(0xffffffffu, first, from + 1);
        const uint32_t last0 = __shfl_sync(0xffffffffu, last, from), last1 = __shfl_sync(0xffffffffu, last, from + 1);
        to.sums[n][0] = __byte_perm(first0, first1, t < 2 ? 0x5410 : 0x7632);
        to.sums[n][1] = t < 2 ? last0 | last1 << 16 : 0;
    }
}

// Stages of a warp's ring: what its memory time needs, and no more (65,536 rows of 2,048: 16 tokens 23.4 us with four, 24.3 with six; 24
// tokens 31.0 with four, 31.8 with five; 32 tokens 38.1 with five, 39.1 with four; a fourth for 16 warps has no room beside four steps a join).
template <int NT, int WARPS>
constexpr int kStages = WARPS == 16 ? 3 : NT <= 3 ? 4 : 5;

// Shared memory: the factors [warp][NT][4][4][2]; two of the warps' sums, [step of the unit][warp][token][row]; the ring
// [warp][stage] of tiles; where K is more than a chunk, the sums so far of a block's steps, [step][token][row].
struct Layout {
    int warps, nt, tiles_log, stages, block_bytes;
    __host__ __device__ int join() const { return warps * nt * 128; }
    __host__ __device__ int join_bytes() const { return ((warps * 8 * nt * kPitch + kSkew) * 4) << tiles_log; }
    __host__ __device__ int ring() const { return join() + 2 * join_bytes(); }
    __host__ __device__ int block() const { return ring() + warps * stages * kTileBytes; }
    __host__ __device__ int total() const { return block() + block_bytes; }
};

template <int NT, int WARPS, bool VEC, bool CODES>
__global__ void __launch_bounds__(WARPS * 32, 1) matvec_kernel(const __grid_constant__ MatvecArgs a)
{
    constexpr int kThreads = WARPS * 32, kSums = 8 * NT * kPitch, kS = kStages<NT, WARPS>;
    extern __shared__ __align__(128) unsigned char smem[];
    pdl_trigger();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    // a chunk is per_chunk quads of K, one for each of wk warps
    const int groups = a.K / 64, all_quads = (groups + 3) / 4, per_chunk = a.per_chunk;
    const int wk = 1 << a.wk_log, wm = WARPS >> a.wk_log, wm_log = 31 - __clz(wm);  // warps along K, along rows
    const int k_warp = warp & (wk - 1), m_warp = warp >> a.wk_log;
    const int my_chunks = k_warp < per_chunk && k_warp < all_quads ? (all_quads - k_warp - 1) / per_chunk + 1 : 0;  // those in which this warp has a quad
    // A step is a tile of each of the warps along rows; a unit, between joins, 2^tiles_log steps; a block, between chunks, block_steps.
    // A CTA takes steps that follow one another.
    const int tiles_log = a.tiles_log, step_rows = wm * 16;
    const int first_step = blockIdx.x * a.steps_each + min(static_cast<int>(blockIdx.x), a.steps_more);
    const int last_step = first_step + a.steps_each + (static_cast<int>(blockIdx.x) < a.steps_more ? 1 : 0);
    const Layout L{WARPS, NT, tiles_log, kS, 0};
    float *factors = reinterpret_cast<float *>(smem) + warp * (NT * 32);
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
    const int p_step = step_rows * groups, last_row = min(last_step * step_rows, a.rows);  // past this CTA's rows
    int load_chunk = 0, load_block = first_step, load_row = first_step * step_rows + m_warp * 16, load_end = 0;
    uint32_t load_to = ring_to;
    const uint8_t *from_w = nullptr;
    long long from_p = 0;
    auto aim = [&]() {  // at the first tile of a chunk of a block
        const int q = load_chunk * per_chunk + k_warp;
        load_row = load_block * step_rows + m_warp * 16;
        load_end = min(min(load_block + a.block_steps, last_step) * step_rows, a.rows);
        from_w = a.w + (load_row + row_w) * half + q * 128 + piece * 16;
        from_p = static_cast<long long>(load_row + lane % 16) * groups + q * 4;
    };
    aim();
    auto load = [&]() {
        if (load_chunk < my_chunks && load_row < last_row) {
            const int q = load_chunk * per_chunk + k_warp;
            if (load_row + 16 <= a.rows && (VEC || q < all_quads - 1)) {
#pragma unroll
                for (int i = 0; i < 4; ++i) copy<16>(load_to + to_w + i * 512, from_w + 4 * i * half);
                if (VEC) {
                    copy<8>(load_to + to_p, params + from_p);
                } else {
                    const uint16_t *p = params + (from_p & ~1ll);
                    copy<4>(load_to + to_p, p);
                    copy<4>(load_to + to_p + 4, p + 2);
                    if (from_p & 1) copy<4>(load_to + to_p + 8, p + 4, 2);  // the row's fourth
                }
            } else {  // rows past the end and, in the last quad, groups past the end are zeros
                const int pieces = (groups - q * 4) * 2;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool on = load_row + 4 * i + row_w < a.rows && piece < pieces;
                    copy<16>(load_to + to_w + i * 512, on ? from_w + 4 * i * half : a.w, on ? 16 : 0);
                }
                const bool on = load_row + lane % 16 < a.rows;
                if (VEC) {
                    copy<8>(load_to + to_p, on ? params + from_p : params, on ? 8 : 0);
                } else {
#pragma unroll
                    for (int k = 0; k < 3; ++k) {
                        const long long word = (from_p & ~1ll) + 2 * k, left = on ? param_end - word : 0;
                        copy<4>(load_to + to_p + 4 * k, left > 0 ? params + word : params, left <= 0 ? 0 : left < 2 ? 2 : 4);
                    }
                }
            }
            load_to += kTileBytes;
            if (load_to == ring_to + kS * kTileBytes) load_to = ring_to;
            load_row += step_rows;
            from_w += w_step;
            from_p += p_step;
            if (load_row >= load_end && a.per_chunk < all_quads) {  // the next chunk, or the next block's first
                if (++load_chunk >= my_chunks) {
                    load_chunk = 0;
                    load_block += a.block_steps;
                }
                aim();
            }
        }
        copy_commit();
    };
    // The matrix may come from a kernel before, so the copies stand behind the wait.  Ahead of it the first tiles are called to L2, which
    // every store goes through: no value is taken.  (1 token on 5,120 rows of 2,048: 4.0 us, 4.4 without; 16 tokens on 65,536
    // 23.4 against 24.2; 32 tokens on 65,536, where registers are short, 38.7 against 38.1.)
    if (NT <= 3 && my_chunks > 0) {
#pragma unroll
        for (int i = 0; i < kS - 1; ++i) {
            const int row = load_row + i * step_rows + lane % 16;
            if (row < load_end) {
                if (lane < 16) {
                    prefetch_l2(a.w + row * half + k_warp * 128);
                } else {
                    const long long at = static_cast<long long>(row) * groups + k_warp * 4;
                    prefetch_l2(a.s + at);
                    prefetch_l2(a.b + at);
                }
            }
        }
    }
    pdl_wait();
    for (int i = 0; i < kS - 1; ++i) load();
    const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const unsigned char *tile = ring;
    const unsigned char *const ring_end = ring + kS * kTileBytes;
    const int fours_log = 29 - __clz(step_rows << tiles_log), items = a.T << fours_log;  // items of the join: [token][row / 4]
    int turn = 0;
    for (int block = first_step; block < last_step; block += a.block_steps)
        for (int c0 = 0; c0 < all_quads; c0 += per_chunk) {
            Tokens<NT, CODES> x;
            const bool works = k_warp < per_chunk && c0 + k_warp < all_quads;
            if (works) {
                __syncwarp();  // all lanes are done with the factors before
                load_tokens<NT, VEC, CODES>(x, a, (c0 + k_warp) * 4, groups, lane, factors);
                __syncwarp();
            }
            const int block_end = min(block + a.block_steps, last_step);
            const bool first_chunk = c0 == 0, last_chunk = c0 + per_chunk >= all_quads;
            for (int step = block; step < block_end; turn ^= 1) {
                float *sums = reinterpret_cast<float *>(smem + L.join() + turn * L.join_bytes()) + warp * kSums + t * (2 * kPitch) + g;
                const int unit_step = step, steps = min(1 << tiles_log, block_end - step);
                for (int r = 0; r < steps; ++r, ++step, sums += WARPS * kSums + kSkew) {
                    const int row0 = step * step_rows + m_warp * 16;
                    float part[NT][4];
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int k = 0; k < 4; ++k) part[n][k] = 0.0f;
                    if (works && row0 < a.rows) {
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
                                const int left = groups - (c0 + k_warp) * 4;
                                if (left < 4) {
                                    s[h].y = left > 2 ? s[h].y & 0xFFFFu : 0;
                                    s[h].x = left > 1 ? s[h].x : s[h].x & 0xFFFFu;
                                    const int mine = left - t % 2 * 2;
                                    b[h] = mine > 1 ? b[h] : mine > 0 ? b[h] & 0xFFFFu : 0;
                                }
                            }
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma_bf16(part[n], b[0], b[1], x.sums[n][0], x.sums[n][1], zero);
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
                            for (int n = 0; n < NT; ++n) mma_f16(acc[n], c[0], x.x[n][j][0], x.x[n][j][1], zero);
#pragma unroll
                            for (int k = 1; k < 4; ++k)
#pragma unroll
                                for (int n = 0; n < NT; ++n) mma_f16(acc[n], c[k], x.x[n][j][2 * k], x.x[n][j][2 * k + 1], acc[n]);
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                if (CODES) {
                                    const float2 f = *reinterpret_cast<const float2 *>(factors + (n * 4 + t) * 8 + j * 2);
                                    mul2(acc[n][0], acc[n][1], f.x, f.y);
                                    mul2(acc[n][2], acc[n][3], f.x, f.y);
                                }
                                // two at once where registers are left for the pairs (16 tokens 23.4 us against 24.0, 32 tokens 39.4 against 38.1)
                                if (NT <= 2) {
                                    fma2(part[n][0], part[n][1], acc[n][0], acc[n][1], by[0]);
                                    fma2(part[n][2], part[n][3], acc[n][2], acc[n][3], by[1]);
                                } else {
#pragma unroll
                                    for (int k = 0; k < 4; ++k) part[n][k] = fmaf(by[k / 2], acc[n][k], part[n][k]);
                                }
                            }
                        }
                        if (!CODES) {
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                const float *f = x.factor[CODES ? 0 : n];
                                mul2(part[n][0], part[n][1], f[0], f[1]);
                                mul2(part[n][2], part[n][3], f[0], f[1]);
                            }
                        }
                        tile += kTileBytes;
                        if (tile == ring_end) tile = ring;
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) sums[(n * 8 + i % 2) * kPitch + i / 2 * 8] = part[n][i];
                }
                // Join: a thread takes four rows of a token.  Two buffers: the barrier of the next unit stands between this one's reads and
                // the next but one's writes.  The sums so far are the same thread's in every chunk.
                __syncthreads();
                const float *joined = reinterpret_cast<const float *>(smem + L.join() + turn * L.join_bytes());
                float4 *so_far = reinterpret_cast<float4 *>(smem + L.block()) + (unit_step - block) * a.T * (step_rows / 4);
                const int end_row = min((unit_step + steps) * step_rows, a.rows);
                for (int i = threadIdx.x; i < items; i += kThreads) {
                    const int token = i >> fours_log, n = (i & (1 << fours_log) - 1) * 4, row = unit_step * step_rows + n;
                    if (row >= end_row) continue;
                    const int of_unit = n / 16 >> wm_log;  // step of the unit
                    const float *from = joined + (of_unit * WARPS + ((n >> 4 & wm - 1) << a.wk_log)) * kSums + of_unit * kSkew + token * kPitch + n % 16;
                    float4 sum = *reinterpret_cast<const float4 *>(from);
#pragma unroll 8
                    for (int k = 1; k < wk; ++k) {
                        const float4 v = *reinterpret_cast<const float4 *>(from + k * kSums);
                        sum = make_float4(sum.x + v.x, sum.y + v.y, sum.z + v.z, sum.w + v.w);
                    }
                    if (!first_chunk) {
                        const float4 v = so_far[i];
                        sum = make_float4(sum.x + v.x, sum.y + v.y, sum.z + v.z, sum.w + v.w);
                    }
                    if (!last_chunk) {
                        so_far[i] = sum;
                        continue;
                    }
                    constexpr float kUnit = 1024.0f;  // codes times 2^-24, bf16 x times 2^14 over its factor, e4m3 x times 2^6 and its factor 2^8
                    const float v[4] = {sum.x * kUnit, sum.y * kUnit, sum.z * kUnit, sum.w * kUnit};
                    const long long o = static_cast<long long>(token) * a.rows + row;
                    if (a.rows % 4 == 0) {
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
                }
            }
        }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

int log2_at_least(int n)
{
    int log = 0;
    while ((1 << log) < n) ++log;
    return log;
}

template <int NT, int WARPS, bool VEC, bool CODES>
cudaError_t launch(MatvecArgs a, const Layout &L, int num_sms, cudaStream_t stream)
{
    const int step_rows = (WARPS >> a.wk_log) * 16, steps = (a.rows + step_rows - 1) / step_rows, ctas = std::min(steps, num_sms);
    a.steps_each = steps / ctas;
    a.steps_more = steps % ctas;
    auto kernel = matvec_kernel<NT, WARPS, VEC, CODES>;
    const cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void *>(kernel), L.total());
    return e != cudaSuccess ? e : launch_pdl(kernel, dim3(ctas), dim3(WARPS * 32), static_cast<size_t>(L.total()), stream, a);
}

template <int NT, int WARPS>
cudaError_t launch(const MatvecArgs &args, int num_sms, cudaStream_t stream)
{
    MatvecArgs a = args;
    const int quads = (a.K / 64 + 3) / 4, chunks = (quads + WARPS - 1) / WARPS;
    a.per_chunk = (quads + chunks - 1) / chunks;
    a.wk_log = log2_at_least(a.per_chunk);
    // A unit is as many steps as some CTA has, up to four, which leaves a quarter of the barriers (8,192 rows of 2,048 and 1 token: 4.6 us
    // against 4.9 with two; 130,001 of 2,048 and 4 tokens 28.0 against 29.1; 4,096 of 16,384 14.8 against 16.1 with one); above 8 tokens
    // shared memory has room for two, and above 16 they pay where each CTA has two (32 tokens on 65,536 of 2,048 38.1 us against 39.4
    // with one, but on 4,096 of 16,384, where some CTAs have one step, 48.5 against 47.3).
    const int step_rows = (WARPS >> a.wk_log) * 16;
    const long long wave = static_cast<long long>(step_rows) * num_sms;
    a.tiles_log = NT == 1 && a.rows > 2 * wave ? 2 : a.rows > (NT <= 2 ? 1 : 2) * wave ? 1 : 0;
    Layout L{WARPS, NT, a.tiles_log, kStages<NT, WARPS>, 0};
    a.block_steps = 1 << 30;
    if (chunks > 1) {
        a.block_steps = (kMaxSmem - L.total()) / (step_rows * a.T * 4) >> a.tiles_log << a.tiles_log;
        L.block_bytes = a.block_steps * step_rows * a.T * 4;
    }
    const bool vec = a.K % 256 == 0;
    if (a.x_scale) return vec ? launch<NT, WARPS, true, true>(a, L, num_sms, stream) : launch<NT, WARPS, false, true>(a, L, num_sms, stream);
    return vec ? launch<NT, WARPS, true, false>(a, L, num_sms, stream) : launch<NT, WARPS, false, false>(a, L, num_sms, stream);
}

}  // namespace

cudaError_t launch_matvec(const MatvecArgs &a, int num_sms, cudaStream_t stream)
{
    // Up to 8 tokens half the warps start sooner and join less, where they hold all of K and a CTA has up to eight steps (1,024 rows
    // of 1,024: 2.5 us against 3.3; 10,240 of 2,048 5.5 against 5.7; 19,456 6.9 against 7.0; 65,536 17.2 against 15.8).
    const int quads = (a.K + 255) / 256;
    if (a.T <= 8 && quads <= 8 && a.rows <= 8ll * (8 >> log2_at_least(quads)) * 16 * num_sms) return launch<1, 8>(a, num_sms, stream);
    if (a.T <= 8) return launch<1, 16>(a, num_sms, stream);
    if (a.T <= 16) return launch<2, 8>(a, num_sms, stream);
    if (a.T <= 24) return launch<3, 8>(a, num_sms, stream);
    return launch<4, 8>(a, num_sms, stream);
}

}  // namespace lily
