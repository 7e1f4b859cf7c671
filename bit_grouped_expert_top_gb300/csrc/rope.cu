// Rotary positions on queries and keys, for sm_103a.
//
// Pair i of a head is turned by the angle pos * f_i:
//   (a, b) -> amplitude * (a cos - b sin, a sin + b cos)
// with the pair's channels (i, i + rot/2) or (2i, 2i + 1) of the first `rot`.
// f_i / 2 pi is held as a 64-bit fraction of a turn (53 bits of it, as it comes from fp64), so the turns of a position
// modulo one are an integer product modulo 2^64: exact for that fraction, at any position.  Its top 32 bits, cut by up to
// 2^-31 half-turns and rounded to fp32 by up to 2^-25 (as much as sincospif's own error), go to sincospif.  In
// fp32, pos * f_i alone would be off by 2^-5 at position 2^20.
//
// Bound: HBM (4 bytes a channel) for a prompt, latency for a step.  A thread has the 16 channels of a pair of
// 16-byte vectors (eight pairs to turn, or a piece of the tail to copy), and takes `heads_each` heads with the sines and
// cosines that it works out once: with one head a thread a prompt is bound by its instructions.  The threads that turn
// come first, so that no warp does both.
#include <cstdint>

#include "lily_internal.h"

namespace lily {
namespace {

constexpr int kThreads = 256;

template <bool NEXT>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a)
{
    pdl_trigger();
    const int turn = a.rot / 16, tail = a.copy ? (a.D - a.rot) / 16 : 0;
    const int heads = a.H_q + a.H_k, slices = a.slices;
    // units of (token, slice of the heads, part): the parts that turn, then, from a block's border on, the tail
    unsigned unit = blockIdx.x * kThreads + threadIdx.x;
    const bool turns = blockIdx.x < a.turn_blocks;
    if (!turns) unit -= a.turn_blocks * kThreads;
    const unsigned parts = turns ? turn : tail;
    const int part = unit % parts;
    const unsigned rest = unit / parts;
    const long long n = rest / slices;
    const int slice = rest % slices;
    if (n >= a.N) return;
    // the two vectors of this part, in channels from the head's first
    const int v0 = turns ? part * 8 : a.rot + part * 8;
    const int v1 = v0 + (turns ? a.rot : a.D - a.rot) / 2;
    pdl_wait();
    float c[8], s[8];
    if (turns) {
        const long long pos = a.positions[n];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            // half: pairs v0 .. v0 + 7; next: four pairs from each vector
            const int pair = NEXT ? (j < 4 ? v0 / 2 + j : v1 / 2 + j - 4) : v0 + j;
            const unsigned long long fraction = static_cast<unsigned long long>(pos) * a.table[pair];
            const float half_turns = static_cast<float>(static_cast<int>(fraction >> 32)) * 0x1p-31f;
            sincospif(half_turns, &s[j], &c[j]);
            s[j] *= a.amplitude;
            c[j] *= a.amplitude;
        }
    }
    const int last = min(heads, (slice + 1) * a.heads_each);
    constexpr int kBatch = 3;
    for (int h0 = slice * a.heads_each; h0 < last; h0 += kBatch) {
        uint4 in[kBatch][2];
        uint16_t *dst[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int h = h0 + i;
            if (h >= last) break;
            const bool is_q = h < a.H_q;
            const uint16_t *src = is_q ? a.q + n * a.q_stride + h * a.D : a.k + n * a.k_stride + (h - a.H_q) * a.D;
            dst[i] = is_q ? a.q_out + n * a.q_out_stride + h * a.D : a.k_out + n * a.k_out_stride + (h - a.H_q) * a.D;
            in[i][0] = *reinterpret_cast<const uint4 *>(src + v0);
            in[i][1] = *reinterpret_cast<const uint4 *>(src + v1);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (h0 + i >= last) break;
            const uint4 x = in[i][0], y = in[i][1];
            uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
            if (turns) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float x0 = __uint_as_float(xs[j] << 16), x1 = __uint_as_float(xs[j] & 0xFFFF0000u);
                    const float y0 = __uint_as_float(ys[j] << 16), y1 = __uint_as_float(ys[j] & 0xFFFF0000u);
                    __nv_bfloat162 p, q;
                    if (NEXT) {  // (x0, x1) is pair j of the first vector, (y0, y1) of the second
                        p = __floats2bfloat162_rn(x0 * c[j] - x1 * s[j], x0 * s[j] + x1 * c[j]);
                        q = __floats2bfloat162_rn(y0 * c[j + 4] - y1 * s[j + 4], y0 * s[j + 4] + y1 * c[j + 4]);
                    } else {  // (x0, y0) and (x1, y1) are pairs 2j and 2j + 1
                        p = __floats2bfloat162_rn(x0 * c[2 * j] - y0 * s[2 * j], x1 * c[2 * j + 1] - y1 * s[2 * j + 1]);
                        q = __floats2bfloat162_rn(x0 * s[2 * j] + y0 * c[2 * j], x1 * s[2 * j + 1] + y1 * c[2 * j + 1]);
                    }
                    xs[j] = *reinterpret_cast<const uint32_t *>(&p);
                    ys[j] = *reinterpret_cast<const uint32_t *>(&q);
                }
            }
            *reinterpret_cast<uint4 *>(dst[i] + v0) = make_uint4(xs[0], xs[1], xs[2], xs[3]);
            *reinterpret_cast<uint4 *>(dst[i] + v1) = make_uint4(ys[0], ys[1], ys[2], ys[3]);
        }
    }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &args, int num_sms, cudaStream_t stream)
{
    RopeArgs a = args;
    const int heads = a.H_q + a.H_k;
    // As many heads a thread as leave 512 threads an SM that turn.  8,192 tokens of 18 heads of 256, a quarter of which turns: 24.9 us
    // (6.1 TB/s); 33.4 with 2,048 threads an SM, 25.6 with 1,024, 28.0 with 128.  1,001 tokens of 16 heads of 128, all of which turns, have
    // one head a thread: 4.3 us; 6.1 with 128 threads an SM.
    const long long wave = num_sms * 512ll, turning = static_cast<long long>(a.N) * (a.rot / 16);
    const long long most = turning * heads / wave;
    a.heads_each = static_cast<int>(most < 1 ? 1 : most < heads ? most : heads);
    a.slices = (heads + a.heads_each - 1) / a.heads_each;
    a.heads_each = (heads + a.slices - 1) / a.slices;
    auto blocks = [&](int parts) { return static_cast<unsigned>((static_cast<long long>(a.N) * a.slices * parts + kThreads - 1) / kThreads); };
    a.turn_blocks = blocks(a.rot / 16);
    const dim3 grid(a.turn_blocks + (a.copy ? blocks((a.D - a.rot) / 16) : 0)), block(kThreads);
    return a.next ? launch_pdl(rope_kernel<true>, grid, block, 0, stream, a)
                  : launch_pdl(rope_kernel<false>, grid, block, 0, stream, a);
}

}  // namespace lily
