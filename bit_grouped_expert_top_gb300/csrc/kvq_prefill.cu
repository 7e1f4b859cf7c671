// Prefill attention over the quantised KV cache (a chunk of query tokens per
// sequence, causal), for sm_103a: query i of the m of sequence b, head h,
//   o = sum_{t < L - m + i + 1} softmax_t(scale q . k_t) v_t,
// k_t and v_t the values code * scale + bias of row t of KV head g = h / (H_q / H_kv).
//
// The tensor cores bound this one: 4 D operations per (query head, token) pair.  A CTA
// takes 128 query rows, the G query heads of a KV head for TQ = 128 / G tokens (one
// rebuilt K and V serves them all), against the cache in chunks of 64 tokens; a pair of
// CTAs shares an item of 2 TQ tokens and each rebuilds half of K and V, since with D = 256 the
// rebuild and not the MMAs bounds a CTA alone (2,048 queries on 32,768 tokens at the time: 669 us with
// pairs, 835 without; with D = 64 and 128 it is the chain of a tile's scores, softmax and product, which takes
// as long as with 256).  The chunks of all items form one list that the pairs, one per two SMs,
// share evenly (a long prompt's later tiles have more of them); an item cut between pairs
// leaves partial results that a second kernel joins.
// Per CTA, with every wait bounded:
//   warps 0..7   two threads per query row (32 of a chunk's 64 tokens each; four where a
//                tile has 32 rows, which leaves the warps for the rebuild): q into
//                tensor memory as fp16 (times a power of two per row, so q has no range
//                limit), then per chunk S from tensor memory, the softmax weights back
//                into it as fp16 (the A operand of P V), at the end O out of it.  The
//                running maximum moves only when a score passes it by 8 (in powers of
//                two; the weights then stay below 2^15, see kLift), so O in tensor memory is
//                rescaled rarely.  The next item's q is converted before O is read, so
//                its first scores are computed meanwhile.
//   warps 8..15  rebuild K and V of a chunk in fp16 (rounded once) into swizzled
//                shared memory, two to four buffers each: a thread takes one (token, group
//                of 64 channels); its codes are loaded one chunk ahead.  Rows behind the
//                sequence become zeros.
//   warp 16      issues tcgen05.mma (of a pair: the first CTA's): S = Q K^T (A from tensor
//                memory, B K-major) of chunk i + 1, then O += P V (B with the channels
//                contiguous) of chunk i, so the softmax runs beside them.
//   warp 17      one thread copies the next item's q into shared memory (TMA).
// K and V must stay within fp16: |value| >= 65520, or one that is no number, records LILY_ERR_DEVICE_RANGE.
// Measured (16 query heads on 2 KV heads of 256, 4 bits): 2,048 queries at the end of
// 32,768 tokens 677 us (1,573 TFLOP/s, 0.82 of the measured burst matrix rate), a prompt of
// 8,192 tokens 400 us (0.72: an item's start and end cost about eight chunks).
#include <cmath>
#include <cstdint>

#include "kvq_device.cuh"
#include "lily_internal.h"

namespace lily {
namespace {

constexpr int kRows = 128;                 // query rows of a tile
constexpr int kChunk = 64;                 // cache tokens per step
// Taking up an item (its q, the first scores, its output) costs about eight chunks,
// which the shares of the work list count: an 8K prompt 413 us with 6, 397 with 8, 402
// with 10, 406 with 12.
constexpr int kItemCost = 8;
// Cutting an item costs about sixteen chunks (its parts, their join): where there are no more
// items than shares, and the longest is not longer by more than that than an even share, each
// share is an item.  A prompt of 1,024 tokens 43 us cut, 35 with items; of 512 33 and 28.
// (With a limit of 8 chunks as if cut; with 32, four tokens each on four contexts of 1,000
// take 30 us instead of 21.)
constexpr int kUncut = 16;
// Warps by the quarters NQ of the tile's 128 rows that hold queries: softmax warps (eight:
// two a quarter; one quarter: four; a quarter's warps have its index modulo 4, as they reach
// its lanes of tensor memory), rebuild warps, MMA issuer, query loader.
template <int NQ>
struct Roles {
    static constexpr int parts = NQ == 1 ? 4 : 2;  // softmax warps of a quarter: each has 64 / parts of a chunk's tokens
    static constexpr int soft = parts * NQ, deq = NQ == 1 ? 16 : 8, mma = soft + deq, load = mma + 1, threads = (load + 1) * 32;
    __device__ static __forceinline__ bool is_soft(int warp) { return warp < 4 * parts && (warp & 3) < NQ; }
    __device__ static __forceinline__ int deq_index(int warp) { return NQ == 1 ? (warp < 16 ? warp - 1 - warp / 4 : warp - 4) : warp - soft; }
};
constexpr int kMaxWarps = Roles<1>::threads / 32;
constexpr int kBarPair = 1;                // named barriers 1..4: the softmax warps of 32 rows
constexpr int kBox = kChunk * 128;         // [64 tokens][64 channels] fp16, 128-byte swizzle
constexpr int kMaxBufs = 4;                // buffers of K and of V, at most
constexpr uint32_t kTmemCols = 512;
constexpr float kNoMax = -1.7e38f;
// Weights are taken against the running maximum less kLift: a row's largest one is 2^7 to 2^15, so that fp16 rounds
// the others by 2^-11 of themselves down to 2^-21 of it, and smaller ones by 2^-32 of it at most (as
// many small weights beside a large one may be all that a row is made of).
constexpr float kLift = 7.0f;

struct Fixed {
    uint64_t k_full[kMaxBufs], k_free[kMaxBufs], v_full[kMaxBufs], v_free[kMaxBufs], s_full[2], p_full[2];
    uint64_t pv_done[2], q_full, q_loaded, q_free, o_free, drain;
    uint32_t tmem;
    int abort, b0, m0, L0, q0;
    long long pre, per, begin, total, used, sum[kMaxWarps];
    float xch[2][4][kRows];  // [chunk parity][part of the columns][row]
#ifdef LILY_TEST_STALL_T
    uint64_t never;  // test builds only: a barrier nothing arrives on
#endif
};
constexpr int kFixed = 5120;
static_assert(sizeof(Fixed) <= kFixed, "barriers and scratch");
constexpr int kQBox = kRows * 128;         // [128 rows][64 channels] bf16, 128-byte swizzle
// CG: the CTAs that share an item's K and V.  The MMAs of a pair read half of K's tokens
// and of V's channels from each CTA's shared memory, so each rebuilds half.
__host__ __device__ constexpr int buf_bytes(int GR, int CG) { return GR * kBox / CG; }
__host__ __device__ constexpr int bufs_for(int GR, int CG) { return buf_bytes(GR, CG) > 16384 ? 2 : kMaxBufs; }
// More than half of an SM's, so that no two CTAs that allocate tensor memory meet on
// one SM: two pairs that each hold one of two SMs would wait for each other.
constexpr int kSmemLeast = 120 * 1024;
constexpr int smem_bytes(int GR, int CG)
{
    const int n = 1024 + kFixed + 2 * bufs_for(GR, CG) * buf_bytes(GR, CG) + GR * kQBox;
    return n > kSmemLeast ? n : kSmemLeast;
}

// Tensor-memory columns: O [0, D), S / P two buffers of 64, Q D / 2.
template <int GR>
struct Cols {
    static constexpr uint32_t O = 0, S = 64 * GR, Q = 64 * GR + 128;
};

// Channel, within eight, of position p in the order in which the codes unpack.
template <int BITS>
__device__ __forceinline__ constexpr int unpacked(int p)
{
    return BITS == 4 ? (p < 4 ? 2 * p : 2 * (p - 4) + 1) : (p & 4) + ((p & 3) == 0 ? 0 : (p & 3) == 1 ? 2 : (p & 3) == 2 ? 1 : 3);
}

__device__ __forceinline__ void sts128(uint32_t addr, uint4 v)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// 32 lanes x 32 columns, complete on return: the load and its wait are one statement, as
// nothing (not even a register copy) may touch the result between them.
__device__ __forceinline__ void tmem_ld_x32(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
// The same of 16 columns.
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[32]) { tmem_ld_x32(taddr, r); }
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[16]) { tmem_ld_x16(taddr, r); }
// Descriptor of an operand with its M/N side contiguous (128-byte swizzle): boxes of
// 64 contiguous elements x rows of 128 bytes; `lead` bytes between boxes, 1024 bytes
// between groups of eight rows.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t smem_addr, uint32_t lead)
{
    uint64_t d = 0;
    d |= static_cast<uint64_t>((smem_addr >> 4) & 0x3FFF);
    d |= static_cast<uint64_t>((lead >> 4) & 0x3FFF) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_x8(uint32_t taddr, const uint32_t (&r)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st_cols(uint32_t taddr, const uint32_t (&r)[16]) { tmem_st_x16(taddr, r); }
__device__ __forceinline__ void tmem_st_cols(uint32_t taddr, const uint32_t (&r)[8]) { tmem_st_x8(taddr, r); }
__device__ __forceinline__ uint4 lds128(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1, int c2)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
        : "memory");
}

// ---- a pair of CTAs
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
template <int CG>
__device__ __forceinline__ void pair_sync()  // every thread of the CTA, or of both
{
    __syncwarp();
    if constexpr (CG == 1)
        __syncthreads();
    else
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Arrives on a barrier of the first CTA of the pair.  What it announces is memory of this CTA that the MMAs of the
// first one read, so the arrival and the wait for it are of cluster scope.  Tensor memory needs no more than that between
// before_thread_sync and after_thread_sync.  For shared memory (kShared; made visible to the tensor cores by the
// writers' proxy fences) a release fence comes before the arrival, restricted to shared memory, and first_wait acquires.
// (An arrival of the plain form releases to its own CTA only; release.cluster waits for every access in flight:
// 2,048 tokens on 32,768 took 676 us with the first, 959 with the second, 686 with this fence before every arrival,
// 677 so.)
template <int CG, bool kShared>
__device__ __forceinline__ void arrive_first(uint64_t *bar)
{
    if constexpr (CG == 1) {
        mbar_arrive(bar);
    } else {
        if constexpr (kShared) asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
        asm volatile(
            "{\n\t.reg .b32 r;\n\t"
            "mapa.shared::cluster.u32 r, %0, 0;\n\t"
            "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [r];\n\t}" ::"r"(smem_u32(bar))
            : "memory");
    }
}
// The first CTA's wait for such a barrier, by a whole warp: mbar_wait with acquire at cluster scope.
template <int CG>
__device__ __forceinline__ bool first_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag, int *status)
{
    if constexpr (CG == 1) return warp_wait(bar, parity, abort_flag, status);
    const uint32_t addr = smem_u32(bar);
    auto done = [&]() {
        uint32_t r;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(r)
            : "r"(addr), "r"(parity), "r"(20000u)
            : "memory");
        return r != 0;
    };
    bool ok = done();
    if (!ok) {
        const uint64_t t0 = global_timer_ns();
#pragma unroll 1
        while (!(ok = done()) && !*abort_flag) {
            if (global_timer_ns() - t0 > LILY_WAIT_LIMIT_NS) {
                record_error(status, kErrDeviceTimeout);
                *abort_flag = 1;
                break;
            }
        }
    }
    return __all_sync(0xffffffffu, ok);
}
template <int CG>
__device__ __forceinline__ void alloc_tmem(uint32_t *dst)
{
    if constexpr (CG == 1) {
        tmem_alloc(dst, kTmemCols);
        tmem_relinquish();
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n\t"
                     "tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::"r"(smem_u32(dst)), "r"(kTmemCols)
                     : "memory");
    }
}
template <int CG>
__device__ __forceinline__ void free_tmem(uint32_t taddr)
{
    if constexpr (CG == 1)
        tmem_dealloc(taddr, kTmemCols);
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(kTmemCols) : "memory");
}
template <int CG>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    if constexpr (CG == 1)
        umma_ts(d, a, b, idesc, accumulate);
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
            "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
}
// Arrives on this barrier of every CTA of the pair when the MMAs issued so far are done.
template <int CG>
__device__ __forceinline__ void commit(uint64_t *bar)
{
    if constexpr (CG == 1)
        umma_commit(bar);
    else
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
                     "h"(static_cast<uint16_t>(3))
                     : "memory");
}

__device__ __forceinline__ uint64_t join64(uint32_t lo, uint32_t hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}

// ------------------------------------------------------------------ work list
__device__ __forceinline__ int length_of(const KvqAttnArgs &a, int L)
{
    const int cap = a.max_blocks * a.c.bs;
    if (L < 0 || L > cap) {
        record_error(&a.ctrl->status, kErrDeviceIndex);
        L = L < 0 ? 0 : cap;
    }
    return L;
}
// Query tokens of a sequence from row q0 on (rows outside the call's N are none).
__device__ __forceinline__ int queries_of(const KvqAttnArgs &a, int b, int &q0)
{
    q0 = a.cu_q[b];
    const int q1 = min(a.cu_q[b + 1], a.N);
    return q0 < 0 || q1 <= q0 ? 0 : q1 - q0;
}
__device__ __forceinline__ int tile_chunks(int m, int L, int t, int TQ)
{
    const int limit = min(L, L - m + min(m, (t + 1) * TQ));
    return limit > 0 ? (limit + kChunk - 1) / kChunk : 1;
}
// Chunks of the tiles [0, t) of a sequence, without the items' own cost.  All but the last tile have the limit
// x + i TQ, x = L - m + TQ: the sum of ceil(. / 64) is the arithmetic series less the
// residues, which repeat with period 64 / gcd(TQ, 64).
__device__ __forceinline__ long long chunks_before(int m, int L, int t, int TQ)
{
    const int n = (m + TQ - 1) / TQ, k = min(t, n - 1);
    if (k <= 0) return t >= n ? tile_chunks(m, L, n - 1, TQ) : 0;
    int x = L - m + TQ, z = 0;
    if (x <= 0) {  // tiles that see nothing count as one chunk
        z = min(k, -x / TQ + 1);
        x += z * TQ;
    }
    const long long cnt = k - z, y = x + kChunk - 1;
    long long total = cnt * y + TQ * (cnt * (cnt - 1) / 2);
    const int g = min(TQ & -TQ, kChunk), P = kChunk / g;
    const int full = static_cast<int>(cnt / P), rest = static_cast<int>(cnt % P);
    long long res = static_cast<long long>(full) * (P * (y % g) + g * (P * (P - 1) / 2));
    int r = static_cast<int>(y % kChunk);
    for (int i = 0; i < rest; ++i) {
        res += r;
        r = (r + TQ) % kChunk;
    }
    return z + (total - res) / kChunk + (t >= n ? tile_chunks(m, L, n - 1, TQ) : 0);
}

// The same in places of the work list: an item of n chunks has kItemCost + n, the first
// ones for taking it up.
__device__ __forceinline__ long long places_before(int m, int L, int t, int TQ)
{
    return chunks_before(m, L, t, TQ) + static_cast<long long>(kItemCost) * t;
}

// A CTA's place in the list: item (b, g, t) from place s0 on, `left` places in all.
struct Walk {
    int b, g, t, m, L, s0, q0;  // q0: the sequence's first query row
    long long left;
};
// Its share of the item: chunks [j0, j0 + n) of nch, `take` places.
struct Share {
    int j0, n, nch, take;
};
__device__ __forceinline__ Share share_of(const Walk &w, int TQ)
{
    Share h;
    h.nch = tile_chunks(w.m, w.L, w.t, TQ);
    h.take = static_cast<int>(min(static_cast<long long>(h.nch + kItemCost - w.s0), w.left));
    h.j0 = max(w.s0 - kItemCost, 0);
    h.n = max(w.s0 + h.take - kItemCost, 0) - h.j0;
    return h;
}

// c of `shares`: which share of the list; TQ: query tokens of an item.
template <int NT>  // threads of the CTA
__device__ __forceinline__ Walk first_item(const KvqAttnArgs &a, Fixed &F, int TQ, int c, int shares)
{
    Walk w{};
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    long long off, per_head;  // of share c's first place within its sequence; the sequence's places per KV head
    if (a.B <= 32) {
        // every warp for itself, a sequence per lane
        int m = 0, L = 0, q0 = 0;
        if (lane < a.B) {
            L = a.seq_lens[lane];
            m = queries_of(a, lane, q0);
        }
        long long per = 0;
        if (m > 0) {
            L = length_of(a, L);
            per = places_before(m, L, (m + TQ - 1) / TQ, TQ);
        }
        long long inc = per * a.c.H_kv;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long up = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += up;
        }
        const long long total = __shfl_sync(0xffffffffu, inc, 31), used = min(total, static_cast<long long>(shares));
        // an item for each share, where the longest is not much more than an even share
        const int tiles = (m + TQ - 1) / TQ;
        const int longest = __reduce_max_sync(0xffffffffu, m > 0 ? tile_chunks(m, L, tiles - 1, TQ) + kItemCost : 0);
        const int mine = static_cast<int>(min(static_cast<long long>(tiles) * a.c.H_kv, 4096LL));
        if (static_cast<int>(__reduce_add_sync(0xffffffffu, mine)) <= shares && longest <= total / shares + kUncut) {
            int upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += up;
            }
            const uint32_t in = __ballot_sync(0xffffffffu, c < upto);
            if (in == 0) return w;
            w.b = __ffs(in) - 1;
            w.m = __shfl_sync(0xffffffffu, m, w.b);
            w.L = __shfl_sync(0xffffffffu, L, w.b);
            w.q0 = __shfl_sync(0xffffffffu, q0, w.b);
            const int i = c - __shfl_sync(0xffffffffu, upto - mine, w.b), n = (w.m + TQ - 1) / TQ;
            w.g = i / n;
            w.t = i % n;
            w.left = tile_chunks(w.m, w.L, w.t, TQ) + kItemCost;
            return w;
        }
        if (c >= used) return w;
        const long long begin = total * c / used;
        w.left = total * (c + 1) / used - begin;
        w.b = __ffs(__ballot_sync(0xffffffffu, begin < inc)) - 1;
        w.m = __shfl_sync(0xffffffffu, m, w.b);
        w.L = __shfl_sync(0xffffffffu, L, w.b);
        w.q0 = __shfl_sync(0xffffffffu, q0, w.b);
        per_head = __shfl_sync(0xffffffffu, per, w.b);
        off = begin - (__shfl_sync(0xffffffffu, inc, w.b) - per_head * a.c.H_kv);
        if (tid == 0) {
            F.begin = begin;
            F.total = total;
            F.used = used;
        }
    } else {
        int m = 0, L = 0, q0 = 0;
        long long per = 0, before = 0, all = 0;  // this thread's sequence: places per KV head
        auto scan = [&](int s0) {
            m = L = 0;
            per = 0;
            if (s0 + tid < a.B && (m = queries_of(a, s0 + tid, q0)) > 0) {
                L = length_of(a, a.seq_lens[s0 + tid]);
                per = places_before(m, L, (m + TQ - 1) / TQ, TQ);
            }
            const long long n = per * a.c.H_kv;
            long long inc = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long up = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += up;
            }
            __syncthreads();
            if (lane == 31) F.sum[warp] = inc;
            __syncthreads();
            before = inc - n;
            all = 0;
            for (int i = 0; i < NT / 32; ++i) {
                if (i < warp) before += F.sum[i];
                all += F.sum[i];
            }
        };
        long long total = 0;
        for (int s0 = 0; s0 < a.B; s0 += NT) {
            scan(s0);
            total += all;
        }
        // no more CTAs than places: every CTA between an item's first and last has a part of it
        const long long used = min(total, static_cast<long long>(shares));
        if (c >= used) return w;
        const long long begin = total * c / used;
        w.left = total * (c + 1) / used - begin;
        long long pre = 0;
        for (int s0 = 0; s0 < a.B; s0 += NT) {
            if (a.B > NT) scan(s0);
            const long long lo = pre + before;
            if (begin >= lo && begin < lo + per * a.c.H_kv) {
                F.b0 = s0 + tid;
                F.m0 = m;
                F.L0 = L;
                F.q0 = q0;
                F.pre = lo;
                F.per = per;
                F.begin = begin;
                F.total = total;
                F.used = used;
            }
            pre += all;
            if (begin < pre) break;
        }
        __syncthreads();
        w.b = F.b0;
        w.m = F.m0;
        w.L = F.L0;
        w.q0 = F.q0;
        off = begin - F.pre;
        per_head = F.per;
    }
    w.g = static_cast<int>(off / per_head);
    const long long r = off % per_head;
    // the tile that place r falls into: the last t with places_before(t) <= r, 32 candidates at a time
    int t_lo = 0, t_hi = (w.m + TQ - 1) / TQ;  // places_before(t_lo) <= r < places_before(t_hi)
    while (t_hi - t_lo > 1) {
        const int step = (t_hi - t_lo + 31) / 32, t = min(t_lo + lane * step, t_hi);
        const uint32_t ok = __ballot_sync(0xffffffffu, t < t_hi && places_before(w.m, w.L, t, TQ) <= r);
        const int last = 31 - __clz(ok);
        t_lo += last * step;
        t_hi = min(t_lo + step, t_hi);
    }
    w.t = t_lo;
    w.s0 = static_cast<int>(r - places_before(w.m, w.L, t_lo, TQ));
    return w;
}

// The next item after `take` places of this one.
__device__ __forceinline__ void advance(const KvqAttnArgs &a, Walk &w, int take, int TQ)
{
    w.left -= take;
    w.s0 = 0;
    if (w.left <= 0) return;
    if (++w.t * TQ < w.m) return;
    w.t = 0;
    if (++w.g < a.c.H_kv) return;
    w.g = 0;
    do {
        w.m = queries_of(a, ++w.b, w.q0);
    } while (w.m == 0 && w.b + 1 < a.B);  // places are still to come, so there is one
    w.L = length_of(a, a.seq_lens[w.b]);
}
// From here to an item with chunks for this CTA (only its last item may have none).
__device__ __forceinline__ bool next_share(const KvqAttnArgs &a, const Walk &w, Share &h, int TQ)
{
    if (w.left <= 0) return false;
    h = share_of(w, TQ);
    return h.n > 0;
}

// ------------------------------------------------------------------ the kernel
// Codes of one (token, group) in registers.
template <int BITS>
struct Raw {
    uint4 q[BITS / 2];
    uint32_t sb;
};

// Values in fp16, the multiply-add in fp32.
template <int BITS>
__device__ __noinline__ void rebuild_f32(const uint32_t *codes, float s, float b, uint32_t row_addr)
{
    constexpr uint32_t L = (1u << BITS) - 1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const unsigned long long w = BITS == 4 ? codes[i] : codes[2 * i] | static_cast<unsigned long long>(codes[2 * i + 1]) << 32;
        uint32_t v[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const int c0 = BITS * unpacked<BITS>(2 * p), c1 = BITS * unpacked<BITS>(2 * p + 1);
            v[p] = pack_f16(fmaf(__uint2float_rn(static_cast<uint32_t>(w >> c0) & L), s, b),
                            fmaf(__uint2float_rn(static_cast<uint32_t>(w >> c1) & L), s, b));
        }
        sts128(row_addr ^ (i << 4), make_uint4(v[0], v[1], v[2], v[3]));
    }
}

// Values code * scale + bias in fp16, each rounded once.  4 bits: the nibbles are e2m3
// bit patterns of code / 8, which converts exactly, and the multiply-add gets 8 scale.
// 8 bits: the code under the exponent of 128 is 128 + code / 8, so 128 is taken off exactly
// first.  That needs 8 scale and the bias to be fp16 numbers, which the test at the end makes sure of:
// scales from 2^-20 to 8176 and biases from 2^-17 are (8 significant bits above 2^-24), and 4-bit groups from
// about -61000 to 61000 have larger scales; what a smaller scale lost the code would multiply, by up to 32.
// The rare group that fails the test is done over in fp32.  The test comes after the stores
// so that nothing waits for it (a 2K chunk at the end of 32K 669 us without it, 673 here, 686 with it first).  Where
// every group fails it (V of 2^-24), that chunk takes 1.3 times as long.
template <int BITS>
__device__ __forceinline__ void rebuild(const Raw<BITS> &raw, bool exists, uint32_t row_addr, int *status)
{
    const uint32_t sb = exists ? raw.sb : 0u;  // rows behind the sequence, whatever they hold
    const float s = lo_bf16(sb), b = hi_bf16(sb);
    constexpr float L = BITS == 4 ? 15.0f : 255.0f;
    const uint32_t *q = reinterpret_cast<const uint32_t *>(raw.q);
    const __half2 s2 = __float2half2_rn(s * 8.0f), b2 = __float2half2_rn(b);
    auto value = [&](uint32_t w) {
        const uint32_t x = (w & 0x00FF00FFu) | 0x58005800u, off = 0xD800D800u;
        const __half2 v = __hfma2(__hadd2(*reinterpret_cast<const __half2 *>(&x), *reinterpret_cast<const __half2 *>(&off)), s2, b2);
        return *reinterpret_cast<const uint32_t *>(&v);
    };
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint4 v;
        if constexpr (BITS == 4)  // channels (0, 2), (4, 6), (1, 3), (5, 7)
            v = dequant8_f16_e2m3(q[i], s2, b2);
        else                      // channels (0, 2), (1, 3), (4, 6), (5, 7)
            v = make_uint4(value(q[2 * i]), value(q[2 * i] >> 8), value(q[2 * i + 1]), value(q[2 * i + 1] >> 8));
        sts128(row_addr ^ (i << 4), v);
    }
    if (!(__low2float(s2) == s * 8.0f && __low2float(b2) == b && fmaf(L, fabsf(s), fabsf(b)) < 65504.0f)) {
        // (a NaN is in no range)
        if (!(fabsf(b) < 65520.0f && fabsf(fmaf(L, s, b)) < 65520.0f)) record_error(status, kErrDeviceRange);
        Raw<BITS> copy = raw;
        rebuild_f32<BITS>(reinterpret_cast<const uint32_t *>(copy.q), s, b, row_addr);
    }
}

template <int BITS, int GR, int CG, int NQ>
__global__ void __launch_bounds__(Roles<NQ>::threads, 1) kvq_prefill_kernel(const __grid_constant__ KvqAttnArgs a, const __grid_constant__ CUtensorMap tmQ)
{
    constexpr int D = 64 * GR, GB = 8 * BITS;
    extern __shared__ uint8_t dsm_raw[];
    uint8_t *base = dsm_raw + ((1024 - (smem_u32(dsm_raw) & 1023)) & 1023);
    Fixed &F = *reinterpret_cast<Fixed *>(base);
    constexpr int kBufs = bufs_for(GR, CG), BB = buf_bytes(GR, CG), kKBox = kBox / CG;  // BB: bytes of a K or V buffer, kKBox: of a K box
    constexpr int VG = GR / CG, NK = 2 * GR / CG;         // groups of V in this CTA; warps for K of a chunk, and for V
    const uint32_t k_smem = smem_u32(base) + kFixed, v_smem = k_smem + kBufs * BB, q_smem = v_smem + kBufs * BB;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = CG == 1 ? 0 : static_cast<int>(cluster_rank()), share = blockIdx.x / CG;
    using R = Roles<NQ>;
    const int G = a.group, TQ = 32 * NQ / G, TI = CG * TQ;  // query tokens of this CTA's rows, of an item
    int *status = &a.ctrl->status;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kBufs; ++i) {
            mbar_init(&F.k_full[i], CG * NK);
            mbar_init(&F.v_full[i], CG * NK);
            mbar_init(&F.k_free[i], 1);
            mbar_init(&F.v_free[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&F.s_full[i], 1);
            mbar_init(&F.p_full[i], CG * R::soft);
            mbar_init(&F.pv_done[i], 1);
        }
        mbar_init(&F.q_full, CG * R::soft);
        mbar_init(&F.q_loaded, 1);
        mbar_init(&F.q_free, R::soft);
        mbar_init(&F.o_free, CG * R::soft);
        mbar_init(&F.drain, 1);
#ifdef LILY_TEST_STALL_T
        mbar_init(&F.never, 1);
#endif
        F.abort = 0;
        fence_mbar_init();
    }
    if (warp == R::mma) alloc_tmem<CG>(&F.tmem);
    tc_fence_before();
    pair_sync<CG>();
    tc_fence_after();
    // the next kernel may start only now: its CTAs must not take the tensor memory that these wait for
    pdl_trigger();
    pdl_wait();
    const uint32_t tmem = F.tmem;
    Walk w = first_item<R::threads>(a, F, TI, share, kKvqPrefillCtas / CG);
    bool ok = true;

    if (R::is_soft(warp)) {
        // ------------------------------------------------ two or four threads per query row
        constexpr int NP = R::parts, NC = kChunk / NP;  // of a row, and its columns of a chunk
        const int quarter = warp & 3, part = warp >> 2, row = quarter * 32 + lane;
        auto quarter_sync = [&]() { named_barrier_sync(kBarPair + quarter, NP * 32); };
        // over the row's threads; all of them are done with xch[s] afterwards, if a quarter_sync comes before its next use
        auto others = [&](int s, float x, auto op) {
            F.xch[s][part][row] = x;
            quarter_sync();
#pragma unroll
            for (int o = 1; o < NP; ++o) x = op(x, F.xch[s][(part + o) & (NP - 1)][row]);
            return x;
        };
        auto larger = [](float x, float y) { return fmaxf(x, y); };
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        Share h, h2;
        bool more = next_share(a, w, h, TI);
        int it = 0, items = 0, mine = 1;  // mine: this CTA's meta entry is still to be written
        long long done = 0;
        float mul = 0.0f;

        // item x's q from shared memory to tensor memory: this thread's row, every second group of 64 channels
        auto take_q = [&](int x) {
            ok = ok && warp_wait(&F.q_loaded, x & 1, &F.abort, status);
            const uint32_t src = q_smem + row * 128;
            const int sw = row & 7;
            float big = 0.0f;
#pragma unroll
            for (int c = part; c < GR; c += NP)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint4 y = lds128(src + c * kQBox + ((i ^ sw) << 4));
                    big = fmaxf(big, fmaxf(fmaxf(fabsf(lo_bf16(y.x)), fabsf(hi_bf16(y.x))), fmaxf(fabsf(lo_bf16(y.y)), fabsf(hi_bf16(y.y)))));
                    big = fmaxf(big, fmaxf(fmaxf(fabsf(lo_bf16(y.z)), fabsf(hi_bf16(y.z))), fmaxf(fabsf(lo_bf16(y.w)), fabsf(hi_bf16(y.w)))));
                }
            quarter_sync();  // the others are done with xch
            big = others(0, big, larger);
            quarter_sync();
            // times 2^(14 - floor(log2 big)), within the normal numbers, and the sign of the scale
            const int ef = big > 0.0f ? min(268 - max(static_cast<int>(__float_as_uint(big) >> 23), 1), 253) : 127;
            const float up = copysignf(__uint_as_float(static_cast<uint32_t>(ef) << 23), a.scale_log2);
            // never 0: a masked score is -inf, and stays it
            mul = fmaxf(fabsf(a.scale_log2) * __uint_as_float(static_cast<uint32_t>(254 - ef) << 23), 1.17549435e-38f);
#pragma unroll
            for (int c = part; c < GR; c += NP) {
                uint32_t r[32];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint4 y = lds128(src + c * kQBox + ((i ^ sw) << 4));
                    const uint32_t xs[4] = {y.x, y.y, y.z, y.w};
                    float f[8];
#pragma unroll
                    for (int p = 0; p < 8; ++p) {
                        const int ch = unpacked<BITS>(p);
                        f[p] = (ch & 1 ? hi_bf16(xs[ch / 2]) : lo_bf16(xs[ch / 2])) * up;
                    }
#pragma unroll
                    for (int p = 0; p < 4; ++p) r[4 * i + p] = pack_f16(f[2 * p], f[2 * p + 1]);
                }
                if (ok) tmem_st_32x32b_x32(lanes + Cols<GR>::Q + c * 32, r);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                arrive_first<CG, false>(&F.q_full);
                mbar_arrive(&F.q_free);
            }
        };
        // A warp whose wait gave up goes on through the named barriers (its partner may be in one), without the work.
        if (more) take_q(0);
        while (more) {
            const int tq = w.t * TI + rank * TQ + row / G, head = w.g * G + row % G;
            const bool valid = row < TQ * G && tq < w.m;
            const int limit = valid ? w.L - w.m + tq + 1 : 0;  // tokens this row sees (may be <= 0)
            const bool any_row = __any_sync(0xffffffffu, valid);
            float m_run = kNoMax, l_run = 0.0f;
            const float item_mul = mul;
            for (int i = 0; i < h.n; ++i, ++it) {
                const int sb = it & 1;
#ifdef LILY_TEST_STALL_T
                // Test builds only: with that many query tokens the first chunk of every second CTA waits for a barrier that
                // nothing completes, so that the wait runs out and every role of its pair gives up.
                if (a.N == LILY_TEST_STALL_T && blockIdx.x % 2 == 0 && threadIdx.x < 32 && it == 0) ok = ok && warp_wait(&F.never, 0, &F.abort, status);
#endif
                ok = ok && warp_wait(&F.s_full[sb], (it >> 1) & 1, &F.abort, status);
                if (any_row) {
                    tc_fence_after();
                    const int vis = limit - (h.j0 + i) * kChunk - part * NC;  // of this thread's columns, those the row sees
                    uint32_t s[NC] = {};
                    if (ok) tmem_ld_cols(lanes + Cols<GR>::S + sb * 64 + part * NC, s);
                    if (__any_sync(0xffffffffu, vis < NC)) {
#pragma unroll
                        for (int x = 0; x < NC; ++x)
                            if (x >= vis) s[x] = 0xFF800000u;  // -inf
                    }
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int x = 0; x < NC; x += 2)  // three operands a step
                        mx[(x >> 1) & 3] = fmaxf(fmaxf(mx[(x >> 1) & 3], __uint_as_float(s[x])), __uint_as_float(s[x + 1]));
                    // (after its barrier all of the row's S is in registers, so P may overwrite it)
                    const float top = others(sb, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), larger);
                    const float mn = top > -INFINITY ? fmaf(top, item_mul, -kLift) : kNoMax;
                    if (__any_sync(0xffffffffu, mn > m_run + 8.0f)) {  // the same in all parts
                        const float to = fmaxf(m_run, mn), al = ex2(m_run - to);
                        m_run = to;
                        l_run *= al;
                        if (i > 0) {
                            // O of the chunks before this one, once their products are done
                            ok = ok && warp_wait(&F.pv_done[(it - 1) & 1], ((it - 1) >> 1) & 1, &F.abort, status);
                            tc_fence_after();
#pragma unroll 1
                            for (int c = part; c < D / 32 && ok; c += NP) {
                                uint32_t o[32];
                                tmem_ld_x32(lanes + Cols<GR>::O + c * 32, o);
#pragma unroll
                                for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * al);
                                tmem_st_32x32b_x32(lanes + Cols<GR>::O + c * 32, o);
                            }
                            tmem_st_wait();
                        }
                    }
                    uint32_t p[NC / 2];
                    unsigned long long sum[2] = {0ull, 0ull};
                    const unsigned long long mul2 = pair(item_mul, item_mul), neg2 = pair(-m_run, -m_run);
#pragma unroll
                    for (int x = 0; x < NC / 2; ++x) {
                        float e0, e1;
                        unpair(fma2(pair(__uint_as_float(s[2 * x]), __uint_as_float(s[2 * x + 1])), mul2, neg2), e0, e1);
                        e0 = ex2(e0);
                        e1 = ex2(e1);
                        sum[x & 1] = add2(sum[x & 1], pair(e0, e1));
                        p[x] = pack_f16(e0, e1);
                    }
                    {
                        float a0, a1;
                        unpair(add2(sum[0], sum[1]), a0, a1);
                        l_run += a0 + a1;
                    }
                    if (ok) tmem_st_cols(lanes + Cols<GR>::S + sb * 64 + part * (NC / 2), p);
                    tmem_st_wait();
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) arrive_first<CG, false>(&F.p_full[sb]);
            }
            // ---- the item's end.  The next item's q first: the last scores of this one are in (S is full), so Q is free
            Walk w2 = w;
            advance(a, w2, h.take, TI);
            const bool more2 = next_share(a, w2, h2, TI);
            if (more2) take_q(items + 1);
            ok = ok && warp_wait(&F.pv_done[(it - 1) & 1], ((it - 1) >> 1) & 1, &F.abort, status);
            tc_fence_after();
            const bool starts = h.j0 == 0, ends = h.j0 + h.n == h.nch;
            const size_t part_row = static_cast<size_t>(2 * share + (starts ? 1 : 0)) * (CG * kRows) + rank * kRows + row;
            if (any_row) {
                quarter_sync();
                l_run = others(0, l_run, [](float x, float y) { return x + y; });
                quarter_sync();
                const bool seen = l_run > 0.0f;  // a row that saw nothing has zeros
                const float r = seen ? 1.0f / l_run : 0.0f;
                const long long n = w.q0 + tq;
                uint16_t *dst = a.out + (n * a.H_q + head) * D;
                float *pdst = a.part_acc + part_row * D;
#pragma unroll 1
                for (int c = part; c < D / 32 && ok; c += NP) {
                    uint32_t o[32];
                    tmem_ld_x32(lanes + Cols<GR>::O + c * 32, o);
                    if (valid) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float x[8];
#pragma unroll
                            for (int p = 0; p < 8; ++p) x[unpacked<BITS>(p)] = seen ? __uint_as_float(o[8 * i + p]) : 0.0f;
                            if (starts && ends) {
                                uint32_t y[4];
#pragma unroll
                                for (int p = 0; p < 4; ++p) {
                                    const __nv_bfloat162 t = __floats2bfloat162_rn(x[2 * p] * r, x[2 * p + 1] * r);
                                    y[p] = *reinterpret_cast<const uint32_t *>(&t);
                                }
                                *reinterpret_cast<uint4 *>(dst + c * 32 + i * 8) = make_uint4(y[0], y[1], y[2], y[3]);
                            } else {
                                *reinterpret_cast<float4 *>(pdst + c * 32 + i * 8) = make_float4(x[0], x[1], x[2], x[3]);
                                *reinterpret_cast<float4 *>(pdst + c * 32 + i * 8 + 4) = make_float4(x[4], x[5], x[6], x[7]);
                            }
                        }
                    }
                    __syncwarp();
                }
                if (valid && part == 0 && !(starts && ends))
                    *reinterpret_cast<float2 *>(a.part_ml + part_row * 2) = make_float2(m_run, l_run);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_first<CG, false>(&F.o_free);
            if (threadIdx.x == 0 && rank == 0 && starts && !ends) {
                // who joins the parts of an item that starts here and goes on: up to the CTA with its last place
                const long long last = ((F.begin + done - w.s0 + h.nch + kItemCost) * F.used - 1) / F.total;
                a.meta[share] = make_int4(w.q0 + w.t * TI, w.g, w.m - w.t * TI, static_cast<int>(last));
                mine = 0;
            }
            done += h.take;
            ++items;
            w = w2;
            h = h2;
            more = more2;
        }
        if (threadIdx.x == 0 && rank == 0 && mine) a.meta[share] = make_int4(-1, 0, 0, 0);
    } else if (warp < R::soft + R::deq) {
        // ------------------------------------------------ K and V of the chunks into shared memory
        // The chunk's (K or V, group, 32 tokens) are dealt to the warps: one each (two for one CTA with D = 256);
        // with fewer of them than warps, the warps take chunks in turn.  Of a pair, this CTA has half of the
        // chunk's tokens of K, and half of the groups of V.
        constexpr int kItems = 2 * NK > R::deq ? 2 * NK / R::deq : 1, kWarps = 2 * NK / kItems, kTurns = R::deq / kWarps;
        const int dw = R::deq_index(warp) % kWarps, turn = R::deq_index(warp) / kWarps;
        struct Item {
            uint32_t addr;  // this lane's row of the group in buffer 0
            int row, group, half;
            bool isv;
        } item[kItems];
#pragma unroll
        for (int x = 0; x < kItems; ++x) {
            Item &m = item[x];
            const int n = dw + x * kWarps, idx = n % NK;
            m.isv = n >= NK;
            m.half = !m.isv && CG == 2 ? rank : idx & 1;
            const int here = !m.isv && CG == 2 ? idx : idx >> 1;  // group within this CTA's
            m.group = m.isv && CG == 2 ? rank * VG + here : here;
            m.row = m.half * 32 + lane;
            const int r = !m.isv && CG == 2 ? lane : m.row;
            m.addr = (m.isv ? v_smem + here * kBox : k_smem + here * kKBox) + r * 128 + ((r & 7) << 4);
        }
        // every item of a warp has the same tokens (two items: K and V of the same group and half)
        const int half = item[0].half, row = item[0].row;
        const int bs_log = 31 - __clz(a.c.bs), block_rows = a.c.H_kv * GR * a.c.bs;
        int it = 0;
        Share h;
        while (ok && next_share(a, w, h, TI)) {
            const int end = h.j0 + h.n;
            // the table entries of this warp's 32 tokens of its next 32 chunks, one chunk per lane
            const int *table = a.block_table + static_cast<size_t>(w.b) * a.max_blocks;
            auto entries = [&](int c0) {
                const int j = c0 + lane * kTurns, tok = j * kChunk + half * 32;
                int e = 0;
                if (j < end && tok < w.L) {
                    e = table[tok >> bs_log];
                    if (e < 0 || e >= a.c.n_blocks) {
                        record_error(status, kErrDeviceIndex);
                        e = 0;
                    }
                }
                return e;
            };
            Raw<BITS> raw[kItems];
            auto fetch = [&](int x, int j, int block) {
                const uint32_t group0 = (static_cast<uint32_t>(w.g) * GR + item[x].group) << bs_log;  // rows before the group's in a block
                const long long gi = static_cast<long long>(block) * block_rows + (group0 + ((j * kChunk + row) & (a.c.bs - 1)));
                const uint4 *src = reinterpret_cast<const uint4 *>((item[x].isv ? a.c.v_q : a.c.k_q) + gi * GB);
#pragma unroll
                for (int y = 0; y < BITS / 2; ++y) raw[x].q[y] = src[y];
                raw[x].sb = reinterpret_cast<const uint32_t *>(item[x].isv ? a.c.v_sb : a.c.k_sb)[gi];
            };
            int j = h.j0 + ((turn - it) & (kTurns - 1)), cnt = 0, tab = entries(j);
            const int block0 = __shfl_sync(0xffffffffu, tab, 0);
#pragma unroll
            for (int x = 0; x < kItems; ++x)
                if (j < end) fetch(x, j, block0);
            for (; j < end && ok; j += kTurns) {
                const int x = it + j - h.j0, buf = x % kBufs, use = x / kBufs;
                uint32_t is_free[kItems];
#pragma unroll
                for (int y = 0; y < kItems; ++y)
                    is_free[y] = use > 0 ? phase_done(item[y].isv ? &F.v_free[buf] : &F.k_free[buf], (use - 1) & 1) : 1u;
                if ((++cnt & 31) == 0) tab = entries(j + kTurns);
                const int next = __shfl_sync(0xffffffffu, tab, cnt & 31);
#pragma unroll
                for (int y = 0; y < kItems; ++y) {
                    if (!__all_sync(0xffffffffu, is_free[y]) &&
                        !(ok = ok && warp_wait(item[y].isv ? &F.v_free[buf] : &F.k_free[buf], (use - 1) & 1, &F.abort, status)))
                        break;
                    rebuild<BITS>(raw[y], j * kChunk + row < w.L, item[y].addr + buf * BB, status);
                    fence_async_shared();
                    __syncwarp();
                    if (lane == 0) arrive_first<CG, true>(item[y].isv ? &F.v_full[buf] : &F.k_full[buf]);
                    if (j + kTurns < end) fetch(y, j + kTurns, next);
                }
            }
            it += h.n;
            advance(a, w, h.take, TI);
        }
    } else if (warp == R::load) {
        // ------------------------------------------------ q of the items, one ahead
        if (lane == 0) {
            prefetch_tmap(&tmQ);
            Share h;
            int items = 0;
            while (next_share(a, w, h, TI)) {
                if (items > 0 && !mbar_wait(&F.q_free, (items - 1) & 1, &F.abort, status)) break;
                mbar_arrive_expect_tx(&F.q_loaded, static_cast<uint32_t>(GR * TQ * G * 128));
#pragma unroll
                for (int c = 0; c < GR; ++c)
                    tma_load_3d(base + kFixed + 2 * kBufs * BB + c * kQBox, &tmQ, &F.q_loaded, c * 64, w.g * G,
                                w.q0 + w.t * TI + rank * TQ);
                ++items;
                advance(a, w, h.take, TI);
            }
            // no copy into this CTA's shared memory may still be in flight at exit
            if (items > 0) {
                const uint32_t addr = smem_u32(&F.q_loaded);
                const uint64_t t0 = global_timer_ns();
                while (!mbar_try_wait(addr, (items - 1) & 1))
                    if (global_timer_ns() - t0 > LILY_DRAIN_LIMIT_NS) {
                        record_error(status, kErrDeviceTimeout);
                        break;
                    }
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------ MMA issuer (of the pair's first CTA)
        // The whole warp walks the list, so that every operand of an MMA is warp-uniform, and one elected
        // lane issues: issuing from inside `if (lane == 0)` took ~87 cycles an MMA, more than it runs.
        constexpr uint32_t kIdescS = idesc_f32acc(kFmtF16, CG * kRows, kChunk);
        constexpr uint32_t kIdescO = idesc_f32acc(kFmtF16, CG * kRows, D) | (1u << 16);  // B: channels contiguous
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint64_t kd = sdesc_sw128(k_smem), vd = sdesc_mn_sw128(v_smem, kBox);
        int it = 0, items = 0;
        Share h;
        while (rank == 0 && ok && next_share(a, w, h, TI)) {
            const int n = __shfl_sync(0xffffffffu, h.n, 0);
            if (!(ok = first_wait<CG>(&F.q_full, items & 1, &F.abort, status))) break;
            tc_fence_after();
            for (int i = 0; i <= n && ok; ++i) {
                if (i < n) {
                    const int x = it + i, buf = x % kBufs, sb = x & 1;
                    if (!(ok = first_wait<CG>(&F.k_full[buf], (x / kBufs) & 1, &F.abort, status))) break;
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t lo = static_cast<uint32_t>(kd) + buf * (BB >> 4), hi = static_cast<uint32_t>(kd >> 32);
#pragma unroll
                        for (int c = 0; c < GR; ++c)
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                mma_ts<CG>(tm + Cols<GR>::S + sb * 64, tm + Cols<GR>::Q + c * 32 + kk * 8,
                                           join64(lo + c * (kKBox >> 4) + kk * 2, hi), kIdescS, (c | kk) != 0);
                        commit<CG>(&F.k_free[buf]);
                        commit<CG>(&F.s_full[sb]);
                    }
                    __syncwarp();
                }
                if (i > 0) {
                    const int x = it + i - 1, buf = x % kBufs, sb = x & 1;
                    if (i == 1 && items > 0 && !(ok = first_wait<CG>(&F.o_free, (items - 1) & 1, &F.abort, status))) break;
                    if (!(ok = first_wait<CG>(&F.v_full[buf], (x / kBufs) & 1, &F.abort, status))) break;
                    if (!(ok = first_wait<CG>(&F.p_full[sb], (x >> 1) & 1, &F.abort, status))) break;
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t lo = static_cast<uint32_t>(vd) + buf * (BB >> 4), hi = static_cast<uint32_t>(vd >> 32);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_ts<CG>(tm + Cols<GR>::O, tm + Cols<GR>::S + sb * 64 + kk * 8, join64(lo + kk * (2048 >> 4), hi), kIdescO,
                                       i > 1 || kk > 0);
                        commit<CG>(&F.v_free[buf]);
                        commit<CG>(&F.pv_done[sb]);
                    }
                    __syncwarp();
                }
            }
            it += n;
            ++items;
            advance(a, w, h.take, TI);
        }
        if (rank == 0 && elect_one()) {
            // all tensor-core work must finish before tensor memory is freed (the pair's other CTA waits below)
            commit<CG>(&F.drain);
            const uint32_t addr = smem_u32(&F.drain);
            const uint64_t t0 = global_timer_ns();
            while (!mbar_try_wait(addr, 0))
                if (global_timer_ns() - t0 > LILY_DRAIN_LIMIT_NS) {
                    record_error(status, kErrDeviceTimeout);
                    break;
                }
        }
        __syncwarp();
    }
    // no CTA of a pair leaves while the other may still signal it or read its shared memory
    tc_fence_before();
    __syncwarp();
    pair_sync<CG>();
    tc_fence_after();
    if (warp == R::mma) free_tmem<CG>(tmem);
}

// Joins the parts of an item that was cut: CTA (first share of the item, four rows, every
// gridDim.y-th four of them), 64 threads a row, a float4 column each, on a running maximum.
// An item of a pair is cut in two as a rule: two parts in flight with many CTAs on an SM (an
// 8K prompt's join 9 us; eight in flight 15).  One row per CTA took 20 us to launch.  The part
// of the first share c0 is in slot 2 c0 + 1, those of the following ones c in slot 2 c.
template <int CG>
__global__ void __launch_bounds__(256, CG == 2 ? 8 : 2) kvq_prefill_join_kernel(const __grid_constant__ KvqAttnArgs a)
{
    constexpr int kBatch = CG == 2 ? 2 : 8;
    pdl_trigger();
    pdl_wait();
    const int4 meta = a.meta[blockIdx.x];
    if (meta.x < 0) return;
    const int G = a.group, TQ = kRows / G, d4 = threadIdx.x % 64, c0 = blockIdx.x, S = meta.w - c0 + 1;
    if (d4 * 4 >= a.D) return;
    for (int row = blockIdx.y * 4 + threadIdx.x / 64; row < CG * kRows; row += gridDim.y * 4) {
        const int r = row % kRows, tq = row / kRows * TQ + r / G;  // query token within the item
        if (r >= TQ * G || tq >= meta.z) continue;
        auto slot = [&](int s) { return static_cast<size_t>(s == 0 ? 2 * c0 + 1 : 2 * (c0 + s)) * (CG * kRows) + row; };
        float M = kNoMax, den = 0.0f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s0 = 0; s0 < S; s0 += kBatch) {
            float2 ml[kBatch];
            float4 x[kBatch];
            float to = M;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int s = s0 + k;
                ml[k] = s < S ? *reinterpret_cast<const float2 *>(a.part_ml + slot(s) * 2) : make_float2(kNoMax, 0.0f);
                x[k] = s < S ? reinterpret_cast<const float4 *>(a.part_acc + slot(s) * a.D)[d4] : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) to = fmaxf(to, ml[k].x);
            const float c = ex2(M - to);
            M = to;
            den *= c;
            o.x *= c;
            o.y *= c;
            o.z *= c;
            o.w *= c;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const float e = ex2(ml[k].x - to);
                den = fmaf(e, ml[k].y, den);
                o.x = fmaf(e, x[k].x, o.x);
                o.y = fmaf(e, x[k].y, o.y);
                o.z = fmaf(e, x[k].z, o.z);
                o.w = fmaf(e, x[k].w, o.w);
            }
        }
        const float inv = den > 0.0f ? 1.0f / den : 0.0f;
        uint2 y;
        const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * inv, o.y * inv), hi = __floats2bfloat162_rn(o.z * inv, o.w * inv);
        y.x = *reinterpret_cast<const uint32_t *>(&lo);
        y.y = *reinterpret_cast<const uint32_t *>(&hi);
        const long long n = meta.x + tq;
        reinterpret_cast<uint2 *>(a.out + (n * a.H_q + meta.y * G + r % G) * a.D)[d4] = y;
    }
}

// The same where items are few (no more than shares) and may have up to 152 parts or not be cut
// at all: the query rows of the cut ones are one list that the CTAs go through, found by
// a scan over the shares' entries.  64 threads take a row; where an item has more parts than
// a thread has loads in flight, a CTA takes one row and its four groups of 64 threads every
// fourth part each, joined through shared memory in a fixed order.  16 tokens on 32,768: 35 us
// for the call, 45 with the kernel above (which is the faster where items are many: a prompt of
// 8,192 tokens 396 us, 402 with the list).
template <int CG, int NQ>
__global__ void __launch_bounds__(256, 2) kvq_prefill_join_few_kernel(const __grid_constant__ KvqAttnArgs a)
{
    constexpr int kBatch = 8, kShares = kKvqPrefillCtas / CG;
    __shared__ int4 metas[kShares];
    __shared__ int upto[kShares], warp_sum[8];  // units of the shares up to this one
    __shared__ float4 part[4][64];
    __shared__ float2 part_ml[4];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, d4 = tid % 64, slot0 = tid / 64;
    const int G = a.group, TQ = 32 * NQ / G;
    pdl_trigger();
    pdl_wait();
    const int4 mine = tid < kShares ? a.meta[tid] : make_int4(-1, 0, 0, 0);
    const int rows = mine.x >= 0 ? min(mine.z, CG * TQ) * G : 0;
    const bool by_row = __syncthreads_or(mine.x >= 0 && mine.w - tid + 1 > kBatch);
    int inc = by_row ? rows : (rows + 3) / 4;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += up;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    for (int i = 0; i < warp; ++i) inc += warp_sum[i];
    if (tid < kShares) {
        metas[tid] = mine;
        upto[tid] = inc;
    }
    __syncthreads();
    const int total = upto[kShares - 1];
    for (int u = blockIdx.x; u < total; u += gridDim.x) {
        int c0 = -1, last = kShares - 1;  // the first share with upto > u
        while (last - c0 > 1) {
            const int mid = (c0 + last) >> 1;
            if (upto[mid] > u)
                last = mid;
            else
                c0 = mid;
        }
        const int local = u - (c0 >= 0 ? upto[c0] : 0);
        c0 = last;
        const int4 meta = metas[c0];
        const int S = meta.w - c0 + 1, i = by_row ? local : local * 4 + slot0, tq = i / G, h = i % G;  // query token, head
        const bool valid = tq < min(meta.z, CG * TQ) && d4 * 4 < a.D;
        const int row = tq / TQ * kRows + tq % TQ * G + h;
        auto slot = [&](int s) { return static_cast<size_t>(s == 0 ? 2 * c0 + 1 : 2 * (c0 + s)) * (CG * kRows) + row; };
        float M = kNoMax, den = 0.0f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        auto add = [&](float e, float l, const float4 &x) {
            den = fmaf(e, l, den);
            o.x = fmaf(e, x.x, o.x);
            o.y = fmaf(e, x.y, o.y);
            o.z = fmaf(e, x.z, o.z);
            o.w = fmaf(e, x.w, o.w);
        };
        const int step = by_row ? 4 : 1;
        for (int s0 = by_row ? slot0 : 0; valid && s0 < S; s0 += kBatch * step) {
            float2 ml[kBatch];
            float4 x[kBatch];
            float to = M;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int s = s0 + k * step;
                ml[k] = s < S ? *reinterpret_cast<const float2 *>(a.part_ml + slot(s) * 2) : make_float2(kNoMax, 0.0f);
                x[k] = s < S ? reinterpret_cast<const float4 *>(a.part_acc + slot(s) * a.D)[d4] : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) to = fmaxf(to, ml[k].x);
            const float4 before = o;
            const float e = ex2(M - to), l = den;
            M = to;
            den = 0.0f;
            o = make_float4(0.f, 0.f, 0.f, 0.f);
            add(e, l, before);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) add(ex2(ml[k].x - to), ml[k].y, x[k]);
        }
        if (by_row) {
            __syncthreads();  // the last row's are read
            part[slot0][d4] = o;
            if (d4 == 0) part_ml[slot0] = make_float2(M, den);
            __syncthreads();
            if (slot0 > 0) continue;
            M = kNoMax;
            for (int k = 0; k < 4; ++k) M = fmaxf(M, part_ml[k].x);
            den = 0.0f;
            o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k = 0; k < 4; ++k) add(ex2(part_ml[k].x - M), part_ml[k].y, part[k][d4]);
        }
        if (!valid) continue;
        const float inv = den > 0.0f ? 1.0f / den : 0.0f;
        uint2 y;
        const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * inv, o.y * inv), hi = __floats2bfloat162_rn(o.z * inv, o.w * inv);
        y.x = *reinterpret_cast<const uint32_t *>(&lo);
        y.y = *reinterpret_cast<const uint32_t *>(&hi);
        const long long n = meta.x + tq;
        reinterpret_cast<uint2 *>(a.out + (n * a.H_q + meta.y * G + h) * a.D)[d4] = y;
    }
}

// Whether no sequence need have more query tokens than `rows` rows hold.
bool few_queries(const KvqAttnArgs &a, int rows) { return a.N <= static_cast<long long>(a.B) * (rows / a.group); }

template <int BITS, int GR, int CG, int NQ>
cudaError_t launch(const KvqAttnArgs &a, const CUtensorMap &tmQ, cudaStream_t stream)
{
    constexpr int smem = smem_bytes(GR, CG);
    cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void *>(kvq_prefill_kernel<BITS, GR, CG, NQ>), smem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CG;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(kKvqPrefillCtas);
    cfg.blockDim = dim3(Roles<NQ>::threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if ((e = cudaLaunchKernelEx(&cfg, kvq_prefill_kernel<BITS, GR, CG, NQ>, a, tmQ)) != cudaSuccess) return e;
    const long long items = (a.N / (CG * (32 * NQ / a.group)) + static_cast<long long>(a.B)) * a.c.H_kv;  // at most
    if (few_queries(a, kRows) || items <= kKvqPrefillCtas / CG)
        return launch_pdl(kvq_prefill_join_few_kernel<CG, NQ>, dim3(4 * kKvqPrefillCtas), dim3(256), 0, stream, a);
    return launch_pdl(kvq_prefill_join_kernel<CG>, dim3(kKvqPrefillCtas / CG, CG == 1 ? 16 : 64), dim3(256), 0, stream, a);
}

// Pairs, but one CTA an item where D = 64 (its 64 channels of V are one swizzled box and
// do not split) and where no sequence need have more query tokens than one CTA's 128
// rows hold: a pair's second half would idle (eight drafts of four tokens, without the rule below:
// 28 us against 34; prompts and chunks of 1,024 tokens and more are 1.15 to 1.25 times as fast with pairs).
// Where 32 rows hold them, a tile has 32 rows, four threads a row and sixteen rebuild warps
// (28.3 us with the 128-row tile, 25.0 with two threads a row, 24.7 with four).
template <int BITS, int GR>
cudaError_t launch_rows(const KvqAttnArgs &a, const CUtensorMap &tmQ, cudaStream_t stream)
{
    if (few_queries(a, 32)) return launch<BITS, GR, 1, 1>(a, tmQ, stream);
    if (GR == 1 || few_queries(a, kRows)) return launch<BITS, GR, 1, 4>(a, tmQ, stream);
    return launch<BITS, GR, GR == 1 ? 1 : 2, 4>(a, tmQ, stream);
}
template <int BITS>
cudaError_t launch_d(const KvqAttnArgs &a, const CUtensorMap &tmQ, cudaStream_t stream)
{
    return a.D == 64 ? launch_rows<BITS, 1>(a, tmQ, stream) : a.D == 128 ? launch_rows<BITS, 2>(a, tmQ, stream) : launch_rows<BITS, 4>(a, tmQ, stream);
}

}  // namespace

int kvq_prefill_tile_rows(const KvqAttnArgs &a) { return few_queries(a, 32) ? 32 : kRows; }

cudaError_t launch_kvq_prefill(const KvqAttnArgs &a, const CUtensorMap &tmQ, cudaStream_t stream)
{
    return a.c.bits == 4 ? launch_d<4>(a, tmQ, stream) : launch_d<8>(a, tmQ, stream);
}

}  // namespace lily
