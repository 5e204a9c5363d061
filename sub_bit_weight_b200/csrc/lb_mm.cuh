// Matrix products on pairs of SMs: the main loop shared by the training
// operators (loss over the vocabulary, orthogonalised update).
//
//     D[i][j] = sum_k A(i, k) B(j, k),   16-bit operands, fp32 accumulation in tensor memory
//
// Either operand may be K-major (rows of k, as stored [i][k]) or MN-major
// (stored [k][i]): the tensor core reads both, so no operand is transposed in
// memory.  One output tile is 256 x 256 and belongs to a CTA pair
// (tcgen05.mma.cta_group::2, M = 256): each CTA of the pair holds 128 of the
// tile's i in its tensor memory and stages 128 i of A and 128 j of B per 64 k,
// 32 KB for 128 x 256 x 64 multiply-adds.  A CTA by itself with the same
// accumulator would have to stage 48 KB for them, and the operand stream from
// L2 is what paces such a kernel.  A problem with few tiles takes them 128 or
// 64 columns wide.
//
// Roles (12 warps a CTA): warps 0 and 2 issue the TMA copies of their CTA's
// half of A and of B; warp 1 of the pair's first CTA issues the MMAs for both;
// warps 4-11 are the epilogue (128 rows of the CTA, one thread a row and half
// of the columns; an epilogue that holds its columns in registers takes
// registers over from warps 0-3).  Two accumulators of 256 columns let the
// epilogue of one unit overlap the main loop of the next.  Units (tile, or a k
// range of a tile) are dealt to the pairs in order; a launch may hold several
// problems.
//
// What bounds it: 64 k of a 256 x 256 tile are 512 cycles of the tensor cores,
// and the 32 KB a CTA copies for them are 64 bytes a cycle, about what an SM
// gets from L2.  Measured (cycles for 64 k, where a logit GEMM of 2048 x 32000
// x 5120 runs): 786 with one thread for both copies and loop state in shared
// memory, 614 with two threads and registers, 513 with the issuing warps
// converged, so that descriptors stay in uniform registers; that is 1.36 PFLOP/s,
// the clock held down by power.  What adds requests to L2 beside the copies
// costs time at once: prefetches a unit ahead (+27 %), an epilogue whose lanes
// walk a row each (+35 % in the n x n products of lb_orth.cu), and operand rows
// that do not begin on 128 bytes (+30 % with rows of 2320 bytes).
//
// The tensor core adds to its accumulator with truncation (measured: 16 terms
// at a time, about 1.5 * 2^-24 of the accumulator lost on average, toward
// zero), so a long sum of one sign comes out low by 9e-8 of its value per 16
// terms, halved.  An epilogue can ask for `chunk` k blocks at a time and add
// the chunks in registers, rounding to nearest.
//
// A problem is a batch of equal products, its operands arrays [z][row][column].
// With parts = 3 each operand is a pair of halves (the planes z and z + 1: high
// and low), and hi * hi + lo * hi + hi * lo is taken from one copy of the four
// halves of a k block; with parts = 2 one operand is whole and only the other
// has a low half.
// A problem marked symmetric has only its tiles on and above the diagonal.
//
// Every wait is bounded: on timeout an error code is left in g_mm_err and
// the kernel drains its copies and returns.
#pragma once

#include <algorithm>
#include <utility>
#include <vector>

#include "lb_internal.cuh"
#include "lb_tc.cuh"

namespace lb {

constexpr int kMmTile = 256;      // i and j of a unit
constexpr int kMmHalf = 128;      // i and j one CTA of the pair stages
constexpr int kMmBK = 64;         // k of a stage
constexpr int kMmStages = 6;      // even: a k block of halves takes two
constexpr int kMmThreads = 384;
constexpr int kMmEpiWarps = 8;
// Registers a thread: 168 at launch (what 12 warps can have), then 56 and 2 x 224 by group of four warps, the same sum.
constexpr int kMmRegsLaunch = 168, kMmRegsFew = 56, kMmRegsMany = 224;
static_assert(kMmRegsFew + 2 * kMmRegsMany <= 3 * kMmRegsLaunch, "setmaxnreg.inc would wait for good");
constexpr uint32_t kMmOperand = kMmHalf * kMmBK * 2;   // 16 KB: one operand's half of one stage
constexpr int kMmChunkAll = 1 << 28;
constexpr uint32_t kMmSlice = kMmBK * 128;             // MN-major: 64 k rows of 64 elements

// Error code of a bounded wait that gave up, one per source file that has such kernels (mm_status).
static __device__ int g_mm_err;

// One problem of a launch: `batch` products of M x N over nkb 64-deep k blocks.
// a_mn / b_mn: the operand is MN-major.  za, zb: its z planes from one product of the batch to the next.
struct MmProb {
    int a_mn, b_mn;
    int parts, za, zb;
    int b_whole;          // with parts = 2: the low half taken is A's (else B's)
    int M, N;             // rows i, columns j
    int nkb;
    int width;            // columns of a tile: 256, 128 or 64
    int chunk;            // k blocks one accumulator takes
    int ntm, ntn, tiles;  // tiles across, along, and in all (fewer than across times along when symmetric)
    int m_fast;           // units run over i first (else over j first)
    int sym;
    int batch, splits, kb_per;   // k blocks are cut into `splits` ranges of kb_per
    int unit0;            // first unit of this problem
};

// Units by round and pair (kMmNone: the pair has no more), for a launch of few units of different lengths; see mm_deal.
constexpr int kMmMostDealt = 1024, kMmMostRounds = 16;
constexpr uint16_t kMmNone = 0xffff;
struct MmOrder {
    int n;                // entries, a multiple of the pairs; 0: units are dealt in order
    uint16_t unit[kMmMostDealt];
};

template <int kMaxProbs>
struct MmSmem {
    alignas(1024) unsigned char A[kMmStages][kMmOperand];
    alignas(1024) unsigned char B[kMmStages][kMmOperand];
    alignas(1024) unsigned char ST[kMmEpiWarps][32 * 128];   // one 32-row staging block per epilogue warp
    uint64_t full[kMmStages], empty[kMmStages];
    uint64_t accf[2], acce[2];
    MmProb p[kMaxProbs];   // the launch's records: parameters are read from far away, one latency after another
    uint16_t dealt[kMmMostRounds];   // this pair's units, where they are dealt by MmBatch::order
    int ordered;
    uint32_t tmem_base;
    int abort;
};
template <int kMaxProbs>
constexpr size_t kMmSmemBytes = sizeof(MmSmem<kMaxProbs>) + 1024;

static_assert(kMmSmemBytes<16> <= 232448, "the shared memory of one SM");

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;\n" ::: "memory");
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
    return r;
}

// shared::cluster address of this shared-memory object in CTA `rank` of the pair
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(cluster_addr) : "memory");
}

// Copy into this CTA's shared memory, counted on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_3d_pair(void *dst, const CUtensorMap *map, int x, int y, int z,
                                                 uint32_t bar_cluster)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], "
        "[%1, {%2, %3, %4}], [%5];\n" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar_cluster)
        : "memory");
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, int x, int y, uint32_t src)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];\n" ::"l"(map), "r"(x),
                 "r"(y), "r"(src)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, int x, int y, int z, uint32_t src)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];\n" ::"l"(map), "r"(x),
                 "r"(y), "r"(z), "r"(src)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
}

// fp32 add of the block into global memory
__device__ __forceinline__ void tma_add_2d(const CUtensorMap *map, int x, int y, uint32_t src)
{
    asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.bulk_group [%0, {%1, %2}], [%3];\n" ::"l"(map),
                 "r"(x), "r"(y), "r"(src)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
}

__device__ __forceinline__ void tma_store_wait_read()
{
    asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory");
}
__device__ __forceinline__ void tma_store_wait_all() { asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory"); }

__device__ __forceinline__ void tc_commit_pair(uint64_t *bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

__device__ __forceinline__ void tc_mma_f16_pair(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                uint32_t accumulate)
{
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// fp32 accumulator, A and B both bf16 or both fp16, M = 256, N = n (a multiple of 32)
__device__ __forceinline__ uint32_t mm_idesc(bool bf16, bool a_mn, bool b_mn, int n)
{
    return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kMmTile >> 4) << 24);
}

// One lane of the (converged) warp: code under it stays uniform to the compiler, so that the descriptors and barrier
// addresses of the loops below live in uniform registers.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}

// Bounded wait of a whole warp: every lane gets lane 0's answer, so the warp stays together.
__device__ __forceinline__ bool mbar_wait_warp(uint64_t *b, uint32_t parity, volatile int *abort, int *err, int code)
{
    if (__all_sync(0xffffffffu, mbar_try_wait(b, parity))) return true;
    return __all_sync(0xffffffffu, mbar_wait(b, parity, abort, err, code));
}

struct MmUnit {
    int q;             // problem
    int b;             // product of its batch
    int tm, tn, split;
    int half;          // columns one CTA stages: half the tile's, fewer in the last column of tiles
    int kb0, kb1;      // k blocks [kb0, kb1)
};

template <int kMaxProbs>
struct MmBatch {
    CUtensorMap mA[kMaxProbs], mB[kMaxProbs];
    MmProb p[kMaxProbs];
    int n, nunits;
    int extra;            // see mm_nth
    MmOrder order;
};

// The k-th unit of a pair, -1 after its last.  Units are dealt in order, except that where a first problem of long units
// leaves some pairs one short, those pairs first take `extra` units each of what follows, which fills the gap.
template <int kMaxProbs>
__device__ __forceinline__ int mm_nth(const MmBatch<kMaxProbs> &G, const MmSmem<kMaxProbs> &S, int pair, int npairs, int k)
{
    if (S.ordered) {
        const int u = k < kMmMostRounds ? S.dealt[k] : kMmNone;
        return u == kMmNone ? -1 : u;
    }
    const MmProb *const p = S.p;
    if (G.extra == 0) {
        const int u = pair + k * npairs;
        return u < G.nunits ? u : -1;
    }
    const int n0 = p[1].unit0, more = n0 % npairs;   // pairs below `more` have one long unit more
    const int c0 = n0 / npairs + (pair < more ? 1 : 0);
    if (k < c0) return pair + k * npairs;
    k -= c0;
    const int early = npairs - more;
    if (pair >= more) {
        if (k < G.extra) return n0 + (pair - more) + k * early;
        k -= G.extra;
    }
    const int u = n0 + G.extra * early + pair + k * npairs;
    return u < G.nunits ? u : -1;
}

__host__ __device__ __forceinline__ MmUnit mm_unit(const MmProb *p, int nprobs, int u)
{
    MmUnit r;
    r.q = 0;
    for (int i = 1; i < nprobs; ++i)
        if (u >= p[i].unit0) r.q = i;
    const MmProb &P = p[r.q];
    // ranges of k outermost: the units in flight share operands
    int local = u - P.unit0;
    const int per_range = P.tiles * P.batch;
    r.split = P.splits > 1 ? local / per_range : 0;
    local -= r.split * per_range;
    r.b = P.batch > 1 ? local / P.tiles : 0;
    local -= r.b * P.tiles;
    if (P.sym) {
        r.tm = 0;
        // tile row tm has the column tiles from its diagonal block on
        const int per_row = kMmTile / P.width;
        for (int left = P.ntn; local >= left; left -= per_row, ++r.tm) local -= left;
        r.tn = r.tm * per_row + local;
    } else if (P.m_fast) {
        r.tn = local / P.ntm;
        r.tm = local - r.tn * P.ntm;
    } else {
        r.tm = local / P.ntn;
        r.tn = local - r.tm * P.ntn;
    }
    const int columns = (P.N - r.tn * P.width + 31) & ~31;
    r.half = (columns < P.width ? columns : P.width) >> 1;
    r.kb0 = r.split * P.kb_per;
    r.kb1 = r.kb0 + P.kb_per < P.nkb ? r.kb0 + P.kb_per : P.nkb;
    return r;
}

// What an epilogue warp gets for one unit: 32 rows (row = row0 + lane) and `cols` columns from col0 on, which start at
// tensor-memory address `tmem` (lane quarter in the upper half, column in the lower).  cols may be 0.
struct MmTileCtx {
    uint32_t tmem;
    int row0, col0, cols, lane;
    uint32_t st;          // this warp's 4 KB staging block (shared address)
};

// An epilogue `Epi` is called by each of its warps, for each unit: begin() (before the accumulator is there), take() for
// each chunk (`first`, `last`) while the accumulator is held, end() after it has been released.  `State` lives from
// begin() to end(); kManyRegs asks for the register split; `stored` says whether the staging block has copies that may
// still be reading it.
template <bool kBf16, int kMaxProbs, class Epi>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kMmThreads, 1)
    mm_kernel(const __grid_constant__ MmBatch<kMaxProbs> G, const __grid_constant__ typename Epi::Params E)
{
    int *const err = &g_mm_err;
    extern __shared__ __align__(1024) unsigned char mm_raw[];
    const uint32_t raw_addr = smem_u32(mm_raw);
    MmSmem<kMaxProbs> &S = *reinterpret_cast<MmSmem<kMaxProbs> *>(mm_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr));
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    volatile int *abort = &S.abort;
    const int nprobs = G.n;

    for (int i = threadIdx.x; i < nprobs * (int)(sizeof(MmProb) / 4); i += kMmThreads)
        reinterpret_cast<int *>(S.p)[i] = reinterpret_cast<const int *>(G.p)[i];
    if (threadIdx.x < kMmMostRounds) {
        const int i = pair + threadIdx.x * npairs;
        S.dealt[threadIdx.x] = i < G.order.n ? G.order.unit[i] : kMmNone;
        S.ordered = G.order.n;
    }
    if (warp == 3 && lane < nprobs) {
        asm volatile("prefetch.tensormap [%0];\n" ::"l"(&G.mA[lane]) : "memory");
        asm volatile("prefetch.tensormap [%0];\n" ::"l"(&G.mB[lane]) : "memory");
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < kMmStages; ++s) {
            mbar_init(&S.full[s], 1);
            mbar_init(&S.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&S.accf[b], 1);
            mbar_init(&S.acce[b], 2 * kMmEpiWarps);   // both CTAs' warps (the first CTA's barrier is the one used)
        }
        S.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(smem_u32(&S.tmem_base)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = S.tmem_base;
    // Launched to overlap with the kernel before it (see mm_launch), whose memory the copies and the epilogues touch: every
    // warp waits for its end in its first unit, with what can come before done.
    pdl_go();

    if (warp < 4) {
        if constexpr (Epi::kManyRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kMmRegsFew));
        // What the loops below use of a problem is in registers before they start: a k block takes about 500 cycles, and a
        // shared-memory read is 30 of them.
        if (warp == 0 || warp == 2) {
            // ---------------- producers: warp 0 copies A, warp 2 B
            const bool is_a = warp == 0;
            unsigned char *const base = is_a ? S.A[0] : S.B[0];
            const uint32_t full0 = map_rank(smem_u32(&S.full[0]), 0);
            uint32_t s = 0, ph = 0;
            bool ok = true;
            for (int n = 0, u; ok && (u = mm_nth(G, S, pair, npairs, n)) >= 0; ++n) {
                const MmUnit U = mm_unit(S.p, nprobs, u);
                const MmProb &P = S.p[U.q];
                const CUtensorMap *const map = is_a ? &G.mA[U.q] : &G.mB[U.q];
                const bool mn = is_a ? P.a_mn != 0 : P.b_mn != 0;
                const bool two = mn && (is_a || U.half > 64);   // both 64-wide slices
                const int x0 = is_a ? U.tm * kMmTile + (int)rank * kMmHalf : U.tn * P.width + (int)rank * U.half;
                // both CTAs' halves; a K-major box of B has width / 2 rows
                const uint32_t bytes_b = P.b_mn ? (U.half > 64 ? 2 : 1) * kMmSlice : P.width * kMmBK;
                const bool low_a = P.parts == 3 || (P.parts == 2 && P.b_whole), low_b = P.parts == 3 || (P.parts == 2 && !P.b_whole);
                const uint32_t bytes[2] = {2 * (kMmOperand + bytes_b), 2 * ((low_a ? kMmOperand : 0) + (low_b ? bytes_b : 0))};
                const int planes = P.parts > 1 ? 2 : 1, z0 = U.b * (is_a ? P.za : P.zb);
                const bool low = is_a ? low_a : low_b;
                if (n == 0) pdl_wait();
                for (int kb = U.kb0; ok && kb < U.kb1; ++kb)
                    for (int plane = 0; plane < planes; ++plane) {
                        if (!(ok = mbar_wait_warp(&S.empty[s], ph ^ 1, abort, err, 1))) break;
                        const bool one = elect_one();
                        if (one && is_a && rank == 0) mbar_expect_tx(&S.full[s], plane ? bytes[1] : bytes[0]);
                        unsigned char *const dst = base + s * kMmOperand;
                        const uint32_t bar = full0 + s * 8;
                        const int k = kb * kMmBK;
                        if (one && (plane == 0 || low)) {
                            tma_load_3d_pair(dst, map, mn ? x0 : k, mn ? k : x0, z0 + plane, bar);
                            if (two) tma_load_3d_pair(dst + kMmSlice, map, x0 + 64, k, z0 + plane, bar);
                        }
                        __syncwarp();
                        if (++s == kMmStages) {
                            s = 0;
                            ph ^= 1;
                        }
                    }
            }
            if (*abort) {
                // let the copies already issued land before the pair leaves: a wait gives up after two seconds, a copy
                // takes microseconds, so a fixed time is enough
                const long long t0 = clock64();
                while (clock64() - t0 < kWaitCycles / 1000) {
                }
            }
        } else if (warp == 1) {
            // ---------------- MMA issuer (first CTA of the pair)
            if (rank == 0) {
                uint32_t s = 0, ph = 0, acc = 0;   // stage, its phase, accumulators used
                bool ok = true;
                for (int n = 0, u; ok && (u = mm_nth(G, S, pair, npairs, n)) >= 0; ++n) {
                    const MmUnit U = mm_unit(S.p, nprobs, u);
                    const MmProb &P = S.p[U.q];
                    const bool a_mn = P.a_mn != 0, b_mn = P.b_mn != 0;
                    const uint32_t idesc = mm_idesc(kBf16, a_mn, b_mn, 2 * U.half);
                    // 16 k: 32 bytes along a K-major row, or two 8-row groups (2048 bytes) of an MN-major slice
                    const uint64_t step_a = a_mn ? 2048 >> 4 : 32 >> 4, step_b = b_mn ? 2048 >> 4 : 32 >> 4;
                    const uint64_t da0 = a_mn ? smem_desc_mn_sw128(S.A[0], kMmSlice) : smem_desc_sw128(S.A[0]);
                    const uint64_t db0 = b_mn ? smem_desc_mn_sw128(S.B[0], kMmSlice) : smem_desc_sw128(S.B[0]);
                    const int chunk = P.chunk, parts = P.parts;
                    if (n == 0) pdl_wait();   // the bounded waits count from the copies' start
                    const bool low_a = parts == 3 || (parts == 2 && P.b_whole), low_b = parts == 3 || (parts == 2 && !P.b_whole);
                    for (int left = U.kb1 - U.kb0; ok && left > 0; left -= chunk, ++acc) {
                        const int ab = acc & 1;
                        if (!(ok = mbar_wait_warp(&S.acce[ab], ((acc >> 1) & 1) ^ 1, abort, err, 2))) break;
                        tc_fence_after();
                        const uint32_t dacc = tmem + (uint32_t)(ab * kMmTile);
                        uint32_t add = 0;
                        // A k block is one stage of the ring, or two, the high halves and the low ones.
                        auto products = [&](uint32_t sa, uint32_t sb) {
                            const uint64_t da = da0 + sa * (kMmOperand >> 4), db = db0 + sb * (kMmOperand >> 4);
                            tc_mma_f16_pair(dacc, da, db, idesc, add);
#pragma unroll
                            for (int kk = 1; kk < kMmBK / 16; ++kk)
                                tc_mma_f16_pair(dacc, da + kk * step_a, db + kk * step_b, idesc, 1u);
                            add = 1;
                        };
                        for (int i = min(left, chunk); i > 0; --i) {
                            if (!(ok = mbar_wait_warp(&S.full[s], ph, abort, err, 3))) break;
                            tc_fence_after();
                            if (parts == 1) {
                                if (elect_one()) {
                                    products(s, s);
                                    tc_commit_pair(&S.empty[s]);
                                }
                                add = 1;
                            } else {
                                const uint32_t lo = s + 1;   // kMmStages is even
                                if (elect_one()) products(s, s);
                                add = 1;
                                __syncwarp();
                                if (!(ok = mbar_wait_warp(&S.full[lo], ph, abort, err, 3))) break;
                                tc_fence_after();
                                if (elect_one()) {
                                    if (low_a) products(lo, s);
                                    if (low_b) products(s, lo);
                                    tc_commit_pair(&S.empty[s]);
                                    tc_commit_pair(&S.empty[lo]);
                                }
                                ++s;
                            }
                            __syncwarp();
                            if (++s == kMmStages) {
                                s = 0;
                                ph ^= 1;
                            }
                        }
                        if (ok && elect_one()) tc_commit_pair(&S.accf[ab]);
                        __syncwarp();
                    }
                }
            }
        }
    } else {
        if constexpr (Epi::kManyRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kMmRegsMany));
        // ---------------- epilogue (warps 4-11: tensor-memory lanes 32 (warp % 4) .., one half of the columns)
        const int q4 = warp & 3, side = (warp - 4) >> 2;
        uint32_t acc = 0;
        bool stored = false, ok = true;
        MmTileCtx T;
        T.lane = lane;
        T.st = smem_u32(S.ST[warp - 4]);
        for (int n = 0, u; ok && (u = mm_nth(G, S, pair, npairs, n)) >= 0 && !*abort; ++n) {
            const MmUnit U = mm_unit(S.p, nprobs, u);
            const MmProb &P = S.p[U.q];
            T.row0 = U.tm * kMmTile + (int)rank * kMmHalf + q4 * 32;
            T.col0 = U.tn * P.width + side * (P.width / 2);
            T.cols = T.row0 < P.M ? max(0, min(P.width / 2, P.N - T.col0)) : 0;
            typename Epi::State state;
            if (n == 0) pdl_wait();
            Epi::begin(E, P, U, T, state);
            for (int k0 = U.kb0; k0 < U.kb1; k0 += P.chunk, ++acc) {
                const int ab = acc & 1;
                if (!(ok = mbar_wait(&S.accf[ab], (acc >> 1) & 1, abort, err, 4))) break;
                tc_fence_after();
                T.tmem = tmem + ((uint32_t)(q4 * 32) << 16) + (uint32_t)(ab * kMmTile + side * (P.width / 2));
                Epi::take(E, P, U, T, state, k0 == U.kb0, k0 + P.chunk >= U.kb1, stored);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(map_rank(smem_u32(&S.acce[ab]), 0));
            }
            if (ok) Epi::end(E, P, U, T, state, stored);
        }
        if (lane == 0) tma_store_wait_all();
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();   // no CTA of the pair leaves while the other may still signal it or use its operands
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;\n" ::"r"(tmem));
    }
}

// Host: an operand stored as `planes` planes of `rows` rows of `cols` elements, `pitch` elements between rows and
// `plane` between planes.  K-major: a row is an i (or j) and the box is 64 k x `box` rows (128 for A, half a tile's
// columns for B); MN-major: a row is a k and the box is 64 i x 64 k rows.  Everything outside reads as zero.
inline bool mm_operand(CUtensorMap *map, bool bf16, bool mn_major, const void *base, long rows, long cols, long pitch,
                       long planes = 1, int box = kMmHalf, long plane = 0)
{
    return tmap_encode_3d(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, base, cols,
                          rows, planes, pitch * 2, (plane ? plane : pitch * rows) * 2, 64, mn_major ? kMmBK : box);
}

inline int mm_tiles(int ntm, int ntn, bool sym, int width)
{
    if (!sym) return ntm * ntn;
    int t = 0;
    for (int i = 0; i < ntm; ++i) t += std::max(0, ntn - i * (kMmTile / width));
    return t;
}

// Host: tiles and k ranges of a problem whose k blocks are cut into (at most) `splits` ranges.
inline void mm_plan(MmProb &P, int M, int N, long K, bool m_fast, int unit0, int splits, int parts = 1, int batch = 1,
                    bool sym = false, int width = kMmTile)
{
    P.M = M;
    P.N = N;
    P.parts = parts;
    P.batch = batch;
    P.sym = sym ? 1 : 0;
    P.nkb = (int)((K + kMmBK - 1) / kMmBK);
    P.ntm = (M + kMmTile - 1) / kMmTile;
    P.width = width;
    P.ntn = (N + width - 1) / width;
    P.tiles = mm_tiles(P.ntm, P.ntn, sym, width);
    P.chunk = kMmChunkAll;
    P.m_fast = m_fast ? 1 : 0;
    P.unit0 = unit0;
    P.kb_per = (P.nkb + splits - 1) / splits;
    P.splits = (P.nkb + P.kb_per - 1) / P.kb_per;
}
// Host: accumulators of equal lengths, at most `most` k blocks, which the epilogue adds.
inline void mm_chunk(MmProb &P, int most)
{
    const int chunks = (P.kb_per + most - 1) / most;
    P.chunk = (P.kb_per + chunks - 1) / chunks;
}
// Host: CTA pairs that run at once on the current device.
inline cudaError_t mm_pairs(int *pairs)
{
    int sms = 0;
    const cudaError_t e = sm_count_of_current(&sms);
    *pairs = sms / 2 > 0 ? sms / 2 : 1;
    return e;
}
// Host: deal the units of a launch to its pairs, the longest first, each to the pair with least to do: for launches of few
// units of different lengths (where they are equal this is their order).  A k block of a unit takes the tensor cores 512
// cycles for each product of whole tiles, or its copies at about 42 bytes a cycle, which a tile of few columns waits for.
// Of 28 matrices of ranks 800 and 544 (216 units of 9 or 13 k blocks) the first pair ended after 16 us and the last after
// 52 in order, and after 35 and 42 so.
inline void mm_deal(MmOrder &O, const MmProb *p, int nprobs, int nunits, int pairs)
{
    O.n = 0;
    if (nunits <= pairs || nunits > kMmMostDealt) return;
    std::vector<std::pair<long, int>> units(nunits);   // (-cost, unit)
    for (int u = 0; u < nunits; ++u) {
        const MmUnit U = mm_unit(p, nprobs, u);
        const MmProb &P = p[U.q];
        const long planes = P.parts > 1 ? 2 : 1;
        const long products = 512L * P.parts * U.half / kMmHalf, copies = planes * (kMmHalf + U.half) * kMmBK * 2 / 42;
        units[u] = {-(U.kb1 - U.kb0) * std::max(products, copies) - 1000, u};
    }
    std::sort(units.begin(), units.end());
    std::vector<std::pair<long, int>> load(pairs);     // a heap: (-what a pair has to do, pair)
    std::vector<int> taken(pairs, 0);
    for (int i = 0; i < pairs; ++i) load[i] = {0, -i};
    for (uint16_t &u : O.unit) u = kMmNone;
    int rounds = 0;
    for (const auto &[cost, u] : units) {
        std::pop_heap(load.begin(), load.end());
        auto &[left, pair] = load.back();
        const int at = taken[-pair]++ * pairs - pair;
        if (at >= kMmMostDealt || taken[-pair] > kMmMostRounds) return;
        O.unit[at] = (uint16_t)u;
        rounds = std::max(rounds, taken[-pair]);
        left += cost;
        std::push_heap(load.begin(), load.end());
    }
    O.n = std::min(rounds * pairs, kMmMostDealt);
}
inline int mm_units(const MmProb &P) { return P.tiles * P.batch * P.splits; }

template <bool kBf16, int kMaxProbs, class Epi>
inline cudaError_t mm_launch(const MmBatch<kMaxProbs> &G, const typename Epi::Params &E, cudaStream_t s)
{
    if (G.nunits == 0) return cudaSuccess;
    const void *fn = (const void *)mm_kernel<kBf16, kMaxProbs, Epi>;
    cudaError_t e = ensure_dyn_smem(fn, kMmSmemBytes<kMaxProbs>);
    if (e != cudaSuccess) return e;
    if (Epi::kManyRegs) {
        // the register split counts on this: with fewer at launch, setmaxnreg would wait for registers that do not exist
        static const int regs = [fn]() {
            cudaFuncAttributes a;
            return cudaFuncGetAttributes(&a, fn) == cudaSuccess ? a.numRegs : 0;
        }();
        if (regs < kMmRegsLaunch) return cudaErrorInvalidConfiguration;
    }
    int pairs = 0;
    if ((e = mm_pairs(&pairs)) != cudaSuccess) return e;
    if (pairs > G.nunits) pairs = G.nunits;
    // programmatic serialisation: the set-up (barriers, tensor memory, records) may overlap the end of the kernel before
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * pairs);
    cfg.blockDim = dim3(kMmThreads);
    cfg.dynamicSmemBytes = kMmSmemBytes<kMaxProbs>;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, mm_kernel<kBf16, kMaxProbs, Epi>, G, E);
}

// Host: waits for `s`, returns and clears this file's error code.
static inline lb_status mm_status(cudaStream_t s)
{
    int code = 0;
    const int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&code, g_mm_err, sizeof(int), 0, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return status_from(e);
    if (!code) return LB_OK;
    e = cudaMemcpyToSymbolAsync(g_mm_err, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    return e == cudaSuccess ? LB_ERR_TIMEOUT : status_from(e);
}

}  // namespace lb
