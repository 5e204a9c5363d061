// Orthogonalised updates of latent factors: the Newton-Schulz iteration of the
// Muon optimiser (Jordan et al., "Muon: An optimizer for hidden layers in
// neural networks", 2024) for many matrices at once.
//
//     X = G / (|G|_F + eps),   `steps` times:  X <- a X + X (b A + c A^2),  A = X^T X
//     (a, b, c) = (3.4445, -4.7750, 2.0315);   on X^T where G is wide
//
// For a tall m x n matrix (m >= n; n is the latent rank, m the features) this
// is X_0 times a polynomial of A_0 = X_0^T X_0, so the long axis is needed
// twice only, and everything between is n x n:
//
//     p_k = b A_k + c A_k^2,  q_k = a I + p_k,   A_{k+1} = A_k q_k^2,   Q_{k+1} = Q_k q_k,   X_steps = X_0 Q_steps
//
// 2 m n^2 (half of it by symmetry) + 2 m n^2 + steps * 4 * 2 n^3 flops instead
// of steps * (4 m n^2 + 2 n^3).  All these n x n matrices are polynomials of
// A_0: symmetric, and they commute, so only tiles on and above the diagonal
// are computed and either orientation may feed the tensor cores.
//
// Precision.  The small singular values of an update are what the iteration
// blows up (by up to a^steps = 485), and in A_0 they are squared, so an error
// of 2^-11 in A (one binary16 rounding) would move them by percents.  Every
// operand is therefore a pair of binary16 halves, hi + lo, 22 bits, and a
// product is hi hi + lo hi + hi lo in one float32 accumulator for each k block,
// whose halves are copied once for the three.  p is kept rather than q, whose
// diagonal would round by a 2^-23, and the products are made exactly symmetric.
// A_0's sums over the long axis are taken in short pieces (GramEpi).
// Measured against binary64, as parts of the result's norm: 1.7e-3, which is the
// rounding to bfloat16, for Gaussian and gradient-like matrices; at most 2.2e-3
// for spectra that fall off by 1e4 or have one dominant value (plain bfloat16
// iterations: 2e-2 to 2e-1), and the same whatever else is in the call.  That is
// after five steps; singular values below
// some 1e-3 of the norm, lifted to 1 by up to ten steps, come out with relative
// errors of about 2^-22 over their square (1e-2 of the norm for a square Gaussian
// matrix of rank 65 that has one).  Scales are powers of two that keep the halves clear
// of binary16's ends: G is scaled to root mean square 1 (its largest entry is
// then at most sqrt(m n)), A, p and T by 2^13 (their eigenvalues stay below 3),
// Q_k by what a^k leaves.
// bfloat16 G is scaled by a power of two, which makes its high half exact and
// its low half zero: one product for A_0 instead of three, two for X_0 Q.
//
// A matrix of at most 24,576 elements and rank at most 64 is done whole by one
// block, in float32 from shared memory (one launch instead of five: 4 matrices
// of 512 x 16 took 49 us in five, 21 us so).  Ranks up to 64 otherwise run the
// n x n part in one block per matrix, in float32 FMAs (up to rank 48 faster than
// the tensor core, 57 against 78 us a call at 4096 x 33, and 79 against 74 at
// rank 64); ranks up to 128 in one block on its tensor core; larger ranks as
// launches over all matrices (three a step), on CTA pairs.  (One launch for all steps,
// whose units wait for the earlier ones of their own matrix, was no faster: 243
// against 229 us for four odd matrices, 2590 against 2530 us for the 28 of a
// block: a step's latency is in the tiles, not in the launches.)
//
// Copied once, the four halves of 64 k of a tile are 64 KB for three products'
// 1536 cycles of the tensor cores (copied for each product they would be 96):
// 51 us a launch for 28 matrices (12 of rank 800, 16 of rank 544), 96 where
// there are two products of each.

#include <algorithm>
#include <cmath>
#include <cstring>
#include <vector>

#include "lb_mm.cuh"
#include "lb_orth_index.h"
#include "littlebit_train.h"

namespace lb {
namespace {

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
constexpr int kMostMats = 64, kMostGroups = 8;   // of one set of launches
constexpr int kNormBlocks = 592;                 // blocks (and partial sums) a matrix has at most
constexpr int kSmallN = 64;
constexpr float kSA = 8192.0f;                   // scale of A, p and T
constexpr int kMaxSteps = 10;
// k blocks of A_0 one accumulator takes, divided by the products of halves: 60 or 64 additions (see GramEpi).
constexpr int kGramChunk = 16;

// One matrix as the elementwise kernels see it.
struct Mat {
    const void *G;
    __half *X;            // [1 or 2 planes][rows][pitch]
    int rows, cols, pitch;
    int nblocks;          // blocks of the norm
};
struct Mats {
    Mat m[kMostMats];
    int n, bf16;
    float eps;
    double *sums;         // [n][kNormBlocks]
    float2 *scal;         // [n]: (kappa, kappa^2 * kSA), X_0 = kappa * (scaled G)
};

__device__ __forceinline__ float load_g(const void *G, size_t i, int bf16)
{
    return bf16 ? bf16_bits_to_float(reinterpret_cast<const uint16_t *>(G)[i]) : reinterpret_cast<const float *>(G)[i];
}

// Partial sums of squares in binary64 (squares of float32 neither overflow nor vanish there).
__global__ void __launch_bounds__(256) norm_kernel(const __grid_constant__ Mats P)
{
    pdl_go();
    pdl_wait();
    const int which = blockIdx.y;
    const Mat &m = P.m[which];
    if ((int)blockIdx.x >= m.nblocks) return;
    const size_t n = (size_t)m.rows * m.cols;
    const size_t step = (size_t)m.nblocks * 256;
    double s = 0.0;
    if (!P.bf16 && ((uintptr_t)m.G & 15) == 0) {
        const size_t nv = n / 4;
#pragma unroll 4
        for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < nv; i += step) {
            const float4 v = __ldg(reinterpret_cast<const float4 *>(m.G) + i);
            s += ((double)v.x * v.x + (double)v.y * v.y) + ((double)v.z * v.z + (double)v.w * v.w);
        }
        if (blockIdx.x == 0 && threadIdx.x < n % 4) {
            const double v = reinterpret_cast<const float *>(m.G)[nv * 4 + threadIdx.x];
            s += v * v;
        }
    } else {
#pragma unroll 4
        for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += step) {
            const double v = load_g(m.G, i, P.bf16);
            s += v * v;
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    __shared__ double w[8];
    if ((threadIdx.x & 31) == 0) w[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < 8; ++i) s += w[i];
        P.sums[which * kNormBlocks + blockIdx.x] = s;
    }
}

__device__ __forceinline__ void halves(float x, __half &hi, __half &lo)
{
    hi = __float2half_rn(x);
    lo = __float2half_rn(x - __half2float(hi));
}

// Two at once, the first in the lower half of a word: half the conversions.
__device__ __forceinline__ void halves2(float2 x, uint32_t &hi, uint32_t &lo)
{
    const __half2 h = __float22half2_rn(x);
    const float2 back = __half22float2(h);
    const __half2 l = __floats2half2_rn(x.x - back.x, x.y - back.y);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = *reinterpret_cast<const uint32_t *>(&l);
}
__device__ __forceinline__ float2 sum_of(uint32_t hi, uint32_t lo)
{
    const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    const float2 l = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
    return make_float2(h.x + l.x, h.y + l.y);
}

// X = G scaled to root mean square about 1, as binary16 halves.
__global__ void __launch_bounds__(256) split_kernel(const __grid_constant__ Mats P)
{
    pdl_go();
    pdl_wait();
    const int which = blockIdx.y;
    const Mat &m = P.m[which];
    if ((int)blockIdx.x >= m.nblocks) return;
    __shared__ float sc;
    if (threadIdx.x < 32) {
        double s = 0.0;
#pragma unroll 4
        for (int i = threadIdx.x; i < m.nblocks; i += 32) s += P.sums[which * kNormBlocks + i];
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (threadIdx.x == 0) {
            const double norm = sqrt(s);
            double c = fmin(sqrt((double)m.rows * m.cols), 32768.0) / norm;
            if (P.bf16) c = exp2(floor(log2(c)));
            if (c > 0x1p126) c = 0x1p126;                    // also a zero matrix
            sc = (float)c;
            if (blockIdx.x == 0) {
                const double kappa = 1.0 / (c * (norm + (double)P.eps));
                P.scal[which] = norm == 0.0 ? make_float2(0.0f, 0.0f)
                                                 : make_float2((float)kappa, (float)(kappa * kappa * kSA));
            }
        }
    }
    __syncthreads();
    const float c = sc;
    const size_t plane = (size_t)m.rows * m.pitch, total = plane / 8;
    const bool wide_loads = !P.bf16 && m.cols % 4 == 0 && ((uintptr_t)m.G & 15) == 0;
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (size_t)m.nblocks * 256) {
        const SplitVector e = split_vector(i, m.cols, m.pitch);
        float x[8];
        if (wide_loads) {   // e.n is 0, 4 or 8
            const float4 *src = reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(m.G) + e.at);
            const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            const float4 u = e.n >= 4 ? src[0] : zero, v = e.n == 8 ? src[1] : zero;
            x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
            x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = j < e.n ? load_g(m.G, e.at + j, P.bf16) : 0.0f;
        }
        alignas(16) __half hi[8], lo[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) halves(x[j] * c, hi[j], lo[j]);
        *reinterpret_cast<uint4 *>(m.X + i * 8) = *reinterpret_cast<uint4 *>(hi);
        if (!P.bf16) *reinterpret_cast<uint4 *>(m.X + plane + i * 8) = *reinterpret_cast<uint4 *>(lo);
    }
}

// two accumulators times f, as bfloat16
__device__ __forceinline__ uint32_t pack_bf(uint32_t a, uint32_t b, float f)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(__uint_as_float(b) * f), "f"(__uint_as_float(a) * f));
    return r;
}

// ---- products
// A_0: the partial sums of each k range.  The accumulator truncates, and what 2064 additions over 11008 rows lose of A_0
// (up to 9e-5, unevenly) moved small singular values until results were off by 4.5e-3 (1/j^2 spectrum, 800 columns) where
// their rounding is 1.7e-3; so it takes 320 or 1024 rows at a time, and these pieces are added in registers: 1.73e-3, at no
// measurable time (6 of 11008 x 800: 763 -> 766 us a call, the 28 of a block 1695 -> 1695).
struct GramEpi {
    static constexpr bool kManyRegs = true;
    struct Params {
        CUtensorMap mD[kMostGroups];   // float32 [ranges * batch][n][pn]
    };
    struct State {
        float a[kMmHalf];
    };
    static __device__ __forceinline__ void begin(const Params &, const MmProb &, const MmUnit &, const MmTileCtx &, State &S)
    {
#pragma unroll
        for (int i = 0; i < kMmHalf; ++i) S.a[i] = 0.0f;   // taking the first piece as it is spilled registers
    }
    static __device__ __forceinline__ void take(const Params &, const MmProb &, const MmUnit &, const MmTileCtx &T, State &S,
                                                bool, bool, bool &)
    {
        if (T.cols == 0) return;
#pragma unroll
        for (int c = 0; c < kMmHalf; c += 32) {   // columns past the last one hold anything and go nowhere
            uint32_t v[32];
            tmem_ld32(T.tmem + c, v);
#pragma unroll
            for (int i = 0; i < 32; ++i) S.a[c + i] += __uint_as_float(v[i]);
        }
    }
    static __device__ __forceinline__ void end(const Params &E, const MmProb &P, const MmUnit &U, const MmTileCtx &T,
                                               State &S, bool &stored)
    {
#pragma unroll
        for (int c = 0; c < kMmHalf; c += 32) {
            if (c >= T.cols) continue;
            if (stored) {
                if (T.lane == 0) tma_store_wait_read();
                __syncwarp();
            }
            stored = true;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float *a = S.a + c + 4 * i;
                sts128(T.st + sw128(T.lane, i), make_uint4(__float_as_uint(a[0]), __float_as_uint(a[1]),
                                                           __float_as_uint(a[2]), __float_as_uint(a[3])));
            }
            fence_proxy_async();
            __syncwarp();
            if (T.lane == 0) tma_store_3d(&E.mD[U.q], T.col0 + c, T.row0, U.split * P.batch + U.b, T.st);
        }
    }
};

enum { kSym = 0, kOut = 1 };
constexpr int kMostProbs = 2 * kMostGroups;
struct OrthProb {
    int kind;
    int pn;               // row pitch of the n x n arrays
    int first;            // index of the batch's first matrix
    float alpha, beta;    // kSym: alpha * product + beta * C;  kOut: alpha * kappa * product
    const __half *C;      // [batch][2][n][pn]
    __half *D;
    __half *D2;           // null, or the same plus gamma * I
    float gamma;
    int ldo;              // kOut: columns of the output
};
struct OrthEpi {
    static constexpr bool kManyRegs = true;
    struct Params {
        OrthProb p[kMostProbs];
        uint16_t *out[kMostMats];
        const float2 *scal;
    };
    // A warp's 32 x 32 block of a symmetric matrix (two planes of binary16) moves between memory and registers through
    // its staging block, so that four lanes touch the 64 bytes of a row together: a lane that walks its own row alone
    // makes four times as many requests to L2, which slowed the operands' copies to half.
    struct State {
        uint4 c[2][4];   // kSym: the first block of C; part i of a lane is chunk lane % 4 of row 8 i + lane / 4
    };
    // 16-byte chunk `chunk` of row `row` of plane p in the staging block: 64-byte rows, chunks permuted by the row so
    // that eight rows fall on all banks
    static __device__ __forceinline__ uint32_t stage(uint32_t st, int p, int row, int chunk)
    {
        return st + 2048u * p + 64u * row + 16u * (uint32_t)(chunk ^ ((row >> 1) & 3));
    }
    static __device__ __forceinline__ void load_c(const OrthProb &O, const MmProb &P, const MmUnit &U, const MmTileCtx &T,
                                                  int col0, State &S)
    {
        const size_t plane = (size_t)P.N * O.pn;
        const int row = T.row0 + (T.lane >> 2), col = col0 + 8 * (T.lane & 3);
        const __half *C = O.C + (size_t)U.b * 2 * plane + (size_t)row * O.pn + col;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool in = row + 8 * i < P.M && col < O.pn && col0 >= T.row0;
#pragma unroll
            for (int p = 0; p < 2; ++p)
                S.c[p][i] = in ? *reinterpret_cast<const uint4 *>(C + p * plane + (size_t)(8 * i) * O.pn)
                               : make_uint4(0, 0, 0, 0);
        }
    }
    // the staged block to rows row0 .. and columns col0 .. of both planes of D
    static __device__ __forceinline__ void write_block(uint32_t st, int lane, __half *D, size_t plane, int pn, int row0,
                                                       int col0, int n)
    {
        const int row = row0 + (lane >> 2), col = col0 + 8 * (lane & 3);
        __half *dst = D + (size_t)row * pn + col;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const uint4 v = lds128(stage(st, p, 8 * i + (lane >> 2), lane & 3));
                if (row + 8 * i < n && col < pn) *reinterpret_cast<uint4 *>(dst + p * plane + (size_t)(8 * i) * pn) = v;
            }
    }
    static __device__ __forceinline__ void begin(const Params &E, const MmProb &P, const MmUnit &U, const MmTileCtx &T,
                                                 State &S)
    {
        if (E.p[U.q].kind == kSym && T.cols > 0) load_c(E.p[U.q], P, U, T, T.col0, S);
    }
    static __device__ __forceinline__ void end(const Params &, const MmProb &, const MmUnit &, const MmTileCtx &, State &,
                                               bool &)
    {
    }
    static __device__ __forceinline__ void take(const Params &E, const MmProb &P, const MmUnit &U, const MmTileCtx &T,
                                                State &S, bool, bool, bool &)
    {
        const OrthProb &O = E.p[U.q];
        const int row = T.row0 + T.lane;
        uint32_t v[32];
        if (O.kind == kOut) {
            if (T.cols == 0) return;
            uint16_t *const base = E.out[O.first + U.b];
            const float f = O.alpha * E.scal[O.first + U.b].x;
            const bool vec = O.ldo % 8 == 0 && ((uintptr_t)base & 15) == 0;
            if (vec) {   // 64 columns at a time through the staging block, eight lanes to the 128 bytes of a row
                for (int c = 0; c < T.cols; c += 64) {
                    __syncwarp();
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (h && c + 32 >= T.cols) break;
                        tmem_ld32(T.tmem + c + 32 * h, v);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            sts128(T.st + sw128(T.lane, 4 * h + i),
                                   make_uint4(pack_bf(v[8 * i], v[8 * i + 1], f), pack_bf(v[8 * i + 2], v[8 * i + 3], f),
                                              pack_bf(v[8 * i + 4], v[8 * i + 5], f), pack_bf(v[8 * i + 6], v[8 * i + 7], f)));
                    }
                    __syncwarp();
                    const int r0 = T.lane >> 3, col = c + 8 * (T.lane & 7);
                    uint16_t *dst = base + (size_t)(T.row0 + r0) * O.ldo + T.col0 + col;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint4 y = lds128(T.st + sw128(r0 + 4 * i, T.lane & 7));
                        if (T.row0 + r0 + 4 * i < P.M && col < T.cols)
                            *reinterpret_cast<uint4 *>(dst + (size_t)(4 * i) * O.ldo) = y;
                    }
                }
                return;
            }
            // rows without alignment: through the staging block (32 rows of 32, 66 bytes apart), then one row of 32
            // columns at a time
            for (int c = 0; c < T.cols; c += 32) {
                tmem_ld32(T.tmem + c, v);
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const uint32_t w = pack_bf(v[2 * i], v[2 * i + 1], f);
                    asm volatile("st.shared.u16 [%0], %1;\n" ::"r"(T.st + (uint32_t)(T.lane * 66 + 4 * i)),
                                 "h"((uint16_t)w)
                                 : "memory");
                    asm volatile("st.shared.u16 [%0], %1;\n" ::"r"(T.st + (uint32_t)(T.lane * 66 + 4 * i + 2)),
                                 "h"((uint16_t)(w >> 16))
                                 : "memory");
                }
                __syncwarp();
                const int rows = min(32, P.M - T.row0);
                uint16_t *dst = base + (size_t)T.row0 * O.ldo + T.col0 + c + T.lane;
                if (c + T.lane < T.cols)
#pragma unroll 8
                    for (int r = 0; r < rows; ++r) {
                        uint16_t y;
                        asm volatile("ld.shared.u16 %0, [%1];\n" : "=h"(y) : "r"(T.st + (uint32_t)(r * 66 + 2 * T.lane)));
                        dst[(size_t)r * O.ldo] = y;
                    }
            }
            return;
        }
        // A symmetric n x n matrix, in 32 x 32 blocks: one above the diagonal is computed once and written to both its
        // places, one on the diagonal takes its lower half from its upper.  (The products of a polynomial's factors are
        // symmetric only up to rounding, and a difference between the triangles would grow by q(0)^2 = 12 a step.)
        const size_t plane = (size_t)P.N * O.pn;
        for (int c = 0; c < T.cols; c += 32) {
            const int col0 = T.col0 + c;
            if (col0 < T.row0) {
                if (c + 32 < T.cols) load_c(O, P, U, T, col0 + 32, S);
                continue;
            }
            __syncwarp();
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int i = 0; i < 4; ++i) sts128(stage(T.st, p, 8 * i + (T.lane >> 2), T.lane & 3), S.c[p][i]);
            if (c + 32 < T.cols) load_c(O, P, U, T, col0 + 32, S);
            tmem_ld32(T.tmem + c, v);
            __syncwarp();
            float x[32];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 h = lds128(stage(T.st, 0, T.lane, i)), l = lds128(stage(T.st, 1, T.lane, i));
                const uint32_t ch[4] = {h.x, h.y, h.z, h.w}, cl[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 c2 = sum_of(ch[j], cl[j]);
                    x[8 * i + 2 * j] = fmaf(__uint_as_float(v[8 * i + 2 * j]), O.alpha, O.beta * c2.x);
                    x[8 * i + 2 * j + 1] = fmaf(__uint_as_float(v[8 * i + 2 * j + 1]), O.alpha, O.beta * c2.y);
                }
            }
            put(x, O.D + (size_t)U.b * 2 * plane, plane, O.pn, T, col0, P.N);
            if (O.D2) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (col0 + i == row) x[i] += O.gamma;
                put(x, O.D2 + (size_t)U.b * 2 * plane, plane, O.pn, T, col0, P.N);
            }
        }
    }
    static __device__ __forceinline__ void put(const float (&x)[32], __half *D, size_t plane, int pn, const MmTileCtx &T,
                                               int col0, int n)
    {
        uint32_t w[2][16];   // the row's halves, two to a word
#pragma unroll
        for (int i = 0; i < 16; ++i) halves2(make_float2(x[2 * i], x[2 * i + 1]), w[0][i], w[1][i]);
        // the transpose
        __syncwarp();
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int i = 0; i < 32; ++i)
                asm volatile("st.shared.u16 [%0], %1;\n" ::"r"(stage(T.st, p, i, T.lane >> 3) + 2u * (T.lane & 7)),
                             "h"((uint16_t)(i & 1 ? w[p][i >> 1] >> 16 : w[p][i >> 1]))
                             : "memory");
        __syncwarp();
        if (col0 == T.row0) {   // on the diagonal: the lower half from the upper
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                uint4 t[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) t[i] = lds128(stage(T.st, p, T.lane, i));
                const uint32_t *tw = reinterpret_cast<const uint32_t *>(t);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    if (2 * i < T.lane) w[p][i] = (w[p][i] & 0xffff0000u) | (tw[i] & 0xffffu);
                    if (2 * i + 1 < T.lane) w[p][i] = (w[p][i] & 0xffffu) | (tw[i] & 0xffff0000u);
                }
            }
        } else {
            write_block(T.st, T.lane, D, plane, pn, col0, T.row0, n);
        }
        __syncwarp();
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                sts128(stage(T.st, p, T.lane, i), make_uint4(w[p][4 * i], w[p][4 * i + 1], w[p][4 * i + 2], w[p][4 * i + 3]));
        __syncwarp();
        write_block(T.st, T.lane, D, plane, pn, T.row0, col0, n);
    }
};

// ---- A_0 from the Gram product's partial sums (tiles on and above the diagonal)
struct GroupArg {
    const float *part;    // [ranges][batch][n][pn]
    __half *A;            // [batch][2][n][pn]
    int n, pn, ranges, batch, first, b0;   // b0: first matrix of this group in the grid
};
struct Groups {
    GroupArg g[kMostGroups];
    int n;
    const float2 *scal;
    float q_scale[kMaxSteps + 1];   // after each step, for mid_kernel
};

// n > 128: 64 x 64 blocks on and above the diagonal, written to both places
__global__ void __launch_bounds__(256) gram_kernel(const __grid_constant__ Groups P)
{
    __shared__ float tile[64][65];
    pdl_go();
    pdl_wait();
    int q = 0;
    for (int i = 1; i < P.n; ++i)
        if ((int)blockIdx.y >= P.g[i].b0) q = i;
    const GroupArg &g = P.g[q];
    const int b = blockIdx.y - g.b0, nb = (g.n + 63) / 64;
    int ti = 0, t = blockIdx.x;
    if (t >= nb * (nb + 1) / 2) return;
    for (int left = nb; t >= left; --left, ++ti) t -= left;
    const int tj = ti + t;
    const float f = P.scal[g.first + b].y;
    const size_t plane = (size_t)g.n * g.pn;
    __half *A = g.A + (size_t)b * 2 * plane;
    const int x = threadIdx.x & 15, y = threadIdx.x >> 4;   // 4 columns; rows y, y + 16, ..
    auto put = [&](int i, int j, const float (&v)[4]) {
        alignas(8) __half hi[4], lo[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) halves(v[k], hi[k], lo[k]);
        *reinterpret_cast<uint2 *>(A + (size_t)i * g.pn + j) = *reinterpret_cast<uint2 *>(hi);
        *reinterpret_cast<uint2 *>(A + plane + (size_t)i * g.pn + j) = *reinterpret_cast<uint2 *>(lo);
    };
    const int j = tj * 64 + 4 * x;
    const float *part = g.part + (size_t)b * plane + (size_t)(ti * 64 + y) * g.pn + j;
    const size_t step = (size_t)g.batch * plane;
    float4 s[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) s[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int r = 0; r < g.ranges; ++r)
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (ti * 64 + y + 16 * k < g.n && j < g.pn) {
                const float4 v = *reinterpret_cast<const float4 *>(part + r * step + (size_t)(16 * k) * g.pn);
                s[k].x += v.x, s[k].y += v.y, s[k].z += v.z, s[k].w += v.w;
            }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int i = ti * 64 + y + 16 * k;
        const float v[4] = {s[k].x * f, s[k].y * f, s[k].z * f, s[k].w * f};
        if (i < g.n && j < g.pn) put(i, j, v);
#pragma unroll
        for (int c = 0; c < 4; ++c) tile[y + 16 * k][4 * x + c] = v[c];
    }
    if (ti == tj) return;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int i = tj * 64 + y + 16 * k, jj = ti * 64 + 4 * x;
        const float v[4] = {tile[4 * x][y + 16 * k], tile[4 * x + 1][y + 16 * k], tile[4 * x + 2][y + 16 * k],
                            tile[4 * x + 3][y + 16 * k]};
        if (i < g.n && jj < g.pn) put(i, jj, v);
    }
}

// ---- n <= 64: the whole polynomial in one block of 1024 threads, float32 from shared memory
// Only elements on and above the diagonal are computed, each written to both its places (see OrthEpi).  Up to rank 32 a
// thread has one of them: a product is then as long as one dot product (4 matrices of 512 x 16: 27 us with 4 x 4 elements
// a thread, 21 us so).  Above, 256 of the threads have 4 x 4 each, since one word of shared memory per multiply-add would
// bound the products (4 of 64 x 64: 127 us with single elements, 60 us so).
// Rows are 68 words apart, so that 4 columns can be read at once.
constexpr int kSmallP = 68;
constexpr int kSmallThreads = 1024;
constexpr int kSmallMat = 64 * kSmallP;

struct SmallOne {
    float c;
    int i, j;
    bool mine;
    __device__ __forceinline__ SmallOne(int n) : c(0.0f), i(threadIdx.x >> 5), j(threadIdx.x & 31), mine(i <= j && j < n) {}
    // c = s X Y + t D for symmetric X (its row k serves as its column k)
    __device__ __forceinline__ void mul(const float *X, const float *Y, const float *D, float s, float t, int n)
    {
        if (!mine) return;
        float u = 0.0f, v = 0.0f;
        int k = 0;
#pragma unroll 4
        for (; k + 1 < n; k += 2) {
            u = fmaf(X[k * kSmallP + i], Y[k * kSmallP + j], u);
            v = fmaf(X[(k + 1) * kSmallP + i], Y[(k + 1) * kSmallP + j], v);
        }
        if (k < n) u = fmaf(X[k * kSmallP + i], Y[k * kSmallP + j], u);
        c = fmaf(s, u + v, t * D[i * kSmallP + j]);
    }
    __device__ __forceinline__ void put(float *D, int, float diagonal = 0.0f) const
    {
        if (mine) D[i * kSmallP + j] = D[j * kSmallP + i] = c + (i == j ? diagonal : 0.0f);
    }
};

struct SmallTile {
    float c[4][4];
    int ty, tx;
    bool mine;
    __device__ __forceinline__ SmallTile(int n) : ty(threadIdx.x >> 4), tx(threadIdx.x & 15), mine(ty <= tx && 4 * tx < n) {}
    __device__ __forceinline__ void mul(const float *X, const float *Y, const float *D, float s, float t, int n)
    {
        if (!mine) return;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) c[i][j] = 0.0f;
#pragma unroll 4
        for (int k = 0; k < n; ++k) {
            const float4 x = *reinterpret_cast<const float4 *>(X + k * kSmallP + 4 * ty);
            const float4 y = *reinterpret_cast<const float4 *>(Y + k * kSmallP + 4 * tx);
            const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) c[i][j] = fmaf(xs[i], ys[j], c[i][j]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) c[i][j] = fmaf(s, c[i][j], t * D[(4 * ty + i) * kSmallP + 4 * tx + j]);
    }
    __device__ __forceinline__ void put(float *D, int n, float diagonal = 0.0f) const
    {
        if (!mine) return;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (4 * ty + i <= 4 * tx + j && 4 * tx + j < n)
                    D[(4 * ty + i) * kSmallP + 4 * tx + j] = D[(4 * tx + j) * kSmallP + 4 * ty + i] =
                        c[i][j] + (4 * ty + i == 4 * tx + j ? diagonal : 0.0f);
    }
};

// Q_steps from A (shared memory, kSmallMat floats each; p and T are scratch); ends synchronised
template <class E>
__device__ __forceinline__ void small_chain_of(float *A, float *p, float *T, float *Q, int n, int steps)
{
    E c(n), d(n);
    for (int k = 0; k < steps; ++k) {
        c.mul(A, A, A, kC, kB, n);
        c.put(p, n);
        if (k == 0) c.put(Q, n, kA);
        __syncthreads();
        if (k > 0) d.mul(Q, p, Q, 1.0f, kA, n);
        if (k + 1 < steps) {
            c.mul(A, p, A, 1.0f, kA, n);
            c.put(T, n);
        }
        __syncthreads();
        if (k > 0) d.put(Q, n);
        if (k + 1 < steps) {
            c.mul(T, p, T, 1.0f, kA, n);
            c.put(A, n);
        }
        __syncthreads();
    }
}

__device__ __forceinline__ void small_chain(float *A, float *p, float *T, float *Q, int n, int steps)
{
    if (n <= 32) small_chain_of<SmallOne>(A, p, T, Q, n, steps);
    else small_chain_of<SmallTile>(A, p, T, Q, n, steps);
}

__global__ void __launch_bounds__(kSmallThreads) small_kernel(const __grid_constant__ Groups P, int steps, float q_scale)
{
    extern __shared__ __align__(16) float sm[];
    float *A = sm, *p = A + kSmallMat, *T = p + kSmallMat, *Q = T + kSmallMat;
    pdl_go();
    pdl_wait();
    int w = 0;
    for (int i = 1; i < P.n; ++i)
        if ((int)blockIdx.x >= P.g[i].b0) w = i;
    const GroupArg &g = P.g[w];
    const int b = blockIdx.x - g.b0, n = g.n;
    const float f = P.scal[g.first + b].y * (1.0f / kSA);
    const size_t plane = (size_t)n * g.pn;
    for (int e = threadIdx.x; e < 64 * 64; e += kSmallThreads) {
        const int i = e >> 6, j = e & 63;
        if (i >= n || j >= n) continue;
        const float *part = g.part + (size_t)b * plane + (size_t)i * g.pn + j;
        float a = 0.0f;
#pragma unroll 4
        for (int r = 0; r < g.ranges; ++r) a += part[(size_t)r * g.batch * plane];
        A[i * kSmallP + j] = a * f;
    }
    __syncthreads();
    small_chain(A, p, T, Q, n, steps);
    __half *D = g.A + (size_t)b * 2 * plane;
    for (int e = threadIdx.x; e < 64 * 64; e += kSmallThreads) {
        const int i = e >> 6, j = e & 63;
        if (i < n && j < n) {
            __half hi, lo;
            halves(Q[i * kSmallP + j] * q_scale, hi, lo);
            D[(size_t)i * g.pn + j] = hi;
            D[plane + (size_t)i * g.pn + j] = lo;
        }
    }
}

// ---- 64 < n <= 128: the whole polynomial in one block, on its tensor core
// A (and T over it), p and Q stay in shared memory as binary16 halves in the tensor core's layout, 64 KB each, padded with
// zeros to 128.  A product is 24 MMAs of 128 x 128 x 16 (1500 cycles, the tensor core's rate), its epilogue 2750: it adds
// the linear term from the operand it replaces and writes each element of one triangle to both places.  Q's epilogue runs
// beside the product T p, and T's beside Q p.  Three launches a step took 113 to 161 us a call for one to four matrices of
// rank 65 to 100, this 71 to 93 (ranks above 128 would not fit).  The epilogue is not inlined: ten copies
// of it ran out of the instruction caches, at 4200 cycles each.
constexpr int kMidN = 128, kMidThreads = 512;
constexpr uint32_t kMidPlane = 2 * 128 * 128;      // one plane: two blocks of 64 k, 128 rows of 128 bytes each
constexpr uint32_t kMidSlot = 2 * kMidPlane;       // high and low
constexpr size_t kMidSmemBytes = 3 * kMidSlot + 1024 + 64;

__device__ __forceinline__ uint32_t mid_at(int row, int col)   // byte of an element in its plane
{
    return (uint32_t)(col >> 6) * 16384u + (uint32_t)row * 128u + (uint32_t)((((col & 63) >> 3) ^ (row & 7)) << 4) +
           (uint32_t)(col & 7) * 2u;
}

__device__ __forceinline__ void sts16(uint32_t addr, uint16_t v)
{
    asm volatile("st.shared.u16 [%0], %1;\n" ::"r"(addr), "h"(v) : "memory");
}

// acc = X Y for symmetric X and Y: the three products of their halves
__device__ __forceinline__ void mid_mma(uint32_t acc, const unsigned char *X, const unsigned char *Y)
{
    constexpr uint32_t idesc = (1u << 4) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
    uint32_t add = 0;
#pragma unroll
    for (int part = 0; part < 3; ++part) {   // low halves first: the accumulator truncates
        const uint64_t dx = smem_desc_sw128(X + (part == 0 ? kMidPlane : 0)), dy = smem_desc_sw128(Y + (part == 1 ? kMidPlane : 0));
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint64_t off = (uint64_t)((k >> 2) * (16384 >> 4) + (k & 3) * (32 >> 4));
            tc_mma_f16(acc, dx + off, dy + off, idesc, add);
            add = 1;
        }
    }
}

// D = alpha * accumulator + beta * C + diagonal * I, of a 32 x 32 block, a row a lane, to both its places.  D may be C: an
// element and its mirror are read and written by this warp only, and it reads each before it writes it.
template <bool kDiag>
__device__ __noinline__ void mid_block(uint32_t acc, uint32_t C, uint32_t D, int row, int col0, float alpha, float beta,
                                          float diagonal)
{
    uint32_t v[32];
    tmem_ld32(acc, v);
    const uint32_t low_row = (uint32_t)(row >> 6) * 16384u + (uint32_t)(row & 7) * 2u, chunk = (uint32_t)(row & 63) >> 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c0 = col0 + 8 * i;
        const uint32_t at = mid_at(row, c0);
        const uint4 h = lds128(C + at), l = lds128(C + kMidPlane + at);
        const uint32_t ch[4] = {h.x, h.y, h.z, h.w}, cl[4] = {l.x, l.y, l.z, l.w};
        uint32_t oh[4], ol[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 c2 = sum_of(ch[j], cl[j]);
            float2 x = make_float2(fmaf(__uint_as_float(v[8 * i + 2 * j]), alpha, beta * c2.x),
                                   fmaf(__uint_as_float(v[8 * i + 2 * j + 1]), alpha, beta * c2.y));
            if (kDiag) {
                x.x += c0 + 2 * j == row ? diagonal : 0.0f;
                x.y += c0 + 2 * j + 1 == row ? diagonal : 0.0f;
            }
            halves2(x, oh[j], ol[j]);
        }
        if (kDiag) {
            __syncwarp();   // a lane's mirrors are in the others' rows
        } else {
            sts128(D + at, make_uint4(oh[0], oh[1], oh[2], oh[3]));
            sts128(D + kMidPlane + at, make_uint4(ol[0], ol[1], ol[2], ol[3]));
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint16_t hi = (uint16_t)(j & 1 ? oh[j / 2] >> 16 : oh[j / 2]), lo = (uint16_t)(j & 1 ? ol[j / 2] >> 16 : ol[j / 2]);
            const uint32_t mirror = D + low_row + (uint32_t)(c0 + j) * 128u + ((chunk ^ (uint32_t)j) << 4);
            if (!kDiag || c0 + j >= row) {
                sts16(mirror, hi);
                sts16(mirror + kMidPlane, lo);
            }
            if (kDiag && c0 + j > row) {
                sts16(D + at + 2 * j, hi);
                sts16(D + kMidPlane + at + 2 * j, lo);
            }
        }
    }
}

__global__ void __launch_bounds__(kMidThreads, 1) mid_kernel(const __grid_constant__ Groups P, int steps)
{
    extern __shared__ __align__(1024) unsigned char mid_raw[];
    __shared__ uint64_t bars[2];
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    const uint32_t raw = smem_u32(mid_raw);
    unsigned char *const A = mid_raw + (((raw + 1023u) & ~1023u) - raw), *const Pm = A + kMidSlot, *const Q = Pm + kMidSlot;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    volatile int *abort = &abort_flag;
    if (tid == 0) {
        mbar_init(&bars[0], 1);
        mbar_init(&bars[1], 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 256;\n" ::"r"(smem_u32(&tmem_base)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
    }
    pdl_go();
    pdl_wait();
    int w = 0;
    for (int i = 1; i < P.n; ++i)
        if ((int)blockIdx.x >= P.g[i].b0) w = i;
    const GroupArg &g = P.g[w];
    const int b = blockIdx.x - g.b0, n = g.n;
    const float f = P.scal[g.first + b].y;
    const size_t plane = (size_t)n * g.pn;
    const uint32_t sA = smem_u32(A), sP = smem_u32(Pm), sQ = smem_u32(Q);
    // A_0 from the partial sums, on and above the diagonal; zeros around it.  Rows of four elements, four rows and four
    // ranges of a thread in flight together.
    constexpr int kRows = 4, kAtOnce = 4;
    const int jq = lane * 4;
    const size_t range = (size_t)g.batch * plane;
    for (int i0 = warp; i0 < kMidN; i0 += kRows * (kMidThreads / 32)) {
        float4 a[kRows];
        bool in[kRows];
        const float *src[kRows];
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const int i = i0 + u * (kMidThreads / 32);
            a[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            in[u] = i < n && jq < g.pn && jq + 3 >= i;
            src[u] = g.part + (size_t)b * plane + (size_t)i * g.pn + jq;
        }
        for (int r = 0; r < g.ranges; r += kAtOnce) {
            float4 v[kAtOnce][kRows];
#pragma unroll
            for (int q = 0; q < kAtOnce; ++q)
#pragma unroll
                for (int u = 0; u < kRows; ++u)
                    v[q][u] = in[u] && r + q < g.ranges ? *reinterpret_cast<const float4 *>(src[u] + (r + q) * range)
                                                        : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int q = 0; q < kAtOnce; ++q)
#pragma unroll
                for (int u = 0; u < kRows; ++u) a[u].x += v[q][u].x, a[u].y += v[q][u].y, a[u].z += v[q][u].z, a[u].w += v[q][u].w;
        }
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const int i = i0 + u * (kMidThreads / 32);
            const float x[4] = {a[u].x, a[u].y, a[u].z, a[u].w};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int jc = jq + c;
                if (jc < i) continue;
                __half hi, lo;
                halves(jc < n ? x[c] * f : 0.0f, hi, lo);
                sts16(sA + mid_at(i, jc), __half_as_ushort(hi));
                sts16(sA + kMidPlane + mid_at(i, jc), __half_as_ushort(lo));
                sts16(sA + mid_at(jc, i), __half_as_ushort(hi));
                sts16(sA + kMidPlane + mid_at(jc, i), __half_as_ushort(lo));
            }
        }
    }
    fence_proxy_async();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    // The 4 blocks on the diagonal and one of each mirrored pair: 3, 3, 2 and 2 for the four row quarters, each of which
    // only the warps of one scheduler can read
    const int quarter = warp & 3, col0 = ((quarter + (warp >> 2)) & 3) * 32, row0 = quarter * 32, row = row0 + lane;
    const bool mine = warp < 8 || (warp < 12 && quarter < 2);
    const uint32_t acc = tmem + ((uint32_t)row0 << 16) + (uint32_t)col0;
    auto block = [&](uint32_t from, uint32_t C, uint32_t D, float alpha, float beta, float diagonal) {
        if (!mine) return;
        if (warp < 4) mid_block<true>(from, C, D, row, col0, alpha, beta, diagonal);
        else mid_block<false>(from, C, D, row, col0, alpha, beta, 0.0f);
    };
    // the accumulators of bars[w] are there for every thread, or the wait gave up (bounded) and all leave
    uint32_t phase[2] = {0, 0};
    auto finished = [&](int w) -> bool {
        const bool ok = mbar_wait(&bars[w], phase[w], abort, &g_mm_err, 6);
        phase[w] ^= 1;
        tc_fence_after();
        return __syncthreads_and(ok) != 0;
    };
    // what was written is there for the next products
    auto written = [&]() {
        fence_proxy_async();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    };
    // Products are issued by a warp that has no epilogue: issuing waits for the tensor core
    auto product = [&](int w, const unsigned char *X, const unsigned char *Y) {
        if (warp == kMidThreads / 32 - 1 && elect_one()) {
            mid_mma(tmem + 128 * w, X, Y);
            tc_commit(&bars[w]);
        }
        __syncwarp();
    };
    float scale = kSA;   // of Q
    bool ok = true;
    for (int k = 0; k < steps; ++k) {
        // p = b A + c A^2; the first also gives Q_1 = a I + p
        product(0, A, A);
        if (!(ok = finished(0))) break;
        block(acc, sA, sP, kC / kSA, kB, 0.0f);
        if (k == 0) block(acc, sA, sQ, kC / kSA, kB, kA * kSA);
        written();
        // T = a A + A p over A while Q p runs, then Q <- a Q + Q p while T p runs
        const bool more = k + 1 < steps;
        if (more) product(0, A, Pm);
        if (k) product(1, Q, Pm);
        if (more) {
            if (!(ok = finished(0))) break;
            block(acc, sA, sA, 1.0f / kSA, kA, 0.0f);
            written();
            product(0, A, Pm);
        }
        if (k) {
            if (!(ok = finished(1))) break;
            const float next = P.q_scale[k + 1], fq = next / scale;
            block(acc + 128, sQ, sQ, fq / kSA, kA * fq, 0.0f);
            scale = next;
        }
        if (more) {   // A <- a T + T p
            if (!(ok = finished(0))) break;
            block(acc, sA, sA, 1.0f / kSA, kA, 0.0f);
        }
        written();
    }
    if (ok) {
        __half *const D = g.A + (size_t)b * 2 * plane;
        for (int e = tid; e < 2 * n * 16; e += kMidThreads) {   // 16-byte chunks of both planes' rows
            const int p = e / (n * 16), r = (e / 16) % n, c = (e & 15) * 8;
            if (c < n)
                *reinterpret_cast<uint4 *>(D + p * plane + (size_t)r * g.pn + c) = lds128(sQ + p * kMidPlane + mid_at(r, c));
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 256;\n" ::"r"(tmem));
    }
}

// ---- a whole small matrix in one block
constexpr int kTinyElems = 24576;   // m times n rounded up to 4
struct TinyMat {
    const void *G;
    uint16_t *O;
    int rows, cols;
};
struct Tinies {
    TinyMat m[kMostMats];
    int bf16, steps;
    float eps;
};

__global__ void __launch_bounds__(kSmallThreads) tiny_kernel(const __grid_constant__ Tinies P)
{
    extern __shared__ __align__(16) float sm[];
    float *X = sm;                                        // m x pitch: G, or its transpose
    __shared__ double sums[32], scale;
    const TinyMat &M = P.m[blockIdx.x];
    const int rows = M.rows, cols = M.cols, tid = threadIdx.x;
    const bool wide = rows < cols;
    const int m = max(rows, cols), n = min(rows, cols), pitch = (n + 3) & ~3;
    const int total = rows * cols, size = m * pitch;
    float *A = X + size, *p = A + kSmallMat, *T = p + kSmallMat, *Q = T + kSmallMat;

    if (pitch != n)
        for (int e = tid; e < size; e += kSmallThreads) X[e] = 0.0f;
    if (pitch != n) __syncthreads();
    double s = 0.0;
    const float inv = 1.0f / (float)cols;   // total < 2^15: the quotient below is exact
#pragma unroll 8
    for (int e = tid; e < total; e += kSmallThreads) {
        const float x = load_g(M.G, e, P.bf16);
        const int r = (int)(((float)e + 0.5f) * inv), c = e - r * cols;
        X[wide ? c * pitch + r : r * pitch + c] = x;
        s += (double)x * x;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((tid & 31) == 0) sums[tid >> 5] = s;
    __syncthreads();
    if (tid < 32) {
        s = sums[tid];
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (tid == 0) {
            const double norm = sqrt(s);
            scale = norm == 0.0 ? 0.0 : 1.0 / (norm + (double)P.eps);
        }
    }
    __syncthreads();
    const double f = scale;
    for (int e = tid; e < size; e += kSmallThreads) X[e] = (float)(X[e] * f);
    __syncthreads();

    // A = X^T X: 4 x 4 tiles, the rows of X dealt to as many groups of threads as there are
    {
        const int td = pitch / 4, tiles = td * td, groups = min(kSmallThreads / tiles, 3 * kSmallMat / (pitch * pitch));
        const int g = tid / tiles, t = tid - g * tiles, ty = t / td, tx = t - ty * td;
        float *const part = p;   // the groups' sums in p, T and Q, which are one array, then added in order
        if (g < groups) {
            float c[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) c[i][j] = 0.0f;
#pragma unroll 4
            for (int k = g; k < m; k += groups) {
                const float4 x = *reinterpret_cast<const float4 *>(X + k * pitch + 4 * ty);
                const float4 y = *reinterpret_cast<const float4 *>(X + k * pitch + 4 * tx);
                const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) c[i][j] = fmaf(xs[i], ys[j], c[i][j]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) part[(g * pitch + 4 * ty + i) * pitch + 4 * tx + j] = c[i][j];
        }
        __syncthreads();
        for (int e = tid; e < pitch * pitch; e += kSmallThreads) {
            float a = 0.0f;
#pragma unroll 8
            for (int i = 0; i < groups; ++i) a += part[i * pitch * pitch + e];
            A[e / pitch * kSmallP + e % pitch] = a;
        }
        __syncthreads();
    }
    small_chain(A, p, T, Q, n, P.steps);

    // Q with rows of 64, for reads of 4 columns at once (into A and p, which are done with)
    float *const Q4 = reinterpret_cast<float *>(((uintptr_t)A + 15) & ~(uintptr_t)15);
    for (int e = tid; e < n * 64; e += kSmallThreads) Q4[e] = (e & 63) < n ? Q[(e >> 6) * kSmallP + (e & 63)] : 0.0f;
    for (int e = n * 64 + tid; e < pitch * 64; e += kSmallThreads) Q4[e] = 0.0f;
    __syncthreads();
    // the update, 4 columns of a row of X Q at a time; neighbours take the other columns of the row
    const int nj = pitch / 4;
    const float inv_nj = 1.0f / (float)nj;
    const bool vec = !wide && n % 4 == 0 && ((uintptr_t)M.O & 7) == 0;
    for (int e = tid; e < m * nj; e += kSmallThreads) {
        const int i = (int)(((float)e + 0.5f) * inv_nj), j = 4 * (e - i * nj);
        float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 2
        for (int k = 0; k < pitch; k += 4) {
            const float4 x4 = *reinterpret_cast<const float4 *>(X + i * pitch + k);
            const float x[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float4 q = *reinterpret_cast<const float4 *>(Q4 + (k + u) * 64 + j);
                a.x = fmaf(x[u], q.x, a.x);
                a.y = fmaf(x[u], q.y, a.y);
                a.z = fmaf(x[u], q.z, a.z);
                a.w = fmaf(x[u], q.w, a.w);
            }
        }
        const uint32_t lo = pack_bf(__float_as_uint(a.x), __float_as_uint(a.y), 1.0f);
        const uint32_t hi = pack_bf(__float_as_uint(a.z), __float_as_uint(a.w), 1.0f);
        if (vec) {
            *reinterpret_cast<uint2 *>(M.O + (size_t)i * n + j) = make_uint2(lo, hi);
        } else {
            const uint16_t o[4] = {(uint16_t)lo, (uint16_t)(lo >> 16), (uint16_t)hi, (uint16_t)(hi >> 16)};
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (j + u < n) M.O[wide ? (size_t)(j + u) * m + i : (size_t)i * n + j + u] = o[u];
        }
    }
}

// ---- host
size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }
bool misaligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) != 0; }

// Matrices of one shape, consecutive in the order of a set of launches.
struct Group {
    int rows, cols, m, n, pn, pitch, first, batch, ranges;
    size_t X, part, A, q, T, Q0, Q1;   // workspace offsets; part shares its place with q, T, Q0 and Q1
    bool wide;
};
struct Chunk {
    std::vector<int> order;
    std::vector<Group> groups;
    size_t sums, scal, bytes;
    bool tiny;
};

bool is_tiny(int r, int c)
{
    const long n = std::min(r, c), m = std::max(r, c);
    return n <= kSmallN && m * ((n + 3) & ~3L) <= kTinyElems;
}

// Sets of at most kMostMats matrices and kMostGroups shapes, the longest units first in each.
void orth_chunks(std::vector<Chunk> &out, const int *rows, const int *cols, int count, bool bf16)
{
    std::vector<int> idx(count);
    for (int i = 0; i < count; ++i) idx[i] = i;
    std::sort(idx.begin(), idx.end(), [&](int a, int b) {
        const int na = std::min(rows[a], cols[a]), nb = std::min(rows[b], cols[b]);
        const bool ta = is_tiny(rows[a], cols[a]), tb = is_tiny(rows[b], cols[b]);
        if (ta != tb) return tb;
        if (na != nb) return na > nb;
        if (rows[a] != rows[b]) return rows[a] > rows[b];
        if (cols[a] != cols[b]) return cols[a] > cols[b];
        return a < b;
    });
    for (int at = 0; at < count;) {
        Chunk C;
        C.tiny = is_tiny(rows[idx[at]], cols[idx[at]]);
        C.bytes = 0;
        while (at < count && (int)C.order.size() < kMostMats) {
            const int i = idx[at];
            if (is_tiny(rows[i], cols[i]) != C.tiny) break;
            if (C.tiny) {
                C.order.push_back(i);
                ++at;
                continue;
            }
            if (C.groups.empty() || C.groups.back().rows != rows[i] || C.groups.back().cols != cols[i]) {
                if ((int)C.groups.size() == kMostGroups) break;
                Group g;
                memset(&g, 0, sizeof(g));
                g.rows = rows[i];
                g.cols = cols[i];
                g.wide = rows[i] < cols[i];
                g.m = std::max(rows[i], cols[i]);
                g.n = std::min(rows[i], cols[i]);
                g.pn = (g.n + 63) & ~63;
                g.pitch = (cols[i] + 63) & ~63;
                g.first = (int)C.order.size();
                C.groups.push_back(g);
            }
            ++C.groups.back().batch;
            C.order.push_back(i);
            ++at;
        }
        if (C.tiny) {
            out.push_back(std::move(C));
            continue;
        }
        // Ranges of the Gram products, in products of 64 deep by a pair (0.27 us): the longest list of units as they are
        // dealt, and the writing and reading of the ranges' partial sums at the copy rate.  Units of at least 24 of them.
        const int parts = bf16 ? 1 : 3, pairs = 74;
        auto blocks = [&](const Group &g) { return (long)(g.m + kMmBK - 1) / kMmBK; };
        auto tiles = [&](const Group &g) {
            const int nt = (g.n + kMmTile - 1) / kMmTile;
            return (long)mm_tiles(nt, nt, true, kMmTile) * g.batch;
        };
        auto cut = [&](const Group &g, long unit) {   // as mm_plan cuts
            // no range above 256 blocks, some 50 of the pieces that are added in a row
            const long k = blocks(g), most = std::max(64L, (k + 255) / 256);
            const long r = std::min(most, std::max((k + 255) / 256, (k * parts + unit - 1) / unit)), per = (k + r - 1) / r;
            return (k + per - 1) / per;
        };
        double total = 0.0;
        for (const Group &g : C.groups) total += (double)tiles(g) * blocks(g) * parts;
        long unit = 24;
        double best = 1e300;
        for (int c = 1; c <= 12; ++c) {
            const long u = std::max(24L, (long)(total / (pairs * c)) + 1);
            std::vector<double> load(pairs, 0.0);
            double bytes = 0.0;
            long at_unit = 0;
            for (const Group &g : C.groups) {
                const long r = cut(g, u);
                for (long x = 0; x < tiles(g) * r; ++x) load[at_unit++ % pairs] += (double)blocks(g) * parts / r + 4.0;
                bytes += (double)r * g.batch * g.n * g.pn * 4.0 * 2.0;
            }
            const double cost = *std::max_element(load.begin(), load.end()) + bytes / 1.8e6;
            if (cost < best) {
                best = cost;
                unit = u;
            }
            if (u == 24) break;
        }
        size_t o = 0;
        auto take = [&](size_t b) {
            const size_t r = o;
            o = up256(o + b);
            return r;
        };
        C.sums = take(C.order.size() * kNormBlocks * sizeof(double));
        C.scal = take(C.order.size() * sizeof(float2));
        for (Group &g : C.groups) {
            g.ranges = (int)cut(g, unit);
            const size_t nn = (size_t)g.batch * 2 * g.n * g.pn * 2;
            g.X = take((size_t)g.batch * (bf16 ? 1 : 2) * g.rows * g.pitch * 2);
            g.A = take(nn);
            g.part = o;
            g.q = take(nn);
            g.T = take(nn);
            g.Q0 = take(nn);
            g.Q1 = take(nn);
            o = std::max(o, up256(g.part + (size_t)g.ranges * g.batch * g.n * g.pn * 4));
        }
        C.bytes = o;
        out.push_back(std::move(C));
    }
}

float q_scale_after(int k) { return exp2f(floorf(log2f(50000.0f / powf(kA, (float)k)))); }

lb_status orth_chunk(const Chunk &C, const void *const *Gs, bool bf16, int steps, float eps, uint16_t *const *Os,
                     unsigned char *ws, cudaStream_t s, int *launches)
{
    Mats M;
    memset(&M, 0, sizeof(M));
    M.n = (int)C.order.size();
    M.bf16 = bf16 ? 1 : 0;
    M.eps = eps;
    M.sums = (double *)(ws + C.sums);
    M.scal = (float2 *)(ws + C.scal);
    int most_blocks = 1;
    for (const Group &g : C.groups)
        for (int b = 0; b < g.batch; ++b) {
            Mat &m = M.m[g.first + b];
            m.G = Gs[C.order[g.first + b]];
            m.X = (__half *)(ws + g.X) + (size_t)b * (bf16 ? 1 : 2) * g.rows * g.pitch;
            m.rows = g.rows;
            m.cols = g.cols;
            m.pitch = g.pitch;
            const size_t n = (size_t)g.rows * g.cols;
            m.nblocks = (int)std::min<size_t>(kNormBlocks, (n + 8191) / 8192);
            most_blocks = std::max(most_blocks, m.nblocks);
        }
    const dim3 blocks_of_all(most_blocks, M.n);
    cudaError_t e = launch_after(norm_kernel, blocks_of_all, 256, s, M);
    if (e != cudaSuccess) return status_from(e);
    if ((e = launch_after(split_kernel, blocks_of_all, 256, s, M)) != cudaSuccess) return status_from(e);
    *launches += 2;

    MmBatch<kMostProbs> B;
    OrthEpi::Params E;
    memset(&E, 0, sizeof(E));
    E.scal = M.scal;
    for (int i = 0; i < M.n; ++i) E.out[i] = Os[C.order[i]];
    const int parts = bf16 ? 1 : 3, xz = bf16 ? 1 : 2;
    int pairs = 0;
    if ((e = mm_pairs(&pairs)) != cudaSuccess) return status_from(e);
    // Widest tiles of a launch that still give every pair of SMs one: a few small matrices are bound by the length of one
    // tile's chain (copy, products, epilogue), many or large ones by the operands read per tile.
    auto width_of = [&](auto &&tiles) {
        int w = kMmTile;
        while (w > 64 && tiles(w) < pairs) w >>= 1;
        return w;
    };
    auto square_tiles = [&](int w) {
        long t = 0;
        for (const Group &g : C.groups)
            if (g.n > kMidN)
                t += (long)g.batch * mm_tiles((g.n + kMmTile - 1) / kMmTile, (g.n + w - 1) / w, true, w);
        return t;
    };
    auto update_tiles = [&](int w) {
        long t = 0;
        for (const Group &g : C.groups)
            t += (long)g.batch * ((g.rows + kMmTile - 1) / kMmTile) * ((g.cols + w - 1) / w);
        return t;
    };
    const int wq = width_of(square_tiles), wo = width_of(update_tiles);
    bool ok = true;
    auto begin = [&]() { memset(&B, 0, sizeof(B)); };
    MmOrder one, two;   // of the launches with one product of each matrix, and with two
    one.n = two.n = -1;
    auto deal = [&](MmOrder &O) {
        if (O.n < 0) mm_deal(O, B.p, B.n, B.nunits, pairs);
        B.order = O;
    };
    auto launch = [&]() -> cudaError_t {
        if (B.n == 0) return cudaSuccess;
        ++*launches;
        return mm_launch<false, kMostProbs, OrthEpi>(B, E, s);
    };

    // A_0: both operands are X, contracted over the long axis
    MmBatch<kMostGroups> R;
    GramEpi::Params D;
    memset(&R, 0, sizeof(R));
    for (const Group &g : C.groups) {
        MmProb &P = R.p[R.n];
        mm_plan(P, g.n, g.n, g.m, false, R.nunits, g.ranges, parts, g.batch, true);
        mm_chunk(P, kGramChunk / parts);
        P.a_mn = P.b_mn = g.wide ? 0 : 1;
        P.za = P.zb = xz;
        ok = ok && mm_operand(&R.mA[R.n], false, P.a_mn, ws + g.X, g.rows, g.cols, g.pitch, (long)g.batch * xz);
        R.mB[R.n] = R.mA[R.n];
        ok = ok && tmap_encode_3d(&D.mD[R.n], CU_TENSOR_MAP_DATA_TYPE_FLOAT32, ws + g.part, g.pn, g.n,
                                  (long)g.ranges * g.batch, (long)g.pn * 4, (long)g.n * g.pn * 4, 32, 32);
        R.nunits += mm_units(P);
        ++R.n;
    }
    mm_deal(R.order, R.p, R.n, R.nunits, pairs);
    if (!ok) return LB_ERR_CUDA;
    ++*launches;
    if ((e = mm_launch<false, kMostGroups, GramEpi>(R, D, s)) != cudaSuccess) return status_from(e);

    // the small ranks' polynomials, the others' A_0
    Groups big, mid, small;
    memset(&big, 0, sizeof(big));
    memset(&mid, 0, sizeof(mid));
    memset(&small, 0, sizeof(small));
    big.scal = mid.scal = small.scal = M.scal;
    for (int k = 0; k <= steps; ++k) mid.q_scale[k] = q_scale_after(k);
    int bigs = 0, mids = 0, smalls = 0, blocks = 0;
    for (const Group &g : C.groups) {
        Groups &to = g.n <= kSmallN ? small : g.n <= kMidN ? mid : big;
        int &count = g.n <= kSmallN ? smalls : g.n <= kMidN ? mids : bigs;
        GroupArg &a = to.g[to.n++];
        a.part = (const float *)(ws + g.part);
        a.A = (__half *)(ws + g.A);
        a.n = g.n;
        a.pn = g.pn;
        a.ranges = g.ranges;
        a.batch = g.batch;
        a.first = g.first;
        a.b0 = count;
        count += g.batch;
        const int nb = (g.n + 63) / 64;
        if (g.n > kMidN) blocks = std::max(blocks, nb * (nb + 1) / 2);
    }
    if (bigs) {
        if ((e = launch_after(gram_kernel, dim3(blocks, bigs), 256, s, big)) != cudaSuccess) return status_from(e);
        ++*launches;
    }
    if (mids) {
        if ((e = ensure_dyn_smem((const void *)mid_kernel, kMidSmemBytes)) != cudaSuccess) return status_from(e);
        if ((e = launch_after_smem(mid_kernel, dim3(mids), kMidThreads, kMidSmemBytes, s, mid, steps)) != cudaSuccess)
            return status_from(e);
        ++*launches;
    }
    if (smalls) {
        const size_t smem = 4 * kSmallMat * sizeof(float);
        if ((e = ensure_dyn_smem((const void *)small_kernel, smem)) != cudaSuccess) return status_from(e);
        if ((e = launch_after_smem(small_kernel, dim3(smalls), kSmallThreads, smem, s, small, steps, q_scale_after(steps))) != cudaSuccess)
            return status_from(e);
        ++*launches;
    }

    // n > 128: three launches a step
    // d = alpha * x y + beta * c
    auto square = [&](const Group &g, size_t x, size_t y, size_t d, float alpha, float beta, size_t c) -> OrthProb & {
        MmProb &P = B.p[B.n];
        OrthProb &O = E.p[B.n];
        mm_plan(P, g.n, g.n, g.n, false, B.nunits, 1, 3, g.batch, true, wq);
        P.za = P.zb = 2;
        ok = ok && mm_operand(&B.mA[B.n], false, false, ws + x, g.n, g.n, g.pn, 2L * g.batch) &&
             mm_operand(&B.mB[B.n], false, false, ws + y, g.n, g.n, g.pn, 2L * g.batch, wq / 2);
        O.kind = kSym;
        O.pn = g.pn;
        O.first = g.first;
        O.alpha = alpha;
        O.beta = beta;
        O.C = (const __half *)(ws + c);
        O.D = (__half *)(ws + d);
        O.D2 = nullptr;
        B.nunits += mm_units(P);
        ++B.n;
        return O;
    };
    for (int k = 0; bigs && k < steps; ++k) {
        begin();   // p = b A + c A^2; the first also gives Q_1 = a I + p
        for (const Group &g : C.groups) {
            if (g.n <= kMidN) continue;
            OrthProb &O = square(g, g.A, g.A, g.q, kC / kSA, kB, g.A);
            if (k == 0) {
                O.D2 = (__half *)(ws + g.Q0);
                O.gamma = kA * kSA;
            }
        }
        deal(one);
        if (!ok) return LB_ERR_CUDA;
        if ((e = launch()) != cudaSuccess) return status_from(e);
        if (k + 1 == steps && k == 0) break;
        begin();   // T = a A + A p, and Q <- a Q + Q p
        for (const Group &g : C.groups) {
            if (g.n <= kMidN) continue;
            if (k + 1 < steps) square(g, g.A, g.q, g.T, 1.0f / kSA, kA, g.A);
            if (k) {
                const size_t from = k & 1 ? g.Q0 : g.Q1, to = k & 1 ? g.Q1 : g.Q0;
                const float f = q_scale_after(k + 1) / (k == 1 ? kSA : q_scale_after(k));
                square(g, from, g.q, to, f / kSA, kA * f, from);
            }
        }
        deal(k && k + 1 < steps ? two : one);
        if (!ok) return LB_ERR_CUDA;
        if ((e = launch()) != cudaSuccess) return status_from(e);
        if (k + 1 == steps) break;
        begin();   // A <- a T + T p
        for (const Group &g : C.groups)
            if (g.n > kMidN) square(g, g.T, g.q, g.A, 1.0f / kSA, kA, g.T);
        deal(one);
        if (!ok) return LB_ERR_CUDA;
        if ((e = launch()) != cudaSuccess) return status_from(e);
    }

    // the update: X Q, or Q X of a wide matrix
    begin();
    for (const Group &g : C.groups) {
        MmProb &P = B.p[B.n];
        OrthProb &O = E.p[B.n];
        const bool sm = g.n <= kMidN;   // Q is where A_0 would be
        const size_t Q = sm ? g.A : (steps - 1) & 1 ? g.Q1 : g.Q0;
        mm_plan(P, g.rows, g.cols, g.n, false, B.nunits, 1, bf16 ? 2 : 3, g.batch, false, wo);
        CUtensorMap mQ, mX;
        ok = ok && mm_operand(&mQ, false, false, ws + Q, g.n, g.n, g.pn, 2L * g.batch, g.wide ? kMmHalf : wo / 2) &&
             mm_operand(&mX, false, g.wide, ws + g.X, g.rows, g.cols, g.pitch, (long)g.batch * xz);
        B.mA[B.n] = g.wide ? mQ : mX;
        B.mB[B.n] = g.wide ? mX : mQ;
        P.b_mn = g.wide ? 1 : 0;
        P.b_whole = g.wide ? 1 : 0;
        P.za = g.wide ? 2 : xz;
        P.zb = g.wide ? xz : 2;
        O.kind = kOut;
        O.first = g.first;
        O.alpha = 1.0f / (g.n > kSmallN && steps == 1 ? kSA : q_scale_after(steps));
        O.ldo = g.cols;
        B.nunits += mm_units(P);
        ++B.n;
    }
    mm_deal(B.order, B.p, B.n, B.nunits, pairs);
    if (!ok) return LB_ERR_CUDA;
    if ((e = launch()) != cudaSuccess) return status_from(e);
    return status_from(cudaGetLastError());
}

lb_status tiny_chunk(const Chunk &C, const void *const *Gs, const int *rows, const int *cols, bool bf16, int steps, float eps,
                     uint16_t *const *Os, cudaStream_t s, int *launches)
{
    Tinies T;
    memset(&T, 0, sizeof(T));
    T.bf16 = bf16 ? 1 : 0;
    T.steps = steps;
    T.eps = eps;
    int most = 0;
    for (size_t k = 0; k < C.order.size(); ++k) {
        const int i = C.order[k], n = std::min(rows[i], cols[i]), m = std::max(rows[i], cols[i]);
        T.m[k] = TinyMat{Gs[i], Os[i], rows[i], cols[i]};
        most = std::max(most, m * ((n + 3) & ~3));
    }
    const size_t smem = (size_t)(4 * kSmallMat + most) * sizeof(float);
    const cudaError_t e = ensure_dyn_smem((const void *)tiny_kernel, smem);
    if (e != cudaSuccess) return status_from(e);
    tiny_kernel<<<(unsigned)C.order.size(), kSmallThreads, smem, s>>>(T);
    ++*launches;
    return status_from(cudaGetLastError());
}

bool orth_shapes_ok(const int *rows, const int *cols, int n)
{
    if (n < 0 || (n > 0 && (!rows || !cols))) return false;
    for (int i = 0; i < n; ++i)
        if (rows[i] < 1 || cols[i] < 1) return false;
    return true;
}
bool orth_supported(int rows, int cols)
{
    return std::min(rows, cols) <= LB_MAX_RANK && std::max(rows, cols) <= (1 << 24);
}

}  // namespace

lb_status orth_status(cudaStream_t s) { return mm_status(s); }

}  // namespace lb

using namespace lb;

extern "C" size_t lb_orthogonalise_workspace_bytes(const int *rows, const int *cols, int n, int dtype)
{
    if (!orth_shapes_ok(rows, cols, n) || (dtype != LB_F32 && dtype != LB_BF16)) return 0;
    for (int i = 0; i < n; ++i)
        if (!orth_supported(rows[i], cols[i])) return 0;
    try {
        std::vector<Chunk> chunks;
        orth_chunks(chunks, rows, cols, n, dtype == LB_BF16);
        size_t most = 0;
        for (const Chunk &c : chunks) most = std::max(most, c.bytes);
        return most;
    } catch (...) {
        return 0;
    }
}

extern "C" lb_status lb_orthogonalise(const void *const *G, int dtype, const int *rows, const int *cols, int n, int steps,
                                      float eps, uint16_t *const *O, void *workspace, size_t workspace_bytes,
                                      void *stream)
{
    set_launch_count(0);
    if (!orth_shapes_ok(rows, cols, n) || (dtype != LB_F32 && dtype != LB_BF16) || steps < 1 || !(eps >= 0.0f))
        return LB_ERR_INVALID_ARG;
    if (steps > kMaxSteps) return LB_ERR_UNSUPPORTED;
    if (n == 0) return LB_OK;
    if (!G || !O) return LB_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i) {
        if (!G[i] || !O[i] || misaligned(G[i], dtype == LB_F32 ? 4 : 2) || misaligned(O[i], 2)) return LB_ERR_INVALID_ARG;
        if (!orth_supported(rows[i], cols[i])) return LB_ERR_UNSUPPORTED;
    }
    try {
        std::vector<Chunk> chunks;
        orth_chunks(chunks, rows, cols, n, dtype == LB_BF16);
        for (const Chunk &c : chunks)
            if (c.bytes && (!workspace || misaligned(workspace, 256) || workspace_bytes < c.bytes)) return LB_ERR_INVALID_ARG;
        if (tmap_encoder_ready() != cudaSuccess) return LB_ERR_UNSUPPORTED;
        int launches = 0;
        for (const Chunk &c : chunks) {
            const bool bf16 = dtype == LB_BF16;
            cudaStream_t s = (cudaStream_t)stream;
            const lb_status st = c.tiny ? tiny_chunk(c, G, rows, cols, bf16, steps, eps, O, s, &launches)
                                        : orth_chunk(c, G, bf16, steps, eps, O, (unsigned char *)workspace, s, &launches);
            if (st != LB_OK) return st;
        }
        set_launch_count(launches);
    } catch (const std::bad_alloc &) {
        return LB_ERR_OOM;
    } catch (...) {
        return LB_ERR_INVALID_ARG;
    }
    return LB_OK;
}
