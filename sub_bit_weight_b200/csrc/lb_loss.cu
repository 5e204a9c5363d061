// Softmax cross entropy of hidden states H [M][D] against a vocabulary matrix
// W [V][D], with the gradients of both, without keeping the logits.
//
//     z = H W^T,  lse = log sum_v exp z_v,  loss = lse - z_label
//     G = w (softmax(z) - onehot),  dH = G W,  dW = G^T H
//
// Floor: 2 M V D flops for the loss and 6 M V D with both gradients (H and W
// are read once from memory: at the sizes of a training step the tensor cores
// bound all three products).  So every logit is computed once:
//
//   1  z tiles (256 rows x 256 vocabulary entries) on CTA pairs.  The epilogue
//      takes each row's maximum m and sum of exp(z - m) over the tile (one
//      thread a row and 128 columns, which it holds in registers) and, for the gradient,
//      leaves e = 2^15 exp(z - m) in binary16: at most 2^15, right to 2^-11
//      down to 2^-29 of the maximum of those columns and to 2^-40 of that
//      maximum below (so less than that is 0).
//   2  one block per row and 8192 entries: lse from the tiles' (m, s), then
//      G / max w = w / max w (e exp(m - lse) 2^-15 - onehot), rounded to
//      bfloat16, over e, and what this rounding left of the label's entry.
//   3  dH = G W, with that rest, and dW = G^T H in one launch; G and W (dH) and
//      G and H (dW) are read in the orientation they are stored in, whichever
//      index is contracted.
//
// Keeping e costs 2 bytes a logit of one piece of rows, written, turned into G
// and read twice; recomputing z instead would cost a third more flops.

#include <algorithm>
#include <cmath>
#include <cstring>

#include "lb_mm.cuh"
#include "littlebit_train.h"

namespace lb {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kEScale = 15.0f;        // e is stored times 2^15
constexpr int kChunk = 16;             // k blocks (1024 k) one accumulator takes, see lb_mm.cuh
constexpr int kGradCols = 8192;         // entries of a row one block of the second step takes, or up to four times that
constexpr int kRowsDefault = 8192, kRowsMost = 32768;

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ uint32_t pack_bf2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// value where at == i, else `other`; opaque, so that a loop of them is not turned into an indexed copy of the registers
__device__ __forceinline__ uint32_t pick(int at, int i, uint32_t value, uint32_t other)
{
    uint32_t r;
    asm("{\n.reg .pred p;\nsetp.eq.s32 p, %1, %2;\nselp.b32 %0, %3, %4, p;\n}\n"
        : "=r"(r)
        : "r"(at), "r"(i), "r"(value), "r"(other));
    return r;
}

// Before the staging block is written again, its last copy must have been read.
__device__ __forceinline__ void staging_free(bool &stored, int lane)
{
    if (stored) {
        if (lane == 0) tma_store_wait_read();
        __syncwarp();
    }
    stored = true;
}

// ---- 1: statistics of 128 columns of a row of logits (kKeep: and e)
template <bool kKeep>
struct LogitEpi {
    static constexpr bool kManyRegs = true;
    struct Params {
        CUtensorMap mE;            // binary16 [rows][Vp]
        const int64_t *labels;
        float2 *stat;              // [rows][nst]: (reference exponent, sum), base 2, of each 128 columns
        float *target;             // [rows]: z of the label
        int M, V, nst;
    };
    struct State {
        float z[kMmHalf];          // the row's logits
        int at;                    // column of the label, -1 if it is not among them
    };
    static __device__ __forceinline__ void begin(const Params &E, const MmProb &, const MmUnit &, const MmTileCtx &T,
                                                 State &S)
    {
        const int row = T.row0 + T.lane;
        const long long lab = T.cols > 0 && row < E.M ? E.labels[row] : -1;
        S.at = lab >= T.col0 && lab < T.col0 + T.cols ? (int)(lab - T.col0) : -1;
    }
    static __device__ __forceinline__ void take(const Params &, const MmProb &, const MmUnit &, const MmTileCtx &T,
                                                State &S, bool first, bool, bool &)
    {
        if (T.cols == 0) return;
#pragma unroll
        for (int c = 0; c < kMmHalf; c += 32) {
            uint32_t v[32];
            tmem_ld32(T.tmem + c, v);
#pragma unroll
            for (int i = 0; i < 32; ++i)
                S.z[c + i] = first ? __uint_as_float(v[i]) : S.z[c + i] + __uint_as_float(v[i]);
        }
    }
    static __device__ __forceinline__ void end(const Params &E, const MmProb &, const MmUnit &, const MmTileCtx &T,
                                               State &S, bool &stored)
    {
        if (T.cols == 0) return;
        const int row = T.row0 + T.lane;
        if (T.cols < kMmHalf) {
#pragma unroll
            for (int i = 0; i < kMmHalf; ++i)
                if (i >= T.cols) S.z[i] = -INFINITY;
        }
        float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < kMmHalf; ++i) m[i & 3] = fmaxf(m[i & 3], S.z[i]);
        if (S.at >= 0) {
            uint32_t z = 0;
#pragma unroll
            for (int i = 0; i < kMmHalf; ++i) z = pick(S.at, i, __float_as_uint(S.z[i]), z);
            E.target[row] = __uint_as_float(z);
        }
        const float mx = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
        const float ref = fmaf(mx, kLog2e, -kEScale);
        const float sub = mx == -INFINITY ? 0.0f : ref;   // nothing but -inf (or NaN): weights 0 (or NaN)
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < kMmHalf; ++i) {
            S.z[i] = ex2(fmaf(S.z[i], kLog2e, -sub));
            s[i & 3] += S.z[i];
        }
        if (row < E.M)
            E.stat[(size_t)row * E.nst + T.col0 / kMmHalf] = make_float2(ref, (s[0] + s[1]) + (s[2] + s[3]));
        if (kKeep) {
#pragma unroll
            for (int c = 0; c < kMmHalf; c += 64) {
                if (c >= T.cols) break;
                staging_free(stored, T.lane);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float *e = S.z + c + 8 * i;
                    sts128(T.st + sw128(T.lane, i), make_uint4(pack_h2(e[0], e[1]), pack_h2(e[2], e[3]),
                                                               pack_h2(e[4], e[5]), pack_h2(e[6], e[7])));
                }
                fence_proxy_async();
                __syncwarp();
                if (T.lane == 0) tma_store_2d(&E.mE, T.col0 + c, T.row0, T.st);
            }
        }
    }
};

// ---- few rows: the logits of one k range, transposed ([V][M]: the vocabulary is the 256-wide side of the tiles, the few
// rows their columns), float32, for few_kernel to add up
struct FewEpi {
    static constexpr bool kManyRegs = false;
    struct Params {
        CUtensorMap mD;            // float32 [ranges][V][Mp]
    };
    struct State {
        float z[kMmHalf / 2];
    };
    static __device__ __forceinline__ void begin(const Params &, const MmProb &, const MmUnit &, const MmTileCtx &, State &)
    {
    }
    static __device__ __forceinline__ void take(const Params &, const MmProb &, const MmUnit &, const MmTileCtx &T,
                                                State &S, bool first, bool, bool &)
    {
#pragma unroll
        for (int c = 0; c < kMmHalf / 2; c += 32) {
            if (c >= T.cols) continue;
            uint32_t v[32];
            tmem_ld32(T.tmem + c, v);
#pragma unroll
            for (int i = 0; i < 32; ++i) S.z[c + i] = first ? __uint_as_float(v[i]) : S.z[c + i] + __uint_as_float(v[i]);
        }
    }
    static __device__ __forceinline__ void end(const Params &E, const MmProb &, const MmUnit &U, const MmTileCtx &T,
                                               State &S, bool &stored)
    {
#pragma unroll
        for (int c = 0; c < kMmHalf / 2; c += 32) {
            if (c >= T.cols) continue;
            staging_free(stored, T.lane);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float *z = S.z + c + 4 * i;
                sts128(T.st + sw128(T.lane, i), make_uint4(__float_as_uint(z[0]), __float_as_uint(z[1]),
                                                           __float_as_uint(z[2]), __float_as_uint(z[3])));
            }
            fence_proxy_async();
            __syncwarp();
            if (T.lane == 0) tma_store_3d(&E.mD, T.col0 + c, T.row0, U.split, T.st);
        }
    }
};

// ---- lse (base 2) of a row from its tiles' statistics, by a group of kThreads threads (a warp, or a block)
__device__ __forceinline__ float2 lse_merge(float2 a, float2 b)
{
    // (m, s): sum of s 2^m.  NaN in either sum stays; an empty side (-inf, 0) adds nothing.
    const float m = fmaxf(a.x, b.x);
    if (m == -INFINITY) return make_float2(m, a.y + b.y);
    return make_float2(m, a.y * ex2(a.x - m) + b.y * ex2(b.x - m));
}

__device__ __forceinline__ float2 lse_warp(float2 a)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float2 b = make_float2(__shfl_xor_sync(0xffffffffu, a.x, o), __shfl_xor_sync(0xffffffffu, a.y, o));
        a = lse_merge(a, b);
    }
    return a;
}

// Few rows: statistics of 64 vocabulary entries for every row, from the ranges' logits, added in order.  A lane has a row
// and eight entries (with 16 rows or fewer the other lanes of the warp share them), all their loads in flight at once.
constexpr int kFewEntries = 64;
__global__ void __launch_bounds__(256) few_kernel(const float *__restrict__ part, int ranges, int M, int V, int Mp,
                                                  int row_lanes, const int64_t *__restrict__ labels,
                                                  float2 *__restrict__ stat, float *__restrict__ target)
{
    __shared__ float2 all[8][32];
    pdl_go();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane / row_lanes, subs = 32 / row_lanes;   // which of the lanes that share a row's entries
    const int v0 = blockIdx.x * kFewEntries + warp * 8;
    const size_t step = (size_t)V * Mp;
    for (int m0 = 0; m0 < M; m0 += row_lanes) {
        const int m = m0 + lane % row_lanes;
        float z[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = -INFINITY;
        if (m < M) {
            const float *p = part + (size_t)v0 * Mp + m;
            for (int r = 0; r < ranges; ++r, p += step)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i % subs == sub && v0 + i < V) z[i] = r ? z[i] + p[i * Mp] : p[i * Mp];
            const long long lab = labels[m] - v0;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (lab == i && i % subs == sub && v0 + i < V) target[m] = z[i];
        }
        float top = z[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) top = fmaxf(top, z[i]);
        const float ref = top * kLog2e, from = top == -INFINITY ? 0.0f : ref;
        float2 s = make_float2(ref, 0.0f);
#pragma unroll
        for (int i = 0; i < 8; ++i) s.y += ex2(fmaf(z[i], kLog2e, -from));
        for (int o = row_lanes; o < 32; o <<= 1)
            s = lse_merge(s, make_float2(__shfl_xor_sync(0xffffffffu, s.x, o), __shfl_xor_sync(0xffffffffu, s.y, o)));
        all[warp][lane] = s;
        __syncthreads();
        if (warp == 0 && sub == 0 && m < M) {
            for (int i = 1; i < 8; ++i) s = lse_merge(s, all[i][lane]);
            stat[(size_t)m * gridDim.x + blockIdx.x] = s;
        }
        __syncthreads();
    }
}

__global__ void __launch_bounds__(256) lse_kernel(const float2 *__restrict__ stat, const float *__restrict__ target,
                                                  const int64_t *__restrict__ labels, int M, int V, int nst,
                                                  float *__restrict__ loss, float *__restrict__ lse)
{
    const int lane = threadIdx.x & 31, row = blockIdx.x * 8 + (threadIdx.x >> 5);
    pdl_wait();
    if (row >= M) return;
    float2 a = make_float2(-INFINITY, 0.0f);
    for (int t = lane; t < nst; t += 32) a = lse_merge(a, stat[(size_t)row * nst + t]);
    a = lse_warp(a);
    if (lane == 0) {
        const long long lab = labels[row];
        const float l = (a.x + log2f(a.y)) * kLn2;
        lse[row] = l;
        loss[row] = lab >= 0 && lab < V ? l - target[row] : 0.0f;
    }
}

// The largest finite |weight| of a row that counts (1 if there is none): G is held relative to it, so that with equal
// weights, a mean, the entries of G are p and p - 1 themselves.  Where p is small the one that dominates a row is then
// rounded by p at most, to -1, while w (p - 1) could be off by 2^-8 of itself, the same way in every row.  From p = 1e-3 on
// p - 1 is off by up to 2^-9 all the same, differently from row to row: dH makes up for that (ProductEpi); in dW the rows
// would have to be brought together by label, and what they leave stays below the rounding of the result (1.90e-3 of the
// norm with it, 1.66e-3 without, at 4096 rows, D 4096, V 32000).
__global__ void __launch_bounds__(1024) wref_kernel(const float *__restrict__ weight, const int64_t *__restrict__ labels,
                                                    int M, int V, float *__restrict__ wref)
{
    float m = 0.0f;
#pragma unroll 4
    for (int i = threadIdx.x; i < M; i += 1024) {
        const float w = fabsf(weight[i]);
        const long long lab = labels[i];
        if (lab >= 0 && lab < V && w < INFINITY) m = fmaxf(m, w);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    __shared__ float part[32];
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x < 32) {
        m = part[threadIdx.x];
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (threadIdx.x == 0) *wref = m > 0.0f ? m : 1.0f;
    }
}

// ---- 2: G over e, the loss, and (Hc) H with the rows that do not count zeroed, the operand of dW
__global__ void __launch_bounds__(256) grad_kernel(uint4 *__restrict__ E, const float2 *__restrict__ stat,
                                                   const float *__restrict__ target,
                                                   const int64_t *__restrict__ labels,
                                                   const float *__restrict__ weight,
                                                   const float *__restrict__ wref, int V, int Vp, int nst, int D,
                                                   const uint4 *__restrict__ H, uint4 *__restrict__ Hc,
                                                   float *__restrict__ loss, float *__restrict__ rest, int cols)
{
    const int row = blockIdx.y, chunk = blockIdx.x;
    pdl_go();
    pdl_wait();
    const long long lab = labels[row];
    const bool counts = lab >= 0 && lab < V;
    if (chunk == 0 && Hc) {
        const int nv = D / 8;
        const size_t base = (size_t)row * nv;
        for (int i = threadIdx.x; i < nv; i += 256) Hc[base + i] = counts ? H[base + i] : make_uint4(0, 0, 0, 0);
    }
    const int v0 = chunk * (cols / 8), v1 = min(Vp / 8, v0 + cols / 8);   // vectors of 8 entries
    uint4 *out = E + (size_t)row * (Vp / 8);
    if (!counts) {
        for (int i = v0 + threadIdx.x; i < v1; i += 256) out[i] = make_uint4(0, 0, 0, 0);
        if (chunk == 0 && threadIdx.x == 0) loss[row] = rest[row] = 0.0f;
        return;
    }
    const float2 *st = stat + (size_t)row * nst;
    float2 a = make_float2(-INFINITY, 0.0f);
    for (int t = threadIdx.x; t < nst; t += 256) a = lse_merge(a, st[t]);
    a = lse_warp(a);
    __shared__ float2 part[8];
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = a;
    __syncthreads();
    a = lse_warp(part[threadIdx.x & 7]);   // every warp: the eight parts, four times over
    a.y *= 0.25f;
    const float lse2 = a.x + log2f(a.y);
    const float w = weight[row] / *wref, z = target[row];
    if (chunk == 0 && threadIdx.x == 0) loss[row] = lse2 * kLn2 - z;
    // the label's entry from the float32 logit: p - 1 of a sure row is far below the rounding of p
    const float at_label = w * (ex2(fmaf(z, kLog2e, -lse2)) - 1.0f);
#pragma unroll 4
    for (int i = v0 + threadIdx.x; i < v1; i += 256) {
        const uint4 q = out[i];
        const float f = w * ex2(st[i >> 4].x - lse2);   // 16 vectors to 128 entries
        const uint32_t in[4] = {q.x, q.y, q.z, q.w};
        float g[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 e = __half22float2(*reinterpret_cast<const __half2 *>(&in[j]));
            g[2 * j] = e.x * f;
            g[2 * j + 1] = e.y * f;
        }
        if (lab >> 3 == i) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if ((lab & 7) == j) g[j] = at_label;
            rest[row] = at_label - __uint_as_float(pack_bf2(0.0f, at_label));   // the upper half is the rounded entry
        }
        out[i] = make_uint4(pack_bf2(g[0], g[1]), pack_bf2(g[2], g[3]), pack_bf2(g[4], g[5]), pack_bf2(g[6], g[7]));
    }
}

// ---- 3: the two products
// Their sums run over the whole vocabulary (dH) or all rows of a piece (dW): pieces of an accumulator, as for the logits,
// are added in registers.  (One accumulator over 131,072 entries of one sign came out up to 1e-3 low.)
enum { kOutBf16 = 0, kOutF32 = 1, kOutF32Add = 2 };
struct ProductEpi {
    static constexpr bool kManyRegs = true;
    struct Params {
        CUtensorMap mD[2];
        int kind[2];
        int split_rows[2];   // rows between the partial results of consecutive k ranges
        const float *wref;
        // What the rounding of G left of each row's label entry, up to 2^-9: by itself more than the other entries' roundings
        // together where none of them is large, and a multiple of W[label] in dH's row, so it is made up for there:
        // dH += rest W[label] (1.91e-3 -> 1.66e-3 of the norm, which is the rounding of the result, at 4096 rows, D 4096,
        // V 32000).  This takes 2 to 5 us of a call of few rows (205 -> 208 us at 1 row, D 4096, V 32000), and about 1 % of
        // larger ones together with the pieces.
        const float *rest;
        const int64_t *labels;
        const uint16_t *W;
        int M, D;
    };
    struct State {
        float a[kMmHalf];
    };
    static __device__ __forceinline__ void begin(const Params &, const MmProb &, const MmUnit &, const MmTileCtx &, State &S)
    {
#pragma unroll
        for (int i = 0; i < kMmHalf; ++i) S.a[i] = 0.0f;
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
    static __device__ __forceinline__ void end(const Params &E, const MmProb &, const MmUnit &U, const MmTileCtx &T,
                                               State &S, bool &stored)
    {
        const int kind = E.kind[U.q], y = T.row0 + U.split * E.split_rows[U.q];
        const CUtensorMap *map = &E.mD[U.q];
        const int row = T.row0 + T.lane;
        if (U.q == 0 && U.split == 0 && T.cols > 0 && row < E.M) {
            const float r = E.rest[row];
            if (r != 0.0f) {   // a row that counts
                const uint4 *w = reinterpret_cast<const uint4 *>(E.W + E.labels[row] * E.D + T.col0);
#pragma unroll
                for (int c = 0; c < kMmHalf; c += 32) {
                    uint4 q[4];   // four reads in flight
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        q[j] = c + 8 * j < T.cols ? __ldg(w + c / 8 + j) : make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t h[4] = {q[j].x, q[j].y, q[j].z, q[j].w};
                        float *const a = S.a + c + 8 * j;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            a[2 * i] = fmaf(r, __uint_as_float(h[i] << 16), a[2 * i]);
                            a[2 * i + 1] = fmaf(r, __uint_as_float(h[i] & 0xffff0000u), a[2 * i + 1]);
                        }
                    }
                }
            }
        }
        if (kind == kOutBf16) {
            const float f = *E.wref;
#pragma unroll
            for (int c = 0; c < kMmHalf; c += 64) {
                if (c >= T.cols) break;
                staging_free(stored, T.lane);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float *a = S.a + c + 8 * i;
                    sts128(T.st + sw128(T.lane, i), make_uint4(pack_bf2(a[0] * f, a[1] * f), pack_bf2(a[2] * f, a[3] * f),
                                                               pack_bf2(a[4] * f, a[5] * f), pack_bf2(a[6] * f, a[7] * f)));
                }
                fence_proxy_async();
                __syncwarp();
                if (T.lane == 0) tma_store_2d(map, T.col0 + c, y, T.st);
            }
            return;
        }
#pragma unroll
        for (int c = 0; c < kMmHalf; c += 32) {
            if (c >= T.cols) break;
            staging_free(stored, T.lane);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float *a = S.a + c + 4 * i;
                sts128(T.st + sw128(T.lane, i), make_uint4(__float_as_uint(a[0]), __float_as_uint(a[1]),
                                                           __float_as_uint(a[2]), __float_as_uint(a[3])));
            }
            fence_proxy_async();
            __syncwarp();
            if (T.lane == 0) {
                if (kind == kOutF32) tma_store_2d(map, T.col0 + c, y, T.st);
                else tma_add_2d(map, T.col0 + c, y, T.st);
            }
        }
    }
};

// out = bfloat16(*wref * sum of n fp32 parts `stride` elements apart), in order; 8 elements a thread
__global__ void __launch_bounds__(256) round_sum_kernel(const float4 *__restrict__ part, size_t stride4, int n,
                                                        size_t nvec, const float *__restrict__ wref,
                                                        uint4 *__restrict__ out)
{
    pdl_wait();
    const float f = *wref;
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < nvec; i += (size_t)gridDim.x * 256) {
        float4 a = part[2 * i], b = part[2 * i + 1];
        for (int s = 1; s < n; ++s) {
            const float4 c = part[s * stride4 + 2 * i], d = part[s * stride4 + 2 * i + 1];
            a.x += c.x, a.y += c.y, a.z += c.z, a.w += c.w;
            b.x += d.x, b.y += d.y, b.z += d.z, b.w += d.w;
        }
        out[i] = make_uint4(pack_bf2(a.x * f, a.y * f), pack_bf2(a.z * f, a.w * f), pack_bf2(b.x * f, b.y * f),
                            pack_bf2(b.z * f, b.w * f));
    }
}

// ---- host
size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }

// What a unit of the two products costs, in 64-deep k blocks of a pair (0.27 us): its k blocks, but at least its epilogue,
// 2.4 us for 256 x 256 outputs, which is all there is where few rows are contracted into dW.
constexpr long kEpilogueBlocks = 9;
long unit_cost(long kb) { return std::max(kb, kEpilogueBlocks); }

// K ranges of dH: k is the whole vocabulary, so a few rows give few, long tiles.  The time of `s` ranges in 64-deep k
// blocks of a pair: the launch's longest chain, plus the write and read of the fp32 partial results at the copy rate
// (1.8 MB in that time), which one range does not need.  With M = 777, D = 1160, V = 32003 (20 tiles of 501 k blocks, 7
// ranges) the product takes 62 us and the adding 7; whole, a chain of 501 k blocks alone would be 135.
int dh_splits(int M, int D, int V, bool with_dW, int pairs)
{
    const long tiles = (long)((M + kMmTile - 1) / kMmTile) * ((D + kMmTile - 1) / kMmTile);
    const long nkb = ((long)V + kMmBK - 1) / kMmBK;
    const long dw_len = unit_cost((M + kMmBK - 1) / kMmBK);
    const double dw = with_dW ? (double)((V + kMmTile - 1) / kMmTile) * ((D + kMmTile - 1) / kMmTile) * dw_len : 0.0;
    int best = 1;
    double best_cost = 1e300;
    for (int s = 1; s <= 16 && s <= nkb; ++s) {
        const long len = (nkb + s - 1) / s, units = tiles * s;
        const double chain = (double)((units + pairs - 1) / pairs) * len;
        const double even = ((double)units * len + dw) / pairs + (with_dW ? dw_len : 0);
        const double cost = std::max(chain, even) + (s > 1 ? 8.0 + (double)s * M * D * 8.0 / 1.8e6 : 0.0);
        if (cost < best_cost) {
            best_cost = cost;
            best = s;
        }
    }
    return best;
}

// A forward pass of at most 128 rows is bound by reading W.  With the rows as the 256-wide side of the tiles the tensor
// cores multiply mostly zeros, and take longer than the reading (118 us at M = 16, D = 8192, V = 32000); so W is that
// side, and the rows are the columns (as few as 32): 101 us.  Its tiles (256 vocabulary entries) divide badly, 125 on 74
// pairs take as long as 148, which cutting k into ranges evens out; the ranges' logits have to be written, read and added.
// In bytes a pair waits for: the longest list of units, and its share of the logits.
int few_ranges(int M, int D, int V)
{
    if (M > kMmHalf) return 0;
    const long pairs = 74, tiles = ((long)V + kMmTile - 1) / kMmTile, nkb = ((long)D + kMmBK - 1) / kMmBK;
    long best = 1;
    double best_cost = 0.0;
    for (long s = 1; s <= 16 && s <= nkb; ++s) {
        const double rounds = (double)((tiles * s + pairs - 1) / pairs);
        const double unit = (double)((nkb + s - 1) / s) * kMmBK * kMmTile * 2;
        const double cost = rounds * unit + (double)s * M * V * 8 / pairs;
        if (s == 1 || cost < 0.98 * best_cost) {
            best_cost = cost;
            best = s;
        }
    }
    const long per = (nkb + best - 1) / best;   // as mm_plan cuts
    return (int)((nkb + per - 1) / per);
}

struct LossPlan {
    int rows, npieces, ntn, nst, Vp, splits;
    int ranges, Mp;   // forward pass of few rows: k ranges whose logits are written (0: not few), pitch of the logits
    size_t stat, target, rest, wref, E, Hc, part, acc, bytes;   // workspace offsets
};

// false: sizes that the operators refuse
bool loss_plan(LossPlan &L, int M, int D, int V, bool grad, bool with_dW, int rows)
{
    if (M < 0 || D < 1 || V < 1 || rows < 0 || D % 8 || D > (1 << 20) || V > (1 << 28) || M > (1 << 28)) return false;
    memset(&L, 0, sizeof(L));
    L.rows = std::min(std::max(M, 1), grad ? (rows ? std::min(rows, kRowsMost) : kRowsDefault) : std::max(M, 1));
    L.npieces = M ? (M + L.rows - 1) / L.rows : 0;
    L.ntn = (V + kMmTile - 1) / kMmTile;
    L.nst = (V + kMmHalf - 1) / kMmHalf;
    L.Vp = (V + 63) & ~63;   // rows of e begin on 128-byte lines: 16 bytes off, every store splits its sectors
    const size_t tiles_m = (L.rows + kMmTile - 1) / kMmTile, tiles_d = (D + kMmTile - 1) / kMmTile, tiles_n = L.ntn;
    if (tiles_m * tiles_n > (1u << 28)) return false;   // units of a launch, with its k ranges an int
    size_t at = 0;
    auto take = [&](size_t b) {
        const size_t o = at;
        at = up256(at + b);
        return o;
    };
    if (!grad && (L.ranges = few_ranges(L.rows, D, V)) > 0) L.nst = (V + kFewEntries - 1) / kFewEntries;
    L.stat = take((size_t)L.rows * L.nst * sizeof(float2));
    L.target = take((size_t)L.rows * 4);
    L.rest = take(grad ? (size_t)L.rows * 4 : 0);
    L.wref = take(grad ? 4 : 0);
    if (L.ranges) {
        L.Mp = (L.rows + 3) & ~3;
        L.part = take((size_t)L.ranges * V * L.Mp * 4);
    }
    if (grad) {
        // the plan's pairs: those of the B200's 148 SMs, whatever the current device, so that the size is one number
        L.splits = dh_splits(L.rows, D, V, with_dW, 74);
        if (tiles_n * tiles_d > (1u << 28) || tiles_m * tiles_d * L.splits > (1u << 28)) return false;
        L.E = take((size_t)L.rows * L.Vp * 2);
        const size_t tile_rows = (size_t)((L.rows + kMmTile - 1) / kMmTile) * kMmTile;
        L.part = take(L.splits > 1 ? (size_t)L.splits * tile_rows * D * 4 : 0);
        L.Hc = take(with_dW ? (size_t)L.rows * D * 2 : 0);
        L.acc = take(with_dW && L.npieces > 1 ? (size_t)V * D * 4 : 0);
    }
    L.bytes = at;
    return true;
}

bool misaligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) != 0; }

lb_status few_logits(const LossPlan &L, const uint16_t *H, const uint16_t *W, int M, int D, int V, unsigned char *ws,
                     cudaStream_t s)
{
    MmBatch<1> G;
    FewEpi::Params E;
    memset(&G, 0, sizeof(G));
    const int width = M <= 64 ? 64 : 128;
    G.n = 1;
    mm_plan(G.p[0], V, M, D, true, 0, L.ranges, 1, 1, false, width);
    mm_chunk(G.p[0], kChunk);
    G.nunits = mm_units(G.p[0]);
    if (!mm_operand(&G.mA[0], true, false, W, V, D, D) ||
        !mm_operand(&G.mB[0], true, false, H, M, D, D, 1, width / 2) ||
        !tmap_encode_3d(&E.mD, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, ws + L.part, L.Mp, V, L.ranges, (long)L.Mp * 4,
                        (long)V * L.Mp * 4, 32, 32))
        return LB_ERR_CUDA;
    return status_from(mm_launch<true, 1, FewEpi>(G, E, s));
}

lb_status logits(const LossPlan &L, const uint16_t *H, const uint16_t *W, const int64_t *labels, int M, int D, int V,
                 unsigned char *ws, bool keep, cudaStream_t s)
{
    MmBatch<1> G;
    memset(&G, 0, sizeof(G));
    G.n = 1;
    mm_plan(G.p[0], M, V, D, true, 0, 1);
    mm_chunk(G.p[0], kChunk);
    G.nunits = mm_units(G.p[0]);
    if (!mm_operand(&G.mA[0], true, false, H, M, D, D) || !mm_operand(&G.mB[0], true, false, W, V, D, D))
        return LB_ERR_CUDA;
    auto fill = [&](auto &E) {
        memset(&E, 0, sizeof(E));
        E.labels = labels;
        E.stat = (float2 *)(ws + L.stat);
        E.target = (float *)(ws + L.target);
        E.M = M;
        E.V = V;
        E.nst = L.nst;
    };
    if (keep) {
        LogitEpi<true>::Params E;
        fill(E);
        if (!tmap_encode_2d(&E.mE, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, ws + L.E, L.Vp, M, (long)L.Vp * 2, 64, 32))
            return LB_ERR_CUDA;
        return status_from(mm_launch<true, 1, LogitEpi<true>>(G, E, s));
    }
    LogitEpi<false>::Params E;
    fill(E);
    return status_from(mm_launch<true, 1, LogitEpi<false>>(G, E, s));
}

// dH (and dW) of one piece of M rows
lb_status products(const LossPlan &L, const uint16_t *W, const int64_t *labels, int M, int D, int V, uint16_t *dH,
                   uint16_t *dW, bool first, unsigned char *ws, cudaStream_t s, int *launches)
{
    MmBatch<2> G;
    ProductEpi::Params E;
    memset(&G, 0, sizeof(G));
    memset(&E, 0, sizeof(E));
    const void *Gm = ws + L.E;
    E.wref = (const float *)(ws + L.wref);
    E.rest = (const float *)(ws + L.rest);
    E.labels = labels;
    E.W = W;
    E.M = M;
    E.D = D;
    MmProb &P = G.p[0];
    mm_plan(P, M, D, V, true, 0, L.splits);
    mm_chunk(P, kChunk);
    P.b_mn = 1;
    if (!mm_operand(&G.mA[0], true, false, Gm, M, L.Vp, L.Vp) || !mm_operand(&G.mB[0], true, true, W, V, D, D))
        return LB_ERR_CUDA;
    const int tile_rows = P.ntm * kMmTile;
    bool ok;
    if (P.splits > 1) {
        E.kind[0] = kOutF32;
        E.split_rows[0] = tile_rows;
        ok = tmap_encode_2d(&E.mD[0], CU_TENSOR_MAP_DATA_TYPE_FLOAT32, ws + L.part, D, (long)tile_rows * P.splits,
                            (long)D * 4, 32, 32);
    } else {
        E.kind[0] = kOutBf16;
        ok = tmap_encode_2d(&E.mD[0], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dH, D, M, (long)D * 2, 64, 32);
    }
    if (!ok) return LB_ERR_CUDA;
    G.n = 1;
    G.nunits = mm_units(P);
    if (dW) {
        MmProb &Q = G.p[1];
        mm_plan(Q, V, D, M, false, G.nunits, 1);
        mm_chunk(Q, kChunk);
        Q.a_mn = Q.b_mn = 1;
        if (!mm_operand(&G.mA[1], true, true, Gm, M, L.Vp, L.Vp) || !mm_operand(&G.mB[1], true, true, ws + L.Hc, M, D, D))
            return LB_ERR_CUDA;
        if (L.npieces > 1) {
            E.kind[1] = first ? kOutF32 : kOutF32Add;
            ok = tmap_encode_2d(&E.mD[1], CU_TENSOR_MAP_DATA_TYPE_FLOAT32, ws + L.acc, D, V, (long)D * 4, 32, 32);
        } else {
            E.kind[1] = kOutBf16;
            ok = tmap_encode_2d(&E.mD[1], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dW, D, V, (long)D * 2, 64, 32);
        }
        if (!ok) return LB_ERR_CUDA;
        int pairs = 0;
        const cudaError_t e = mm_pairs(&pairs);
        if (e != cudaSuccess) return status_from(e);
        const int n1 = mm_units(Q), more = G.nunits % pairs;
        const long c0 = unit_cost(P.kb_per), c1 = unit_cost(Q.kb_per);
        if (more) G.extra = (int)std::min<long>((c0 + c1 / 2) / c1, n1 / (pairs - more));
        G.n = 2;
        G.nunits += n1;
        if (pairs > G.nunits) G.extra = 0;   // fewer pairs are launched than the rule above counted with
    }
    const cudaError_t e = mm_launch<true, 2, ProductEpi>(G, E, s);
    if (e != cudaSuccess) return status_from(e);
    ++*launches;
    if (P.splits > 1) {
        const size_t nvec = (size_t)M * D / 8;
        const int grid = (int)std::min<size_t>((nvec + 255) / 256, 148 * 8);
        const cudaError_t r = launch_after(round_sum_kernel, dim3(grid), 256, s, (const float4 *)(ws + L.part),
                                           (size_t)tile_rows * D / 4, P.splits, nvec, E.wref, (uint4 *)dH);
        if (r != cudaSuccess) return status_from(r);
        ++*launches;
    }
    return status_from(cudaGetLastError());
}

}  // namespace

lb_status orth_status(cudaStream_t s);

}  // namespace lb

using namespace lb;

extern "C" size_t lb_cross_entropy_forward_workspace_bytes(int M, int D, int V)
{
    LossPlan L;
    return loss_plan(L, M, D, V, false, false, 0) ? L.bytes : 0;
}

extern "C" size_t lb_cross_entropy_gradient_workspace_bytes(int M, int D, int V, int with_dW, int rows)
{
    LossPlan L;
    return loss_plan(L, M, D, V, true, with_dW != 0, rows) ? L.bytes : 0;
}

extern "C" lb_status lb_cross_entropy_forward(const uint16_t *H, const uint16_t *W, const int64_t *labels, int M, int D,
                                              int V, float *loss, float *lse, void *workspace, size_t workspace_bytes,
                                              void *stream)
{
    set_launch_count(0);
    LossPlan L;
    if (M < 0 || D < 1 || V < 1) return LB_ERR_INVALID_ARG;
    if (!loss_plan(L, M, D, V, false, false, 0)) return LB_ERR_UNSUPPORTED;
    if (M == 0) return LB_OK;
    if (!H || !W || !labels || !loss || !lse || !workspace) return LB_ERR_INVALID_ARG;
    if (misaligned(H, 16) || misaligned(W, 16) || misaligned(labels, 8) || misaligned(loss, 4) || misaligned(lse, 4) ||
        misaligned(workspace, 256) || workspace_bytes < L.bytes)
        return LB_ERR_INVALID_ARG;
    if (tmap_encoder_ready() != cudaSuccess) return LB_ERR_UNSUPPORTED;
    unsigned char *ws = (unsigned char *)workspace;
    cudaStream_t s = (cudaStream_t)stream;
    const lb_status st = L.ranges ? few_logits(L, H, W, M, D, V, ws, s) : logits(L, H, W, labels, M, D, V, ws, false, s);
    if (st != LB_OK) return st;
    cudaError_t e;
    if (L.ranges) {
        int row_lanes = 4;
        while (row_lanes < 32 && row_lanes < M) row_lanes <<= 1;
        e = launch_after(few_kernel, dim3(L.nst), 256, s, (const float *)(ws + L.part), L.ranges, M, V, L.Mp, row_lanes,
                         labels, (float2 *)(ws + L.stat), (float *)(ws + L.target));
        if (e != cudaSuccess) return status_from(e);
    }
    e = launch_after(lse_kernel, dim3((M + 7) / 8), 256, s, (const float2 *)(ws + L.stat), (const float *)(ws + L.target),
                     labels, M, V, L.nst, loss, lse);
    set_launch_count(L.ranges ? 3 : 2);
    return status_from(e);
}

extern "C" lb_status lb_cross_entropy_gradient(const uint16_t *H, const uint16_t *W, const int64_t *labels,
                                               const float *weight, int M, int D, int V, int rows, float *loss,
                                               uint16_t *dH, uint16_t *dW, void *workspace, size_t workspace_bytes,
                                               void *stream)
{
    set_launch_count(0);
    LossPlan L;
    if (M < 0 || D < 1 || V < 1 || rows < 0) return LB_ERR_INVALID_ARG;
    if (!loss_plan(L, M, D, V, true, dW != nullptr, rows)) return LB_ERR_UNSUPPORTED;
    if (misaligned(dW, 16)) return LB_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    if (M == 0) {   // no rows: the gradient of W is zero
        if (!dW) return LB_OK;
        return status_from(cudaMemsetAsync(dW, 0, (size_t)V * D * 2, s));
    }
    if (!H || !W || !labels || !weight || !loss || !dH || !workspace) return LB_ERR_INVALID_ARG;
    if (misaligned(H, 16) || misaligned(W, 16) || misaligned(labels, 8) || misaligned(weight, 4) ||
        misaligned(loss, 4) || misaligned(dH, 16) || misaligned(workspace, 256) || workspace_bytes < L.bytes)
        return LB_ERR_INVALID_ARG;
    if (tmap_encoder_ready() != cudaSuccess) return LB_ERR_UNSUPPORTED;
    unsigned char *ws = (unsigned char *)workspace;
    int launches = 1;
    wref_kernel<<<1, 1024, 0, s>>>(weight, labels, M, V, (float *)(ws + L.wref));
    for (int p = 0; p < L.npieces; ++p) {
        const int r0 = p * L.rows, m = std::min(L.rows, M - r0);
        const uint16_t *Hp = H + (size_t)r0 * D;
        lb_status st = logits(L, Hp, W, labels + r0, m, D, V, ws, true, s);
        if (st != LB_OK) return st;
        // every block adds up its row's statistics first: as long a part of the row as leaves the GPU full of blocks
        int cols = kGradCols;
        while (cols < 4 * kGradCols && (long)m * ((L.Vp + 2 * cols - 1) / (2 * cols)) >= 148 * 8) cols *= 2;
        const dim3 grid((L.Vp + cols - 1) / cols, m);
        cudaError_t e = launch_after(grad_kernel, grid, 256, s, (uint4 *)(ws + L.E), (const float2 *)(ws + L.stat),
                                         (const float *)(ws + L.target), labels + r0, weight + r0,
                                         (const float *)(ws + L.wref), V, L.Vp, L.nst, D,
                                         (const uint4 *)Hp, dW ? (uint4 *)(ws + L.Hc) : nullptr, loss + r0,
                                         (float *)(ws + L.rest), cols);
        if (e != cudaSuccess) return status_from(e);
        launches += 2;
        st = products(L, W, labels + r0, m, D, V, dH + (size_t)r0 * D, dW, p == 0, ws, s, &launches);
        if (st != LB_OK) return st;
    }
    if (dW && L.npieces > 1) {
        const size_t nvec = (size_t)V * D / 8;
        const int grid = (int)std::min<size_t>((nvec + 255) / 256, 148 * 8);
        const cudaError_t e = launch_after(round_sum_kernel, dim3(grid), 256, s, (const float4 *)(ws + L.acc), 0, 1, nvec,
                                           (const float *)(ws + L.wref), (uint4 *)dW);
        if (e != cudaSuccess) return status_from(e);
        ++launches;
    }
    set_launch_count(launches);
    return status_from(cudaGetLastError());
}

extern "C" lb_status lb_train_status(void *stream)
{
    const lb_status a = mm_status((cudaStream_t)stream), b = orth_status((cudaStream_t)stream);
    return a != LB_OK ? a : b;
}
