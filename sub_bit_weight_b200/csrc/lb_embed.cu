// Token embedding: lookup with scaling, and its gradient by sorted tokens.
//
//     out[m] = scale * table[id_m]             dtable[v] = scale * sum over m with id_m = v of dout[m]
//
// Both are bound by memory.  The lookup reads the rows it names and writes M D
// elements.  The gradient reads M D elements and writes all V D (rows without
// a token are zero), in a fixed order of additions:
//
//   1  every (id, position) pair's place among the sorted pairs is the number
//      of smaller ones, counted directly against up to 16,384 ids in shared
//      memory (the pairs are distinct, so the order is unique): 8192^2
//      comparisons are 4 us for the whole GPU and need no exchange between
//      blocks, where a sort in one block took 20 us.  The same blocks write the
//      zeros of the rows that no token names, most of the output in a real
//      vocabulary;
//   2  (more than 16,384 tokens) every pair finds its place among the other
//      chunks' sorted runs;
//   3  a block takes 8 or 32 consecutive pairs and 256 vectors of columns, adds
//      the rows of each token in float32 and writes the tokens that lie inside
//      its pairs; a token that crosses into other blocks (a frequent one)
//      leaves float32 partial sums there;
//   4  the partial sums of each crossing token are added in order.

#include <algorithm>
#include <cstring>

#include "lb_internal.cuh"
#include "littlebit_train.h"

namespace lb {
namespace {

constexpr int kSortMost = 16384;    // ids of a chunk (64 KB of shared memory)
constexpr int kZeroRows = 4096;     // rows a block looks after at a time
constexpr int kOrderThreads = 512;  // of a block's 1024 threads, those that count while the others write zeros

template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
    T v[N];
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x)
{
    return x;
}
template <>
__device__ __forceinline__ uint16_t from_f<uint16_t>(float x)
{
    uint16_t r;
    asm("cvt.rn.bf16.f32 %0, %1;\n" : "=h"(r) : "f"(x));
    return r;
}

// ---- lookup: one row per blockIdx.x, up to 4 vectors a thread in flight
template <typename TI, typename TO, int N>
__global__ void __launch_bounds__(256) lookup_kernel(const int64_t *__restrict__ ids, const TI *__restrict__ table,
                                                     long long V, int D, float scale, TO *__restrict__ out)
{
    const long long id = ids[blockIdx.x];
    const bool ok = id >= 0 && id < V;
    const int nv = D / N;
    const Vec<TI, N> *src = reinterpret_cast<const Vec<TI, N> *>(table + (ok ? id : 0) * (long long)D);
    Vec<TO, N> *dst = reinterpret_cast<Vec<TO, N> *>(out + (long long)blockIdx.x * D);
    const int c0 = blockIdx.y * 1024 + threadIdx.x;
    Vec<TI, N> x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (ok && c0 + 256 * j < nv) x[j] = src[c0 + 256 * j];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (c0 + 256 * j >= nv) break;
        Vec<TO, N> y;
#pragma unroll
        for (int i = 0; i < N; ++i) y.v[i] = ok ? from_f<TO>(to_f(x[j].v[i]) * scale) : from_f<TO>(0.0f);
        dst[c0 + 256 * j] = y;
    }
}

// ---- 1: order, and zeros of the rows without a token
// Pairs are (id << 32 | position); an id outside 0 .. V-1 sorts behind every other, as V.
// `split` threads count for one pair, each a share of the chunk's ids.
__global__ void __launch_bounds__(1024) order_zero_kernel(const int64_t *__restrict__ ids, long long M, int V,
                                                          size_t row_bytes, int nchunks, int chunk, int split,
                                                          unsigned long long *__restrict__ pairs,
                                                          unsigned char *__restrict__ out)
{
    extern __shared__ __align__(16) unsigned char e_raw[];
    uint32_t *const k = reinterpret_cast<uint32_t *>(e_raw);
    unsigned char *const seen = e_raw + ((chunk + 3) & ~3) * 4;
    const int tid = threadIdx.x;
    const int per = (int)(((long long)V + gridDim.x - 1) / gridDim.x);
    const long long r0 = (long long)blockIdx.x * per, r1 = min((long long)V, r0 + per);   // rows of this block
    const int first = (int)min((long long)kZeroRows, max(0LL, r1 - r0));
    // zeros in the rows [v0, v0 + rows) without a token, by the threads t, t + n, ..; `lanes` threads a row
    int lanes = 4;
    while (lanes < 128 && (size_t)lanes * 16 < row_bytes) lanes <<= 1;
    auto zeros = [&](long long v0, int rows, int t, int n) {
        for (int r = t / lanes; r < rows; r += n / lanes) {
            if (seen[r]) continue;
            unsigned char *const dst = out + (v0 + r) * row_bytes;
            // to the first 16-byte boundary and from the last one in elements of 2 bytes
            const size_t head = min((size_t)(-(uintptr_t)dst & 15), row_bytes), body = (row_bytes - head) / 16;
            const size_t l = t & (lanes - 1);
            for (size_t i = l; i < head / 2; i += lanes) reinterpret_cast<uint16_t *>(dst)[i] = 0;
            for (size_t i = l; i < body; i += lanes) reinterpret_cast<uint4 *>(dst + head)[i] = make_uint4(0, 0, 0, 0);
            for (size_t i = head + body * 16 + 2 * l; i < row_bytes; i += 2 * lanes)
                *reinterpret_cast<uint16_t *>(dst + i) = 0;
        }
    };
    pdl_go();
    for (int i = tid; i < first; i += 1024) seen[i] = 0;
    for (int c = 0; c < nchunks; ++c) {
        const long long base = (long long)c * chunk;
        const int n = (int)min((long long)chunk, M - base), n4 = (n + 3) & ~3;
        __syncthreads();
        for (int i = tid; i < n4; i += 1024) {
            long long id = i < n ? ids[base + i] : (long long)V;
            if (id < 0 || id >= V) id = V;
            k[i] = (uint32_t)id;
            if (id >= r0 && id - r0 < first) seen[id - r0] = 1;
        }
        __syncthreads();
        if (tid >= kOrderThreads) {   // the last chunk's flags are complete: write zeros beside the counting
            if (c + 1 == nchunks) zeros(r0, first, tid - kOrderThreads, 1024 - kOrderThreads);
            continue;
        }
        const int groups = kOrderThreads / split, part = tid % split;
        const uint32_t mates = (split == 32 ? ~0u : (1u << split) - 1) << ((tid & 31) - part);   // of one pair
        for (int i = blockIdx.x * groups + tid / split; i < n; i += gridDim.x * groups) {
            const uint32_t id = k[i];   // unsigned: V, and id + 1, may be 2^31 - 1 and one more
            const int at = i >> 2;
            int count = 0;
#pragma unroll 4
            for (int j = part; j < n4 / 4; j += split) {
                const uint4 q = reinterpret_cast<const uint4 *>(k)[j];
                const uint32_t t = id + (j < at ? 1 : 0);   // an equal id at an earlier position is smaller
                if (j != at) {
                    count += (q.x < t) + (q.y < t) + (q.z < t) + (q.w < t);
                } else {
                    const int o = i & 3;
                    count += (q.x < id + (o > 0)) + (q.y < id + (o > 1)) + (q.z < id + (o > 2)) + (q.w < id);
                }
            }
            for (int o = split >> 1; o; o >>= 1) count += __shfl_xor_sync(mates, count, o);
            if (part == 0)
                pairs[base + count] = ((unsigned long long)id << 32) | (uint32_t)(base + i);
        }
    }
    if (nchunks == 0) {
        __syncthreads();
        zeros(r0, first, tid, 1024);
    }
    for (long long v0 = r0 + kZeroRows; v0 < r1; v0 += kZeroRows) {   // more rows than one set of flags
        const int rows = (int)min((long long)kZeroRows, r1 - v0);
        __syncthreads();
        for (int i = tid; i < rows; i += 1024) seen[i] = 0;
        __syncthreads();
        for (long long i = tid; i < M; i += 1024) {
            const long long r = ids[i] - v0;
            if (r >= 0 && r < rows) seen[r] = 1;
        }
        __syncthreads();
        zeros(v0, rows, tid, 1024);
    }
}

// ---- 2: place of every pair in the union of the sorted chunks
__global__ void __launch_bounds__(256) merge_kernel(const unsigned long long *__restrict__ in, long long M, int nsort,
                                                    int chunk, unsigned long long *__restrict__ out)
{
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    pdl_go();
    pdl_wait();
    if (i >= M) return;
    const unsigned long long key = in[i];
    const int own = (int)(i / chunk);
    long long at = i - (long long)own * chunk;
    for (int c = 0; c < nsort; ++c) {
        if (c == own) continue;
        const unsigned long long *p = in + (long long)c * chunk;
        int lo = 0, hi = (int)min((long long)chunk, M - (long long)c * chunk);
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (p[mid] < key) lo = mid + 1;
            else hi = mid;
        }
        at += lo;
    }
    out[at] = key;
}

// ---- 3: sums of kPairs pairs.  A token whose pairs begin before or end after this block's leaves its sum in part[2 b]
// (it began before; also a token that fills the block) or part[2 b + 1] (it begins here and goes on).
template <typename TI, typename TO, int N, int kPairs>
__global__ void __launch_bounds__(256) sum_kernel(const unsigned long long *__restrict__ pairs, long long M, int V, int D,
                                                  const TI *__restrict__ dout, float scale, TO *__restrict__ out,
                                                  float *__restrict__ part)
{
    __shared__ unsigned long long k[kPairs + 2];   // the pair before, kPairs, the pair after (~0 where there is none)
    const long long base = (long long)blockIdx.x * kPairs;
    const int n = (int)min((long long)kPairs, M - base);
    pdl_go();
    pdl_wait();
    if (threadIdx.x < kPairs + 2) {
        const long long i = base + (int)threadIdx.x - 1;
        k[threadIdx.x] = i >= 0 && i < M && (int)threadIdx.x <= n + 1 ? pairs[i] : ~0ull;
    }
    __syncthreads();
    const int c = blockIdx.y * 256 + threadIdx.x;
    if (c >= D / N) return;
    float acc[N];
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] = 0.0f;
    int first = 0;   // first pair of the current token in this block
    constexpr int kAhead = 8;
    for (int i0 = 0; i0 < n; i0 += kAhead) {
        Vec<TI, N> x[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (i0 + u < n && (int)(k[i0 + u + 1] >> 32) < V)
                x[u] = reinterpret_cast<const Vec<TI, N> *>(dout + (long long)(uint32_t)k[i0 + u + 1] * D)[c];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = i0 + u;
            if (i >= n) break;
            const uint32_t id = (uint32_t)(k[i + 1] >> 32);
            if ((int)id >= V) return;   // the rest names no row
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] += to_f(x[u].v[j]);
            const bool last = i + 1 == n;
            if (last || (uint32_t)(k[i + 2] >> 32) != id) {
                const bool before = first == 0 && (uint32_t)(k[0] >> 32) == id;
                const bool after = last && (uint32_t)(k[i + 2] >> 32) == id;
                if (before || after) {
                    Vec<float, N> *p = reinterpret_cast<Vec<float, N> *>(
                        part + ((long long)blockIdx.x * 2 + (before ? 0 : 1)) * D);
                    Vec<float, N> y;
#pragma unroll
                    for (int j = 0; j < N; ++j) y.v[j] = acc[j];
                    p[c] = y;
                } else {
                    Vec<TO, N> y;
#pragma unroll
                    for (int j = 0; j < N; ++j) y.v[j] = from_f<TO>(acc[j] * scale);
                    reinterpret_cast<Vec<TO, N> *>(out + (long long)id * D)[c] = y;
                }
#pragma unroll
                for (int j = 0; j < N; ++j) acc[j] = 0.0f;
                first = i + 1;
            }
        }
    }
}

// ---- 4: a token that begins in block b's pairs and goes on past them
template <typename TO, int N, int kPairs>
__global__ void __launch_bounds__(256) join_kernel(const unsigned long long *__restrict__ pairs, long long M, int V, int D,
                                                   const float *__restrict__ part, float scale, TO *__restrict__ out)
{
    pdl_wait();
    const long long b = blockIdx.x, lastp = (b + 1) * kPairs - 1;
    if (lastp + 1 >= M) return;
    const uint32_t id = (uint32_t)(pairs[lastp] >> 32);
    if ((int)id >= V || (uint32_t)(pairs[lastp + 1] >> 32) != id) return;   // nothing goes on
    if (b > 0 && (uint32_t)(pairs[b * kPairs - 1] >> 32) == id) return;     // it began before this block
    // last block that holds a pair of this token: the blocks whose first pair is one follow each other
    long long e = b;
    for (int more = 256; more == 256; e += more) {
        const long long q = e + 1 + threadIdx.x;
        more = __syncthreads_count(q * kPairs < M && (uint32_t)(pairs[q * kPairs] >> 32) == id);
    }
    const int c = blockIdx.y * 256 + threadIdx.x;
    if (c >= D / N) return;
    Vec<float, N> a = reinterpret_cast<const Vec<float, N> *>(part + (2 * b + 1) * D)[c];
#pragma unroll 8
    for (long long q = b + 1; q <= e; ++q) {
        const Vec<float, N> x = reinterpret_cast<const Vec<float, N> *>(part + 2 * q * D)[c];
#pragma unroll
        for (int j = 0; j < N; ++j) a.v[j] += x.v[j];
    }
    Vec<TO, N> y;
#pragma unroll
    for (int j = 0; j < N; ++j) y.v[j] = from_f<TO>(a.v[j] * scale);
    reinterpret_cast<Vec<TO, N> *>(out + (long long)id * D)[c] = y;
}

// ---- host
size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }
size_t size_of(int dt) { return dt == LB_F32 ? 4 : 2; }
bool known(int dt) { return dt == LB_F32 || dt == LB_BF16; }
bool misaligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) != 0; }

// Largest vector (in elements, at most `most`) that divides a row and to which both arrays are aligned.
int vector_of(int D, int most, const void *a, size_t sa, const void *b, size_t sb)
{
    int n = most;
    while (n > 1 && (D % n || misaligned(a, n * sa) || misaligned(b, n * sb))) n >>= 1;
    return n;
}

struct EmbedPlan {
    int nchunks, chunk, per;   // chunks of ids, pairs a block of step 3 takes
    long long nsum;
    size_t pairs, sorted, part, bytes;
};

bool embed_plan(EmbedPlan &L, long long M, int V, int D)
{
    if (M < 0 || V < 1 || D < 1 || M > (1LL << 31) - 1 || D > (1 << 23)) return false;
    const long long c = M ? (M + kSortMost - 1) / kSortMost : 0;
    L.nchunks = (int)c;
    L.chunk = c ? (int)((M + c - 1) / c) : 0;
    // few tokens: more blocks, each with all its rows in flight at once; many: half as many partial sums per row
    L.per = M <= 4096 ? 8 : 32;
    L.nsum = (M + L.per - 1) / L.per;
    size_t at = 0;
    auto take = [&](size_t b) {
        const size_t o = at;
        at = up256(at + b);
        return o;
    };
    L.pairs = take((size_t)M * 8);
    L.sorted = take(L.nchunks > 1 ? (size_t)M * 8 : 0);
    L.part = take((size_t)L.nsum * 2 * D * 4);
    L.bytes = at;
    return true;
}

template <typename TI, typename TO, int N>
cudaError_t launch_lookup(const int64_t *ids, long long M, const void *table, int V, int D, float scale, void *out,
                          cudaStream_t s)
{
    const dim3 grid((unsigned)M, (D / N + 1023) / 1024);
    lookup_kernel<TI, TO, N><<<grid, 256, 0, s>>>(ids, (const TI *)table, V, D, scale, (TO *)out);
    return cudaGetLastError();
}

template <typename TI, typename TO>
cudaError_t lookup(int n, const int64_t *ids, long long M, const void *table, int V, int D, float scale, void *out,
                   cudaStream_t s)
{
    constexpr int kMost = sizeof(TI) == 2 && sizeof(TO) == 2 ? 8 : 4;
    if constexpr (kMost == 8)
        if (n == 8) return launch_lookup<TI, TO, 8>(ids, M, table, V, D, scale, out, s);
    if (n == 4) return launch_lookup<TI, TO, 4>(ids, M, table, V, D, scale, out, s);
    if (n == 2) return launch_lookup<TI, TO, 2>(ids, M, table, V, D, scale, out, s);
    return launch_lookup<TI, TO, 1>(ids, M, table, V, D, scale, out, s);
}

template <typename TI, typename TO, int N, int kPairs>
cudaError_t launch_sums(const EmbedPlan &L, const unsigned long long *pairs, long long M, const void *dout, int V, int D,
                        float scale, void *dtable, float *part, cudaStream_t s)
{
    const dim3 grid((unsigned)L.nsum, (D / N + 255) / 256);
    const cudaError_t e = launch_after(sum_kernel<TI, TO, N, kPairs>, grid, 256, s, pairs, M, V, D, (const TI *)dout, scale,
                                       (TO *)dtable, part);
    if (e != cudaSuccess) return e;
    return launch_after(join_kernel<TO, N, kPairs>, grid, 256, s, pairs, M, V, D, (const float *)part, scale, (TO *)dtable);
}

template <typename TI, typename TO, int N>
cudaError_t launch_grad(const EmbedPlan &L, const int64_t *ids, long long M, const void *dout, int V, int D, float scale,
                        void *dtable, unsigned char *ws, cudaStream_t s, int *launches)
{
    int sms = 0;
    cudaError_t e = sm_count_of_current(&sms);
    if (e != cudaSuccess) return e;
    const int blocks = (int)std::min<long long>(sms, std::max<long long>(V, (M + 31) / 32));
    int split = 1;   // threads per pair: as many as keep every thread busy
    while (split < 32 && (long long)L.chunk * split * 2 <= (long long)blocks * kOrderThreads) split <<= 1;
    const size_t smem = (size_t)((L.chunk + 3) & ~3) * 4 + kZeroRows;
    if ((e = ensure_dyn_smem((const void *)order_zero_kernel, smem)) != cudaSuccess) return e;
    unsigned long long *pairs = (unsigned long long *)(ws + L.pairs);
    order_zero_kernel<<<blocks, 1024, smem, s>>>(ids, M, V, (size_t)D * sizeof(TO), L.nchunks, L.chunk, split, pairs,
                                                 (unsigned char *)dtable);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    ++*launches;
    if (M == 0) return cudaSuccess;
    if (L.nchunks > 1) {
        unsigned long long *sorted = (unsigned long long *)(ws + L.sorted);
        e = launch_after(merge_kernel, dim3((unsigned)((M + 255) / 256)), 256, s, (const unsigned long long *)pairs, M, L.nchunks,
                         L.chunk, sorted);
        if (e != cudaSuccess) return e;
        pairs = sorted;
        ++*launches;
    }
    *launches += 2;
    float *const part = (float *)(ws + L.part);
    return L.per == 8 ? launch_sums<TI, TO, N, 8>(L, pairs, M, dout, V, D, scale, dtable, part, s)
                      : launch_sums<TI, TO, N, 32>(L, pairs, M, dout, V, D, scale, dtable, part, s);
}

template <typename TI, typename TO>
cudaError_t grad(int n, const EmbedPlan &L, const int64_t *ids, long long M, const void *dout, int V, int D, float scale,
                 void *dtable, unsigned char *ws, cudaStream_t s, int *launches)
{
    if constexpr (sizeof(TI) == 2)
        if (n == 8) return launch_grad<TI, TO, 8>(L, ids, M, dout, V, D, scale, dtable, ws, s, launches);
    if (n == 4) return launch_grad<TI, TO, 4>(L, ids, M, dout, V, D, scale, dtable, ws, s, launches);
    if (n == 2) return launch_grad<TI, TO, 2>(L, ids, M, dout, V, D, scale, dtable, ws, s, launches);
    return launch_grad<TI, TO, 1>(L, ids, M, dout, V, D, scale, dtable, ws, s, launches);
}

}  // namespace
}  // namespace lb

using namespace lb;

extern "C" lb_status lb_embedding_forward(const int64_t *ids, int64_t M, const void *table, int table_dtype, int V, int D,
                                          float scale, void *out, int out_dtype, void *stream)
{
    set_launch_count(0);
    if (M < 0 || V < 1 || D < 1 || !known(table_dtype) || !known(out_dtype)) return LB_ERR_INVALID_ARG;
    if (M > (1LL << 31) - 1 || D > (1 << 25)) return LB_ERR_UNSUPPORTED;
    if (M == 0) return LB_OK;
    const size_t si = size_of(table_dtype), so = size_of(out_dtype);
    if (!ids || !table || !out || misaligned(ids, 8) || misaligned(table, si) || misaligned(out, so))
        return LB_ERR_INVALID_ARG;
    const int n = vector_of(D, si == 2 && so == 2 ? 8 : 4, table, si, out, so);
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (table_dtype == LB_F32)
        e = out_dtype == LB_F32 ? lookup<float, float>(n, ids, M, table, V, D, scale, out, s)
                                : lookup<float, uint16_t>(n, ids, M, table, V, D, scale, out, s);
    else
        e = out_dtype == LB_F32 ? lookup<uint16_t, float>(n, ids, M, table, V, D, scale, out, s)
                                : lookup<uint16_t, uint16_t>(n, ids, M, table, V, D, scale, out, s);
    set_launch_count(1);
    return status_from(e);
}

extern "C" size_t lb_embedding_backward_workspace_bytes(int64_t M, int V, int D)
{
    EmbedPlan L;
    return embed_plan(L, M, V, D) ? L.bytes : 0;
}

extern "C" lb_status lb_embedding_backward(const int64_t *ids, int64_t M, const void *dout, int dout_dtype, int V, int D,
                                           float scale, void *dtable, int dtable_dtype, void *workspace,
                                           size_t workspace_bytes, void *stream)
{
    set_launch_count(0);
    EmbedPlan L;
    if (M < 0 || V < 1 || D < 1 || !known(dout_dtype) || !known(dtable_dtype)) return LB_ERR_INVALID_ARG;
    if (!embed_plan(L, M, V, D)) return LB_ERR_UNSUPPORTED;
    const size_t si = size_of(dout_dtype), so = size_of(dtable_dtype);
    if (!dtable || misaligned(dtable, so)) return LB_ERR_INVALID_ARG;
    if (M > 0 && (!ids || !dout || !workspace || misaligned(ids, 8) || misaligned(dout, si) ||
                  misaligned(workspace, 256) || workspace_bytes < L.bytes))
        return LB_ERR_INVALID_ARG;
    const int n = vector_of(D, si == 2 ? 8 : 4, M ? dout : dtable, M ? si : so, dtable, so);
    unsigned char *ws = (unsigned char *)workspace;
    cudaStream_t s = (cudaStream_t)stream;
    int launches = 0;
    cudaError_t e;
    if (dout_dtype == LB_F32)
        e = dtable_dtype == LB_F32 ? grad<float, float>(n, L, ids, M, dout, V, D, scale, dtable, ws, s, &launches)
                                   : grad<float, uint16_t>(n, L, ids, M, dout, V, D, scale, dtable, ws, s, &launches);
    else
        e = dtable_dtype == LB_F32 ? grad<uint16_t, float>(n, L, ids, M, dout, V, D, scale, dtable, ws, s, &launches)
                                   : grad<uint16_t, uint16_t>(n, L, ids, M, dout, V, D, scale, dtable, ws, s, &launches);
    set_launch_count(launches);
    return status_from(e);
}
