// Which elements of a matrix one step of the scaling pass of an orthogonalised
// update reads.  A plain header, so that a host program can go through the
// indices of a matrix: a read past its end is found there, not on a GPU.
#pragma once

#include <stddef.h>

#ifdef __CUDACC__
#define LB_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define LB_HOST_DEVICE inline
#endif

namespace lb {

// Vector i of a scaled matrix, whose rows of `cols` elements are padded to `pitch` (a multiple of 8): its 8 columns begin at
// element `at` of the matrix, and the first `n` of them exist there (0 for a vector of padding, which reads nothing).
struct SplitVector {
    size_t at;
    int n;
};
LB_HOST_DEVICE SplitVector split_vector(size_t i, int cols, int pitch)
{
    const int nv = pitch / 8;
    const size_t row = i / nv;
    const int col = (int)(i - row * nv) * 8, left = cols - col;
    return SplitVector{row * cols + col, left < 0 ? 0 : left < 8 ? left : 8};
}

}  // namespace lb
