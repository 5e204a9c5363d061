// The scaling pass of an orthogonalised update, element by element: over all vectors of a padded matrix every element is
// read once and none outside it, whatever the columns leave over of 64 and of 8, and where they are whole groups of four
// so are the reads (the kernel then loads 16 bytes at a time).
#include <cstdio>
#include <vector>

#include "lb_orth_index.h"

static int check(int rows, int cols)
{
    const int pitch = (cols + 63) & ~63;
    const size_t size = (size_t)rows * cols, vectors = (size_t)rows * pitch / 8;
    std::vector<unsigned char> read(size, 0);
    for (size_t i = 0; i < vectors; ++i) {
        const lb::SplitVector v = lb::split_vector(i, cols, pitch);
        const size_t row = i / (pitch / 8), col = i % (pitch / 8) * 8;
        if (v.n < 0 || v.n > 8 || (v.n && v.at + v.n > size)) return 1;
        if (cols % 4 == 0 && (v.n % 4 || (v.n && v.at % 4))) return 2;
        for (int j = 0; j < v.n; ++j) {
            if (v.at + j != row * cols + col + j || col + j >= (size_t)cols) return 3;
            if (read[v.at + j]++) return 4;
        }
    }
    for (size_t e = 0; e < size; ++e)
        if (!read[e]) return 5;
    return 0;
}

int main()
{
    for (int cols = 1; cols <= 200; ++cols)
        for (int rows : {1, 2, 3, 7, 64, 65})
            if (const int what = check(rows, cols)) {
                std::fprintf(stderr, "%d x %d: %d\n", rows, cols, what);
                return 1;
            }
    for (int cols : {1023, 1024, 1025, 2044, 2047, 2048, 4097, 65536})
        if (const int what = check(5, cols)) {
            std::fprintf(stderr, "5 x %d: %d\n", cols, what);
            return 1;
        }
    // offsets past 32 bits: the last row of 2^24 x 2048
    const lb::SplitVector far = lb::split_vector((((size_t)1 << 24) - 1) * 256 + 255, 2048, 2048);
    if (far.at + 8 != (size_t)1 << 35 || far.n != 8) return 1;
    std::puts("orth index ok");
    return 0;
}
