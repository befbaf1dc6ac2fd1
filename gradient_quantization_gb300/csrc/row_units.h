// row_units.h -- how many CTAs (or clusters) share the rows of a layer norm call, and how
// many rows of partial sums its workspace holds.  Host arithmetic without CUDA.
#pragma once

#include <cstdint>

namespace agoq {

// Rows of partial sums of dw and db: at most two an SM of 152, and more of short rows,
// whose CTAs are small (as many bytes as 304 rows of 4096 elements); no more than T.
inline int ln_partials(int64_t T, int64_t H) {
    const int64_t fit = H < 4096 ? 4096 / H : 1, most = 304 * (fit < 8 ? fit : 8);
    return (int)(T < most ? T : most);
}

// CTAs (clusters) of the kernels for any alignment, of `n` that are resident: a multiple of
// eight where one takes several rows, so that its rows start at the same place between
// 16-byte boundaries.  Never more than T or `most`: each writes a row of partial sums.  (Up
// to eight rows take a unit each, resident at once or not.)
inline int by_eights(int n, int64_t T, int most) {
    if (n < 8) n = 8;
    if (n > most) n = most;
    return n >= T ? (int)T : n > 8 ? n / 8 * 8 : n;
}

}  // namespace agoq
