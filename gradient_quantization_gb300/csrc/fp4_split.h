// fp4_split.h -- how many CTAs of a cluster share the K of a tile of the FP4 product.  Host
// arithmetic without CUDA.
#pragma once

#include <algorithm>
#include <cstdint>

namespace agoq {

// CTAs of `split` that have stages where each takes ceil(stages / split) of them: the others
// would hold tensor memory and join barriers to add zeros.
inline int64_t fp4_with_stages(int64_t stages, int64_t split) {
    const int64_t per = (stages + split - 1) / split;
    return (stages + per - 1) / per;
}

// One operand has at most 64 rows.  As many CTAs a tile as the GPU has room for (two an SM), with
// four stages each, or four CTAs where the stages are few.  1 x 11008 x 4096: 8.7 us with three, 9.2
// with two, 13.8 with four (more than fit); 16 x 4096 x 4096: 7.0 us with four, 7.5 with eight, 10.6
// with one; 32 x 1024 x 1024: 5.5 us with four, 6.5 with one.
inline int fp4_split_few_rows(int64_t stages, int64_t tiles, int sms) {
    const int64_t room = 2 * sms / tiles, most = std::max(stages / 4, std::min<int64_t>(stages, 4));
    return (int)fp4_with_stages(stages, std::max<int64_t>(1, std::min<int64_t>({8, room, most})));
}

// Few tiles of 128 x 128 over a long K, a CTA an SM, eight stages each (0 to 2: not shared).  300 x
// 200 x 9000: 10 us, 15 us without; but 512 x 512 x 4096, with four CTAs of four stages each: 8.8 us,
// 8.2 without.
inline int fp4_split_few_tiles(int64_t stages, int64_t tiles, int sms) {
    const int64_t split = std::min<int64_t>({8, sms / tiles, stages / 8});
    return split > 0 ? (int)fp4_with_stages(stages, split) : 0;
}

}  // namespace agoq
