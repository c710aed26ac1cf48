// norm_shape.h -- how the norm kernels hold a row of C columns, and the shared memory that a block takes for it.
// Plain host arithmetic, which the tests walk over every width.
#pragma once

#include <stddef.h>

namespace gspn {
namespace seq {

enum { kWPost, kBPost, kScale, kWPre, kBPre, kParams };   // a norm call's parameters

// Elements of a thread, threads of a block (128 = four warps with a row each, `warp`), up to seven places
// kept free for the phase; `wide`: the kernels for wide rows.
struct Shape {
    int e, threads;
    bool warp, wide;
};
inline Shape shape_for(int C) {
    const int n = C % 8 != 0 ? C + 7 : C;
    if (n <= 256) return {8, 128, true, false};
    if (n <= 2048) return {8, (n + 255) / 256 * 32, false, false};
    if (n <= 4096) return {16, (n + 511) / 512 * 32, false, false};
    return {16, (C + 511) / 512 * 32, false, true};
}
// Dynamic shared memory: parameters and the backward pass's column sums (`slots` of them); of wide rows the latter only.
inline size_t smem_for(const Shape& s, int slots) {
    if (s.wide) return (size_t)slots * 8 * s.threads * 8;
    return (size_t)s.threads * s.e * (kParams + slots) * sizeof(float);
}
// The kernels' own arrays beside it (the sums over a row), at most.
constexpr size_t kStaticSmem = 768;
// Whether a launch has to ask for more than the 48 KB that every block may have. Those 48 KB are for both kinds
// of shared memory together: one column sum of 2048 columns takes exactly 48 KB of the dynamic kind.
inline bool over_48k(size_t dynamic) { return dynamic + kStaticSmem > 48 * 1024; }

}  // namespace seq
}  // namespace gspn
