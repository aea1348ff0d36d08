// backward.hpp -- the product of gradients with the codes, D W, as its callers have it (backward.hip).
#pragma once
#include "linear_codes.hpp"

namespace gptq {

// Y [t, n] = sum over up to two matrices of D_m [t, rows] W_m [rows, n]: D_m's columns start at m side of D.
struct BackArgs {
    const void* D;
    int64_t ldd;
    int side;
    int mats, rows, G, n;
    const uint8_t* codes[2];
    const float* scale[2];
    int t;
    void* Y;
    int64_t ldy;
    float* part;  // [splits, t, n] sums of pieces of the rows, or NULL
};
// How it is laid out: 16 tt tokens a wave, `waves` of a workgroup and `splits` pieces cut the rows between them.
struct BackPlan {
    int tt, waves, splits;
};
BackPlan back_plan(int64_t t, int64_t rows, int mats, int64_t n);
inline size_t back_part_bytes(const BackPlan& p, int64_t t, int64_t n) {
    return p.splits > 1 ? align256(sizeof(float) * (size_t)p.splits * (size_t)t * (size_t)n) : 0;
}
// D of type dd (the type dt of Y, or f32); rows of D at 16 bytes, whole 8 elements.  Returns a status.
int back_run(BackArgs a, const BackPlan& p, int dd, int dt, int bits, hipStream_t st);

}  // namespace gptq
