// The FP8 block-scaled product of few tokens with bfloat16 results, and how it runs.
#include "dh_fp8_few.cuh"

namespace dh {
namespace f8 {

// Fewest microseconds over the clusters that fit: rounds of tiles times a step's time (0.35 us, 0.38
// for 64 tokens) and a tile's end, which an exchange makes longer, by
// the tokens; quantising takes 0.6 us for every 32 blocks of 128 in the kernel, 3 before it.
// Measured, us (in the kernel / before it): 16 tokens x 64,026 x 2,560 39 / 33, 16 x 2,560 x 5,120
// 9.0 / 10, 32 x 4,608 x 2,560 in 4 CTAs 10.6 / 9.1; 1 x 4,608 x 2,560 in 1 CTA 7.2, in 4 5.9; 64 x
// 4,608 x 2,560 in 1 CTA 10.1, in 4 11.1.
template <int NT, bool FUSED>
void consider(int M, int tiles, int steps, FewPlan& best) {
    using F = Few<NT, FUSED>;
    for (int s = 1; s <= kMaxSplits; ++s) {
        const int per = ceil_div(steps, s);
        if ((s - 1) * per >= steps || F::rest(per, s) + 3 * F::kStage > kSpace) continue;
        const float end = s == 1 ? 0.9f : 3.7f + 0.047f * M;
        const float us = ceil_div(tiles, kClusters[s]) * (per * (NT < 64 ? 0.35f : 0.38f) + end) +
                         (FUSED ? M * per * (0.6f / 32) : 3.0f);
        if (best.splits == 0 || us < best.us) best = {NT, s, FUSED, us};
    }
}

FewPlan few_plan(int M, int out, int width) {
    const int tiles = ceil_div(out, kBlock), steps = ceil_div(width, kBlock);
    FewPlan p = {};
    if (M <= 16) {
        consider<16, true>(M, tiles, steps, p);
        consider<32, false>(M, tiles, steps, p);
    } else if (M <= 32) {
        consider<32, true>(M, tiles, steps, p);
        consider<32, false>(M, tiles, steps, p);
    } else if (M <= kFewTokens) {
        consider<64, true>(M, tiles, steps, p);
        consider<64, false>(M, tiles, steps, p);
    }
    return p;
}

template cudaError_t launch_few<__nv_bfloat16>(const Fp8BlockArgs&, const FewPlan&, const uint8_t*, int, const float*, cudaStream_t);

}  // namespace f8
}  // namespace dh
