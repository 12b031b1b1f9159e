// The FP8 block-scaled product of few tokens with bfloat16 results, and how it runs.
#include "dh_fp8_few.cuh"

namespace dh {
namespace f8 {

// Fewest microseconds over the clusters that fit: rounds of tiles times a step's time (0.40 us; 0.60
// where 128 tokens' sums are what takes it) and a tile's end, which an exchange makes longer by
// the tokens; quantising in the kernel costs 0.85 us for every 32 blocks of 128 (less what the
// first boxes take to come), before it 3. Measured, us: 24
// tokens x 4,608 x 2,560 9.2, 64 12, 128 16 (4 CTAs each, quantised before); 32 x 64,026 x 2,560
// 36 (1 CTA).
template <int NT, bool FUSED>
void consider(int M, int tiles, int steps, FewPlan& best) {
    using F = Few<NT, FUSED>;
    for (int s = 1; s <= kMaxSplits; ++s) {
        const int per = ceil_div(steps, s);
        if ((s - 1) * per >= steps || F::rest(per, s) + 3 * F::kStage > kSpace) continue;
        const float end = s == 1 ? 0.6f : 1.5f + 0.06f * NT;
        const int blocks = ceil_div(M * per, 32);
        const float us = ceil_div(tiles, kClusters[s]) * (per * (NT < 128 ? 0.40f : 0.60f) + end) +
                         (FUSED ? (blocks > 2 ? 0.85f * (blocks - 2) : 0.0f) : 3.0f);
        if (best.splits == 0 || us < best.us) best = {NT, s, FUSED, us};
    }
}

FewPlan few_plan(int M, int out, int width) {
    const int tiles = ceil_div(out, kBlock), steps = ceil_div(width, kBlock);
    FewPlan p = {};
    if (M <= 16) {
        consider<16, true>(M, tiles, steps, p);
    } else if (M <= 32) {
        consider<32, true>(M, tiles, steps, p);
        consider<32, false>(M, tiles, steps, p);
    } else if (M <= 64) {
        consider<64, true>(M, tiles, steps, p);
        consider<64, false>(M, tiles, steps, p);
    } else if (M <= kFewTokens) {
        consider<128, false>(M, tiles, steps, p);
    }
    return p;
}

template cudaError_t launch_few<__nv_bfloat16>(const Fp8BlockArgs&, const FewPlan&, const uint8_t*, int, const float*, cudaStream_t);

}  // namespace f8
}  // namespace dh
