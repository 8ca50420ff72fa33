// How the backward pass of the gated feed-forward block launches its products,
// for sizes "m f k" read from the input, one line each: "dx dw paired", dx and dw
// being "big" (256 x 256 tiles), "mid" (128 x 128) or "split" (128 x 128, the
// contraction in parts), paired 1 where both go out in one launch.  Built for the
// host alone; without a GPU the plans are those of 256 compute units.
#include <cstdio>

#include "gated_ffn_backward.hip"

static const char *kind(const fp8bsq::TilePlan &p) { return p.big ? "big" : p.parts > 1 ? "split" : "mid"; }

int main() {
  long long m, f, k;
  while (std::scanf("%lld %lld %lld", &m, &f, &k) == 3) {
    const fp8bsq::TilePlan in = fp8bsq::input_plan(m, f, k), alone = fp8bsq::weight_plan(m, f, k);
    const fp8bsq::TilePlan wt = in.big ? alone : fp8bsq::paired_weight_plan(m, f, k);
    std::printf("%s %s %d %s\n", kind(in), kind(wt), in.big == wt.big, kind(alone));
  }
}
