// Which kernel the experts' products take, for sizes "gated rows experts f k" read from
// the input, one line each.  Built for the host alone, for 256 compute units.
#include <cstdio>

#include "expert_gemm.hip"

int main() {
  long long gated, rows, experts, f, k;
  while (std::scanf("%lld %lld %lld %lld %lld", &gated, &rows, &experts, &f, &k) == 5) {
    using fp8bsq::Shape;
    const Shape s = fp8bsq::product_shape(rows, experts, f, k, gated != 0, 256);
    const bool by_four = fp8bsq::scales_by_four((int)(k / 128), nullptr);
    std::puts(s == Shape::kLong32 ? "long32" : s == Shape::kLong64 ? "long64" : s == Shape::kFew ? "few" : s == Shape::kSome ? "some"
                                  : by_four ? "many by four" : "many");
  }
}
