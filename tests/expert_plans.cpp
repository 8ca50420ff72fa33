// Which kernel the experts' products take, for sizes "gated rows experts f k" read from
// the input, one line each.  With an argument,
// instead, the LDS bytes that launches for tiles of 16 and of 64 rows ask for with so
// many experts.  Built for the host alone, for 256 compute units.
#include <cstdio>
#include <cstdlib>

#include "expert_gemm.hip"

int main(int argc, char **argv) {
  if (argc > 1) {
    const long long all = std::atoll(argv[1]);
    std::printf("%zu %zu\n", fp8bsq::StreamShape<16>::lds(all), fp8bsq::StreamShape<64>::lds(all));
    return 0;
  }
  long long gated, rows, experts, f, k;
  while (std::scanf("%lld %lld %lld %lld %lld", &gated, &rows, &experts, &f, &k) == 5) {
    using fp8bsq::Shape;
    const Shape s = fp8bsq::product_shape(rows, experts, f, k, gated != 0, 256);
    const bool by_four = fp8bsq::scales_by_four((int)(k / 128), nullptr);
    std::puts(s == Shape::kLong32 ? "long32" : s == Shape::kLong64 ? "long64" : s == Shape::kFew ? "few" : s == Shape::kSome ? "some"
                                  : by_four ? "many by four" : "many");
  }
}
