// The form of each call asked for on standard input (operator, type, T, d, f
// in numbers), from the library's own header: a line for each, in the words of
// tests/product_forms.py.
#include <cstdio>
#include <cstring>

#include "product_plan.hpp"

using namespace gift;

int main() {
  char op[16], type[16];
  long T, d, f;
  while (std::scanf("%15s %15s %ld %ld %ld", op, type, &T, &d, &f) == 5) {
    const int dtype = std::strcmp(type, "fp32") ? GIFT_BF16 : GIFT_FP32;
    const int planes = dtype == GIFT_FP32 ? 6 : 1;
    ProdPlan p{};
    if (!std::strcmp(op, "forward")) {
      if (glu_by_tokens(dtype, T, (int)d, (int)f)) {
        std::printf("tokens %d\n", 16 * glu_token_units(dtype, T, (int)f));
        continue;
      }
      p = product_plan(kEpiGlu, false, false, f, T, d, planes);
    } else if (!std::strcmp(op, "dx")) {
      if (glu_backward_by_tokens(dtype, T, false)) {
        std::printf("tokens\n");
        continue;
      }
      p = product_plan(kEpiStore, true, false, d, T, f, 2 * planes);
    } else {
      p = product_plan(kEpiGrad, true, true, d, f, T, planes);
    }
    std::printf("%d %s%s\n", p.side, p.deep ? "deep " : "",
                p.split == 0 ? "none" : p.split == p.nbm * p.nbn ? "all" : "some");
  }
}
