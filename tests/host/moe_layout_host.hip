// Host program over csrc/moe_layout.h: lines "pad COUNT ALIGN" -> the padded run; "rows FIRST END LANE" -> the number of rows, the
// first and the last of them (0 0 0 for none).
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "../../bit_block_scaled_quantize_amd/csrc/moe_layout.h"

int main() {
  char what[8];
  long long a, b;
  while (std::scanf("%7s %lld %lld", what, &a, &b) == 3) {
    if (std::strcmp(what, "pad") == 0) {
      std::printf("%d\n", nvfp4::padded_run((int)a, (int)b));
      continue;
    }
    long long lane, n = 0, first = 0, last = 0;
    if (std::scanf("%lld", &lane) != 1) return 1;
    nvfp4::each_64th((int)a, (int)b, (int)lane, [&](int64_t r) {
      if (n++ == 0) first = r;
      last = r;
      if (n > 1000000) std::fputs("runs on\n", stdout), std::exit(2);
    });
    std::printf("%lld %lld %lld\n", n, first, last);
  }
}
