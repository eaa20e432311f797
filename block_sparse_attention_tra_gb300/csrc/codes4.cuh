// codes4.cuh -- e2m1 codes as f16, for the kernels over the 4-bit cache.
#pragma once

#include <stdint.h>

namespace bsa {

// The eight codes of a word as four f16x2, two neighbours each.
__device__ __forceinline__ void f16_of_codes(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}

}  // namespace bsa
