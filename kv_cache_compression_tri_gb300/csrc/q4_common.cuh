// q4_common.cuh -- rows in 4 bits: d / 2 bytes of codes, then (scale, minimum) in
// fp16 for each quarter of the row (the header has the order of the codes).
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace tri {
namespace {

constexpr float Q4_MOST = 30656.f;  // largest magnitude stored: scales stay below 2^12, an fp16 number times 16

template <int D>
struct Q4Row {
  static constexpr int CODES = D / 2;          // bytes of codes
  static constexpr int BYTES = CODES + 16;
  static constexpr int WORDS = D / 32;         // 32-bit words of codes per lane of four
};

}  // namespace
}  // namespace tri
