// Arithmetic of sizes, for host code of any compiler.
#pragma once

#include <cstdint>

namespace wgs {

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace wgs
