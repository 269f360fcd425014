// Sizes and alignments, in plain C++.
#pragma once

#include <stddef.h>
#include <stdint.h>

#ifdef __CUDACC__
#define GDP_HD __host__ __device__
#else
#define GDP_HD
#endif

namespace gdp {

constexpr size_t kAlign = 256;
GDP_HD inline size_t align_up(size_t x, size_t a = kAlign) { return (x + a - 1) / a * a; }
GDP_HD inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace gdp
