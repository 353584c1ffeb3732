// fp8.h -- internal declarations of the 8-bit serving head: block sizes, the
// e4m3 conversions and the argument checks its entry points share.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ce.h"

namespace ce {

constexpr int kFp8Block = 128;             // columns (and rows of a weight) that share a scale
constexpr float kE4m3Max = 448.f;          // the largest e4m3 value
constexpr float kFp8MinScale = 1.17549435e-38f;  // 2^-126: blocks of zeros, and those below it, have this scale

inline bool fp8_on(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline int fp8_elem(int dtype) { return dtype == CE_DT_F32 ? 4 : 2; }
inline bool fp8_dtype_ok(int dtype) { return dtype == CE_DT_F32 || dtype == CE_DT_BF16 || dtype == CE_DT_F16; }

// Two row-major buffers of n rows share no byte. (Two views side by side of one
// wider buffer count as overlapping here.)
inline bool fp8_apart(const void *a, int64_t a_bytes, const void *b, int64_t b_bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x + static_cast<uintptr_t>(a_bytes) <= y || y + static_cast<uintptr_t>(b_bytes) <= x;
}

// 2-D matrix of bytes [rows, cols], row stride ld (a multiple of 16), boxes of
// 128 columns x box_rows, 128-byte swizzle, zeros out of bounds (flce.cu).
cudaError_t make_tmap_bytes(CUtensorMap *m, const void *ptr, uint64_t rows, uint64_t cols, uint64_t ld,
                            uint32_t box_rows);

}  // namespace ce
