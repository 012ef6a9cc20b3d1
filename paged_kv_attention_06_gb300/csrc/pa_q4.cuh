// The 4-bit rows of a page pool: 128 elements in 80 bytes. Bytes 0-63 are the
// codes (element d in byte d / 2, even d in the low half); then for each group of
// 32 elements its step s and its least value m as f16: s0 m0 s1 m1 s2 m2 s3 m3. A code
// c stands for m + s c.
#pragma once

#include <stdint.h>

namespace pa {

constexpr int kQ4RowBytes = 80;
constexpr int kQ4CodeBytes = 64;
constexpr int kQ4Group = 32;
// Magnitudes are cut to e4m3's largest, so that 1024 s and 32 m are f16 (a decode kernel
// turns codes into f16 by the one, and adds the least values up by the other).
constexpr float kQ4Max = 448.f;

}  // namespace pa
