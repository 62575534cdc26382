// Rotary positions: the angles and the turn of sixteen channels, as the kernels
// of rotary.cu and ragged_append.cu use them.
//
// A unit is 16 channels of a row, eight pairs: channels 8u .. 8u + 7 with
// rot / 2 + 8u .., or 16u .. 16u + 15 (neighbours, and channels that are only
// copied).  A thread keeps the eight cosines and sines of its token's unit and
// takes the unit of several heads with them.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "../../include/diffattn_rotary.h"

namespace diffattn {

// False where the table's own fields are wrong (d: channels of a row).
inline bool rotary_table_ok(const diffrotary_table &t, int64_t d) {
  return t.freq != nullptr && (reinterpret_cast<uintptr_t>(t.freq) & 7) == 0 && t.rot >= 16 &&
         t.rot % 16 == 0 && t.rot <= d && t.reserved == 0 && (t.neighbours == 0 || t.neighbours == 1);
}

struct Turn {
  float c[8], s[8];
};

// The turn of pairs 8u .. 8u + 7 at position pos (negated: the turn back).  The product with the
// 64-bit fraction wraps at whole turns; its upper 32 bits are the angle to 2^-32 of a turn.
// kShort (bf16 outputs, whose rounding hides 2^-21): the sine and cosine by the approximate
// instructions, within half a turn of zero off by at most 2^-21.41 and 2^-21.19; eight pairs by
// sincospif take as long as the memory of four heads' units (221 MB of packed rows 35.3 us, so
// 34.8).  Not where fp32 or e4m3 is written: e4m3's wide steps show the last bits of a value next to
// the border between two (of 12.7 million, 27 to 33 fell to the wrong side, so 3 to 6, as with sines
// worked out in 64 bits and rounded once; 120 MB 22.6 us, so 23.9).
template <bool kShort>
__device__ __forceinline__ Turn make_turn(const uint64_t *freq, int u, int64_t pos, float scale) {
  Turn t;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint64_t angle = static_cast<uint64_t>(pos) * freq[8 * u + i];
    const int32_t part = static_cast<int32_t>(angle >> 32);  // of 2^31: half a turn
    constexpr float kStep = 1.4629180792671596e-9f;          // pi 2^-31
    if constexpr (kShort) {
      const float x = static_cast<float>(part) * kStep;
      t.s[i] = __sinf(x);
      t.c[i] = __cosf(x);
    } else {
      // fp32 has the upper 24 bits; the last eight are a turn of d <= 2^-21.3 more, to first order.
      float s, c;
      sincospif(static_cast<float>(part & ~0xFF) * 0x1p-31f, &s, &c);
      const float d = static_cast<float>(part & 0xFF) * kStep;
      t.s[i] = fmaf(c, d, s);
      t.c[i] = fmaf(-s, d, c);
    }
    t.s[i] *= scale;
    t.c[i] *= scale;
  }
  return t;
}

// Channel offsets of the two halves of a unit.
struct UnitAt {
  int a, b;
};
__device__ __forceinline__ UnitAt unit_at(int u, int rot, bool neighbours) {
  const bool apart = !neighbours && 16 * u < rot;
  return apart ? UnitAt{8 * u, rot / 2 + 8 * u} : UnitAt{16 * u, 16 * u + 8};
}

__device__ __forceinline__ void turn_unit(float (&x)[16], const Turn &t, bool neighbours) {
  if (neighbours) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = a * t.c[i] - b * t.s[i];
      x[2 * i + 1] = a * t.s[i] + b * t.c[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = x[i], b = x[8 + i];
      x[i] = a * t.c[i] - b * t.s[i];
      x[8 + i] = a * t.s[i] + b * t.c[i];
    }
  }
}

// Eight channels of bf16 (one 16-byte unit) or fp32 (two).
__device__ __forceinline__ void widen(const uint4 &q, float *x) {
  const uint32_t in[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(in[i] << 16);
    x[2 * i + 1] = __uint_as_float(in[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 narrow_bf16(const float *x) {
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(out[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
  return make_uint4(out[0], out[1], out[2], out[3]);
}
__device__ __forceinline__ uint2 narrow_e4m3(const float *x) {
  uint32_t half[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    half[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i], x[2 * i + 1]), __NV_SATFINITE,
                                       __NV_E4M3);
  return make_uint2(half[0] | (half[1] << 16), half[2] | (half[3] << 16));
}

}  // namespace diffattn
