// A tile's softmax as the d = 64 forwards do it (two threads a row, 64 of a tile's 128 keys each,
// read through the two-threads-per-lane shape), and the e4m3 operands of their first products.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace diffattn {
namespace {

constexpr int kTileColumns = 128;     // keys of a tile
constexpr float CERT_SUM = 65536.0f;    // half-row sums up to 2^16 certify a tile
// When the exact path sets the reference maximum it places it this far (log2
// units) above the tile's maximum: P then starts at most 2^-24 and later
// tiles may climb 24 + 16 units before the certificate fails again.  Only the
// scale of P, O and the sums changes (their relative precision does not); an
// entry more than about 100 units below the maximum flushes to zero, where
// its weight (below 2^-100 of the maximum's) is already far below rounding.
constexpr float M_HEADROOM = 24.0f;

// e4m3 operands (kind::f8f6f4): instruction descriptor with A and B both
// E4M3 (format code 0), fp32 D, K-major; and the shared-memory descriptor of
// a tile of 64-byte rows with 64-byte swizzle (layout code 4, 8-row groups
// 512 bytes apart).
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(uint32_t M, uint32_t N) {
  return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
__device__ __forceinline__ uint64_t smem_desc_sw64(uint32_t saddr) {
  uint64_t desc = 0;
  desc |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  desc |= static_cast<uint64_t>(1) << 16;
  desc |= static_cast<uint64_t>(512 >> 4) << 32;
  desc |= static_cast<uint64_t>(1) << 46;
  desc |= static_cast<uint64_t>(4) << 61;
  return desc;
}
// Issued by one elected lane of a converged warp (as umma_bf16_ss_lo_warp).
__device__ __forceinline__ void umma_e4m3_ss_warp(uint32_t d_tmem, uint64_t a_desc,
                                                  uint64_t b_desc, uint32_t idesc,
                                                  uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// acc += the two numbers of a bf16 pair, in fp32.
__device__ __forceinline__ void add_bf16x2(float2 &acc, uint32_t pair) {
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
      "add.f32.bf16 %0, lo, %0;\n\tadd.f32.bf16 %1, hi, %1;\n\t}"
      : "+f"(acc.x), "+f"(acc.y)
      : "r"(pair));
}

// One 32-key chunk of a half row: mask (key key0 + i visible iff key0 + i <=
// lim), x = s * log2(e)/sqrt(d) - m, p = 2^x, accumulate the sum in four
// packed partial sums and pack p as bf16 pairs into pk[pk0 ..].  kRounded: the
// sum is of the packed numbers instead.
template <bool kMasked, bool kRounded = false>
__device__ __forceinline__ void softmax_chunk_exp(const uint32_t (&x)[32], int key0, int pk0,
                                                  float m, float sl2, int lim, float2 (&acc)[4],
                                                  uint32_t (&pk)[kTileColumns / 4]) {
  const float2 scale = make_float2(sl2, sl2), negm = make_float2(-m, -m);
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    float a = __uint_as_float(x[i]), b = __uint_as_float(x[i + 1]);
    if (kMasked) {
      a = (key0 + i <= lim) ? a : -INFINITY;
      b = (key0 + i + 1 <= lim) ? b : -INFINITY;
    }
    float2 e = __ffma2_rn(make_float2(a, b), scale, negm);
    e.x = ex2_approx(e.x);
    e.y = ex2_approx(e.y);
    pk[pk0 + i / 2] = pack_bf16x2(e.x, e.y);
    if constexpr (kRounded)
      add_bf16x2(acc[(i / 2) % 4], pk[pk0 + i / 2]);
    else
      acc[(i / 2) % 4] = __fadd2_rn(acc[(i / 2) % 4], e);
  }
}

// Exponentials of this thread's 64 keys of an S row (keys key0 .. key0 + 63,
// read through the two-threads-per-lane shape) against reference maximum m.
// Returns the half row's sum of the unrounded exponentials or, kRounded, of
// the rounded ones.
template <bool kMasked, bool kRounded = false>
__device__ __forceinline__ float softmax_half_exp(uint32_t t_s, int key0, float m, float sl2,
                                                  int lim, uint32_t (&pk)[kTileColumns / 4]) {
  float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                   make_float2(0.f, 0.f)};
  uint32_t a[32], b[32];
  tmem_ld16_x32_nowait(t_s, a);
  tmem_ld16_x32_nowait(t_s + 32, b);
  tmem_ld_wait_x32(a);
  tmem_ld_wait_x32(b);
  softmax_chunk_exp<kMasked, kRounded>(a, key0, 0, m, sl2, lim, acc, pk);
  softmax_chunk_exp<kMasked, kRounded>(b, key0 + 32, 16, m, sl2, lim, acc, pk);
  const float2 s01 = __fadd2_rn(acc[0], acc[1]), s23 = __fadd2_rn(acc[2], acc[3]);
  return (s01.x + s01.y) + (s23.x + s23.y);
}

// Maximum of this thread's 64 keys of an S row over the visible ones.
template <bool kMasked>
__device__ __forceinline__ float softmax_half_max(uint32_t t_s, int key0, int lim) {
  uint32_t a[32], b[32];
  tmem_ld16_x32_nowait(t_s, a);
  tmem_ld16_x32_nowait(t_s + 32, b);
  tmem_ld_wait_x32(a);
  tmem_ld_wait_x32(b);
  float v[64];
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    v[i] = __uint_as_float(a[i]);
    v[32 + i] = __uint_as_float(b[i]);
  }
  if (kMasked) {
#pragma unroll
    for (int i = 0; i < 64; ++i) v[i] = (key0 + i <= lim) ? v[i] : -INFINITY;
  }
#pragma unroll
  for (int w = 32; w >= 1; w /= 2) {
#pragma unroll
    for (int i = 0; i < w; ++i) v[i] = fmaxf(v[i], v[i + w]);
  }
  return v[0];
}

// A row's first tile, whose reference is not known yet: the maximum of its visible keys (both halves'
// threads) from the registers that the exponentials are then taken from, so that S is read once.
// Sets m (-infinity where no key is visible or all logits are) and returns the half row's sum, which
// is of the rounded exponentials: weights that the products take then add up to one, so that a row of
// one key gets the value itself and a row of few (the first of a prompt, where both maps nearly
// cancel) keeps the precision of fp32 statistics.  The d = 128 forward adds the rounded ones in all
// tiles (it costs up to 1 %), so that rows whose maps both lean on one key keep it wherever the key is.
// At d = 64 later tiles add the unrounded ones, two at once: over many keys the roundings average out,
// and all tiles rounded took 1215 to 1238 us for 1146 to 1157 (2048 tokens behind 32768 keys), 259 for
// 247 (a mixed batch); only tiles that hold much of a row's sum, by a vote, 1211 and 272.
__device__ __forceinline__ float softmax_half_first(uint32_t t_s, int key0, float sl2, int lim,
                                                    bool masked, float &m,
                                                    uint32_t (&pk)[kTileColumns / 4]) {
  float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                   make_float2(0.f, 0.f)};
  uint32_t a[32], b[32];
  tmem_ld16_x32_nowait(t_s, a);
  tmem_ld16_x32_nowait(t_s + 32, b);
  tmem_ld_wait_x32(a);
  tmem_ld_wait_x32(b);
  if (masked) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      a[i] = key0 + i <= lim ? a[i] : 0xFF800000u;  // -infinity
      b[i] = key0 + 32 + i <= lim ? b[i] : 0xFF800000u;
    }
  }
  float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int i = 0; i < 32; ++i)
    top[i % 4] = fmaxf(top[i % 4], fmaxf(__uint_as_float(a[i]), __uint_as_float(b[i])));
  float mt = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
  mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 16));
  m = mt * sl2 + M_HEADROOM;
  const float m_use = m == -INFINITY ? 0.f : m;
  softmax_chunk_exp<false, true>(a, key0, 0, m_use, sl2, lim, acc, pk);
  softmax_chunk_exp<false, true>(b, key0 + 32, 16, m_use, sl2, lim, acc, pk);
  const float2 s01 = __fadd2_rn(acc[0], acc[1]), s23 = __fadd2_rn(acc[2], acc[3]);
  return (s01.x + s01.y) + (s23.x + s23.y);
}

}  // namespace
}  // namespace diffattn
