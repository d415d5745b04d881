// pa_fp4.cuh -- the 4-bit pools: layout, quantiser and widening.
//
// A pool is [num_blocks, Hkv, block_size / 8] tiles of eight tokens; a tile is eight
// rows of D / 2 bytes of E2M1 codes (element 2i in the low half of byte i), then eight
// rows of D / 16 E4M3 scales, one for each group of 16 elements.  A tile is contiguous
// (4.5 D bytes, a multiple of 16) and so are the tiles of a (block, head), so any run of
// tokens that starts at a multiple of eight is one copy.  A value is code * scale * S, S
// the head's fp32 scale.
#pragma once

#include "pa_device.cuh"

namespace pa {
namespace fp4 {

template <int D>
struct Tile {
  static constexpr int kRowBytes = D / 2;        // codes of a token
  static constexpr int kScaleBytes = D / 16;     // scales of a token
  static constexpr int kScales = 8 * kRowBytes;  // offset of the scales
  static constexpr int kBytes = kScales + 8 * kScaleBytes;
};

// A head's scale is usable between 2^-64 and 2^64: then 6 S, the group scales times S
// and the quotients below are normal numbers (or round to code 0).
__device__ __forceinline__ bool head_scale_ok(float s) {
  return s >= 5.421010862427522e-20f && s <= 1.8446744073709552e19f;
}

// E4M3(x) in the low byte: nearest, ties to even, at most 448 (x >= 0).
__device__ __forceinline__ uint32_t to_e4m3(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r;
}
// Two E4M3 bytes (low half of w) as fp16 pairs; exact.
__device__ __forceinline__ uint32_t e4m3_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(w)));
  return r;
}
// The four bytes of a word of codes: byte b as the fp16 pair (low half, high half); exact.
__device__ __forceinline__ void widen8(uint32_t w, uint32_t &r0, uint32_t &r1, uint32_t &r2,
                                       uint32_t &r3) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
      : "r"(w));
}
// Eight values -> eight codes: nearest, ties to even, at most 6.
__device__ __forceinline__ uint32_t to_e2m1(const float *f) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return r;
}

// The larger magnitudes of two pairs of 16-bit values; NaN where either is.
template <class E>
__device__ __forceinline__ typename E::T2 max_abs(typename E::T2 a, uint32_t w) {
  return __hmax2_nan(a, __habs2(*reinterpret_cast<typename E::T2 *>(&w)));
}

// What a head's groups share: its scale S (0: unusable), 6 S and RN(1 / (6 S)).
struct HeadScale {
  float s, six, r;
  __device__ __forceinline__ HeadScale(float S) {
    s = head_scale_ok(S) ? S : 0.f;
    six = __fmul_rn(6.f, S);
    r = __frcp_rn(six);
  }
};

// One group: 16 values (eight words of two) -> 16 codes and their scale's byte.  With S
// the head's scale and every operation in fp32, rounded to nearest:
//   c = E4M3(max |x| / (6 S)), w = value(c) S, codes E2M1(x / w); c = 0: codes 0.
// NaN counts as 0.  Both divisors are normal numbers (w >= 2^-73), so their correctly
// rounded quotients take a reciprocal, a product and two fused steps (div_rn_recip), and
// while no value is NaN or infinite and c not at its end, none of its special cases.
template <class E>
__device__ __forceinline__ uint2 quantise16(const uint32_t (&v)[8], const HeadScale &h,
                                            uint32_t &scale) {
  scale = 0;
  if (h.s == 0.f) return make_uint2(0, 0);
  typename E::T2 m2 = max_abs<E>(*reinterpret_cast<const typename E::T2 *>(&v[0]), v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m2 = max_abs<E>(m2, v[i]);
  const uint32_t mw = *reinterpret_cast<const uint32_t *>(&m2);
  float m = fmaxf(fabsf(E::lo(mw)), fabsf(E::hi(mw)));
  const bool odd = !(fabsf(E::lo(mw)) + fabsf(E::hi(mw)) < INFINITY);
  float x[16];
  if (odd) {
    m = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float y = i & 1 ? E::hi(v[i / 2]) : E::lo(v[i / 2]);
      m = fmaxf(m, y != y ? 0.f : fabsf(y));
    }
  }
  scale = to_e4m3(div_rn_recip(m, h.six, h.r));
  if (scale == 0) return make_uint2(0, 0);
  const float w = __fmul_rn(F16::lo(e4m3_to_f16x2(scale)), h.s), r = __frcp_rn(w);
  if (odd || scale == 126) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float y = i & 1 ? E::hi(v[i / 2]) : E::lo(v[i / 2]);
      x[i] = div_rn_recip(y != y ? 0.f : y, w, r);
    }
  } else {
    // two at a time, from -x: q = (-x)(-r), e = q w - x, q - e r, which leaves -0 as it is
    const uint64_t w2 = f2_pack(w, w), nr = f2_pack(-r, -r);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t n = v[i] ^ 0x80008000u;
      const uint64_t nx = f2_pack(E::lo(n), E::hi(n)), q = f2_mul(nx, nr);
      f2_unpack(f2_fma(f2_fma(q, w2, nx), nr, q), x[2 * i], x[2 * i + 1]);
    }
  }
  return make_uint2(to_e2m1(x), to_e2m1(x + 8));
}

}  // namespace fp4
}  // namespace pa
