// kv4_sm100.cuh -- the 4-bit form of keys and values in the paged cache.
//
// 32 neighbouring values of a row share a scale and a minimum, both bf16:
//   mn = min rounded down, sc = (max - mn) / 15 rounded up (2^-126 at least, or
//   0), n = rint((x - mn) / sc)
// and the value read back is sc n + mn.  n is 0 .. 15 by itself.  Rounding mn down
// and sc up keeps every value inside [mn, mn + 15 sc], so no value is off by
// more than sc / 2.  Codes are those of the exact quotient: with the bf16 inputs
// of the values exact ties are common, and they go to the even code.  A group
// that holds a NaN or an infinity, or whose spread does not fit, reads back as NaN.
//
// A record is 16 rows of one head: the codes (8 D bytes), then [16][D / 32]
// pairs (sc, mn).  The code order is the one in which a warp's m16n8k16
// tensor-core fragments are made from it without an exchange, each lane from
// whole 16-byte (D = 64: 8-byte) pieces:
//   keys:   row r at r D / 2; a 32-bit word holds the 8 values d = 8 m .. 8 m + 7,
//           value 2 i in nibble i and 2 i + 1 in nibble i + 4, so a mask and a
//           shift leave neighbouring values in the two halves of a register;
//           word m stands at (m % 4) (D / 32) + m / 4: a lane's words, one of
//           each group, are contiguous.
//   values: a 32-bit word holds the same 4 values d = 32 g' + 4 g + i of two
//           neighbouring rows r, r + 1 (low and high half, nibble i); the words
//           of the D / 32 groups g' are contiguous, at lane 4 g + (r / 2) % 4,
//           the two halves of the record (r / 8) after each other.
#pragma once

#include <cfloat>
#include <cstdint>

#include "sm100_ptx.cuh"

namespace sskip {

template <int D>
struct Kv4 {
  static constexpr int kGroups = D / 32;
  static constexpr int kCodes = 8 * D;              // bytes of 16 rows' codes
  static constexpr int kRecord = kCodes + 16 * kGroups * 4;
};

__device__ __forceinline__ void kv4_bounds(const float (&x)[8], float& lo, float& hi) {
  lo = min_nan(min_nan(x[0], x[1], x[2]), min_nan(x[3], x[4], x[5]), min_nan(x[6], x[7]));
  hi = max_nan(max_nan(x[0], x[1], x[2]), max_nan(x[3], x[4], x[5]), max_nan(x[6], x[7]));
}

// rint(y / sc), ties to even, for 0 <= y <= about 15 sc, in the low bits of a
// float (kCodeBias + code).  The quotient is the correctly rounded one: an
// estimate by the correctly rounded reciprocal, and one correction by the exact
// remainder (Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990; scales within 2^23 of the smallest can have a
// subnormal, so inexact, remainder, and then an ulp is off).  One division a
// group, not one a value: the reciprocal unit takes 8 clocks of a sub-partition
// for a warp.  No clamp: sc is (max - mn) / 15 to an ulp at least, so no quotient
// of a finite group comes near 15.5; one that holds a NaN or an infinity leaves
// any codes, in words of its own, under a scale that is NaN.
constexpr uint32_t kCodeBias = 0x4B400000u;  // 1.5 * 2^23: adding it rounds to an integer
__device__ __forceinline__ uint32_t kv4_code(float y, float sc, float inv) {
  const float q = y * inv;
  const float exact = fmaf(fmaf(-q, sc, y), inv, q);
  return __float_as_uint(exact + __uint_as_float(kCodeBias));
}

// Store row r of a record.  The D / 16 lanes of a head hold chunks m0 and m1
// (8 values each) of it; all 32 lanes call, `live` ones write.  split: how many
// lanes of a head hold chunks (j, j + split), which `apart` says of this one;
// the others hold (2 j, 2 j + 1).
template <int D>
__device__ __forceinline__ void kv4_store_row(uint8_t* rec, int r, bool value, bool live, int split,
                                              bool apart, int m0, int m1, const float (&x0)[8],
                                              const float (&x1)[8]) {
  constexpr int LH = D / 16, NG = Kv4<D>::kGroups;
  constexpr uint32_t kAll = 0xffffffffu;
  float lo[2], hi[2];  // of the groups of the two chunks
  kv4_bounds(x0, lo[0], hi[0]);
  kv4_bounds(x1, lo[1], hi[1]);
  if (split <= 2 || split % 4 == 0) {
    // A group's four chunks are both chunks of a pair of lanes, or (apart,
    // split a multiple of 4) one chunk each of four neighbours.
    const bool quad = apart && split > 2;
    if (!quad) {
      lo[0] = lo[1] = min_nan(lo[0], lo[1]);
      hi[0] = hi[1] = max_nan(hi[0], hi[1]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      lo[i] = min_nan(lo[i], __shfl_xor_sync(kAll, lo[i], 1));
      hi[i] = max_nan(hi[i], __shfl_xor_sync(kAll, hi[i], 1));
      const float l2 = __shfl_xor_sync(kAll, lo[i], 2), h2 = __shfl_xor_sync(kAll, hi[i], 2);
      if (quad) {
        lo[i] = min_nan(lo[i], l2);
        hi[i] = max_nan(hi[i], h2);
      }
    }
  } else {
    const float clo[2] = {lo[0], lo[1]}, chi[2] = {hi[0], hi[1]};
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      float l = min_nan((m0 >> 2) == g ? clo[0] : INFINITY, (m1 >> 2) == g ? clo[1] : INFINITY);
      float h = max_nan((m0 >> 2) == g ? chi[0] : -INFINITY, (m1 >> 2) == g ? chi[1] : -INFINITY);
#pragma unroll
      for (int o = LH / 2; o > 0; o >>= 1) {
        l = min_nan(l, __shfl_xor_sync(kAll, l, o));
        h = max_nan(h, __shfl_xor_sync(kAll, h, o));
      }
      if ((m0 >> 2) == g) { lo[0] = l; hi[0] = h; }
      if ((m1 >> 2) == g) { lo[1] = l; hi[1] = h; }
    }
  }
  if (!live) return;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int m = i ? m1 : m0;
    const float mn = __bfloat162float(__float2bfloat16_rd(lo[i]));
    float sc = __bfloat162float(__float2bfloat16_ru(__fdiv_rn(hi[i] - mn, 15.f)));
    // A NaN or an infinity in the group, or a spread that does not fit.
    const bool bad = !(sc <= FLT_MAX) || !(fabsf(mn) <= FLT_MAX);
    if (sc > 0.f) sc = fmaxf(sc, FLT_MIN);  // its reciprocal stays finite
    const float inv = sc > 0.f ? __frcp_rn(sc) : 0.f;
    uint32_t n[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) n[e] = kv4_code((i ? x1[e] : x0[e]) - mn, sc, inv);
    if ((m & 3) == 0) {
      const uint32_t w = bad ? 0x7FFF7FFFu : pack_bf16x2(sc, mn);
      *reinterpret_cast<uint32_t*>(rec + Kv4<D>::kCodes + (r * NG + (m >> 2)) * 4) = w;
    }
    // Codes side by side: the biases add up to a constant.
    if (!value) {
      uint32_t w = 0, bias = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        w += n[e] << (4 * ((e >> 1) + (e & 1) * 4));
        bias += kCodeBias << (4 * ((e >> 1) + (e & 1) * 4));
      }
      *reinterpret_cast<uint32_t*>(rec + r * (D / 2) + ((m & 3) * NG + (m >> 2)) * 4) = w - bias;
    } else {
#pragma unroll
      for (int qd = 0; qd < 2; ++qd) {
        const int g = (2 * m + qd) & 7;
        // kCodeBias has no low bits: 16 bits of the sum are the codes alone
        const uint32_t w = n[4 * qd] + (n[4 * qd + 1] << 4) + (n[4 * qd + 2] << 8) + (n[4 * qd + 3] << 12);
        *reinterpret_cast<uint16_t*>(rec + ((r >> 3) * 32 + g * 4 + ((r >> 1) & 3)) * NG * 4 +
                                     (m >> 2) * 4 + (r & 1) * 2) = (uint16_t)w;
      }
    }
  }
}

// Values 8 m .. 8 m + 7 of row r.
template <int D>
__device__ __forceinline__ void kv4_load_chunk(const uint8_t* rec, int r, bool value, int m,
                                               float (&x)[8]) {
  constexpr int NG = Kv4<D>::kGroups;
  const uint32_t par = *reinterpret_cast<const uint32_t*>(rec + Kv4<D>::kCodes +
                                                          (r * NG + (m >> 2)) * 4);
  const float sc = __uint_as_float(par << 16), mn = __uint_as_float(par & 0xFFFF0000u);
  if (!value) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(rec + r * (D / 2) +
                                                          ((m & 3) * NG + (m >> 2)) * 4);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      x[e] = fmaf((float)((w >> (4 * ((e >> 1) + (e & 1) * 4))) & 15u), sc, mn);
  } else {
#pragma unroll
    for (int qd = 0; qd < 2; ++qd) {
      const int g = (2 * m + qd) & 7;
      const uint32_t w = *reinterpret_cast<const uint16_t*>(
          rec + ((r >> 3) * 32 + g * 4 + ((r >> 1) & 3)) * NG * 4 + (m >> 2) * 4 + (r & 1) * 2);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[4 * qd + i] = fmaf((float)((w >> (4 * i)) & 15u), sc, mn);
    }
  }
}

}  // namespace sskip
