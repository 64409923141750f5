// append_kernel.cuh -- writes new tokens into a paged latent cache: RMSNorm of
// the compressed latent, rotation of its RoPE dims at the token's position,
// quantisation to the cache's row format, and the scatter to physical slots.
// (The cache formats: [FlashMLA (AI Wiki), "The FP8 and FP4 KV cache"].)
//
// Per token with latent x (d = 576 for the bf16 and 656-byte rows, 512 for the
// V4.1 rows) and physical slot s (block * 64 + offset, negative = no slot):
//   y_i = x_i g_i / sqrt(mean_{j<512}(x_j^2) + eps)        (i < 512, optional)
//   the last 64 dims rotated in pairs (2k, 2k + 1) by pos * base^(-2k/64)
//                                                          (optional)
//   1152 bytes  bf16(y)
//    656 bytes  scale = absmax/448 per 128 dims (fp32, 1 for a zero group),
//               codes e4m3(y 448 / absmax), the 64 RoPE dims in bf16
//               (y / scale where the scale is not a normal fp32 number)
//    528 bytes  scale = the least 2^e >= absmax/448 per 32 dims (E8M0)
//    288 bytes  scale = e4m3(absmax/6) per 16 dims (1 where that is 0),
//               codes e2m1(y / scale)
// The V4.1 latent includes its RoPE dims, so its norm covers them and the
// rotation follows the norm.  Optionally the rows are also written as the
// cache stands for them: bf16(code * scale), what the attention kernels read.
//
// One warp per token: lane l holds the 16-byte units l and l + 32 (8 dims
// each) of the first 512 dims, and lanes 0..7 the eight units behind them, so
// that a quantisation group is 16, 4 or 2 neighbouring lanes of one unit index
// and its maximum takes 4, 2 or 1 shuffles.  The gains lie in shared memory; a warp
// strides over the tokens.
//
// Precision: the norm's sum of squares and 1/sqrt are formed in fp64, y in fp32
// with the exact products' low parts carried along (one rounding), quotients with
// one more; with the rounded maximum and scale that is 2^-22 of a quotient.  One
// that lies within 2^-21 of a rounding border is decided in fp64 from the latent
// (rotated dims, whose error is relative to their pair: within 2^-18), and so are the
// 528- and 288-byte scales, so that the codes are those of the definition in fp64, but
// for rotated dims that cancel to less than a 16th of their pair.  A latent without
// norm needs none of that: its quotients are rounded once, the right way at a border.
// (32768 tokens with norm into FP4 rows: 27.5 us; 24 us
// without the second look, where a few codes in a million differ, and 21 us with
// the squares in fp32 and y = x (g / rms), where some ten do.)
//
// Bound: bulk calls by instructions (some 550 a token and warp; the quotients by
// one multiplication and one correction each, not by division), steps of a few
// tokens by one chain of latencies, so the slot, the position and the row are
// read side by side.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "combine_kernel.cuh"
#include "sparse_gather.cuh"

namespace mla {

constexpr int kRow1152 = 2 * kD;  // bf16 cache row
constexpr int kAppendWarps = 4;
constexpr int kAppendCtas = 6;  // CTAs per SM of a full grid

struct AppendParams {
  const __nv_bfloat16* kv;  // [n] rows of d values, kv_stride values apart
  long long kv_stride;
  const int32_t* slots;      // [n]
  const int32_t* positions;  // [n], or null: no rotation
  const float* gain;         // [512], or null: no norm
  double eps;
  double turns[kRope / 2];   // base^(-2k/64) / (2 pi), computed on the host in fp64
  int n;
  uint8_t* cache;  // [num_slots, row bytes]
  long long num_slots;
  __nv_bfloat16* rows;  // [n, d], or null
};

// x * g * inv with one rounding, inv = inv_hi + inv_lo: the product x g is held
// exactly as hi + lo, and the small products join hi * inv_hi inside the last fma.
__device__ __forceinline__ float mul3_once(float x, float g, float inv_hi, float inv_lo) {
  const float hi = x * g;
  const float lo = fmaf(x, g, -hi);
  return fmaf(hi, inv_hi, fmaf(lo, inv_hi, hi * inv_lo));
}

// 1/sqrt(v) for v in fp32's normal range: the fp32 value (2^-22) and one Newton
// step in fp64 (3/8 of its error squared: below 2^-44).
__device__ __forceinline__ double inv_root(double v) {
  const double r = static_cast<double>(rsqrtf(static_cast<float>(v)));
  return fma(0.5 * r, fma(-v * r, r, 1.0), r);
}

// The same outside of it, kept out of line.
__device__ __noinline__ double inv_root_far(double v) { return 1.0 / sqrt(v); }

// y / scale for eight values, of a scale between 2^-100 and 2^100.
__device__ __forceinline__ void quotients8(const float* y, float scale, float* c) {
  const float inv = __frcp_rn(scale);
#pragma unroll
  for (int k = 0; k < 8; ++k) c[k] = div_by(y[k], scale, inv);
}

// y 448 / amax for eight values of a group with maximum amax; y / scale where
// scale = amax/448 is not a normal number.  One rounding where y is a bf16 value (the
// product with 7/16 is exact, 1024 a power of two), and two such values whose quotient
// is no rounding border of the codes lie 2^-13 of it away from one: the codes are then
// the definition's, ties to even among them.  (y / scale takes the scale's rounding
// along, by which some 45 codes in a million differed.)
__device__ __forceinline__ void quotients8_of_max(const float* y, float amax, float scale,
                                                  float* c) {
  float n[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) n[k] = y[k] * 0.4375f;
  const float d = amax * 0x1p-10f;
  quotients8(n, d, c);
  if (!(d > 0x1p-100f && d < 0x1p+100f)) {
    const bool normal = amax >= 448 * 0x1p-126f;
#pragma unroll
    for (int k = 0; k < 8; ++k) c[k] = normal ? n[k] / amax * 1024.f : y[k] / scale;
  }
}

// Eight fp32 values -> eight E2M1 codes (nearest, ties to even, saturating),
// code 2i in the low nibble of byte i, and the values that the codes stand for
// as f16 pairs (exact), taken from the bytes before they are packed.
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float* v, uint32_t (&h)[4]) {
  uint32_t w;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %8, %7;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %10, %9;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %12, %11;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %4, b3;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(w), "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return w;
}

// E2M1 code pair (low nibble first) -> two fp32 values (exact).
__device__ __forceinline__ float2 e2m1x2_to_float2(uint32_t byte) {
  uint32_t h;
  asm("{\n\t.reg .b8 b0, b1;\n\t"
      "mov.b16 {b0, b1}, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t}"
      : "=r"(h)
      : "h"(static_cast<uint16_t>(byte)));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// E4M3 code pair -> two fp32 values (exact).
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t pair) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(pair)));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// bf16(code * scale) of eight codes, each product rounded once.  kExact: the
// product is exact in fp32 (a code of at most four significand bits times a
// power of two or a four-bit scale).
template <bool kExact>
__device__ __forceinline__ uint4 scaled_bf16x8(const float* c, float scale) {
  float v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = kExact ? c[k] * scale : mul_round_odd(c[k], scale);
  return make_uint4(ptx::pack_bf16x2(v[0], v[1]), ptx::pack_bf16x2(v[2], v[3]),
                    ptx::pack_bf16x2(v[4], v[5]), ptx::pack_bf16x2(v[6], v[7]));
}

__device__ __forceinline__ uint4 pack_bf16x8(const float* y) {
  return make_uint4(ptx::pack_bf16x2(y[0], y[1]), ptx::pack_bf16x2(y[2], y[3]),
                    ptx::pack_bf16x2(y[4], y[5]), ptx::pack_bf16x2(y[6], y[7]));
}

__device__ __forceinline__ void unpack_bf16x8(const uint4 w, float* x) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(u[e] << 16);
    x[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
  }
}

// fp64 -> fp32 rounded to odd: rounding that to nearest in a shorter format gives
// the correctly rounded value of v.
__device__ __forceinline__ float round_odd(double v) {
  const float f = __double2float_rz(v);
  return static_cast<double>(f) != v ? __uint_as_float(__float_as_uint(f) | 1u) : f;
}

// A lane's unit (8 dims) formed in fp64 from the latent.  gain: of the unit, or
// null; rotated: lanes 24.. hold units to rotate, lane l the `turns` of pair l.
// Every lane of the warp calls it.
__device__ __forceinline__ void unit_by_fp64(uint4 raw, const float* gain, double inv, bool rotated,
                                             int position, double turns, double (&y)[8]) {
  const int lane = threadIdx.x & 31;
  float x[8];
  unpack_bf16x8(raw, x);
#pragma unroll
  for (int k = 0; k < 8; ++k) y[k] = gain ? static_cast<double>(x[k]) * gain[k] * inv : x[k];
  if (!rotated) return;
#pragma unroll 1
  for (int k = 0; k < 4; ++k) {
    const double a = position * __shfl_sync(0xffffffffu, turns, (4 * (lane - 24) + k) & 31);
    double s, c;
    sincospi(2.0 * (a - rint(a)), &s, &c);
    if (lane < 24) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e)  // (indexes known to the compiler)
      if (e == k) {
        const double p = y[2 * e], q = y[2 * e + 1];
        y[2 * e] = p * c - q * s;
        y[2 * e + 1] = p * s + q * c;
      }
  }
}

// Its group's maximum magnitude.
template <int kGroupLanes>
__device__ __forceinline__ double amax_by_fp64(const double (&y)[8]) {
  double amax = 0.0;
#pragma unroll
  for (int k = 0; k < 8; ++k) amax = fmax(amax, fabs(y[k]));
#pragma unroll
  for (int o = kGroupLanes / 2; o > 0; o >>= 1)
    amax = fmax(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  return amax;
}

// Rarely called, by a whole warp, and kept out of line: a unit's codes as fp64 has them (E4M3 in .x
// and .y, or E2M1 in .x; scale: as stored, in place of which the 656-byte rows take the
// group's own absmax/448, unrounded, where that is a normal number), and the E4M3 code of
// absmax/6.
template <int kRowBytes>
__device__ __noinline__ uint2 codes_by_fp64(uint4 raw, const float* gain, double inv, bool rotated,
                                            int position, double turns, float scale) {
  double y[8], unit = scale;
  unit_by_fp64(raw, gain, inv, rotated, position, turns, y);
  if constexpr (kRowBytes == kRow656) {
    const double amax = amax_by_fp64<16>(y);
    if (amax >= 448 * 0x1p-126) {
      unit = amax;
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] *= 448.0;
    }
  }
  float c[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) c[k] = round_odd(y[k] / unit);
  if constexpr (kRowBytes == kRow288) {
    uint32_t h[4];
    return make_uint2(cvt_e2m1x8(c, h), 0u);
  } else {
    return make_uint2(cvt_e4m3x4(c[0], c[1], c[2], c[3]), cvt_e4m3x4(c[4], c[5], c[6], c[7]));
  }
}
// Exponent e of the least power of two >= amax/448: amax = m 2^x with 1 <= m < 2 and
// 448 = 1.75 * 2^8, so that e = x - 8, one more where m > 1.75; 0 of a zero group, -127
// at least.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return amax > 0.f ? max(e, -127) : 0;  // at most 127 - 7 for a finite amax
}
// The same of a unit's group (4 lanes) from the latent.
__device__ __noinline__ int scale_exponent_by_fp64(uint4 raw, const float* gain, double inv,
                                                   bool rotated, int position, double turns) {
  double y[8];
  unit_by_fp64(raw, gain, inv, rotated, position, turns, y);
  const double amax = amax_by_fp64<4>(y);
  const unsigned long long bits = __double_as_longlong(amax);
  const int e = static_cast<int>(bits >> 52) - 1023 - 8 +
                ((bits & 0xFFFFFFFFFFFFFull) > 0xC000000000000ull ? 1 : 0);
  return amax > 0.0 ? max(min(e, 127 - 7), -127) : 0;
}
__device__ __noinline__ uint32_t scale_by_fp64(uint4 raw, const float* gain, double inv,
                                               bool rotated, int position, double turns) {
  double y[8];
  unit_by_fp64(raw, gain, inv, rotated, position, turns, y);
  return cvt_e4m3x4(round_odd(amax_by_fp64<2>(y) / 6.0), 0.f, 0.f, 0.f) & 0xFFu;
}

// Rotates the unit's four pairs 4u .. 4u + 3; lane k holds pair k's cos, sin.
// Every lane of the warp calls it (the shuffles); `mine` lanes take the result.
__device__ __forceinline__ void rotate_unit(float* y, int u, bool mine, float cs, float sn) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float c = __shfl_sync(0xffffffffu, cs, (4 * u + e) & 31);
    const float s = __shfl_sync(0xffffffffu, sn, (4 * u + e) & 31);
    const float a = y[2 * e], b = y[2 * e + 1];
    if (mine) {
      y[2 * e] = a * c - b * s;
      y[2 * e + 1] = a * s + b * c;
    }
  }
}

template <int kRowBytes>
__global__ void __launch_bounds__(32 * kAppendWarps, kAppendCtas)
    mla_append_kernel(const AppendParams P) {
  static_assert(kRowBytes == kRow1152 || kRowBytes == kRow656 || kRowBytes == kRow528 ||
                    kRowBytes == kRow288,
                "1152-, 656-, 528- or 288-byte rows");
  constexpr bool kWide = kRowBytes == kRow1152 || kRowBytes == kRow656;  // 576-dim latent
  constexpr int kDim = kWide ? kD : kNope;
  constexpr int kGroupLanes = kRowBytes == kRow656 ? 16 : kRowBytes == kRow528 ? 4 : 2;
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const double turns = P.turns[lane];
  __shared__ __align__(16) float s_gain[kNope];
  if (P.gain) {
    for (int i = threadIdx.x; i < kNope; i += 32 * kAppendWarps) s_gain[i] = __ldg(P.gain + i);
    __syncthreads();
  }

  for (long long t = (long long)blockIdx.x * kAppendWarps + warp; t < P.n;
       t += (long long)gridDim.x * kAppendWarps) {
    const int slot = P.slots[t];
    const int position = P.positions ? P.positions[t] : 0;
    const __nv_bfloat16* src = P.kv + t * P.kv_stride;
    uint4 raw[3];
#pragma unroll
    for (int j = 0; j < 2; ++j)
      raw[j] = *reinterpret_cast<const uint4*>(src + (lane + 32 * j) * 8);
    raw[2] = make_uint4(0, 0, 0, 0);
    if (kWide && lane < 8) raw[2] = *reinterpret_cast<const uint4*>(src + kNope + lane * 8);
    if (slot < 0 || slot >= P.num_slots) {  // no slot: whatever the row holds is not used
      if (slot >= 0 && lane == 0) ptx::set_error(MLA_DEVERR_BAD_INDEX, 0x71);
      continue;
    }
    float cs = 1.f, sn = 0.f;
    if (P.positions) {
      // the angle in turns, its whole turns dropped in fp64, the rest in fp32
      const double a = static_cast<double>(position) * turns;
      sincospif(2.f * static_cast<float>(a - rint(a)), &sn, &cs);
    }
    float y[2][8], yr[8];
#pragma unroll
    for (int j = 0; j < 2; ++j) unpack_bf16x8(raw[j], y[j]);
    unpack_bf16x8(raw[2], yr);

    double inv = 1.0;
    if (P.gain) {
      double s0 = 0.0, s1 = 0.0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {  // the squares are exact in fp64
        const double a = static_cast<double>(y[0][e]), b = static_cast<double>(y[1][e]);
        s0 = fma(a, a, s0);
        s1 = fma(b, b, s1);
      }
      double ss = s0 + s1;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const double v = ss * (1.0 / kNope) + P.eps;
      inv = v > 0x1p-100 && v < 0x1p+100 ? inv_root(v) : inv_root_far(v);
      const float inv_hi = static_cast<float>(inv);
      const float inv_lo = static_cast<float>(inv - static_cast<double>(inv_hi));
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float4* g = reinterpret_cast<const float4*>(s_gain + (lane + 32 * j) * 8);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float4 f = g[e];
          y[j][4 * e] = mul3_once(y[j][4 * e], f.x, inv_hi, inv_lo);
          y[j][4 * e + 1] = mul3_once(y[j][4 * e + 1], f.y, inv_hi, inv_lo);
          y[j][4 * e + 2] = mul3_once(y[j][4 * e + 2], f.z, inv_hi, inv_lo);
          y[j][4 * e + 3] = mul3_once(y[j][4 * e + 3], f.w, inv_hi, inv_lo);
        }
      }
    }
    if (P.positions) {
      if (kWide)
        rotate_unit(yr, lane, lane < 8, cs, sn);  // dims 512..575
      else
        rotate_unit(y[1], lane - 24, lane >= 24, cs, sn);  // dims 448..511
    }

    uint8_t* row = P.cache + static_cast<size_t>(slot) * kRowBytes;
    __nv_bfloat16* out = P.rows ? P.rows + t * kDim : nullptr;
    if constexpr (kRowBytes == kRow1152) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint4 w = pack_bf16x8(y[j]);
        *reinterpret_cast<uint4*>(row + (lane + 32 * j) * 16) = w;
        if (out) *reinterpret_cast<uint4*>(out + (lane + 32 * j) * 8) = w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int u = lane + 32 * j;
        const int group = u / kGroupLanes;
        // Without norm or rotation a dim is exact, and so is its code (and bf16 values
        // often lie on a border); otherwise a quotient within eps of a rounding border
        // is decided in fp64.
        const bool rotated = !kWide && P.positions && j == 1;
        const float eps = rotated && lane >= 24 ? 0x1p-18f : P.gain ? 0x1p-21f : 0.f;
        float more = 1.f + eps, less = 1.f - eps;
        const float* gain = P.gain ? s_gain + u * 8 : nullptr;
        float amax = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(y[j][e]));
#pragma unroll
        for (int o = kGroupLanes / 2; o > 0; o >>= 1)
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        float c[8];
        float scale;
        if constexpr (kRowBytes == kRow528) {
          int e = scale_exponent(amax * more);
          const bool near = e != scale_exponent(amax * less);
          if (__any_sync(0xffffffffu, near)) {
            const int exact = scale_exponent_by_fp64(raw[j], gain, inv, rotated, position, turns);
            if (near) e = exact;
          }
          scale = e8m0_to_float(static_cast<uint32_t>(e + 127));
          const float up = ldexpf(1.f, -e);  // exact: y * 2^-e is y / scale
#pragma unroll
          for (int k = 0; k < 8; ++k) c[k] = y[j][k] * up;
          if (lane % kGroupLanes == 0) row[kNope + group] = static_cast<uint8_t>(e + 127);
        } else if constexpr (kRowBytes == kRow656) {
          scale = amax > 0.f ? amax / 448.f : 1.f;
          if (!(scale > 0.f)) scale = 1.f;  // absmax/448 below the least fp32 value
          quotients8_of_max(y[j], amax, scale, c);
          if (scale < 0x1p-126f) {  // y / scale, rounded
            more = 1.f + 0x1p-21f;
            less = 1.f - 0x1p-21f;
          }
          if (lane % kGroupLanes == 0)
            *reinterpret_cast<float*>(row + kNope + 4 * group) = scale;
        } else {
          const float sixth = div_by(amax, 6.f, 1.f / 6.f);
          const uint32_t both = cvt_e4m3x4(sixth * more, sixth * less, 0.f, 0.f);
          uint32_t code = both & 0xFFu;
          if (__any_sync(0xffffffffu, code != (both >> 8 & 0xFFu)))
            code = scale_by_fp64(raw[j], gain, inv, rotated, position, turns);
          if (code == 0) code = 0x38;  // 1.0, of a zero or tiny group
          scale = e4m3x2_to_float2(code).x;
          quotients8(y[j], scale, c);
          if (lane % kGroupLanes == 0) row[kNope / 2 + group] = static_cast<uint8_t>(code);
        }
        if constexpr (kRowBytes == kRow288) {
          float up[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            up[k] = c[k] * more;
            c[k] *= less;
          }
          uint32_t h[4], other[4];
          uint32_t w = cvt_e2m1x8(up, h);
          const uint32_t near = __ballot_sync(0xffffffffu, w != cvt_e2m1x8(c, other));
          if (near) {
            const uint2 exact = codes_by_fp64<kRowBytes>(
                raw[j], gain, inv, rotated && near >> 24, position, turns, scale);
            if (near >> lane & 1) w = exact.x;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 f = e2m1x2_to_float2((w >> (8 * k)) & 0xFFu);
              const __half2 hv = __floats2half2_rn(f.x, f.y);
              h[k] = *reinterpret_cast<const uint32_t*>(&hv);
            }
          }
          *reinterpret_cast<uint32_t*>(row + u * 4) = w;
          if (out) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[k]));
              c[2 * k] = f.x;
              c[2 * k + 1] = f.y;
            }
            *reinterpret_cast<uint4*>(out + u * 8) = scaled_bf16x8<true>(c, scale);
          }
        } else {
          uint32_t lo = cvt_e4m3x4(c[0] * more, c[1] * more, c[2] * more, c[3] * more);
          uint32_t hi = cvt_e4m3x4(c[4] * more, c[5] * more, c[6] * more, c[7] * more);
          const uint32_t near = __ballot_sync(
              0xffffffffu, lo != cvt_e4m3x4(c[0] * less, c[1] * less, c[2] * less, c[3] * less) ||
                               hi != cvt_e4m3x4(c[4] * less, c[5] * less, c[6] * less, c[7] * less));
          if (near) {
            const uint2 exact = codes_by_fp64<kRowBytes>(
                raw[j], gain, inv, rotated && near >> 24, position, turns, scale);
            if (near >> lane & 1) {
              lo = exact.x;
              hi = exact.y;
            }
          }
          *reinterpret_cast<uint2*>(row + u * 8) = make_uint2(lo, hi);
          if (out) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 f = e4m3x2_to_float2((k < 2 ? lo : hi) >> (16 * (k & 1)));
              c[2 * k] = f.x;
              c[2 * k + 1] = f.y;
            }
            *reinterpret_cast<uint4*>(out + u * 8) = scaled_bf16x8<kRowBytes == kRow528>(c, scale);
          }
        }
      }
    }
    if (kWide && lane < 8) {
      const uint4 w = pack_bf16x8(yr);
      *reinterpret_cast<uint4*>(row + (kRowBytes == kRow1152 ? 2 * kNope : kNope + 16) +
                                lane * 16) = w;
      if (out) *reinterpret_cast<uint4*>(out + kNope + lane * 8) = w;
    }
  }
}

}  // namespace mla
