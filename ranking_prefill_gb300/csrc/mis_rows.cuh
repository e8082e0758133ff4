// Device helpers of the row kernels around the 8-bit cache: rotation angles,
// root mean square norms, and e4m3 codes with a power of two per row.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

namespace mis {
namespace dev {

// Exponents of a quantised row: |x| up to 448 * 2^kQ8MaxExp covers bf16, and
// what lies below 2^(kQ8MinExp - 10) is kept as zero.
constexpr int kQ8MinExp = -56, kQ8MaxExp = 120;

__device__ __forceinline__ void bf16x8_to_float(const uint4& u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// A source row's 16 bytes, read once.
__device__ __forceinline__ uint4 ld_row16(const __nv_bfloat16* ptr) {
  uint4 u;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(ptr));
  return u;
}

// sin and cos of position p times a frequency given as a 64-bit fraction f of
// a turn. p * f modulo 2^64 is the fraction left after whole turns, whatever p.
// Its top bits name the nearest quarter turn, the rest is an angle a in
// [-pi/4, pi/4], kept to 2^-25 of itself, whose sine and cosine are the Taylor
// sums up to a^9 / 9! and a^10 / 10! (the next terms are below 2^-29).
__device__ __forceinline__ void sincos_quarters(int32_t p, uint64_t f, float& sn, float& cs) {
  const uint64_t turn = (uint64_t)(int64_t)p * f;
  const uint64_t near = turn + (1ull << 61);            // half a quarter up
  const int32_t rest = (int32_t)((turn - (near & (3ull << 62))) >> 32);
  const float a = (float)rest * 1.46291807926715968e-9f;   // 2 pi / 2^32
  const float b = a * a;
  const float s = fmaf(a * b, fmaf(b, fmaf(b, fmaf(b, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6), a);
  const float c = fmaf(b, fmaf(b, fmaf(b, fmaf(b, fmaf(b, -1.f / 3628800, 1.f / 40320), -1.f / 720),
                                       1.f / 24), -0.5f), 1.f);
  const uint32_t quarter = (uint32_t)(near >> 62);
  const float u = quarter & 1 ? c : s, v = quarter & 1 ? s : c;
  sn = quarter & 2 ? -u : u;
  cs = (quarter + 1) & 2 ? -v : v;
}

// The N lanes (a power of two, aligned) that share a row, and sums and maxima over
// them
template <int N>
__device__ __forceinline__ uint32_t row_lanes() {
  return N == 32 ? 0xffffffffu : ((1u << N) - 1u) << ((threadIdx.x & 31) & ~(N - 1));
}
// of U values, their exchanges side by side
template <int N, int U>
__device__ __forceinline__ void row_sums(float* x, uint32_t lanes) {
#pragma unroll
  for (int o = N / 2; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < U; ++i) x[i] += __shfl_xor_sync(lanes, x[i], o);
}
template <int N, int U>
__device__ __forceinline__ void row_maxima(float* x, uint32_t lanes) {
#pragma unroll
  for (int o = N / 2; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < U; ++i) x[i] = fmaxf(x[i], __shfl_xor_sync(lanes, x[i], o));
}
template <int N>
__device__ __forceinline__ float row_max(float x, uint32_t lanes) {
  row_maxima<N, 1>(&x, lanes);
  return x;
}

// A lane's 8 + 8 elements of U rows (x: of their first halves, y: of their
// second) times w / sqrt(mean(x^2) + eps). Squares of bf16 leave fp32 at both ends:
// rows whose sum comes near its largest number, or whose mean and eps together are
// that small, are taken 2^-80 or 2^100 times as large first (each row's lanes see
// the same sum; a row that holds infinities or NaN gives the same either way). The
// look costs 0.3 us of 7.2 at 4,099 tokens of 16 heads, nothing that shows at 128K of 24.
template <int D, int U>
__device__ __forceinline__ void norm_rows(float (*x)[8], float (*y)[8], const float* wx, const float* wy, float eps,
                                          uint32_t lanes) {
  float s[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    s[i] = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s[i] = fmaf(x[i][e], x[i][e], fmaf(y[i][e], y[i][e], s[i]));
  }
  row_sums<D / 16, U>(s, lanes);
  bool far = false;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    s[i] = fmaf(s[i], 1.f / D, eps);
    far |= !(s[i] < 1e36f && s[i] > 1e-33f);
  }
  if (__builtin_expect(far, 0)) {
    float t[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const float k = !(s[i] < 1e36f) ? 8.2718061e-25f : s[i] > 1e-33f ? 1.f : 1.2676506e30f;   // 2^-80, 2^100
      t[i] = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[i][e] *= k;
        y[i][e] *= k;
        t[i] = fmaf(x[i][e], x[i][e], fmaf(y[i][e], y[i][e], t[i]));
      }
      s[i] = eps * k * k;
    }
    row_sums<D / 16, U>(t, lanes);
#pragma unroll
    for (int i = 0; i < U; ++i) s[i] = fmaf(t[i], 1.f / D, s[i]);
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const float r = __frsqrt_rn(s[i]);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[i][e] = x[i][e] * r * wx[e];
      y[i][e] = y[i][e] * r * wy[e];
    }
  }
}

__device__ __forceinline__ void rotate_row(float* x, float* y, const float* sn, const float* cs) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float a = x[e], b = y[e];
    x[e] = a * cs[e] - b * sn[e];
    y[e] = b * cs[e] + a * sn[e];
  }
}

// 2^e as fp32, e in [-126, 127].
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// The exponent byte of a row as stored (e + 127), brought into range.
__device__ __forceinline__ int q8_exp(uint32_t byte) {
  return min(max((int)byte - 127, kQ8MinExp), kQ8MaxExp);
}

// Least e in range with a <= 448 * 2^e (448 = 1.75 * 2^8, the largest e4m3).
__device__ __forceinline__ int q8_exp_of(float a) {
  const int bits = __float_as_int(a);
  const int e = (bits >> 23) - 127 - 8 + ((bits & 0x7fffff) > 0x600000);
  return min(max(e, kQ8MinExp), kQ8MaxExp);
}

// Four codes, the first in the lowest byte. NaN gives the NaN code.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | (uint32_t)hi << 16;
}
// Two codes (the low 16 bits) as half floats, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint16_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(codes));
  return h;
}

__device__ __forceinline__ void half2_to_float(uint32_t h, float& lo, float& hi) {
  asm("{.reg .f16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}" : "=f"(lo), "=f"(hi) : "r"(h));
}

}  // namespace dev
}  // namespace mis
