// mx4.cuh - the microscaled 4-bit formats on the device and the host: block scales, e2m1
// rounding, the scale layout, and the description of a 4-bit matrix that the kernels take.
#pragma once

#include <cuda_fp16.h>

#include "../../include/moe_mx4.h"
#include "common.cuh"

namespace moe {

constexpr int kMx4MaxGroups = 1024;

// elements that share a scale
__host__ __device__ constexpr int mx4_block(bool nv) { return nv ? 16 : 32; }

// A 4-bit matrix as the kernels see it (moe_mx4_t without the buffers).
struct Mx4Rows {
  const int32_t* offsets;   // ragged groups, or null
  int rows, K, groups, group_rows;

  __device__ __forceinline__ int begin(int g) const { return offsets ? offsets[g] : g * group_rows; }
};

// Byte offset of the scale of block b in row l of the group that starts at row o_g: pieces of
// 128 rows x 4 blocks, 512 bytes each, as tcgen05.cp hands them to the tensor cores (32 lanes
// of 16 bytes: lane l % 32 holds the four scales of its rows l % 32 + 0, 32, 64, 96).
// `chunks` is the number of pieces along K.
__device__ __forceinline__ size_t mx4_scale_at(int o_g, int g, int l, int b, int chunks) {
  const size_t tile = (size_t)(o_g >> 7) + g + (l >> 7);
  return (tile * chunks + (b >> 2)) * 512 + (l & 31) * 16 + ((l & 127) >> 5) * 4 + (b & 3);
}

// Group of row r, for a whole warp with one r: the groups' starts are searched 32 at a time.
// -1 when no group has the row. Returns the group's first row in o_g.
__device__ __forceinline__ int mx4_find_group(const Mx4Rows& m, int r, int& o_g) {
  if (r >= m.rows) return -1;
  if (!m.offsets) {
    const int g = r / m.group_rows;
    o_g = g * m.group_rows;
    return g;
  }
  // the last start that is <= r; empty groups share their start with the next one
  const int lane = threadIdx.x & 31;
  int lo = 0, n = m.groups + 1;         // starts [lo, lo + n) are candidates
  while (n > 32) {
    const int step = (n + 31) / 32;
    const int at = lo + lane * step;
    const unsigned le = __ballot_sync(0xffffffffu, lane * step < n && m.offsets[at] <= r);
    if (!le) return -1;
    const int k = 31 - __clz(le);
    lo += k * step;
    n = min(step, n - k * step);
  }
  const unsigned le = __ballot_sync(0xffffffffu, lane < n && m.offsets[lo + min(lane, n - 1)] <= r);
  if (!le) return -1;
  const int g = lo + 31 - __clz(le);
  if (g >= m.groups) return -1;
  o_g = max(m.offsets[g], 0);
  return g;
}

// Groups of 32 rows at once, lane l's row r (negative: none): 32 starts that all lanes load together,
// then each lane's own search between two of them. For a token's picks, whose rows lie anywhere: one
// after the other they took 7 us of a single token's 10 us.
__device__ __forceinline__ int mx4_find_groups(const Mx4Rows& m, int r, int& o_g) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = m.groups + 1;
  const int step = (n + 31) / 32;
  const int start = lane * step < n ? m.begin(lane * step) : INT32_MAX;
  int k = 0;
#pragma unroll
  for (int s = 16; s > 0; s >>= 1)
    if (__shfl_sync(0xffffffffu, start, k + s) <= r) k += s;
  lo = k * step;
  n = min(step, n - lo);
  if (r < 0 || r >= m.rows) return -1;
  while (n > 1) {               // starts [lo, lo + n), the first one <= r
    const int half = n / 2;
    if (m.begin(lo + half) <= r) {
      lo += half;
      n -= half;
    } else {
      n = half;
    }
  }
  o_g = max(m.begin(lo), 0);
  return lo < m.groups && m.begin(lo) <= r ? lo : -1;
}

// Two floats -> two e2m1 numbers in a byte (a in the low half), nearest even, at most 6.
__device__ __forceinline__ uint32_t e2m1x2(float a, float b) {
  uint32_t r;
  asm("{\n\t.reg .b8 q;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 q, %2, %1;\n\t"
      "cvt.u32.u8 %0, q;\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b));
  return r;
}

// Eight of them, the first in the low bits.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}
// The values of eight codes.
__device__ __forceinline__ void e2m1x8_values(uint32_t code, float (&v)[8]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(code));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

// Nearest e4m3 number of a non-negative float, at most 448; NaN for a NaN.
__device__ __forceinline__ uint32_t e4m3(float a) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(a));
  return r & 0xFFu;
}
__device__ __forceinline__ float e4m3_value(uint32_t byte) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)byte));
  __half_raw v;
  v.x = (unsigned short)(h & 0xFFFFu);
  return __half2float(__half(v));
}
// 2^(byte - 127); 255 is NaN
__device__ __forceinline__ float e8m0_value(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7FC00000u : byte ? byte << 23 : 1u << 22);
}

// max(a, |b|) of non-negative a, NaN if either is one.
__device__ __forceinline__ float max_abs(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
  return r;
}

// The same of |a|, |b| and |c|.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The correctly rounded quotient x / d from r, the correctly rounded reciprocal of d: with t = x r it
// is t + r (x - t d) (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990) while nothing underflows. 3 operations for a division's dozen.
__device__ __forceinline__ float quotient(float x, float d, float r) {
  const float t = __fmul_rn(x, r);
  return __fmaf_rn(r, __fmaf_rn(-t, d, x), t);
}
// d for which quotient() is good while |x / d| is below 2^66 or so: an x so small beside d that x - t d
// underflows has a quotient below 2^-40, which rounds to 0 on every grid here. (A larger x would make
// x r infinite, and the correction of that a NaN.)
__device__ __forceinline__ bool quotient_ok(float d) { return d >= 0x1p-60f && d <= 0x1p60f; }

// t of an NVFP4 matrix with what its scales are made with.
struct Mx4Factor {
  float t, six, r;         // t, 6 t, 1 / (6 t)
};
__device__ __forceinline__ Mx4Factor mx4_factor(float t) {
  const float six = __fmul_rn(6.0f, t);
  return Mx4Factor{t, six, __frcp_rn(six)};
}

// A block's scale byte, and what its elements are divided (NVFP4) or multiplied (MXFP4) by before
// rounding, from the block's largest magnitude. `by` is 0 where every element becomes 0: an empty
// NVFP4 block, or a block without a finite scale.
template <bool NV>
__device__ __forceinline__ uint32_t mx4_scale(float amax, const Mx4Factor& f, float& by) {
  const uint32_t bits = __float_as_uint(amax);
  by = 0.f;
  if (NV) {
    if (bits >= 0x7F800000u) return 0x7Fu;
    // 448 is the largest scale: every quotient from there on gives it, the quotients' own range ends nowhere
    const float a = fminf(amax, 512.0f * f.six);
    const uint32_t s = e4m3(quotient_ok(f.six) ? quotient(a, f.six, f.r) : __fdiv_rn(a, f.six));
    by = __fmul_rn(e4m3_value(s), f.t);
    return s;
  }
  const uint32_t e = bits >> 23;
  if (e == 255u) return 255u;
  const uint32_t b = e > 2u ? e - 2u : 0u;
  by = __uint_as_float((254u - b) << 23);
  return b;
}
// The codes of 4 or 8 elements of a block (the first in the low bits) whose largest magnitude is amax.
template <bool NV, int N>
__device__ __forceinline__ uint32_t mx4_codes(const float (&x)[N], float by, float amax) {
  float q[N];
  // a block of zeros must not end in the divisions (17081 rows of 768, a quarter of whose lanes have
  // none, took 22 us instead of 10)
  const float d = by != 0.f ? by : 1.0f;
  if (!NV) {
    const uint64_t s = pack_f32x2(d, d);
#pragma unroll
    for (int i = 0; i < N; i += 2) unpack_f32x2(mul_f32x2(pack_f32x2(x[i], x[i + 1]), s), q[i], q[i + 1]);
  } else if (quotient_ok(d) && amax <= 0x1p66f * d) {
    const float r = __frcp_rn(d);
    const uint64_t r2 = pack_f32x2(r, r), minus = pack_f32x2(-d, -d);
#pragma unroll
    for (int i = 0; i < N; i += 2) {       // quotient() of two elements at once
      const uint64_t v = pack_f32x2(x[i], x[i + 1]), n = mul_f32x2(v, r2);
      unpack_f32x2(fma_f32x2(r2, fma_f32x2(n, minus, v), n), q[i], q[i + 1]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = __fdiv_rn(x[i], d);   // infinite past the range: at most 6
  }
  uint32_t c;
  if constexpr (N == 8) c = e2m1x8(q);
  else c = e2m1x2(q[0], q[1]) | e2m1x2(q[2], q[3]) << 8;
  return by != 0.f ? c : 0u;
}

// ---- host side -------------------------------------------------------------------------------
// Checks a matrix's sizes (MOE_OK or an error).
int mx4_check(const moe_mx4_t* m);
inline bool is_nv(const moe_mx4_t& m) { return m.format == MOE_MX4_NVFP4; }
inline size_t mx4_scale_tiles(const moe_mx4_t& m) { return (size_t)(m.rows / 128) + m.groups; }
inline size_t mx4_scale_size(const moe_mx4_t& m) {
  return mx4_scale_tiles(m) * (m.K / (4 * mx4_block(is_nv(m)))) * 512;
}
inline Mx4Rows mx4_rows(const moe_mx4_t& m) {
  return Mx4Rows{m.offsets, m.rows, m.K, m.groups, m.group_rows};
}

}  // namespace moe
