// mx4_quant.cu - rows to microscaled 4 bits and back, and a checkpoint's scales into the
// tensor cores' layout (moe_mx4_quantize, moe_mx4_dequantize, moe_mx4_pack_scales).
//
// Every kernel here moves bytes: per element 2 (bf16) or 4 (fp32) on one side and 0.5 plus the
// block's share of a scale byte on the other, against a dozen instructions. One lane holds 8
// elements (16 bytes of bf16, 4 bytes of codes), so a warp moves 512 contiguous bytes in and
// 128 out; a block's largest magnitude is a butterfly over its 4 (MXFP4) or 2 (NVFP4) lanes,
// and the four scale bytes of a piece's row go out as one word. A warp takes up to 6 steps of
// 256 elements of a row, all their loads in flight at once, and looks for the row's group once for
// them: 32768 rows of 6144 to MXFP4 took 208, 147, 118, 107 and 121 us with 1, 2, 4, 6 and 8 steps.
// The number of steps is the smallest that covers a row in as few warps (6 steps for rows of 768
// leave half of the lanes' work empty: 36 us for 17081 rows instead of 20).
#include "checks.cuh"
#include "kernels.cuh"
#include "launch.cuh"
#include "mx4.cuh"

namespace moe {
namespace {

constexpr int kMaxSteps = 6;                  // 256-element steps of a warp
constexpr int kQuantThreads = 128;

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 q = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
template <>
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                            pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

struct QuantArgs {
  Mx4Rows m;
  const void* x;
  int64_t ld;
  const int32_t* row_of;    // or null: row t of x is row t of m
  int tokens, picks;
  const float* factor;
  int factor_per_group;
  uint8_t* codes;
  uint8_t* scales;
  int* status;
};

// One warp: S steps of 256 elements of one row of x, to one row of m or to the rows of its picks.
template <typename T, bool NV, int S>
__global__ void __launch_bounds__(kQuantThreads) k_mx4_quantize(const QuantArgs q) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * (kQuantThreads / 32) + (threadIdx.x >> 5);
  if (t >= q.tokens) return;
  const int k0 = blockIdx.y * (S * 256);
  const int chunks = q.m.K / (4 * mx4_block(NV));
  // the destinations: lane p holds pick p's row
  int dst = -1;
  if (q.row_of) {
    if (lane < q.picks) dst = q.row_of[(int64_t)t * q.picks + lane];
  } else if (lane == 0) {
    dst = t;
  }
  unsigned left = __ballot_sync(0xffffffffu, dst >= 0);
  if (!left) return;
  const T* src = static_cast<const T*>(q.x) + (int64_t)t * q.ld;
  float v[S][8];
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int k = k0 + s * 256 + lane * 8;
    if (k < q.m.K) {
      load8(src + k, v[s]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[s][i] = 0.f;
    }
  }
  // its group, looked for while the loads are under way: of the row, or of lane p's pick
  int g, o_g = 0, row = t;
  if (q.row_of) {
    g = mx4_find_groups(q.m, dst, o_g);
    if (dst >= 0 && g < 0) set_status(q.status, MOE_ERR_DEVICE_CHECK);
    left = __ballot_sync(0xffffffffu, g >= 0);
  } else {
    g = mx4_find_group(q.m, row, o_g);
    if (g < 0) return;
  }
  const int my_g = g, my_o = o_g;
  const Mx4Factor f = mx4_factor(NV && q.factor ? q.factor[q.factor_per_group ? g : 0] : 1.0f);

  uint32_t code[S], scale[S];
#pragma unroll
  for (int s = 0; s < S; ++s) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max_abs(top, v[s][i]);
#pragma unroll
    for (int o = 1; o < mx4_block(NV) / 8; o <<= 1) top = max_abs(top, __shfl_xor_sync(0xffffffffu, top, o));
    float by;
    const uint32_t byte = mx4_scale<NV>(top, f, by);
    code[s] = mx4_codes<NV>(v[s], by);
    // the four scales of one piece's row, gathered from its 16 (8) lanes into a word
    constexpr int kLanes = mx4_block(NV) / 8;
    uint32_t w = byte << (8 * ((lane / kLanes) & 3));
    w |= __shfl_xor_sync(0xffffffffu, w, kLanes);
    w |= __shfl_xor_sync(0xffffffffu, w, 2 * kLanes);
    scale[s] = w;
  }
  while (left) {
    const int p = __ffs(left) - 1;
    left &= left - 1;
    if (q.row_of) {
      row = __shfl_sync(0xffffffffu, dst, p);
      g = __shfl_sync(0xffffffffu, my_g, p);
      o_g = __shfl_sync(0xffffffffu, my_o, p);
    }
    uint8_t* codes = q.codes + (int64_t)row * (q.m.K / 2);
    constexpr int kPiece = mx4_block(NV) / 2;     // lanes of a piece's row: 4 blocks of 8-element lanes
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int k = k0 + s * 256 + lane * 8;
      if (k < q.m.K) {
        *reinterpret_cast<uint32_t*>(codes + k / 2) = code[s];
        if ((lane & (kPiece - 1)) == 0)
          *reinterpret_cast<uint32_t*>(q.scales + mx4_scale_at(o_g, g, row - o_g, k / mx4_block(NV), chunks)) =
              scale[s];
      }
    }
  }
}

struct DequantArgs {
  Mx4Rows m;
  const float* factor;
  int factor_per_group;
  const uint8_t* codes;
  const uint8_t* scales;
  void* out;
  int64_t ld;
};

// One warp: S steps of one row.
template <typename T, bool NV, int S>
__global__ void __launch_bounds__(kQuantThreads) k_mx4_dequantize(const DequantArgs q) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x * (kQuantThreads / 32) + (threadIdx.x >> 5);
  if (row >= q.m.rows) return;
  const int k0 = blockIdx.y * (S * 256);
  const int chunks = q.m.K / (4 * mx4_block(NV));
  int o_g = 0;
  const int g = mx4_find_group(q.m, row, o_g);
  if (g < 0) return;
  const float f = NV && q.factor ? q.factor[q.factor_per_group ? g : 0] : 1.0f;
  uint32_t code[S], byte[S];
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int k = k0 + s * 256 + lane * 8;
    code[s] = byte[s] = 0;
    if (k < q.m.K) {
      code[s] = *reinterpret_cast<const uint32_t*>(q.codes + (int64_t)row * (q.m.K / 2) + k / 2);
      byte[s] = q.scales[mx4_scale_at(o_g, g, row - o_g, k / mx4_block(NV), chunks)];
    }
  }
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int k = k0 + s * 256 + lane * 8;
    const float sc = NV ? __fmul_rn(e4m3_value(byte[s]), f) : e8m0_value(byte[s]);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // magnitude code m: 0, 0.5, then 1 + half a low bit with exponent m / 2 - 1
      const uint32_t c = code[s] >> (4 * i), m = c & 7u;
      const uint32_t bits = m < 2u ? (m ? 0x3F000000u : 0u) : ((126u + (m >> 1)) << 23) | ((m & 1u) << 22);
      v[i] = __fmul_rn(__uint_as_float(bits | ((c & 8u) << 28)), sc);
    }
    if (k < q.m.K) store8(static_cast<T*>(q.out) + (int64_t)row * q.ld + k, v);
  }
}

// Row-major scale bytes into the pieces: a thread moves the four bytes of a piece's row.
__global__ void __launch_bounds__(256) k_mx4_pack_scales(const Mx4Rows m, int chunks,
                                                         const uint32_t* in, uint8_t* scales) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t warps = (int64_t)gridDim.x * (blockDim.x / 32);
  for (int64_t row = (int64_t)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5); row < m.rows; row += warps) {
    int o_g = 0;
    const int g = mx4_find_group(m, (int)row, o_g);
    if (g < 0) continue;
    for (int c = threadIdx.x & 31; c < chunks; c += 32)
      *reinterpret_cast<uint32_t*>(scales + mx4_scale_at(o_g, g, (int)row - o_g, 4 * c, chunks)) =
          in[row * chunks + c];
  }
}

// The grid of one warp per S steps of each row, and S; MOE_ERR_UNSUPPORTED beyond the grid's limit.
int step_grid(int rows, int K, dim3* grid, int* S) {
  const int steps = (K + 255) / 256;
  const int warps = (steps + kMaxSteps - 1) / kMaxSteps;         // along a row
  *S = (steps + warps - 1) / warps;
  if (*S == 5) *S = 6;                                           // not built
  if (warps > 65535) return MOE_ERR_UNSUPPORTED;
  *grid = dim3((unsigned)((rows + (int64_t)kQuantThreads / 32 - 1) / (kQuantThreads / 32)), (unsigned)warps);
  return MOE_OK;
}

#define MX4_STEPS(KERN, T, NV) \
  (S == 1 ? KERN<T, NV, 1> : S == 2 ? KERN<T, NV, 2> : S == 3 ? KERN<T, NV, 3> : S == 4 ? KERN<T, NV, 4> : KERN<T, NV, 6>)
#define MX4_KERNEL(KERN)                                                                              \
  (dtype == MOE_BF16 ? (is_nv(*m) ? MX4_STEPS(KERN, __nv_bfloat16, true) : MX4_STEPS(KERN, __nv_bfloat16, false)) \
                     : (is_nv(*m) ? MX4_STEPS(KERN, float, true) : MX4_STEPS(KERN, float, false)))

int check_ld(const moe_mx4_t* m, int32_t dtype, int64_t ld) {
  if (dtype != MOE_BF16 && dtype != MOE_FP32) return MOE_ERR_INVALID_ARG;
  if (ld < m->K) return MOE_ERR_INVALID_ARG;
  if (ld * (dtype == MOE_BF16 ? 2 : 4) % 16 != 0) return MOE_ERR_ALIGNMENT;
  return MOE_OK;
}

}  // namespace

int mx4_check(const moe_mx4_t* m) {
  if (!m) return MOE_ERR_INVALID_ARG;
  if (m->format != MOE_MX4_MXFP4 && m->format != MOE_MX4_NVFP4) return MOE_ERR_INVALID_ARG;
  if (m->rows < 0 || m->K <= 0 || m->groups <= 0 || m->group_rows < 0) return MOE_ERR_INVALID_ARG;
  if (m->factor_per_group != 0 && m->factor_per_group != 1) return MOE_ERR_INVALID_ARG;
  if (m->groups > kMx4MaxGroups || m->K % 128 != 0) return MOE_ERR_UNSUPPORTED;
  // (the last tile's coordinates may run on by a tile)
  if (m->rows >= INT32_MAX - 1024 || (int64_t)m->rows * m->K >= (1ll << 46)) return MOE_ERR_UNSUPPORTED;
  if (m->offsets) {
    if (m->group_rows != 0) return MOE_ERR_INVALID_ARG;
    if (!aligned16(m->offsets)) return MOE_ERR_ALIGNMENT;
  } else if ((int64_t)m->groups * m->group_rows != m->rows) {
    return MOE_ERR_INVALID_ARG;
  }
  if (m->format == MOE_MX4_MXFP4 && (m->factor || m->factor_per_group)) return MOE_ERR_INVALID_ARG;
  if (m->factor && (reinterpret_cast<uintptr_t>(m->factor) & 3u)) return MOE_ERR_ALIGNMENT;
  return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" {

int moe_mx4_scale_bytes(const moe_mx4_t* m, size_t* bytes) {
  if (!m || !bytes) return MOE_ERR_INVALID_ARG;
  // ragged or uniform: the size depends on the rows and the number of groups alone
  moe_mx4_t s = *m;
  s.offsets = nullptr;
  s.factor = nullptr;
  s.factor_per_group = 0;
  if (s.group_rows == 0 && s.rows > 0) s.group_rows = s.rows, s.groups = 1;
  MOE_TRY(mx4_check(&s));
  if (m->groups <= 0) return MOE_ERR_INVALID_ARG;
  if (m->groups > kMx4MaxGroups) return MOE_ERR_UNSUPPORTED;
  *bytes = mx4_scale_size(*m);
  return MOE_OK;
}

int moe_mx4_quantize(const moe_mx4_t* m, const void* x, int32_t dtype, int64_t ld,
                     const int32_t* row_of, int32_t tokens, int32_t picks, int32_t* status,
                     void* stream) {
  MOE_TRY(mx4_check(m));
  MOE_TRY(check_ld(m, dtype, ld));
  if (tokens < 0) return MOE_ERR_INVALID_ARG;
  if (row_of) {
    if (picks <= 0 || m->factor_per_group) return MOE_ERR_INVALID_ARG;
    if (picks > 32) return MOE_ERR_UNSUPPORTED;
  } else if (tokens != m->rows) {
    return MOE_ERR_INVALID_ARG;
  }
  if (tokens == 0 || m->rows == 0) return MOE_OK;
  MOE_TRY(check_ptrs({x, m->codes, m->scales}));
  MOE_TRY(check_opt({row_of}));
  QuantArgs q{};
  dim3 grid;
  int S;
  MOE_TRY(step_grid(tokens, m->K, &grid, &S));
  DeviceInfo dev;
  MOE_TRY(current_device_info(&dev));
  q.m = mx4_rows(*m);
  q.x = x;
  q.ld = ld;
  q.row_of = row_of;
  q.tokens = tokens;
  q.picks = picks;
  q.factor = m->factor;
  q.factor_per_group = m->factor_per_group;
  q.codes = static_cast<uint8_t*>(m->codes);
  q.scales = static_cast<uint8_t*>(m->scales);
  q.status = status;
  auto kern = MX4_KERNEL(k_mx4_quantize);
  const cudaError_t e = launch_kernel(kern, grid, kQuantThreads, 0, as_stream(stream), 1, q);
  count_launch();
  return cuda_rc(e);
}

int moe_mx4_dequantize(const moe_mx4_t* m, void* out, int32_t dtype, int64_t ld, void* stream) {
  MOE_TRY(mx4_check(m));
  MOE_TRY(check_ld(m, dtype, ld));
  if (m->rows == 0) return MOE_OK;
  MOE_TRY(check_ptrs({out, m->codes, m->scales}));
  dim3 grid;
  int S;
  MOE_TRY(step_grid(m->rows, m->K, &grid, &S));
  DeviceInfo dev;
  MOE_TRY(current_device_info(&dev));
  DequantArgs q{};
  q.m = mx4_rows(*m);
  q.factor = m->factor;
  q.factor_per_group = m->factor_per_group;
  q.codes = static_cast<const uint8_t*>(m->codes);
  q.scales = static_cast<const uint8_t*>(m->scales);
  q.out = out;
  q.ld = ld;
  auto kern = MX4_KERNEL(k_mx4_dequantize);
  const cudaError_t e = launch_kernel(kern, grid, kQuantThreads, 0, as_stream(stream), 1, q);
  count_launch();
  return cuda_rc(e);
}

int moe_mx4_pack_scales(const moe_mx4_t* m, const void* row_major, void* stream) {
  MOE_TRY(mx4_check(m));
  if (m->rows == 0) return MOE_OK;
  MOE_TRY(check_ptrs({row_major, m->scales}));
  DeviceInfo dev;
  MOE_TRY(current_device_info(&dev));
  const int chunks = m->K / (4 * mx4_block(is_nv(*m)));
  const unsigned grid = (unsigned)min((m->rows + 7ll) / 8, (long long)dev.sm_count * 8);
  const cudaError_t e = launch_kernel(k_mx4_pack_scales, grid, 256, 0, as_stream(stream), 1, mx4_rows(*m),
                                      chunks, static_cast<const uint32_t*>(row_major),
                                      static_cast<uint8_t*>(m->scales));
  count_launch();
  return cuda_rc(e);
}

}  // extern "C"
