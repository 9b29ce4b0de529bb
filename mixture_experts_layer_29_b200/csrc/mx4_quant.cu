// mx4_quant.cu - rows to microscaled 4 bits and back, and a checkpoint's scales into the
// tensor cores' layout (moe_mx4_quantize, moe_mx4_dequantize, moe_mx4_pack_scales).
//
// Every kernel here moves bytes: per element 2 (bf16) or 4 (fp32) on one side and 0.5 plus the block's
// share of a scale byte on the other, against a few instructions, and both sides have to be kept low.
//  * quantise: a lane holds 16 elements (32 bytes of bf16 in one load, 8 bytes of codes), which are an
//    NVFP4 block, or half of an MXFP4 one whose largest magnitude takes one shuffle; the four scale
//    bytes of a piece's row go out as one word. With 8 elements per lane twice as many lanes worked out
//    each scale: 8192 rows of 6144 to NVFP4 took 35.6 us instead of 26.6 (4.8 TB/s), 32768 to MXFP4 89
//    instead of 76 (6.6 TB/s, the card's copy rate). A warp takes up to 3 steps of 512 elements of a row
//    (4 steps: 2 % less for the latter, nothing for the former, and 2.24 us instead of 2.05 for 128 rows), all their loads in flight at
//    once, and looks for the row's group once for them.
//  * dequantise: 8 elements per lane, up to 6 steps of 256 elements per warp (23 us for 8192 rows of
//    6144 from NVFP4; 33.5 with the values made by integer operations instead of conversions).
// The number of steps is the smallest that covers a row in as few warps.
#include "checks.cuh"
#include "kernels.cuh"
#include "launch.cuh"
#include "mx4.cuh"

namespace moe {
namespace {

constexpr int kQuantSteps = 3;                // of a warp, of 512 elements
constexpr int kDequantSteps = 6;              // of 256
constexpr int kQuantThreads = 128;

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                            pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// 16 elements as they are in memory: 32 bytes in one load where they are aligned to that, else in two.
template <typename T>
struct Sixteen {
  uint4 q[sizeof(T)];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) q[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void load(const T* p, bool wide) {
    const uint4* s = reinterpret_cast<const uint4*>(p);
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); i += 2) {
      if (wide) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(q[i].x), "=r"(q[i].y), "=r"(q[i].z), "=r"(q[i].w), "=r"(q[i + 1].x), "=r"(q[i + 1].y),
                       "=r"(q[i + 1].z), "=r"(q[i + 1].w)
                     : "l"(s + i));
      } else {
        q[i] = s[i];
        q[i + 1] = s[i + 1];
      }
    }
  }
  // elements 8 h to 8 h + 7
  __device__ __forceinline__ void half(int h, float (&v)[8]) const {
    if constexpr (sizeof(T) == 2) {
      const uint32_t w[4] = {q[h].x, q[h].y, q[h].z, q[h].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4& a = q[2 * h + i];
        v[4 * i] = __uint_as_float(a.x);
        v[4 * i + 1] = __uint_as_float(a.y);
        v[4 * i + 2] = __uint_as_float(a.z);
        v[4 * i + 3] = __uint_as_float(a.w);
      }
    }
  }
};

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
  bool wide;                // rows of x are 32-byte aligned
};

// One warp: S steps of 512 elements of one row of x, to one row of m or to the rows of its picks.
template <typename T, bool NV, int S>
__global__ void __launch_bounds__(kQuantThreads) k_mx4_quantize(const QuantArgs q) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * (kQuantThreads / 32) + (threadIdx.x >> 5);
  if (t >= q.tokens) return;
  const int k0 = blockIdx.y * (S * 512);
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
  Sixteen<T> v[S];
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int k = k0 + s * 512 + lane * 16;
    if (k < q.m.K) v[s].load(src + k, q.wide);
    else v[s].clear();
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

  constexpr int kLanes = mx4_block(NV) / 16;      // of a block
  uint2 code[S];
  uint32_t scale[S];
#pragma unroll
  for (int s = 0; s < S; ++s) {
    float a[8], b[8];
    v[s].half(0, a);
    v[s].half(1, b);
    float top = max_abs(max_abs(a[0], a[1], a[2]), a[3], a[4]);
    top = max_abs(max_abs(top, a[5], a[6]), a[7], b[0]);
    top = max_abs(max_abs(top, b[1], b[2]), b[3], b[4]);
    top = max_abs(max_abs(top, b[5], b[6]), b[7]);
    if (kLanes == 2) top = max_abs(top, __shfl_xor_sync(0xffffffffu, top, 1));
    float by;
    const uint32_t byte = mx4_scale<NV>(top, f, by);
    code[s] = make_uint2(mx4_codes<NV>(a, by, top), mx4_codes<NV>(b, by, top));
    // the four scales of one piece's row, gathered from its 8 (4) lanes into a word
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
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int k = k0 + s * 512 + lane * 16;
      if (k < q.m.K) {
        *reinterpret_cast<uint2*>(codes + k / 2) = code[s];
        if ((lane & (4 * kLanes - 1)) == 0)
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
    e2m1x8_values(code[s], v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(v[i], sc);
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

// The grid of one warp per S steps (at most most, of `step` elements) of each row, and S;
// MOE_ERR_UNSUPPORTED beyond the grid's limit.
int step_grid(int rows, int K, int step, int most, dim3* grid, int* S) {
  const int steps = (K + step - 1) / step;
  const int warps = (steps + most - 1) / most;                   // along a row
  *S = (steps + warps - 1) / warps;
  if (*S == 5) *S = 6;                                           // not built
  if (warps > 65535) return MOE_ERR_UNSUPPORTED;
  *grid = dim3((unsigned)((rows + (int64_t)kQuantThreads / 32 - 1) / (kQuantThreads / 32)), (unsigned)warps);
  return MOE_OK;
}

#define MX4_QUANT(T, NV) \
  (S == 1 ? k_mx4_quantize<T, NV, 1> : S == 2 ? k_mx4_quantize<T, NV, 2> : k_mx4_quantize<T, NV, 3>)
#define MX4_DEQUANT(T, NV)                                                                                   \
  (S == 1 ? k_mx4_dequantize<T, NV, 1> : S == 2 ? k_mx4_dequantize<T, NV, 2> : S == 3 ? k_mx4_dequantize<T, NV, 3> \
   : S == 4 ? k_mx4_dequantize<T, NV, 4> : k_mx4_dequantize<T, NV, 6>)
#define MX4_KERNEL(WHICH)                                                              \
  (dtype == MOE_BF16 ? (is_nv(*m) ? WHICH(__nv_bfloat16, true) : WHICH(__nv_bfloat16, false)) \
                     : (is_nv(*m) ? WHICH(float, true) : WHICH(float, false)))

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
  if (reinterpret_cast<uintptr_t>(status) & 3u) return MOE_ERR_ALIGNMENT;
  QuantArgs q{};
  dim3 grid;
  int S;
  MOE_TRY(step_grid(tokens, m->K, 512, kQuantSteps, &grid, &S));
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
  q.wide = (reinterpret_cast<uintptr_t>(x) | (uintptr_t)(ld * (dtype == MOE_BF16 ? 2 : 4))) % 32 == 0;
  auto kern = MX4_KERNEL(MX4_QUANT);
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
  MOE_TRY(step_grid(m->rows, m->K, 256, kDequantSteps, &grid, &S));
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
  auto kern = MX4_KERNEL(MX4_DEQUANT);
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
