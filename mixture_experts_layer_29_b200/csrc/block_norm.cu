// block_norm.cu - the norm after a block, its gate and residual scale, the residual add and the
// norm before the next block in one pass, and the gradients (moe_block_norm,
// moe_block_norm_backward).
//
//   n1 = w_post * b * rb          rb = rstd(b)
//   r  = res + s * gate * n1      rounded to the stream's type
//   n2 = w_pre * r * rr           rr = rstd(r) of the rounded r
// Backward, with c = d_n2 * w_pre, rhat = r rr, bhat = b rb:
//   g   = d_r + rr (c - rhat <c, rhat> / H)          d_res = g
//   dn1 = s gate g,  c' = dn1 * w_post,  d_b = rb (c' - bhat <c', bhat> / H)
//   d_gate = s sum g n1,  d_w_post = sum_t dn1 bhat,  d_w_pre = sum_t d_n2 rhat
//
// Bound by memory: 4 rows of H elements in and out per token forward, 6 backward, against some
// 10 and 22 flops per element. One CTA holds a token's row in registers (16-byte vectors), so
// each array is read once; the two norms are two block reductions in a row, the second on what
// the first produced. Forward: one CTA per token. Backward: persistent CTAs, so that the sums
// over tokens (d_w_post, d_w_pre, d_gate per channel) stay in registers; each CTA writes its
// partial sums once and a second kernel adds them in order (no atomics: bit-reproducible).
#include "checks.cuh"
#include "kernels.cuh"
#include "launch.cuh"

#include "../../include/moe_norm.h"
#include "common.cuh"

namespace moe {
namespace {

constexpr int kMaxH = 16384;

template <typename T>
struct Row;      // 16 bytes of a row
template <>
struct Row<__nv_bfloat16> {
  static constexpr int N = 8;
  __device__ static __forceinline__ void unpack(const uint4& q, float (&v)[8]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ static __forceinline__ uint4 pack(const float (&v)[8]) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
  }
};
template <>
struct Row<float> {
  static constexpr int N = 4;
  __device__ static __forceinline__ void unpack(const uint4& q, float (&v)[4]) {
    v[0] = __uint_as_float(q.x); v[1] = __uint_as_float(q.y);
    v[2] = __uint_as_float(q.z); v[3] = __uint_as_float(q.w);
  }
  __device__ static __forceinline__ uint4 pack(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                      __float_as_uint(v[3]));
  }
};

__device__ __forceinline__ float warp_sum_f(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Sum over the block, the same bits in every thread. `part` holds one float per warp (two
// calls in a row use two arrays).
__device__ __forceinline__ float block_sum(float v, float* part) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = (blockDim.x + 31) >> 5;
  v = warp_sum_f(v);
  if (lane == 0) part[warp] = v;
  __syncthreads();
  return warp_sum_f(lane < warps ? part[lane] : 0.f);
}

struct FwdArgs {
  int H, gate;
  float eps, scale;
  const void *residual, *block;
  const float *w_post, *g, *w_pre;
  void *residual_out, *normed;
  float *rstd_block, *rstd_res;
};

__device__ __forceinline__ float rstd_of(float sum_sq, int H, float eps) {
  return 1.0f / sqrtf(sum_sq / (float)H + eps);
}

// fp32 parameters of the 16-byte vector at column c
template <int N>
__device__ __forceinline__ void load_param(const float* p, int c, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const float4 q = *reinterpret_cast<const float4*>(p + c + i);
    v[i] = q.x; v[i + 1] = q.y; v[i + 2] = q.z; v[i + 3] = q.w;
  }
}

// VPT vectors per thread, strided by the block so that a warp's loads are contiguous.
template <typename T, int VPT>
__global__ void __launch_bounds__(1024) k_block_norm(const FwdArgs a) {
  constexpr int N = Row<T>::N;
  __shared__ float part[2][32];
  pdl_launch_dependents();
  pdl_wait();
  const size_t t = blockIdx.x;
  const int nvec = a.H / N;
  const uint4* res = reinterpret_cast<const uint4*>(static_cast<const T*>(a.residual) + t * a.H);
  float r[VPT][N];
  if (a.block) {
    const uint4* blk = reinterpret_cast<const uint4*>(static_cast<const T*>(a.block) + t * a.H);
    uint4 rq[VPT];
    float b[VPT][N], sq = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      const uint4 q = v < nvec ? blk[v] : make_uint4(0, 0, 0, 0);
      rq[i] = v < nvec ? res[v] : make_uint4(0, 0, 0, 0);
      Row<T>::unpack(q, b[i]);
    }
    float rb = 1.0f;
    if (a.w_post) {
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) sq = fmaf(b[i][j], b[i][j], sq);
      rb = rstd_of(block_sum(sq, part[0]), a.H, a.eps);
      if (a.rstd_block && threadIdx.x == 0) a.rstd_block[t] = rb;
    }
    const float gt = a.scale * (a.gate == MOE_GATE_TOKEN ? a.g[t] : 1.0f);
    uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(a.residual_out) + t * a.H);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      Row<T>::unpack(rq[i], r[i]);
      if (v >= nvec) continue;
      float w[N], gc[N];
#pragma unroll
      for (int j = 0; j < N; ++j) w[j] = gc[j] = 1.0f;
      if (a.w_post) load_param(a.w_post, v * N, w);
      if (a.gate == MOE_GATE_CHANNEL) load_param(a.g, v * N, gc);
#pragma unroll
      for (int j = 0; j < N; ++j) r[i][j] = fmaf(gt * gc[j], b[i][j] * rb * w[j], r[i][j]);
      const uint4 q = Row<T>::pack(r[i]);
      out[v] = q;
      Row<T>::unpack(q, r[i]);       // the next norm reads the stream as it is stored
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      Row<T>::unpack(v < nvec ? res[v] : make_uint4(0, 0, 0, 0), r[i]);
    }
  }
  if (!a.w_pre) return;
  float sq = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) sq = fmaf(r[i][j], r[i][j], sq);
  const float rr = rstd_of(block_sum(sq, part[1]), a.H, a.eps);
  if (a.rstd_res && threadIdx.x == 0) a.rstd_res[t] = rr;
  uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(a.normed) + t * a.H);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v >= nvec) continue;
    float w[N];
    load_param(a.w_pre, v * N, w);
#pragma unroll
    for (int j = 0; j < N; ++j) r[i][j] = r[i][j] * rr * w[j];
    out[v] = Row<T>::pack(r[i]);
  }
}

struct BwdArgs {
  int T, H, gate;
  float scale;
  const void *d_res_out, *d_normed, *res_out, *block;
  const float *w_post, *g, *w_pre, *rstd_block, *rstd_res;
  void *d_residual, *d_block;
  float* d_gate;         // per token: written here; per channel: through the partial sums
  float* partial;        // [grid, 3, H]: d_w_post, d_w_pre, d_gate (the parts that exist)
};

// A token's rows as they are loaded.
template <int VPT>
struct RawRows {
  uint4 d[VPT], n[VPT], r[VPT], b[VPT];
  float rr, rb;
};
template <typename T, int VPT>
__device__ __forceinline__ void load_rows(const BwdArgs& a, size_t t, int nvec, RawRows<VPT>& q) {
  const size_t o = t * a.H;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const auto vec = [&](const void* p, int v) { return reinterpret_cast<const uint4*>(static_cast<const T*>(p) + o)[v]; };
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    const bool in = v < nvec;
    q.n[i] = in && a.w_pre ? vec(a.d_normed, v) : zero;
    q.r[i] = in && a.w_pre ? vec(a.res_out, v) : zero;
    q.d[i] = in && a.d_res_out ? vec(a.d_res_out, v) : zero;
    q.b[i] = in && a.block ? vec(a.block, v) : zero;
  }
  q.rr = a.w_pre ? a.rstd_res[t] : 0.f;
  q.rb = a.w_post ? a.rstd_block[t] : 1.f;
}

// MAXT: most threads of a CTA. A CTA of a wide row has an SM to itself (its sums take 24 registers per
// 8 columns), so it loads the next token's rows before it works on the ones it has.
template <typename T, int VPT, int MAXT>
__global__ void __launch_bounds__(MAXT) k_block_norm_bwd(const BwdArgs a) {
  constexpr int N = Row<T>::N;
  __shared__ float part[2][32];
  pdl_launch_dependents();
  pdl_wait();
  const int nvec = a.H / N;
  const bool chan = a.block && a.gate == MOE_GATE_CHANNEL;
  float sw_post[VPT][N], sw_pre[VPT][N], s_gate[VPT][N];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) sw_post[i][j] = sw_pre[i][j] = s_gate[i][j] = 0.f;

  RawRows<VPT> q;
  if (blockIdx.x < (unsigned)a.T) load_rows<T, VPT>(a, blockIdx.x, nvec, q);
  for (size_t t = blockIdx.x; t < (size_t)a.T; t += gridDim.x) {
    const size_t o = t * a.H;
    uint4 qd[VPT], qb[VPT];
    float g[VPT][N], rhat[VPT][N], sum = 0.f;
    const float rr = q.rr, rb = q.rb;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      Row<T>::unpack(q.n[i], g[i]);
      Row<T>::unpack(q.r[i], rhat[i]);
      qd[i] = q.d[i];
      qb[i] = q.b[i];
    }
    if (t + gridDim.x < (size_t)a.T) load_rows<T, VPT>(a, t + gridDim.x, nvec, q);
    if (a.w_pre) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v >= nvec) continue;
        float w[N];
        load_param(a.w_pre, v * N, w);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          rhat[i][j] *= rr;
          sw_pre[i][j] = fmaf(g[i][j], rhat[i][j], sw_pre[i][j]);
          g[i][j] *= w[j];                                  // c
          sum = fmaf(g[i][j], rhat[i][j], sum);
        }
      }
      sum = block_sum(sum, part[0]) / (float)a.H;
    }
    // g: the gradient of the residual stream
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      float d[N];
      Row<T>::unpack(qd[i], d);
#pragma unroll
      for (int j = 0; j < N; ++j) g[i][j] = fmaf(rr, g[i][j] - rhat[i][j] * sum, d[j]);
      if (v < nvec) reinterpret_cast<uint4*>(static_cast<T*>(a.d_residual) + o)[v] = Row<T>::pack(g[i]);
    }
    if (!a.block) {
      __syncthreads();                                      // part[0] is free again
      continue;
    }
    // bhat in rhat's registers; c' in g's
    const float gt = a.scale * (a.gate == MOE_GATE_TOKEN ? a.g[t] : 1.0f);
    float dot = 0.f;                                        // <g w_post gate_c, bhat>
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      Row<T>::unpack(qb[i], rhat[i]);
      if (v >= nvec) continue;
      float w[N], gc[N];
#pragma unroll
      for (int j = 0; j < N; ++j) w[j] = gc[j] = 1.0f;
      if (a.w_post) load_param(a.w_post, v * N, w);
      if (chan) load_param(a.g, v * N, gc);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float bhat = rhat[i][j] * rb;
        rhat[i][j] = bhat;
        if (chan) s_gate[i][j] = fmaf(g[i][j], bhat * w[j], s_gate[i][j]);
        sw_post[i][j] = fmaf(gt * gc[j] * g[i][j], bhat, sw_post[i][j]);
        g[i][j] *= w[j] * gc[j];
        dot = fmaf(g[i][j], bhat, dot);
      }
    }
    float mean = 0.f;
    if (a.w_post || a.gate == MOE_GATE_TOKEN) {
      dot = block_sum(dot, part[1]);
      if (a.gate == MOE_GATE_TOKEN && threadIdx.x == 0) a.d_gate[t] = a.scale * dot;
      if (a.w_post) mean = dot / (float)a.H;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
#pragma unroll
      for (int j = 0; j < N; ++j) g[i][j] = gt * rb * (g[i][j] - rhat[i][j] * mean);
      if (v < nvec) reinterpret_cast<uint4*>(static_cast<T*>(a.d_block) + o)[v] = Row<T>::pack(g[i]);
    }
    __syncthreads();                                        // both partial arrays are free again
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v >= nvec) continue;
    float* p = a.partial + (size_t)blockIdx.x * 3 * a.H + v * N;
#pragma unroll
    for (int j = 0; j < N; j += 4) {
      if (a.w_post)
        *reinterpret_cast<float4*>(p + j) = make_float4(sw_post[i][j], sw_post[i][j + 1], sw_post[i][j + 2], sw_post[i][j + 3]);
      if (a.w_pre)
        *reinterpret_cast<float4*>(p + a.H + j) = make_float4(sw_pre[i][j], sw_pre[i][j + 1], sw_pre[i][j + 2], sw_pre[i][j + 3]);
      if (chan)
        *reinterpret_cast<float4*>(p + 2 * a.H + j) =
            make_float4(a.scale * s_gate[i][j], a.scale * s_gate[i][j + 1], a.scale * s_gate[i][j + 2], a.scale * s_gate[i][j + 3]);
    }
  }
}

// out[k][c] = sum over the CTAs' partial sums, for the arrays that are wanted: 32 columns per block,
// whose 32 warps share the CTAs; each warp adds its ones in order, then the warps' sums in order.
__global__ void __launch_bounds__(1024) k_block_norm_sum(const float* partial, int n, int H, float* w_post,
                                                         float* w_pre, float* gate) {
  pdl_launch_dependents();
  pdl_wait();
  float* out = blockIdx.y == 0 ? w_post : blockIdx.y == 1 ? w_pre : gate;
  if (!out) return;
  __shared__ float part[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < H) {
#pragma unroll 4
    for (int i = warp; i < n; i += 32) s += partial[((size_t)i * 3 + blockIdx.y) * H + c];
  }
  part[lane][warp] = s;
  __syncthreads();
  // warp w adds up column w
  const float v = warp_sum_f(part[warp][lane]);
  if (lane == 0 && blockIdx.x * 32 + warp < H) out[blockIdx.x * 32 + warp] = v;
}

int check_norm(const moe_norm_t* n) {
  if (!n) return MOE_ERR_INVALID_ARG;
  if (n->T < 0 || n->H <= 0) return MOE_ERR_INVALID_ARG;
  if (n->dtype != MOE_BF16 && n->dtype != MOE_FP32) return MOE_ERR_INVALID_ARG;
  if (n->gate < MOE_GATE_NONE || n->gate > MOE_GATE_CHANNEL) return MOE_ERR_INVALID_ARG;
  if (!(n->eps > 0.f) || n->eps > 3.4e38f || !(n->scale - n->scale == 0.f)) return MOE_ERR_INVALID_ARG;
  if (n->H % 16 != 0 || n->H > kMaxH || n->T >= (1 << 24)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Threads of a row's CTA and the vectors each holds (1 to 4): whole warps, `most` threads where four
// vectors suffice for that, else up to 1024.
void row_shape(int nvec, int most, int* vpt, int* threads) {
  if (nvec > 4 * most) most = 1024;
  *vpt = (nvec + most - 1) / most;
  *threads = ((nvec + *vpt - 1) / *vpt + 31) / 32 * 32;
}

// The backward's CTAs: up to 768 threads a row (the register file holds 768 with their sums), and as
// many CTAs as make up 768 threads per SM.
constexpr int kBwdThreads = 768;
void bwd_shape(const moe_norm_t& n, int* vpt, int* threads, int* per_sm) {
  row_shape(n.H / (n.dtype == MOE_BF16 ? 8 : 4), kBwdThreads, vpt, threads);
  *per_sm = max(1, kBwdThreads / *threads);
}
constexpr int kMaxSms = 256;

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_block_norm(const moe_norm_t* n, const void* residual, const void* block, const float* w_post,
                   const float* gate, const float* w_pre, void* residual_out, void* normed,
                   float* rstd_block, float* rstd_res, void* stream) {
  MOE_TRY(check_norm(n));
  if (n->T == 0) return MOE_OK;
  MOE_TRY(check_ptrs({residual}));
  MOE_TRY(check_opt({block, w_post, gate, w_pre, residual_out, normed, rstd_block, rstd_res}));
  if (!block && !w_pre) return MOE_ERR_INVALID_ARG;
  if (!block && (w_post || residual_out || rstd_block || n->gate != MOE_GATE_NONE)) return MOE_ERR_INVALID_ARG;
  if (block && !residual_out) return MOE_ERR_INVALID_ARG;
  if (rstd_block && !w_post) return MOE_ERR_INVALID_ARG;
  if ((n->gate != MOE_GATE_NONE) != (gate != nullptr)) return MOE_ERR_INVALID_ARG;
  if ((w_pre != nullptr) != (normed != nullptr) || (rstd_res && !w_pre)) return MOE_ERR_INVALID_ARG;
  DeviceInfo dev;
  MOE_TRY(current_device_info(&dev));
  FwdArgs a{n->H, n->gate, n->eps, n->scale, residual, block, w_post, gate, w_pre, residual_out, normed,
            rstd_block, rstd_res};
  const bool bf16 = n->dtype == MOE_BF16;
  // few tokens: many threads per row, for the shortest way through; more: 256, so that an SM has
  // several rows under way (8192 x 6144 bf16: 108, 82, 73, 75 us with 768, 384, 256, 192 threads)
  int vpt, threads;
  row_shape(n->H / (bf16 ? 8 : 4), n->T > 2 * dev.sm_count ? 256 : 1024, &vpt, &threads);
#define NORM_VPT(T) \
  (vpt == 1 ? k_block_norm<T, 1> : vpt == 2 ? k_block_norm<T, 2> : vpt == 3 ? k_block_norm<T, 3> : k_block_norm<T, 4>)
  void (*kern)(FwdArgs) = bf16 ? NORM_VPT(__nv_bfloat16) : NORM_VPT(float);
  const cudaError_t e = launch_kernel(kern, n->T, threads, 0, as_stream(stream), 1, a);
  count_launch();
  return cuda_rc(e);
}

int moe_block_norm_workspace_size(const moe_norm_t* n, size_t* bytes) {
  MOE_TRY(check_norm(n));
  if (!bytes) return MOE_ERR_INVALID_ARG;
  int vpt, threads, per_sm;
  bwd_shape(*n, &vpt, &threads, &per_sm);
  *bytes = (size_t)max(1, min(n->T, kMaxSms * per_sm)) * 3 * n->H * sizeof(float);
  return MOE_OK;
}

int moe_block_norm_backward(const moe_norm_t* n, const void* d_residual_out, const void* d_normed,
                            const void* residual_out, const void* block, const float* w_post,
                            const float* gate, const float* w_pre, const float* rstd_block,
                            const float* rstd_res, void* d_residual, void* d_block, float* d_w_post,
                            float* d_gate, float* d_w_pre, void* ws, size_t ws_bytes, void* stream) {
  size_t need;
  MOE_TRY(moe_block_norm_workspace_size(n, &need));
  if (n->T > 0) {
    MOE_TRY(check_ptrs({d_residual}));
    MOE_TRY(check_opt({d_residual_out, d_normed, residual_out, block, w_post, gate, w_pre, rstd_block, rstd_res,
                       d_block, d_w_post, d_gate, d_w_pre}));
    if (!block && !w_pre) return MOE_ERR_INVALID_ARG;
    if (!block && (w_post || n->gate != MOE_GATE_NONE)) return MOE_ERR_INVALID_ARG;
    if ((n->gate != MOE_GATE_NONE) != (gate != nullptr)) return MOE_ERR_INVALID_ARG;
    // each part's tensors come together
    const auto agree = [](bool have, std::initializer_list<const void*> ps) {
      for (const void* p : ps)
        if ((p != nullptr) != have) return false;
      return true;
    };
    if (!agree(block != nullptr, {d_block}) || !agree(w_post != nullptr, {rstd_block, d_w_post}) ||
        !agree(gate != nullptr, {d_gate}) || !agree(w_pre != nullptr, {d_normed, residual_out, rstd_res, d_w_pre}))
      return MOE_ERR_INVALID_ARG;
    if (!d_residual_out && !w_pre) return MOE_ERR_INVALID_ARG;
  }
  if (ws_bytes < need) return MOE_ERR_WORKSPACE;
  MOE_TRY(check_ptrs({ws}));
  MOE_TRY(check_opt({d_w_post, d_w_pre, d_gate}));
  DeviceInfo dev;
  const cudaStream_t st = as_stream(stream);
  MOE_TRY(current_device_info(&dev));
  BwdArgs a{n->T, n->H, n->gate, n->scale, d_residual_out, d_normed, residual_out, block, w_post, gate, w_pre,
            rstd_block, rstd_res, d_residual, d_block, n->gate == MOE_GATE_TOKEN ? d_gate : nullptr,
            static_cast<float*>(ws)};
  const bool bf16 = n->dtype == MOE_BF16;
  int vpt, threads, per_sm;
  bwd_shape(*n, &vpt, &threads, &per_sm);
#define NORM_BWD(T, MAXT)                                                            \
  (vpt == 1 ? k_block_norm_bwd<T, 1, MAXT> : vpt == 2 ? k_block_norm_bwd<T, 2, MAXT> \
   : vpt == 3 ? k_block_norm_bwd<T, 3, MAXT> : k_block_norm_bwd<T, 4, MAXT>)
  void (*kern)(BwdArgs) = threads > kBwdThreads ? (bf16 ? NORM_BWD(__nv_bfloat16, 1024) : NORM_BWD(float, 1024))
                                                : (bf16 ? NORM_BWD(__nv_bfloat16, kBwdThreads) : NORM_BWD(float, kBwdThreads));
  const int grid = min(n->T, min(dev.sm_count, kMaxSms) * per_sm);
  if (n->T > 0) {
    MOE_TRY(cuda_rc(launch_kernel(kern, grid, threads, 0, st, 1, a)));
    count_launch();
  }
  float* chan = n->gate == MOE_GATE_CHANNEL ? d_gate : nullptr;
  if (!d_w_post && !d_w_pre && !chan) return MOE_OK;
  const cudaError_t e = launch_kernel(k_block_norm_sum, dim3((n->H + 31) / 32, 3), 1024, 0, st, 1,
                                      static_cast<const float*>(ws), grid, n->H, d_w_post, d_w_pre, chan);
  count_launch();
  return cuda_rc(e);
}

}  // extern "C"
