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
// 10 and 22 flops per element (the backward's done two at a time, which took 3 % off 8192 x 6144 bf16 and a
// fifth off 4096 x 8192): 70 and 112 us for 8192 x 6144 bf16, 5.8 and 5.4 TB/s. One CTA holds a token's row in registers (16-byte vectors), so
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

// Sum of the squares of a thread's vectors.
template <typename T, int VPT>
__device__ __forceinline__ float squares(const uint4 (&q)[VPT]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    float v[Row<T>::N];
    Row<T>::unpack(q[i], v);
#pragma unroll
    for (int j = 0; j < Row<T>::N; ++j) s = fmaf(v[j], v[j], s);
  }
  return s;
}

// A CTA's most threads (row_shape gives three and four vectors of bf16 to 256 threads only), and the CTAs
// per SM that the registers have to allow (0: as the compiler likes). Five, not four, of 6144 columns:
// 69.0 us instead of 72.8 for 8192 rows, six 70.6; four, not three, of 8192: 96 us instead of 111.
template <typename T>
constexpr int fwd_threads(int vpt) { return sizeof(T) == 2 && vpt >= 3 ? 256 : 1024; }
template <typename T>
constexpr int fwd_blocks(int vpt) { return sizeof(T) == 2 && vpt == 3 ? 5 : sizeof(T) == 2 && vpt == 4 ? 4 : 0; }

// VPT vectors per thread, strided by the block so that a warp's loads are contiguous.
template <typename T, int VPT>
__global__ void __launch_bounds__(fwd_threads<T>(VPT), fwd_blocks<T>(VPT)) k_block_norm(const FwdArgs a) {
  constexpr int N = Row<T>::N;
  __shared__ float part[2][32];
  pdl_launch_dependents();
  pdl_wait();
  const size_t t = blockIdx.x;
  const int nvec = a.H / N;
  const uint4* res = reinterpret_cast<const uint4*>(static_cast<const T*>(a.residual) + t * a.H);
  // the rows stay as they are in memory (12 registers for 6144 columns of bf16 on 256 threads, not 24) and
  // are unpacked where they are used: more rows fit on an SM
  uint4 r[VPT];
  if (a.block) {
    const uint4* blk = reinterpret_cast<const uint4*>(static_cast<const T*>(a.block) + t * a.H);
    uint4 b[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      b[i] = v < nvec ? blk[v] : make_uint4(0, 0, 0, 0);
      r[i] = v < nvec ? res[v] : make_uint4(0, 0, 0, 0);
    }
    float rb = 1.0f;
    if (a.w_post) {
      rb = rstd_of(block_sum(squares<T, VPT>(b), part[0]), a.H, a.eps);
      if (a.rstd_block && threadIdx.x == 0) a.rstd_block[t] = rb;
    }
    const float gt = a.scale * (a.gate == MOE_GATE_TOKEN ? a.g[t] : 1.0f);
    uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(a.residual_out) + t * a.H);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v >= nvec) continue;
      float w[N], gc[N], x[N], y[N];
#pragma unroll
      for (int j = 0; j < N; ++j) w[j] = gc[j] = 1.0f;
      if (a.w_post) load_param(a.w_post, v * N, w);
      if (a.gate == MOE_GATE_CHANNEL) load_param(a.g, v * N, gc);
      Row<T>::unpack(b[i], x);
      Row<T>::unpack(r[i], y);
#pragma unroll
      for (int j = 0; j < N; ++j) y[j] = fmaf(gt * gc[j], x[j] * rb * w[j], y[j]);
      r[i] = Row<T>::pack(y);        // the next norm reads the stream as it is stored
      out[v] = r[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      r[i] = v < nvec ? res[v] : make_uint4(0, 0, 0, 0);
    }
  }
  if (!a.w_pre) return;
  const float rr = rstd_of(block_sum(squares<T, VPT>(r), part[1]), a.H, a.eps);
  if (a.rstd_res && threadIdx.x == 0) a.rstd_res[t] = rr;
  uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(a.normed) + t * a.H);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v >= nvec) continue;
    float w[N], x[N];
    load_param(a.w_pre, v * N, w);
    Row<T>::unpack(r[i], x);
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] = x[j] * rr * w[j];
    out[v] = Row<T>::pack(x);
  }
}

struct BwdArgs {
  int T, H, gate;
  float scale;
  const void *d_res_out, *d_normed, *res_out, *block;
  const float *w_post, *g, *w_pre, *rstd_block, *rstd_res;
  void *d_residual, *d_block;
  float* d_gate;         // per token
  float* partial;        // [grid, 2, H]: sum of gate_t g bhat and of d_normed rhat (the parts that exist)
  int* status;
};

// A token's norms and gate. (Loading them a token ahead was a sixth slower for 8192 x 6144
// bf16.)
struct TokenScalars {
  float rr, rb, gt;
};
__device__ __forceinline__ TokenScalars load_scalars(const BwdArgs& a, size_t t) {
  return TokenScalars{a.w_pre ? a.rstd_res[t] : 0.f, a.w_post ? a.rstd_block[t] : 1.f,
                      a.gate == MOE_GATE_TOKEN ? a.g[t] : 1.f};
}

// Elements j and j + 1 as a register pair, back, and their sum.
template <int N>
__device__ __forceinline__ uint64_t pair(const float (&v)[N], int j) {
  return pack_f32x2(v[j], v[j + 1]);
}
template <int N>
__device__ __forceinline__ void put(uint64_t p, float (&v)[N], int j) {
  unpack_f32x2(p, v[j], v[j + 1]);
}
__device__ __forceinline__ float both(uint64_t p) {
  float a, b;
  unpack_f32x2(p, a, b);
  return a + b;
}

// One token's gradients, for the VPT vectors of a thread: its rows (d_normed and res_out unpacked into
// g and rhat, d_res_out and block as loaded) and its sums over tokens. wg = w_post * gate of the column;
// the sum p of gate_t g bhat serves both d_w_post (scale * gate_c * p) and d_gate_c (scale * w_post * p).
template <typename T, int VPT, class PRE, class POST>
__device__ __forceinline__ void token_gradients(const BwdArgs& a, size_t t, int nvec, float (&g)[VPT][Row<T>::N],
                                                float (&rhat)[VPT][Row<T>::N], const uint4 (&qd)[VPT],
                                                const uint4 (&qb)[VPT], const TokenScalars& k, float inv_h,
                                                float (&s_post)[VPT][Row<T>::N], float (&s_pre)[VPT][Row<T>::N],
                                                float (*part)[32], const PRE& w_pre, const POST& wg) {
  constexpr int N = Row<T>::N;
  const size_t o = t * a.H;
  float sum = 0.f;
  if (a.w_pre) {
    const uint64_t rr = pack_f32x2(k.rr, k.rr);
    uint64_t sums = 0;                                      // of the even and of the odd elements
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float w[N];
      w_pre(i, w);
#pragma unroll
      for (int j = 0; j < N; j += 2) {
        const uint64_t rh = mul_f32x2(pair(rhat[i], j), rr);
        put(fma_f32x2(pair(g[i], j), rh, pair(s_pre[i], j)), s_pre[i], j);
        const uint64_t c = mul_f32x2(pair(g[i], j), pair(w, j));
        sums = fma_f32x2(c, rh, sums);
        put(rh, rhat[i], j);
        put(c, g[i], j);
      }
    }
    sum = both(sums);
    sum = block_sum(sum, part[0]) * inv_h;
  } else {
    __syncthreads();
  }
  // g: the gradient of the residual stream
  const uint64_t rr = pack_f32x2(k.rr, k.rr), minus = pack_f32x2(-sum, -sum);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    float d[N];
    Row<T>::unpack(qd[i], d);
#pragma unroll
    for (int j = 0; j < N; j += 2)
      put(fma_f32x2(rr, fma_f32x2(pair(rhat[i], j), minus, pair(g[i], j)), pair(d, j)), g[i], j);
    if (v < nvec) reinterpret_cast<uint4*>(static_cast<T*>(a.d_residual) + o)[v] = Row<T>::pack(g[i]);
  }
  if (!a.block) {
    __syncthreads();                                        // part[0] is free again
    return;
  }
  // bhat in rhat's registers
  uint64_t dots = 0;                                        // <g wg, bhat>
  const uint64_t rb = pack_f32x2(k.rb, k.rb), gt = pack_f32x2(k.gt, k.gt);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    float w[N], b[N];
    wg(i, w);
    Row<T>::unpack(qb[i], b);
#pragma unroll
    for (int j = 0; j < N; j += 2) {
      const uint64_t bh = mul_f32x2(pair(b, j), rb), h = mul_f32x2(pair(g[i], j), bh);
      put(fma_f32x2(gt, h, pair(s_post[i], j)), s_post[i], j);
      dots = fma_f32x2(h, pair(w, j), dots);
      put(mul_f32x2(pair(g[i], j), pair(w, j)), g[i], j);
      put(bh, rhat[i], j);
    }
  }
  float dot = both(dots);
  float mean = 0.f;
  if (a.w_post || a.gate == MOE_GATE_TOKEN) {
    dot = block_sum(dot, part[1]);
    if (a.gate == MOE_GATE_TOKEN && threadIdx.x == 0) a.d_gate[t] = a.scale * dot;
    if (a.w_post) mean = dot * inv_h;
  }
  const float f = a.scale * k.gt * k.rb;
  const uint64_t ff = pack_f32x2(f, f), less = pack_f32x2(-mean, -mean);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
#pragma unroll
    for (int j = 0; j < N; j += 2)
      put(mul_f32x2(ff, fma_f32x2(pair(rhat[i], j), less, pair(g[i], j))), g[i], j);
    if (v < nvec) reinterpret_cast<uint4*>(static_cast<T*>(a.d_block) + o)[v] = Row<T>::pack(g[i]);
  }
  // part[0] may be written again: every thread has read it before the second sum's barrier
  if (!(a.w_post || a.gate == MOE_GATE_TOKEN)) __syncthreads();
}

// w_post * gate (per channel), each 1 where it is absent, of the vector at column c.
template <int N>
__device__ __forceinline__ void load_wg(const BwdArgs& a, int c, float (&w)[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j) w[j] = 1.0f;
  if (a.w_post) load_param(a.w_post, c, w);
  if (a.gate == MOE_GATE_CHANNEL) {
    float g[N];
    load_param(a.g, c, g);
#pragma unroll
    for (int j = 0; j < N; ++j) w[j] *= g[j];
  }
}

template <typename T, int VPT>
__device__ __forceinline__ void store_partial(const BwdArgs& a, int nvec, const float (&s_post)[VPT][Row<T>::N],
                                              const float (&s_pre)[VPT][Row<T>::N]) {
  constexpr int N = Row<T>::N;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v >= nvec) continue;
    float* p = a.partial + (size_t)blockIdx.x * 2 * a.H + v * N;
#pragma unroll
    for (int j = 0; j < N; j += 4) {
      if (a.block) *reinterpret_cast<float4*>(p + j) = make_float4(s_post[i][j], s_post[i][j + 1], s_post[i][j + 2], s_post[i][j + 3]);
      if (a.w_pre) *reinterpret_cast<float4*>(p + a.H + j) = make_float4(s_pre[i][j], s_pre[i][j + 1], s_pre[i][j + 2], s_pre[i][j + 3]);
    }
  }
}

// Rows straight into registers: for rows of which two tokens' do not fit in shared memory.
template <typename T, int VPT>
__global__ void __launch_bounds__(1024) k_block_norm_bwd(const BwdArgs a) {
  constexpr int N = Row<T>::N;
  __shared__ float part[2][32];
  pdl_launch_dependents();
  pdl_wait();
  const int nvec = a.H / N;
  float s_post[VPT][N] = {}, s_pre[VPT][N] = {};
  for (size_t t = blockIdx.x; t < (size_t)a.T; t += gridDim.x) {
    uint4 qd[VPT], qb[VPT];
    float g[VPT][N], rhat[VPT][N];
    const auto vec = [&](const void* p, int v) {
      return p && v < nvec ? reinterpret_cast<const uint4*>(static_cast<const T*>(p) + t * a.H)[v] : make_uint4(0, 0, 0, 0);
    };
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      Row<T>::unpack(vec(a.w_pre ? a.d_normed : nullptr, v), g[i]);
      Row<T>::unpack(vec(a.w_pre ? a.res_out : nullptr, v), rhat[i]);
      qd[i] = vec(a.d_res_out, v);
      qb[i] = vec(a.block, v);
    }
    token_gradients<T, VPT>(
        a, t, nvec, g, rhat, qd, qb, load_scalars(a, t), 1.0f / (float)a.H, s_post, s_pre, part,
        [&](int i, float (&w)[N]) { load_param(a.w_pre, min((int)(threadIdx.x + i * blockDim.x), nvec - 1) * N, w); },
        [&](int i, float (&w)[N]) { load_wg(a, min((int)(threadIdx.x + i * blockDim.x), nvec - 1) * N, w); });
  }
  store_partial<T, VPT>(a, nvec, s_post, s_pre);
}

// Rows through a ring in shared memory, filled by bulk copies: a CTA of a wide row has an SM to itself
// (its sums over tokens stay in registers), so the loads of the next tokens go on under the two block
// reductions of this one. (Loading the next token into registers instead gained nothing.) The ring has
// `depth` tokens of up to four rows (stall: testing, MOE_TUNE_TEST_STALL, the first place of CTA 0 is not
// filled). A CTA of at most 512 threads may use 128 registers a thread: with the parameters and both vectors'
// sums in them 4096 x 8192 bf16 take 84 us instead of 148 with the parameters read for every token, 4096 x
// 6144 fp32 119 instead of 137. (bf16 rows of 8208 to 12288 columns, 1026 to 1536 vectors, have 80 registers
// and spill some 90 of them: 200 us for 4096 x 12288, 45 % of the copy rate.)
constexpr int kMaxDepth = 4;
constexpr int kRingThreads = 768;      // what the register file holds with their sums

template <typename T, int VPT, int THREADS>
__global__ void __launch_bounds__(THREADS) k_block_norm_bwd_ring(const BwdArgs a, int depth, int stall) {
  constexpr int N = Row<T>::N;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float part[2][32];
  __shared__ uint64_t full[kMaxDepth];
  __shared__ int abort_flag;
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < depth; ++i) mbar_init(&full[i], 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  pdl_wait();
  __syncthreads();
  const int nvec = a.H / N;
  const uint32_t row = (uint32_t)a.H * sizeof(T);
  const auto fill = [&](int s, size_t t) {
    const void* src[4] = {a.w_pre ? a.d_normed : nullptr, a.w_pre ? a.res_out : nullptr, a.d_res_out, a.block};
    uint32_t n = 0;
    for (int i = 0; i < 4; ++i) n += src[i] ? 1 : 0;
    mbar_arrive_expect_tx(&full[s], n * row);
    for (int i = 0; i < 4; ++i)
      if (src[i])
        bulk_load(ring + (size_t)(s * 4 + i) * row, static_cast<const char*>(src[i]) + t * row, row, &full[s]);
  };
  if (threadIdx.x == 0)
    for (int s = blockIdx.x ? 0 : stall; s < depth; ++s)
      if (blockIdx.x + (size_t)s * gridDim.x < (size_t)a.T) fill(s, blockIdx.x + (size_t)s * gridDim.x);

  // the columns' parameters stay in registers
  float wp[VPT][N], wg[VPT][N];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = min((int)(threadIdx.x + i * blockDim.x), nvec - 1) * N;
    if (a.w_pre) load_param(a.w_pre, c, wp[i]);
    load_wg(a, c, wg[i]);
  }
  float s_post[VPT][N] = {}, s_pre[VPT][N] = {};
  const float inv_h = 1.0f / (float)a.H;
  int s = 0;
  uint32_t phase = 0;
  bool ok = true;
  for (size_t t = blockIdx.x; t < (size_t)a.T; t += gridDim.x) {
    const TokenScalars k = load_scalars(a, t);
    // (a thread whose wait ran out works on what there is, since it has to keep up with the block's
    // barriers, and waits for no token after that)
    ok = ok && mbar_wait(&full[s], phase, &abort_flag);
    uint4 qd[VPT], qb[VPT];
    float g[VPT][N], rhat[VPT][N];
    const auto vec = [&](bool have, int i, int v) {
      return have && v < nvec ? reinterpret_cast<const uint4*>(ring + (size_t)(s * 4 + i) * row)[v] : make_uint4(0, 0, 0, 0);
    };
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      Row<T>::unpack(vec(a.w_pre, 0, v), g[i]);
      Row<T>::unpack(vec(a.w_pre, 1, v), rhat[i]);
      qd[i] = vec(a.d_res_out, 2, v);
      qb[i] = vec(a.block, 3, v);
    }
    token_gradients<T, VPT>(
        a, t, nvec, g, rhat, qd, qb, k, inv_h, s_post, s_pre, part,
        [&](int i, float (&w)[N]) {
#pragma unroll
          for (int j = 0; j < N; ++j) w[j] = wp[i][j];
        },
        [&](int i, float (&w)[N]) {
#pragma unroll
          for (int j = 0; j < N; ++j) w[j] = wg[i][j];
        });
    // every thread has used its rows before the token's last barrier (loads that are only under way
    // there would not do): the place is free. Filling it at the end of the token keeps the copies'
    // issue, some 140 cycles each, out of the block's way (an eighth of the time for 8192 x 6144 bf16)
    const size_t next = t + (size_t)depth * gridDim.x;
    if (threadIdx.x == 0 && next < (size_t)a.T) fill(s, next);
    if (++s == depth) {
      s = 0;
      phase ^= 1u;
    }
  }
  store_partial<T, VPT>(a, nvec, s_post, s_pre);
  __syncthreads();
  if (abort_flag && threadIdx.x == 0) {
    set_status(a.status, MOE_ERR_TIMEOUT);
    // let copies already in flight land before the CTA's memory goes away
    const unsigned long long t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 2000000ull) __nanosleep(1000);
  }
}

// Sums the CTAs' partial sums p (blockIdx.y 0: d_w_post = scale * gate_c * p and d_gate_c = scale *
// w_post * p, 1: d_w_pre = p): 32 columns per block, whose 32 warps share the CTAs; each warp adds its
// ones in order, then the warps' sums are added in order.
struct SumArgs {
  const float* partial;
  int n, H;
  float scale;
  const float *w_post, *gate_c;      // or null: 1
  float *d_w_post, *d_w_pre, *d_gate;
};
__global__ void __launch_bounds__(1024) k_block_norm_sum(const SumArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const bool pre = blockIdx.y == 1;
  if (pre ? !a.d_w_pre : !a.d_w_post && !a.d_gate) return;
  __shared__ float part[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < a.H) {
#pragma unroll 4
    for (int i = warp; i < a.n; i += 32) s += a.partial[((size_t)i * 2 + blockIdx.y) * a.H + c];
  }
  part[lane][warp] = s;
  __syncthreads();
  // warp w adds up column w
  const float v = warp_sum_f(part[warp][lane]);
  const int col = blockIdx.x * 32 + warp;
  if (lane != 0 || col >= a.H) return;
  if (pre) {
    a.d_w_pre[col] = v;
  } else {
    if (a.d_w_post) a.d_w_post[col] = a.scale * (a.gate_c ? a.gate_c[col] : 1.0f) * v;
    if (a.d_gate) a.d_gate[col] = a.scale * (a.w_post ? a.w_post[col] : 1.0f) * v;
  }
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

// The backward's CTAs. With the ring, for rows of up to 2 x 768 vectors of which two tokens' fit: up to 768
// threads of one or two vectors, as many CTAs as make up 768 threads per SM. Without (depth 0): up to 1024
// threads, one CTA per SM.
constexpr size_t kRingBytes = 200 * 1024;      // of an SM's rings
struct BwdShape {
  int vpt, threads, per_sm, depth;
  size_t smem;
};
BwdShape bwd_shape(const moe_norm_t& n) {
  BwdShape b{};
  const size_t esz = n.dtype == MOE_BF16 ? 2 : 4, token = 4 * esz * n.H;
  const int nvec = (int)(n.H * esz / 16);
  const bool narrow = nvec <= 2 * kRingThreads;
  row_shape(nvec, narrow ? kRingThreads : 1024, &b.vpt, &b.threads);
  b.per_sm = max(1, kRingThreads / b.threads);
  // One-vector CTAs that make up at most three quarters of those 768 threads (a row of 288, or of 416 to 576
  // threads) leave the rest unused. CTAs of two vectors take their place where together they have as many
  // threads (768 in fp32; in bf16, with 128 registers a thread, 512, which rows of 416 to 512 threads meet):
  // 8192 x 4096 bf16 75 us instead of 94, x 2048 fp32 77 instead of 83. (Where one vector fills the SM two
  // cost: an eighth more at 6144; and so they do with few tokens per CTA: 13.1 instead of 11.2 for 512 x 2048.)
  if (b.vpt == 1 && n.T >= 2048 && 4 * b.per_sm * b.threads <= 3 * kRingThreads) {
    int vpt, threads;
    row_shape(nvec, (nvec + 1) / 2, &vpt, &threads);
    const int per_sm = (esz == 2 ? 512 : kRingThreads) / threads;
    if (per_sm * threads >= b.per_sm * b.threads) b.vpt = vpt, b.threads = threads, b.per_sm = per_sm;
  }
  b.depth = (int)min((size_t)kMaxDepth, kRingBytes / b.per_sm / token);
  if (b.depth < 2 || !narrow) b.depth = 0;
  b.smem = b.depth * token;
  return b;
}
constexpr int kMaxSms = 256;
constexpr size_t kStatusBytes = 256;

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
  // several rows under way (8192 x 6144 bf16, before: 108, 82, 73, 75 us with 768, 384, 256, 192 threads)
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
  *bytes = kStatusBytes + (size_t)max(1, min(n->T, kMaxSms * bwd_shape(*n).per_sm)) * 2 * n->H * sizeof(float);
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
            at<float>(ws, kStatusBytes), at<int>(ws, 0)};
  const bool bf16 = n->dtype == MOE_BF16;
  const BwdShape b = bwd_shape(*n);
  const int grid = min(n->T, min(dev.sm_count, kMaxSms) * b.per_sm);
  if (n->T > 0) {
    cudaError_t e;
    if (b.depth) {
      // (the kernels for 512 threads take 128 registers in bf16 and 88 in fp32, the others 80)
#define NORM_RING(T, ROOM)                                              \
  (b.vpt == 1                   ? k_block_norm_bwd_ring<T, 1, kRingThreads> \
   : b.threads * b.per_sm <= ROOM && b.threads <= 512 ? k_block_norm_bwd_ring<T, 2, 512> \
                                : k_block_norm_bwd_ring<T, 2, kRingThreads>)
      auto kern = bf16 ? NORM_RING(__nv_bfloat16, 512) : NORM_RING(float, 704);
      // the same value for every shape: the limit is the kernel's, and a call from another thread may set it
      // between this call's setting and its launch
      if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRingBytes) != cudaSuccess)
        return MOE_ERR_CUDA;
      e = launch_kernel(kern, grid, b.threads, b.smem, st, 1, a, b.depth, take_test_stall(2) ? 1 : 0);
    } else {
      // more than 12288 (bf16) or 6144 (fp32) elements: 2, or 2 to 4 vectors
      auto kern = bf16         ? k_block_norm_bwd<__nv_bfloat16, 2>
                  : b.vpt == 2 ? k_block_norm_bwd<float, 2>
                  : b.vpt == 3 ? k_block_norm_bwd<float, 3>
                               : k_block_norm_bwd<float, 4>;
      e = launch_kernel(kern, grid, b.threads, 0, st, 1, a);
    }
    MOE_TRY(cuda_rc(e));
    count_launch();
  }
  float* chan = n->gate == MOE_GATE_CHANNEL ? d_gate : nullptr;
  if (!d_w_post && !d_w_pre && !chan) return MOE_OK;
  const SumArgs sum{at<float>(ws, kStatusBytes), grid, n->H, n->scale, w_post,
                    n->gate == MOE_GATE_CHANNEL ? gate : nullptr, d_w_post, d_w_pre, chan};
  const cudaError_t e = launch_kernel(k_block_norm_sum, dim3((n->H + 31) / 32, 2), 1024, 0, st, 1, sum);
  count_launch();
  return cuda_rc(e);
}

}  // extern "C"
