// mx4_gemm.cu - ragged grouped products of two 4-bit operands on the 5th-generation tensor
// cores (tcgen05.mma with block scales), and the SwiGLU FFN of 4-bit experts made of them.
//
//   y[r, n] = sum_k A[r, k] W[g(r)][n, k]            (moe_mx4_grouped_gemm, and the FFN's down)
//   h[r, i] = q(silu(A Wg^T) * (A Wu^T))             (the FFN's gate and up)
//
// The weights are the M side of the MMA (128 rows), a group's rows the N side. A decode step has
// a few rows per group and then is bound by streaming the weights, so the side that is padded to
// 128 is the one that has the rows, and N shrinks with the group to 16. Each tile holds two
// weight blocks of 128 rows, which share the tile's rows: the gate and up rows of the same 128
// channels of h, or 256 outputs of a plain product. TMEM lane = output channel, column = row.
//
// Kernel structure (one CTA per SM, persistent, static round-robin over tiles):
//   warp 0      TMA producer: per stage of K = 256 elements (128 bytes, 128-byte swizzle) two
//               weight boxes of 128 rows, the tile's rows in boxes of 64 and 16, and the block
//               scales as plain bulk copies of the 512-byte pieces
//   warp 1      TMEM owner and MMA issuer: tcgen05.cp moves each piece of scales to its 4 TMEM
//               columns, then 4 x 2 tcgen05.mma M128 K64 per stage
//   warps 2-9   epilogue: tcgen05.ld, math, global stores
// The scales of a stage alternate between two TMEM slots: before it overwrites a slot the issuer
// waits until the MMAs of two stages ago have completed.
//
// Tiles: a group of `count` rows has ceil(count / NT) tiles along its rows; the table is built in
// shared memory from `offsets` by every CTA, so the host never reads the counts. Columns past
// the group's last row are computed from whatever is there (each depends on its own row only)
// and never stored. Every wait is bounded (MOE_ERR_TIMEOUT in the status word).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cstddef>

#include "checks.cuh"
#include "common.cuh"
#include "kernels.cuh"
#include "launch.cuh"
#include "mx4.cuh"

namespace moe {
namespace {

constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + kEpiWarps * 32;
constexpr uint32_t kTmemCols = 512;
constexpr int W_BYTES = 128 * 128;                  // a weight block's stage: 128 rows x 128 bytes

enum Mode : int { kStore = 0, kAtomic = 1, kSwiglu = 2 };

struct Args {
  Mx4Rows a;              // the rows' groups
  int n_out;              // output channels per group: N, or I for kSwiglu
  int w_rows;             // weight rows per group: N, or 2I
  int w_second;           // from a tile's first weight block to its second: 128, or I
  int n_tiles;            // tiles along the channels
  int kstages;            // ceil(K / 256)
  int chunks;             // 512-byte scale pieces along K
  const uint8_t* a_scales;
  const uint8_t* w_scales;
  const float* a_factor;  // or null: 1
  const float* w_factor;
  int w_factor_per_group;
  int mode;
  void* out;              // kStore: [rows, n_out]; kAtomic: fp32 [*, n_out]; kSwiglu: h's codes
  int out_fp32;
  uint8_t* h_scales;      // kSwiglu
  const float* h_factor;
  const int32_t* perm_token;   // kAtomic
  const float* row_gate;
  float scale;
  int* status;
};

// NT: rows of a tile. CPS: scale pieces of a stage along K (2: MXFP4, 4: NVFP4).
template <int NT, int CPS>
struct Cfg {
  static constexpr bool kNv = CPS == 4;
  static constexpr int T_BYTES = NT * 128;
  static constexpr int SFT_TILES = NT > 64 ? 2 : 1;       // 128-row scale tiles that NT rows span
  static constexpr int SFW_BYTES = CPS * 512;
  static constexpr int STAGE = 2 * W_BYTES + T_BYTES + (2 + SFT_TILES) * SFW_BYTES;
  static constexpr int STAGES = (227 * 1024 - 12 * 1024) / STAGE;
  static constexpr int ACCS = NT > 64 ? 1 : 2;            // accumulator sets of 2 NT columns
  static constexpr int SF_COL = ACCS * 2 * NT;            // TMEM columns of the scales' slots
  static constexpr int SF_SLOT = CPS * 16;                // W0: CPS x 4, W1: CPS x 4, rows: CPS x 8
  static_assert(STAGE % 1024 == 0, "128-byte-swizzled boxes need 1024-byte alignment");
  static_assert(SF_COL + 2 * SF_SLOT <= (int)kTmemCols, "TMEM budget");
};

template <int STAGES, int STAGE>
struct alignas(1024) Storage {
  uint8_t ring[STAGES][STAGE];
  uint64_t full[STAGES];
  uint64_t empty[STAGES];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint32_t tmem_base;
  int abort_flag;
  int offs[kMx4MaxGroups + 1];
  int toff[kMx4MaxGroups + 1];
};

struct Tile {
  int g, row0, row_end, o_g, n0, n;   // n: rows of the tile
  int blocks;                         // weight blocks of 128 rows: 1 or 2
};

// Tile order: group by group, inside a group channel tile by channel tile with the row tiles
// fastest, so that the CTAs that run at once share each weight block through L2.
template <class S>
__device__ __forceinline__ Tile decode(const S& s, const Args& g, int tile, int NT) {
  Tile t;
  const int any = tile / g.n_tiles;
  int lo = 0, hi = g.a.groups - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s.toff[mid] <= any) lo = mid; else hi = mid - 1;
  }
  const int rt = s.toff[lo + 1] - s.toff[lo];
  const int l = tile - s.toff[lo] * g.n_tiles;
  const int nt = l / rt;
  t.g = lo;
  t.o_g = s.offs[lo];
  t.row0 = t.o_g + (l - nt * rt) * NT;
  t.row_end = s.offs[lo + 1];
  t.n = min(NT, t.row_end - t.row0);
  const int per = g.mode == kSwiglu ? 128 : 256;
  t.n0 = nt * per;
  t.blocks = g.mode == kSwiglu || t.n0 + 128 < g.n_out ? 2 : 1;
  return t;
}

// ---- tcgen05 with block scales ---------------------------------------------------------------
// 32 rows of 16 bytes in shared memory -> 4 TMEM columns of lanes 0-31, repeated in the other
// three lane quarters.
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint32_t smem_addr) {
  // no swizzle: 8-row groups of 16-byte rows, 128 bytes apart
  const uint64_t desc = static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu) |
                        (static_cast<uint64_t>(128u >> 4) << 32) | (static_cast<uint64_t>(1u) << 46);
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// D (+)= (A * scales of A) (B * scales of B)^T, both operands e2m1, fp32 accumulate.
template <bool NV>
__device__ __forceinline__ void umma_mx4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  if (NV) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], "
        "[%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], "
        "[%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  }
}

// Instruction descriptor, block-scaled 4-bit kinds: A and B e2m1 (bits 7-9 and 10-11 = 1), both
// K-major, N >> 3 in bits 17-22, scale type in bit 23 (1: e8m0, 0: e4m3), M >> 7 in bits 27-28;
// the byte of the scales' 32-bit columns that the MMA starts at: bits 4-5 (B), 29-30 (A).
template <bool NV>
__device__ __forceinline__ uint32_t idesc_mx4(int N, uint32_t sf_id) {
  return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (NV ? 0u : (1u << 23)) |
         (1u << 27) | (sf_id << 4) | (sf_id << 29);
}

// Untiled bulk copy global -> shared, completion counted on `bar`; 16-byte aligned both sides.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void tmem_ld_32x32b_x8(uint32_t taddr, float (&r)[8]) {
  uint32_t u[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
               : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = __uint_as_float(u[i]);
}

// Lane i of each 8-lane group holds 8 four-bit values, value j for column j; afterwards lane j
// holds column j's values, value i from lane i.
__device__ __forceinline__ uint32_t transpose_nibbles(uint32_t v, int lane) {
  uint32_t o = __shfl_xor_sync(0xffffffffu, v, 4);
  v = lane & 4 ? (v & 0xFFFF0000u) | (o >> 16) : (v & 0xFFFFu) | (o << 16);
  o = __shfl_xor_sync(0xffffffffu, v, 2);
  v = lane & 2 ? (v & 0xFF00FF00u) | ((o >> 8) & 0x00FF00FFu) : (v & 0x00FF00FFu) | ((o & 0x00FF00FFu) << 8);
  o = __shfl_xor_sync(0xffffffffu, v, 1);
  v = lane & 1 ? (v & 0xF0F0F0F0u) | ((o >> 4) & 0x0F0F0F0Fu) : (v & 0x0F0F0F0Fu) | ((o & 0x0F0F0F0Fu) << 4);
  return v;
}

// ---- epilogues: 8 columns (rows of the tile) at a time, lane = channel -------------------------
// h: 32 channels of a warp are one (MXFP4) or two (NVFP4) blocks of each of the 8 rows.
template <bool NV>
__device__ __forceinline__ void epi_swiglu(const Args& a, const Tile& t, int c, int q, int lane, float f,
                                           float (&gate)[8], float (&up)[8], float hf) {
  uint32_t byte[8], v = 0;
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    float s[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float G = gate[j + i] * f, U = up[j + i] * f;
      const float h = __fdividef(G, 1.0f + __expf(-G)) * U;
      const uint32_t bits = __float_as_uint(h) & 0x7FFFFFFFu;
      uint32_t top;
      if (NV) {
        const uint32_t lo = __reduce_max_sync(0xffffffffu, lane < 16 ? bits : 0u);
        const uint32_t hi = __reduce_max_sync(0xffffffffu, lane < 16 ? 0u : bits);
        top = lane < 16 ? lo : hi;
      } else {
        top = __reduce_max_sync(0xffffffffu, bits);
      }
      float by;
      byte[j + i] = mx4_scale<NV>(top, hf, by);
      s[i] = mx4_scaled<NV>(h, by);
    }
    v |= e2m1x2(s[0], s[1]) << (4 * j);
  }
  v = transpose_nibbles(v, lane);
  const int j = lane & 7, quad = lane >> 3;
  const int row = t.row0 + c + j;
  // this lane's block's scale of row j
  uint32_t b = byte[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) b = j == i ? byte[i] : b;
  if (c + j >= t.n) return;
  const int ch = t.n0 + 32 * q;
  *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.out) + (size_t)row * (a.n_out / 2) + ch / 2 + 4 * quad) = v;
  if (quad == 0 || (NV && quad == 2)) {
    const int block = (ch + 8 * quad) / mx4_block(NV);
    a.h_scales[mx4_scale_at(t.o_g, t.g, row - t.o_g, block, a.n_out / (4 * mx4_block(NV)))] = (uint8_t)b;
  }
}

__device__ __forceinline__ void epi_plain(const Args& a, const Tile& t, int c, int ch, float f,
                                          const float (&y)[8]) {
  if (ch >= a.n_out) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (c + j >= t.n) break;
    const int row = t.row0 + c + j;
    if (a.mode == kAtomic) {
      atomicAdd(static_cast<float*>(a.out) + (size_t)a.perm_token[row] * a.n_out + ch,
                a.scale * a.row_gate[row] * f * y[j]);
    } else if (a.out_fp32) {
      static_cast<float*>(a.out)[(size_t)row * a.n_out + ch] = f * y[j];
    } else {
      static_cast<__nv_bfloat16*>(a.out)[(size_t)row * a.n_out + ch] = __float2bfloat16_rn(f * y[j]);
    }
  }
}

template <int NT, int CPS, bool SWIGLU>
__global__ void __launch_bounds__(kThreads, 1)
    k_mx4_gemm(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA64,
               const __grid_constant__ CUtensorMap tmA16, const Args g) {
  using C = Cfg<NT, CPS>;
  constexpr bool NV = C::kNv;
  constexpr int STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  auto& s = *reinterpret_cast<Storage<STAGES, C::STAGE>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.tfull[i], 1);
      mbar_init(&s.tempty[i], kEpiWarps * 32);
    }
    s.abort_flag = 0;
    fence_barrier_init();
    prefetch_tensormap(&tmW);
    prefetch_tensormap(&tmA64);
    prefetch_tensormap(&tmA16);
  }
  if (warp == 1) {
    tmem_alloc(&s.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  pdl_wait();
  for (int i = threadIdx.x; i <= g.a.groups; i += kThreads) s.offs[i] = g.a.begin(i);
  __syncthreads();
  if (warp == 2) {
    // toff[e] = sum over e' < e of ceil(count_e' / NT)
    const int per = (g.a.groups + 31) / 32;
    const int b = lane * per;
    auto tiles_of = [&](int e) { return (s.offs[e + 1] - s.offs[e] + NT - 1) / NT; };
    int local = 0;
    for (int i = 0; i < per; ++i)
      if (b + i < g.a.groups) local += tiles_of(b + i);
    const int inc = warp_inclusive_scan(local);
    int run = inc - local;
    for (int i = 0; i < per; ++i)
      if (b + i < g.a.groups) {
        s.toff[b + i] = run;
        run += tiles_of(b + i);
      }
    if (lane == 31) s.toff[g.a.groups] = inc;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;
  const int total = s.toff[g.a.groups] * g.n_tiles;
  volatile int* abort_flag = &s.abort_flag;

  if (warp == 0) {
    // ---- TMA producer --------------------------------------------------------------------
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      for (int tile = blockIdx.x; tile < total && !*abort_flag; tile += gridDim.x) {
        const Tile t = decode(s, g, tile, NT);
        const int big = t.n / 64, small = (t.n % 64 + 15) / 16;
        const int l0 = t.row0 - t.o_g;
        const int sft = ((l0 & 127) + t.n + 127) / 128;      // scale tiles of the rows
        const int wrow = t.g * g.w_rows + t.n0;
        const size_t wtile = (size_t)((t.g * (int64_t)g.w_rows) >> 7) + t.g;
        const uint8_t* sw = g.w_scales + (wtile + t.n0 / 128) * g.chunks * 512;
        const uint8_t* sw2 = sw + (size_t)(g.w_second / 128) * g.chunks * 512;
        const uint8_t* sa = g.a_scales + ((size_t)(t.o_g >> 7) + t.g + (l0 >> 7)) * g.chunks * 512;
        for (int kb = 0; kb < g.kstages; ++kb) {
          if (!mbar_wait(&s.empty[stage], phase ^ 1u, abort_flag)) break;
          uint8_t* st = s.ring[stage];
          uint64_t* bar = &s.full[stage];
          const uint32_t sfb = 512u * (uint32_t)min(CPS, g.chunks - kb * CPS);
          mbar_arrive_expect_tx(bar, t.blocks * (W_BYTES + sfb) + (big * 64 + small * 16) * 128 + sft * sfb);
          tma_load_2d(st, &tmW, kb * 128, wrow, bar);
          if (t.blocks == 2) tma_load_2d(st + W_BYTES, &tmW, kb * 128, wrow + g.w_second, bar);
          uint8_t* rows = st + 2 * W_BYTES;
          for (int i = 0; i < big; ++i) tma_load_2d(rows + i * 64 * 128, &tmA64, kb * 128, t.row0 + i * 64, bar);
          for (int i = 0; i < small; ++i)
            tma_load_2d(rows + (big * 64 + i * 16) * 128, &tmA16, kb * 128, t.row0 + big * 64 + i * 16, bar);
          uint8_t* sf = rows + C::T_BYTES;
          const size_t at = (size_t)kb * CPS * 512;
          bulk_load(sf, sw + at, sfb, bar);
          if (t.blocks == 2) bulk_load(sf + C::SFW_BYTES, sw2 + at, sfb, bar);
          for (int i = 0; i < sft; ++i)
            bulk_load(sf + (2 + i) * C::SFW_BYTES, sa + (size_t)i * g.chunks * 512 + at, sfb, bar);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    }
  } else if (warp == 1) {
    // ---- scales to TMEM and MMA ------------------------------------------------------------
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      long long it = 0;          // stages so far
      bool ok = true;
      for (int tile = blockIdx.x; ok && tile < total && !*abort_flag; tile += gridDim.x) {
        const Tile t = decode(s, g, tile, NT);
        const int npad = (t.n + 15) & ~15;
        const int l0 = t.row0 - t.o_g;
        const int sft = ((l0 & 127) + t.n + 127) / 128;
        const uint32_t sft_col = (uint32_t)(l0 & 127) / 32u;
        if (!mbar_wait(&s.tempty[acc], acc_phase ^ 1u, abort_flag)) break;
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(acc * 2 * NT);
        for (int kb = 0; kb < g.kstages; ++kb, ++it) {
          if (!mbar_wait(&s.full[stage], phase, abort_flag)) { ok = false; break; }
          // the slot's previous MMAs (two stages ago) have read their scales
          if (it >= 2) {
            const long long p = it - 2;
            if (!mbar_wait(&s.empty[p % STAGES], (uint32_t)(p / STAGES) & 1u, abort_flag)) { ok = false; break; }
          }
          tc_fence_after();
          const uint32_t w0 = smem_u32(s.ring[stage]);
          const uint32_t rows = w0 + 2 * W_BYTES;
          const uint32_t sf = rows + C::T_BYTES;
          const uint32_t slot = tmem + C::SF_COL + (uint32_t)(it & 1) * C::SF_SLOT;
          const int pieces = min(CPS, g.chunks - kb * CPS);
          for (int p = 0; p < pieces; ++p) {
            tmem_cp_scales(slot + 4 * p, sf + p * 512);
            if (t.blocks == 2) tmem_cp_scales(slot + CPS * 4 + 4 * p, sf + C::SFW_BYTES + p * 512);
            for (int i = 0; i < sft; ++i)
              tmem_cp_scales(slot + CPS * 8 + 8 * p + 4 * i, sf + (2 + i) * C::SFW_BYTES + p * 512);
          }
          const int ksteps = pieces * (4 / CPS);             // K = 64 each
          for (int k = 0; k < ksteps; ++k) {
            const uint32_t p = k / (4 / CPS);
            const uint32_t idesc = idesc_mx4<NV>(npad, NV ? 0u : 2u * (k & 1));
            const uint64_t db = sw128_kmajor_desc(rows + k * 32);
            const uint32_t sfb = slot + CPS * 8 + 8 * p + sft_col;
            const uint32_t go = (kb > 0 || k > 0) ? 1u : 0u;
            umma_mx4<NV>(d, sw128_kmajor_desc(w0 + k * 32), db, idesc, slot + 4 * p, sfb, go);
            if (t.blocks == 2)
              umma_mx4<NV>(d + NT, sw128_kmajor_desc(w0 + W_BYTES + k * 32), db, idesc, slot + CPS * 4 + 4 * p,
                           sfb, go);
          }
          umma_commit(&s.empty[stage]);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        umma_commit(&s.tfull[acc]);
        if (C::ACCS == 2) acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
    }
  } else {
    // ---- epilogue: TMEM lane quarter = warp % 4; the two warps of a quarter take turns over
    // groups of 8 columns ---------------------------------------------------------------------
    const int q = warp & 3;
    const int half = (warp - 2) >> 2;
    int acc = 0;
    uint32_t acc_phase = 0;
    const float af = NV && g.a_factor ? *g.a_factor : 1.0f;
    const float hf = NV && SWIGLU && g.h_factor ? *g.h_factor : 1.0f;
    for (int tile = blockIdx.x; tile < total; tile += gridDim.x) {
      const Tile t = decode(s, g, tile, NT);
      const float f = NV && g.w_factor ? af * g.w_factor[g.w_factor_per_group ? t.g : 0] : af;
      int w_ok = 1;
      if (lane == 0) w_ok = mbar_wait(&s.tfull[acc], acc_phase, abort_flag) ? 1 : 0;
      w_ok = __shfl_sync(0xffffffffu, w_ok, 0);
      if (!w_ok) break;
      tc_fence_after();
      const uint32_t base = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * 2 * NT);
#pragma unroll 1
      for (int c = 8 * half; c < t.n; c += 16) {
        float v0[8], v1[8];
        tmem_ld_32x32b_x8(base + c, v0);
        if (t.blocks == 2) tmem_ld_32x32b_x8(base + NT + c, v1);
        tmem_ld_wait();
        if (SWIGLU) {
          epi_swiglu<NV>(g, t, c, q, lane, f, v0, v1, hf);
        } else {
          epi_plain(g, t, c, t.n0 + 32 * q + lane, f, v0);
          if (t.blocks == 2) epi_plain(g, t, c, t.n0 + 128 + 32 * q + lane, f, v1);
        }
        __syncwarp();
      }
      tc_fence_before();
      mbar_arrive(&s.tempty[acc]);
      if (C::ACCS == 2) acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
  }

  if (*abort_flag) {
    set_status(g.status, MOE_ERR_TIMEOUT);
    // let copies and MMAs already in flight land before the CTA's memory goes away
    const unsigned long long t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 2000000ull) __nanosleep(1000);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ---- host side -------------------------------------------------------------------------------
template <int NT, int CPS, bool SWIGLU>
int launch_as(const CUtensorMap& w, const CUtensorMap& a64, const CUtensorMap& a16, const Args& g,
              int sm_count, cudaStream_t st) {
  using C = Cfg<NT, CPS>;
  constexpr size_t smem = sizeof(Storage<C::STAGES, C::STAGE>) + 1024;
  static_assert(smem <= 227 * 1024 && C::STAGES >= 3, "shared memory budget");
  auto kern = k_mx4_gemm<NT, CPS, SWIGLU>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return MOE_ERR_CUDA;
  const cudaError_t e = launch_kernel(kern, sm_count, kThreads, smem, st, 1, w, a64, a16, g);
  count_launch();
  return cuda_rc(e);
}

// One grouped product of a (its rows' groups) with w; g holds the epilogue's arguments.
int launch_product(const moe_mx4_t& a, const moe_mx4_t& w, Args g, const DeviceInfo& dev, cudaStream_t st) {
  const bool swiglu = g.mode == kSwiglu;
  g.a = mx4_rows(a);
  g.w_rows = w.group_rows;
  g.n_out = swiglu ? w.group_rows / 2 : w.group_rows;
  g.w_second = swiglu ? g.n_out : 128;
  g.n_tiles = (g.n_out + (swiglu ? 127 : 255)) / (swiglu ? 128 : 256);
  g.kstages = (a.K + 255) / 256;
  g.chunks = a.K / (4 * mx4_block(is_nv(a)));
  g.a_scales = static_cast<const uint8_t*>(a.scales);
  g.w_scales = static_cast<const uint8_t*>(w.scales);
  g.a_factor = a.factor;
  g.w_factor = w.factor;
  g.w_factor_per_group = w.factor_per_group;
  CUtensorMap mw, a64, a16;
  MOE_TRY(make_byte_map(&mw, w.codes, (uint64_t)w.rows, a.K / 2, 128));
  MOE_TRY(make_byte_map(&a64, a.codes, (uint64_t)a.rows, a.K / 2, 64));
  MOE_TRY(make_byte_map(&a16, a.codes, (uint64_t)a.rows, a.K / 2, 16));
  // Few rows per group on average: a tile of 64 rows leaves room for more stages of weights in
  // flight and a second accumulator. Else 192 rows, so that fewer tiles re-read the weights.
  const bool few = a.rows <= 64ll * a.groups;
#define MX4_LAUNCH(NT, CPS) \
  (swiglu ? launch_as<NT, CPS, true>(mw, a64, a16, g, dev.sm_count, st) \
          : launch_as<NT, CPS, false>(mw, a64, a16, g, dev.sm_count, st))
  return is_nv(a) ? (few ? MX4_LAUNCH(64, 4) : MX4_LAUNCH(192, 4))
               : (few ? MX4_LAUNCH(64, 2) : MX4_LAUNCH(192, 2));
#undef MX4_LAUNCH
}

// a: the rows; w: uniform groups of n_rows rows, as many as a has
int check_operands(const moe_mx4_t* a, const moe_mx4_t* w, int n_rows) {
  MOE_TRY(mx4_check(a));
  MOE_TRY(mx4_check(w));
  if (w->offsets || w->format != a->format || w->groups != a->groups || w->K != a->K) return MOE_ERR_INVALID_ARG;
  if (a->factor_per_group) return MOE_ERR_INVALID_ARG;
  if (n_rows > 0 && w->group_rows != n_rows) return MOE_ERR_INVALID_ARG;
  if (w->group_rows <= 0) return MOE_ERR_INVALID_ARG;
  // every tile index fits 32 bits: at most rows / NT + groups row tiles per channel tile
  if (((int64_t)a->rows / 64 + a->groups) * ((w->group_rows + 127) / 128) >= (1ll << 31)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

constexpr size_t kStatusBytes = 1024;

struct FfnLayout {
  size_t codes, scales, total;
};
FfnLayout ffn_layout(const moe_mx4_t& a, int I) {
  moe_mx4_t h = a;
  h.K = I;
  FfnLayout L{};
  L.codes = kStatusBytes;
  L.scales = (L.codes + (size_t)a.rows * (I / 2) + 1023) / 1024 * 1024;
  L.total = L.scales + mx4_scale_size(h);
  return L;
}

int check_ffn(const moe_mx4_t* a, const moe_mx4_t* w_gate_up) {
  MOE_TRY(check_operands(a, w_gate_up, 0));
  if (w_gate_up->group_rows % 2 != 0) return MOE_ERR_INVALID_ARG;
  if (w_gate_up->group_rows % 256 != 0) return MOE_ERR_UNSUPPORTED;      // I % 128
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_mx4_gemm_workspace_size(size_t* bytes) {
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = kStatusBytes;
  return MOE_OK;
}

int moe_mx4_grouped_gemm(const moe_mx4_t* a, const moe_mx4_t* w, void* out, int32_t dtype, void* ws,
                         size_t ws_bytes, void* stream) {
  MOE_TRY(check_operands(a, w, 0));
  if (dtype != MOE_BF16 && dtype != MOE_FP32) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < kStatusBytes) return MOE_ERR_WORKSPACE;
  MOE_TRY(check_ptrs({ws}));
  if (a->rows == 0) return MOE_OK;
  MOE_TRY(check_ptrs({a->codes, a->scales, w->codes, w->scales, out}));
  DeviceInfo dev;
  MOE_TRY(current_device_info(&dev));
  Args g{};
  g.mode = kStore;
  g.out = out;
  g.out_fp32 = dtype == MOE_FP32;
  g.status = static_cast<int*>(ws);
  return launch_product(*a, *w, g, dev, as_stream(stream));
}

int moe_mx4_ffn_workspace_size(const moe_mx4_t* a, const moe_mx4_t* w_gate_up, size_t* bytes) {
  MOE_TRY(check_ffn(a, w_gate_up));
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = ffn_layout(*a, w_gate_up->group_rows / 2).total;
  return MOE_OK;
}

int moe_mx4_grouped_ffn(const moe_mx4_t* a, const moe_mx4_t* w_gate_up, const moe_mx4_t* w_down,
                        const float* h_factor, const int32_t* perm_token, const float* row_gate,
                        float scale, void* out, int32_t dtype, void* ws, size_t ws_bytes, void* stream) {
  MOE_TRY(check_ffn(a, w_gate_up));
  const int I = w_gate_up->group_rows / 2;
  // h: the same rows and groups, I elements each, in the workspace
  const FfnLayout L = ffn_layout(*a, I);
  moe_mx4_t h = *a;
  h.K = I;
  h.factor = h_factor;
  h.codes = static_cast<char*>(ws) + L.codes;
  h.scales = static_cast<char*>(ws) + L.scales;
  MOE_TRY(check_operands(&h, w_down, a->K));
  if (dtype != MOE_BF16 && dtype != MOE_FP32) return MOE_ERR_INVALID_ARG;
  if (!(scale == scale)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < L.total) return MOE_ERR_WORKSPACE;
  MOE_TRY(check_ptrs({ws}));
  if (perm_token) {
    if (dtype != MOE_FP32) return MOE_ERR_INVALID_ARG;
    MOE_TRY(check_ptrs({perm_token, row_gate}));
  }
  if (a->rows == 0) return MOE_OK;
  MOE_TRY(check_ptrs({a->codes, a->scales, w_gate_up->codes, w_gate_up->scales, w_down->codes, w_down->scales, out}));
  DeviceInfo dev;
  MOE_TRY(current_device_info(&dev));
  Args g{};
  g.mode = kSwiglu;
  g.out = h.codes;
  g.h_scales = static_cast<uint8_t*>(h.scales);
  g.h_factor = h_factor;
  g.status = static_cast<int*>(ws);
  MOE_TRY(launch_product(*a, *w_gate_up, g, dev, as_stream(stream)));
  Args d{};
  d.mode = perm_token ? kAtomic : kStore;
  d.out = out;
  d.out_fp32 = dtype == MOE_FP32;
  d.perm_token = perm_token;
  d.row_gate = row_gate;
  d.scale = scale;
  d.status = static_cast<int*>(ws);
  return launch_product(h, *w_down, d, dev, as_stream(stream));
}

}  // extern "C"
