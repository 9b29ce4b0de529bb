// mx4_gemm.cu - ragged grouped products of two 4-bit operands on the 5th-generation tensor
// cores (tcgen05.mma with block scales), and the SwiGLU FFN of 4-bit experts made of them.
//
//   y[r, n] = sum_k A[r, k] W[g(r)][n, k]            (moe_mx4_grouped_gemm, and the FFN's down)
//   h[r, i] = q(silu(A Wg^T) * (A Wu^T))             (the FFN's gate and up)
//
// The weights are the M side of the MMA (128 rows), a group's rows the N side. A decode step has
// a few rows per group and then is bound by streaming the weights, so it is the weights' side that
// comes in blocks of 128, and N shrinks with the group to 16. Each tile holds two
// weight blocks of 128 rows, which share the tile's rows: the gate and up rows of the same 128
// channels of h, or 256 outputs of a plain product. TMEM lane = output channel, column = row.
//
// Two kernels, both persistent with a static round-robin over tiles:
//  * k_mx4_gemm, one CTA per SM, for few rows per group: a tile is two blocks of 128 weight rows
//    (the gate and up rows of 128 channels of h, or 256 outputs of a plain product) by up to 64
//    rows of the group. Bound by streaming the weights.
//  * k_mx4_gemm_pair, CTA pairs (cta_group::2), for many rows: a tile is 256 weight rows, 128 per
//    CTA (64 gate and the same 64 up rows, or 128 outputs), by up to 192 rows of the group, half
//    of which each CTA holds. An e2m1 MMA of one CTA reads both operands from its shared memory
//    at about the rate that memory has (107 bytes a cycle at N = 192 besides what TMA writes); in
//    a pair each CTA reads half of the rows. Two accumulators let the epilogue of a tile overlap
//    the MMAs of the next. Of 352 us for 32768 x 4096 x 6144 (4.7 PFLOP/s) the loads alone take 274,
//    59 bytes a cycle into each SM, and the MMAs alone some 255: the two meet in shared memory.
// Warps, one CTA:
//   0           TMA producer: per stage of K = 256 elements (128 bytes, 128-byte swizzle) the
//               weight boxes, the tile's rows in a few boxes, and the block scales as plain bulk
//               copies of the 512-byte pieces
//   1           TMEM owner and MMA issuer: 4 tcgen05.mma of K = 64 per stage and weight block
//   2-9         epilogue: tcgen05.ld, math, global stores
//   10-13       scales: each warp copies the stage's pieces from shared memory to its lane quarter
//               of TMEM with tcgen05.st (the MMA reads them in all four quarters)
// and the pair, in each CTA: 0 the operands' TMA producer, 1 the MMA issuer (the leader's), then 8 or 12
// epilogue warps, 8 for the scales (four for every other stage) and the scales' TMA producer.
// tcgen05.cp would copy the scales without these warps, but each copy of 512 bytes holds up the tensor
// pipe for some 90 cycles (8 to 16 copies per stage of 768): 64 experts' gate/up at a decode batch
// took 214 us with it.
// The scales of the stages take turns over the TMEM columns that are left, in the pair 3 slots (NVFP4)
// or 6: with fewer slots than stages the scale warps wait, before they overwrite a slot, until the MMAs
// that read it have completed. (Two slots held the pair kernel up: from one MMA's end to the next
// scales in TMEM takes about as long as a stage's MMAs; 594 us instead of 390 at 32768 rows.)
// A lane of the epilogue reads one channel of 8 rows; the warp turns them around, so that a lane has 8
// channels of one row, rounds h with one block scale and stores 16 or 32 bytes at once (one channel
// per lane took 190 us of 750 at 32768 rows, in 2-byte stores). In the pair kernel, whose MMAs keep
// shared memory busy, plain products do it by shuffles (352 us instead of 359, and 143 instead of 150
// for the FFN's down product of 16384 rows); elsewhere it goes through shared memory.
//
// Tiles: a group of `count` rows has ceil(count / NT) tiles along its rows; the table is built in
// shared memory from `offsets` by every CTA, so the host never reads the counts. Columns past
// the group's last row are computed from whatever is there (each depends on its own row only)
// and never stored. Every wait is bounded (MOE_ERR_TIMEOUT in the status word).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cstddef>
#include <mutex>

#include "checks.cuh"
#include "common.cuh"
#include "kernels.cuh"
#include "launch.cuh"
#include "mx4.cuh"

namespace moe {
namespace {

constexpr int kEpiWarps = 8;                        // two per TMEM lane quarter
constexpr int kScaleWarps = 4;
constexpr int kThreads = 64 + (kEpiWarps + kScaleWarps) * 32;
constexpr uint32_t kTmemCols = 512;
// a warp's staging rows: 8 rows of 32 channels, 4 floats apart from a multiple of 32, so that
// neither the writes (a row at a time) nor the reads (16 bytes of 8 rows) meet in a bank
constexpr int kStageLd = 36;
constexpr int kGroupLd = 132;
constexpr int kEpiFloats = kEpiWarps * 8 * kStageLd;
constexpr int kEpiBytes = kEpiFloats * 4;
static_assert(kEpiFloats >= kEpiWarps / 4 * 8 * kGroupLd, "staging rows");
constexpr int W_BYTES = 128 * 128;                  // a weight block's stage: 128 rows x 128 bytes

// kStore: y in bf16; kFp32: y in fp32, stored or added to the tokens' sums; kSwiglu: h in 4 bits
enum Mode : int { kStore = 0, kFp32 = 1, kSwiglu = 2 };

// Pair kernel: plain products have a third epilogue warp per quarter (17081 rows of the 768-wide layer
// in 20.2 us instead of 21.5, 20.6 now). The rounding of h gains nothing by one, and it takes issue slots from the
// other roles (229 to 236 us instead of 221 for 16384 rows' gate and up).
constexpr int pair_epi_warps(int mode) { return mode == kSwiglu ? kEpiWarps : 12; }
constexpr int pair_threads(int mode) { return (2 + pair_epi_warps(mode) + 2 * kScaleWarps + 1) * 32; }

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
  void* out;              // kStore, kFp32: [rows, n_out] (or tokens); kSwiglu: h's codes
  uint8_t* h_scales;      // kSwiglu
  const float* h_factor;
  const int32_t* perm_token;   // kFp32: row r is added to out[perm_token[r]]; or null
  const float* row_gate;
  float scale;
  int* status;
  int test_stall;         // testing (MOE_TUNE_TEST_STALL): tile 0 leaves its first stage unloaded
};

// CPS: scale pieces of a stage along K (2: MXFP4, 4: NVFP4); NT: rows of a tile
template <int CPS>
struct One {
  static constexpr int NT = 64;
  static constexpr int T_BYTES = NT * 128;
  static constexpr int SF_BYTES = CPS * 512;               // a stage's pieces of 128 rows
  static constexpr int STAGE = 2 * W_BYTES + T_BYTES + 3 * SF_BYTES;   // two weight blocks, the rows
  static constexpr int STAGES = (227 * 1024 - 12 * 1024 - kEpiBytes) / STAGE;
  static constexpr int SF_STAGE = 16, SF_STAGES = 1;       // no ring of scales: they come with the operands
  static constexpr int SF_COL = 4 * NT;                    // after two accumulators of two blocks
  static constexpr int SF_SLOT = CPS * 10;                 // W0: CPS x 4, W1: CPS x 4, rows: CPS x 2
  static constexpr int SLOTS = STAGES;
  static_assert(STAGE % 1024 == 0, "128-byte-swizzled boxes need 1024-byte alignment");
  static_assert(SF_COL + SLOTS * SF_SLOT <= (int)kTmemCols, "TMEM budget");
};
template <int CPS>
struct Pair {
  static constexpr int NT = 192;
  static constexpr int T_BYTES = NT / 2 * 128;             // this CTA's half of the rows
  static constexpr int SF_BYTES = CPS * 512;
  static constexpr int STAGE = W_BYTES + T_BYTES;
  static constexpr int STAGES = 6;
  static constexpr int SF_STAGE = 4 * SF_BYTES;            // gate and up (or W), the rows: two scale tiles
  static constexpr int SF_BOX = CPS * 64;                  // a stage's pieces in 8-byte elements
  static constexpr int SF_STAGES = CPS == 4 ? 4 : 6;       // of a ring of their own
  static constexpr int SF_COL = 2 * NT;                    // after two accumulators
  static constexpr int SF_SLOT = CPS * 10;                 // W: CPS x 4, rows: CPS x 6
  static constexpr int FIT = ((int)kTmemCols - SF_COL) / SF_SLOT;
  static constexpr int SLOTS = FIT < STAGES ? FIT : STAGES;
  static_assert(STAGE % 1024 == 0, "128-byte-swizzled boxes need 1024-byte alignment");
  static_assert(SLOTS >= 3, "TMEM budget");
  // each of the two sets of scale warps keeps to its own stages of this ring, so that it sees every
  // phase of their barriers (one that misses a phase takes the phase before for the one it waits for)
  static_assert(SF_STAGES % 2 == 0, "a stage of scales belongs to one set of warps");
};

template <class C>
struct alignas(1024) Storage {
  uint8_t ring[C::STAGES][C::STAGE];
  alignas(128) uint8_t sring[C::SF_STAGES][C::SF_STAGE];
  uint64_t full[C::STAGES];   // operands have landed; pair, on the leader: those of both CTAs, and the
                              // scales of both CTAs are in TMEM
  uint64_t empty[C::STAGES];
  uint64_t sland[C::SF_STAGES];    // pair: this CTA's scales have landed, and have been read
  uint64_t sempty[C::SF_STAGES];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t sfull[C::SLOTS];   // one CTA: a slot of scales is in TMEM
  uint32_t tmem_base;
  int abort_flag;
  int offs[kMx4MaxGroups + 1];
  int toff[kMx4MaxGroups + 1];
  int turn_ok[kEpiWarps];     // the warps of a column range tell each other whether to go on
  // staging rows of the epilogue: [warp][8][kStageLd], or [four warps][8][kGroupLd] where the
  // warps of a channel range work together
  alignas(16) float turn[kEpiFloats];
};

struct Tile {
  int g, row0, row_end, o_g, n0, n;   // n: rows of the tile, n0: its first channel
  int blocks;                         // one CTA: weight blocks of 128 rows, 1 or 2
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
  t.n0 = nt * (g.mode == kSwiglu ? 128 : 256);
  t.blocks = g.mode == kSwiglu || t.n0 + 128 < g.n_out ? 2 : 1;
  return t;
}

// ---- tcgen05 with block scales ---------------------------------------------------------------
__device__ __forceinline__ void tmem_st_x4(uint32_t taddr, const uint4& v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ void tmem_st_x2(uint32_t taddr, uint32_t a, uint32_t b) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};" ::"r"(taddr), "r"(a), "r"(b) : "memory");
}
// P pieces of scales (512 bytes each, one after another) -> 4 P TMEM columns from taddr on, this
// warp's lane quarter: lane l holds bytes [16 l, 16 l + 16) of each piece.
template <int P>
__device__ __forceinline__ void tmem_st_scales(uint32_t taddr, const uint8_t* pieces, int lane) {
#pragma unroll
  for (int p = 0; p < P; ++p)
    tmem_st_x4(taddr + 4 * p, *reinterpret_cast<const uint4*>(pieces + p * 512 + lane * 16));
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
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

// The same by a CTA pair, issued by its leader: M = 256, 128 rows of A and N / 2 of B per CTA; each
// CTA's TMEM holds the scales of its rows of A and of all N rows of B.
template <bool NV>
__device__ __forceinline__ void umma_mx4_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                              uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  if (NV) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], "
        "[%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], "
        "[%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  }
}

// Arrive on the mbarrier at `bar` (this CTA's shared memory) and on the one at the same place in the
// pair's other CTA once the tcgen05.mma issued so far have completed.
__device__ __forceinline__ void umma_commit_both(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}

// Instruction descriptor, block-scaled 4-bit kinds: A and B e2m1 (bits 7-9 and 10-11 = 1), both
// K-major, N >> 3 in bits 17-22, scale type in bit 23 (1: e8m0, 0: e4m3), M >> 7 in bits 27-28;
// the byte of the scales' 32-bit columns that the MMA starts at: bits 4-5 (B), 29-30 (A).
template <bool NV>
__device__ __forceinline__ uint32_t idesc_mx4(int M, int N, uint32_t sf_id) {
  return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (NV ? 0u : (1u << 23)) |
         (static_cast<uint32_t>(M >> 7) << 27) | (sf_id << 4) | (sf_id << 29);
}

// The value of lane 0, which the compiler then knows to be the same in every lane.
__device__ __forceinline__ int uni(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// mbar_wait by every lane of the warp, the same answer in each: lanes that go on to read what the
// barrier guards have to wait themselves, a value shuffled from one that did orders no memory.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag));
}

// Whether the phase of the given parity is over, without waiting for it.
__device__ __forceinline__ uint32_t mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok;
}

// Tiled TMA loads of more dimensions: for a CTA pair, counted on an mbarrier of either CTA (cluster
// address), and plain ones.
__device__ __forceinline__ void tma_load_3d_pair(void* dst, const void* tmap, int c0, int c1, int c2,
                                                 uint32_t bar_cluster_addr) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(bar_cluster_addr)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(void* dst, const void* tmap, int c0, int c1, int c2, int c3, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
      : "memory");
}

// The warp's 32 channels (one per lane) of 8 rows, v[j] of row j, turned around: afterwards v[i]
// is channel 8 (lane / 8) + i of row lane % 8.
__device__ __forceinline__ void turn_around(float (&v)[8], float (*stg)[kStageLd], int lane) {
#pragma unroll
  for (int j = 0; j < 8; ++j) stg[j][lane] = v[j];
  __syncwarp();
  const float4* p = reinterpret_cast<const float4*>(&stg[lane & 7][lane & 24]);
  const float4 a = p[0], b = p[1];
  __syncwarp();                // the rows may be written again
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// The same in registers: in step b = 1, 2, 4, lanes l and l ^ b exchange the halves that the other keeps.
__device__ __forceinline__ void turn_in_registers(float (&v)[8], int lane) {
#pragma unroll
  for (int b = 1; b < 8; b <<= 1) {
    const bool up = lane & b;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j & b) continue;
      const float got = __shfl_xor_sync(0xffffffffu, up ? v[j] : v[j | b], b);
      if (up) v[j] = got;
      else v[j | b] = got;
    }
  }
}
// And rounded to bf16 on the way, two rows (then two channels) in a register.
__device__ __forceinline__ uint4 turn_to_bf16(const float (&v)[8], float f, int lane) {
  uint32_t q[4];
  const uint32_t sel = lane & 1 ? 0x3276u : 0x5410u;      // (got, own) high halves, or (own, got) low ones
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t own = pack_bf16x2(v[2 * k] * f, v[2 * k + 1] * f);
    q[k] = __byte_perm(own, __shfl_xor_sync(0xffffffffu, own, 1), sel);
  }
#pragma unroll
  for (int b = 1; b < 4; b <<= 1) {
    const bool up = lane & (2 * b);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k & b) continue;
      const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? q[k] : q[k | b], 2 * b);
      if (up) q[k] = got;
      else q[k | b] = got;
    }
  }
  return make_uint4(q[0], q[1], q[2], q[3]);
}

// The product of the two factors, each from 2^-100 to 2^100: f, after a multiplication of the sums by `by`,
// a power of two that is 1 unless the product itself leaves fp32's range. A sum other than 0 has a magnitude
// from 2^-20 on: by f and `by` it becomes infinite, or smaller than any number, only where the result is.
struct Factors {
  float f, by;
};
template <bool NV>
__device__ __forceinline__ Factors factors(const Args& g, float a, int group) {
  if (!NV || !g.w_factor) return Factors{a, 1.0f};
  const float w = g.w_factor[g.w_factor_per_group ? group : 0], f = a * w;
  if (f >= 0x1p-126f && f <= 0x1p126f) return Factors{f, 1.0f};
  return f > 1.0f ? Factors{a * 0x1p-100f * w, 0x1p100f} : Factors{a * 0x1p100f * w, 0x1p-100f};
}
// The sums as loaded, times `by`.
template <int N>
__device__ __forceinline__ void prescale(uint32_t (&v)[N], float by) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * by);
}

// silu(x) u = x / (1 + e^-x) u, in that order, each step to fp32's last place or two: h goes on to 4 bits,
// where the last places decide which way a value goes that lies half way between two numbers. (With __expf
// and __fdividef up to 16 of the 33 million elements of 16384 rows' h went another way than by fp32's own
// operations, with these none does.) The reciprocal is the hardware's estimate with one step of Newton's
// method on 1 / d; d infinite (x below -88) gives 0. It costs 16384 rows' FFN 2 % (373 us), expf and a
// division 3 %.
__device__ __forceinline__ float swiglu(float x, float u) {
  const float d = 1.0f + expf(-x);
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(d));
  const float c = fmaf(-d, r, 1.0f);
  r = fabsf(c) < 1.0f ? fmaf(r, c, r) : r;
  return x * r * u;
}

// ---- epilogues: 8 rows of the tile from row c on; v: 8 channels, from channel ch on, of row
// c + lane % 8 ------------------------------------------------------------------------------
// h rounded to 4 bits: the warp's 32 channels are one (MXFP4) or two (NVFP4) blocks of each row.
template <bool NV>
__device__ __forceinline__ void epi_round_h(const Args& a, const Tile& t, int c, int ch, int lane,
                                            const float (&h)[8], const Mx4Factor& hf) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(h[i]) & 0x7FFFFFFFu);
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 8));
  if (!NV) top = max(top, __shfl_xor_sync(0xffffffffu, top, 16));
  float by;
  const uint32_t byte = mx4_scale<NV>(__uint_as_float(top), hf, by);
  const uint32_t v = mx4_codes<NV>(h, by, __uint_as_float(top));
  const int j = lane & 7;
  if (c + j >= t.n) return;
  const int row = t.row0 + c + j;
  *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.out) + (size_t)row * (a.n_out / 2) + ch / 2) = v;
  if (lane < 8 || (NV && (lane & 8) == 0))
    a.h_scales[mx4_scale_at(t.o_g, t.g, row - t.o_g, ch / mx4_block(NV), a.n_out / (4 * mx4_block(NV)))] =
        (uint8_t)byte;
}

// y, times f: 16 (bf16) or 32 bytes per lane, 64 or 128 contiguous bytes per row and warp, where
// rows are 16-byte aligned; else value by value.
template <int MODE>
__device__ __forceinline__ void epi_store(const Args& a, const Tile& t, int c, int ch, int lane, float f,
                                          float (&v)[8]) {
  if (c + (lane & 7) >= t.n || ch >= a.n_out) return;
  const int row = t.row0 + c + (lane & 7);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= f;
  if (MODE == kStore) {
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + (size_t)row * a.n_out + ch;
    if ((a.n_out & 7) == 0) {
      *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                  pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (ch + i < a.n_out) dst[i] = __float2bfloat16_rn(v[i]);
    }
    return;
  }
  const bool add = a.perm_token != nullptr;
  const float s = add ? a.scale * a.row_gate[row] : 1.0f;
  float* dst = static_cast<float*>(a.out) + (size_t)(add ? a.perm_token[row] : row) * a.n_out + ch;
  if ((a.n_out & 7) == 0) {
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const float4 q = make_float4(s * v[i], s * v[i + 1], s * v[i + 2], s * v[i + 3]);
      if (add) atomicAdd(reinterpret_cast<float4*>(dst + i), q);
      else *reinterpret_cast<float4*>(dst + i) = q;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (ch + i >= a.n_out) break;
      if (add) atomicAdd(dst + i, s * v[i]);
      else dst[i] = v[i];
    }
  }
}

// y in bf16, rounded before it was turned around.
__device__ __forceinline__ void epi_store_bf16(const Args& a, const Tile& t, int c, int ch, int lane, const uint4& q) {
  if (c + (lane & 7) >= t.n || ch >= a.n_out) return;
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + (size_t)(t.row0 + c + (lane & 7)) * a.n_out + ch;
  if ((a.n_out & 7) == 0) {
    *reinterpret_cast<uint4*>(dst) = q;
  } else {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (ch + i < a.n_out) reinterpret_cast<uint16_t*>(dst)[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
  }
}

// The tables of the groups' rows and row tiles, by every thread of the CTA. Offsets outside the matrix are
// clamped and reported; where some are out of order there are no tiles at all (their rows, counted several
// times, would have no bound that the tiles' indices are made for).
template <class S>
__device__ __forceinline__ void build_table(S& s, const Args& g, int NT) {
  for (int i = threadIdx.x; i <= g.a.groups; i += blockDim.x) {
    const int o = g.a.begin(i), c = min(max(o, 0), g.a.rows);
    if (o != c || (i == 0 && o != 0)) set_status(g.status, MOE_ERR_DEVICE_CHECK);
    s.offs[i] = c;
  }
  __syncthreads();
  if (threadIdx.x >= 64 && threadIdx.x < 96) {
    // toff[e] = sum over e' < e of ceil(count_e' / NT)
    const int lane = threadIdx.x & 31;
    const int per = (g.a.groups + 31) / 32;
    const int b = lane * per;
    bool ordered = true;
    auto tiles_of = [&](int e) {
      const int n = s.offs[e + 1] - s.offs[e];
      if (n < 0) ordered = false;
      return n > 0 ? (n + NT - 1) / NT : 0;
    };
    int local = 0;
    for (int i = 0; i < per; ++i)
      if (b + i < g.a.groups) local += tiles_of(b + i);
    if (!__all_sync(0xffffffffu, ordered)) {
      set_status(g.status, MOE_ERR_DEVICE_CHECK);
      if (lane == 31) s.toff[g.a.groups] = 0;
      return;
    }
    const int inc = warp_inclusive_scan(local);
    int run = inc - local;
    for (int i = 0; i < per; ++i)
      if (b + i < g.a.groups) {
        s.toff[b + i] = run;
        run += tiles_of(b + i);
      }
    if (lane == 31) s.toff[g.a.groups] = inc;
  }
}

// The first scale pieces of the 128-row tile of group g that has its row l.
__device__ __forceinline__ const uint8_t* scale_tile(const uint8_t* scales, int64_t o_g, int g, int l, int chunks) {
  return scales + ((size_t)(o_g >> 7) + g + (l >> 7)) * chunks * 512;
}

template <int CPS, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    k_mx4_gemm(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA64,
               const __grid_constant__ CUtensorMap tmA16, const Args g) {
  using C = One<CPS>;
  constexpr bool NV = CPS == 4;
  constexpr int STAGES = C::STAGES, NT = C::NT;
  extern __shared__ uint8_t smem_raw[];
  auto& s = *reinterpret_cast<Storage<C>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = uni(threadIdx.x >> 5), lane = threadIdx.x & 31;
  pdl_launch_dependents();

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.tfull[i], 1);
      mbar_init(&s.tempty[i], kEpiWarps);
    }
    for (int i = 0; i < C::SLOTS; ++i) mbar_init(&s.sfull[i], kScaleWarps);
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
  build_table(s, g, NT);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;
  const int total = uni(s.toff[g.a.groups] * g.n_tiles);
  volatile int* abort_flag = &s.abort_flag;

  // The producer and the issuer run as whole warps in step, on values that the compiler knows to be
  // uniform, and one lane issues: TMA, MMA and commit take their operands from uniform registers.
  if (warp == 0) {
    // ---- TMA producer --------------------------------------------------------------------
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int tile = blockIdx.x; ok && tile < total; tile += gridDim.x) {
      const Tile t = decode(s, g, tile, NT);
      const int n = uni(t.n), grp = uni(t.g), n0 = uni(t.n0), row0 = uni(t.row0), o_g = uni(t.o_g);
      const bool two = uni(t.blocks) == 2;
      const int small = n < NT ? (n + 15) / 16 : 0;          // boxes of 16 rows, or one of 64
      const int wrow = grp * g.w_rows + n0;
      const int64_t wo = (int64_t)grp * g.w_rows;
      const uint8_t* sw = scale_tile(g.w_scales, wo, grp, n0, g.chunks);
      const uint8_t* sw2 = scale_tile(g.w_scales, wo, grp, n0 + g.w_second, g.chunks);
      const uint8_t* sa = scale_tile(g.a_scales, o_g, grp, row0 - o_g, g.chunks);
      for (int kb = 0; kb < g.kstages; ++kb) {
        ok = warp_wait(&s.empty[stage], phase ^ 1u, abort_flag);
        if (!ok) break;
        if (!(g.test_stall && tile + kb == 0) && elect_one()) {
          uint8_t* st = s.ring[stage];
          uint64_t* bar = &s.full[stage];
          const uint32_t sfb = 512u * (uint32_t)min(CPS, g.chunks - kb * CPS);
          mbar_arrive_expect_tx(bar, (two ? 2 : 1) * (W_BYTES + sfb) + (small ? small * 16 : NT) * 128 + sfb);
          tma_load_2d(st, &tmW, kb * 128, wrow, bar);
          if (two) tma_load_2d(st + W_BYTES, &tmW, kb * 128, wrow + g.w_second, bar);
          uint8_t* rows = st + 2 * W_BYTES;
          if (!small) tma_load_2d(rows, &tmA64, kb * 128, row0, bar);
          for (int i = 0; i < small; ++i) tma_load_2d(rows + i * 16 * 128, &tmA16, kb * 128, row0 + i * 16, bar);
          uint8_t* sf = rows + C::T_BYTES;
          const size_t at = (size_t)kb * CPS * 512;
          bulk_load(sf, sw + at, sfb, bar);
          if (two) bulk_load(sf + C::SF_BYTES, sw2 + at, sfb, bar);
          bulk_load(sf + 2 * C::SF_BYTES, sa + at, sfb, bar);     // 64 rows lie in one scale tile
        }
        __syncwarp();
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp == 1) {
    // ---- MMA issuer --------------------------------------------------------------------------
    int stage = 0;
    uint32_t phase = 0;
    int acc = 0;
    uint32_t acc_phase = 0;
    int sl = 0;                // slot of scales
    uint32_t sl_phase = 0;
    bool ok = true;
    for (int tile = blockIdx.x; ok && tile < total; tile += gridDim.x) {
      const Tile t = decode(s, g, tile, NT);
      const int npad = (uni(t.n) + 15) & ~15;
      const bool two = uni(t.blocks) == 2;
      ok = warp_wait(&s.tempty[acc], acc_phase ^ 1u, abort_flag);
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem + (uint32_t)(acc * 2 * NT);
      for (int kb = 0; kb < g.kstages; ++kb) {
        ok = warp_wait(&s.full[stage], phase, abort_flag) && warp_wait(&s.sfull[sl], sl_phase, abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t w0 = smem_u32(s.ring[stage]);
          const uint32_t rows = w0 + 2 * W_BYTES;
          const uint32_t slot = tmem + C::SF_COL + (uint32_t)sl * C::SF_SLOT;
          const int ksteps = min(CPS, g.chunks - kb * CPS) * (4 / CPS);      // K = 64 each
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (k >= ksteps) break;
            const uint32_t p = k / (4 / CPS);
            const uint32_t idesc = idesc_mx4<NV>(128, npad, NV ? 0u : 2u * (k & 1));
            const uint64_t db = sw128_kmajor_desc(rows + k * 32);
            const uint32_t sfb = slot + CPS * 8 + 2 * p;
            const uint32_t go = (kb > 0 || k > 0) ? 1u : 0u;
            umma_mx4<NV>(d, sw128_kmajor_desc(w0 + k * 32), db, idesc, slot + 4 * p, sfb, go);
            if (two)
              umma_mx4<NV>(d + NT, sw128_kmajor_desc(w0 + W_BYTES + k * 32), db, idesc, slot + CPS * 4 + 4 * p,
                           sfb, go);
          }
          umma_commit(&s.empty[stage]);
        }
        __syncwarp();
        if (++sl == C::SLOTS) {
          sl = 0;
          sl_phase ^= 1u;
        }
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      if (elect_one()) umma_commit(&s.tfull[acc]);
      __syncwarp();
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
  } else if (warp >= 2 + kEpiWarps) {
    // ---- scales: shared memory -> this warp's lane quarter of TMEM ----------------------------
    const uint32_t quarter = (uint32_t)((warp & 3) * 32) << 16;
    int stage = 0;
    uint32_t phase = 0;
    int sl = 0;
    bool ok = true;
    for (int tile = blockIdx.x; ok && tile < total; tile += gridDim.x) {
      const Tile t = decode(s, g, tile, NT);
      const int upper = ((t.row0 - t.o_g) & 64) / 8;         // the rows' half of their scale tile
      for (int kb = 0; kb < g.kstages; ++kb) {
        ok = warp_wait(&s.full[stage], phase, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const uint8_t* sf = s.ring[stage] + 2 * W_BYTES + C::T_BYTES;
        const uint32_t slot = tmem + quarter + C::SF_COL + (uint32_t)sl * C::SF_SLOT;
        // pieces past the row's end hold an earlier stage's scales: written, never used
        tmem_st_scales<CPS>(slot, sf, lane);
        if (t.blocks == 2) tmem_st_scales<CPS>(slot + CPS * 4, sf + C::SF_BYTES, lane);
#pragma unroll
        for (int p = 0; p < CPS; ++p) {
          const uint2 v = *reinterpret_cast<const uint2*>(sf + 2 * C::SF_BYTES + p * 512 + lane * 16 + upper);
          tmem_st_x2(slot + CPS * 8 + 2 * p, v.x, v.y);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.sfull[sl]);
        if (++sl == C::SLOTS) sl = 0;
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else {
    // ---- epilogue: TMEM lane quarter = warp % 4; the two warps of a quarter take turns over
    // chunks of 16 columns ----------------------------------------------------------------------
    const int q = warp & 3;
    const int part = (warp - 2) >> 2;
    float (*stg)[kStageLd] = reinterpret_cast<float (*)[kStageLd]>(s.turn + (warp - 2) * 8 * kStageLd);
    int acc = 0;
    uint32_t acc_phase = 0;
    const float af = NV && g.a_factor ? *g.a_factor : 1.0f;
    const Mx4Factor hf = mx4_factor(NV && MODE == kSwiglu && g.h_factor ? *g.h_factor : 1.0f);
    for (int tile = blockIdx.x; tile < total; tile += gridDim.x) {
      const Tile t = decode(s, g, tile, NT);
      const auto [f, by] = factors<NV>(g, af, t.g);
      if (!warp_wait(&s.tfull[acc], acc_phase, abort_flag)) break;
      tc_fence_after();
      const uint32_t base = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * 2 * NT);
      const int ch = t.n0 + 32 * q + (lane & ~7);
#pragma unroll 1
      for (int c = 16 * part; c < t.n; c += 16 * (kEpiWarps / 4)) {
        uint32_t v[2][16];
        tmem_ld_32x32b_x16(base + c, v[0]);
        tmem_ld_32x32b_x16(base + NT + c, v[1]);
        tmem_ld_wait_for(v[0], v[1]);
        if (NV && by != 1.0f) {
          prescale(v[0], by);
          prescale(v[1], by);
        }
#pragma unroll
        for (int e = 0; e < 16; e += 8) {
          float x[8];
          if constexpr (MODE == kSwiglu) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              x[j] = swiglu(__uint_as_float(v[0][e + j]) * f, __uint_as_float(v[1][e + j]) * f);
            turn_around(x, stg, lane);
            epi_round_h<NV>(g, t, c + e, ch, lane, x, hf);
            __syncwarp();
          } else {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              if (b == t.blocks) break;
#pragma unroll
              for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(v[b][e + j]);
              turn_around(x, stg, lane);
              epi_store<MODE>(g, t, c + e, ch + 128 * b, lane, f, x);
              __syncwarp();
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.tempty[acc]);
      acc ^= 1;
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

// ---- CTA pairs ---------------------------------------------------------------------------------
// h of the pair kernel, where lanes 0-63 hold the gate and 64-127 the up rows of the CTA's 64
// channels: the four warps of a column range (one per lane quarter) have staged 8 rows from c on as
// S[row][TMEM lane]; this warp takes rows 2 q and 2 q + 1, 4 channels per lane. ch: the CTA's first
// channel.
template <bool NV>
__device__ __forceinline__ void epi_round_h_pair(const Args& a, const Tile& t, int c, int ch, int q, int lane, float f,
                                                 const float (*S)[kGroupLd], const Mx4Factor& hf) {
  const int r = 2 * q + (lane >> 4), k = 4 * (lane & 15);
  const float4 G = *reinterpret_cast<const float4*>(&S[r][k]);
  const float4 U = *reinterpret_cast<const float4*>(&S[r][64 + k]);
  const float gv[4] = {G.x, G.y, G.z, G.w}, uv[4] = {U.x, U.y, U.z, U.w};
  float h[4];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = swiglu(gv[i] * f, uv[i] * f);
    top = max(top, __float_as_uint(h[i]) & 0x7FFFFFFFu);
  }
#pragma unroll
  for (int o = 1; o < mx4_block(NV) / 4; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  float by;
  const uint32_t byte = mx4_scale<NV>(__uint_as_float(top), hf, by);
  const uint32_t v = mx4_codes<NV>(h, by, __uint_as_float(top));
  if (c + r < t.n) {
    const int row = t.row0 + c + r;
    *reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(a.out) + (size_t)row * (a.n_out / 2) + (ch + k) / 2) = (uint16_t)v;
    if (k % mx4_block(NV) == 0)
      a.h_scales[mx4_scale_at(t.o_g, t.g, row - t.o_g, (ch + k) / mx4_block(NV), a.n_out / (4 * mx4_block(NV)))] =
          (uint8_t)byte;
  }
}

// The epilogue warps of one column range (four warps) meet here; named barriers 1 and 2.
__device__ __forceinline__ void range_bar(int part) { asm volatile("bar.sync %0, 128;" ::"r"(part + 1) : "memory"); }

template <int CPS, int MODE>
__global__ void __launch_bounds__(pair_threads(MODE), 1)
    k_mx4_gemm_pair(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA96,
                    const __grid_constant__ CUtensorMap tmA16, const __grid_constant__ CUtensorMap tmSW,
                    const __grid_constant__ CUtensorMap tmSA, const Args g) {
  using C = Pair<CPS>;
  constexpr bool NV = CPS == 4;
  constexpr int STAGES = C::STAGES, NT = C::NT, EPI = pair_epi_warps(MODE);
  extern __shared__ uint8_t smem_raw[];
  auto& s = *reinterpret_cast<Storage<C>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = uni(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();            // 0: leader, 1: peer
  const int cluster = blockIdx.x >> 1, nclusters = gridDim.x >> 1;
  pdl_launch_dependents();

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&s.full[i], 1 + 2 * kScaleWarps);
      mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < C::SF_STAGES; ++i) {
      mbar_init(&s.sland[i], 1);
      mbar_init(&s.sempty[i], kScaleWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.tfull[i], 1);
      mbar_init(&s.tempty[i], 2 * EPI);
    }
    s.abort_flag = 0;
    fence_barrier_init();
    prefetch_tensormap(&tmW);
    prefetch_tensormap(&tmA96);
    prefetch_tensormap(&tmA16);
    prefetch_tensormap(&tmSW);
    prefetch_tensormap(&tmSA);
  }
  pdl_wait();
  __syncthreads();
  cluster_sync();                                     // both CTAs' barriers initialised
  if (warp == 1) {
    tmem_alloc_pair(&s.tmem_base, kTmemCols);
    tmem_relinquish_pair();
  }
  build_table(s, g, NT);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;
  const int total = uni(s.toff[g.a.groups] * g.n_tiles);
  volatile int* abort_flag = &s.abort_flag;

  // whole warps in step with one lane issuing, as in k_mx4_gemm
  if (warp == 0) {
    // ---- TMA producer of the operands (both CTAs), counted on the leader. A thread issues a copy every
    // 140 cycles or so, whatever its size: two copies per stage here and two of scales below
    // (one thread for all seven plain ones took 600 us for 32768 rows) -----------------------------
    int stage = 0;
    uint32_t phase = 0;
    uint32_t ready = 0;          // the coming stage was seen to be empty
    bool ok = true;
    for (int tile = cluster; ok && tile < total; tile += nclusters) {
      const Tile t = decode(s, g, tile, NT);
      const int mine = ((uni(t.n) + 31) & ~31) / 2;          // rows of this CTA's half
      const int arow = uni(t.row0) + mine * (int)rank;
      const int grp = uni(t.g);
      // this CTA's first weight row in its group; past the group's end (an odd number of 128-row
      // blocks) the boxes read on or are zeros: those channels are dropped
      const int wl = uni(t.n0) + (MODE == kSwiglu ? 64 : 128) * (int)rank;
      for (int kb = 0; kb < g.kstages; ++kb) {
        if (!__all_sync(0xffffffffu, ready)) ok = warp_wait(&s.empty[stage], phase ^ 1u, abort_flag);
        if (!ok) break;
        const int next = stage + 1 == STAGES ? 0 : stage + 1;
        ready = mbar_test(&s.empty[next], next ? phase ^ 1u : phase);
        if (!(g.test_stall && tile + kb == 0) && elect_one()) {      // (neither CTA loads)
          uint8_t* st = s.ring[stage];
          const uint32_t full = mapa_shared(smem_u32(&s.full[stage]), 0);
          if (rank == 0) mbar_arrive_expect_tx(&s.full[stage], 2 * (W_BYTES + mine * 128));
          if (MODE == kSwiglu) tma_load_3d_pair(st, &tmW, kb * 128, wl, 2 * grp, full);
          else tma_load_2d_pair(st, &tmW, kb * 128, grp * g.w_rows + wl, full);
          uint8_t* rows = st + W_BYTES;
          if (mine == NT / 2) {
            tma_load_2d_pair(rows, &tmA96, kb * 128, arow, full);
          } else {
            for (int i = 0; i < mine; i += 16) tma_load_2d_pair(rows + i * 128, &tmA16, kb * 128, arow + i, full);
          }
        }
        __syncwarp();
        stage = next;
        if (next == 0) phase ^= 1u;
      }
    }
  } else if (warp == 2 + EPI + 2 * kScaleWarps) {
    // ---- TMA producer of the scales, counted on this CTA, into a ring that the scale warps free
    // as soon as they have read a stage. Always two scale tiles of rows: what the tile does not have
    // of them is any group's or zeros, and not used ----------------------------------------------
    int stage = 0;
    uint32_t phase = 0;
    uint32_t ready = 0;
    bool ok = true;
    for (int tile = cluster; ok && tile < total; tile += nclusters) {
      const Tile t = decode(s, g, tile, NT);
      const int grp = uni(t.g), o_g = uni(t.o_g);
      const int ta = (o_g >> 7) + grp + ((uni(t.row0) - o_g) >> 7);
      // kSwiglu: the tile of the 128 channels; else the CTA's own one, the group's last one where the
      // CTA has no channels
      const int wl = uni(t.n0) + (MODE == kSwiglu ? 0 : min(128 * (int)rank, g.w_rows - 1 - uni(t.n0)));
      const int tw = MODE == kSwiglu ? wl >> 7 : (int)(((int64_t)grp * g.w_rows) >> 7) + grp + (wl >> 7);
      for (int kb = 0; kb < g.kstages; ++kb) {
        if (!__all_sync(0xffffffffu, ready)) ok = warp_wait(&s.sempty[stage], phase ^ 1u, abort_flag);
        if (!ok) break;
        const int next = stage + 1 == C::SF_STAGES ? 0 : stage + 1;
        ready = mbar_test(&s.sempty[next], next ? phase ^ 1u : phase);
        if (elect_one()) {
          uint8_t* sf = s.sring[stage];
          uint64_t* bar = &s.sland[stage];
          mbar_arrive_expect_tx(bar, C::SF_BYTES * (MODE == kSwiglu ? 4 : 3));
          if (MODE == kSwiglu) tma_load_4d(sf, &tmSW, kb * C::SF_BOX, tw, 0, grp, bar);
          else tma_load_2d(sf, &tmSW, kb * C::SF_BOX, tw, bar);
          tma_load_2d(sf + 2 * C::SF_BYTES, &tmSA, kb * C::SF_BOX, ta, bar);
        }
        __syncwarp();
        stage = next;
        if (next == 0) phase ^= 1u;
      }
    }
  } else if (warp == 1) {
    // ---- MMA issuer (leader only) ------------------------------------------------------------
    int stage = 0;
    uint32_t phase = 0;
    int acc = 0;
    uint32_t acc_phase = 0;
    int sl = 0;                // slot of scales
    uint32_t ready = 0;        // the coming stage was seen to be full
    bool ok = rank == 0;
    for (int tile = cluster; ok && tile < total; tile += nclusters) {
      const Tile t = decode(s, g, tile, NT);
      const int npad = (uni(t.n) + 31) & ~31;
      ok = warp_wait(&s.tempty[acc], acc_phase ^ 1u, abort_flag);
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem + (uint32_t)(acc * NT);
      for (int kb = 0; kb < g.kstages; ++kb) {
        if (!__all_sync(0xffffffffu, ready)) ok = warp_wait(&s.full[stage], phase, abort_flag);
        if (!ok) break;
        tc_fence_after();
        // look at the next stage's barrier before this stage's MMAs: the answer takes a while
        const int next = stage + 1 == STAGES ? 0 : stage + 1;
        ready = mbar_test(&s.full[next], next ? phase : phase ^ 1u);
        if (elect_one()) {
          const uint32_t w0 = smem_u32(s.ring[stage]);
          const uint32_t rows = w0 + W_BYTES;
          const uint32_t slot = tmem + C::SF_COL + (uint32_t)sl * C::SF_SLOT;
          const int ksteps = min(CPS, g.chunks - kb * CPS) * (4 / CPS);      // K = 64 each
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (k >= ksteps) break;
            const uint32_t p = k / (4 / CPS);
            umma_mx4_pair<NV>(d, sw128_kmajor_desc(w0 + k * 32), sw128_kmajor_desc(rows + k * 32),
                              idesc_mx4<NV>(256, npad, NV ? 0u : 2u * (k & 1)), slot + 4 * p,
                              slot + CPS * 4 + 6 * p, (kb > 0 || k > 0) ? 1u : 0u);
          }
          umma_commit_both(&s.empty[stage]);
        }
        __syncwarp();
        if (++sl == C::SLOTS) sl = 0;
        stage = next;
        if (next == 0) phase ^= 1u;
      }
      if (!ok) break;
      if (elect_one()) umma_commit_both(&s.tfull[acc]);
      __syncwarp();
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
  } else if (warp >= 2 + EPI) {
    // ---- scales of both CTAs: shared memory -> this warp's lane quarter of TMEM. A stage takes a
    // warp some 560 cycles, longer than its MMAs: two sets of four warps take turns ---------------
    const uint32_t quarter = (uint32_t)((warp & 3) * 32) << 16;
    const int set = (warp - 2 - EPI) / kScaleWarps;
    int turn = 0;                // of the set whose stage it is
    int stage = set;             // this set's next one, of the scales' ring,
    uint32_t phase = 0;
    int ostage = set;            // of the operands' ring,
    int sl = set;                // and its slot
    // the stage SLOTS ago, whose MMAs read the slot last
    int before = STAGES - C::SLOTS + set;
    uint32_t before_phase = 1;   // the first waits return at once
    bool ok = true;
    for (int tile = cluster; ok && tile < total; tile += nclusters) {
      const Tile t = decode(s, g, tile, NT);
      // the rows start at the first or the third of their first scale tile's four columns
      const int off = (t.row0 - t.o_g) & 127;
      const bool two = off + t.n > 128;
      // kSwiglu: the CTA's 64 channels are the first or the second half of their scale tile
      const int upper = MODE == kSwiglu ? 8 * (int)rank : 0;
      for (int kb = 0; kb < g.kstages; ++kb) {
        turn ^= 1;
        if ((turn ^ 1) != set) continue;
        ok = warp_wait(&s.sland[stage], phase, abort_flag);
        if (!ok) break;
        // (pieces past the row's end are zeros: written, never used)
        const uint8_t* sf = s.sring[stage] + lane * 16;
        uint4 w[CPS], r[CPS];
        uint2 r2[CPS];
#pragma unroll
        for (int p = 0; p < CPS; ++p) {
          if (MODE == kSwiglu) {
            // columns 0, 1: 64 gate rows, 2, 3: the same up rows
            const uint2 a = *reinterpret_cast<const uint2*>(sf + p * 512 + upper);
            const uint2 b = *reinterpret_cast<const uint2*>(sf + C::SF_BYTES + p * 512 + upper);
            w[p] = make_uint4(a.x, a.y, b.x, b.y);
          } else {
            w[p] = *reinterpret_cast<const uint4*>(sf + p * 512);
          }
          const uint8_t* piece = sf + 2 * C::SF_BYTES + p * 512;
          const uint4 a = *reinterpret_cast<const uint4*>(piece);
          const uint4 b = two ? *reinterpret_cast<const uint4*>(piece + C::SF_BYTES) : make_uint4(0, 0, 0, 0);
          r[p] = off ? make_uint4(a.z, a.w, b.x, b.y) : a;
          r2[p] = off ? make_uint2(b.z, b.w) : make_uint2(b.x, b.y);
        }
        ok = warp_wait(&s.empty[before], before_phase, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const uint32_t slot = tmem + quarter + C::SF_COL + (uint32_t)sl * C::SF_SLOT;
#pragma unroll
        for (int p = 0; p < CPS; ++p) {
          tmem_st_x4(slot + 4 * p, w[p]);
          tmem_st_x4(slot + CPS * 4 + 6 * p, r[p]);
          tmem_st_x2(slot + CPS * 4 + 6 * p + 4, r2[p].x, r2[p].y);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        // Like the accumulators, TMEM columns are handed over by the tcgen05 fences. The place in the
        // ring is free only now that the stores have taken the scales: an arrival does not wait for
        // loads that are under way, and those here take long, with the MMAs reading shared memory at
        // its rate. (Freed after the loads, places were filled again in the middle of them: 88 of 1600
        // products of 32768 rows, or all, by the wait before it, had channels with a later stage's scales.)
        if (lane == 0) {
          mbar_arrive_cluster(mapa_shared(smem_u32(&s.full[ostage]), 0));
          mbar_arrive(&s.sempty[stage]);
        }
        ostage += 2;
        if (ostage >= STAGES) ostage -= STAGES;
        sl += 2;
        if (sl >= C::SLOTS) sl -= C::SLOTS;
        before += 2;
        if (before >= STAGES) {
          before -= STAGES;
          before_phase ^= 1u;
        }
        stage += 2;
        if (stage >= C::SF_STAGES) {
          stage -= C::SF_STAGES;
          phase ^= 1u;
        }
      }
    }
  } else {
    // ---- epilogue (both CTAs): this CTA's 128 weight rows; the warps of a quarter take turns
    // over chunks of 16 columns -----------------------------------------------------------
    const int q = warp & 3;
    const int part = (warp - 2) >> 2;
    float (*S)[kGroupLd] = reinterpret_cast<float (*)[kGroupLd]>(s.turn + part * 8 * kGroupLd);
    int acc = 0;
    uint32_t acc_phase = 0;
    const float af = NV && g.a_factor ? *g.a_factor : 1.0f;
    const Mx4Factor hf = mx4_factor(NV && MODE == kSwiglu && g.h_factor ? *g.h_factor : 1.0f);
    for (int tile = cluster; tile < total; tile += nclusters) {
      const Tile t = decode(s, g, tile, NT);
      const auto [f, by] = factors<NV>(g, af, t.g);
      int w_ok = warp_wait(&s.tfull[acc], acc_phase, abort_flag) ? 1 : 0;
      // all four warps of a range leave together: they meet at its barrier
      if (MODE == kSwiglu) {
        if (lane == 0) s.turn_ok[warp - 2] = w_ok;
        range_bar(part);
        w_ok = s.turn_ok[4 * part] & s.turn_ok[4 * part + 1] & s.turn_ok[4 * part + 2] & s.turn_ok[4 * part + 3];
        range_bar(part);
      }
      if (!w_ok) break;
      tc_fence_after();
      const uint32_t base = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * NT);
#pragma unroll 1
      for (int c = 16 * part; c < t.n; c += 16 * (EPI / 4)) {
        uint32_t v[16];
        tmem_ld_32x32b_x16(base + c, v);
        tmem_ld_wait_for(v);
        if (NV && by != 1.0f) prescale(v, by);
        if constexpr (MODE == kSwiglu) {
#pragma unroll
          for (int e = 0; e < 16; e += 8) {
#pragma unroll
            for (int j = 0; j < 8; ++j) S[j][32 * q + lane] = __uint_as_float(v[e + j]);
            range_bar(part);
            epi_round_h_pair<NV>(g, t, c + e, t.n0 + 64 * (int)rank, q, lane, f, S, hf);
            range_bar(part);                         // the rows may be written again
          }
        } else {
#pragma unroll
          for (int e = 0; e < 16; e += 8) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(v[e + j]);
            const int ch = t.n0 + 128 * (int)rank + 32 * q + (lane & ~7);
            if constexpr (MODE == kStore) {
              epi_store_bf16(g, t, c + e, ch, lane, turn_to_bf16(x, f, lane));
            } else {
              turn_in_registers(x, lane);
              epi_store<MODE>(g, t, c + e, ch, lane, f, x);
            }
            __syncwarp();
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&s.tempty[acc]), 0));
      acc ^= 1;
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
  cluster_sync();            // neither CTA leaves while the other may still signal it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// ---- host side -------------------------------------------------------------------------------
template <int CPS, int MODE>
int launch_one(const moe_mx4_t& a, const moe_mx4_t& w, const Args& g, const DeviceInfo& dev, cudaStream_t st) {
  constexpr size_t smem = sizeof(Storage<One<CPS>>) + 1024;
  static_assert(smem <= 227 * 1024 && One<CPS>::STAGES >= 3, "shared memory budget");
  CUtensorMap mw, a64, a16;
  MOE_TRY(make_byte_map(&mw, w.codes, (uint64_t)w.rows, a.K / 2, 128));
  MOE_TRY(make_byte_map(&a64, a.codes, (uint64_t)a.rows, a.K / 2, 64));
  MOE_TRY(make_byte_map(&a16, a.codes, (uint64_t)a.rows, a.K / 2, 16));
  auto kern = k_mx4_gemm<CPS, MODE>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return MOE_ERR_CUDA;
  const cudaError_t e = launch_kernel(kern, dev.sm_count, kThreads, smem, st, 1, mw, a64, a16, g);
  count_launch();
  return cuda_rc(e);
}

template <int CPS, int MODE>
int launch_pair(const moe_mx4_t& a, const moe_mx4_t& w, const Args& g, const DeviceInfo& dev, cudaStream_t st) {
  constexpr size_t smem = sizeof(Storage<Pair<CPS>>) + 1024;
  static_assert(smem <= 227 * 1024 && Pair<CPS>::STAGES >= 3, "shared memory budget");
  CUtensorMap mw, a96, a16, sw, sa;
  const uint64_t half = a.K / 2, piece_row = (uint64_t)g.chunks * 512;
  const CUtensorMapDataType eight = CU_TENSOR_MAP_DATA_TYPE_FLOAT64;    // 8 bytes an element: boxes of 256
  if (MODE == kSwiglu) {
    // [groups, gate | up, I rows]: one box has 64 gate rows and the same up rows
    const uint64_t I = g.n_out, tiles = I / 128;
    const uint64_t wd[3] = {half, I, 2ull * w.groups}, ws[2] = {half, I * half};
    const uint32_t wb[3] = {128, 64, 2};
    MOE_TRY(make_tiled_map(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, w.codes, 3, wd, ws, wb, true));
    // a group has 2 I / 128 scale tiles and one to spare
    const uint64_t sd[4] = {piece_row / 8, tiles, 2, (uint64_t)w.groups};
    const uint64_t ss[3] = {piece_row, tiles * piece_row, (2 * tiles + 1) * piece_row};
    const uint32_t sb[4] = {Pair<CPS>::SF_BOX, 1, 2, 1};
    MOE_TRY(make_tiled_map(&sw, eight, w.scales, 4, sd, ss, sb, false));
  } else {
    MOE_TRY(make_byte_map(&mw, w.codes, (uint64_t)w.rows, half, 128));
    const uint64_t sd[2] = {piece_row / 8, mx4_scale_tiles(w)}, ss[1] = {piece_row};
    const uint32_t sb[2] = {Pair<CPS>::SF_BOX, 1};
    MOE_TRY(make_tiled_map(&sw, eight, w.scales, 2, sd, ss, sb, false));
  }
  MOE_TRY(make_byte_map(&a96, a.codes, (uint64_t)a.rows, half, 96));
  MOE_TRY(make_byte_map(&a16, a.codes, (uint64_t)a.rows, half, 16));
  const uint64_t ad[2] = {piece_row / 8, mx4_scale_tiles(a)}, as[1] = {piece_row};
  const uint32_t ab[2] = {Pair<CPS>::SF_BOX, 2};
  MOE_TRY(make_tiled_map(&sa, eight, a.scales, 2, ad, as, ab, false));
  auto kern = k_mx4_gemm_pair<CPS, MODE>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return MOE_ERR_CUDA;
  // as many clusters as fit at once (cached per device), so that no CTA of the persistent tile
  // loop waits for a cluster's place
  static std::mutex mu;
  static int clusters_of[64] = {0};
  int n;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (clusters_of[dev.device] == 0) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 2;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.gridDim = dim3(dev.sm_count & ~1);
      cfg.blockDim = dim3(pair_threads(MODE));
      cfg.dynamicSmemBytes = smem;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int fit = 0;
      if (cudaOccupancyMaxActiveClusters(&fit, kern, &cfg) != cudaSuccess || fit < 1) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
      }
      clusters_of[dev.device] = min(fit, dev.sm_count / 2);
    }
    n = clusters_of[dev.device];
  }
  const cudaError_t e = launch_kernel(kern, 2 * n, pair_threads(MODE), smem, st, 2, mw, a96, a16, sw, sa, g);
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
  g.test_stall = take_test_stall(3) ? 1 : 0;
  // Up to 64 rows per group on average (of the rows there may be: the host does not know the groups' sizes):
  // one CTA per tile. In us, one CTA / pairs, MXFP4, 512 groups with 4096 x 6144 weights, of which some have
  // rows, as many each:
  //   rows each        16          64          96          128         256        512
  //   512 groups   1024 / 1132 1104 / 1235 2147 / 1320 1959 / 1413
  //   60            130 / 135   140 / 143   178 / 149   188 / 156   337 / 256   697 / 402
  //   20             56 / 57     61 / 60     73 / 62     75 / 63    122 / 90    235 / 137
  // The border is 64 rows of a group that has any. Where few of many groups have them, the rule keeps to the
  // one-CTA kernel past it.
  const bool few = a.rows <= 64ll * a.groups;
#define MX4_LAUNCH(KERNEL, CPS)                                              \
  (swiglu             ? KERNEL<CPS, kSwiglu>(a, w, g, dev, st)               \
   : g.mode == kStore ? KERNEL<CPS, kStore>(a, w, g, dev, st)                \
                      : KERNEL<CPS, kFp32>(a, w, g, dev, st))
  return is_nv(a) ? (few ? MX4_LAUNCH(launch_one, 4) : MX4_LAUNCH(launch_pair, 4))
                  : (few ? MX4_LAUNCH(launch_one, 2) : MX4_LAUNCH(launch_pair, 2));
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
  g.mode = dtype == MOE_FP32 ? kFp32 : kStore;
  g.out = out;
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
  } else if (row_gate) {
    return MOE_ERR_INVALID_ARG;
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
  d.mode = dtype == MOE_FP32 ? kFp32 : kStore;
  d.out = out;
  d.perm_token = perm_token;
  d.row_gate = row_gate;
  d.scale = scale;
  d.status = static_cast<int*>(ws);
  return launch_product(h, *w_down, d, dev, as_stream(stream));
}

}  // extern "C"
