// kda_gdr_prefill.hip - the gated delta rule over whole prompts, in chunks
// of 32 tokens (16 for fp32 rows of 128 keys) on the matrix cores
// (kda_gdr_prefill).
//
// Mathematics.  One decay per token and head, G_i its log summed from the
// chunk's start, S0 the state before the chunk:
//   A_ij = beta_i e^(G_i - G_j) kh_i.kh_j          (i > j)
//   T    = (I + A)^-1 diag(beta)                   (lower triangular)
//   U    = T (V - diag(e^G) Kh S0)
//   P_ij = e^(G_i - G_j) qh_i.kh_j / scale         (i >= j)
//   O    = diag(e^G) Qh S0 + scale P U
//   S    = e^(G_last) S0 + (diag(e^(G_last - G)) Kh)^T U
// Unlike a decay per key channel, a decay per token factors out of the
// products: A and P are plain Gram matrices of the raw q and k with factors
// on rows and columns.
//
// Precision.  All products run on the fp16 matrix instructions with fp32
// sums.  fp16 has 11 significant bits and little range, so operands enter
// as follows:
//   - a row of q or k is divided by a power of two near its norm; a bf16 row
//     then is exact in fp16 (but for values below 2^-17 of the norm, off by
//     at most 2^-25 of it), an fp32 row is taken as hi + lo, 22 bits;
//   - the state, R = V - diag(e^G) Kh S0 and U are held in a unit 2^sig per
//     value column, which keeps them below 2^15, and taken as hi + lo; T and P,
//     whose entries are at most 1 in size, times 2^14 as hi + lo.
// |T_ij| <= 1: T_ij = -beta_i kh_i^T [product of contractions] kh_j.  The
// lo.lo terms (2^-22) are dropped.  So an operand carries about 22 bits and
// the result is close to fp32's; two bf16 terms would leave 16 bits.  G is
// kept as a sum of two floats (summed in fp64): only differences of it count
// and an fp32 sum of strong decays loses them.
//
// Range.  hi + lo has the exponents of one fp16: beside the largest value of its
// column and chunk (the bound X that the unit comes from) a value is off by up to
// 2^-25 of the unit, 2^-39 X.  R, U and the K^T operand each bring one such rounding
// in, so what a column holds at a token, M, has an error below 2^-20 M (decode's
// bound is of that size) while X < 2^17 M.  M is taken as max |v| over a lane's group
// of tokens, or what the chunk leaves of S0 if that is more.  Where a group is
// smaller - an outlier beside small tokens, a large state that a gate closes - the
// state wave takes the chunk token by token in fp32 (`wide` below): 19 us for 1.4
// (16 columns).  Normal values do not come near that; v of which half is zero does in
// one chunk of 25 (16384 tokens x 32 heads 0.7 -> 1.2 ms).
//
// Work split.  Value columns never interact, so a workgroup owns one
// (request, value head) tile and NCW * 16 * NCS of its columns.  The chain
// from chunk to chunk (S0 -> R -> U -> S) runs in NCW state waves, each
// with 16 * NCS columns, all keys in registers, and no exchange with other
// waves.  What does not depend on the state is made ahead by four helper
// waves, each a chunk further on:
//   0  K: fp16 rows in operand order (K for K S0 and the Gram
//      products, K^T for the state update), norms      chunk c + 3
//   1  Q: the same without K^T; the gates: G and beta  chunk c + 3
//   2  the Gram products: A, P, the factor tables      chunk c + 2
//   3  T: two 16 x 16 triangular inverses, joined      chunk c + 1
// with one barrier per chunk.  The accumulator layout of one product (four
// consecutive rows per lane) is the operand layout of the next once the
// operands' order of k is permuted to match, so the chain never leaves its
// registers.

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "kda.h"
#include "kda_device.h"
#include "kda_internal.h"
#include "kda_tile.h"

namespace kda {
namespace {

constexpr int kHelpers = 4;
constexpr int kRing = 4;          // chunks of q and k held in LDS
constexpr int kRingP = 3;         // of P, made a chunk later
constexpr float kUnitT = 16384.0f;   // T and P are stored times this
constexpr int kWide = 17;         // powers of two between a chunk's bound and its smallest group (`wide`)

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Blocks of 16 tokens in a chunk: 32 tokens, and 16 where fp32 rows of 128 keys
// (hi and lo) would need twice the LDS.
template <int DK, bool F32>
constexpr int kBlocks = F32 && DK == 128 ? 1 : 2;

__device__ __forceinline__ f32x4 mfma(h8 a, h8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ f32x4 mfma(h4 a, h4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x16f16(a, b, c, 0, 0, 0);
}

// x * s as hi + lo in fp16 (s a power of two).  The packed hi is made opaque
// so that lo is taken from it and not from conversions of its own, in one
// mixed-precision FMA each.
__device__ __forceinline__ h2 low_part(float x0, float x1, float s, h2& hi) {
  asm("" : "+v"(hi));
  _Float16 lo = static_cast<_Float16>(__builtin_fmaf(x0, s, -static_cast<float>(hi.x)));
  asm("" : "+v"(lo));   // not a packed conversion of two separate FMAs
  return h2{lo, static_cast<_Float16>(__builtin_fmaf(x1, s, -static_cast<float>(hi.y)))};
}

__device__ __forceinline__ void split2(float x0, float x1, float s, h2& hi, h2& lo) {
  hi = h2{static_cast<_Float16>(x0 * s), static_cast<_Float16>(x1 * s)};
  lo = low_part(x0, x1, s, hi);
}

// The same with s = 1 for two accumulators' rows, as an operand.  `one` is a
// 1.0f that the compiler does not see as such: it would take the FMA apart.
__device__ __forceinline__ void split8(const f32x4& x, const f32x4& y, float one, h8& hi, h8& lo) {
  h2 h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x0 = i < 2 ? x[2 * i] : y[2 * i - 4], x1 = i < 2 ? x[2 * i + 1] : y[2 * i - 3];
    h[i] = h2{static_cast<_Float16>(x0), static_cast<_Float16>(x1)};
    l[i] = low_part(x0, x1, one, h[i]);
  }
  hi = h8{h[0].x, h[0].y, h[1].x, h[1].y, h[2].x, h[2].y, h[3].x, h[3].y};
  lo = h8{l[0].x, l[0].y, l[1].x, l[1].y, l[2].x, l[2].y, l[3].x, l[3].y};
}

// A chunk's rows (NB accumulators) as an operand over its tokens.
__device__ __forceinline__ void split_rows(const f32x4 (&x)[2], float one, h8& hi, h8& lo) {
  split8(x[0], x[1], one, hi, lo);
}

__device__ __forceinline__ void split_rows(const f32x4 (&x)[1], float one, h4& hi, h4& lo) {
  h2 h[2], l[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    h[i] = h2{static_cast<_Float16>(x[0][2 * i]), static_cast<_Float16>(x[0][2 * i + 1])};
    l[i] = low_part(x[0][2 * i], x[0][2 * i + 1], one, h[i]);
  }
  hi = h4{h[0].x, h[0].y, h[1].x, h[1].y};
  lo = h4{l[0].x, l[0].y, l[1].x, l[1].y};
}

// The unit of a state column is 2^sig: the least one in which a bound on the
// column, 2^e <= bound < 2^(e + 1), is below 2^15, but not below 2^kSigMin nor
// 2^100 times smaller than the old one (the factors between them stay finite).
// Bounds are handled by their exponents: a bound on v in the unit of a state
// that is zero or tiny does not fit fp32.
constexpr int kSigMin = -100;

// floor(log2(x)) + 127 of a normal x > 0; 0 for zero and below the normal range.
constexpr int kBias = 127;
__device__ __forceinline__ int exponent(float x) { return static_cast<int>(__float_as_uint(x) >> 23); }

__device__ __forceinline__ int unit_for(int e, int min) {   // e biased
  const int to = e - kBias - 14;
  min = min < kSigMin ? kSigMin : min;
  return to < min ? min : to;
}

__device__ __forceinline__ int max16_32(int x) {   // over lanes that share lane % 16
  const auto p = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  x = max(static_cast<int>(p[0]), static_cast<int>(p[1]));
  const auto q = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  return max(static_cast<int>(q[0]), static_cast<int>(q[1]));
}

// A double moved within its row of 16 lanes (0 where none comes in), and
// lane 15's.
template <int CTRL>
__device__ __forceinline__ double dpp_f64(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(u), CTRL, 0xf, 0xf, true);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(u >> 32), CTRL, 0xf, 0xf, true);
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

__device__ __forceinline__ double lane15_f64(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(u), 15);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(u >> 32), 15);
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

// ---------------------------------------------------------------------------
// LDS
// ---------------------------------------------------------------------------

// Operand order.  A 16-row operand of one matrix instruction is 64 slots of
// 8 halves; lane l = 16 g + row holds k positions 8 g + 0..7, which stand for
// k = 4 g + 0..3 and 16 + 4 g + 0..3 of the 32 (the rows that lane group g
// holds of two stacked accumulators).  Slots are permuted within their row
// of 16 so that the writes of one token spread over the banks.
__device__ __forceinline__ int row_slot(int s, int g, int row) {
  return g * 16 + (row ^ (((g >> 1) + 2 * s) & 7));
}

// The same for key block j of K^T, whose writers hold one channel of every
// other block at a time.
__device__ __forceinline__ int kt_slot(int j, int g, int channel) { return g * 16 + (channel ^ (j & 7)); }

template <int DK, bool F32>
struct Shared {
  static constexpr int KS = DK / 32;       // 32-key steps
  static constexpr int TERMS = F32 ? 2 : 1;
  static constexpr int NB = kBlocks<DK, F32>;
  static constexpr int C = 16 * NB;
  static constexpr int TK = 4 * NB;        // a lane's positions of an operand over tokens
  _Float16 k[kRing][TERMS][NB][KS][64][8];         // K rows: [token block][key step]
  _Float16 q[kRing][TERMS][NB][KS][64][8];
  _Float16 kt[kRing][TERMS][DK / 16][64][TK];      // K^T: [key block], k = token
  _Float16 p[kRingP][2][NB][64][TK];               // P hi, lo: [token block]
  _Float16 t[2][2][NB][64][TK];                    // T hi, lo, beta included
  float a[2][2 * NB - 1][16][16];                  // A: blocks 00, 11, 10; row-major
  float join[NB][16][16];                          // diagonal blocks of (I + A)^-1, row-major
  float norm_k[kRing][C], norm_q[kRing][C];        // kh = norm_k * stored row
  float g_hi[2][C], g_lo[2][C], beta[2][C];
  float tab[kRing][4][C];                          // 2^14 beta; e^G norm_k; scale e^G norm_q; norm_k e^(last - G)
  float last[kRing];                               // e^(G_last)
};

// ---------------------------------------------------------------------------
// the rows of k or q
// ---------------------------------------------------------------------------

// A window of rows of a packed tensor: rows of `row` bytes every `stride`
// bytes, `n` of them (n >= 1).  Loads past the last row give zero and stores
// are dropped by the hardware's range check, so a chunk's tail needs no masks;
// all offsets are in the vector offset, which the check covers.
template <int C>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_resource(const void* base, int64_t offset, int n, int stride,
                                                                int row) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(static_cast<const char*>(base)) + offset,
                                           static_cast<short>(0), ((n < C ? n : C) - 1) * stride + row,
                                           kRawBufferWord3);
}

// A lane holds 8 channels of TL tokens: dk / 8 lanes cover a token, and lane
// group q of them has operand positions P = q TL .. q TL + TL - 1, where
// position P = TK g + p is token 4 g + p % 4 + 16 (p / 4) (TK = 8, or 4 with
// one block of tokens).
template <int DK, bool F32>
struct RowLoader {
  static constexpr int LANES = DK / 8;
  static constexpr int TK = 4 * kBlocks<DK, F32>;
  static constexpr int TL = TK * LANES / 16;
  static constexpr int WORDS = F32 ? 2 : 1;
  u32x4 w[TL][WORDS];

  static __device__ __forceinline__ int position(int lane) { return (lane / LANES) * TL; }
  static __device__ __forceinline__ int token(int lane) {   // of the lane's first position
    const int P = position(lane);
    return 4 * (P / TK) + P % 4 + 16 * (P % TK / 4);
  }
  static constexpr __device__ int step(int i) { return i % 4 + 16 * (i / 4); }   // token i's distance from it

  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, int voff, int stride) {
#pragma unroll
    for (int i = 0; i < TL; ++i)
#pragma unroll
      for (int x = 0; x < WORDS; ++x)
        w[i][x] = __builtin_amdgcn_raw_buffer_load_b128(r, voff + step(i) * stride + 16 * x, 0, 0);
  }

  __device__ __forceinline__ void unpack(int i, float (&x)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (F32) x[e] = __uint_as_float(w[i][e / 4][e % 4]);
      else x[e] = e % 2 ? __uint_as_float(w[i][0][e / 2] & 0xffff0000u) : __uint_as_float(w[i][0][e / 2] << 16);
    }
  }
};

// Sums over the LANES lanes of a group, to all of them; level by level, so
// that the moves of one sum hide the latency of another's.
template <int LANES, int N>
__device__ __forceinline__ void group_sums(float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] += dpp<kDppXor1>(x[i]);
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] += dpp<kDppXor2>(x[i]);
  if constexpr (LANES == 8) {   // quads are uniform by now
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] += dpp<kDppHalfMirror>(x[i]);
  }
  if constexpr (LANES == 16) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] += dpp<kDppRowRor4>(x[i]);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] += dpp<kDppRowRor8>(x[i]);
  }
}

// A row's power of two 2^-e, with 2^e <= norm < 2^(e + 1), from the exponent of
// its square; and the factor that makes the row times 2^-e a unit row.  A row
// whose square is not finite is multiplied by 0, as by 1 / sqrt(inf): finite
// values give kh = 0, infinities and NaN give NaN.
__device__ __forceinline__ float row_down(float square) {
  const uint32_t ex = __float_as_uint(square) >> 23;
  return ex < 255u ? __uint_as_float((191u - ((ex + 1u) >> 1)) << 23) : 0.0f;   // e = (ex + 1) / 2 - 64
}

__device__ __forceinline__ float row_factor(float square, float l2_eps) {
  const uint32_t ex = __float_as_uint(square) >> 23;
  return ex < 255u ? __uint_as_float((63u + ((ex + 1u) >> 1)) << 23) * rsqrt_f(square + l2_eps) : 0.0f;
}

// Converts a chunk's rows: fp16 rows in operand order, their factors
// (norm[token] * stored row = unit row), and for k the transposed operand.
template <int DK, bool F32, bool KT>
__device__ __forceinline__ void convert_rows(const RowLoader<DK, F32>& in, float l2_eps, int lane,
                                             _Float16 (*rows)[kBlocks<DK, F32>][DK / 32][64][8],
                                             _Float16 (*kt)[DK / 16][64][4 * kBlocks<DK, F32>],
                                             float* norm) {
  using L = RowLoader<DK, F32>;
  constexpr int TL = L::TL;
  const int c = 8 * (lane % L::LANES);
  const int s = c / 32, half = (c % 32) / 16, g = (c % 16) / 4;   // the lane's channels: operand groups g, g + 1
  const int first = L::token(lane);
  float sums[TL];
#pragma unroll
  for (int i = 0; i < TL; ++i) {
    float x[8];
    in.unpack(i, x);
    sums[i] = x[0] * x[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) sums[i] = fmaf(x[e], x[e], sums[i]);
  }
  group_sums<L::LANES>(sums);
  // lane i of a group writes the factor of the group's token i
  const int mine = lane % L::LANES;
  float own = sums[0];
#pragma unroll
  for (int i = 1; i < TL; ++i) own = mine == i ? sums[i] : own;
  if (mine < TL) norm[first + L::step(mine)] = row_factor(own, l2_eps);
  h2 hi[TL][4], lo[TL][4];
#pragma unroll
  for (int i = 0; i < TL; ++i) {
    float x[8];
    in.unpack(i, x);
    const float down = row_down(sums[i]);
    const int t = first + L::step(i);
#pragma unroll
    for (int e2 = 0; e2 < 4; ++e2) {
      if constexpr (F32) {
        split2(x[2 * e2], x[2 * e2 + 1], down, hi[i][e2], lo[i][e2]);
      } else {
        hi[i][e2] = h2{static_cast<_Float16>(x[2 * e2] * down), static_cast<_Float16>(x[2 * e2 + 1] * down)};
      }
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int at = row_slot(s, g + q, t % 16);
      *reinterpret_cast<h4*>(&rows[0][t / 16][s][at][half * 4]) =
          h4{hi[i][2 * q].x, hi[i][2 * q].y, hi[i][2 * q + 1].x, hi[i][2 * q + 1].y};
      if constexpr (F32)
        *reinterpret_cast<h4*>(&rows[1][t / 16][s][at][half * 4]) =
            h4{lo[i][2 * q].x, lo[i][2 * q].y, lo[i][2 * q + 1].x, lo[i][2 * q + 1].y};
    }
  }
  if constexpr (KT) {
    typedef _Float16 run __attribute__((ext_vector_type(TL)));
    const int P = L::position(lane);
    constexpr int TK = L::TK;
#pragma unroll
    for (int ch = 0; ch < 8; ++ch) {
      const int cc = c + ch;
      run v;
#pragma unroll
      for (int i = 0; i < TL; ++i) v[i] = hi[i][ch / 2][ch % 2];
      *reinterpret_cast<run*>(&kt[0][cc / 16][kt_slot(cc / 16, P / TK, cc % 16)][P % TK]) = v;
      if constexpr (F32) {
#pragma unroll
        for (int i = 0; i < TL; ++i) v[i] = lo[i][ch / 2][ch % 2];
        *reinterpret_cast<run*>(&kt[1][cc / 16][kt_slot(cc / 16, P / TK, cc % 16)][P % TK]) = v;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------

// State columns of a lane.  With two column sets a lane's columns are
// neighbours (2 n, 2 n + 1), so v, o and key-first rows move in pairs.
template <int NCS>
__device__ __forceinline__ int column(int lane, int cs) {
  return NCS == 2 ? 2 * (lane % 16) + cs : lane % 16;
}

// NCS neighbouring values of a row of v or out.
template <bool F32, int NCS>
struct Columns {
  static constexpr int W = F32 ? NCS : 1;
  uint32_t w[W];
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, int voff) {
    if constexpr (F32 && NCS == 2) {
      const u32x2 x = __builtin_amdgcn_raw_buffer_load_b64(r, voff, 0, 0);
      w[0] = x.x;
      w[1] = x.y;
    } else if constexpr (F32 || NCS == 2) {
      w[0] = __builtin_amdgcn_raw_buffer_load_b32(r, voff, 0, 0);
    } else {
      w[0] = __builtin_amdgcn_raw_buffer_load_b16(r, voff, 0, 0);
    }
  }
  __device__ __forceinline__ void unpack(float (&x)[NCS]) const {
    if constexpr (F32) {
#pragma unroll
      for (int c = 0; c < NCS; ++c) x[c] = __uint_as_float(w[c]);
    } else {
      x[0] = bf16_to_f32(w[0]);
      if constexpr (NCS == 2) x[1] = __uint_as_float(w[0] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, int voff, const float (&x)[NCS]) {
    if constexpr (F32 && NCS == 2) {
      __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(x[0]), __float_as_uint(x[1])}, r, voff, 0, 0);
    } else if constexpr (F32) {
      __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x[0]), r, voff, 0, 0);
    } else if constexpr (NCS == 2) {
      __builtin_amdgcn_raw_buffer_store_b32(f32x2_to_bf16x2_rne(x[0], x[1]), r, voff, 0, 0);
    } else {
      __builtin_amdgcn_raw_buffer_store_b16(static_cast<uint16_t>(f32_to_bf16_rne(x[0])), r, voff, 0, 0);
    }
  }
};

// The wave's columns of the state tile, from or to memory: a lane's keys
// 16 j + 4 g + 0..3 are one access of a value-first tile, its NCS columns one
// of a key-first tile.
template <bool STORE, int KB, int NCS, bool V_FIRST, bool BF16>
__device__ __forceinline__ void slab_form(__amdgpu_buffer_rsrc_t res, int dv, int col, int lane, f32x4 (&S)[KB][NCS]) {
  constexpr int E = BF16 ? 2 : 4;
  const int key0 = 4 * (lane / 16);
#pragma unroll
  for (int j = 0; j < KB; ++j) {
    if constexpr (V_FIRST) {
      using IO = StateIO<BF16, 4, 0>;
#pragma unroll
      for (int cs = 0; cs < NCS; ++cs) {
        const int voff = ((col + column<NCS>(lane, cs)) * (KB * 16) + key0) * E;
        float x[4] = {S[j][cs][0], S[j][cs][1], S[j][cs][2], S[j][cs][3]};
        if constexpr (STORE) IO::store(res, voff, 16 * j * E, x);
        else IO::load(res, voff, 16 * j * E, x);
        S[j][cs] = f32x4{x[0], x[1], x[2], x[3]};
      }
    } else {
      const int voff = (key0 * dv + col + column<NCS>(lane, 0)) * E;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int at = voff + (16 * j + r) * dv * E;
        float x[NCS];
        if constexpr (STORE) {
#pragma unroll
          for (int cs = 0; cs < NCS; ++cs) x[cs] = S[j][cs][r];
          Columns<!BF16, NCS>::store(res, at, x);
        } else {
          Columns<!BF16, NCS> c;
          c.load(res, at);
          c.unpack(x);
#pragma unroll
          for (int cs = 0; cs < NCS; ++cs) S[j][cs][r] = x[cs];
        }
      }
    }
  }
}

template <bool STORE, int KB, int NCS>
__device__ __forceinline__ void slab_io(__amdgpu_buffer_rsrc_t res, int layout, int bf16, int dv, int col, int lane,
                                        f32x4 (&S)[KB][NCS]) {
  asm("" : "+v"(lane));   // addresses are made here, not kept through the chunks
  if (layout == KDA_STATE_V_FIRST) {
    if (bf16) slab_form<STORE, KB, NCS, true, true>(res, dv, col, lane, S);
    else slab_form<STORE, KB, NCS, true, false>(res, dv, col, lane, S);
  } else {
    if (bf16) slab_form<STORE, KB, NCS, false, true>(res, dv, col, lane, S);
    else slab_form<STORE, KB, NCS, false, false>(res, dv, col, lane, S);
  }
}

// max |S| of the lane's share of a column.
template <int KB, int NCS>
__device__ __forceinline__ float largest(const f32x4 (&S)[KB][NCS], int cs) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < KB; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r) m = fmaxf(m, fabsf(S[j][cs][r]));
  return m;
}

struct Tile {
  int b, hv, h, slot, col0;   // col0: first column of the workgroup
  int t0, n;                  // first row and tokens
};

// Log decay of a token: raw gate plus bias -> g, at least -200 (exp(-200) is 0 in
// fp32, and sums stay finite).
__device__ __forceinline__ float log_decay(const DecodeArgs& a, float x, float amp) {
  const float g = a.gate_mode == KDA_GATE_SOFTPLUS ? -amp * softplus_f(x) : a.lower_bound * sigmoid_f(amp * x);
  return g < -200.0f ? -200.0f : g;
}

// One chunk token by token, in fp32 and without a unit: with the decay applied
// first, u = v - kh^T S, S += beta kh u^T, o = qh^T S = qh^T S_old + (qh.kh) beta u.
// q and k come as the helpers left them in LDS.  A lane's keys are 16 j + 4 g + r.
template <int KB, int NCS, int DK, bool F32>
__device__ __forceinline__ void walk_chunk(const DecodeArgs& a, const Shared<DK, F32>& sh, const Tile& w, int ring,
                                           int first, int n, __amdgpu_buffer_rsrc_t rv, __amdgpu_buffer_rsrc_t ro,
                                           int voff, int stride, int lane, int (&sig)[NCS], f32x4 (&S)[KB][NCS]) {
  const int g = lane / 16;
  // the decay of token lane % C (row `first` of the request and on)
  const int64_t row = static_cast<int64_t>(w.t0) + first + (lane % Shared<DK, F32>::C < n ? lane % Shared<DK, F32>::C : 0);
  const float decays = exp_f(log_decay(a, a.raw_gate[row * a.HV + w.hv] + a.dt_bias[w.hv], exp_f(a.a_log[w.hv])));
#pragma unroll
  for (int cs = 0; cs < NCS; ++cs) {
    const float f = __builtin_ldexpf(1.0f, sig[cs]);
#pragma unroll
    for (int j = 0; j < KB; ++j) S[j][cs] *= f;
  }
  Columns<F32, NCS> next;
  next.load(rv, voff);
#pragma unroll 1
  for (int t = 0; t < n; ++t) {
    float v[NCS];
    next.unpack(v);
    if (t + 1 < n) next.load(rv, voff + (t + 1) * stride);
    const float alpha = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(decays), t));
    const float nk = sh.norm_k[ring][t], nq = a.scale * sh.norm_q[ring][t];
    const float beta = sh.tab[ring][0][t] * (1.0f / kUnitT);
    float qk = 0.0f, ks[NCS], qs[NCS];
#pragma unroll
    for (int cs = 0; cs < NCS; ++cs) ks[cs] = qs[cs] = 0.0f;
    h8 kr[F32 ? 2 : 1][DK / 32], qr[F32 ? 2 : 1][DK / 32];
#pragma unroll
    for (int term = 0; term < (F32 ? 2 : 1); ++term)
#pragma unroll
      for (int s = 0; s < DK / 32; ++s) {
        kr[term][s] = *reinterpret_cast<const h8*>(&sh.k[ring][term][t / 16][s][row_slot(s, g, t % 16)][0]);
        qr[term][s] = *reinterpret_cast<const h8*>(&sh.q[ring][term][t / 16][s][row_slot(s, g, t % 16)][0]);
      }
    const auto value = [](const auto& rows, int s, int e) {
      if constexpr (F32) return static_cast<float>(rows[0][s][e]) + static_cast<float>(rows[1][s][e]);
      else return static_cast<float>(rows[0][s][e]);
    };
#pragma unroll
    for (int s = 0; s < DK / 32; ++s)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float k = value(kr, s, e), q = value(qr, s, e);
        qk = fmaf(q, k, qk);
#pragma unroll
        for (int cs = 0; cs < NCS; ++cs) {
          const float x = S[2 * s + e / 4][cs][e % 4] * alpha;
          S[2 * s + e / 4][cs][e % 4] = x;
          ks[cs] = fmaf(k, x, ks[cs]);
          qs[cs] = fmaf(q, x, qs[cs]);
        }
      }
    qk = swap16_add(qk, qk);
    qk = swap32_add(qk, qk);
    float write[NCS], o[NCS];
#pragma unroll
    for (int cs = 0; cs < NCS; ++cs) {
      ks[cs] = swap16_add(ks[cs], ks[cs]);
      ks[cs] = swap32_add(ks[cs], ks[cs]);
      qs[cs] = swap16_add(qs[cs], qs[cs]);
      qs[cs] = swap32_add(qs[cs], qs[cs]);
      write[cs] = beta * nk * fmaf(-nk, ks[cs], v[cs]);
      o[cs] = nq * fmaf(qk, write[cs], qs[cs]);
    }
#pragma unroll
    for (int s = 0; s < DK / 32; ++s)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float k = value(kr, s, e);
#pragma unroll
        for (int cs = 0; cs < NCS; ++cs) S[2 * s + e / 4][cs][e % 4] = fmaf(k, write[cs], S[2 * s + e / 4][cs][e % 4]);
      }
    if (g == 0) Columns<F32, NCS>::store(ro, voff + t * stride, o);
  }
#pragma unroll
  for (int cs = 0; cs < NCS; ++cs) {
    sig[cs] = unit_for(max16_32(exponent(largest(S, cs))), kSigMin);
    const float f = __builtin_ldexpf(1.0f, -sig[cs]);
#pragma unroll
    for (int j = 0; j < KB; ++j) S[j][cs] *= f;
  }
}

// At dk = 32 two workgroups fit a CU where they hold up to 128 registers (128
// columns, 8 prompts x 1024 tokens x 96 heads: 159 us with 126 and 188 with 131).
template <int NCW, int NCS, int DK, bool F32>
__global__ void __launch_bounds__((NCW + kHelpers) * kWave, DK == 32 ? 4 : 1)
gdr_prefill(const DecodeArgs a, const int dv, const int layout, const int state_bf16) {
  constexpr int KS = DK / 32;          // key steps of 32
  constexpr int KB = DK / 16;          // key blocks of 16
  constexpr int NC = NCW * 16 * NCS;   // columns of the workgroup
  constexpr int TERMS = F32 ? 2 : 1;
  using Sh = Shared<DK, F32>;
  constexpr int NB = Sh::NB;           // blocks of 16 tokens
  constexpr int C = Sh::C;             // tokens per chunk
  constexpr int M = 2 * NB - 1;        // blocks of the lower triangle
  using ht = std::conditional_t<NB == 2, h8, h4>;   // an operand over tokens
  extern __shared__ __attribute__((aligned(16))) char lds[];
  Sh& sh = *reinterpret_cast<Sh*>(lds);

  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int g = lane / 16;

  // XCD-aware id -> (tile, slab): the slabs of a tile read the same q and k
  const int slabs = dv / NC;
  const uint32_t wg = blockIdx.x, nwg = gridDim.x;
  const uint32_t xcd = wg % kXcds, per = nwg / kXcds, extra = nwg % kXcds;
  const uint32_t logical = xcd * per + (xcd < extra ? xcd : extra) + wg / kXcds;
  Tile w;
  w.col0 = static_cast<int>(logical % slabs) * NC;
  const int tile = static_cast<int>(logical / slabs);
  w.b = tile / a.HV;
  w.hv = tile - w.b * a.HV;
  w.h = w.hv / a.G;
  int t0 = a.cu_seqlens[w.b], t1 = a.cu_seqlens[w.b + 1];
  t0 = t0 < 0 ? 0 : (t0 > a.T ? a.T : t0);
  t1 = t1 < t0 ? t0 : (t1 > a.T ? a.T : t1);
  w.t0 = t0;
  w.n = t1 - t0;
  w.slot = a.state_indices[w.b];

  if (w.slot < 0 || w.slot >= a.N) {   // skipped: zero rows, no state
    for (int64_t i = threadIdx.x; i < static_cast<int64_t>(w.n) * NC; i += blockDim.x) {
      const int64_t off = ((t0 + i / NC) * a.HV + w.hv) * dv + w.col0 + i % NC;
      store_scalar<!F32>(a.out, off, 0.0f);
    }
    return;
  }
  if (w.n == 0) return;
  const int chunks = (w.n + C - 1) / C;
  constexpr int E = F32 ? 4 : 2;
  // Waves i and i + 4 share a SIMD.  With fewer than four state waves they get
  // SIMDs of their own and the helpers share the others.
  constexpr uint32_t kRoles = NCW == 1 ? 0x3f102u : NCW == 2 ? 0x13ff02u : NCW == 4 ? 0x3210ffffu : 0u;
  const int role = static_cast<int>(kRoles >> (4 * wave) & 15u);   // 15: state wave
  const int cw = NCW == 1 ? 0 : NCW == 2 ? wave - 2 : wave;

  // the upper blocks of P and T stay zero
  if constexpr (NB == 2) {
    for (int i = threadIdx.x; i < kRingP * 2 * 64; i += blockDim.x)
      *reinterpret_cast<h4*>(&sh.p[i / 128][(i / 64) % 2][0][i % 64][4]) = h4{0, 0, 0, 0};
    for (int i = threadIdx.x; i < 2 * 2 * 64; i += blockDim.x)
      *reinterpret_cast<h4*>(&sh.t[i / 128][(i / 64) % 2][0][i % 64][4]) = h4{0, 0, 0, 0};
  }

  if (role == 0 || role == 1) {
    // ---- helpers 0 and 1: k / q rows of chunk it + 3, and with q the gates ----
    using L = RowLoader<DK, F32>;
    const void* const src = role == 0 ? a.k : a.q;
    const int stride = a.H * DK * E;
    const int voff = L::token(lane) * stride + 8 * (lane % L::LANES) * E;
    auto chunk_rows = [&](int c) {
      return rows_resource<C>(src, ((static_cast<int64_t>(t0) + c * C) * a.H + w.h) * (DK * E), w.n - c * C, stride,
                           DK * E);
    };
    L raw;
    raw.load(chunk_rows(0), voff, stride);
    const float amp = exp_f(a.a_log[w.hv]);
    const float bias = a.dt_bias[w.hv];
    const int tl = lane % C;
    auto gate_at = [&](int c) {   // raw gate and beta logit of the lane's token
      const int t = c * C + tl;
      const int64_t off = (static_cast<int64_t>(t0) + (t < w.n ? t : 0)) * a.HV + w.hv;
      return make_float2(a.raw_gate[off], a.beta_logits[off]);
    };
    float2 gate = make_float2(0.0f, 0.0f);
    if (role == 1) gate = gate_at(0);
    lds_barrier();
    for (int it = -3; it < chunks; ++it) {
      const int c = it + 3;
      if (c < chunks) {
        const L cur = raw;
        const float2 gb = gate;
        if (c + 1 < chunks) {
          raw.load(chunk_rows(c + 1), voff, stride);
          if (role == 1) gate = gate_at(c + 1);
        }
        const int ring = c % kRing, two = c % 2;
        if (role == 0) {
          convert_rows<DK, F32, true>(cur, a.l2_eps, lane, sh.k[ring], sh.kt[ring], sh.norm_k[ring]);
        } else {
          convert_rows<DK, F32, false>(cur, a.l2_eps, lane, sh.q[ring], nullptr, sh.norm_q[ring]);
          const bool live = c * C + tl < w.n;
          double sum = live ? static_cast<double>(log_decay(a, gb.x + bias, amp)) : 0.0;
          sum += dpp_f64<0x111>(sum);   // row_shr 1, 2, 4, 8: zero comes in
          sum += dpp_f64<0x112>(sum);
          sum += dpp_f64<0x114>(sum);
          sum += dpp_f64<0x118>(sum);
          if constexpr (NB == 2) {
            const double row0 = lane15_f64(sum);
            if (tl >= 16) sum += row0;
          }
          if (lane < C) {
            const float hi = static_cast<float>(sum);
            sh.g_hi[two][tl] = hi;
            sh.g_lo[two][tl] = static_cast<float>(sum - static_cast<double>(hi));
            sh.beta[two][tl] = live ? sigmoid_f(gb.y) : 0.0f;
          }
        }
      }
      lds_barrier();
    }
  } else if (role == 2) {
    // ---- helper 2: Gram products of chunk it + 2 ----
    lds_barrier();
    int third = 0;   // c % kRingP
    for (int it = -3; it < chunks; ++it) {
      const int c = it + 2;
      if (c >= 0 && c < chunks) {
        const int ring = c % kRing, two = c % 2;
        f32x4 ka[M], pa[M];   // blocks 00, 11, 10
#pragma unroll
        for (int m = 0; m < M; ++m) ka[m] = pa[m] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const int at = row_slot(s, g, lane % 16);
          h8 kk[TERMS][NB], qq[TERMS][NB];
#pragma unroll
          for (int term = 0; term < TERMS; ++term)
#pragma unroll
            for (int rb = 0; rb < NB; ++rb) {
              kk[term][rb] = *reinterpret_cast<const h8*>(&sh.k[ring][term][rb][s][at][0]);
              qq[term][rb] = *reinterpret_cast<const h8*>(&sh.q[ring][term][rb][s][at][0]);
            }
#pragma unroll
          for (int m = 0; m < M; ++m) {
            const int i = m > 0, j = m == 1;   // row block i, column block j
            // transposed: a lane holds row lane % 16 of block i, columns 4 g + 0..3 of block j
            ka[m] = mfma(kk[0][j], kk[0][i], ka[m]);
            pa[m] = mfma(kk[0][j], qq[0][i], pa[m]);
            if constexpr (F32) {
              ka[m] = mfma(kk[0][j], kk[1][i], ka[m]);
              ka[m] = mfma(kk[1][j], kk[0][i], ka[m]);
              pa[m] = mfma(kk[0][j], qq[1][i], pa[m]);
              pa[m] = mfma(kk[1][j], qq[0][i], pa[m]);
            }
          }
        }
        const float g_last = sh.g_hi[two][C - 1], g_last_lo = sh.g_lo[two][C - 1];
#pragma unroll
        for (int m = 0; m < M; ++m) {
          const int i = m > 0, j = m == 1;
          const int row = 16 * i + lane % 16, col = 16 * j + 4 * g;
          const float gh = sh.g_hi[two][row], gl = sh.g_lo[two][row];
          const float nq = kUnitT * sh.norm_q[ring][row], nk = sh.norm_k[ring][row] * sh.beta[two][row];
          const f32x4 ch = *reinterpret_cast<const f32x4*>(&sh.g_hi[two][col]);
          const f32x4 cl = *reinterpret_cast<const f32x4*>(&sh.g_lo[two][col]);
          const f32x4 ck = *reinterpret_cast<const f32x4*>(&sh.norm_k[ring][col]);
          f32x4 y;
          float x[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            // e^(G_row - G_col) norm_col; above the diagonal the exponent may
            // be positive, and is not used
            const float d = exp_f((gh - ch[r]) + (gl - cl[r])) * ck[r];
            y[r] = col + r < row ? ka[m][r] * nk * d : 0.0f;
            x[r] = col + r <= row ? pa[m][r] * nq * d : 0.0f;
          }
          *reinterpret_cast<f32x4*>(&sh.a[two][m][lane % 16][4 * g]) = y;
          {
            h2 hi0, lo0, hi1, lo1;
            split2(x[0], x[1], 1.0f, hi0, lo0);
            split2(x[2], x[3], 1.0f, hi1, lo1);
            *reinterpret_cast<h4*>(&sh.p[third][0][i][lane][4 * j]) = h4{hi0.x, hi0.y, hi1.x, hi1.y};
            *reinterpret_cast<h4*>(&sh.p[third][1][i][lane][4 * j]) = h4{lo0.x, lo0.y, lo1.x, lo1.y};
          }
        }
        if (lane < C) {
          const float gh = sh.g_hi[two][lane], gl = sh.g_lo[two][lane];
          const float nk = sh.norm_k[ring][lane];
          const float eg = exp_f(gh + gl);
          sh.tab[ring][0][lane] = kUnitT * sh.beta[two][lane];
          sh.tab[ring][1][lane] = eg * nk;
          sh.tab[ring][2][lane] = a.scale * eg * sh.norm_q[ring][lane];
          sh.tab[ring][3][lane] = nk * exp_f((g_last - gh) + (g_last_lo - gl));
          if (lane == C - 1) sh.last[ring] = eg;
        }
        third = third == kRingP - 1 ? 0 : third + 1;
      }
      lds_barrier();
    }
  } else if (role == 3) {
    // ---- helper 3: T of chunk it + 1 ----
    lds_barrier();
    for (int it = -3; it < chunks; ++it) {
      const int c = it + 1;
      if (c >= 0 && c < chunks) {
        const int two = c % 2;
        // lane: row `row` of diagonal block `blk` (lanes 32.. repeat), x (I + A)
        // = e_row, from the last column back: with x_k known, row k of A is
        // taken off all columns before it
        const int blk = (lane / 16) % NB, row = lane % 16;
        float x[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = row == j ? 1.0f : 0.0f;
#pragma unroll
        for (int k = 15; k > 0; --k) {
#pragma unroll
          for (int j4 = 0; j4 < (k + 3) / 4; ++j4) {
            const f32x4 ar = *reinterpret_cast<const f32x4*>(&sh.a[two][blk][k][4 * j4]);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (4 * j4 + j < k) x[4 * j4 + j] = fmaf(-x[k], ar[j], x[4 * j4 + j]);
          }
        }
        if (lane < C) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const f32x4 xj = {x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]};
            *reinterpret_cast<f32x4*>(&sh.join[blk][row][4 * j]) = xj;
            const f32x4 xb = xj * *reinterpret_cast<const f32x4*>(&sh.tab[c % kRing][0][16 * blk + 4 * j]);
            h2 hi0, lo0, hi1, lo1;
            split2(xb[0], xb[1], 1.0f, hi0, lo0);
            split2(xb[2], xb[3], 1.0f, hi1, lo1);
            *reinterpret_cast<h4*>(&sh.t[two][0][blk][16 * j + row][4 * blk]) = h4{hi0.x, hi0.y, hi1.x, hi1.y};
            *reinterpret_cast<h4*>(&sh.t[two][1][blk][16 * j + row][4 * blk]) = h4{lo0.x, lo0.y, lo1.x, lo1.y};
          }
        }
        if constexpr (NB == 2) {
          __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront", "local");
          // T10^T = -T00^T (A10^T T11^T) on the fp32 matrix instruction
          f32x4 z = {0, 0, 0, 0}, y = {0, 0, 0, 0};
          const f32x4 bt = *reinterpret_cast<const f32x4*>(&sh.join[1][lane % 16][4 * g]);      // T11[lane % 16][4g + r]
#pragma unroll
          for (int r = 0; r < 4; ++r) z = __builtin_amdgcn_mfma_f32_16x16x4f32(sh.a[two][2][4 * g + r][lane % 16], bt[r], z, 0, 0, 0);
#pragma unroll
          for (int r = 0; r < 4; ++r) y = __builtin_amdgcn_mfma_f32_16x16x4f32(sh.join[0][4 * g + r][lane % 16], z[r], y, 0, 0, 0);
          // y: column (row of T10) lane % 16, rows (columns of T10) 4 g + 0..3
          y *= -*reinterpret_cast<const f32x4*>(&sh.tab[c % kRing][0][4 * g]);
          h2 hi0, lo0, hi1, lo1;
          split2(y[0], y[1], 1.0f, hi0, lo0);
          split2(y[2], y[3], 1.0f, hi1, lo1);
          *reinterpret_cast<h4*>(&sh.t[two][0][1][lane][0]) = h4{hi0.x, hi0.y, hi1.x, hi1.y};
          *reinterpret_cast<h4*>(&sh.t[two][1][1][lane][0]) = h4{lo0.x, lo0.y, lo1.x, lo1.y};
        }
      }
      lds_barrier();
    }
  } else {
    // ---- state waves ----
    const int colw = w.col0 + cw * 16 * NCS;
    const int elem = state_bf16 ? 2 : 4;
    char* const tile_base = static_cast<char*>(a.state_pool) +
                            (static_cast<int64_t>(w.slot) * a.HV + w.hv) * (static_cast<int64_t>(DK) * dv * elem);
    const __amdgpu_buffer_rsrc_t res = tile_resource(tile_base, DK * dv * elem);
    f32x4 S[KB][NCS];
    slab_io<false, KB, NCS>(res, layout, state_bf16, dv, colw, lane, S);

    // v and out of a chunk: the lane's rows 16 rb + 4 g + r, NCS columns
    const int stride = a.HV * dv * E;
    int voff[NB][4];
#pragma unroll
    for (int rb = 0; rb < NB; ++rb)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        voff[rb][r] = (16 * rb + 4 * g + r) * stride + (colw + column<NCS>(lane, 0)) * E;
    auto chunk_rows = [&](const void* base, int c) {
      return rows_resource<C>(base, ((static_cast<int64_t>(t0) + c * C) * a.HV + w.hv) * (dv * E), w.n - c * C, stride,
                              dv * E);
    };
    Columns<F32, NCS> v[NB][4];
    // a last chunk's groups of less than four tokens go with the one before, if there
    // is one: an exponent that is not the smallest.  In the second 16 of 32 tokens they
    // belong to a group of four in the first 16, so only groups without a token do.
    const int fewest = C * (chunks - 1) % 32 ? 1 : 4;
    const int past = g > 0 && 4 * g + fewest > w.n - (chunks - 1) * C ? 512 : 0;
    auto load_v = [&](int c) {
      const __amdgpu_buffer_rsrc_t r0 = chunk_rows(a.v, c);
#pragma unroll
      for (int rb = 0; rb < NB; ++rb)
#pragma unroll
        for (int r = 0; r < 4; ++r) v[rb][r].load(r0, voff[rb][r]);
    };
    load_v(0);
    // S of column cs is held divided by 2^sig[cs], below 2^15 in size
    int sig[NCS];
    float one = 1.0f;
    asm("" : "+s"(one));
    int third = 0;   // it % kRingP
#pragma unroll
    for (int cs = 0; cs < NCS; ++cs) {
      sig[cs] = unit_for(max16_32(exponent(largest(S, cs))), kSigMin);
      const float f = __builtin_ldexpf(1.0f, -sig[cs]);
#pragma unroll
      for (int j = 0; j < KB; ++j) S[j][cs] *= f;
    }
    lds_barrier();
    for (int it = -3; it < chunks; ++it) {
      if (it >= 0) {
        const int ring = it % kRing;
        // K S and Q S, the state as hi + lo
        f32x4 ks[NB][NCS], qs[NB][NCS];
#pragma unroll
        for (int rb = 0; rb < NB; ++rb)
#pragma unroll
          for (int cs = 0; cs < NCS; ++cs) ks[rb][cs] = qs[rb][cs] = f32x4{0, 0, 0, 0};
        if constexpr (NCS == 1) {
          // Operands are read and S is split a step ahead of the products, and products
          // into one accumulator stand apart (one prompt of 16384 tokens x 32 heads 737 ->
          // 671 us; with two column sets, as below, the products stand apart by themselves
          // and this costs 1%).
          h8 kr[2][TERMS][NB], qr[2][TERMS][NB], hi[2][NCS], lo[2][NCS];
          const auto stage = [&](int s) {
            const int at = row_slot(s, g, lane % 16);
#pragma unroll
            for (int term = 0; term < TERMS; ++term)
#pragma unroll
              for (int rb = 0; rb < NB; ++rb) {
                kr[s % 2][term][rb] = *reinterpret_cast<const h8*>(&sh.k[ring][term][rb][s][at][0]);
                qr[s % 2][term][rb] = *reinterpret_cast<const h8*>(&sh.q[ring][term][rb][s][at][0]);
              }
#pragma unroll
            for (int cs = 0; cs < NCS; ++cs) split8(S[2 * s][cs], S[2 * s + 1][cs], one, hi[s % 2][cs], lo[s % 2][cs]);
          };
          stage(0);
#pragma unroll
          for (int s = 0; s < KS; ++s) {
            if (s + 1 < KS) stage(s + 1);
#pragma unroll
            for (int part = 0; part < TERMS + 1; ++part)   // hi hi, hi lo, lo hi
#pragma unroll
              for (int cs = 0; cs < NCS; ++cs)
#pragma unroll
                for (int rb = 0; rb < NB; ++rb) {
                  const h8 x = part == 1 ? lo[s % 2][cs] : hi[s % 2][cs];
                  ks[rb][cs] = mfma(kr[s % 2][part == 2 ? TERMS - 1 : 0][rb], x, ks[rb][cs]);
                  qs[rb][cs] = mfma(qr[s % 2][part == 2 ? TERMS - 1 : 0][rb], x, qs[rb][cs]);
                }
          }
        } else {
#pragma unroll
          for (int s = 0; s < KS; ++s) {
            h8 hi[NCS], lo[NCS];
#pragma unroll
            for (int cs = 0; cs < NCS; ++cs) split8(S[2 * s][cs], S[2 * s + 1][cs], one, hi[cs], lo[cs]);
            const int at = row_slot(s, g, lane % 16);
#pragma unroll
            for (int rb = 0; rb < NB; ++rb) {
              const h8 k0 = *reinterpret_cast<const h8*>(&sh.k[ring][0][rb][s][at][0]);
              const h8 q0 = *reinterpret_cast<const h8*>(&sh.q[ring][0][rb][s][at][0]);
#pragma unroll
              for (int cs = 0; cs < NCS; ++cs) {
                ks[rb][cs] = mfma(k0, hi[cs], ks[rb][cs]);
                qs[rb][cs] = mfma(q0, hi[cs], qs[rb][cs]);
                ks[rb][cs] = mfma(k0, lo[cs], ks[rb][cs]);
                qs[rb][cs] = mfma(q0, lo[cs], qs[rb][cs]);
              }
              if constexpr (F32) {
                const h8 k1 = *reinterpret_cast<const h8*>(&sh.k[ring][1][rb][s][at][0]);
                const h8 q1 = *reinterpret_cast<const h8*>(&sh.q[ring][1][rb][s][at][0]);
#pragma unroll
                for (int cs = 0; cs < NCS; ++cs) {
                  ks[rb][cs] = mfma(k1, hi[cs], ks[rb][cs]);
                  qs[rb][cs] = mfma(q1, hi[cs], qs[rb][cs]);
                }
              }
            }
          }
        }
        // The chunk's unit, while these products run.  In one column, a step
        // S <- alpha (I - beta kh kh^T) S + beta kh v lengthens S by at most
        // |v|, so S stays within |S0|_2 + C max|v| through the chunk, and the
        // corrections U_j and R within max|v| more; |S0|_2 <= sqrt(dk) max|S0|.
        // 2 max(sqrt(dk) max|S0|, (C + 1) max|v|) covers them all.
        const float last = sh.last[ring];
        f32x4 R[NCS][NB], U[NCS][NB];
        int to[NCS];
        bool wide = false;
        const int last_log = exponent(last) - kBias;
        const int past_now = it == chunks - 1 ? past : 0;
#pragma unroll
        for (int cs = 0; cs < NCS; ++cs)
#pragma unroll
          for (int rb = 0; rb < NB; ++rb)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              float x[NCS];
              v[rb][r].unpack(x);
              R[cs][rb][r] = x[cs];
            }
#pragma unroll
        for (int cs = 0; cs < NCS; ++cs) {
          constexpr float kRoot = DK == 128 ? 11.4f : DK == 64 ? 8.0f : 5.7f;
          constexpr int kRootLog = DK == 128 ? 3 : 4;   // floor(-log2(2 kRoot / 2^kDown))
          constexpr int kTopLog = NB == 2 ? 1 : 2;      // floor(-log2(2 (C + 1) / 2^kDown))
          constexpr int kDown = 8;   // the bounds' exponents are taken 2^8 lower: no finite v or S overflows
          float m = 0.0f;            // max |v| of the lane's group of tokens
#pragma unroll
          for (int rb = 0; rb < NB; ++rb)
#pragma unroll
            for (int r = 0; r < 4; ++r) m = fmaxf(m, fabsf(R[cs][rb][r]));
          const int ev = exponent(m * (2.0f * (C + 1) / (1 << kDown)));
          const int es = exponent(largest(S, cs) * (2.0f * kRoot / (1 << kDown))) + sig[cs];
          const int e = max16_32(max(ev, es));
          to[cs] = unit_for(e + kDown, sig[cs] - 100);
          // max |S| of the lane's keys and max |v| of its group, rounded down, by how much
          // they exceed a state of zero (-1: it is one).  S0 as the chunk's decay leaves
          // it bounds a group from below; a group without v goes with S0, and gives zero
          // where that is zero.
          constexpr int kNone = kSigMin + kRootLog + 1;
          const int s0 = es + kRootLog - kNone, v0 = ev + kTopLog + past_now - kNone;
          const int from_s = ev == 0 ? s0 : max(s0 + last_log, 0);
          const uint32_t least = max(max(static_cast<uint32_t>(v0), static_cast<uint32_t>(from_s)),
                                     static_cast<uint32_t>(kSigMin + kBias + 1 - kNone));
          // The old unit counts like the bound that it came from (twice, for the sum over
          // keys), as S is split in it.
          wide |= least <= static_cast<uint32_t>(max(e, sig[cs] + kBias + 15 - kDown) - (kWide - kDown) - kNone);
        }
        // A chunk that goes token by token runs through the lines below as well, with S
        // kept as it is and no outputs stored, so that the others need not wait for this
        // verdict.
        const bool walks = __any(wide);   // uniform
        const float scale_u = walks ? 0.0f : 1.0f / kUnitT;
        float keep[NCS], up_old[NCS], up_new[NCS], down[NCS], shift[NCS];
#pragma unroll
        for (int cs = 0; cs < NCS; ++cs) {
          const int d = to[cs] - sig[cs];
          up_old[cs] = __builtin_ldexpf(1.0f, sig[cs]);
          shift[cs] = __builtin_ldexpf(1.0f, -d);   // 0 where the new unit dwarfs all of S
          keep[cs] = walks ? 1.0f : __builtin_ldexpf(last, -d);
          down[cs] = __builtin_ldexpf(1.0f, -to[cs]);
          up_new[cs] = __builtin_ldexpf(1.0f / kUnitT, to[cs]);
        }
        // R = v - e^G kh^T S, in the new unit (zero past the end)
#pragma unroll
        for (int rb = 0; rb < NB; ++rb) {
          const f32x4 ck = *reinterpret_cast<const f32x4*>(&sh.tab[ring][1][16 * rb + 4 * g]);
#pragma unroll
          for (int cs = 0; cs < NCS; ++cs)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              R[cs][rb][r] = fmaf(-ck[r] * shift[cs], ks[rb][cs][r], down[cs] * R[cs][rb][r]);
        }
        if (it + 1 < chunks) load_v(it + 1);
#pragma unroll
        for (int cs = 0; cs < NCS; ++cs) {
          // U = T R
          ht hi, lo;
          split_rows(R[cs], one, hi, lo);
#pragma unroll
          for (int rb = 0; rb < NB; ++rb) {
            const ht t0h = *reinterpret_cast<const ht*>(&sh.t[it % 2][0][rb][lane][0]);
            const ht t0l = *reinterpret_cast<const ht*>(&sh.t[it % 2][1][rb][lane][0]);
            f32x4 acc = {0, 0, 0, 0};
            acc = mfma(t0l, hi, acc);
            acc = mfma(t0h, lo, acc);
            U[cs][rb] = mfma(t0h, hi, acc) * scale_u;
          }
        }
#pragma unroll
        for (int cs = 0; cs < NCS; ++cs) sig[cs] = walks ? sig[cs] : to[cs];
        // S = e^(G_last) S + (diag(e^(G_last - G)) Kh)^T U
#pragma unroll
        for (int cs = 0; cs < NCS; ++cs) {
          ht hi, lo;
          f32x4 wu[NB];
#pragma unroll
          for (int rb = 0; rb < NB; ++rb)
            wu[rb] = U[cs][rb] * *reinterpret_cast<const f32x4*>(&sh.tab[ring][3][16 * rb + 4 * g]);
          split_rows(wu, one, hi, lo);
#pragma unroll
          for (int j = 0; j < KB; ++j) {
            const int at = kt_slot(j, g, lane % 16);
            f32x4 acc = S[j][cs] * keep[cs];
            if constexpr (F32) acc = mfma(*reinterpret_cast<const ht*>(&sh.kt[ring][1][j][at][0]), hi, acc);
            const ht k0 = *reinterpret_cast<const ht*>(&sh.kt[ring][0][j][at][0]);
            acc = mfma(k0, lo, acc);
            S[j][cs] = mfma(k0, hi, acc);
          }
        }
        // O = e^G Qh S0 + P U
#pragma unroll
        for (int cs = 0; cs < NCS; ++cs) {
          ht hi, lo;
          split_rows(U[cs], one, hi, lo);
#pragma unroll
          for (int rb = 0; rb < NB; ++rb) {
            const ht p0 = *reinterpret_cast<const ht*>(&sh.p[third][0][rb][lane][0]);
            const ht p1 = *reinterpret_cast<const ht*>(&sh.p[third][1][rb][lane][0]);
            f32x4 acc = {0, 0, 0, 0};
            acc = mfma(p1, hi, acc);
            acc = mfma(p0, lo, acc);
            acc = mfma(p0, hi, acc);
            const f32x4 cq = *reinterpret_cast<const f32x4*>(&sh.tab[ring][2][16 * rb + 4 * g]);
#pragma unroll
            for (int r = 0; r < 4; ++r)
              qs[rb][cs][r] = fmaf(cq[r] * up_old[cs], qs[rb][cs][r], a.scale * up_new[cs] * acc[r]);
          }
        }
        const __amdgpu_buffer_rsrc_t ro = chunk_rows(a.out, it);
        const int gone = walks ? static_cast<int>(0x80000000u) : 0;   // past every row: dropped
#pragma unroll
        for (int rb = 0; rb < NB; ++rb)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float x[NCS];
#pragma unroll
            for (int cs = 0; cs < NCS; ++cs) x[cs] = qs[rb][cs][r];
            Columns<F32, NCS>::store(ro, voff[rb][r] | gone, x);
          }
        if (__builtin_expect(walks, 0)) {
          walk_chunk<KB, NCS, DK, F32>(a, sh, w, ring, it * C, min(w.n - it * C, C), chunk_rows(a.v, it),
                                       ro, voff[0][0] - 4 * g * stride, stride, lane, sig, S);
          __builtin_amdgcn_s_waitcnt(0x0f70);   // vmcnt(0): waits of the usual form then count on its own loads alone
        }
        third = third == kRingP - 1 ? 0 : third + 1;
      }
      lds_barrier();
    }
#pragma unroll
    for (int cs = 0; cs < NCS; ++cs) {
      const float f = __builtin_ldexpf(1.0f, sig[cs]);
#pragma unroll
      for (int j = 0; j < KB; ++j) S[j][cs] *= f;
    }
    slab_io<true, KB, NCS>(res, layout, state_bf16, dv, colw, lane, S);
  }
}

// ---------------------------------------------------------------------------
// dispatch
// ---------------------------------------------------------------------------

constexpr int kCus = 256;

template <int NCW, int NCS, int DK, bool F32>
hipError_t launch_form(const DecodeArgs& args, int dv, int layout, int state_bf16, hipStream_t stream) {
  const void* fn = reinterpret_cast<const void*>(&gdr_prefill<NCW, NCS, DK, F32>);
  const int64_t nwg = static_cast<int64_t>(args.B) * args.HV * (dv / (NCW * 16 * NCS));
  void* kargs[] = {const_cast<DecodeArgs*>(&args), &dv, &layout, &state_bf16};
  const size_t lds = sizeof(Shared<DK, F32>);
  if (lds > 65536) {   // beyond the default limit of dynamic LDS
    const hipError_t rc = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds));
    if (rc != hipSuccess) return rc;
  }
  return hipLaunchKernel(fn, dim3(static_cast<uint32_t>(nwg)), dim3((NCW + kHelpers) * kWave), kargs, lds, stream);
}

// A workgroup takes a CU's issue slots, or all of its LDS, so the time is the number
// of rounds of 256 workgroups times a form's time per chunk (at dk <= 64 two fit a CU
// with bf16 rows, but then share its issue slots: 64 tiles below).  The fewer
// columns, the shorter the chain of a chunk, but the more workgroups: the narrowest
// form that is one round, else the widest.  1024 tokens, us by number of tiles (forms
// of 16 / 32 / 64 / 128 columns), bf16 rows:
//               dk = dv = 128              dk = 64, dv = 128          dk = 32, dv = 128
//      8 tiles    49   58   65   84         42   43   47   62         45   45   47   57
//     32          50   60   66   86         42   43   48   63         46   46   47   59
//     64          96   61   68   86         62   44   50   63         56   47   48   60
//    128         191  118   72   87        150   67   52   64        109   59   50   60
//    192         285  174  131   88        204   99   78   65        162   97   70   61
//    256         381  234  143  100        256  159   84   74        213  114   72   63
//    384         572  351  208  181        381  225  126  130        315  171  107   96
//    768        1142  702  436  309        758  457  262  225        624  354  225  167
// Between rounds the widest may lose a little (fp32 rows, dk = 64, 384 tiles: 179 us
// with 64 columns, 198 with 128).
// 16 columns per state wave beat 32 (64 columns in two waves 86 us against 65
// in four) but for the 128-column form, where eight waves of 16 columns and the
// helpers are short of registers and issue slots (652 us against 624 on 768
// tiles x 2048 tokens).
template <int DK, bool F32>
hipError_t launch_dk(const DecodeArgs& args, int dv, int layout, int state_bf16, hipStream_t stream) {
  const int64_t tiles = static_cast<int64_t>(args.B) * args.HV;
  const auto one_round = [&](int columns) { return tiles * (dv / columns) <= kCus; };
  if (one_round(16)) return launch_form<1, 1, DK, F32>(args, dv, layout, state_bf16, stream);
  if (dv == 32 || one_round(32)) return launch_form<2, 1, DK, F32>(args, dv, layout, state_bf16, stream);
  if (dv == 64 || one_round(64)) return launch_form<4, 1, DK, F32>(args, dv, layout, state_bf16, stream);
  return launch_form<4, 2, DK, F32>(args, dv, layout, state_bf16, stream);
}

}  // namespace

int launch_gdr_prefill(const DecodeArgs& args, int dk, int dv, bool qkv_bf16, bool state_bf16, int state_layout,
                       hipStream_t stream) {
  hipError_t rc = hipSuccess;
  switch (dk) {
    case 32: rc = qkv_bf16 ? launch_dk<32, false>(args, dv, state_layout, state_bf16, stream)
                           : launch_dk<32, true>(args, dv, state_layout, state_bf16, stream); break;
    case 64: rc = qkv_bf16 ? launch_dk<64, false>(args, dv, state_layout, state_bf16, stream)
                           : launch_dk<64, true>(args, dv, state_layout, state_bf16, stream); break;
    case 128: rc = qkv_bf16 ? launch_dk<128, false>(args, dv, state_layout, state_bf16, stream)
                            : launch_dk<128, true>(args, dv, state_layout, state_bf16, stream); break;
    default: return KDA_ERR_UNSUPPORTED;
  }
  return rc == hipSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}

}  // namespace kda
