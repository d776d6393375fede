// kda_gdr_prefill.hip - the gated delta rule over whole prompts, in chunks
// of 32 tokens on the matrix cores (kda_gdr_prefill).
//
// Mathematics.  One decay per token and head, G_i its log summed from the
// chunk's start, S0 the state before the chunk:
//   A_ij = beta_i e^(G_i - G_j) kh_i.kh_j          (i > j)
//   T    = (I + A)^-1                              (unit lower triangular)
//   U    = T diag(beta) (V - diag(e^G) Kh S0)
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
//   - the state, R = diag(beta)(V - ...) and U are scaled by a power of two
//     per value column and taken as hi + lo; T and P, whose entries are at
//     most 1 in size, as hi + lo.
// |T_ij| <= 1: T_ij = -beta_i kh_i^T [product of contractions] kh_j.  The
// lo.lo terms (2^-22) are dropped.  So an operand carries about 22 bits and
// the result is close to fp32's; two bf16 terms would leave 16 bits.  G is
// kept as a sum of two floats (summed in fp64): only differences of it count
// and an fp32 sum of strong decays loses them.
//
// Work split.  Value columns never interact, so a workgroup owns one
// (request, value head) tile and NCW * 16 * NCS of its columns.  The chain
// from chunk to chunk (S0 -> R -> U -> S) runs in NCW state waves, each
// with 16 * NCS columns, all keys in registers, and no exchange with other
// waves.  What does not depend on the state is made ahead by four helper
// waves, each a chunk further on:
//   wave 0  K: fp16 rows in operand order (K for K S0 and the Gram
//           products, K^T for the state update), norms      chunk c + 3
//   wave 1  Q: the same, and the gates (g, G, beta)           chunk c + 3
//   wave 2  the Gram products: A, P, the factor tables        chunk c + 2
//   wave 3  T: two 16 x 16 triangular inverses and their join chunk c + 1
//   others  the state chain                                   chunk c
// with one barrier per chunk.  The accumulator layout of one product (four
// consecutive rows per lane) is the operand layout of the next once the
// operands' order of k is permuted to match, so the chain never leaves its
// registers.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "kda.h"
#include "kda_device.h"
#include "kda_internal.h"
#include "kda_tile.h"

namespace kda {
namespace {

constexpr int kC = 32;            // tokens per chunk
constexpr int kHelpers = 4;
constexpr int kRing = 4;          // chunks of q and k held in LDS

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

__device__ __forceinline__ f32x4 mfma(h8 a, h8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// x * s as hi + lo in fp16 (s a power of two).  The packed hi is made opaque
// so that lo is taken from it and not from conversions of its own.
__device__ __forceinline__ void split2(float x0, float x1, float s, h2& hi, h2& lo) {
  hi = h2{static_cast<_Float16>(x0 * s), static_cast<_Float16>(x1 * s)};
  asm("" : "+v"(hi));
  lo = h2{static_cast<_Float16>(__builtin_fmaf(x0, s, -static_cast<float>(hi.x))),
          static_cast<_Float16>(__builtin_fmaf(x1, s, -static_cast<float>(hi.y)))};
}

__device__ __forceinline__ void split8(const f32x4& x, const f32x4& y, float s, h8& hi, h8& lo) {
  h2 h[4], l[4];
  split2(x[0], x[1], s, h[0], l[0]);
  split2(x[2], x[3], s, h[1], l[1]);
  split2(y[0], y[1], s, h[2], l[2]);
  split2(y[2], y[3], s, h[3], l[3]);
  hi = h8{h[0].x, h[0].y, h[1].x, h[1].y, h[2].x, h[2].y, h[3].x, h[3].y};
  lo = h8{l[0].x, l[0].y, l[1].x, l[1].y, l[2].x, l[2].y, l[3].x, l[3].y};
}

// The power of two that brings m (>= 0) into [2^P, 2^(P + 1)), and its
// inverse; below 2^-100 the factor stays where it is there (zero included).
template <int P>
__device__ __forceinline__ float scale_for(float m, float& inverse) {
  uint32_t e = __float_as_uint(m) >> 23;
  e = e < 27u ? 27u : e;
  inverse = __uint_as_float((e - P) << 23);
  return __uint_as_float((254u + P - e) << 23);
}

__device__ __forceinline__ float max16_32(float x) {   // over lanes that share lane % 16
  const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
  const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
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
  return g * 16 + (row ^ ((g + 4 * s) & 7));
}

template <int DK, bool F32>
struct Shared {
  static constexpr int KS = DK / 32;       // 32-key steps
  static constexpr int TERMS = F32 ? 2 : 1;
  _Float16 k[kRing][TERMS][2][KS][64][8];          // K rows: [token block][key step]
  _Float16 q[kRing][TERMS][2][KS][64][8];
  _Float16 kt[kRing][TERMS][DK / 16][64][8];       // K^T: [key block], k = token
  _Float16 p[kRing][2][2][64][8];                  // P hi, lo: [token block]
  _Float16 t[2][2][2][64][8];                      // T hi, lo
  float a[2][3][16][16];                           // A: blocks 00, 11, 10; [column][row]
  float join[2][16][16];                           // T's diagonal blocks, row-major
  float norm_k[2][kC], norm_q[2][kC];              // kh = norm_k * stored row
  float g_hi[2][kC], g_lo[2][kC], beta[2][kC];
  float tab[kRing][4][kC];                         // beta; beta e^G norm_k; scale e^G norm_q; norm_k e^(last - G)
  float last[kRing];                               // e^(G_last)
};

// ---------------------------------------------------------------------------
// helper waves 0 and 1: rows of k or q
// ---------------------------------------------------------------------------

// A lane holds a pair of channels of TL = 8 NG tokens: dk / 2 lanes cover a
// token, 128 / dk lane groups share the chunk's tokens, each with NG of the
// four operand groups g.  Token i of group gi is 4 g + i % 4 + 16 (i / 4).
template <int DK, bool F32>
struct RowLoader {
  static constexpr int LANES = DK / 2;
  static constexpr int SPLIT = kWave / LANES;
  static constexpr int NG = 4 / SPLIT;
  static constexpr int TL = 8 * NG;
  uint32_t w[TL * (F32 ? 2 : 1)];

  static __device__ __forceinline__ int token(int lane, int i) {
    const int g = (lane / LANES) * NG + i / 8;
    return 4 * g + i % 4 + 16 * ((i / 4) % 2);
  }

  // rows t0 .. t0 + n - 1 of head h (n >= 1); rows past them are zero
  __device__ __forceinline__ void load(const void* base, int64_t t0, int n, int H, int h, int lane) {
    const int c = 2 * (lane % LANES);
#pragma unroll
    for (int i = 0; i < TL; ++i) {
      const int t = token(lane, i);
      const int64_t off = ((t0 + (t < n ? t : 0)) * H + h) * DK + c;
      if constexpr (F32) {
        const u32x2 x = *reinterpret_cast<const u32x2*>(static_cast<const float*>(base) + off);
        w[2 * i] = t < n ? x.x : 0u;
        w[2 * i + 1] = t < n ? x.y : 0u;
      } else {
        const uint32_t x = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(base) + off);
        w[i] = t < n ? x : 0u;
      }
    }
  }

  __device__ __forceinline__ void unpack(int i, float& x, float& y) const {
    if constexpr (F32) {
      x = __uint_as_float(w[2 * i]);
      y = __uint_as_float(w[2 * i + 1]);
    } else {
      x = bf16_to_f32(w[i] & 0xffffu);
      y = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};

// Converts a chunk's rows: fp16 rows in operand order, their factors
// (norm[token] * stored row = unit row), and for k the transposed operand.
template <int DK, bool F32, bool KT>
__device__ __forceinline__ void convert_rows(const RowLoader<DK, F32>& in, float l2_eps, int lane,
                                             _Float16 (*rows)[2][DK / 32][64][8], _Float16 (*kt)[DK / 16][64][8],
                                             float* norm) {
  using L = RowLoader<DK, F32>;
  constexpr int TL = L::TL;
  constexpr int LOG_LANES = log2_exact<L::LANES>();
  constexpr int LOG_TL = log2_exact<TL>();
  static_assert(LOG_LANES == LOG_TL + 1, "one level of plain sums");
  float sq[TL];
#pragma unroll
  for (int i = 0; i < TL; ++i) {
    float x, y;
    in.unpack(i, x, y);
    sq[i] = fmaf(x, x, y * y);
  }
  // lane bits LOG_LANES - 1 .. 1 pick the token, bit 0 is summed
  transpose_levels<TL / 2, LOG_LANES - 1>(sq, lane);
  const float sum = xchg_level<0>(false, sq[0], sq[0]);
  const int mine = (lane % L::LANES) >> 1;   // index of this lane's token
  // 2^-e with 2^e <= norm < 2^(e + 1), from the exponent of the square.  A row
  // whose square is not finite is multiplied by 0, as by 1 / sqrt(inf): finite
  // values give kh = 0, infinities and NaN give NaN.
  const uint32_t ex = __float_as_uint(sum) >> 23;
  const int e = (static_cast<int>(ex) - 127) >> 1;
  const bool usable = ex < 255u;
  const float down = usable ? __uint_as_float(static_cast<uint32_t>(127 - e) << 23) : 0.0f;
  const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
  if ((lane & 1) == 0) norm[L::token(lane, mine)] = usable ? up * rsqrt_f(sum + l2_eps) : 0.0f;

  const int c = 2 * (lane % L::LANES);
  const int s = c / 32, half = (c % 32) / 16, g = (c % 16) / 4, r = c % 4;
  constexpr int NG = L::NG;
  h2 hi[TL], lo[TL];
#pragma unroll
  for (int i = 0; i < TL; ++i) {
    // this lane group's token i is held by its lanes 2 i, 2 i + 1
    const float f = __shfl(down, (lane & ~(L::LANES - 1)) + 2 * i);
    float x, y;
    in.unpack(i, x, y);
    if constexpr (F32) split2(x, y, f, hi[i], lo[i]);
    else hi[i] = h2{static_cast<_Float16>(x * f), static_cast<_Float16>(y * f)};
    const int t = L::token(lane, i);
    const int at = row_slot(s, g, t % 16);
    *reinterpret_cast<h2*>(&rows[0][t / 16][s][at][half * 4 + r]) = hi[i];
    if constexpr (F32) *reinterpret_cast<h2*>(&rows[1][t / 16][s][at][half * 4 + r]) = lo[i];
  }
  if constexpr (KT) {
#pragma unroll
    for (int gi = 0; gi < NG; ++gi) {
      const int tg = (lane / L::LANES) * NG + gi;   // operand group: these 8 tokens
#pragma unroll
      for (int ch = 0; ch < 2; ++ch) {
        const int cc = c + ch;
        const int at = tg * 16 + (cc % 16);
        h8 v;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = ch ? hi[8 * gi + i].y : hi[8 * gi + i].x;
        *reinterpret_cast<h8*>(&kt[0][cc / 16][at][0]) = v;
        if constexpr (F32) {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = ch ? lo[8 * gi + i].y : lo[8 * gi + i].x;
          *reinterpret_cast<h8*>(&kt[1][cc / 16][at][0]) = v;
        }
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

struct Tile {
  int b, hv, h, slot, col0;   // col0: first column of the workgroup
  int t0, n;                  // first row and tokens
};

template <int NCW, int NCS, int DK, bool F32>
__global__ void __launch_bounds__((NCW + kHelpers) * kWave, 1)
gdr_prefill(const DecodeArgs a, const int dv, const int layout, const int state_bf16) {
  constexpr int KS = DK / 32;          // key steps of 32
  constexpr int KB = DK / 16;          // key blocks of 16
  constexpr int NC = NCW * 16 * NCS;   // columns of the workgroup
  constexpr int TERMS = F32 ? 2 : 1;
  using Sh = Shared<DK, F32>;
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
  const int chunks = (w.n + kC - 1) / kC;

  // the upper blocks of P and T stay zero
  for (int i = threadIdx.x; i < kRing * 2 * 64; i += blockDim.x)
    *reinterpret_cast<h4*>(&sh.p[i / 128][(i / 64) % 2][0][i % 64][4]) = h4{0, 0, 0, 0};
  for (int i = threadIdx.x; i < 2 * 2 * 64; i += blockDim.x)
    *reinterpret_cast<h4*>(&sh.t[i / 128][(i / 64) % 2][0][i % 64][4]) = h4{0, 0, 0, 0};

  if (wave < 2) {
    // ---- helpers 0 and 1: k / q rows of chunk it + 3 ----
    RowLoader<DK, F32> raw;
    const void* const src = wave == 0 ? a.k : a.q;
    raw.load(src, t0, w.n, a.H, w.h, lane);
    const float amp = exp_f(a.a_log[w.hv]);
    const float bias = a.dt_bias[w.hv];
    const int tl = lane % kC;
    auto gate_at = [&](int c) {   // raw gate and beta logit of the lane's token
      const int t = c * kC + tl;
      const int64_t off = (static_cast<int64_t>(t0) + (t < w.n ? t : 0)) * a.HV + w.hv;
      return make_float2(a.raw_gate[off], a.beta_logits[off]);
    };
    float2 gate = make_float2(0.0f, 0.0f);
    if (wave == 1) gate = gate_at(0);
    lds_barrier();
    for (int it = -3; it < chunks; ++it) {
      const int c = it + 3;
      if (c < chunks) {
        const RowLoader<DK, F32> cur = raw;
        const float2 gb = gate;
        if (c + 1 < chunks) {
          raw.load(src, static_cast<int64_t>(t0) + (c + 1) * kC, w.n - (c + 1) * kC, a.H, w.h, lane);
          if (wave == 1) gate = gate_at(c + 1);
        }
        const int ring = c % kRing, two = c % 2;
        if (wave == 0) {
          convert_rows<DK, F32, true>(cur, a.l2_eps, lane, sh.k[ring], sh.kt[ring], sh.norm_k[two]);
        } else {
          convert_rows<DK, F32, false>(cur, a.l2_eps, lane, sh.q[ring], nullptr, sh.norm_q[two]);
          const bool live = c * kC + tl < w.n;
          const float x = gb.x + bias;
          float gv = a.gate_mode == KDA_GATE_SOFTPLUS ? -amp * softplus_f(x) : a.lower_bound * sigmoid_f(amp * x);
          gv = gv < -200.0f ? -200.0f : gv;   // exp(-200) is 0 in fp32, and sums stay finite
          double sum = live ? static_cast<double>(gv) : 0.0;
#pragma unroll
          for (int m = 1; m < kC; m *= 2) {
            const double y = __shfl_up(sum, m, kC);
            if (tl >= m) sum += y;
          }
          if (lane < kC) {
            const float hi = static_cast<float>(sum);
            sh.g_hi[two][tl] = hi;
            sh.g_lo[two][tl] = static_cast<float>(sum - static_cast<double>(hi));
            sh.beta[two][tl] = live ? sigmoid_f(gb.y) : 0.0f;
          }
        }
      }
      lds_barrier();
    }
  } else if (wave == 2) {
    // ---- helper 2: Gram products of chunk it + 2 ----
    lds_barrier();
    for (int it = -3; it < chunks; ++it) {
      const int c = it + 2;
      if (c >= 0 && c < chunks) {
        const int ring = c % kRing, two = c % 2;
        f32x4 ka[3], pa[3];   // blocks 00, 11, 10
#pragma unroll
        for (int m = 0; m < 3; ++m) ka[m] = pa[m] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const int at = row_slot(s, g, lane % 16);
          h8 kk[TERMS][2], qq[TERMS][2];
#pragma unroll
          for (int term = 0; term < TERMS; ++term)
#pragma unroll
            for (int rb = 0; rb < 2; ++rb) {
              kk[term][rb] = *reinterpret_cast<const h8*>(&sh.k[ring][term][rb][s][at][0]);
              qq[term][rb] = *reinterpret_cast<const h8*>(&sh.q[ring][term][rb][s][at][0]);
            }
#pragma unroll
          for (int m = 0; m < 3; ++m) {
            const int i = m > 0, j = m == 1;   // row block i, column block j
            ka[m] = mfma(kk[0][i], kk[0][j], ka[m]);   // rows i, columns j
            pa[m] = mfma(kk[0][j], qq[0][i], pa[m]);   // rows j, columns i
            if constexpr (F32) {
              ka[m] = mfma(kk[0][i], kk[1][j], ka[m]);
              ka[m] = mfma(kk[1][i], kk[0][j], ka[m]);
              pa[m] = mfma(kk[0][j], qq[1][i], pa[m]);
              pa[m] = mfma(kk[1][j], qq[0][i], pa[m]);
            }
          }
        }
        const float g_last = sh.g_hi[two][kC - 1], g_last_lo = sh.g_lo[two][kC - 1];
#pragma unroll
        for (int m = 0; m < 3; ++m) {
          const int i = m > 0, j = m == 1;
          // A: column 16 j + lane % 16, rows 16 i + 4 g + 0..3
          {
            const int col = 16 * j + lane % 16, row = 16 * i + 4 * g;
            const float gh = sh.g_hi[two][col], gl = sh.g_lo[two][col], nk = sh.norm_k[two][col];
            const f32x4 rh = *reinterpret_cast<const f32x4*>(&sh.g_hi[two][row]);
            const f32x4 rl = *reinterpret_cast<const f32x4*>(&sh.g_lo[two][row]);
            const f32x4 rk = *reinterpret_cast<const f32x4*>(&sh.norm_k[two][row]);
            const f32x4 rb = *reinterpret_cast<const f32x4*>(&sh.beta[two][row]);
            f32x4 x;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float d = exp_f((rh[r] - gh) + (rl[r] - gl));
              x[r] = row + r > col ? ka[m][r] * nk * (rk[r] * rb[r]) * d : 0.0f;
            }
            *reinterpret_cast<f32x4*>(&sh.a[two][m][lane % 16][4 * g]) = x;
          }
          // P: row 16 i + lane % 16, columns 16 j + 4 g + 0..3
          {
            const int row = 16 * i + lane % 16, col = 16 * j + 4 * g;
            const float gh = sh.g_hi[two][row], gl = sh.g_lo[two][row], nq = sh.norm_q[two][row];
            const f32x4 ch = *reinterpret_cast<const f32x4*>(&sh.g_hi[two][col]);
            const f32x4 cl = *reinterpret_cast<const f32x4*>(&sh.g_lo[two][col]);
            const f32x4 ck = *reinterpret_cast<const f32x4*>(&sh.norm_k[two][col]);
            float x[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float d = exp_f((gh - ch[r]) + (gl - cl[r]));
              x[r] = col + r <= row ? pa[m][r] * nq * ck[r] * d : 0.0f;
            }
            h2 hi0, lo0, hi1, lo1;
            split2(x[0], x[1], 1.0f, hi0, lo0);
            split2(x[2], x[3], 1.0f, hi1, lo1);
            *reinterpret_cast<h4*>(&sh.p[ring][0][i][lane][4 * j]) = h4{hi0.x, hi0.y, hi1.x, hi1.y};
            *reinterpret_cast<h4*>(&sh.p[ring][1][i][lane][4 * j]) = h4{lo0.x, lo0.y, lo1.x, lo1.y};
          }
        }
        if (lane < kC) {
          const float gh = sh.g_hi[two][lane], gl = sh.g_lo[two][lane];
          const float nk = sh.norm_k[two][lane], be = sh.beta[two][lane];
          const float eg = exp_f(gh + gl);
          sh.tab[ring][0][lane] = be;
          sh.tab[ring][1][lane] = be * eg * nk;
          sh.tab[ring][2][lane] = a.scale * eg * sh.norm_q[two][lane];
          sh.tab[ring][3][lane] = nk * exp_f((g_last - gh) + (g_last_lo - gl));
          if (lane == kC - 1) sh.last[ring] = eg;
        }
      }
      lds_barrier();
    }
  } else if (wave == 3) {
    // ---- helper 3: T of chunk it + 1 ----
    lds_barrier();
    for (int it = -3; it < chunks; ++it) {
      const int c = it + 1;
      if (c >= 0 && c < chunks) {
        const int two = c % 2;
        // lane: row `row` of diagonal block `blk` (lanes 32.. repeat); x (I + A)
        // = e_row solved from the last column back
        const int blk = (lane / 16) % 2, row = lane % 16;
        float x[16];
#pragma unroll
        for (int j = 15; j >= 0; --j) {
          float acc = row == j ? 1.0f : 0.0f;
#pragma unroll
          for (int k = 15; k > j; --k) acc = fmaf(-x[k], sh.a[two][blk][j][k], acc);
          x[j] = acc;
        }
        if (lane < 32) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            *reinterpret_cast<f32x4*>(&sh.join[blk][row][4 * j]) = f32x4{x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]};
            h2 hi0, lo0, hi1, lo1;
            split2(x[4 * j], x[4 * j + 1], 1.0f, hi0, lo0);
            split2(x[4 * j + 2], x[4 * j + 3], 1.0f, hi1, lo1);
            *reinterpret_cast<h4*>(&sh.t[two][0][blk][16 * j + row][4 * blk]) = h4{hi0.x, hi0.y, hi1.x, hi1.y};
            *reinterpret_cast<h4*>(&sh.t[two][1][blk][16 * j + row][4 * blk]) = h4{lo0.x, lo0.y, lo1.x, lo1.y};
          }
        }
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront", "local");
        // T10^T = -T00^T (A10^T T11^T) on the fp32 matrix instruction
        f32x4 z = {0, 0, 0, 0}, y = {0, 0, 0, 0};
        const f32x4 at = *reinterpret_cast<const f32x4*>(&sh.a[two][2][lane % 16][4 * g]);    // A10[4g + r][lane % 16]
        const f32x4 bt = *reinterpret_cast<const f32x4*>(&sh.join[1][lane % 16][4 * g]);      // T11[lane % 16][4g + r]
#pragma unroll
        for (int r = 0; r < 4; ++r) z = __builtin_amdgcn_mfma_f32_16x16x4f32(at[r], bt[r], z, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < 4; ++r) y = __builtin_amdgcn_mfma_f32_16x16x4f32(sh.join[0][4 * g + r][lane % 16], z[r], y, 0, 0, 0);
        // y: column (row of T10) lane % 16, rows (columns of T10) 4 g + 0..3
        h2 hi0, lo0, hi1, lo1;
        split2(-y[0], -y[1], 1.0f, hi0, lo0);
        split2(-y[2], -y[3], 1.0f, hi1, lo1);
        *reinterpret_cast<h4*>(&sh.t[two][0][1][lane][0]) = h4{hi0.x, hi0.y, hi1.x, hi1.y};
        *reinterpret_cast<h4*>(&sh.t[two][1][1][lane][0]) = h4{lo0.x, lo0.y, lo1.x, lo1.y};
      }
      lds_barrier();
    }
  } else {
    // ---- state waves ----
    const int cw = wave - kHelpers;
    const int colw = w.col0 + cw * 16 * NCS;
    const int64_t tile_off = (static_cast<int64_t>(w.slot) * a.HV + w.hv) * (static_cast<int64_t>(DK) * dv);
    auto state_at = [&](int j, int r, int cs) {   // element of key 16 j + 4 g + r
      const int key = 16 * j + 4 * g + r, col = colw + column<NCS>(lane, cs);
      return tile_off + (layout == KDA_STATE_V_FIRST ? static_cast<int64_t>(col) * DK + key
                                                     : static_cast<int64_t>(key) * dv + col);
    };
    f32x4 S[KB][NCS];
#pragma unroll
    for (int j = 0; j < KB; ++j)
#pragma unroll
      for (int cs = 0; cs < NCS; ++cs)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          S[j][cs][r] = state_bf16 ? load_scalar<true>(a.state_pool, state_at(j, r, cs))
                                   : load_scalar<false>(a.state_pool, state_at(j, r, cs));

    const int64_t vcol = static_cast<int64_t>(w.hv) * dv + colw + column<NCS>(lane, 0);
    RawRun<!F32, NCS> v[2][4];
    auto load_v = [&](int c) {
#pragma unroll
      for (int rb = 0; rb < 2; ++rb)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int t = c * kC + 16 * rb + 4 * g + r;
          v[rb][r].load(a.v, (static_cast<int64_t>(t0) + (t < w.n ? t : 0)) * a.HV * dv + vcol);
        }
    };
    load_v(0);
    lds_barrier();
    for (int it = -3; it < chunks; ++it) {
      if (it >= 0) {
        const int ring = it % kRing;
        // K S and Q S, the state as hi + lo
        f32x4 ks[2][NCS], qs[2][NCS];
        float down_s[NCS], up_s[NCS];
#pragma unroll
        for (int cs = 0; cs < NCS; ++cs) {
          float m = 0.0f;
#pragma unroll
          for (int j = 0; j < KB; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) m = fmaxf(m, fabsf(S[j][cs][r]));
          down_s[cs] = scale_for<13>(max16_32(m), up_s[cs]);
#pragma unroll
          for (int rb = 0; rb < 2; ++rb) ks[rb][cs] = qs[rb][cs] = f32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          h8 hi[NCS], lo[NCS];
#pragma unroll
          for (int cs = 0; cs < NCS; ++cs) split8(S[2 * s][cs], S[2 * s + 1][cs], down_s[cs], hi[cs], lo[cs]);
          const int at = row_slot(s, g, lane % 16);
#pragma unroll
          for (int rb = 0; rb < 2; ++rb) {
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
        // R = beta v - beta e^G kh^T S
        f32x4 R[2][NCS];
#pragma unroll
        for (int rb = 0; rb < 2; ++rb) {
          const f32x4 be = *reinterpret_cast<const f32x4*>(&sh.tab[ring][0][16 * rb + 4 * g]);
          const f32x4 ck = *reinterpret_cast<const f32x4*>(&sh.tab[ring][1][16 * rb + 4 * g]);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float x[NCS];
            v[rb][r].unpack(x);
            const bool live = it * kC + 16 * rb + 4 * g + r < w.n;
#pragma unroll
            for (int cs = 0; cs < NCS; ++cs)
              R[rb][cs][r] = live ? fmaf(-ck[r] * up_s[cs], ks[rb][cs][r], be[r] * x[cs]) : 0.0f;
          }
        }
        if (it + 1 < chunks) load_v(it + 1);
        // U = T R
        f32x4 U[2][NCS];
        float up_u[NCS];
#pragma unroll
        for (int cs = 0; cs < NCS; ++cs) {
          float m = 0.0f;
#pragma unroll
          for (int rb = 0; rb < 2; ++rb)
#pragma unroll
            for (int r = 0; r < 4; ++r) m = fmaxf(m, fabsf(R[rb][cs][r]));
          const float down = scale_for<9>(max16_32(m), up_u[cs]);   // |U| <= 32 max|R|
          h8 hi, lo;
          split8(R[0][cs], R[1][cs], down, hi, lo);
#pragma unroll
          for (int rb = 0; rb < 2; ++rb) {
            const h8 t0h = *reinterpret_cast<const h8*>(&sh.t[it % 2][0][rb][lane][0]);
            const h8 t0l = *reinterpret_cast<const h8*>(&sh.t[it % 2][1][rb][lane][0]);
            f32x4 acc = {0, 0, 0, 0};
            acc = mfma(t0l, hi, acc);
            acc = mfma(t0h, lo, acc);
            U[rb][cs] = mfma(t0h, hi, acc);
          }
        }
        // S = e^(G_last) S + (diag(e^(G_last - G)) Kh)^T U
        const float last = sh.last[ring];
        const f32x4 w0 = *reinterpret_cast<const f32x4*>(&sh.tab[ring][3][4 * g]);
        const f32x4 w1 = *reinterpret_cast<const f32x4*>(&sh.tab[ring][3][16 + 4 * g]);
#pragma unroll
        for (int cs = 0; cs < NCS; ++cs) {
          h8 hi, lo;
          split8(U[0][cs] * w0, U[1][cs] * w1, 1.0f, hi, lo);
#pragma unroll
          for (int j = 0; j < KB; ++j) {
            const h8 k0 = *reinterpret_cast<const h8*>(&sh.kt[ring][0][j][lane][0]);
            f32x4 acc = {0, 0, 0, 0};
            if constexpr (F32) acc = mfma(*reinterpret_cast<const h8*>(&sh.kt[ring][1][j][lane][0]), hi, acc);
            acc = mfma(k0, lo, acc);
            acc = mfma(k0, hi, acc);
#pragma unroll
            for (int r = 0; r < 4; ++r) S[j][cs][r] = fmaf(acc[r], up_u[cs], last * S[j][cs][r]);
          }
        }
        // O = e^G Qh S0 + P U
#pragma unroll
        for (int cs = 0; cs < NCS; ++cs) {
          h8 hi, lo;
          split8(U[0][cs], U[1][cs], 1.0f, hi, lo);
#pragma unroll
          for (int rb = 0; rb < 2; ++rb) {
            const h8 p0 = *reinterpret_cast<const h8*>(&sh.p[ring][0][rb][lane][0]);
            const h8 p1 = *reinterpret_cast<const h8*>(&sh.p[ring][1][rb][lane][0]);
            f32x4 acc = {0, 0, 0, 0};
            acc = mfma(p1, hi, acc);
            acc = mfma(p0, lo, acc);
            acc = mfma(p0, hi, acc);
            const f32x4 cq = *reinterpret_cast<const f32x4*>(&sh.tab[ring][2][16 * rb + 4 * g]);
#pragma unroll
            for (int r = 0; r < 4; ++r)
              qs[rb][cs][r] = fmaf(cq[r] * up_s[cs], qs[rb][cs][r], a.scale * up_u[cs] * acc[r]);
          }
        }
#pragma unroll
        for (int rb = 0; rb < 2; ++rb)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int t = it * kC + 16 * rb + 4 * g + r;
            if (t < w.n) {
              const int64_t off = (static_cast<int64_t>(t0) + t) * a.HV * dv + vcol;
              if constexpr (NCS == 2) store_pair<!F32>(a.out, off, qs[rb][0][r], qs[rb][1][r]);
              else store_scalar<!F32>(a.out, off, qs[rb][0][r]);
            }
          }
      }
      lds_barrier();
    }
#pragma unroll
    for (int j = 0; j < KB; ++j)
#pragma unroll
      for (int cs = 0; cs < NCS; ++cs)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if (state_bf16) store_scalar<true>(a.state_pool, state_at(j, r, cs), S[j][cs][r]);
          else store_scalar<false>(a.state_pool, state_at(j, r, cs), S[j][cs][r]);
        }
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

template <int DK, bool F32>
hipError_t launch_dk(const DecodeArgs& args, int dv, int layout, int state_bf16, hipStream_t stream) {
  const int64_t tiles = static_cast<int64_t>(args.B) * args.HV;
  if (dv >= 128 && tiles >= kCus) return launch_form<4, 2, DK, F32>(args, dv, layout, state_bf16, stream);
  if (dv >= 64 && tiles * (dv / 64) >= kCus) return launch_form<2, 2, DK, F32>(args, dv, layout, state_bf16, stream);
  if (tiles * (dv / 32) >= kCus) return launch_form<1, 2, DK, F32>(args, dv, layout, state_bf16, stream);
  return launch_form<1, 1, DK, F32>(args, dv, layout, state_bf16, stream);
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
    case 128: rc = launch_dk<128, false>(args, dv, state_layout, state_bf16, stream); break;
    default: return KDA_ERR_UNSUPPORTED;
  }
  return rc == hipSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}

}  // namespace kda
