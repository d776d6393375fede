// kda_ssm_prefill.hip - the selective state space scan over whole prompts
// (kda_ssm_prefill), in chunks of 64 tokens on the matrix cores.
//
// With g_t = -exp(a_log) step_t and c_t its running sum since the chunk's
// start, S0 the state before the chunk and x', B, C the convolved channels:
//     y_t = exp(c_t) C_t^T S0 + sum_{s<=t} (C_t.B_s) exp(c_t - c_s) step_s x'_s + d_skip x'_t
//     S   = exp(c_last) S0 + sum_s B_s (exp(c_last - c_s) step_s x'_s)^T
// Every factor is at most one, so nothing overflows that the scan does not.
//
// ssm_keys, one workgroup per (chunk, group): convolves B and C, which all
// heads of the group share, and leaves them and C.B in the order in which the
// matrix instructions take them, in bf16 terms.  It also sets the windows.
// ssm_scan, one wave per (request, value head, up to 64 value columns): walks
// the chunks with the state in its accumulators.  The accumulators of two
// 16-key tiles are the instruction's other operand for 32 keys in the order
// that ssm_keys stores C in, and the pairs (C.B) arrive in operand order, so
// no value moves between lanes.  It convolves its own columns of x.
// Where a batch has few heads for the chip, requests are split into segments:
// ssm_scan (kSegment) runs all segments from a zero state, ssm_join passes
// the states on, and ssm_scan (kJoined) runs the segments from there.
//
// Precision: an fp32 value is the sum of three bf16 terms, 8 bits each, taken
// by truncation, so that no term leaves the value's range.  Products of three
// terms each keep about 24 bits (six matrix instructions), of two about 16
// (three): the state takes three for an fp32 pool or fp32 activations, and
// what only reaches bf16 outputs or a bf16 pool takes two.  c is summed in
// fp64 and kept in two fp32 parts: differences of large sums are what counts.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "kda.h"
#include "kda_device.h"
#include "kda_internal.h"
#include "kda_ssm.h"
#include "kda_tile.h"

#ifndef KDA_SSM_DK
#error "compile with -DKDA_SSM_DK=32, 64 or 128"
#endif

namespace kda {
namespace {

constexpr int DK = KDA_SSM_DK;
constexpr int Q = kSsmChunk;
constexpr int kKeySteps = DK / 32;      // matrix steps of 32 over the keys
constexpr int kKeyTiles = DK / 16;
constexpr int kWaves = 4;               // per workgroup
constexpr int kMostTerms = 3;
constexpr int kMinSegment = 256;        // tokens

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------------------------
// workspace
// ---------------------------------------------------------------------------

// What ssm_keys leaves of a chunk and group: fragments of 64 lanes x 16 bytes.
struct Keys {
  u32x4 b[kMostTerms][kKeyTiles][2][kWave];   // rows: 16 keys; 32 tokens
  u32x4 c[kMostTerms][4][kKeySteps][kWave];   // rows: 16 tokens; 32 keys in the accumulators' order
  f32x4 pairs[4][2][2][kWave];                // rows: 16 tokens t; 32 tokens s; C_t.B_s
};
static_assert(sizeof(Keys) == 4 * (192 * DK + 4096), "KDA_SSM_WORKSPACE");

struct Plan {
  SsmArgs a;
  Keys* keys;           // [chunk slot][H]
  float* windows;       // [B][K-1][C], as they were
  float* states;        // [segment slot][HV][DK][DV]: what a segment adds, then the state before it
  float* decays;        // [segment slot][HV]
  int32_t segment;      // tokens per segment, 0: not split
  int32_t units;        // segment slots, or B
};

// Requests' chunks (or segments) are numbered through: request b's begin at
// slot(b) = t0 / length + b, which leaves each of them enough.
struct Unit {
  int b, i;
};

__device__ __forceinline__ Unit find_unit(const SsmArgs& a, int slot, int length) {
  int lo = 0, hi = a.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (request_range(a, mid).t0 / length + mid <= slot) lo = mid;
    else hi = mid - 1;
  }
  return {lo, slot - (request_range(a, lo).t0 / length + lo)};
}

// ---------------------------------------------------------------------------
// bf16 terms
// ---------------------------------------------------------------------------

__device__ __forceinline__ uint32_t high_halves(float lo, float hi) {
  return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}
__device__ __forceinline__ float truncated(float x) { return __uint_as_float(__float_as_uint(x) & 0xffff0000u); }

// Eight values as N bf16 terms.  The last of two terms is rounded to nearest;
// the last of three holds all bits that are left.
template <int N>
__device__ __forceinline__ void split(const float (&x)[8], u32x4 (&term)[N]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float x0 = x[2 * e], x1 = x[2 * e + 1];
    term[0][e] = high_halves(x0, x1);
    const float r0 = x0 - truncated(x0), r1 = x1 - truncated(x1);
    if constexpr (N == 2) {
      term[1][e] = f32x2_to_bf16x2_rne(r0, r1);
    } else {
      term[1][e] = high_halves(r0, r1);
      term[2][e] = high_halves(r0 - truncated(r0), r1 - truncated(r1));
    }
  }
}

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                 0);
}

// c += a b in N terms each, small products first.
template <int N>
__device__ __forceinline__ f32x4 product(const u32x4 (&a)[N], const u32x4 (&b)[N], f32x4 c) {
  if constexpr (N == 3) {
    c = mfma(a[0], b[2], c);
    c = mfma(a[2], b[0], c);
    c = mfma(a[1], b[1], c);
  }
  c = mfma(a[0], b[1], c);
  c = mfma(a[1], b[0], c);
  return mfma(a[0], b[0], c);
}

// ---------------------------------------------------------------------------
// keys
// ---------------------------------------------------------------------------

// The workgroup of a request's first chunk keeps the old windows of its
// group's channels and sets the new ones; no other reads them.
template <bool BF16>
__device__ void set_windows(const Plan& p, const Range& range, int b, int slot, int h) {
  const SsmArgs& a = p.a;
  const int dv = (a.C - 2 * a.H * DK) / a.HV;
  const int mine = a.G * dv;
  for (int i = threadIdx.x; i < mine + 2 * DK; i += 256) {
    const int keys = a.HV * dv + h * DK;
    const int c = i < mine ? h * mine + i : (i < mine + DK ? keys + (i - mine) : keys + a.H * DK + (i - mine - DK));
    float* const win = a.conv_win + static_cast<int64_t>(slot) * (a.K - 1) * a.C + c;
    float* const kept = p.windows + static_cast<int64_t>(b) * (a.K - 1) * a.C + c;
    float x[kPast];
    for (int j = 0; j < a.K - 1; ++j) kept[static_cast<int64_t>(j) * a.C] = win[static_cast<int64_t>(j) * a.C];
    for (int j = 0; j < a.K - 1; ++j) {
      const int t = range.n - (a.K - 1) + j;
      x[j] = t >= 0 ? load_scalar<BF16>(a.xbc, (static_cast<int64_t>(range.t0) + t) * a.C + c)
                    : win[static_cast<int64_t>(a.K - 1 + t) * a.C];
    }
    for (int j = 0; j < a.K - 1; ++j) win[static_cast<int64_t>(j) * a.C] = x[j];
  }
}

template <bool BF16>
__global__ void __launch_bounds__(256) ssm_keys(Plan p) {
  const SsmArgs& a = p.a;
  constexpr int STRIDE = DK + 2;        // rows 8 apart start 16 banks apart
  __shared__ __attribute__((aligned(16))) float rows[2][Q][STRIDE];   // B, C
  const int h = blockIdx.x % a.H;
  const Unit u = find_unit(a, blockIdx.x / a.H, Q);
  const Range range = request_range(a, u.b);
  const int slot = request_slot(a, u.b);
  if (slot < 0 || u.i < 0 || static_cast<int64_t>(u.i) * Q >= range.n) return;
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int begin = u.i * Q, valid = min(Q, range.n - begin);

  // a channel per thread, over all tokens or a part of them
  {
    constexpr int PARTS = 256 / (2 * DK), TOKENS = Q / PARTS;
    const int i = tid % (2 * DK), part = tid / (2 * DK);
    const int which = i / DK, k = i % DK;
    const int c = a.C - 2 * a.H * DK + which * a.H * DK + h * DK + k;
    Taps taps;
    taps.load(a, c);
    float past[kPast];
#pragma unroll
    for (int j = 0; j < kPast; ++j) {
      const int t = begin + part * TOKENS - kPast + j;      // of the request
      float x = 0.0f;
      if (t >= 0) {
        if (t < range.n) x = load_scalar<BF16>(a.xbc, (static_cast<int64_t>(range.t0) + t) * a.C + c);
      } else if (a.K - 1 + t >= 0) {
        x = a.conv_win[(static_cast<int64_t>(slot) * (a.K - 1) + a.K - 1 + t) * a.C + c];
      }
      past[j] = x;
    }
    const int64_t at = (static_cast<int64_t>(range.t0) + begin) * a.C + c;
#pragma unroll 16
    for (int j = 0; j < TOKENS; ++j) {
      const int t = part * TOKENS + j;
      const float x = load_scalar<BF16>(a.xbc, at + static_cast<int64_t>(min(t, valid - 1)) * a.C);
      const float y = silu_f(taps.dot(a.K, past[0], past[1], past[2], x));
      past[0] = past[1];
      past[1] = past[2];
      past[2] = x;
      rows[which][t][k] = t < valid ? y : 0.0f;
    }
  }
  __syncthreads();
  if (u.i == 0) set_windows<BF16>(p, range, u.b, slot, h);

  Keys& out = p.keys[(static_cast<int64_t>(range.t0 / Q) + u.b + u.i) * a.H + h];
  const int col = lane % 16, quad = lane / 16;
#pragma unroll
  for (int f = 0; f < kKeyTiles * 2 / kWaves; ++f) {
    const int tile = (f * kWaves + wave) / 2, step = (f * kWaves + wave) % 2;
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = rows[0][step * 32 + quad * 8 + j][tile * 16 + col];
    u32x4 term[kMostTerms];
    split(x, term);
#pragma unroll
    for (int n = 0; n < kMostTerms; ++n) out.b[n][tile][step][lane] = term[n];
  }
  f32x4 pairs[4];
#pragma unroll
  for (int st = 0; st < 4; ++st) pairs[st] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int step = 0; step < kKeySteps; ++step) {
    // 32 keys in the accumulators' order: four of each of two tiles
    auto fragment = [&](const float (&row)[STRIDE], u32x4 (&term)[kMostTerms]) {
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = row[step * 32 + (j / 4) * 16 + quad * 4 + j % 4];
      split(x, term);
    };
    u32x4 c[kMostTerms];
    fragment(rows[1][wave * 16 + col], c);
#pragma unroll
    for (int n = 0; n < kMostTerms; ++n) out.c[n][wave][step][lane] = c[n];
#pragma unroll
    for (int st = 0; st < 4; ++st) {
      if (st > wave) break;
      u32x4 b[kMostTerms];
      fragment(rows[0][st * 16 + col], b);
      pairs[st] = product(c, b, pairs[st]);
    }
  }
  // rows t, columns s -> operand order, through LDS
  __syncthreads();
  constexpr int PSTRIDE = Q + 4;
  float* const square = &rows[0][0][0];
  static_assert(Q * PSTRIDE <= 2 * Q * STRIDE, "the pairs fit where B and C were");
#pragma unroll
  for (int st = 0; st < 4; ++st)
#pragma unroll
    for (int i = 0; i < 4; ++i) square[(wave * 16 + quad * 4 + i) * PSTRIDE + st * 16 + col] = pairs[st][i];
  __syncthreads();
#pragma unroll
  for (int step = 0; step < 2; ++step)
#pragma unroll
    for (int half = 0; half < 2; ++half)
      out.pairs[wave][step][half][lane] =
          *reinterpret_cast<const f32x4*>(square + (wave * 16 + col) * PSTRIDE + step * 32 + quad * 8 + half * 4);
}

// ---------------------------------------------------------------------------
// scan
// ---------------------------------------------------------------------------

enum Mode { kWhole, kSegment, kJoined };

// NT values per lane of one row of x: adjacent columns.
template <int NT, bool BF16>
__device__ __forceinline__ void load_row(const void* base, int64_t at, float (&x)[NT]) {
  if constexpr (BF16) {
    const uint16_t* const p = static_cast<const uint16_t*>(base) + at;
    if constexpr (NT == 4) {
      const u32x2 w = *reinterpret_cast<const u32x2*>(p);
      x[0] = bf16_to_f32(w.x & 0xffffu);
      x[1] = __uint_as_float(w.x & 0xffff0000u);
      x[2] = bf16_to_f32(w.y & 0xffffu);
      x[3] = __uint_as_float(w.y & 0xffff0000u);
    } else {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
      x[0] = bf16_to_f32(w & 0xffffu);
      x[1] = __uint_as_float(w & 0xffff0000u);
    }
  } else {
    const float* const p = static_cast<const float*>(base) + at;
    if constexpr (NT == 4) {
      const f32x4 w = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
      for (int n = 0; n < 4; ++n) x[n] = w[n];
    } else {
      const float2 w = *reinterpret_cast<const float2*>(p);
      x[0] = w.x;
      x[1] = w.y;
    }
  }
}

template <int NT, bool BF16>
__device__ __forceinline__ void store_row(void* base, int64_t at, const float (&x)[NT]) {
#pragma unroll
  for (int n = 0; n < NT; n += 2) store_pair<BF16>(base, at + n, x[n], x[n + 1]);
}

template <int NT, bool BF16, int TY, int TS, int MODE>
__global__ void __launch_bounds__(256, 1) ssm_scan(Plan p, bool state_bf16, bool v_first) {
  const SsmArgs& a = p.a;
  constexpr int COLS = NT * 16;
  __shared__ __attribute__((aligned(16))) float sums[kWaves][3][Q];   // c in two parts (base 2), step
  const int dv = (a.C - 2 * a.H * DK) / a.HV;
  const int slabs = dv / COLS;
  const int waves = a.HV * slabs, blocks = (waves + kWaves - 1) / kWaves;

  // workgroups of a unit share its keys: on one XCD, where there are units
  // for all of them
  int unit, block;
  if (p.units >= kXcds) {
    const int xcd = blockIdx.x % kXcds, i = blockIdx.x / kXcds;
    unit = i / blocks * kXcds + xcd;
    block = i % blocks;
  } else {
    unit = blockIdx.x / blocks;
    block = blockIdx.x % blocks;
  }
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int w = block * kWaves + wave;
  if (unit >= p.units || w >= waves) return;
  const int hv = w / slabs, slab = w % slabs;
  Unit u = {unit, 0};
  if constexpr (MODE != kWhole) u = find_unit(a, unit, p.segment);
  const Range range = request_range(a, u.b);
  const int slot = request_slot(a, u.b);
  // tokens begin .. end - 1 of the request
  const int64_t wide_begin = MODE == kWhole ? 0 : static_cast<int64_t>(u.i) * p.segment;
  if (u.i < 0 || wide_begin >= range.n) return;
  const int begin = static_cast<int>(wide_begin);
  const int end = MODE == kWhole || range.n - begin < p.segment ? range.n : begin + p.segment;
  const int col = lane % 16, quad = lane / 16;
  const int column = hv * dv + slab * COLS + col * NT;      // the lane's first column: of out, and channel of x
  const int64_t out_row = static_cast<int64_t>(a.HV) * dv;
  if (slot < 0) {
    if constexpr (MODE != kSegment) {
      const float zero[NT] = {};
      for (int t = begin + quad; t < end; t += 4)
        store_row<NT, BF16>(a.out, (static_cast<int64_t>(range.t0) + t) * out_row + column, zero);
    }
    return;
  }

  // state tile: keys kt * 16 + quad * 4 + i, columns col * NT + n
  f32x4 S[kKeyTiles][NT];
  const int64_t tile = (static_cast<int64_t>(slot) * a.HV + hv) * DK * dv;
  const int vcol = slab * COLS + col * NT;
  const int64_t here = static_cast<int64_t>(range.t0 / (MODE == kWhole ? 1 : p.segment)) + u.b + u.i;
  float* const kept = MODE == kWhole ? nullptr : p.states + (here * a.HV + hv) * DK * dv;
  if constexpr (MODE == kWhole) {
#pragma unroll
    for (int kt = 0; kt < kKeyTiles; ++kt)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int k = kt * 16 + quad * 4 + i;
          const int64_t at = tile + (v_first ? static_cast<int64_t>(vcol + n) * DK + k
                                             : static_cast<int64_t>(k) * dv + vcol + n);
          S[kt][n][i] = state_bf16 ? load_scalar<true>(a.state_pool, at) : load_scalar<false>(a.state_pool, at);
        }
  } else {
#pragma unroll
    for (int kt = 0; kt < kKeyTiles; ++kt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x[NT] = {};
        if constexpr (MODE == kJoined)
          load_row<NT, false>(kept, static_cast<int64_t>(kt * 16 + quad * 4 + i) * dv + vcol, x);
#pragma unroll
        for (int n = 0; n < NT; ++n) S[kt][n][i] = x[n];
      }
  }

  Taps taps[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) taps[n].load(a, column + n);
  const float amp = exp_f(a.a_log[hv]), bias = a.dt_bias[hv];
  const float skip = a.d_skip != nullptr ? a.d_skip[hv] : 0.0f;
  const int h = hv / a.G;
  const int64_t first_key = static_cast<int64_t>(range.t0 / Q) + u.b;
  float* const hi = sums[wave][0];
  float* const lo = sums[wave][1];
  float* const steps = sums[wave][2];
  double gone = 0.0;                    // log2 of the segment's decay

  for (int t0 = begin; t0 < end; t0 += Q) {
    const int valid = min(Q, end - t0);
    const Keys& keys = p.keys[(first_key + t0 / Q) * a.H + h];
    // steps and the running sum of the decays, one token per lane
    double c;
    {
      const int64_t t = static_cast<int64_t>(range.t0) + t0 + min(lane, valid - 1);
      const float step = lane < valid ? softplus_f(a.dt[t * a.HV + hv] + bias) : 0.0f;
      c = static_cast<double>(step) * static_cast<double>(-amp) * 1.4426950408889634;
#pragma unroll
      for (int d = 1; d < kWave; d *= 2) {
        const double before = __shfl_up(c, d);
        if (lane >= d) c += before;
      }
      const float part = static_cast<float>(c);
      __builtin_amdgcn_wave_barrier();
      hi[lane] = part;
      lo[lane] = static_cast<float>(c - static_cast<double>(part));
      steps[lane] = step;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
    const double total = __shfl(c, kWave - 1);
    gone += total;
    const float total_hi = static_cast<float>(total);
    const float total_lo = static_cast<float>(total - static_cast<double>(total_hi));

    f32x4 y[4][NT];
    if constexpr (MODE != kSegment) {
#pragma unroll
      for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int n = 0; n < NT; ++n) y[mt][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      // C^T S0
#pragma unroll
      for (int step = 0; step < kKeySteps; ++step) {
        u32x4 s[NT][TY];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float x[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = S[2 * step + j / 4][n][j % 4];
          split(x, s[n]);
        }
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
          u32x4 ck[TY];
#pragma unroll
          for (int m = 0; m < TY; ++m) ck[m] = keys.c[m][mt][step][lane];
#pragma unroll
          for (int n = 0; n < NT; ++n) y[mt][n] = product(ck, s[n], y[mt][n]);
        }
      }
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) {
        const f32x4 ch = *reinterpret_cast<const f32x4*>(hi + mt * 16 + quad * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float f = __builtin_amdgcn_exp2f(ch[i]);
#pragma unroll
          for (int n = 0; n < NT; ++n) y[mt][n][i] *= f;
        }
      }
    }
    const bool update = MODE != kJoined || t0 + Q < end;     // a joined segment's last state is not used
    {
      const float f = __builtin_amdgcn_exp2f(total_hi);
#pragma unroll
      for (int kt = 0; kt < kKeyTiles; ++kt)
#pragma unroll
        for (int n = 0; n < NT; ++n) S[kt][n] *= f;
    }

#pragma unroll
    for (int step = 0; step < 2; ++step) {
      const int first = step * 32 + quad * 8;       // the lane's eight tokens of the chunk
      if (step * 32 >= valid) break;
      float x[8][NT];
      {
        float in[8 + kPast][NT];
#pragma unroll
        for (int j = 0; j < 8 + kPast; ++j) {
          const int t = min(max(t0 + first + j - kPast, 0), end - 1);
          load_row<NT, BF16>(a.xbc, (static_cast<int64_t>(range.t0) + t) * a.C + column, in[j]);
        }
        if (t0 == 0 && step == 0) {                 // the window of before
#pragma unroll
          for (int j = 0; j < kPast; ++j) {
            const int r = a.K - 1 - kPast + j;
            if (quad == 0) {
              if (r >= 0)
                load_row<NT, false>(p.windows, (static_cast<int64_t>(u.b) * (a.K - 1) + r) * a.C + column, in[j]);
            }
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const float z = silu_f(taps[n].dot(a.K, in[j][n], in[j + 1][n], in[j + 2][n], in[j + 3][n]));
            x[j][n] = first + j < valid ? z : 0.0f;
          }
      }
      const f32x4 h0 = *reinterpret_cast<const f32x4*>(hi + first), h1 = *reinterpret_cast<const f32x4*>(hi + first + 4);
      const f32x4 l0 = *reinterpret_cast<const f32x4*>(lo + first), l1 = *reinterpret_cast<const f32x4*>(lo + first + 4);
      const f32x4 d0 = *reinterpret_cast<const f32x4*>(steps + first);
      const f32x4 d1 = *reinterpret_cast<const f32x4*>(steps + first + 4);
      if constexpr (MODE != kSegment) {
        u32x4 xs[NT][TY];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = x[j][n];
          split(v, xs[n]);
        }
#pragma unroll
        for (int mt = 2 * step; mt < 4; ++mt) {
          const int t = mt * 16 + col;
          const float th = hi[t], tl = lo[t];
          const f32x4 p0 = keys.pairs[mt][step][0][lane], p1 = keys.pairs[mt][step][1][lane];
          float m[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float ch = j < 4 ? h0[j % 4] : h1[j % 4], cl = j < 4 ? l0[j % 4] : l1[j % 4];
            const float pair = (j < 4 ? p0[j % 4] : p1[j % 4]) * (j < 4 ? d0[j % 4] : d1[j % 4]);
            const float f = pair * __builtin_amdgcn_exp2f((th - ch) + (tl - cl));
            m[j] = first + j < t ? f : (first + j == t ? pair + skip : 0.0f);
          }
          u32x4 ms[TY];
          split(m, ms);
#pragma unroll
          for (int n = 0; n < NT; ++n) y[mt][n] = product(ms, xs[n], y[mt][n]);
        }
      }
      if (update) {
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float ch = j < 4 ? h0[j % 4] : h1[j % 4], cl = j < 4 ? l0[j % 4] : l1[j % 4];
          f[j] = __builtin_amdgcn_exp2f((total_hi - ch) + (total_lo - cl)) * (j < 4 ? d0[j % 4] : d1[j % 4]);
        }
        u32x4 xs[NT][TS];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = x[j][n] * f[j];
          split(v, xs[n]);
        }
#pragma unroll
        for (int kt = 0; kt < kKeyTiles; ++kt) {
          u32x4 bk[TS];
#pragma unroll
          for (int m = 0; m < TS; ++m) bk[m] = keys.b[m][kt][step][lane];
#pragma unroll
          for (int n = 0; n < NT; ++n) S[kt][n] = product(bk, xs[n], S[kt][n]);
        }
      }
    }
    if constexpr (MODE != kSegment) {
#pragma unroll
      for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = mt * 16 + quad * 4 + i;
          float o[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n) o[n] = y[mt][n][i];
          if (t < valid)
            store_row<NT, BF16>(a.out, (static_cast<int64_t>(range.t0) + t0 + t) * out_row + column, o);
        }
    }
  }

  if constexpr (MODE == kWhole) {
#pragma unroll
    for (int kt = 0; kt < kKeyTiles; ++kt)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int k = kt * 16 + quad * 4 + i;
          const int64_t at = tile + (v_first ? static_cast<int64_t>(vcol + n) * DK + k
                                             : static_cast<int64_t>(k) * dv + vcol + n);
          if (state_bf16) store_scalar<true>(a.state_pool, at, S[kt][n][i]);
          else store_scalar<false>(a.state_pool, at, S[kt][n][i]);
        }
  } else if constexpr (MODE == kSegment) {
#pragma unroll
    for (int kt = 0; kt < kKeyTiles; ++kt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float o[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) o[n] = S[kt][n][i];
        store_row<NT, false>(kept, static_cast<int64_t>(kt * 16 + quad * 4 + i) * dv + vcol, o);
      }
    if (slab == 0 && lane == 0) p.decays[here * a.HV + hv] = static_cast<float>(exp2(gone));
  }
}

// The states before the segments of a request, and after its last: four
// adjacent columns per thread.
__global__ void __launch_bounds__(256) ssm_join(Plan p, bool state_bf16, bool v_first) {
  const SsmArgs& a = p.a;
  const int dv = (a.C - 2 * a.H * DK) / a.HV;
  const int parts = DK * dv / 1024;
  const int part = blockIdx.x % parts, head = blockIdx.x / parts;
  const int hv = head % a.HV, b = head / a.HV;
  const Range range = request_range(a, b);
  const int slot = request_slot(a, b);
  if (slot < 0 || range.n == 0) return;
  const int at = (part * 256 + threadIdx.x) * 4;
  const int k = at / dv, v = at % dv;
  const int64_t tile = (static_cast<int64_t>(slot) * a.HV + hv) * DK * dv;
  f32x4 s;
  int64_t where[4];
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    where[n] = tile + (v_first ? static_cast<int64_t>(v + n) * DK + k : static_cast<int64_t>(k) * dv + v + n);
    s[n] = state_bf16 ? load_scalar<true>(a.state_pool, where[n]) : load_scalar<false>(a.state_pool, where[n]);
  }
  const int64_t first = static_cast<int64_t>(range.t0 / p.segment) + b;
  const int segments = (range.n - 1) / p.segment + 1;
  const int64_t stride = static_cast<int64_t>(a.HV) * DK * dv;
  float* const states = p.states + first * stride + static_cast<int64_t>(hv) * DK * dv + at;
  const float* const decays = p.decays + first * a.HV + hv;
#pragma unroll 4
  for (int i = 0; i < segments; ++i) {
    f32x4* const state = reinterpret_cast<f32x4*>(states + i * stride);
    const f32x4 own = *state;
    const float decay = decays[static_cast<int64_t>(i) * a.HV];
    *state = s;
#pragma unroll
    for (int n = 0; n < 4; ++n) s[n] = fmaf(decay, s[n], own[n]);
  }
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    if (state_bf16) store_scalar<true>(a.state_pool, where[n], s[n]);
    else store_scalar<false>(a.state_pool, where[n], s[n]);
  }
}

// ---------------------------------------------------------------------------
// launch
// ---------------------------------------------------------------------------

template <int NT, bool BF16, int TY, int TS, int MODE>
hipError_t scan(const Plan& plan, int dv, bool state_bf16, bool v_first, hipStream_t stream) {
  const int64_t blocks = (static_cast<int64_t>(plan.a.HV) * (dv / (NT * 16)) + kWaves - 1) / kWaves;
  const int64_t units = plan.units >= kXcds ? (plan.units + kXcds - 1) / kXcds * kXcds : plan.units;
  void* kargs[] = {const_cast<Plan*>(&plan), &state_bf16, &v_first};
  return hipLaunchKernel(reinterpret_cast<const void*>(&ssm_scan<NT, BF16, TY, TS, MODE>),
                         dim3(static_cast<uint32_t>(units * blocks)), dim3(kWaves * kWave), kargs, 0, stream);
}

template <int NT, bool BF16, int TY, int TS>
hipError_t scans(const Plan& plan, int dv, bool state_bf16, bool v_first, hipStream_t stream) {
  if (plan.segment == 0) return scan<NT, BF16, TY, TS, kWhole>(plan, dv, state_bf16, v_first, stream);
  hipError_t rc = scan<NT, BF16, TY, TS, kSegment>(plan, dv, state_bf16, v_first, stream);
  if (rc != hipSuccess) return rc;
  void* kargs[] = {const_cast<Plan*>(&plan), &state_bf16, &v_first};
  const int64_t blocks = static_cast<int64_t>(plan.a.B) * plan.a.HV * (DK * dv / 1024);
  rc = hipLaunchKernel(reinterpret_cast<const void*>(&ssm_join), dim3(static_cast<uint32_t>(blocks)), dim3(256), kargs,
                       0, stream);
  if (rc != hipSuccess) return rc;
  // the state of a joined segment only reaches its outputs
  return scan<NT, BF16, TY, TY, kJoined>(plan, dv, state_bf16, v_first, stream);
}

template <int NT>
hipError_t scans(const Plan& plan, int dv, bool bf16, bool state_bf16, bool v_first, hipStream_t stream) {
  if (!bf16) return scans<NT, false, 3, 3>(plan, dv, state_bf16, v_first, stream);
  if (state_bf16) return scans<NT, true, 2, 2>(plan, dv, state_bf16, v_first, stream);
  return scans<NT, true, 2, 3>(plan, dv, state_bf16, v_first, stream);
}

}  // namespace

template <>
int launch_ssm_prefill_dk<DK>(const SsmArgs& args, int dv, bool bf16, bool state_bf16, int state_layout,
                              hipStream_t stream) {
  Plan plan{};
  plan.a = args;
  const int64_t chunks = static_cast<int64_t>(args.T) / Q + args.B;
  plan.keys = reinterpret_cast<Keys*>(args.workspace);
  plan.windows = reinterpret_cast<float*>(plan.keys + chunks * args.H);
  plan.states = plan.windows + static_cast<int64_t>(args.B) * (args.K - 1) * args.C;
  const int64_t waves = static_cast<int64_t>(args.HV) * (dv > 64 ? 2 : 1);
  plan.units = args.B;
  const int64_t most = KDA_SSM_SPLIT / waves;       // segments that the workspace has room for, beyond one a request
  if (args.B * waves < 1024 && most >= 2) {
    int64_t length = (args.T + most - 1) / most;
    length = (length + Q - 1) / Q * Q;
    if (length < kMinSegment) length = kMinSegment;
    if (length < args.T) {
      plan.segment = static_cast<int32_t>(length);
      plan.units = static_cast<int32_t>(args.T / length + args.B);
      plan.decays = plan.states + static_cast<int64_t>(plan.units) * args.HV * DK * dv;
    }
  }
  void* kargs[] = {&plan};
  const uint32_t blocks = static_cast<uint32_t>(chunks * args.H);
  hipError_t rc = hipLaunchKernel(bf16 ? reinterpret_cast<const void*>(&ssm_keys<true>)
                                       : reinterpret_cast<const void*>(&ssm_keys<false>),
                                  dim3(blocks), dim3(256), kargs, 0, stream);
  if (rc != hipSuccess) return KDA_ERR_LAUNCH;
  const bool v_first = state_layout == KDA_STATE_V_FIRST;
  rc = dv == 32 ? scans<2>(plan, dv, bf16, state_bf16, v_first, stream)
                : scans<4>(plan, dv, bf16, state_bf16, v_first, stream);
  return rc == hipSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}

}  // namespace kda
