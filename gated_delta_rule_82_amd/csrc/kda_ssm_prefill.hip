// kda_ssm_prefill.hip - the selective state space scan over whole prompts
// (kda_ssm_prefill), in chunks of 32 tokens on the matrix cores.
//
// With g_t = -exp(a_log) step_t and c_t its running sum since the chunk's
// start, S0 the state before the chunk and x', B, C the convolved channels:
//     y_t = exp(c_t) C_t^T S0 + sum_{s<=t} (C_t.B_s) exp(c_t - c_s) step_s x'_s + d_skip x'_t
//     S   = exp(c_last) S0 + sum_s B_s (exp(c_last - c_s) step_s x'_s)^T
// Every factor is at most one; what the scan does not form is C.B.
//
// ssm_keys, one workgroup per (chunk, group): convolves B and C, which all
// heads of the group share, and leaves them and C.B in the order in which the
// matrix instructions take them, B and C in bf16 terms.  Further workgroups
// make the steps and decays of 32 tokens and 32 heads, and set the windows.
// ssm_scan, one wave per (request, value head, 32 value columns): walks the
// chunks with the state in its accumulators.  The accumulators of two 16-key
// tiles are the instruction's other operand for 32 keys in the order that
// ssm_keys stores C in, so no value moves between lanes.  Four waves of a group
// share the operands through LDS, and those of a head its factors of C.B; a
// wave convolves its own columns of x.  Two barriers per chunk: behind one the
// outputs, behind the other the update.
// Where a batch has few heads for the chip, requests are split into segments:
// ssm_scan (kSegment) runs all segments from a zero state, ssm_join passes
// the states on, and ssm_scan (kJoined) runs the segments from there.
//
// Precision: an fp32 value is the sum of three bf16 terms, 8 bits each, taken
// by truncation, so that no term leaves the value's range.  Products of three
// terms each are good to 2^-20 of what is added up (six matrix instructions;
// measured 1.3e-7 on the state), of two to 2^-13 (three): the state takes three
// for an fp32 pool or fp32 activations, and what only reaches bf16 outputs or
// a bf16 pool takes two.  c is summed in fp64 and kept in two fp32 parts:
// differences of large sums are what counts.
//
// Bound: vector instructions (splitting the state into terms every 32 tokens,
// the convolution with its SiLU) and the clock under them; 8 x 2048 tokens over
// 96 heads of 128 columns, bf16 pool: 540 us, of which ssm_keys 58 and ssm_scan
// 478, vector units busy 63% of the cycles and matrix units 33%.  16384 tokens
// over 32 heads of 64 columns: 170 us (keys 12, segments 60, join 15, joined 85).

#include <hip/hip_runtime.h>

#include <cstdint>

#include "kda.h"
#include "kda_device.h"
#include "kda_internal.h"
#include "kda_ssm.h"
#include "kda_tile.h"

#if !defined(KDA_SSM_DK) || !defined(KDA_SSM_DV)
#error "compile with -DKDA_SSM_DK and -DKDA_SSM_DV, each 32, 64 or 128"
#endif

namespace kda {
namespace {

constexpr int DK = KDA_SSM_DK;
constexpr int DV = KDA_SSM_DV;
constexpr int Q = kSsmChunk;
constexpr int kKeySteps = DK / 32;      // matrix steps of 32 over the keys
constexpr int kKeyTiles = DK / 16;
constexpr int kMostTerms = 3;
constexpr int kMinSegment = 64;         // tokens; KDA_SSM_WORKSPACE

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------------------------
// workspace
// ---------------------------------------------------------------------------

// What ssm_keys leaves of 32 tokens and a group: fragments of 64 lanes x 16
// bytes.
struct Keys {
  u32x4 b[kMostTerms][kKeyTiles][kWave];      // rows: 16 keys; 32 tokens
  u32x4 c[kMostTerms][2][kKeySteps][kWave];   // rows: 16 tokens; 32 keys in the accumulators' order
  f32x4 pairs[2][2][kWave];                   // rows: 16 tokens t; 32 tokens s; C_t.B_s
};
static_assert(sizeof(Keys) == 4 * (96 * DK + 1024), "KDA_SSM_WORKSPACE");

// ... and of 32 tokens and a head.  c is the running sum of log2 exp(g).
struct Steps {
  float hi[Q], lo[Q];                         // c in two parts
  float decay[Q];                             // exp(g_t)
  float from[Q];                              // exp(c_t)
  float step[Q];
};
constexpr int kSteps = sizeof(Steps) / 4;
static_assert(kSteps == 160, "KDA_SSM_WORKSPACE");

struct Plan {
  SsmArgs a;
  Keys* keys;           // [chunk slot][H]
  Steps* steps;         // [chunk slot][HV]
  float* windows;       // [B][K-1][C], as they were
  float* states;        // [segment slot][HV][DK][DV]: what a segment adds, then the state before it
  float* decays;        // [segment slot][HV]
  int32_t segment;      // tokens per segment, 0: not split
  int32_t units;        // segment slots, or B
  uint32_t key_blocks, window_blocks, step_blocks;    // workgroups of ssm_keys
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

// L values as N bf16 terms.  The last of two terms is rounded to nearest; the
// last of three holds all bits that are left.
template <int N, int L, typename T>
__device__ __forceinline__ void split(const float (&x)[L], T (&term)[N]) {
  static_assert(sizeof(T) == 2 * L, "pairs of bf16");
#pragma unroll
  for (int e = 0; e < L / 2; ++e) {
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

// c[i][n] += a[i] b[n] in N terms each, small products first; term by term over
// all of c, so that an instruction does not wait for the one before it.
template <int M, int N, int L>
__device__ __forceinline__ void products(const u32x4 (&a)[M][N], const u32x4 (&b)[L][N], f32x4 (&c)[M][L]) {
  constexpr int kOrder[6][2] = {{0, 2}, {2, 0}, {1, 1}, {0, 1}, {1, 0}, {0, 0}};
#pragma unroll
  for (int o = N == 3 ? 0 : 3; o < 6; ++o)
#pragma unroll
    for (int i = 0; i < M; ++i)
#pragma unroll
      for (int n = 0; n < L; ++n) c[i][n] = mfma(a[i][kOrder[o][0]], b[n][kOrder[o][1]], c[i][n]);
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

// The new window of request b's channel c; the workspace keeps the old one if
// `keep`.
template <bool BF16>
__device__ __forceinline__ void set_window(const Plan& p, const Range& range, int b, int slot, int c, bool keep) {
  const SsmArgs& a = p.a;
  float* const win = a.conv_win + static_cast<int64_t>(slot) * (a.K - 1) * a.C + c;
  float old[kPast], next[kPast];
#pragma unroll
  for (int j = 0; j < kPast; ++j) {
    if (j >= a.K - 1) continue;
    const int t = range.n - (a.K - 1) + j;      // of the request; below zero: of the old window
    old[j] = win[static_cast<int64_t>(j) * a.C];
    next[j] = t >= 0 ? load_scalar<BF16>(a.xbc, (static_cast<int64_t>(range.t0) + t) * a.C + c)
                     : win[static_cast<int64_t>(a.K - 1 + t) * a.C];
  }
#pragma unroll
  for (int j = 0; j < kPast; ++j) {
    if (j >= a.K - 1) continue;
    if (keep) p.windows[(static_cast<int64_t>(b) * (a.K - 1) + j) * a.C + c] = old[j];
    win[static_cast<int64_t>(j) * a.C] = next[j];
  }
}

template <int CTRL, int ROWS>
__device__ __forceinline__ double add_from(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(u), CTRL, ROWS, 0xf, true);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(u >> 32), CTRL, ROWS, 0xf, true);
  return x + __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

// Sum over this lane and those before it in its half of the wave: within rows
// of 16, then the first row's last lane to the second.
__device__ __forceinline__ double running_sum(double x) {
  x = add_from<0x111, 0xf>(x);
  x = add_from<0x112, 0xf>(x);
  x = add_from<0x114, 0xf>(x);
  x = add_from<0x118, 0xf>(x);
  return add_from<0x142, 0xa>(x);
}

// Steps of 32 tokens and 32 heads: read by rows of heads, a half wave per head.
constexpr int kHeads = 32;
__device__ __forceinline__ void set_steps(const Plan& p, int slot_at, int head0, float (&tile)[kHeads][Q + 1]) {
  const SsmArgs& a = p.a;
  const Unit u = find_unit(a, slot_at, Q);
  const Range range = request_range(a, u.b);
  if (request_slot(a, u.b) < 0 || u.i < 0 || static_cast<int64_t>(u.i) * Q >= range.n) return;
  const int valid = min(Q, range.n - u.i * Q);
  const int64_t first = static_cast<int64_t>(range.t0) + u.i * Q;
  const int lane = threadIdx.x % kHeads, part = threadIdx.x / kHeads;
#pragma unroll
  for (int t = part; t < Q; t += 256 / kHeads)
    tile[lane][t] = a.dt[(first + min(t, valid - 1)) * a.HV + min(head0 + lane, a.HV - 1)];
  constexpr int EACH = kHeads / (256 / Q);      // heads of a half wave
  float bias[EACH], amp[EACH];
#pragma unroll
  for (int e = 0; e < EACH; ++e) {
    const int hv = min(head0 + part * EACH + e, a.HV - 1);
    bias[e] = a.dt_bias[hv];
    amp[e] = a.a_log[hv];
  }
  __syncthreads();
  Steps* const to = p.steps + (static_cast<int64_t>(range.t0 / Q) + u.b + u.i) * a.HV + head0 + part * EACH;
  const int t = lane;
#pragma unroll
  for (int e = 0; e < EACH; ++e) {
    const float step = t < valid ? softplus_f(tile[part * EACH + e][t] + bias[e]) : 0.0f;
    // Without a step nothing decays, whatever a_log; a factor below 2^-10000
    // is zero all the same, and keeps the sums finite.  NaN stays NaN.
    const double rate = static_cast<double>(-exp_f(amp[e])) * 1.4426950408889634;
    const double wide = step * rate;
    const double g = step > 0.0f ? (wide < -1e4 ? -1e4 : wide) : 0.0;
    const double c = running_sum(g);
    const float high = static_cast<float>(c);
    if (head0 + part * EACH + e < a.HV) {
      to[e].hi[t] = high;
      to[e].lo[t] = static_cast<float>(c - static_cast<double>(high));
      to[e].decay[t] = __builtin_amdgcn_exp2f(static_cast<float>(g));
      to[e].from[t] = __builtin_amdgcn_exp2f(high);
      to[e].step[t] = step;
    }
  }
}

// TY terms of C, and of the pairs' operands; TS of B.
template <bool BF16, int TY, int TS>
__global__ void __launch_bounds__(256) ssm_keys(Plan p) {
  const SsmArgs& a = p.a;
  constexpr int STRIDE = DK + (DK == 32 ? 4 : 2);       // rows 8 apart start 16 or 32 banks apart
  __shared__ __attribute__((aligned(16))) float rows[2][Q][STRIDE];   // B, C
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int channels = a.C - 2 * a.H * DK;      // of x
  static_assert(sizeof(rows) >= sizeof(float) * kHeads * (Q + 1), "dt where B and C are otherwise");
  if (blockIdx.x >= p.key_blocks + p.window_blocks) {
    const int tiles = (a.HV + kHeads - 1) / kHeads;
    const int i = blockIdx.x - p.key_blocks - p.window_blocks;
    set_steps(p, i / tiles, i % tiles * kHeads, reinterpret_cast<float (&)[kHeads][Q + 1]>(rows));
    return;
  }
  if (blockIdx.x >= p.key_blocks) {
    // windows of x, which ssm_scan finds in the workspace
    const int blocks = (channels + 255) / 256;
    const int i = blockIdx.x - p.key_blocks, b = i / blocks, c = i % blocks * 256 + tid;
    const Range range = request_range(a, b);
    const int slot = request_slot(a, b);
    if (slot >= 0 && range.n > 0 && c < channels) set_window<BF16>(p, range, b, slot, c, true);
    return;
  }
  const int h = blockIdx.x % a.H;
  const Unit u = find_unit(a, blockIdx.x / a.H, Q);
  const Range range = request_range(a, u.b);
  const int slot = request_slot(a, u.b);
  if (slot < 0 || u.i < 0 || static_cast<int64_t>(u.i) * Q >= range.n) return;
  const int begin = u.i * Q, valid = min(Q, range.n - begin);

  // two adjacent channels per thread, over a part of the tokens
  {
    constexpr int PARTS = 256 / DK, TOKENS = Q / PARTS;
    const int i = tid % DK * 2, part = tid / DK;
    const int which = i / DK, k = i % DK;
    const int c = channels + which * a.H * DK + h * DK + k;
    Taps taps[2];
    load_taps(a, {c, c + 1}, taps);
    float in[TOKENS + kPast][2];
#pragma unroll
    for (int j = 0; j < TOKENS + kPast; ++j) {
      const int t = begin + part * TOKENS - kPast + j;      // of the request
      const int64_t at = (static_cast<int64_t>(range.t0) + min(max(t, 0), range.n - 1)) * a.C + c;
      if constexpr (BF16) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.xbc) + at);
        in[j][0] = bf16_to_f32(w & 0xffffu);
        in[j][1] = __uint_as_float(w & 0xffff0000u);
      } else {
        const float2 w = *reinterpret_cast<const float2*>(static_cast<const float*>(a.xbc) + at);
        in[j][0] = w.x;
        in[j][1] = w.y;
      }
    }
    if (begin == 0 && part * TOKENS < kPast) {              // the window of before
#pragma unroll
      for (int j = 0; j < kPast; ++j) {
        const int r = a.K - 1 - kPast + part * TOKENS + j;  // its row, if below the last
        if (part * TOKENS + j < kPast) {
#pragma unroll
          for (int n = 0; n < 2; ++n)
            in[j][n] = r >= 0 ? a.conv_win[(static_cast<int64_t>(slot) * (a.K - 1) + r) * a.C + c + n] : 0.0f;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < TOKENS; ++j) {
      const int t = part * TOKENS + j;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const float y = silu_f(taps[n].dot(a.K, in[j][n], in[j + 1][n], in[j + 2][n], in[j + 3][n]));
        rows[which][t][k + n] = t < valid ? y : 0.0f;
      }
    }
  }
  __syncthreads();
  if (u.i == 0 && tid < 2 * DK)         // this workgroup alone has read them
    set_window<BF16>(p, range, u.b, slot, channels + tid / DK * a.H * DK + h * DK + tid % DK, false);

  const int64_t here = static_cast<int64_t>(range.t0 / Q) + u.b + u.i;
  Keys& out = p.keys[here * a.H + h];
  const int col = lane % 16, quad = lane / 16;
  for (int tile = wave; tile < kKeyTiles; tile += 4) {
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = rows[0][quad * 8 + j][tile * 16 + col];
    u32x4 term[TS];
    split(x, term);
#pragma unroll
    for (int n = 0; n < TS; ++n) out.b[n][tile][lane] = term[n];
  }
  // C and the pairs: 16 tokens t and every other step over the keys per wave
  const int mt = wave % 2;
  f32x4 pairs[2];
#pragma unroll
  for (int st = 0; st < 2; ++st) pairs[st] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int step = wave / 2; step < kKeySteps; step += 2) {
    // 32 keys in the accumulators' order: four of each of two tiles
    auto fragment = [&](const float (&row)[STRIDE], u32x4 (&term)[TY]) {
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = row[step * 32 + (j / 4) * 16 + quad * 4 + j % 4];
      split(x, term);
    };
    u32x4 c[TY];
    fragment(rows[1][mt * 16 + col], c);
#pragma unroll
    for (int n = 0; n < TY; ++n) out.c[n][mt][step][lane] = c[n];
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      if (st > mt) break;
      u32x4 b[TY];
      fragment(rows[0][st * 16 + col], b);
      pairs[st] = product(c, b, pairs[st]);
    }
  }
  // rows t, columns s -> operand order, and the sum of both waves, through LDS
  constexpr int PSTRIDE = Q + 4;
  static_assert(sizeof(rows) >= sizeof(float) * 2 * Q * PSTRIDE, "the pairs where B and C were");
  auto& squares = reinterpret_cast<float (&)[2][Q][PSTRIDE]>(rows);
  __syncthreads();
#pragma unroll
  for (int st = 0; st < 2; ++st)
#pragma unroll
    for (int i = 0; i < 4; ++i) squares[wave / 2][mt * 16 + quad * 4 + i][st * 16 + col] = pairs[st][i];
  __syncthreads();
  {
    const int part = wave / 2, t = mt * 16 + col, s = quad * 8 + part * 4;
    out.pairs[mt][part][lane] = *reinterpret_cast<const f32x4*>(&squares[0][t][s]) +
                                *reinterpret_cast<const f32x4*>(&squares[1][t][s]);
  }
}

// ---------------------------------------------------------------------------
// scan
// ---------------------------------------------------------------------------

enum Mode { kWhole, kSegment, kJoined };

constexpr int NT = 2;                   // 16-column tiles of a wave; a lane's columns are adjacent
constexpr int kColumns = NT * 16;
constexpr int kSlabs = DV / kColumns;   // waves of a head
constexpr int kWaves = 4;               // of a workgroup, all of one group
constexpr int kThreads = kWaves * kWave;

// A workgroup's LDS: the chunk's operands, which its waves share.
template <int TY, int TS>
struct Shared {
  u32x4 b[TS][kKeyTiles][kWave];
  u32x4 c[TY][2][kKeySteps][kWave];
  u32x2 m[kWaves / kSlabs][TY][2][kWave][2];  // of a head: rows 16 tokens t; 32 tokens s
  Steps steps[kWaves][2];               // of this chunk and the next
};

// N pieces of 16 bytes, from memory to LDS by way of the threads' registers.
template <int N>
struct Staged {
  static constexpr int PER = (N + kThreads - 1) / kThreads;
  u32x4 w[PER];
  __device__ __forceinline__ void load(const u32x4* from) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int at = i * kThreads + static_cast<int>(threadIdx.x);
      if (N % kThreads == 0 || at < N) w[i] = from[at];
    }
  }
  __device__ __forceinline__ void store(u32x4* to) const {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int at = i * kThreads + static_cast<int>(threadIdx.x);
      if (N % kThreads == 0 || at < N) to[at] = w[i];
    }
  }
};

__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// A lane's inputs: tokens 8 quad + 0 .. 7 and the three before them, its two
// columns.
template <bool BF16>
struct Inputs {
  static constexpr int ROWS = 8 + kPast;
  uint32_t w[ROWS][BF16 ? 1 : 2];

  // Rows t0 - 3 .. t0 + valid - 1 of the request, through a resource of just
  // these: others read as zero.  Before the first token there are none.
  __device__ __forceinline__ void load(const SsmArgs& a, const Range& range, int t0, int valid, int quad, int column) {
    constexpr int E = BF16 ? 2 : 4;
    const int before = t0 > 0 ? kPast : 0;
    const int stride = a.C * E;
    const char* const base =
        static_cast<const char*>(a.xbc) + (static_cast<int64_t>(range.t0) + t0 - before) * a.C * E;
    const __amdgpu_buffer_rsrc_t r = tile_resource(const_cast<char*>(base), (valid + before) * stride);
    const int first = (quad * 8 - kPast + before) * stride + column * E;
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      const int at = first + j * stride;        // below zero: out of range as an unsigned offset
      if constexpr (BF16) {
        w[j][0] = __builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0);
      } else {
        const u32x2 x = __builtin_amdgcn_raw_buffer_load_b64(r, at, 0, 0);
        w[j][0] = x.x;
        w[j][1] = x.y;
      }
    }
  }
  __device__ __forceinline__ float get(int j, int n) const {
    if constexpr (BF16) return n == 0 ? __uint_as_float(w[j][0] << 16) : __uint_as_float(w[j][0] & 0xffff0000u);
    else return __uint_as_float(w[j][n]);
  }
};

// A wave's part of a state tile [DK][dv] or [dv][DK] at `tile`: keys
// kt * 16 + quad * 4 + i, columns v + n.
template <bool SBF16, bool VFIRST, bool STORE>
__device__ __forceinline__ void move_state(__amdgpu_buffer_rsrc_t tile, int quad, int v,
                                           f32x4 (&S)[kKeyTiles][NT]) {
  constexpr int E = SBF16 ? 2 : 4;
#pragma unroll
  for (int kt = 0; kt < kKeyTiles; ++kt) {
    if constexpr (VFIRST) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int at = ((v + n) * DK + kt * 16 + quad * 4) * E;
        float x[4];
        if constexpr (STORE) {
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = S[kt][n][i];
          StateIO<SBF16, 4>::store(tile, at, 0, x);
        } else {
          StateIO<SBF16, 4>::load(tile, at, 0, x);
#pragma unroll
          for (int i = 0; i < 4; ++i) S[kt][n][i] = x[i];
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = ((kt * 16 + quad * 4 + i) * DV + v) * E;
        if constexpr (STORE) {
          if constexpr (SBF16) {
            __builtin_amdgcn_raw_buffer_store_b32(f32x2_to_bf16x2_rne(S[kt][0][i], S[kt][1][i]), tile, at, 0, 0);
          } else {
            const u32x2 w = {__float_as_uint(S[kt][0][i]), __float_as_uint(S[kt][1][i])};
            __builtin_amdgcn_raw_buffer_store_b64(w, tile, at, 0, 0);
          }
        } else if constexpr (SBF16) {
          const uint32_t w = __builtin_amdgcn_raw_buffer_load_b32(tile, at, 0, 0);
          S[kt][0][i] = bf16_to_f32(w & 0xffffu);
          S[kt][1][i] = __uint_as_float(w & 0xffff0000u);
        } else {
          const u32x2 w = __builtin_amdgcn_raw_buffer_load_b64(tile, at, 0, 0);
          S[kt][0][i] = __uint_as_float(w.x);
          S[kt][1][i] = __uint_as_float(w.y);
        }
      }
    }
  }
}

template <bool STORE>
__device__ __forceinline__ void move_pool(__amdgpu_buffer_rsrc_t tile, bool state_bf16, bool v_first, int quad, int v,
                                          f32x4 (&S)[kKeyTiles][NT]) {
  if (state_bf16) {
    if (v_first) move_state<true, true, STORE>(tile, quad, v, S);
    else move_state<true, false, STORE>(tile, quad, v, S);
  } else {
    if (v_first) move_state<false, true, STORE>(tile, quad, v, S);
    else move_state<false, false, STORE>(tile, quad, v, S);
  }
}

// The lanes 16 quad + col whose token t = 16 mt + col is at or behind token
// 8 quad + j: constants, one per use.
__device__ __forceinline__ constexpr uint64_t lanes_from(int mt, int j) {
  uint64_t lanes = 0;
  for (int quad = 0; quad < 4; ++quad) {
    const int from = quad * 8 + j - mt * 16;
    const uint64_t row = from <= 0 ? 0xffffu : (from >= 16 ? 0u : 0xffffu << from & 0xffffu);
    lanes |= row << (16 * quad);
  }
  return lanes;
}

// Waves per SIMD, as their registers allow: 16384 tokens over 32 heads of 128
// keys need 240 with outputs; at dk = 64 three waves took the ragged fp32
// prompts from 122 to 111 us (with the shorter segments).
template <int MODE>
constexpr int kResident = MODE == kSegment || DK <= 64 ? 3 : 2;

// Half a fragment of M[t][s] = (C_t.B_s) exp(c_t - c_s) step_s, the lane's
// tokens t = 16 mt + col and s = 8 quad + 4 half + 0 .. 3 (mt and half are the
// wave's); zero for s > t.  The factors exp(c_t - c_s) are taken from the last
// s backwards, one exponential and then the decays in between; one where
// s >= t.
template <int TY>
__device__ __forceinline__ void decayed_pairs(const Steps& of, f32x4 pairs, float skip, int mt, int half, int lane,
                                              u32x2 (&m)[TY][2][kWave][2]) {
  const int t = mt * 16 + lane % 16, s = lane / 16 * 8 + half * 4;
  const f32x4 decay = *reinterpret_cast<const f32x4*>(of.decay + s), step = *reinterpret_cast<const f32x4*>(of.step + s);
  float f = __builtin_amdgcn_exp2f(fminf((of.hi[t] - of.hi[s + 3]) + (of.lo[t] - of.lo[s + 3]), 0.0f));
  auto lanes = [&](int j) {     // one of four constants
    const uint64_t first = half == 0 ? lanes_from(0, j) : lanes_from(0, 4 + j);
    const uint64_t second = half == 0 ? lanes_from(1, j) : lanes_from(1, 4 + j);
    return mt == 0 ? first : second;
  };
  float x[4];
#pragma unroll
  for (int j = 3; j >= 0; --j) {
    const uint64_t reached = lanes(j), passed = lanes(j + 1);   // s <= t, s < t
    if (j < 3) f *= __builtin_amdgcn_inverse_ballot_w64(passed) ? decay[j + 1] : 1.0f;
    const float own = __builtin_amdgcn_inverse_ballot_w64(reached & ~passed) ? skip : 0.0f;
    x[j] = __builtin_amdgcn_inverse_ballot_w64(reached) ? fmaf(pairs[j] * step[j], f, own) : 0.0f;
  }
  u32x2 term[TY];
  split<TY>(x, term);
#pragma unroll
  for (int n = 0; n < TY; ++n) m[n][mt][lane][half] = term[n];
}

template <bool BF16, bool FULL, int TY, int TS, int MODE>
__global__ void __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(kResident<MODE>, kResident<MODE>)))
ssm_scan(Plan p, bool state_bf16, bool v_first) {
  const SsmArgs& a = p.a;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  Shared<TY, TS>& sh = *reinterpret_cast<Shared<TY, TS>*>(lds);
  const int waves = a.G * kSlabs, blocks = (waves + kWaves - 1) / kWaves;    // of a group

  // the workgroups of a unit's group share its keys: on one XCD, where there
  // are groups for all of them
  const int groups = p.units * a.H;
  int group = blockIdx.x / blocks, block = blockIdx.x % blocks;
  if (groups >= kXcds) {
    const int i = blockIdx.x / kXcds;
    group = i / blocks * kXcds + blockIdx.x % kXcds;
    block = i % blocks;
    if (group >= groups) return;
  }
  const int unit = group / a.H, h = group % a.H;
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);    // a scalar
  Unit u = {unit, 0};
  if constexpr (MODE != kWhole) u = find_unit(a, unit, p.segment);
  const Range range = request_range(a, u.b);
  const int slot = request_slot(a, u.b);
  // tokens begin .. end - 1 of the request
  const int64_t wide_begin = MODE == kWhole ? 0 : static_cast<int64_t>(u.i) * p.segment;
  if (u.i < 0 || wide_begin >= range.n) return;
  const int begin = static_cast<int>(wide_begin);
  const int end = MODE == kWhole || range.n - begin < p.segment ? range.n : begin + p.segment;

  // waves behind the group's last help with its operands
  const int w = block * kWaves + wave;
  const bool works = w < waves;
  const int hv = h * a.G + (works ? w / kSlabs : 0), slab = wave % kSlabs;
  const int col = lane % 16, quad = lane / 16;
  const int v = slab * kColumns + col * NT;       // the lane's first column of the head
  const int column = hv * DV + v;                 // ... of out, and its channel of x
  const int out_row = a.HV * DV;
  constexpr int E = BF16 ? 2 : 4;
  if (slot < 0) {
    if (MODE != kSegment && works) {
      for (int t = begin + quad; t < end; t += 4)
        store_pair<BF16>(a.out, (static_cast<int64_t>(range.t0) + t) * out_row + column, 0.0f, 0.0f);
    }
    return;
  }

  f32x4 S[kKeyTiles][NT];
  const int64_t here = MODE == kWhole ? 0 : static_cast<int64_t>(range.t0 / p.segment) + u.b + u.i;
  const int tile_bytes = DK * DV * (MODE == kWhole && state_bf16 ? 2 : 4);
  char* const tile =
      MODE == kWhole ? static_cast<char*>(a.state_pool) + (static_cast<int64_t>(slot) * a.HV + hv) * tile_bytes
                     : reinterpret_cast<char*>(p.states) + (here * a.HV + hv) * tile_bytes;
  if constexpr (MODE == kWhole) {
    move_pool<false>(tile_resource(tile, tile_bytes), state_bf16, v_first, quad, v, S);
  } else if constexpr (MODE == kJoined) {
    move_state<false, false, false>(tile_resource(tile, tile_bytes), quad, v, S);
  } else {
#pragma unroll
    for (int kt = 0; kt < kKeyTiles; ++kt)
#pragma unroll
      for (int n = 0; n < NT; ++n) S[kt][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  Taps taps[NT];
  load_taps(a, {column, column + 1}, taps);
  const float skip = a.d_skip != nullptr ? a.d_skip[hv] : 0.0f;
  float gone = 1.0f;                    // the segment's decay

  constexpr int kC = TY * 2 * kKeySteps * kWave, kB = TS * kKeyTiles * kWave;
  Staged<kC> stage_c;
  Staged<kB> stage_b;
  Inputs<BF16> in;
  const int64_t first_slot = static_cast<int64_t>(range.t0 / Q) + u.b;
  const Keys* const first_keys = p.keys + first_slot * a.H + h;
  auto keys_at = [&](int t0) { return first_keys + static_cast<int64_t>(t0 / Q) * a.H; };
  const float* const first_steps = reinterpret_cast<const float*>(p.steps + first_slot * a.HV + hv);

  // the head's steps, and the wave's share of the pairs
  constexpr int kShare = 4 / kSlabs;          // half fragments
  float steps[3];
  f32x4 pairs[kShare];
  auto load_steps = [&](int t0) {
    const float* const from = first_steps + static_cast<int64_t>(t0 / Q) * a.HV * kSteps;
#pragma unroll
    for (int i = 0; i < 3; ++i) steps[i] = from[min(i * kWave + lane, kSteps - 1)];
    if constexpr (MODE != kSegment) {
#pragma unroll
      for (int i = 0; i < kShare; ++i) {
        const int share = slab + i * kSlabs;
        pairs[i] = keys_at(t0)->pairs[share % 2][share / 2][lane];
      }
    }
  };
  auto store_steps = [&](Steps& to) {
#pragma unroll
    for (int i = 0; i < 3; ++i) reinterpret_cast<float*>(&to)[min(i * kWave + lane, kSteps - 1)] = steps[i];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    if constexpr (MODE != kSegment) {
#pragma unroll
      for (int i = 0; i < kShare; ++i) {
        const int share = slab + i * kSlabs;
        decayed_pairs<TY>(to, pairs[i], skip, share % 2, share / 2, lane, sh.m[wave / kSlabs]);
      }
    }
  };
  // The lane's columns, convolved.  Tokens behind the last have step 0 and keys
  // of zero, but their taps may leave fp32, and zero times that is NaN: x of
  // zero.  The one branch of a step, here, where x is made, costs 0.8% of 8 x
  // 2048 x 96 heads (534 -> 538 us; in front of the outputs 2.5%).
  float x[8][NT];
  auto convolve = [&](const float (&past)[kPast][NT]) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        auto at = [&](int i) { return i < kPast ? past[i][n] : in.get(i, n); };
        x[j][n] = silu_f(taps[n].dot(FULL ? kTaps : a.K, at(j), at(j + 1), at(j + 2), at(j + 3)));
      }
  };
  auto drop_behind = [&](int quad, int valid) {
    if (__builtin_expect(valid < Q, 0)) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int n = 0; n < NT; ++n) x[j][n] = quad * 8 + j < valid ? x[j][n] : 0.0f;
    }
  };
  auto unpack_past = [&](float (&past)[kPast][NT]) {
#pragma unroll
    for (int j = 0; j < kPast; ++j)
#pragma unroll
      for (int n = 0; n < NT; ++n) past[j][n] = in.get(j, n);
  };

  load_steps(begin);
  in.load(a, range, begin, min(Q, end - begin), quad, column);
  if constexpr (MODE != kSegment) {
    stage_c.load(&keys_at(begin)->c[0][0][0][0]);
    stage_c.store(&sh.c[0][0][0][0]);
  }
  store_steps(sh.steps[wave][begin / Q % 2]);
  {
    float past[kPast][NT];
    unpack_past(past);
    if (begin == 0) {                   // the window of before
#pragma unroll
      for (int j = 0; j < kPast; ++j) {
        const int r = a.K - 1 - kPast + j;
        if (r >= 0 && quad == 0) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
            past[j][n] = p.windows[(static_cast<int64_t>(u.b) * (a.K - 1) + r) * a.C + column + n];
        }
      }
    }
    convolve(past);
    drop_behind(quad, end - begin);
  }

  // Per 32 tokens two stretches between barriers, each of products and of
  // other work for the next ones, with one branch: outputs from the state, with
  // the operands of the update; the update, with x and m of the next 32 (behind
  // the last, the last again, which nothing reads).
  for (int t0 = begin; t0 < end; t0 += Q) {
    const int valid = min(Q, end - t0);
    const int next = t0 + Q < end ? t0 + Q : t0;
    // The lane's place, anew for every 32 tokens: addresses made of it would
    // otherwise be kept in registers through all of them.
    int col = lane % 16, quad = lane / 16;
    asm volatile("" : "+v"(col), "+v"(quad));
    const int column = hv * DV + slab * kColumns + col * NT;
    const Steps& of = sh.steps[wave][t0 / Q % 2];
    lds_barrier();            // c and m are there, and b has been read
    stage_b.load(&keys_at(t0)->b[0][0][0]);
    load_steps(next);
    in.load(a, range, next, min(Q, end - next), quad, column);

    f32x4 y[2][NT];
    if constexpr (MODE != kSegment) {
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int n = 0; n < NT; ++n) y[mt][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      // C^T S0
#pragma unroll
      for (int step = 0; step < kKeySteps; ++step) {
        u32x4 s[NT][TY];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float f[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] = S[2 * step + j / 4][n][j % 4];
          split(f, s[n]);
        }
        u32x4 ck[2][TY];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int m = 0; m < TY; ++m) ck[mt][m] = sh.c[m][mt][step][lane];
        products(ck, s, y);
      }
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const f32x4 f = *reinterpret_cast<const f32x4*>(of.from + mt * 16 + quad * 4);
#pragma unroll
        for (int n = 0; n < NT; ++n) y[mt][n] *= f;
      }
      // the 32 tokens' own
      u32x4 xs[NT][TY], ms[2][TY];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = x[j][n];
        split(f, xs[n]);
      }
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int n = 0; n < TY; ++n)
          ms[mt][n] = *reinterpret_cast<const u32x4*>(&sh.m[wave / kSlabs][n][mt][lane][0]);
      products(ms, xs, y);
    }
    // x weighted for the update: step_s exp(c_last - c_s), from the last s
    // backwards
    u32x4 xw[NT][TS];
    {
      const int first = quad * 8;         // the lane's eight tokens s
      float f = __builtin_amdgcn_exp2f((of.hi[Q - 1] - of.hi[first + 7]) + (of.lo[Q - 1] - of.lo[first + 7]));
      float g[8];
#pragma unroll
      for (int j = 4; j >= 0; j -= 4) {
        const f32x4 decay = *reinterpret_cast<const f32x4*>(of.decay + first + j);
        const f32x4 step = *reinterpret_cast<const f32x4*>(of.step + first + j);
#pragma unroll
        for (int i = 3; i >= 0; --i) {
          g[j + i] = f * step[i];
          f *= decay[i];
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = x[j][n] * g[j];
        split(e, xw[n]);
      }
    }
    if constexpr (MODE != kSegment) {
      // rows behind the last, and all of a wave without columns, are dropped
      const __amdgpu_buffer_rsrc_t out =
          tile_resource(static_cast<char*>(a.out) + (static_cast<int64_t>(range.t0) + t0) * out_row * E,
                        works ? valid * out_row * E : 0);
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = ((mt * 16 + quad * 4 + i) * out_row + column) * E;
          if constexpr (BF16) {
            __builtin_amdgcn_raw_buffer_store_b32(f32x2_to_bf16x2_rne(y[mt][0][i], y[mt][1][i]), out, at, 0, 0);
          } else {
            const u32x2 o = {__float_as_uint(y[mt][0][i]), __float_as_uint(y[mt][1][i])};
            __builtin_amdgcn_raw_buffer_store_b64(o, out, at, 0, 0);
          }
        }
    }
    stage_b.store(&sh.b[0][0][0]);
    lds_barrier();            // b is there, and c and m have been read

    if constexpr (MODE != kSegment) stage_c.load(&keys_at(next)->c[0][0][0][0]);
    const float total = of.from[Q - 1];
    gone *= total;
#pragma unroll
    for (int kt = 0; kt < kKeyTiles; kt += 2) {
      u32x4 bk[2][TS];
      f32x4 s[2][NT];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int m = 0; m < TS; ++m) bk[i][m] = sh.b[m][kt + i][lane];
#pragma unroll
        for (int n = 0; n < NT; ++n) s[i][n] = S[kt + i][n] * total;
      }
      products(bk, xw, s);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n) S[kt + i][n] = s[i][n];
    }
    float past[kPast][NT];
    unpack_past(past);
    convolve(past);
    drop_behind(quad, end - next);
    store_steps(sh.steps[wave][next / Q % 2]);
    if constexpr (MODE != kSegment) stage_c.store(&sh.c[0][0][0][0]);
    if constexpr (MODE == kSegment) {
      // Each product followed by its share of the convolution (16384 tokens x
      // 32 heads 64 -> 61 us; with outputs there is enough else to do, and the
      // compiler's own order is better: 541 against 617 us at 8 x 2048 x 96).
      constexpr int kProducts = kKeyTiles * NT * (TS == 3 ? 6 : 3), kOther = 220;
#pragma unroll
      for (int i = 0; i < kProducts; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x2, (kOther + kProducts - 1) / kProducts, 0);
      }
    }
  }

  if (!works) return;
  if constexpr (MODE == kWhole) {
    move_pool<true>(tile_resource(tile, tile_bytes), state_bf16, v_first, quad, v, S);
  } else if constexpr (MODE == kSegment) {
    move_state<false, false, true>(tile_resource(tile, tile_bytes), quad, v, S);
    if (slab == 0 && lane == 0) p.decays[here * a.HV + hv] = gone;
  }
}

// The states before the segments of a request, and after its last: four
// adjacent columns per thread.
__global__ void __launch_bounds__(256) ssm_join(Plan p, bool state_bf16, bool v_first) {
  const SsmArgs& a = p.a;
  constexpr int parts = DK * DV / 1024;
  const int part = blockIdx.x % parts, head = blockIdx.x / parts;
  const int hv = head % a.HV, b = head / a.HV;
  const Range range = request_range(a, b);
  const int slot = request_slot(a, b);
  if (slot < 0 || range.n == 0) return;
  const int at = (part * 256 + threadIdx.x) * 4;
  const int k = at / DV, v = at % DV;
  const int64_t tile = (static_cast<int64_t>(slot) * a.HV + hv) * DK * DV;
  f32x4 s;
  int64_t where[4];
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    where[n] = tile + (v_first ? static_cast<int64_t>(v + n) * DK + k : static_cast<int64_t>(k) * DV + v + n);
    s[n] = state_bf16 ? load_scalar<true>(a.state_pool, where[n]) : load_scalar<false>(a.state_pool, where[n]);
  }
  const int64_t first = static_cast<int64_t>(range.t0 / p.segment) + b;
  const int segments = (range.n - 1) / p.segment + 1;
  const int64_t stride = static_cast<int64_t>(a.HV) * DK * DV;
  float* const states = p.states + first * stride + static_cast<int64_t>(hv) * DK * DV + at;
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

template <bool BF16, int TY, int TS, int MODE>
hipError_t scan(const Plan& plan, bool state_bf16, bool v_first, hipStream_t stream) {
  const void* const fn = plan.a.K == kTaps ? reinterpret_cast<const void*>(&ssm_scan<BF16, true, TY, TS, MODE>)
                                           : reinterpret_cast<const void*>(&ssm_scan<BF16, false, TY, TS, MODE>);
  constexpr int bytes = sizeof(Shared<TY, TS>);
  if constexpr (bytes > 65536) {        // beyond the default limit of dynamic LDS
    const hipError_t rc = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (rc != hipSuccess) return rc;
  }
  const int64_t blocks = (static_cast<int64_t>(plan.a.G) * kSlabs + kWaves - 1) / kWaves;
  int64_t groups = static_cast<int64_t>(plan.units) * plan.a.H;
  if (groups >= kXcds) groups = (groups + kXcds - 1) / kXcds * kXcds;
  void* kargs[] = {const_cast<Plan*>(&plan), &state_bf16, &v_first};
  return hipLaunchKernel(fn, dim3(static_cast<uint32_t>(groups * blocks)), dim3(kThreads), kargs, bytes, stream);
}

template <bool BF16, int TY, int TS>
hipError_t run(const Plan& plan, bool state_bf16, bool v_first, hipStream_t stream) {
  void* kargs[] = {const_cast<Plan*>(&plan), &state_bf16, &v_first};      // ssm_keys takes the first alone
  hipError_t rc = hipLaunchKernel(reinterpret_cast<const void*>(&ssm_keys<BF16, TY, TS>),
                                  dim3(plan.key_blocks + plan.window_blocks + plan.step_blocks), dim3(256), kargs, 0,
                                  stream);
  if (rc != hipSuccess) return rc;
  if (plan.segment == 0) return scan<BF16, TY, TS, kWhole>(plan, state_bf16, v_first, stream);
  rc = scan<BF16, TY, TS, kSegment>(plan, state_bf16, v_first, stream);
  if (rc != hipSuccess) return rc;
  const int64_t blocks = static_cast<int64_t>(plan.a.B) * plan.a.HV * (DK * DV / 1024);
  rc = hipLaunchKernel(reinterpret_cast<const void*>(&ssm_join), dim3(static_cast<uint32_t>(blocks)), dim3(256), kargs,
                       0, stream);
  if (rc != hipSuccess) return rc;
  // the state of a joined segment only reaches its outputs
  return scan<BF16, TY, TY, kJoined>(plan, state_bf16, v_first, stream);
}

// Whether requests are split into segments, which costs a second pass over
// them and two more launches, for waves of 64 columns per request.  By the
// waves that the batch has without (whole / split, us; dk = 128, dv = 64, 2000
// tokens each: 64 heads x 2 requests 213 / 98, x 4 219 / 224, x 6 223 / 326;
// lengths of 1 .. 4000 x 4 384 / 197, x 8 409 / 472; dk = 64, 2000 tokens x 4
// 197 / 149), and by the tokens: 32 heads, one request of 200 tokens 36 / 33,
// 512 64 / 41, 1024 99 / 44.  The longest request is not known here: with
// enough tokens in all there may be a long one, and a batch above the limit runs
// it in one piece (64 heads, 16384 tokens and four requests of 100 353 us, and
// five 1710; 4000 tokens 145 and 431).  Segments of at least
// 64 / 128 / 256 tokens: 512 tokens 41 / 43 / 60, 2048 55 / 50 / 66, 4 x 500
// 57 / 62 / 70.
constexpr int kSplitWaves = KDA_SSM_SPLIT / 16 * 5 * kResident<kJoined> / 3;
static_assert(kSplitWaves * 64 <= KDA_SSM_SPLIT * 20, "a state per request in KDA_SSM_WORKSPACE");

bool splits(const SsmArgs& args, int64_t waves) {
  return args.B * waves <= kSplitWaves && (args.T / args.B >= 192 || args.T >= 1024);
}

}  // namespace

template <>
int launch_ssm_prefill_of<DK, DV>(const SsmArgs& args, bool bf16, bool state_bf16, int state_layout,
                                  hipStream_t stream) {
  Plan plan{};
  plan.a = args;
  const int64_t chunks = static_cast<int64_t>(args.T) / Q + args.B;
  plan.keys = reinterpret_cast<Keys*>(args.workspace);
  plan.steps = reinterpret_cast<Steps*>(plan.keys + chunks * args.H);
  plan.windows = reinterpret_cast<float*>(plan.steps + chunks * args.HV);
  plan.states = plan.windows + static_cast<int64_t>(args.B) * (args.K - 1) * args.C;
  const int64_t waves = static_cast<int64_t>(args.HV) * (DV > 64 ? 2 : 1);
  plan.units = args.B;
  plan.key_blocks = static_cast<uint32_t>(chunks * args.H);
  plan.window_blocks = static_cast<uint32_t>(args.B) * ((args.HV * DV + 255) / 256);
  plan.step_blocks = static_cast<uint32_t>(chunks * ((args.HV + kHeads - 1) / kHeads));
  // segments that the chip holds at once, beyond one a request
  const int64_t most = KDA_SSM_SPLIT * kResident<kJoined> / 3 / waves;
  if (splits(args, waves) && most >= 1) {
    int64_t length = (args.T + most - 1) / most;
    length = (length + Q - 1) / Q * Q;
    if (length < kMinSegment) length = kMinSegment;
    if (length < args.T) {
      plan.segment = static_cast<int32_t>(length);
      plan.units = static_cast<int32_t>(args.T / length + args.B);
      plan.decays = plan.states + static_cast<int64_t>(plan.units) * args.HV * DK * DV;
    }
  }
  const bool v_first = state_layout == KDA_STATE_V_FIRST;
  hipError_t rc;
  if (!bf16) rc = run<false, 3, 3>(plan, state_bf16, v_first, stream);
  else if (state_bf16) rc = run<true, 2, 2>(plan, state_bf16, v_first, stream);
  else rc = run<true, 2, 3>(plan, state_bf16, v_first, stream);
  return rc == hipSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}

}  // namespace kda
