// kda_window.hip - decode windows for CDNA4 (gfx950): the gated delta rule
// with one decay per (token, value head) (kda_gdr_decode), and windows of
// drafted tokens that leave the state behind (kda_decode_window).
//
// Mathematics.  Per token, with alpha = exp(g):
//   u = v - alpha kh^T S,  o = alpha qh^T S + beta (qh.kh) u,
//   S' = alpha S + beta kh u^T
// (the definition with the decay folded into the reads).  The wave keeps its
// slab as S = D S^ with D the pending decay, so a token's write is one FMA
// per element, S^ += (beta / D') kh u^T with D' = D alpha; D' is applied to
// S^ on the last token before the slab is stored and whenever it would drop
// below 2^-64, which keeps 1 / D' finite.  With one decay per key channel
// (kda_decode_window on per-channel gates) D is a vector over the keys.
//
// Both calls walk the tokens of stream 0, write the state, walk those of
// stream 1 and drop what they made of it: a plain decode has its tokens in
// stream 0, a drafted window the previous window's kept tokens (without
// outputs) there and its own in stream 1.  So a window costs the same one
// read and one write of the state as a decode step, and a rejected draft
// never reaches the pool.
//
// Work split: one wave owns a 32-value slab of one (request, value head)
// tile for all dk keys; the value columns never interact, so no wave needs
// another.  Lanes hold the slab as the state layout streams best: key-first
// lane (rs, cq) keys rs + RS i and EPL values, value-first lane (rsub, kc)
// rows rsub + RPI i and EPL keys.
//
// Bound: the state's trip from HBM and back.  With one token a wave is almost
// all state traffic (96 heads x 256 requests, fp32 pool: 512 us, 6.3 TB/s);
// with windows the two sweeps per token (2 + 1 FMA per element) come into
// view, and long ones with one decay per head go 8 tokens at a time, replay
// and window together where that pays (window_chunk below).

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "kda.h"
#include "kda_device.h"
#include "kda_internal.h"
#include "kda_tile.h"

namespace kda {
namespace {

constexpr bool kChannel = KDA_WINDOW_CHANNEL;
constexpr float kDeferFloor = 5.421010862427522e-20f;   // 2^-64

struct Job {
  int b, hv, h, slab, slot;
  int t0, t1;          // rows of the stream with outputs
  int first[2], n[2];  // rows and tokens of each stream
};

__device__ __forceinline__ int clamp_to(int x, int lo, int hi) { return x < lo ? lo : (x > hi ? hi : x); }

template <int SLABS>
__device__ __forceinline__ Job resolve(const WindowArgs& a) {
  // XCD-aware id -> (tile, slab): each XCD takes one contiguous range, so
  // the slabs of a tile meet in one L2
  const uint32_t wg = blockIdx.x, nwg = gridDim.x;
  const uint32_t xcd = wg % kXcds, per = nwg / kXcds, extra = nwg % kXcds;
  const uint32_t logical = xcd * per + (xcd < extra ? xcd : extra) + wg / kXcds;
  Job j;
  j.slab = static_cast<int>(logical % SLABS);
  const int tile = static_cast<int>(logical / SLABS);
  j.b = tile / a.HV;
  j.hv = tile - j.b * a.HV;
  j.h = j.hv / a.G;
  j.slot = a.state_indices[j.b];
  const int T = a.src[a.window].T;
  j.t0 = clamp_to(a.cu_seqlens[j.b], 0, T);
  j.t1 = clamp_to(a.cu_seqlens[j.b + 1], j.t0, T);
  j.first[0] = j.first[1] = j.t0;
  j.n[0] = j.n[1] = j.t1 - j.t0;
  if (a.window) {
    j.first[0] = clamp_to(a.begin[j.b], 0, a.src[0].T);
    j.n[0] = clamp_to(a.count[j.b], 0, a.src[0].T - j.first[0]);
  } else {
    j.n[1] = 0;
  }
  return j;
}

// One token's inputs for one lane, in storage form: q, k and (per-channel
// gates) the gate pre-activation of its CPL setup channels, the NVL v values
// at v_ch, the beta logit and (per-head gates) the gate pre-activation.
template <int DK, int DV, bool QBF16, int CPL, int NVL>
struct TokenIn {
  RawRun<QBF16, CPL> q, k;
  RawRun<false, kChannel ? CPL : 1> x;
  RawRun<QBF16, NVL> v;
  float bl;
  // token i of the job's n[0] + n[1] tokens
  __device__ __forceinline__ void load(const WindowArgs& a, const Job& j, int i, int c0s, int64_t v_ch) {
    const int s = i >= j.n[0];
    const TokenStream& src = a.src[s];
    const int64_t t = j.first[s] + (s ? i - j.n[0] : i);
    const int64_t qk_off = (t * a.H + j.h) * DK + c0s;
    k.load(src.k, qk_off);
    if (src.q != nullptr) q.load(src.q, qk_off);   // uniform; a replay has no q
    else q.load(src.k, qk_off);
    const int64_t th = t * a.HV + j.hv;
    x.load(src.raw_gate, kChannel ? th * DK + c0s : th);
    v.load(src.v, t * a.HV * DV + v_ch);
    bl = src.beta_logits[th];
  }
};

// What a token's setup leaves for the sweeps (uniform over the wave).
struct TokenScalars {
  float beta_qk;   // beta * (qh . kh)
  float ka, qa;    // factors of the two reductions
  float w;         // factor of the write
  float fold;      // decay to apply to the slab first
  bool folds;
};

// Norms, gate and beta of one token; fills the tables
//   per head:    red[c] = {k, q} raw; the norms, decays and beta are scalars
//   per channel: red[c] = {kh m, qh m}, upd[c] = {D', beta kh w}
// where (m, w) = (D', 1 / D') while the decay is deferred and (1, 1) when
// this token folds it into the slab.
template <int DK, int CPL, typename In>
__device__ __forceinline__ TokenScalars setup(const WindowArgs& a, const In& in, int c0, bool chan_lane,
                                              const float (&dtb)[CPL], float amp, float2* red, float2* upd,
                                              float (&pend)[CPL], bool last) {
  float qv[CPL], kv[CPL];
  in.q.unpack(qv);
  in.k.unpack(kv);
  float sq = 0.0f, sk = 0.0f, sqk = 0.0f;
#pragma unroll
  for (int c = 0; c < CPL; ++c) {
    qv[c] = chan_lane ? qv[c] : 0.0f;
    kv[c] = chan_lane ? kv[c] : 0.0f;
    sq = fmaf(qv[c], qv[c], sq);
    sk = fmaf(kv[c], kv[c], sk);
    sqk = fmaf(qv[c], kv[c], sqk);
  }
  constexpr int XN = kChannel ? CPL : 1;
  float x[XN], alpha[XN];
  in.x.unpack(x);
  bool small = false;
#pragma unroll
  for (int c = 0; c < XN; ++c) {
    const float z = x[c] + dtb[c];
    const float g = a.gate_mode == KDA_GATE_SOFTPLUS ? -amp * softplus_f(z) : a.lower_bound * sigmoid_f(amp * z);
    alpha[c] = exp_f(g) * pend[c];   // D'
    small |= (!kChannel || chan_lane) && !(alpha[c] >= kDeferFloor);
  }
  TokenScalars s;
  s.folds = last || __any(small);
  const float beta = sigmoid_f(in.bl);
  if constexpr (!kChannel) {
    if (chan_lane) {
#pragma unroll
      for (int c = 0; c < CPL; ++c) red[c0 + c] = make_float2(kv[c], qv[c]);
    }
  }
  sq = wave_sum(sq);
  sk = wave_sum(sk);
  sqk = wave_sum(sqk);
  const float rq = a.scale * rsqrt_f(sq + a.l2_eps);
  const float rk = rsqrt_f(sk + a.l2_eps);
  s.beta_qk = beta * (sqk * rq * rk);
  if constexpr (kChannel) {
    s.ka = s.qa = s.w = s.fold = 1.0f;
    if (chan_lane) {
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        const float kh = kv[c] * rk, qh = qv[c] * rq;
        const float m = s.folds ? 1.0f : alpha[c];
        const float w = s.folds ? 1.0f : __builtin_amdgcn_rcpf(alpha[c]);
        red[c0 + c] = make_float2(kh * m, qh * m);
        upd[c0 + c] = make_float2(alpha[c], beta * kh * w);
      }
    }
#pragma unroll
    for (int c = 0; c < CPL; ++c) pend[c] = s.folds ? 1.0f : alpha[c];
  } else {
    const float m = s.folds ? 1.0f : alpha[0];
    s.ka = rk * m;
    s.qa = rq * m;
    s.w = beta * rk * (s.folds ? 1.0f : __builtin_amdgcn_rcpf(alpha[0]));
    s.fold = alpha[0];
#pragma unroll
    for (int c = 0; c < CPL; ++c) pend[c] = s.folds ? 1.0f : alpha[0];
  }
  return s;
}

// Skipped request: zero its output rows in this slab, leave every slot alone.
template <int DV, int CW, bool BF16>
__device__ __forceinline__ void zero_rows(const WindowArgs& a, const Job& j, int lane) {
  for (int t = j.t0; t < j.t1; ++t)
    if (lane < CW) store_scalar<BF16>(a.out, (static_cast<int64_t>(t) * a.HV + j.hv) * DV + j.slab * CW + lane, 0.0f);
}

// The gate's parameters of the lane's setup channels.
template <int DK, int CPL>
__device__ __forceinline__ void load_bias(const WindowArgs& a, const Job& j, int c0s, float (&dtb)[CPL]) {
  if constexpr (kChannel) {
    load_f32<CPL>(a.dt_bias + static_cast<int64_t>(j.hv) * DK + c0s, dtb);
  } else {
#pragma unroll
    for (int c = 0; c < CPL; ++c) dtb[c] = a.dt_bias[j.hv];
  }
}

// ---------------------------------------------------------------------------
// key-first layout: state [dk][dv]
// ---------------------------------------------------------------------------

template <int DK, int DV, bool QBF16, bool SBF16>
__global__ __launch_bounds__(kWave) void window_kfirst(const WindowArgs a) {
  constexpr int CW = DV < 32 ? DV : 32;   // value columns of the wave's slab
  constexpr int SLABS = DV / CW;
  // values per lane and key row: 8 bf16 (16 bytes) where dk has a row for
  // each of the row groups that leaves, else 4
  constexpr int EPL = (SBF16 && DK >= kWave * 8 / CW) ? 8 : 4;
  constexpr int CQ = CW / EPL;            // lanes across the slab's columns
  constexpr int RS = kWave / CQ;          // row groups across the wave
  constexpr int R = DK / RS;              // key rows per lane
  constexpr int NV = 2 * EPL;             // partial sums per lane (k and q)
  constexpr int LOG_CQ = log2_exact<CQ>();
  constexpr int LOG_RS = log2_exact<RS>();
  constexpr int LOG_NV = log2_exact<NV>();
  constexpr int CPL = DK >= 2 * kWave ? DK / kWave : 1;   // setup channels per lane
  static_assert(DK % RS == 0 && R >= 1 && LOG_NV <= LOG_RS, "tile shape");
  static_assert(CPL * kWave >= DK && CPL <= 2, "setup split");
  // a 32-column bf16 row is half a cache line, which L2 merges with the
  // neighbouring slab's; whole-line rows stream past the caches
  using IO = StateIO<SBF16, EPL, (SBF16 && CW * 2 < 128) ? 0 : kCachePolicyNT>;

  __shared__ __attribute__((aligned(16))) float2 red_tab[2][DK];
  __shared__ __attribute__((aligned(16))) float2 upd_tab[2][kChannel ? DK : 1];
  __shared__ __attribute__((aligned(16))) float u_tab[CW];

  const int lane = threadIdx.x;
  const int cq = lane % CQ;
  const int rs = lane / CQ;
  const Job j = resolve<SLABS>(a);
  if (j.slot < 0 || j.slot >= a.N) {
    zero_rows<DV, CW, QBF16>(a, j, lane);
    return;
  }
  const int total = j.n[0] + j.n[1];
  if (total == 0) return;

  const int col0 = j.slab * CW + EPL * cq;
  char* const tile = static_cast<char*>(a.state_pool) +
                     (static_cast<int64_t>(j.slot) * a.HV + j.hv) * (DK * DV * IO::kElem);
  const __amdgpu_buffer_rsrc_t res = tile_resource(tile, DK * DV * IO::kElem);
  const int voff = (rs * DV + col0) * IO::kElem;
  constexpr int kRowStep = RS * DV * IO::kElem;
  float S[R][EPL];
#pragma unroll
  for (int i = 0; i < R; ++i) IO::load(res, voff, i * kRowStep, S[i]);

  const int c0 = lane * CPL;
  const bool chan_lane = CPL * kWave == DK || c0 < DK;
  const int c0s = chan_lane ? c0 : 0;
  float dtb[CPL];
  load_bias<DK, CPL>(a, j, c0s, dtb);
  const float amp = exp_f(a.a_log[j.hv]);

  // After the reduction lane rs holds sum m = rs & (NV - 1): k^T S of column
  // col0 + m when m < EPL, else q^T S of column col0 + m - EPL.
  const int m_final = rs & (NV - 1);
  const bool holds_k = m_final < EPL;
  const bool owner = rs < NV;
  const int my_col = col0 + (m_final & (EPL - 1));
  const int64_t v_ch = static_cast<int64_t>(j.hv) * DV + my_col;

  float pend[CPL];
#pragma unroll
  for (int c = 0; c < CPL; ++c) pend[c] = 1.0f;
  using In = TokenIn<DK, DV, QBF16, CPL, 1>;
  In nxt;
  nxt.load(a, j, 0, c0s, v_ch);
  for (int i = 0; i < total; ++i) {
    const In cur = nxt;
    if (i + 1 < total) nxt.load(a, j, i + 1, c0s, v_ch);   // uniform
    const int buf = i & 1;
    float v_mine[1];
    cur.v.unpack(v_mine);
    const TokenScalars ts = setup<DK, CPL>(a, cur, c0, chan_lane, dtb, amp, red_tab[buf], upd_tab[buf], pend,
                                           i + 1 == j.n[0]);
    __syncthreads();
    if (ts.folds) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float f = kChannel ? upd_tab[buf][rs + RS * r].x : ts.fold;
#pragma unroll
        for (int e = 0; e < EPL; ++e) S[r][e] *= f;
      }
    }
    float acc[NV];
#pragma unroll
    for (int m = 0; m < NV; ++m) acc[m] = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float2 p = red_tab[buf][rs + RS * r];
#pragma unroll
      for (int e = 0; e < EPL; ++e) {
        acc[e] = fmaf(p.x, S[r][e], acc[e]);
        acc[EPL + e] = fmaf(p.y, S[r][e], acc[EPL + e]);
      }
    }
    transpose_levels<NV / 2, LOG_CQ + LOG_NV - 1>(acc, lane);
    const float red = sum_levels<LOG_CQ + LOG_RS - 1, LOG_CQ + LOG_NV>(acc[0]) * (holds_k ? ts.ka : ts.qa);
    if (holds_k && owner) u_tab[EPL * cq + m_final] = v_mine[0] - red;
    __syncthreads();
    float u[EPL];
#pragma unroll
    for (int e = 0; e < EPL; e += 4) {
      const float4 x = *reinterpret_cast<const float4*>(&u_tab[EPL * cq + e]);
      u[e] = x.x;
      u[e + 1] = x.y;
      u[e + 2] = x.z;
      u[e + 3] = x.w;
    }
    if (!holds_k && owner && (i >= j.n[0] || !a.window)) {
      const int64_t t = j.t0 + (a.window ? i - j.n[0] : i);
      store_scalar<QBF16>(a.out, t * a.HV * DV + v_ch, fmaf(ts.beta_qk, u[m_final & (EPL - 1)], red));
    }
#pragma unroll
    for (int e = 0; e < EPL; ++e) u[e] *= ts.w;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float p = kChannel ? upd_tab[buf][rs + RS * r].y : red_tab[buf][rs + RS * r].x;
#pragma unroll
      for (int e = 0; e < EPL; ++e) S[r][e] = fmaf(p, u[e], S[r][e]);
    }
    if (i + 1 == j.n[0]) {
#pragma unroll
      for (int r = 0; r < R; ++r) IO::store(res, voff, r * kRowStep, S[r]);
    }
  }
}

// ---------------------------------------------------------------------------
// value-first layout: state [dv][dk]
// ---------------------------------------------------------------------------

template <int DK, int DV, bool QBF16, bool SBF16>
__global__ __launch_bounds__(kWave) void window_vfirst(const WindowArgs a) {
  constexpr int CW = DV < 32 ? DV : 32;   // value rows of the wave's slab
  constexpr int SLABS = DV / CW;
  // keys per lane and value row, as in the decode kernel: 8 where the slab
  // has a row for each of the 512 / dk rows one load instruction covers
  constexpr int EPL = (kWave * 8 / DK <= CW && (SBF16 || DK >= 64)) ? 8 : 4;
  constexpr int Q = EPL / 4;
  constexpr bool ONE_ACCESS = SBF16 && EPL == 8;
  constexpr int KSTEP = ONE_ACCESS ? 8 : 4;          // keys between neighbouring lanes
  constexpr int QSTRIDE = ONE_ACCESS ? 4 : DK / 2;   // keys between a lane's groups
  constexpr int KC = DK / EPL;            // lanes across one row
  constexpr int RPI = kWave / KC;         // rows per load instruction
  constexpr int L = CW / RPI;             // rows per lane
  constexpr int NV = 2 * L;               // partial sums per lane (k and q)
  constexpr int LOG_KC = log2_exact<KC>();
  constexpr int LOG_NV = log2_exact<NV>();
  constexpr int CPL = DK >= 2 * kWave ? DK / kWave : 1;
  static_assert(L >= 1 && LOG_NV <= LOG_KC, "tile shape");
  static_assert(CPL * kWave >= DK && CPL <= 2, "setup split");
  using IO = StateIO<SBF16, ONE_ACCESS ? 8 : 4>;

  __shared__ __attribute__((aligned(16))) float2 red_tab[2][DK];
  __shared__ __attribute__((aligned(16))) float2 upd_tab[2][kChannel ? DK : 1];
  __shared__ __attribute__((aligned(16))) float u_tab[CW];   // [RPI][L]

  const int lane = threadIdx.x;
  const int kc = lane % KC;
  const int rsub = lane / KC;
  const Job j = resolve<SLABS>(a);
  if (j.slot < 0 || j.slot >= a.N) {
    zero_rows<DV, CW, QBF16>(a, j, lane);
    return;
  }
  const int total = j.n[0] + j.n[1];
  if (total == 0) return;

  const int row0 = j.slab * CW + rsub;
  const int key0 = KSTEP * kc;
  char* const tile = static_cast<char*>(a.state_pool) +
                     (static_cast<int64_t>(j.slot) * a.HV + j.hv) * (DK * DV * IO::kElem);
  const __amdgpu_buffer_rsrc_t res = tile_resource(tile, DK * DV * IO::kElem);
  const int voff = (row0 * DK + key0) * IO::kElem;
  constexpr int kRowStep = RPI * DK * IO::kElem;
  constexpr int kGroupStep = QSTRIDE * IO::kElem;
  float S[L][EPL];
#pragma unroll
  for (int l = 0; l < L; ++l) {
    if constexpr (ONE_ACCESS) {
      IO::load(res, voff, l * kRowStep, S[l]);
    } else {
#pragma unroll
      for (int q = 0; q < Q; ++q) IO::load(res, voff + q * kGroupStep, l * kRowStep, &S[l][4 * q]);
    }
  }

  const int c0 = lane * CPL;
  const bool chan_lane = CPL * kWave == DK || c0 < DK;
  const int c0s = chan_lane ? c0 : 0;
  float dtb[CPL];
  load_bias<DK, CPL>(a, j, c0s, dtb);
  const float amp = exp_f(a.a_log[j.hv]);

  // After the reduction lane kc holds sum m of its row group: k^T S of row
  // i = m when m < L, else q^T S of row i = m - L.
  const int m_final = (kc >> (LOG_KC - LOG_NV)) & (NV - 1);
  const bool holds_k = m_final < L;
  const int i_final = m_final & (L - 1);
  const bool owner = (kc & ((1 << (LOG_KC - LOG_NV)) - 1)) == 0;
  const int my_row = row0 + RPI * i_final;
  const int64_t v_ch = static_cast<int64_t>(j.hv) * DV + my_row;

  float pend[CPL];
#pragma unroll
  for (int c = 0; c < CPL; ++c) pend[c] = 1.0f;
  using In = TokenIn<DK, DV, QBF16, CPL, 1>;
  In nxt;
  nxt.load(a, j, 0, c0s, v_ch);
  for (int i = 0; i < total; ++i) {
    const In cur = nxt;
    if (i + 1 < total) nxt.load(a, j, i + 1, c0s, v_ch);   // uniform
    const int buf = i & 1;
    float v_mine[1];
    cur.v.unpack(v_mine);
    const TokenScalars ts = setup<DK, CPL>(a, cur, c0, chan_lane, dtb, amp, red_tab[buf], upd_tab[buf], pend,
                                           i + 1 == j.n[0]);
    __syncthreads();
    if (ts.folds) {
      float f[EPL];
#pragma unroll
      for (int e = 0; e < EPL; ++e) f[e] = kChannel ? upd_tab[buf][key0 + QSTRIDE * (e / 4) + e % 4].x : ts.fold;
#pragma unroll
      for (int l = 0; l < L; ++l)
#pragma unroll
        for (int e = 0; e < EPL; ++e) S[l][e] *= f[e];
    }
    float kq[EPL], qq[EPL];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const float4 r01 = *reinterpret_cast<const float4*>(&red_tab[buf][key0 + QSTRIDE * q]);
      const float4 r23 = *reinterpret_cast<const float4*>(&red_tab[buf][key0 + QSTRIDE * q + 2]);
      kq[4 * q] = r01.x;  qq[4 * q] = r01.y;
      kq[4 * q + 1] = r01.z;  qq[4 * q + 1] = r01.w;
      kq[4 * q + 2] = r23.x;  qq[4 * q + 2] = r23.y;
      kq[4 * q + 3] = r23.z;  qq[4 * q + 3] = r23.w;
    }
    float vals[NV];
#pragma unroll
    for (int l = 0; l < L; ++l) {
      float sa = kq[0] * S[l][0], sb = qq[0] * S[l][0];
#pragma unroll
      for (int e = 1; e < EPL; ++e) {
        sa = fmaf(kq[e], S[l][e], sa);
        sb = fmaf(qq[e], S[l][e], sb);
      }
      vals[l] = sa;
      vals[L + l] = sb;
    }
    transpose_levels<NV / 2, LOG_KC - 1>(vals, lane);
    const float red = sum_levels<LOG_KC - LOG_NV - 1, 0>(vals[0]) * (holds_k ? ts.ka : ts.qa);
    if (holds_k && owner) u_tab[rsub * L + i_final] = v_mine[0] - red;
    __syncthreads();
    if (!holds_k && owner && (i >= j.n[0] || !a.window)) {
      const int64_t t = j.t0 + (a.window ? i - j.n[0] : i);
      store_scalar<QBF16>(a.out, t * a.HV * DV + v_ch, fmaf(ts.beta_qk, u_tab[rsub * L + i_final], red));
    }
    float wk[EPL];
#pragma unroll
    for (int e = 0; e < EPL; ++e)
      wk[e] = kChannel ? upd_tab[buf][key0 + QSTRIDE * (e / 4) + e % 4].y : kq[e] * ts.w;
#pragma unroll
    for (int l = 0; l < L; ++l) {
      const float u = u_tab[rsub * L + l];
#pragma unroll
      for (int e = 0; e < EPL; ++e) S[l][e] = fmaf(wk[e], u, S[l][e]);
    }
    if (i + 1 == j.n[0]) {
#pragma unroll
      for (int l = 0; l < L; ++l) {
        if constexpr (ONE_ACCESS) {
          IO::store(res, voff, l * kRowStep, S[l]);
        } else {
#pragma unroll
          for (int q = 0; q < Q; ++q) IO::store(res, voff + q * kGroupStep, l * kRowStep, &S[l][4 * q]);
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// windows of several tokens with one decay per head: up to 8 tokens at once
// ---------------------------------------------------------------------------

// With a scalar decay a window needs the state only through kh_i^T S0 and
// qh_i^T S0 (G_i: the log decay summed from the window's start):
//   U_i = beta_i (v_i - e^(G_i) kh_i^T S0 - sum_{j<i} e^(G_i - G_j) kh_i.kh_j U_j)
//   o_i = e^(G_i) qh_i^T S0 + sum_{j<=i} e^(G_i - G_j) qh_i.kh_j U_j
//   S'  = e^(G_last) S0 + sum_j e^(G_last - G_j) kh_j U_j^T
// So the sweeps over S are matrix products of 8 rows of k and 8 of q against
// the slab, on the fp32 matrix instruction (exact products of the raw values;
// norms and decays are factors of rows), which run beside the loads and
// leave the vector units with the small triangular solve: about 500
// instructions for up to 8 tokens against 330 for each one.
//
// A lane holds value columns n = lane % 16 (NCS neighbours) and keys 32 s + 8 g
// + 4 b + 0..3 (g = lane / 16): the accumulator layout of the update, the second
// operand of the products, and 16-byte pieces of a value-first row.

constexpr int kW = 8;   // tokens at once

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

template <int DK, int CW>
struct ChunkTables {
  float dots[2 * kW][CW];     // k_i^T S0, q_i^T S0 of the raw rows
  float u[kW][CW];            // e^(G_last - G_j) norm_k U_j
  float k[kW][DK + 4];        // raw k
  float coef[2 * kW][kW];     // of U_j in U_i, and in o_i
  float row[2 * kW];          // norm factors of the rows of k, and of q (times scale)
  float g_hi[kW], g_lo[kW], beta[kW];
  float lead[2 * kW];         // factor of dots[i]
  float tail[kW];             // e^(G_last - G_j) norm_k
  float last;                 // e^(G_last)
};

// Replay and window at once: m replayed and n window tokens of a request with
// m + 2 n <= 16 rows of k and q and m + n <= kMost tokens.  U runs over all of
// them from the one state S0; only the replayed ones go into S'.
constexpr int kMost = 11;

template <int DK, int CW>
struct JointTables {
  float dots[16][CW];
  float u[12][CW];
  float k[12][DK + 4];
  float coef[16][12];
  float row[16], g_hi[16], g_lo[16], beta[16], lead[16], tail[16];
  float last;
};

// exp(G_i - G_j) from two-float sums.
[[maybe_unused]] __device__ __forceinline__ float decay(float hi_i, float lo_i, float hi_j, float lo_j) {
  return exp_f((hi_i - hi_j) + (lo_i - lo_j));
}

[[maybe_unused]] __device__ __forceinline__ double row_shr_f64(double x, int by) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const int lo = static_cast<int>(u), hi = static_cast<int>(u >> 32);
  uint32_t l, h;
  if (by == 1) {
    l = __builtin_amdgcn_update_dpp(0, lo, 0x111, 0xf, 0xf, true);
    h = __builtin_amdgcn_update_dpp(0, hi, 0x111, 0xf, 0xf, true);
  } else if (by == 2) {
    l = __builtin_amdgcn_update_dpp(0, lo, 0x112, 0xf, 0xf, true);
    h = __builtin_amdgcn_update_dpp(0, hi, 0x112, 0xf, 0xf, true);
  } else if (by == 4) {
    l = __builtin_amdgcn_update_dpp(0, lo, 0x114, 0xf, 0xf, true);
    h = __builtin_amdgcn_update_dpp(0, hi, 0x114, 0xf, 0xf, true);
  } else {
    l = __builtin_amdgcn_update_dpp(0, lo, 0x118, 0xf, 0xf, true);
    h = __builtin_amdgcn_update_dpp(0, hi, 0x118, 0xf, 0xf, true);
  }
  return __builtin_bit_cast(double, static_cast<uint64_t>(h) << 32 | l);
}

// 8 keys of a slab that hold bf16 values, as an operand.
[[maybe_unused]] __device__ __forceinline__ bf16x8 pack_slab(const f32x4& x, const f32x4& y) {
  return __builtin_bit_cast(bf16x8, u32x4{f32x2_to_bf16x2_rne(x[0], x[1]), f32x2_to_bf16x2_rne(x[2], x[3]),
                                          f32x2_to_bf16x2_rne(y[0], y[1]), f32x2_to_bf16x2_rne(y[2], y[3])});
}

// Orders the wave's LDS accesses (one wave is the whole workgroup).
[[maybe_unused]] __device__ __forceinline__ void lds_sync() { __syncthreads(); }

// One chunk's inputs in storage form.
template <int DK, int DV, int CW, bool QBF16>
struct ChunkIn {
  static constexpr int KS = DK / 32;
  u32x4 x[KS][QBF16 ? 1 : 2];   // lane row n16 (k 0..7, q 8..15), keys 32 s + 8 g + 0..7
  RawRun<QBF16, 1> v[kW];       // the lane's column of the solve
  float gate, beta;             // of token lane % 8

  // `n` tokens from row t0 of the stream; rows past them repeat row t0 and are
  // dropped where they are used
  __device__ __forceinline__ void load(const WindowArgs& a, const Job& j, const TokenStream& src, int64_t t0, int n,
                                       bool outputs, int lane) {
    const int n16 = lane % 16, tok = n16 % kW;
    const bool live = tok < n && (n16 < kW || outputs);
    const void* const base = n16 < kW || !outputs ? src.k : src.q;
    const int64_t off = ((t0 + (live ? tok : 0)) * a.H + j.h) * DK + 8 * (lane / 16);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      if constexpr (QBF16) {
        x[s][0] = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(base) + off + 32 * s);
      } else {
        x[s][0] = *reinterpret_cast<const u32x4*>(static_cast<const float*>(base) + off + 32 * s);
        x[s][1] = *reinterpret_cast<const u32x4*>(static_cast<const float*>(base) + off + 32 * s + 4);
      }
    }
    const int gt = lane % kW;
    const int64_t goff = (t0 + (gt < n ? gt : 0)) * a.HV + j.hv;
    gate = src.raw_gate[goff];
    beta = src.beta_logits[goff];
#pragma unroll
    for (int i = 0; i < kW; ++i)
      v[i].load(src.v, ((t0 + (i < n ? i : 0)) * a.HV + j.hv) * DV + j.slab * CW + lane % CW);
  }
};

template <int DK, int DV, bool QBF16, bool SBF16, int LAYOUT, int CWT, bool JOINT>
__global__ __launch_bounds__(kWave) void window_chunk(const WindowArgs a) {
  constexpr int CW = DV < CWT ? DV : CWT;
  constexpr int SLABS = DV / CW;
  constexpr int NCS = CW / 16;
  constexpr int KS = DK / 32;
  constexpr int E = SBF16 ? 2 : 4;
  __shared__ __attribute__((aligned(16))) union {
    ChunkTables<DK, CW> chunk;
    std::conditional_t<JOINT, JointTables<DK, CW>, char> joint;
  } tables;
  ChunkTables<DK, CW>& sh = tables.chunk;

  const int lane = threadIdx.x;
  const int n16 = lane % 16, g = lane / 16;
  const Job j = resolve<SLABS>(a);
  if (j.slot < 0 || j.slot >= a.N) {
    zero_rows<DV, CW, QBF16>(a, j, lane);
    return;
  }
  const int total = j.n[0] + j.n[1];
  if (total == 0) return;

  // ---- the slab ----
  char* const tile = static_cast<char*>(a.state_pool) +
                     (static_cast<int64_t>(j.slot) * a.HV + j.hv) * (DK * DV * E);
  const __amdgpu_buffer_rsrc_t res = tile_resource(tile, DK * DV * E);
  f32x4 S[KS][2][NCS];
  const int col = j.slab * CW + NCS * n16;
  const auto slab_io = [&](auto store) {
    constexpr bool STORE = decltype(store)::value;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      if constexpr (LAYOUT == KDA_STATE_V_FIRST) {
#pragma unroll
        for (int cs = 0; cs < NCS; ++cs) {
          const int voff = ((col + cs) * DK + 8 * g) * E;
          float x[8] = {S[s][0][cs][0], S[s][0][cs][1], S[s][0][cs][2], S[s][0][cs][3],
                        S[s][1][cs][0], S[s][1][cs][1], S[s][1][cs][2], S[s][1][cs][3]};
          if constexpr (SBF16) {
            if constexpr (STORE) StateIO<true, 8, 0>::store(res, voff, 32 * s * E, x);
            else StateIO<true, 8, 0>::load(res, voff, 32 * s * E, x);
          } else {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              if constexpr (STORE) StateIO<false, 4, 0>::store(res, voff, (32 * s + 4 * b) * E, x + 4 * b);
              else StateIO<false, 4, 0>::load(res, voff, (32 * s + 4 * b) * E, x + 4 * b);
            }
          }
          if constexpr (!STORE) {
            S[s][0][cs] = f32x4{x[0], x[1], x[2], x[3]};
            S[s][1][cs] = f32x4{x[4], x[5], x[6], x[7]};
          }
        }
      } else {
        const int voff = (8 * g * DV + col) * E;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int soff = (32 * s + 4 * b + r) * DV * E;
            if constexpr (STORE) {
              if constexpr (SBF16 && NCS == 2)
                __builtin_amdgcn_raw_buffer_store_b32(f32x2_to_bf16x2_rne(S[s][b][0][r], S[s][b][1][r]), res, voff, soff, 0);
              else if constexpr (SBF16)
                __builtin_amdgcn_raw_buffer_store_b16(static_cast<uint16_t>(f32_to_bf16_rne(S[s][b][0][r])), res, voff, soff, 0);
              else if constexpr (NCS == 2)
                __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(S[s][b][0][r]), __float_as_uint(S[s][b][1][r])},
                                                      res, voff, soff, kCachePolicyNT);
              else
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[s][b][0][r]), res, voff, soff, 0);
            } else if constexpr (SBF16 && NCS == 2) {
              const uint32_t w = __builtin_amdgcn_raw_buffer_load_b32(res, voff, soff, 0);
              S[s][b][0][r] = bf16_to_f32(w & 0xffffu);
              S[s][b][1][r] = __uint_as_float(w & 0xffff0000u);
            } else if constexpr (SBF16) {
              S[s][b][0][r] = bf16_to_f32(__builtin_amdgcn_raw_buffer_load_b16(res, voff, soff, 0));
            } else if constexpr (NCS == 2) {
              const u32x2 w = __builtin_amdgcn_raw_buffer_load_b64(res, voff, soff, kCachePolicyNT);
              S[s][b][0][r] = __uint_as_float(w.x);
              S[s][b][1][r] = __uint_as_float(w.y);
            } else {
              S[s][b][0][r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(res, voff, soff, 0));
            }
          }
      }
    }
  };
  slab_io(std::false_type{});

  const float amp = exp_f(a.a_log[j.hv]);
  const float bias = a.dt_bias[j.hv];
  const int c = lane % CW;                       // the lane's column in the solve
  constexpr int SHARE = kWave / CW;              // lanes that solve a column; each stores kW / SHARE outputs
  const int part = lane / CW;

  if constexpr (JOINT) {
    const int m = j.n[0], nw = j.n[1];
    if (a.window && m > 0 && nw > 0 && m + 2 * nw <= 16 && m + nw <= kMost) {   // uniform
      JointTables<DK, CW>& jt = tables.joint;
      const int all = m + nw;
      const TokenStream& s0 = a.src[0];
      const TokenStream& s1 = a.src[1];
      // token t of the joint list: its stream's row
      const auto row_of = [&](int t) { return static_cast<int64_t>(t < m ? j.first[0] + t : j.first[1] + t - m); };
      // ---- lane row n16: k of token n16, then q of the window's tokens; keys 32 s + 8 g + 0..7 ----
      const bool is_k = n16 < all, is_q = !is_k && n16 < all + nw;
      const int token = is_k ? n16 : is_q ? n16 - nw : 0;   // q row all + i belongs to token m + i
      const void* const base = is_q ? s1.q : token < m ? s0.k : s1.k;
      const int64_t off = (row_of(token) * a.H + j.h) * DK + 8 * g;
      u32x4 xw[KS][QBF16 ? 1 : 2];
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        if constexpr (QBF16) {
          xw[s][0] = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(base) + off + 32 * s);
        } else {
          xw[s][0] = *reinterpret_cast<const u32x4*>(static_cast<const float*>(base) + off + 32 * s);
          xw[s][1] = *reinterpret_cast<const u32x4*>(static_cast<const float*>(base) + off + 32 * s + 4);
        }
      }
      const int gt = n16 < all ? n16 : 0;
      const int64_t goff = row_of(gt) * a.HV + j.hv;
      const float gate = gt < m ? s0.raw_gate[goff] : s1.raw_gate[goff];
      const float bl = gt < m ? s0.beta_logits[goff] : s1.beta_logits[goff];
      RawRun<QBF16, 1> vw[kMost];
#pragma unroll
      for (int i = 0; i < kMost; ++i) {
        const int t = i < all ? i : 0;
        vw[i].load(t < m ? s0.v : s1.v, (row_of(t) * a.HV + j.hv) * DV + j.slab * CW + c);
      }

      // ---- gates, summed in fp64 over the lanes of a row ----
      {
        const float x = gate + bias;
        float gv = a.gate_mode == KDA_GATE_SOFTPLUS ? -amp * softplus_f(x) : a.lower_bound * sigmoid_f(amp * x);
        gv = gv < -200.0f ? -200.0f : gv;
        double sum = n16 < all ? static_cast<double>(gv) : 0.0;
        sum += row_shr_f64(sum, 1);
        sum += row_shr_f64(sum, 2);
        sum += row_shr_f64(sum, 4);
        sum += row_shr_f64(sum, 8);
        if (lane < 16) {
          const float hi = static_cast<float>(sum);
          jt.g_hi[n16] = hi;
          jt.g_lo[n16] = static_cast<float>(sum - static_cast<double>(hi));
          jt.beta[n16] = n16 < all ? sigmoid_f(bl) : 0.0f;
        }
      }
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int h = 0; h < (QBF16 ? 1 : 2); ++h)
          if (!is_k && !is_q) xw[s][h] = u32x4{0, 0, 0, 0};
      const auto key_value = [&](int s, int e) {   // key 32 s + 8 g + e
        if constexpr (QBF16) return e % 2 ? __uint_as_float(xw[s][0][e / 2] & 0xffff0000u) : __uint_as_float(xw[s][0][e / 2] << 16);
        else return __uint_as_float(xw[s][e / 4][e % 4]);
      };
      float sq = 0.0f;
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int e = 0; e < 8; ++e) sq = fmaf(key_value(s, e), key_value(s, e), sq);
      sq = swap16_add(sq, sq);
      sq = swap32_add(sq, sq);
      if (lane < 16) jt.row[n16] = (is_q ? a.scale : 1.0f) * rsqrt_f(sq + a.l2_eps);
      if (n16 < 12) {   // k of the replayed tokens, zero past them
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            f32x4 x = {key_value(s, 4 * h), key_value(s, 4 * h + 1), key_value(s, 4 * h + 2), key_value(s, 4 * h + 3)};
            if (n16 >= m) x = f32x4{0, 0, 0, 0};
            *reinterpret_cast<f32x4*>(&jt.k[n16][32 * s + 8 * g + 4 * h]) = x;
          }
      }
      // ---- Gram matrix of the rows, rows against the slab ----
      f32x4 gram = {0, 0, 0, 0}, dots[NCS];
#pragma unroll
      for (int cs = 0; cs < NCS; ++cs) dots[cs] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        if constexpr (QBF16) {
          const bf16x8 x = __builtin_bit_cast(bf16x8, xw[s][0]);
          gram = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, x, gram, 0, 0, 0);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            gram = __builtin_amdgcn_mfma_f32_16x16x4f32(key_value(s, e), key_value(s, e), gram, 0, 0, 0);
        }
        if constexpr (SBF16 && QBF16) {
#pragma unroll
          for (int cs = 0; cs < NCS; ++cs)
            dots[cs] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xw[s][0]),
                                                              pack_slab(S[s][0][cs], S[s][1][cs]), dots[cs], 0, 0, 0);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int cs = 0; cs < NCS; ++cs)
              dots[cs] = __builtin_amdgcn_mfma_f32_16x16x4f32(key_value(s, e), S[s][e / 4][cs][e % 4], dots[cs], 0, 0, 0);
        }
      }
      lds_sync();
      // ---- factors ----
      if (lane < 16) {
        const float gh = jt.g_hi[token], gl = jt.g_lo[token];
        const float eg = exp_f(gh + gl);
        jt.lead[n16] = eg * jt.row[n16] * (is_k ? jt.beta[n16] : 1.0f);
        jt.tail[n16] = jt.row[n16] * decay(jt.g_hi[m - 1], jt.g_lo[m - 1], gh, gl);   // of replayed tokens only
        if (n16 == m - 1) jt.last = eg;
      }
      if (n16 < all) {
        const float gh = jt.g_hi[n16], gl = jt.g_lo[n16], nk = jt.row[n16];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 4 * g + r;
          const bool k_row = row < all;
          const int i = k_row ? row : row < all + nw ? row - nw : 0;
          const float f = nk * jt.row[row] * decay(jt.g_hi[i], jt.g_lo[i], gh, gl) * gram[r];
          jt.coef[row][n16] = k_row ? (n16 < i ? f * jt.beta[i] : 0.0f) : (n16 <= i ? f : 0.0f);
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if constexpr (NCS == 2) *reinterpret_cast<float2*>(&jt.dots[4 * g + r][2 * n16]) = make_float2(dots[0][r], dots[1][r]);
        else jt.dots[4 * g + r][n16] = dots[0][r];
      }
      lds_sync();
      // ---- the solve, one column per lane ----
      float U[kMost];
#pragma unroll
      for (int i = 0; i < kMost; ++i) {
        U[i] = 0.0f;
        if (i < all) {
          float v[1];
          vw[i].unpack(v);
          float acc = fmaf(jt.beta[i], v[0], -jt.lead[i] * jt.dots[i][c]);
#pragma unroll
          for (int k = 0; k < i; ++k) acc = fmaf(-jt.coef[i][k], U[k], acc);
          U[i] = acc;
        }
      }
      if (part == 0) {
#pragma unroll
        for (int i = 0; i < 12; ++i) jt.u[i][c] = i < m ? U[i < kMost ? i : 0] * jt.tail[i] : 0.0f;
      }
      for (int i = part; i < nw; i += SHARE) {
        const int row = all + i;
        float o = jt.lead[row] * jt.dots[row][c];
#pragma unroll
        for (int k = 0; k < kMost; ++k) o = k <= m + i ? fmaf(jt.coef[row][k], U[k], o) : o;
        store_scalar<QBF16>(a.out, (row_of(m + i) * a.HV + j.hv) * DV + j.slab * CW + c, o);
      }
      lds_sync();
      // ---- S' of the replayed tokens ----
      const float last = jt.last;
      float ub[3][NCS];
#pragma unroll
      for (int h = 0; h < 3; ++h)
#pragma unroll
        for (int cs = 0; cs < NCS; ++cs) ub[h][cs] = jt.u[4 * h + g][NCS * n16 + cs];
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int key = 32 * s + 8 * (n16 / 4) + 4 * b + n16 % 4;
#pragma unroll
          for (int cs = 0; cs < NCS; ++cs) S[s][b][cs] *= last;
#pragma unroll
          for (int h = 0; h < 3; ++h) {
            if (4 * h < m) {   // uniform
              const float kv = jt.k[4 * h + g][key];
#pragma unroll
              for (int cs = 0; cs < NCS; ++cs)
                S[s][b][cs] = __builtin_amdgcn_mfma_f32_16x16x4f32(kv, ub[h][cs], S[s][b][cs], 0, 0, 0);
            }
          }
        }
      slab_io(std::true_type{});
      return;
    }
  }

  // With few waves the next chunk's inputs are asked for before this one is
  // worked on; with many, that costs the third wave of a SIMD (184 registers
  // for 156: 8-token windows over 96 heads x 256 requests 643 -> 686 us on an
  // fp32 pool, 513 -> 603 on bf16).
  constexpr bool AHEAD = CWT < 32;
  struct Place {
    int st, n;
    int64_t t0;
  };
  const auto place = [&](int done) {
    Place p;
    p.st = done >= j.n[0];               // stream
    const int left = (p.st ? total : j.n[0]) - done;
    p.n = left < kW ? left : kW;
    p.t0 = j.first[p.st] + (p.st ? done - j.n[0] : done);
    return p;
  };
  ChunkIn<DK, DV, CW, QBF16> next;
  Place coming = place(0);
  if constexpr (AHEAD) next.load(a, j, a.src[coming.st], coming.t0, coming.n, coming.st == a.window, lane);
  for (int done = 0; done < total;) {
    const int st = coming.st, n = coming.n;
    const int64_t t0 = coming.t0;
    const bool outputs = st == a.window;
    const bool updates = st == 0 || done + n < total;
    if constexpr (!AHEAD) next.load(a, j, a.src[st], t0, n, outputs, lane);
    ChunkIn<DK, DV, CW, QBF16> cur = next;
    if (done + n < total) {
      coming = place(done + n);
      if constexpr (AHEAD) next.load(a, j, a.src[coming.st], coming.t0, coming.n, coming.st == a.window, lane);
    }
    auto& xw = cur.x;
    auto& vw = cur.v;
    const int tok = n16 % kW;
    const bool live_row = tok < n && (n16 < kW || outputs);
    const int gt = lane % kW;

    // ---- gates: G summed over the 8 lanes of a group of tokens, in fp64 ----
    {
      const float x = cur.gate + bias;
      float gv = a.gate_mode == KDA_GATE_SOFTPLUS ? -amp * softplus_f(x) : a.lower_bound * sigmoid_f(amp * x);
      gv = gv < -200.0f ? -200.0f : gv;   // exp(-200) is 0 in fp32, and sums stay finite
      double sum = gt < n ? static_cast<double>(gv) : 0.0;
      sum += row_shr_f64(sum, 1);
      sum += row_shr_f64(sum, 2);
      sum += row_shr_f64(sum, 4);
      if (lane < kW) {
        const float hi = static_cast<float>(sum);
        sh.g_hi[gt] = hi;
        sh.g_lo[gt] = static_cast<float>(sum - static_cast<double>(hi));
        sh.beta[gt] = gt < n ? sigmoid_f(cur.beta) : 0.0f;
      }
    }

    // ---- rows: norms, k to LDS ----
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int h = 0; h < (QBF16 ? 1 : 2); ++h)
        if (!live_row) xw[s][h] = u32x4{0, 0, 0, 0};
    const auto key_value = [&](int s, int e) {   // key 32 s + 8 g + e
      if constexpr (QBF16) return e % 2 ? __uint_as_float(xw[s][0][e / 2] & 0xffff0000u) : __uint_as_float(xw[s][0][e / 2] << 16);
      else return __uint_as_float(xw[s][e / 4][e % 4]);
    };
    float sq = 0.0f;
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int e = 0; e < 8; ++e) sq = fmaf(key_value(s, e), key_value(s, e), sq);
    sq = swap16_add(sq, sq);
    sq = swap32_add(sq, sq);
    if (lane < 2 * kW) sh.row[n16] = (n16 < kW ? 1.0f : a.scale) * rsqrt_f(sq + a.l2_eps);
    if (n16 < kW && updates) {
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<f32x4*>(&sh.k[n16][32 * s + 8 * g + 4 * h]) =
              f32x4{key_value(s, 4 * h), key_value(s, 4 * h + 1), key_value(s, 4 * h + 2), key_value(s, 4 * h + 3)};
    }

    // ---- Gram matrix of the rows: column n16, rows 4 g + 0..3 ----
    f32x4 gram = {0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      if constexpr (QBF16) {
        const bf16x8 x = __builtin_bit_cast(bf16x8, xw[s][0]);
        gram = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, x, gram, 0, 0, 0);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          gram = __builtin_amdgcn_mfma_f32_16x16x4f32(key_value(s, e), key_value(s, e), gram, 0, 0, 0);
      }
    }

    // ---- rows against the slab ----
    f32x4 dots[NCS];
#pragma unroll
    for (int cs = 0; cs < NCS; ++cs) dots[cs] = f32x4{0, 0, 0, 0};
    // A slab as a bf16 pool holds it goes on the bf16 matrix instruction, the
    // products as exact as on the fp32 one and an eighth of the time.
    if (SBF16 && QBF16 && done == 0) {   // uniform
      if constexpr (SBF16 && QBF16) {
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int cs = 0; cs < NCS; ++cs) {
            dots[cs] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xw[s][0]),
                                                              pack_slab(S[s][0][cs], S[s][1][cs]), dots[cs], 0, 0, 0);
          }
      }
    } else {
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
          for (int cs = 0; cs < NCS; ++cs)
            dots[cs] = __builtin_amdgcn_mfma_f32_16x16x4f32(key_value(s, e), S[s][e / 4][cs][e % 4], dots[cs], 0, 0, 0);
    }

    lds_sync();
    // ---- factors ----
    if (lane < 2 * kW) {
      const float gh = sh.g_hi[tok], gl = sh.g_lo[tok];
      const float eg = exp_f(gh + gl);
      sh.lead[n16] = eg * sh.row[n16] * (n16 < kW ? sh.beta[tok] : 1.0f);
      if (n16 < kW) sh.tail[tok] = sh.row[n16] * decay(sh.g_hi[kW - 1], sh.g_lo[kW - 1], gh, gl);
      if (n16 == kW - 1) sh.last = eg;
    }
    if (n16 < kW) {
      const float gh = sh.g_hi[n16], gl = sh.g_lo[n16], nk = sh.row[n16];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 4 * g + r, i = row % kW;
        const float f = nk * sh.row[row] * decay(sh.g_hi[i], sh.g_lo[i], gh, gl) * gram[r];
        sh.coef[row][n16] = row < kW ? (n16 < i ? f * sh.beta[i] : 0.0f) : (n16 <= i ? f : 0.0f);
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if constexpr (NCS == 2) *reinterpret_cast<float2*>(&sh.dots[4 * g + r][2 * n16]) = make_float2(dots[0][r], dots[1][r]);
      else sh.dots[4 * g + r][n16] = dots[0][r];
    }
    lds_sync();

    // ---- the solve, one column per lane ----
    float U[kW];
#pragma unroll
    for (int i = 0; i < kW; ++i) {
      float v[1];
      vw[i].unpack(v);
      float acc = fmaf(sh.beta[i], v[0], -sh.lead[i] * sh.dots[i][c]);
#pragma unroll
      for (int k = 0; k < i; ++k) acc = fmaf(-sh.coef[i][k], U[k], acc);
      U[i] = i < n ? acc : 0.0f;   // not 0 * U[k], where a token before is not finite
    }
    if (outputs) {
#pragma unroll
      for (int i = 0; i < kW; ++i) {
        float o = sh.lead[kW + i] * sh.dots[kW + i][c];
#pragma unroll
        for (int k = 0; k <= i; ++k) o = fmaf(sh.coef[kW + i][k], U[k], o);
        if (i < n && i / (kW / SHARE) == part)
          store_scalar<QBF16>(a.out, ((t0 + i) * a.HV + j.hv) * DV + j.slab * CW + c, o);
      }
    }
    // ---- S' ----
    if (updates) {
      if (part == 0) {
#pragma unroll
        for (int i = 0; i < kW; ++i) sh.u[i][c] = U[i] * sh.tail[i];
      }
      lds_sync();
      const float last = sh.last;
      float ub[2][NCS];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int cs = 0; cs < NCS; ++cs) ub[h][cs] = sh.u[4 * h + g][NCS * n16 + cs];
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int key = 32 * s + 8 * (n16 / 4) + 4 * b + n16 % 4;
          const float k0 = sh.k[g][key], k1 = sh.k[4 + g][key];
#pragma unroll
          for (int cs = 0; cs < NCS; ++cs) {
            f32x4 acc = S[s][b][cs] * last;
            acc = __builtin_amdgcn_mfma_f32_16x16x4f32(k0, ub[0][cs], acc, 0, 0, 0);
            S[s][b][cs] = __builtin_amdgcn_mfma_f32_16x16x4f32(k1, ub[1][cs], acc, 0, 0, 0);
          }
        }
    }
    done += n;
    if (st == 0 && done == j.n[0]) slab_io(std::true_type{});
    lds_sync();
  }
}

// ---------------------------------------------------------------------------
// dispatch
// ---------------------------------------------------------------------------

// Half tokens per request (on average) from which a window goes 8 tokens at a
// time (window_chunk) rather than token by token.  dk = dv = 128, bf16 q, k, v,
// us token by token / 8 at a time, for 2, 4 and 8 tokens per request over 96
// heads x 256 requests:
//   decode  f32 key-first      544 / 556    550 / 561    612 / 597
//           f32 value-first    559 / 637    558 / 668    618 / 717
//           bf16 key-first     337 / 338    361 / 355    533 / 386
//           bf16 value-first   285 / 322    328 / 338    527 / 367
//   window  f32 key-first      542 / 582    569 / 596    786 / 631
//           f32 value-first    559 / 660    579 / 691    848 / 748
//           bf16 key-first     351 / 422    466 / 435    743 / 462
//           bf16 value-first   310 / 417    456 / 430    755 / 457
// 1..8 tokens over 32 heads x 128 requests, bf16: 79 / 65 and 72 / 62 us.  A
// value-first slab is read in 64-byte pieces of 16 rows here (256 or 512 bytes
// of a row token by token); with the touched-once hint on them the fp32 pool's
// 637 us are 682 and the bf16 pool's 322 are 407.
// Replay and window at once (for requests where they fit) hold 236 registers
// for 156, which a bf16 pool's short windows gain by and an fp32 pool's do not
// (96 heads x 256 requests, 4 tokens: bf16 value-first 430 -> 386, key-first
// 435 -> 390; fp32 key-first 596 -> 751); windows of 8 do not fit (457 -> 570).
// The fp32 value-first decode crosses at 12 tokens: 269 / 268 us at 12 and 331 / 277
// at 16, over 32 heads x 256 requests.  Narrower keys cross earlier, as a token's
// set-up is the same for less of a slab; 32 heads x 512 requests, dk = dv = 64 and,
// after the bar, 32, for 2, 4 and 8 tokens:
//   decode  f32 key-first     103 / 103  109 / 105  133 / 106 |  26 /  31   35 /  32   50 /  33
//           f32 value-first   101 / 107  105 / 109  135 / 120 |  29 /  32   35 /  32   53 /  34
//           bf16 key-first     50 /  50   70 /  52  120 /  56 |  20 /  20   31 /  20   54 /  22
//           bf16 value-first   55 /  52   73 /  54  113 /  58 |  18 /  20   26 /  21   44 /  22
//   window  f32 key-first     103 / 112  120 / 115  178 / 119 |  33 /  38   45 /  39   74 /  41
//           f32 value-first   101 / 129  119 / 133  185 / 142 |  34 /  40   46 /  41   77 /  43
//           bf16 key-first     64 /  61  102 /  67  182 /  89 |  29 /  24   47 /  27   84 /  34
//           bf16 value-first   67 /  62   98 /  68  168 /  89 |  24 /  25   38 /  27   67 /  34
// and dk = 64, dv = 128, value-first: decode f32 195 / 232 and 263 / 252 for 4 and 8
// tokens, bf16 104 / 123 and 137 / 125 for 2 and 4; window bf16 128 / 145 and 191 / 158.
// Few waves (up to half a wave per SIMD) take 16 columns each, replay and
// window at once, and are bound by the chain of latencies; 32 heads x 4
// requests, fp32 pool value-first, token by token / 8 at a time / at once:
//   decode  2: 5.6 / 7.5   4: 7.7 / 7.8   8: 11.5 / 8.1
//   window  2: 7.4 / 9.9 / 8.5   4: 11.1 / 10.1 / 8.8   8: 18.8 / 10.5
constexpr int64_t kFewWaves = 512;   // 32-column waves: half a wave per SIMD
constexpr int64_t kJointTo = 11;     // half tokens of a window

// Slabs in flight.  With one or two tokens a wave is a read, a little work and
// a write, and a CU that holds 16 such waves mixes the reads and writes of too
// many 16 KB slabs; LDS that nothing uses holds it to 8 or 6 of them.  No claim
// / 13000 / 16000 / 23000 bytes, dk = dv = 128, us:
//   f32 key-first, 96 heads x 256 requests, 1 token    534 / 526 / 521 / 512
//   f32 value-first                                    558 / 558 / 547 / 532
//   f32 key-first, 32 heads x 128 requests, 1 token    102 /  95 /  92 /  90
//   f32 key-first, 96 heads x 256 requests, 2 tokens   543 / 528 / 526 / 522
//   f32 key-first, the same, 4 tokens                  551 / 542 / 546 / 567
//   bf16 key-first, 96 x 256, 1 token                  331 / 316 / 309 / 312
//   bf16 value-first                                   275 / 261 / 258 / 267
//   bf16 key-first, 32 x 128, 1 token                 54.6 /55.0 /54.2 /56.6
//   bf16 key-first, 32 x 32, 1 token                  11.9 /14.4 /14.6 /15.7
//   a window of 2 on f32 key-first, 96 x 256           541 / 528 / 527 / 538
//   per-channel window of 1, f32 key-first             542 / 527 / 525 / 540
// and where the rules begin, 32 heads (no claim / 16000 / 23000):
//   f32 key-first, value-first, 1 token, 2048 waves    11.7 / 11.7 / 12.2,   9.9 /  9.9 / 11.5
//                                        4096 waves    25.4 / 25.0 / 23.7,  23.7 / 23.9 / 23.1
//                                        8192 waves    52.8 / 48.3 / 46.5,  48.9 / 48.1 / 47.1
//   the same, 2 tokens, 4096 waves                     24.9 / 25.5 / 26.6,  24.1 / 24.6 / 25.8
//                       8192 waves                     52.8 / 49.5 / 49.5,  49.7 / 49.5 / 49.3
//   per-channel window of 1, 4096 waves                26.4 / 25.8 / 26.8,  25.7 / 26.2 / 25.6
//                            8192 waves                53.3 / 48.9 / 49.6,  51.4 / 49.7 / 49.0
//   bf16, 1 token, 12288 waves                         30.8 / 31.8 / 33.4,  37.2 / 36.8 / 39.2
//                  16384 waves                         40.6 / 41.0 / 42.9,  49.3 / 48.3 / 50.8
//                  32768 waves                         108  / 102  / 108,   95.5 / 90.5 / 93.9
// Longer windows and bf16 pools beyond one token are bound by the waves' own
// work and lose by it (window of 4, f32 key-first, 572 / 603 / 641 / 709), and
// so do launches of a few waves per CU, whose last waves then wait (2 tokens,
// f32 value-first, 20 x 32 heads, 2560 waves: 13.9 none, 17.3 with 16000).
template <int DK, int DV, bool SBF16>
uint32_t idle_lds(const WindowArgs& args, int64_t nwg) {
  if (DK != 128 || DV < 32) return 0;
  const int64_t T = args.src[args.window].T, B = args.B;
  if (SBF16) return !kChannel && !args.window && T <= B && nwg >= 16384 ? 16000 : 0;
  if (T <= B && !kChannel) return nwg >= 4096 ? 23000 : 0;
  return T <= (kChannel ? 1 : 2) * B && nwg >= 8192 ? 16000 : 0;
}

template <int DK, bool SBF16, int LAYOUT>
constexpr int64_t chunk_from(int window) {
  if (DK < 128) {
    if (SBF16) return LAYOUT == KDA_STATE_V_FIRST ? (window ? 6 : 7) : (window ? 4 : 6);
    return DK == 64 && LAYOUT == KDA_STATE_V_FIRST ? (window ? 12 : 14) : 8;
  }
  if (SBF16) return window ? 6 : LAYOUT == KDA_STATE_V_FIRST ? 9 : 8;
  return LAYOUT == KDA_STATE_V_FIRST ? (window ? 14 : 24) : (window ? 10 : 12);
}

template <int DK, int DV, bool QBF16, bool SBF16, int LAYOUT>
hipError_t launch_one(const WindowArgs& args, hipStream_t stream) {
  constexpr int CW = DV < 32 ? DV : 32;
  int64_t nwg = static_cast<int64_t>(args.B) * args.HV * (DV / CW);
  uint32_t lds = idle_lds<DK, DV, SBF16>(args, nwg);
  void* kargs[] = {const_cast<WindowArgs*>(&args)};
  const void* fn = LAYOUT == KDA_STATE_K_FIRST ? reinterpret_cast<const void*>(&window_kfirst<DK, DV, QBF16, SBF16>)
                                               : reinterpret_cast<const void*>(&window_vfirst<DK, DV, QBF16, SBF16>);
  if constexpr (!kChannel && DK >= 32) {
    const bool few = nwg <= kFewWaves;
    const int64_t halves = 2 * static_cast<int64_t>(args.src[args.window].T), B = args.B;
    if (few ? halves >= (args.window ? 5 : 8) * B : halves >= chunk_from<DK, SBF16, LAYOUT>(args.window) * B) {
      lds = 0;
      if (few) {
        fn = reinterpret_cast<const void*>(&window_chunk<DK, DV, QBF16, SBF16, LAYOUT, 16, true>);
        if (DV >= 32) nwg *= 2;
      } else if (SBF16 && args.window && halves <= kJointTo * B) {
        fn = reinterpret_cast<const void*>(&window_chunk<DK, DV, QBF16, SBF16, LAYOUT, 32, SBF16>);
      } else {
        fn = reinterpret_cast<const void*>(&window_chunk<DK, DV, QBF16, SBF16, LAYOUT, 32, false>);
      }
    }
  }
  return hipLaunchKernel(fn, dim3(static_cast<uint32_t>(nwg)), dim3(kWave), kargs, lds, stream);
}

using LaunchFn = hipError_t (*)(const WindowArgs&, hipStream_t);

template <int DK, int DV, bool QBF16, bool SBF16>
LaunchFn pick_layout(int layout) {
  return layout == KDA_STATE_V_FIRST ? &launch_one<DK, DV, QBF16, SBF16, KDA_STATE_V_FIRST>
                                     : &launch_one<DK, DV, QBF16, SBF16, KDA_STATE_K_FIRST>;
}

template <int DK, int DV>
LaunchFn pick(bool qbf16, bool sbf16, int layout) {
  if (qbf16) return sbf16 ? pick_layout<DK, DV, true, true>(layout) : pick_layout<DK, DV, true, false>(layout);
  return sbf16 ? pick_layout<DK, DV, false, true>(layout) : pick_layout<DK, DV, false, false>(layout);
}

template <int DK>
LaunchFn pick_dv(int dv, bool qbf16, bool sbf16, int layout) {
  switch (dv) {
    case 16: return pick<DK, 16>(qbf16, sbf16, layout);
    case 32: return pick<DK, 32>(qbf16, sbf16, layout);
    case 64: return pick<DK, 64>(qbf16, sbf16, layout);
    case 128: return pick<DK, 128>(qbf16, sbf16, layout);
    default: return nullptr;
  }
}

}  // namespace

template <>
int launch_window_gate<kChannel>(const WindowArgs& args, int dk, int dv, bool qkv_bf16, bool state_bf16,
                                 int state_layout, hipStream_t stream) {
  LaunchFn fn = nullptr;
  switch (dk) {
    case 16: fn = pick_dv<16>(dv, qkv_bf16, state_bf16, state_layout); break;
    case 32: fn = pick_dv<32>(dv, qkv_bf16, state_bf16, state_layout); break;
    case 64: fn = pick_dv<64>(dv, qkv_bf16, state_bf16, state_layout); break;
    case 128: fn = pick_dv<128>(dv, qkv_bf16, state_bf16, state_layout); break;
    default: break;
  }
  if (fn == nullptr) return KDA_ERR_UNSUPPORTED;
  return fn(args, stream) == hipSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}

}  // namespace kda
