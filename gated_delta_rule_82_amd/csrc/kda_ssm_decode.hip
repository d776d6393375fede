// kda_ssm_decode.hip - the selective state space scan token by token
// (kda_ssm_decode), with its short causal convolution in front.
//
// ssm_decode: one workgroup per (request, value head, up to 64 value
// columns).  Its waves hold 16 columns of the state each, dk / 16 pieces of
// four values per lane, in the pool's own order: key-first a lane has four
// columns of every 16th row, value-first four keys of some rows.  The state is
// fetched once, advanced through the request's tokens in fp32 and written
// once.  Per token every thread convolves one or two of the head's channels
// (x) or its group's (B and C), which meet in LDS, double-buffered so that one
// barrier per token is enough; C^T S is summed over the wave's lanes.
// ssm_windows: behind it, the new windows.  Every head of a group reads its
// window of B and C, so no workgroup of the first kernel may write it.
//
// Bound: HBM, the state's way in and out.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "kda.h"
#include "kda_device.h"
#include "kda_internal.h"
#include "kda_ssm.h"
#include "kda_tile.h"

namespace kda {
namespace {

template <int DK, int DV, bool BF16, bool SBF16, bool VFIRST>
struct Shape {
  static constexpr int COLS = DV < 64 ? DV : 64;        // value columns of a workgroup
  static constexpr int SLABS = DV / COLS;
  static constexpr int THREADS = COLS * 4;              // 16 columns per wave
  static constexpr int CHANNELS = COLS + 2 * DK;        // convolved by a workgroup: x, B, C
  static constexpr int PER = (CHANNELS + THREADS - 1) / THREADS;
  static constexpr int R = DK / 16;                     // pieces of four values per lane
  static constexpr int LANES = DK / 4;                  // value-first: lanes of a row
  static constexpr int ELEM = SBF16 ? 2 : 4;
};

template <int DK, int DV, bool BF16, bool SBF16, bool VFIRST>
__global__ void __launch_bounds__((Shape<DK, DV, BF16, SBF16, VFIRST>::THREADS)) ssm_decode(SsmArgs a) {
  using S = Shape<DK, DV, BF16, SBF16, VFIRST>;
  using IO = StateIO<SBF16, 4>;
  constexpr int R = S::R, PER = S::PER;
  __shared__ __attribute__((aligned(16))) float conv[2][S::CHANNELS];

  const int slab = blockIdx.x % S::SLABS;
  const int head = blockIdx.x / S::SLABS;
  const int hv = head % a.HV, b = head / a.HV;
  const Range range = request_range(a, b);
  if (range.n == 0) return;
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int slot = request_slot(a, b);
  const int64_t out_row = static_cast<int64_t>(a.HV) * DV;
  int64_t out_at = static_cast<int64_t>(range.t0) * out_row + static_cast<int64_t>(hv) * DV + slab * S::COLS;
  if (slot < 0) {
    for (int i = tid; i < S::COLS; i += S::THREADS)
      for (int t = 0; t < range.n; ++t) store_scalar<BF16>(a.out, out_at + t * out_row + i, 0.0f);
    return;
  }

  // the lane's pieces: rows (key-first: keys; value-first: values) row0 +
  // i * STEP, values col .. col + 3 of them
  const int first = wave * 16 + slab * S::COLS;         // first of the wave's value columns
  constexpr int STEP = VFIRST ? kWave / S::LANES : 16;
  const int row0 = VFIRST ? first + lane / S::LANES : lane >> 2;
  const int col = VFIRST ? (lane % S::LANES) * 4 : first + (lane & 3) * 4;
  constexpr int WIDTH = VFIRST ? DK : DV;
  const int64_t tile = (static_cast<int64_t>(slot) * a.HV + hv) * DK * DV;
  const __amdgpu_buffer_rsrc_t pool =
      tile_resource(static_cast<char*>(a.state_pool) + tile * S::ELEM, DK * DV * S::ELEM);
  const int voff = (row0 * WIDTH + col) * S::ELEM;
  float s[R][4];
#pragma unroll
  for (int i = 0; i < R; ++i) IO::load(pool, voff, i * STEP * WIDTH * S::ELEM, s[i]);

  // the thread's channels: taps, and the inputs before the next token
  const int h = hv / a.G;
  Taps taps[PER];
  float past[PER][kPast];
  int channel[PER];
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    const int i = tid + p * S::THREADS;
    const int keys = a.HV * DV + h * DK;
    int c = i < S::COLS ? hv * DV + slab * S::COLS + i
                        : (i < S::COLS + DK ? keys + (i - S::COLS) : keys + a.H * DK + (i - S::COLS - DK));
    if (i >= S::CHANNELS) c = hv * DV;      // a channel of the head, convolved for nothing
    channel[p] = c;
    taps[p].load(a, c);
#pragma unroll
    for (int j = 0; j < kPast; ++j) {
      const int r = j - (kTaps - a.K);
      past[p][j] = r >= 0 ? a.conv_win[(static_cast<int64_t>(slot) * (a.K - 1) + r) * a.C + c] : 0.0f;
    }
  }
  const float amp = exp_f(a.a_log[hv]), bias = a.dt_bias[hv];
  const bool skips = a.d_skip != nullptr;
  const float skip = skips ? a.d_skip[hv] : 0.0f;

  int64_t in_at = static_cast<int64_t>(range.t0) * a.C;
  const float* dt = a.dt + static_cast<int64_t>(range.t0) * a.HV + hv;
  float next[PER];
#pragma unroll
  for (int p = 0; p < PER; ++p) next[p] = load_scalar<BF16>(a.xbc, in_at + channel[p]);
  for (int t = 0; t < range.n; ++t) {
    float* const buf = conv[t & 1];
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      const float y = taps[p].dot(a.K, past[p][0], past[p][1], past[p][2], next[p]);
      past[p][0] = past[p][1];
      past[p][1] = past[p][2];
      past[p][2] = next[p];
      const int i = tid + p * S::THREADS;
      if (i < S::CHANNELS) buf[i] = silu_f(y);
    }
    const float step = softplus_f(*dt + bias);
    const float decay = exp_f(-amp * step);
    if (t + 1 < range.n) {
      in_at += a.C;
      dt += a.HV;
#pragma unroll
      for (int p = 0; p < PER; ++p) next[p] = load_scalar<BF16>(a.xbc, in_at + channel[p]);
    }
    __syncthreads();
    const float* const x = buf;
    const float* const kb = buf + S::COLS;
    const float* const kc = kb + DK;
    if constexpr (VFIRST) {
      const f32x4 bk = *reinterpret_cast<const f32x4*>(kb + col);
      const f32x4 ck = *reinterpret_cast<const f32x4*>(kc + col);
      float y[R];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float w = step * x[row0 - slab * S::COLS + i * STEP];
        y[i] = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[i][e] = fmaf(bk[e], w, decay * s[i][e]);
          y[i] = fmaf(ck[e], s[i][e], y[i]);
        }
      }
      // lanes of a row: the upper bits pick the piece, the two lowest are summed
      constexpr int TOP = log2_exact<S::LANES>() - 1;
      transpose_levels<R / 2, TOP>(y, lane);
      const float sum = sum_levels<1, 0>(y[0]);
      const int v = row0 - slab * S::COLS + ((lane % S::LANES) >> 2) * STEP;
      if ((lane & 3) == 0) store_scalar<BF16>(a.out, out_at + v, skips ? fmaf(skip, x[v], sum) : sum);
    } else {
      const f32x4 xv = *reinterpret_cast<const f32x4*>(x + col - slab * S::COLS);
      float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float w = step * kb[row0 + i * STEP], ck = kc[row0 + i * STEP];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[i][e] = fmaf(w, xv[e], decay * s[i][e]);
          y[e] = fmaf(ck, s[i][e], y[e]);
        }
      }
      // lanes of a column group differ in bits 2..5: bits 5 and 4 pick the column
      transpose_levels<2, 5>(y, lane);
      const float sum = sum_levels<3, 2>(y[0]);
      const int v = wave * 16 + (lane & 3) * 4 + (lane >> 4 & 1) + (lane >> 5) * 2;
      if ((lane & 12) == 0) store_scalar<BF16>(a.out, out_at + v, skips ? fmaf(skip, x[v], sum) : sum);
    }
    out_at += out_row;
  }
#pragma unroll
  for (int i = 0; i < R; ++i) IO::store(pool, voff, i * STEP * WIDTH * S::ELEM, s[i]);
}

// The last K-1 inputs of every request, one thread per (request, channel).
template <bool BF16>
__global__ void __launch_bounds__(256) ssm_windows(SsmArgs a) {
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (at >= static_cast<int64_t>(a.B) * a.C) return;
  const int b = static_cast<int>(at / a.C), c = static_cast<int>(at % a.C);
  const Range range = request_range(a, b);
  const int slot = request_slot(a, b);
  if (slot < 0 || range.n == 0) return;
  float* const win = a.conv_win + static_cast<int64_t>(slot) * (a.K - 1) * a.C + c;
  float x[kPast];
  for (int j = 0; j < a.K - 1; ++j) {
    const int t = range.n - (a.K - 1) + j;      // of the request; below zero: of the old window
    x[j] = t >= 0 ? load_scalar<BF16>(a.xbc, (static_cast<int64_t>(range.t0) + t) * a.C + c)
                  : win[static_cast<int64_t>(a.K - 1 + t) * a.C];
  }
  for (int j = 0; j < a.K - 1; ++j) win[static_cast<int64_t>(j) * a.C] = x[j];
}

template <int DK, int DV, bool BF16, bool SBF16, bool VFIRST>
hipError_t launch(const SsmArgs& args, hipStream_t stream) {
  using S = Shape<DK, DV, BF16, SBF16, VFIRST>;
  void* kargs[] = {const_cast<SsmArgs*>(&args)};
  const uint32_t blocks = static_cast<uint32_t>(args.B) * static_cast<uint32_t>(args.HV) * S::SLABS;
  hipError_t rc = hipLaunchKernel(reinterpret_cast<const void*>(&ssm_decode<DK, DV, BF16, SBF16, VFIRST>),
                                  dim3(blocks), dim3(S::THREADS), kargs, 0, stream);
  if (rc != hipSuccess) return rc;
  const int64_t channels = static_cast<int64_t>(args.B) * args.C;
  return hipLaunchKernel(reinterpret_cast<const void*>(&ssm_windows<BF16>),
                         dim3(static_cast<uint32_t>((channels + 255) / 256)), dim3(256), kargs, 0, stream);
}

template <int DK, int DV>
hipError_t launch(const SsmArgs& args, bool bf16, bool state_bf16, bool v_first, hipStream_t stream) {
  switch ((bf16 ? 4 : 0) | (state_bf16 ? 2 : 0) | (v_first ? 1 : 0)) {
    case 0: return launch<DK, DV, false, false, false>(args, stream);
    case 1: return launch<DK, DV, false, false, true>(args, stream);
    case 2: return launch<DK, DV, false, true, false>(args, stream);
    case 3: return launch<DK, DV, false, true, true>(args, stream);
    case 4: return launch<DK, DV, true, false, false>(args, stream);
    case 5: return launch<DK, DV, true, false, true>(args, stream);
    case 6: return launch<DK, DV, true, true, false>(args, stream);
    default: return launch<DK, DV, true, true, true>(args, stream);
  }
}

}  // namespace

int launch_ssm_decode(const SsmArgs& args, int dk, int dv, bool bf16, bool state_bf16, int state_layout,
                      hipStream_t stream) {
  const bool v_first = state_layout == KDA_STATE_V_FIRST;
  hipError_t rc = hipErrorInvalidValue;
#define KDA_SSM_CASE(K, V) \
  if (dk == K && dv == V) rc = launch<K, V>(args, bf16, state_bf16, v_first, stream);
  KDA_SSM_CASE(32, 32)
  KDA_SSM_CASE(32, 64)
  KDA_SSM_CASE(32, 128)
  KDA_SSM_CASE(64, 32)
  KDA_SSM_CASE(64, 64)
  KDA_SSM_CASE(64, 128)
  KDA_SSM_CASE(128, 32)
  KDA_SSM_CASE(128, 64)
  KDA_SSM_CASE(128, 128)
#undef KDA_SSM_CASE
  return rc == hipSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}

}  // namespace kda
