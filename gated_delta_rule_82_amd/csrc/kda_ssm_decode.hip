// kda_ssm_decode.hip - the selective state space scan token by token
// (kda_ssm_decode), with its short causal convolution in front.
//
// ssm_decode: one workgroup of four waves (two for dv = 32) per (request, value
// head).  A lane moves its state in 16-byte pieces of the pool's own rows:
// value-first a wave holds its share of the rows of dk keys, key-first the rows
// of its share of the keys.  The state is fetched once, advanced through the
// request's tokens in fp32 and written once.  Per token every thread convolves
// one to three of the head's channels (x) or its group's (B and C), which meet
// in LDS, double-buffered so that one barrier per token is enough.  C^T S is
// summed over the wave's lanes; key-first the waves' parts are added behind
// the next token's barrier.  It sets the window of its own channels of x.
// ssm_windows: behind it, the new windows of B and C.  Every head of a group
// reads them, so no workgroup of the first kernel may write them.
//
// Bound: HBM, the state's way in and out: 256 requests of 64 heads (dk = 128,
// dv = 64, fp32 pool, 1.1 GB moved) 195 us, 5.7 TB/s; one request of 64 heads
// is bound by latency, 6.7 us in the two kernels.

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
  static constexpr int WAVES = DV < 64 ? 2 : 4;
  static constexpr int OWN = DV / WAVES;                // value-first: a wave's rows
  static constexpr int THREADS = WAVES * kWave;
  static constexpr int CHANNELS = DV + 2 * DK;          // convolved by a workgroup: x, B, C
  static constexpr int PER = (CHANNELS + THREADS - 1) / THREADS;
  static constexpr int ELEM = SBF16 ? 2 : 4;
  static constexpr int VEC = 16 / ELEM;                 // values per piece
  static constexpr int LANES = (VFIRST ? DK : DV) / VEC;    // of a row
  static constexpr int STEP = kWave / LANES;            // rows of a wave's piece
  static constexpr int R = (VFIRST ? OWN : DK / WAVES) / STEP;   // pieces per lane
  static_assert(R >= 1, "rows of a wave");
};

template <int DK, int DV, bool BF16, bool SBF16, bool VFIRST>
__global__ void __launch_bounds__((Shape<DK, DV, BF16, SBF16, VFIRST>::THREADS)) ssm_decode(SsmArgs a) {
  using S = Shape<DK, DV, BF16, SBF16, VFIRST>;
  using IO = StateIO<SBF16, S::VEC>;
  constexpr int R = S::R, PER = S::PER, VEC = S::VEC;
  __shared__ __attribute__((aligned(16))) float conv[2][S::CHANNELS];
  __shared__ float parts[2][VFIRST ? 1 : S::WAVES][VFIRST ? 1 : DV];

  const int hv = blockIdx.x % a.HV, b = blockIdx.x / a.HV;
  const Range range = request_range(a, b);
  if (range.n == 0) return;
  const int tid = threadIdx.x, lane = tid % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int slot = request_slot(a, b);
  const int64_t out_row = static_cast<int64_t>(a.HV) * DV;
  int64_t out_at = static_cast<int64_t>(range.t0) * out_row + static_cast<int64_t>(hv) * DV;
  if (slot < 0) {
    for (int i = tid; i < DV; i += S::THREADS)
      for (int t = 0; t < range.n; ++t) store_scalar<BF16>(a.out, out_at + t * out_row + i, 0.0f);
    return;
  }

  // the lane's pieces: rows row0 + i * STEP (key-first: keys; value-first:
  // columns of the workgroup), values col .. col + VEC - 1 of them
  const int row0 = (VFIRST ? wave * S::OWN : wave * (DK / S::WAVES)) + lane / S::LANES;
  const int col = lane % S::LANES * VEC;
  constexpr int WIDTH = VFIRST ? DK : DV;
  const int64_t tile = (static_cast<int64_t>(slot) * a.HV + hv) * DK * DV;
  const __amdgpu_buffer_rsrc_t pool =
      tile_resource(static_cast<char*>(a.state_pool) + tile * S::ELEM, DK * DV * S::ELEM);
  const int voff = (row0 * WIDTH + col) * S::ELEM;
  float s[R][VEC];
#pragma unroll
  for (int i = 0; i < R; ++i) IO::load(pool, voff, i * S::STEP * WIDTH * S::ELEM, s[i]);

  // the thread's channels: taps, and the inputs before the next token
  const int h = hv / a.G;
  Taps taps[PER];
  float past[PER][kPast];
  int channel[PER];
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    const int i = tid + p * S::THREADS;
    const int keys = a.HV * DV + h * DK;
    int c = i < DV ? hv * DV + i
                        : (i < DV + DK ? keys + (i - DV) : keys + a.H * DK + (i - DV - DK));
    if (i >= S::CHANNELS) c = hv * DV;      // a channel of the head, convolved for nothing
    channel[p] = c;
  }
  load_taps(a, channel, taps);
#pragma unroll
  for (int p = 0; p < PER; ++p) {
#pragma unroll
    for (int j = 0; j < kPast; ++j) {
      const int r = j - (kTaps - a.K);
      past[p][j] = r >= 0 ? a.conv_win[(static_cast<int64_t>(slot) * (a.K - 1) + r) * a.C + channel[p]] : 0.0f;
    }
  }
  const float amp = exp_f(a.a_log[hv]), bias = a.dt_bias[hv];
  const bool skips = a.d_skip != nullptr;
  const float skip = skips ? a.d_skip[hv] : 0.0f;

  // key-first: adds the waves' parts of the token before, whose x is `last`
  auto finish = [&](int t, float last) {
    if (tid < DV) {
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < S::WAVES; ++w) sum += parts[t & 1][VFIRST ? 0 : w][VFIRST ? 0 : tid];
      store_scalar<BF16>(a.out, out_at - out_row + tid, skips ? fmaf(skip, last, sum) : sum);
    }
  };

  int64_t in_at = static_cast<int64_t>(range.t0) * a.C;
  float next[PER], last = 0.0f;
#pragma unroll
  for (int p = 0; p < PER; ++p) next[p] = load_scalar<BF16>(a.xbc, in_at + channel[p]);
  float steps = 0.0f, decays = 0.0f;    // of 64 tokens, one per lane
  for (int t = 0; t < range.n; ++t) {
    if (t % kWave == 0) {
      const int64_t at = static_cast<int64_t>(range.t0) + min(t + lane, range.n - 1);
      steps = softplus_f(a.dt[at * a.HV + hv] + bias);
      decays = steps > 0.0f ? exp_f(-amp * steps) : 1.0f;       // without a step nothing decays, whatever a_log
    }
    const float step = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(steps), t % kWave));
    const float decay = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(decays), t % kWave));
    float* const buf = conv[t & 1];
    float mine = 0.0f;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      const float y = silu_f(taps[p].dot(a.K, past[p][0], past[p][1], past[p][2], next[p]));
      past[p][0] = past[p][1];
      past[p][1] = past[p][2];
      past[p][2] = next[p];
      const int i = tid + p * S::THREADS;
      if (i < S::CHANNELS) buf[i] = y;
      if (p == 0) mine = y;
    }
    if (t + 1 < range.n) {
      in_at += a.C;
#pragma unroll
      for (int p = 0; p < PER; ++p) next[p] = load_scalar<BF16>(a.xbc, in_at + channel[p]);
    }
    __syncthreads();
    const float* const x = buf;
    const float* const kb = buf + DV;
    const float* const kc = kb + DK;
    if constexpr (VFIRST) {
      float bk[VEC], ck[VEC], y[R];
#pragma unroll
      for (int e = 0; e < VEC; e += 4) {
        *reinterpret_cast<f32x4*>(bk + e) = *reinterpret_cast<const f32x4*>(kb + col + e);
        *reinterpret_cast<f32x4*>(ck + e) = *reinterpret_cast<const f32x4*>(kc + col + e);
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float w = step * x[row0 + i * S::STEP];
        y[i] = 0.0f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          s[i][e] = fmaf(bk[e], w, decay * s[i][e]);
          y[i] = fmaf(ck[e], s[i][e], y[i]);
        }
      }
      // lanes of a row: the upper bits pick the piece, the lowest are summed
      constexpr int LOW = log2_exact<S::LANES>() - log2_exact<R>();
      static_assert(LOW >= 0, "lanes of a row");
      if constexpr (R > 1) transpose_levels<R / 2, log2_exact<S::LANES>() - 1>(y, lane);
      const float sum = sum_levels<LOW - 1, 0>(y[0]);
      const int v = row0 + ((lane % S::LANES) >> LOW) * S::STEP;
      if ((lane & ((1 << LOW) - 1)) == 0) store_scalar<BF16>(a.out, out_at + v, skips ? fmaf(skip, x[v], sum) : sum);
    } else {
      if (t > 0) finish(t - 1, last);
      last = mine;
      float xv[VEC], y[VEC];
#pragma unroll
      for (int e = 0; e < VEC; e += 4) *reinterpret_cast<f32x4*>(xv + e) = *reinterpret_cast<const f32x4*>(x + col + e);
#pragma unroll
      for (int e = 0; e < VEC; ++e) y[e] = 0.0f;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float w = step * kb[row0 + i * S::STEP], ck = kc[row0 + i * S::STEP];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          s[i][e] = fmaf(w, xv[e], decay * s[i][e]);
          y[e] = fmaf(ck, s[i][e], y[e]);
        }
      }
      // lanes of a column group: their upper bits pick columns, what is left
      // of them is summed; LEFT columns stay in a lane
      constexpr int BITS = log2_exact<S::STEP>(), LOW = log2_exact<S::LANES>();
      constexpr int LEVELS = BITS < log2_exact<VEC>() ? BITS : log2_exact<VEC>(), LEFT = VEC >> LEVELS;
      static_assert(BITS + LOW == 6 && LEVELS > 0 && (LEFT == 1 || LEVELS == BITS), "lanes of a wave");
      transpose_levels<VEC / 2, 5, LEVELS>(y, lane);
      if constexpr (LEFT == 1) y[0] = sum_levels<5 - LEVELS, LOW>(y[0]);
      if (((lane >> LOW) & ((1 << (BITS - LEVELS)) - 1)) == 0) {
#pragma unroll
        for (int e = 0; e < LEFT; ++e) parts[t & 1][wave][col + (lane >> (6 - LEVELS)) * LEFT + e] = y[e];
      }
    }
    out_at += out_row;
  }
#pragma unroll
  for (int i = 0; i < R; ++i) IO::store(pool, voff, i * S::STEP * WIDTH * S::ELEM, s[i]);
  if constexpr (!VFIRST) {
    __syncthreads();
    finish(range.n - 1, last);
  }
  if (tid < DV) {        // a thread's first channel is of x where it has one
#pragma unroll
    for (int j = 0; j < kPast; ++j) {
      const int r = j - (kTaps - a.K);
      if (r >= 0) a.conv_win[(static_cast<int64_t>(slot) * (a.K - 1) + r) * a.C + channel[0]] = past[0][j];
    }
  }
}

// The last K-1 inputs of B and C of every request, one thread per (request,
// channel).
template <bool BF16>
__global__ void __launch_bounds__(256) ssm_windows(SsmArgs a, uint32_t keys) {
  const uint32_t at = blockIdx.x * 256 + threadIdx.x, b = at / keys;
  if (b >= static_cast<uint32_t>(a.B)) return;
  const int c = a.C - keys + static_cast<int>(at % keys);
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

// LDS that nothing uses holds a CU to three workgroups, so that it mixes the
// reads and writes of fewer states.  No claim / 50000 bytes, fp32 pool, one
// token for each of 256 requests of 64 heads, us:
//   dk = 128, dv = 64 key-first 201 / 195, value-first 202 / 198;
//   64 x 128 200 / 194, 203 / 201; 128 x 128 358 / 347, 358 / 359
//   128 requests 101 / 101, 103 / 101; 102 / 101, 102 / 102; 182 / 178, 182 / 184
//   64 requests (128 x 64, key-first) 52.4 / 53.7, 32 requests 28.5 / 30.5.
// Smaller states lose: 64 x 64 104 / 102, 105 / 106; a bf16 pool's 108 / 130.
// So do workgroups with more to do, 256 requests x 2 tokens 203 / 213, and
// batches of long windows among empty requests, 4 tokens for every fourth of
// 256 59 / 72.  Lengths are not known here: as many tokens as requests are taken
// for one each.
template <int DK, int DV, bool SBF16>
uint32_t idle_lds(const SsmArgs& args, uint32_t blocks) {
  return !SBF16 && DK * DV >= 128 * 64 && args.T == args.B && blocks >= 8192 ? 50000 : 0;
}

template <int DK, int DV, bool BF16, bool SBF16, bool VFIRST>
hipError_t launch(const SsmArgs& args, hipStream_t stream) {
  using S = Shape<DK, DV, BF16, SBF16, VFIRST>;
  void* kargs[] = {const_cast<SsmArgs*>(&args)};
  const uint32_t blocks = static_cast<uint32_t>(args.B) * static_cast<uint32_t>(args.HV);
  hipError_t rc = hipLaunchKernel(reinterpret_cast<const void*>(&ssm_decode<DK, DV, BF16, SBF16, VFIRST>),
                                  dim3(blocks), dim3(S::THREADS), kargs,
                                  idle_lds<DK, DV, SBF16>(args, blocks), stream);
  if (rc != hipSuccess) return rc;
  uint32_t keys = 2 * static_cast<uint32_t>(args.H) * DK;
  void* wargs[] = {const_cast<SsmArgs*>(&args), &keys};
  const uint32_t channels = static_cast<uint32_t>(args.B) * keys;     // below 2^31, as B * C is
  return hipLaunchKernel(reinterpret_cast<const void*>(&ssm_windows<BF16>), dim3((channels + 255) / 256), dim3(256),
                         wargs, 0, stream);
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
  KDA_SSM_SIZES(KDA_SSM_CASE)
#undef KDA_SSM_CASE
  return rc == hipSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}

}  // namespace kda
