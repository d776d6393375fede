// kda_ssm.h - what the kernels of the selective state space scan share: a
// request's token range, the taps of the causal convolution and its
// activation.  Included by the .hip sources only; everything has internal
// linkage.
#ifndef KDA_SSM_H_
#define KDA_SSM_H_

#include <hip/hip_runtime.h>

#include <cstdint>

#include "kda_device.h"
#include "kda_internal.h"
#include "kda_tile.h"

namespace kda {
namespace {

constexpr int kTaps = 4;                // most taps
constexpr int kPast = kTaps - 1;        // inputs before a token that its taps reach
constexpr int kSsmChunk = KDA_SSM_CHUNK;

// Tokens of request b, clamped to [0, T].
struct Range {
  int t0, n;
};

__device__ __forceinline__ Range request_range(const SsmArgs& a, int b) {
  int t0 = a.cu_seqlens[b], t1 = a.cu_seqlens[b + 1];
  t0 = t0 < 0 ? 0 : (t0 > a.T ? a.T : t0);
  t1 = t1 < t0 ? t0 : (t1 > a.T ? a.T : t1);
  return {t0, t1 - t0};
}

// Slot of request b, or -1 where it is skipped.
__device__ __forceinline__ int request_slot(const SsmArgs& a, int b) {
  const int s = a.state_indices[b];
  return s < 0 || s >= a.N ? -1 : s;
}

// One channel's taps, newest last; w[kTaps - K ..] are used.
struct Taps {
  float w[kTaps], bias;

  template <bool WBF16>
  __device__ __forceinline__ void load_as(const SsmArgs& a, int c) {
#pragma unroll
    for (int j = 0; j < kTaps; ++j) {
      const int tap = j - (kTaps - a.K);
      w[j] = tap >= 0 ? load_scalar<WBF16>(a.conv_w, static_cast<int64_t>(tap) * a.C + c) : 0.0f;
    }
    bias = a.conv_b != nullptr ? load_scalar<WBF16>(a.conv_b, c) : 0.0f;
  }

  // Inputs oldest first.  Taps that are not there are left out, not
  // multiplied by zero: their inputs may be infinite.
  __device__ __forceinline__ float dot(int K, float x0, float x1, float x2, float x3) const {
    float y = bias;
    if (K > 3) y = fmaf(w[0], x0, y);
    if (K > 2) y = fmaf(w[1], x1, y);
    y = fmaf(w[2], x2, y);
    return fmaf(w[3], x3, y);
  }
};

// Taps of N channels c[0], c[1], ..: one choice of the type, then all loads.
template <int N>
__device__ __forceinline__ void load_taps(const SsmArgs& a, const int (&c)[N], Taps (&taps)[N]) {
  if (a.w_bf16) {
#pragma unroll
    for (int n = 0; n < N; ++n) taps[n].template load_as<true>(a, c[n]);
  } else {
#pragma unroll
    for (int n = 0; n < N; ++n) taps[n].template load_as<false>(a, c[n]);
  }
}

// x * sigmoid(x); exp(-x) = inf for very negative x gives x * 0 = -0.
__device__ __forceinline__ float silu_f(float x) { return x * sigmoid_f(x); }

}  // namespace
}  // namespace kda

#endif  // KDA_SSM_H_
