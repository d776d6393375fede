// kda_norm.hip - norms before and after a block (kda_norm_residual,
// kda_norm_gate).
//
// A row is read once into registers, in pieces of eight values: 16-byte loads
// of bf16, two of fp32, wherever the row starts (the hardware takes them at
// any element).  LANES threads share a row, from 8 of a wave for one head to a
// workgroup of 1024; the squares are summed in fp32 over lanes and, for more
// than one wave, LDS.  The row is normalised from the registers and written.
//
// Sums of squares that leave fp32's comfortable range are taken again in
// fp64, and the factor is applied in two parts so that it stays a normal
// number; a row that needs it is the same for all of its threads.
//
// Bound: HBM, each tensor once: norm_residual of 16384 rows of 8192 in bf16
// 179 us, 6.0 TB/s; norm_gate, gate first, of 16384 rows of 4096 73 us, 5.5.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "kda.h"
#include "kda_device.h"
#include "kda_internal.h"
#include "kda_tile.h"

namespace kda {
namespace {

constexpr int kVec = 8;

// Vectors at any element.
typedef unsigned int any_u32x4 __attribute__((ext_vector_type(4), aligned(2)));
typedef float any_f32x4 __attribute__((ext_vector_type(4), aligned(4)));

template <bool BF16>
__device__ __forceinline__ void load_piece(const void* base, int64_t off, int count, float (&x)[kVec]) {
  if constexpr (BF16) {
    const uint16_t* const p = static_cast<const uint16_t*>(base) + off;
    if (count >= kVec) {
      const any_u32x4 w = *reinterpret_cast<const any_u32x4*>(p);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[2 * e] = bf16_to_f32(w[e] & 0xffffu);
        x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
      }
      return;
    }
#pragma unroll
    for (int e = 0; e < kVec; ++e) x[e] = e < count ? bf16_to_f32(p[e]) : 0.0f;
  } else {
    const float* const p = static_cast<const float*>(base) + off;
    if (count >= kVec) {
      const any_f32x4 lo = *reinterpret_cast<const any_f32x4*>(p), hi = *reinterpret_cast<const any_f32x4*>(p + 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = lo[e];
        x[e + 4] = hi[e];
      }
      return;
    }
#pragma unroll
    for (int e = 0; e < kVec; ++e) x[e] = e < count ? p[e] : 0.0f;
  }
}

template <bool BF16>
__device__ __forceinline__ void store_piece(void* base, int64_t off, int count, const float (&x)[kVec]) {
  if constexpr (BF16) {
    uint16_t* const p = static_cast<uint16_t*>(base) + off;
    if (count >= kVec) {
      any_u32x4 w;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = f32x2_to_bf16x2_rne(x[2 * e], x[2 * e + 1]);
      *reinterpret_cast<any_u32x4*>(p) = w;
      return;
    }
#pragma unroll
    for (int e = 0; e < kVec; ++e)
      if (e < count) p[e] = static_cast<uint16_t>(f32_to_bf16_rne(x[e]));
  } else {
    float* const p = static_cast<float*>(base) + off;
    if (count >= kVec) {
      const any_f32x4 lo = {x[0], x[1], x[2], x[3]}, hi = {x[4], x[5], x[6], x[7]};
      *reinterpret_cast<any_f32x4*>(p) = lo;
      *reinterpret_cast<any_f32x4*>(p + 4) = hi;
      return;
    }
#pragma unroll
    for (int e = 0; e < kVec; ++e)
      if (e < count) p[e] = x[e];
  }
}

// The row's threads: LANES of a wave, or with kBlock a whole workgroup, whose
// waves meet in LDS.
constexpr int kBlock = 0;
constexpr int kMostWaves = 16;

template <int LANES>
struct Row {
  static constexpr bool WHOLE = LANES == kBlock;
  static constexpr int IN_WAVE = WHOLE ? kWave : LANES;
  static constexpr int MOST = WHOLE ? kMostWaves * kWave : 256;     // threads of a workgroup

  static __device__ __forceinline__ int lane() { return WHOLE ? threadIdx.x : threadIdx.x % IN_WAVE; }
  static __device__ __forceinline__ int lanes() { return WHOLE ? blockDim.x : IN_WAVE; }
  static __device__ __forceinline__ int64_t row() {
    return WHOLE ? static_cast<int64_t>(blockIdx.x)
                 : static_cast<int64_t>(blockIdx.x) * (MOST / IN_WAVE) + threadIdx.x / IN_WAVE;
  }

  // The waves' sums, one per lane of 16, to be summed once more.
  template <typename T>
  static __device__ __forceinline__ T meet(T x) {
    __shared__ T part[kMostWaves];
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kMostWaves;
    __syncthreads();            // the last sums have been read
    if (threadIdx.x % kWave == 0) part[wave] = x;
    __syncthreads();
    return lane < static_cast<int>(blockDim.x / kWave) ? part[lane] : T(0);
  }
  static __device__ __forceinline__ float sum(float x) {
    x = sum_levels<log2_exact<IN_WAVE>() - 1, 0>(x);
    if (WHOLE && blockDim.x > kWave) x = sum_levels<log2_exact<kMostWaves>() - 1, 0>(meet(x));
    return x;
  }
  static __device__ double sum(double x) {
#pragma unroll
    for (int m = 1; m < IN_WAVE; m *= 2) x += __shfl_xor(x, m);
    if (WHOLE && blockDim.x > kWave) {
      x = meet(x);
#pragma unroll
      for (int m = 1; m < kMostWaves; m *= 2) x += __shfl_xor(x, m);
    }
    return x;
  }
};

// 1 / sqrt(mean(x^2) + eps) in two factors, their product the value, the
// first applied first; the second is 1 unless the squares leave fp32.  The
// first of a value below one is below one itself: x may be anything up to
// fp32's largest, and x * f must not pass it (a row of 128 with 3e38 alone has
// the value 2^-125 * 1.604).  From one on x * f * g is at most sqrt(D), and f
// is at least one, so that a small x keeps its bits.
struct Factor {
  float f, g;
  __device__ __forceinline__ float operator()(float x) const { return x * f * g; }
};

template <int LANES, int P>
__device__ __forceinline__ Factor norm_factor(const float (&x)[P][kVec], int D, float eps) {
  float ss = 0.0f;
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int e = 0; e < kVec; ++e) ss = fmaf(x[p][e], x[p][e], ss);
  ss = Row<LANES>::sum(ss);
  if (ss > 0x1p-80f && ss < 0x1p120f) return {1.0f / sqrtf(ss / static_cast<float>(D) + eps), 1.0f};
  double wide = 0.0;
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int e = 0; e < kVec; ++e) wide = fma(static_cast<double>(x[p][e]), static_cast<double>(x[p][e]), wide);
  wide = Row<LANES>::sum(wide);
  const double r = 1.0 / sqrt(wide / D + static_cast<double>(eps));
  if (!(r > 0.0 && r < 1e300)) return {static_cast<float>(r), 1.0f};
  const int e = min(max(ilogb(r) + (r < 1.0 ? 1 : 0), -126), 126);
  return {static_cast<float>(ldexp(r, -e)), ldexpf(1.0f, e)};
}

template <int LANES, int P, bool HBF16, bool BF16>
__global__ void __launch_bounds__(Row<LANES>::MOST) norm_residual(ResidualArgs a) {
  const int lane = Row<LANES>::lane(), lanes = Row<LANES>::lanes();
  const int64_t row = Row<LANES>::row();
  if (row >= a.rows) return;      // whole rows: no lane of one is missing
  const int64_t at = row * a.D;
  float y[P][kVec], h[P][kVec];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int i = (p * lanes + lane) * kVec;
    load_piece<BF16>(a.block_out, at + i, a.D - i, y[p]);
    load_piece<HBF16>(a.hidden, at + i, a.D - i, h[p]);
  }
  if (a.post_weight != nullptr) {
    const Factor r = norm_factor<LANES, P>(y, a.D, a.eps);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int i = (p * lanes + lane) * kVec;
      float w[kVec];
      load_piece<false>(a.post_weight, i, a.D - i, w);
#pragma unroll
      for (int e = 0; e < kVec; ++e) y[p][e] = r(y[p][e]) * w[e];
    }
  }
  const float one = a.scale != nullptr ? a.scale[0] : 1.0f;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int i = (p * lanes + lane) * kVec;
    if (a.scale_per_channel) {
      float s[kVec];
      load_piece<false>(a.scale, i, a.D - i, s);
#pragma unroll
      for (int e = 0; e < kVec; ++e) h[p][e] = fmaf(s[e], y[p][e], h[p][e]);
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e) h[p][e] = fmaf(one, y[p][e], h[p][e]);
    }
    store_piece<HBF16>(a.hidden_out, at + i, a.D - i, h[p]);
  }
  const Factor r = norm_factor<LANES, P>(h, a.D, a.eps);
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int i = (p * lanes + lane) * kVec;
    float w[kVec];
    load_piece<false>(a.weight, i, a.D - i, w);
#pragma unroll
    for (int e = 0; e < kVec; ++e) h[p][e] = r(h[p][e]) * w[e];
    store_piece<BF16>(a.normed, at + i, a.D - i, h[p]);
  }
}

template <int LANES, int P, bool FIRST, bool BF16>
__global__ void __launch_bounds__(Row<LANES>::MOST) norm_gate(GateArgs a) {
  const int lane = Row<LANES>::lane(), lanes = Row<LANES>::lanes();
  const int64_t row = Row<LANES>::row();
  if (row >= a.rows) return;
  const int64_t at = row * a.D;
  float x[P][kVec], z[P][kVec];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int i = (p * lanes + lane) * kVec;
    load_piece<BF16>(a.x, at + i, a.D - i, x[p]);
    load_piece<BF16>(a.gate, at + i, a.D - i, z[p]);
  }
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      z[p][e] = a.silu ? z[p][e] * sigmoid_f(z[p][e]) : sigmoid_f(z[p][e]);
      if constexpr (FIRST) x[p][e] *= z[p][e];
    }
  const Factor r = norm_factor<LANES, P>(x, a.D, a.eps);
  const int64_t group = a.groups > 1 ? row % a.groups * a.D : 0;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int i = (p * lanes + lane) * kVec;
    float w[kVec];
    load_piece<false>(a.weight, group + i, a.D - i, w);
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      x[p][e] = r(x[p][e]) * w[e];
      if constexpr (!FIRST) x[p][e] *= z[p][e];
    }
    store_piece<BF16>(a.out, at + i, a.D - i, x[p]);
  }
}

template <int LANES, int P, bool HBF16, bool BF16>
const void* kernel(const ResidualArgs&) {
  return reinterpret_cast<const void*>(&norm_residual<LANES, P, HBF16, BF16>);
}

template <int LANES, int P, bool FIRST, bool BF16>
const void* kernel(const GateArgs&) {
  return reinterpret_cast<const void*>(&norm_gate<LANES, P, FIRST, BF16>);
}

template <int LANES, int P, bool X, bool BF16, typename Args>
int launch(const Args& args, hipStream_t stream) {
  constexpr bool whole = LANES == kBlock;
  constexpr int rows = whole ? 1 : 256 / (whole ? 1 : LANES);
  const int threads = whole ? (args.D + kVec * P * kWave - 1) / (kVec * P * kWave) * kWave : 256;
  const int64_t blocks = (args.rows + rows - 1) / rows;
  if (blocks * threads * P > UINT32_MAX) return KDA_ERR_UNSUPPORTED;      // a dispatch's work-items
  void* kargs[] = {const_cast<Args*>(&args)};
  const hipError_t rc = hipLaunchKernel(kernel<LANES, P, X, BF16>(args), dim3(static_cast<uint32_t>(blocks)),
                                        dim3(static_cast<uint32_t>(threads)), kargs, 0, stream);
  return rc == hipSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}

// One piece per thread, from eight threads to a workgroup of sixteen waves,
// and two where that does not hold the row.  More pieces per thread are
// slower, as fewer rows are under way: norm_residual, bf16, 16384 rows of 8192
// with 256 threads x 4, 512 x 2, 1024 x 1: 205 / 186 / 179 us; of 4096 with
// 64 x 8, 128 x 4, 256 x 2, 512 x 1: 159 / 109 / 96 / 90 us.
template <bool X, bool BF16, typename Args>
int launch(const Args& args, hipStream_t stream) {
  const int D = args.D;
  if (D <= 8 * kVec) return launch<8, 1, X, BF16>(args, stream);
  if (D <= 16 * kVec) return launch<16, 1, X, BF16>(args, stream);
  if (D <= 64 * kVec) return launch<64, 1, X, BF16>(args, stream);
  if (D <= kMostWaves * kWave * kVec) return launch<kBlock, 1, X, BF16>(args, stream);
  static_assert(KDA_NORM_MAX == kMostWaves * kWave * kVec * 2, "the longest row");
  return launch<kBlock, 2, X, BF16>(args, stream);
}

template <bool X, typename Args>
int launch(const Args& args, bool bf16, hipStream_t stream) {
  return bf16 ? launch<X, true>(args, stream) : launch<X, false>(args, stream);
}

}  // namespace

int launch_norm_residual(const ResidualArgs& args, bool hidden_bf16, bool bf16, hipStream_t stream) {
  return hidden_bf16 ? launch<true>(args, bf16, stream) : launch<false>(args, bf16, stream);
}

int launch_norm_gate(const GateArgs& args, bool gate_first, bool bf16, hipStream_t stream) {
  return gate_first ? launch<true>(args, bf16, stream) : launch<false>(args, bf16, stream);
}

}  // namespace kda
