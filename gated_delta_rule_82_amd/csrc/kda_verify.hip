// kda_verify.hip - verification of drafted tokens (kda_verify).
//
// Two kernels.  verify_sum: every wave first finds how many drafts of its
// request stand (one lane per draft, a ballot), which names the one row s of
// the target (and of the draft) that the next token is sampled from; then it
// sums r = max(p - q, 0) over its segments of that row, one fp64 partial per
// segment of 64 lanes x 4 loads of 16 bytes.  verify_pick: one workgroup per
// request scans the partials, finds the segment in which the running sum
// passes u * total, and one wave scans that segment again.
//
// The sums are fp64 because the answer is an index: an fp32 running sum over
// 10^5 tokens is off by more than many tokens' whole mass.  p, q and u are
// fp32 or bf16, so u * q and p - q are compared without rounding in fp64.
//
// Bound: HBM, one row of each distribution per request (all other rows are
// touched at one token only); with few requests the two launches and the
// chain token -> probability -> row.

#include <hip/hip_runtime.h>

#include <cfloat>
#include <cstdint>

#include "kda.h"
#include "kda_device.h"
#include "kda_internal.h"

namespace kda {
namespace {

constexpr int kLoads = 4;      // 16-byte loads per lane and segment
constexpr int kBlock = 256;
constexpr int kHeld = 4;       // rounds of 64 partials that verify_pick keeps

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

template <bool BF16>
constexpr int kVec = BF16 ? 8 : 4;   // probabilities per load

template <bool BF16>
constexpr int kSegment = kWave * kLoads * kVec<BF16>;
static_assert(kSegment<false> == KDA_VERIFY_SEGMENT, "the workspace formula counts fp32 segments");

// NaN, negative and infinite probabilities count as zero.
__device__ __forceinline__ float mass(float x) { return fmaxf(x <= FLT_MAX ? x : 0.0f, 0.0f); }

template <bool BF16>
__device__ __forceinline__ float load_prob(const void* base, int64_t off) {
  return mass(BF16 ? bf16_to_f32(static_cast<const uint16_t*>(base)[off]) : static_cast<const float*>(base)[off]);
}

// The request's window and what stands of it; uniform over the wave.
struct Verdict {
  int n;          // window tokens
  int kept;       // drafts that stand
  bool fell;      // a draft was rejected
  int64_t row;    // row to sample from
};

__device__ __forceinline__ int window(const VerifyArgs& a, int b, int& n) {   // first row and tokens
  int t0 = a.cu_seqlens[b], t1 = a.cu_seqlens[b + 1];
  t0 = t0 < 0 ? 0 : (t0 > a.T ? a.T : t0);
  t1 = t1 < t0 ? t0 : (t1 > a.T ? a.T : t1);
  n = t1 - t0;
  return t0;
}

template <bool BF16>
__device__ __forceinline__ Verdict judge(const VerifyArgs& a, int b, int lane) {
  Verdict v;
  const int t0 = window(a, b, v.n);
  v.kept = v.n > 0 ? v.n - 1 : 0;
  v.fell = false;
  for (int base = 0; base < v.n - 1; base += kWave) {
    const int i = base + lane;
    bool falls = false;
    if (i < v.n - 1) {
      const int64_t t = t0 + i;
      const int x = a.tokens[t + 1];
      if (x < 0 || x >= a.V) {
        falls = true;
      } else {
        const double p = load_prob<BF16>(a.target, t * a.V + x);
        const double q = a.draft != nullptr ? load_prob<BF16>(a.draft, t * a.V + x) : 1.0f;
        falls = !(static_cast<double>(a.u_accept[t]) * q < p);
      }
    }
    const uint64_t mask = __ballot(falls);
    if (mask != 0) {
      v.kept = base + __ffsll(static_cast<unsigned long long>(mask)) - 1;
      v.fell = true;
      break;
    }
  }
  v.row = static_cast<int64_t>(t0) + v.kept;
  return v;
}

// One row's residual r in units of aligned 16-byte groups: group g holds
// tokens g * kVec - shift + 0 .. kVec - 1, where shift is how far the row
// starts behind a 16-byte boundary (target and draft rows alike).
template <bool BF16>
struct Row {
  static constexpr int VEC = kVec<BF16>;
  const char* p;
  const char* q;      // NULL: nothing to subtract
  int V, shift, gone; // gone: token whose mass is dropped (-1: none)
  int64_t groups;

  __device__ __forceinline__ void open(const VerifyArgs& a, const Verdict& v) {
    constexpr int E = BF16 ? 2 : 4;
    const int64_t off = v.row * a.V;
    V = a.V;
    shift = static_cast<int>(off % VEC);
    groups = (static_cast<int64_t>(shift) + a.V + VEC - 1) / VEC;
    p = static_cast<const char*>(a.target) + (off - shift) * E;
    q = v.fell && a.draft != nullptr ? static_cast<const char*>(a.draft) + (off - shift) * E : nullptr;
    gone = v.fell && a.draft == nullptr ? a.tokens[v.row + 1] : -1;
  }

  __device__ __forceinline__ int64_t token(int64_t g) const { return g * VEC - shift; }

  // Whether all of group g lies in the row, so that it may be loaded whole.
  __device__ __forceinline__ bool whole(int64_t g) const { return token(g) >= 0 && token(g) + VEC <= V; }

  static __device__ __forceinline__ void unpack(u32x4 w, float (&x)[VEC]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (BF16) {
        x[2 * e] = bf16_to_f32(w[e] & 0xffffu);
        x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
      } else {
        x[e] = __uint_as_float(w[e]);
      }
    }
  }

  __device__ __forceinline__ void residual(int64_t g, u32x4 wp, u32x4 wq, double (&r)[VEC]) const {
    float x[VEC], y[VEC];
    unpack(wp, x);
    unpack(wq, y);
    const int64_t t = token(g);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const double d = static_cast<double>(mass(x[e])) - static_cast<double>(mass(y[e]));
      r[e] = fmax(d, 0.0);
    }
    if (gone >= t && gone < t + VEC) {
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (t + e == gone) r[e] = 0.0;
    }
  }

  // The groups g, g + 64, ... of a segment, as loaded (groups that reach past
  // the row are left out here).
  struct Raw {
    u32x4 p[kLoads], q[kLoads];
  };

  __device__ __forceinline__ void fetch(int64_t g, Raw& w) const {
#pragma unroll
    for (int l = 0; l < kLoads; ++l) {
      const int64_t at = g + l * kWave;
      w.p[l] = u32x4{0, 0, 0, 0};
      w.q[l] = u32x4{0, 0, 0, 0};
      if (at < groups && whole(at)) {
        w.p[l] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p + at * 16));
        if (q != nullptr) w.q[l] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(q + at * 16));
      }
    }
  }

  // Their r (0 outside the row).
  __device__ __forceinline__ void values(int64_t g, const Raw& w, double (&r)[kLoads][VEC]) const {
#pragma unroll
    for (int l = 0; l < kLoads; ++l) {
      const int64_t at = g + l * kWave;
      if (at < groups && !whole(at)) {   // a row's first or last group
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const int64_t t = token(at) + e;
          double d = 0.0;
          if (t >= 0 && t < V && t != gone) {
            d = load_prob<BF16>(p, at * VEC + e);
            if (q != nullptr) d -= load_prob<BF16>(q, at * VEC + e);
          }
          r[l][e] = fmax(d, 0.0);
        }
      } else {
        residual(at, w.p[l], w.q[l], r[l]);
      }
    }
  }
};

// Moves of a double between lanes: DPP within a row of 16, row swaps across.
template <int CTRL, bool ZERO = false>
__device__ __forceinline__ double dpp_f64(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(u), CTRL, 0xf, 0xf, ZERO);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(u >> 32), CTRL, 0xf, 0xf, ZERO);
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

__device__ __forceinline__ double lane_f64(double x, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(u), lane);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(u >> 32), lane);
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

// Sum of x over lanes 0 .. lane.
__device__ __forceinline__ double wave_scan(double x, int lane) {
  x += dpp_f64<0x111, true>(x);   // row_shr 1, 2, 4, 8: zero comes in
  x += dpp_f64<0x112, true>(x);
  x += dpp_f64<0x114, true>(x);
  x += dpp_f64<0x118, true>(x);
  const double r0 = lane_f64(x, 15), r1 = r0 + lane_f64(x, 31), r2 = r1 + lane_f64(x, 47);
  const int row = lane / 16;
  return x + (row == 0 ? 0.0 : row == 1 ? r0 : row == 2 ? r1 : r2);
}

// Sum over the wave; in lane 0 at least.
__device__ __forceinline__ double wave_total(double x) {
  x += dpp_f64<kDppXor1>(x);
  x += dpp_f64<kDppXor2>(x);
  x += dpp_f64<kDppRowRor4>(x);
  x += dpp_f64<kDppRowRor8>(x);
  return (x + lane_f64(x, 16)) + (lane_f64(x, 32) + lane_f64(x, 48));
}

__device__ __forceinline__ int64_t segments(int V, int segment) { return V / segment + 2; }

// One wave per `run` segments of one request.
template <bool BF16>
__global__ __launch_bounds__(kBlock) void verify_sum(const VerifyArgs a, int blocks_per_request, int run) {
  const int lane = threadIdx.x % kWave;
  const int b = blockIdx.x / blocks_per_request;
  const int64_t first = (static_cast<int64_t>(blockIdx.x % blocks_per_request) * (kBlock / kWave) +
                         threadIdx.x / kWave) * run;
  const Verdict v = judge<BF16>(a, b, lane);
  if (first == 0 && lane == 0) {
    a.n_commit[b] = v.n > 0 ? v.kept + 1 : 0;
  }
  if (v.n == 0) return;
  Row<BF16> row;
  row.open(a, v);
  const int64_t nseg = segments(a.V, kSegment<BF16>);
  double* const part = static_cast<double*>(a.workspace) + b * nseg;
  const int64_t end = first + run < nseg ? first + run : nseg;
  typename Row<BF16>::Raw next;
  row.fetch(first * (kWave * kLoads) + lane, next);   // past the row: nothing
  for (int64_t s = first; s < end; ++s) {
    const int64_t g = s * (kWave * kLoads) + lane;
    const typename Row<BF16>::Raw cur = next;
    if (s + 1 < end) row.fetch(g + kWave * kLoads, next);
    double r[kLoads][kVec<BF16>];
    row.values(g, cur, r);
    double sum = 0.0;
#pragma unroll
    for (int l = 0; l < kLoads; ++l)
#pragma unroll
      for (int e = 0; e < kVec<BF16>; ++e) sum += r[l][e];
    sum = wave_total(sum);
    if (lane == 0) part[s] = sum;
  }
}

// One wave per request.
template <bool BF16>
__global__ __launch_bounds__(kWave) void verify_pick(const VerifyArgs a) {
  constexpr int VEC = kVec<BF16>;
  const int lane = threadIdx.x;
  const int b = blockIdx.x;
  // All that does not hang on another load is asked for at once; the first
  // kHeld rounds of partials and their sums stay in registers.
  const int64_t nseg = segments(a.V, kSegment<BF16>);
  const double* const part = static_cast<const double*>(a.workspace) + b * nseg;
  double held[kHeld], upto[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) held[i] = i * kWave + lane < nseg ? part[i * kWave + lane] : 0.0;
  const float u = a.u_sample[b];
  const int commit = a.n_commit[b];   // the verdict that verify_sum left
  Verdict v;
  const int t0 = window(a, b, v.n);
  if (v.n == 0) {
    if (lane == 0) a.next_token[b] = -1;
    return;
  }
  v.kept = commit - 1;
  v.fell = v.kept < v.n - 1;
  v.row = static_cast<int64_t>(t0) + v.kept;
  // the total, summed in the order in which the search below adds up
  double total = 0.0;
  int64_t last = -1;   // last segment with mass
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const uint64_t some = __ballot(held[i] > 0.0);
    if (some != 0) last = i * kWave + 63 - __clzll(static_cast<long long>(some));
    upto[i] = wave_scan(held[i], lane);
    total += lane_f64(upto[i], kWave - 1);
  }
  for (int64_t s0 = kHeld * kWave; s0 < nseg; s0 += kWave) {
    const double x = s0 + lane < nseg ? part[s0 + lane] : 0.0;
    const uint64_t some = __ballot(x > 0.0);
    if (some != 0) last = s0 + 63 - __clzll(static_cast<long long>(some));
    total += lane_f64(wave_scan(x, lane), kWave - 1);
  }
  if (last < 0) {
    if (lane == 0) a.next_token[b] = -1;
    return;
  }
  const double bar = (u > 0.0f ? static_cast<double>(u) : 0.0) * total;
  // u of one or more: the last token with mass, whatever the sums round to.
  // Below that, only a segment with mass of its own can pass the bar: each
  // lane's prefix rounds in an order of its own, so that of an empty segment
  // may come out above its neighbours'.
  const bool to_end = u >= 1.0f;
  double before = 0.0;   // mass of the segments before `seg`
  int64_t seg = -1;
  const auto search = [&](int64_t s0, double own, double sums) {
    const uint64_t over = __ballot(own > 0.0 && before + sums > bar);
    if (over != 0) {
      const int at = __ffsll(static_cast<unsigned long long>(over)) - 1;
      seg = s0 + at;
      if (at > 0) before += lane_f64(sums, at - 1);
    } else {
      before += lane_f64(sums, kWave - 1);
    }
  };
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (seg < 0 && !to_end) search(i * kWave, held[i], upto[i]);
  for (int64_t s0 = kHeld * kWave; s0 < nseg && seg < 0 && !to_end; s0 += kWave) {
    const double x = s0 + lane < nseg ? part[s0 + lane] : 0.0;
    search(s0, x, wave_scan(x, lane));
  }
  const bool passes = seg >= 0;   // else the last token with mass
  if (!passes) seg = last;
  Row<BF16> row;
  row.open(a, v);
  double r[kLoads][VEC];
  const int64_t g0 = seg * (kWave * kLoads);
  typename Row<BF16>::Raw raw;
  row.fetch(g0 + lane, raw);
  row.values(g0 + lane, raw, r);
  int64_t found = -1, tail = -1;
#pragma unroll
  for (int l = 0; l < kLoads; ++l) {
    double sum = 0.0;
    int some = -1;   // the lane's last element with mass
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      sum += r[l][e];
      if (r[l][e] > 0.0) some = e;
    }
    const double upto = wave_scan(sum, lane);
    double run = before + (upto - sum);   // may round: a token's own sum decides below
    int at = -1;     // the lane's first element past the bar
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      run += r[l][e];
      if (at < 0 && run > bar && r[l][e] > 0.0) at = e;
    }
    const int64_t t = row.token(g0 + l * kWave + lane);
    const uint64_t over = __ballot(passes && at >= 0);
    if (found < 0 && over != 0) {
      const int who = __ffsll(static_cast<unsigned long long>(over)) - 1;
      found = __shfl(static_cast<int>(t + at), who);
    }
    const uint64_t any = __ballot(some >= 0);
    if (any != 0) tail = __shfl(static_cast<int>(t + some), 63 - __clzll(static_cast<long long>(any)));
    before += lane_f64(upto, kWave - 1);
  }
  // a segment whose own running sum rounds to the bar gives its last token
  if (lane == 0) a.next_token[b] = static_cast<int32_t>(found >= 0 ? found : tail);
}

template <bool BF16>
hipError_t launch(const VerifyArgs& args, hipStream_t stream) {
  const int64_t nseg = args.V / kSegment<BF16> + 2;
  // Segments per wave: waves for the chip first, then fewer of them, which
  // share the walk over the drafts.  256 requests over 131072 fp32 tokens, us
  // with at least 2048 / 8192 / 16384 / 65536 waves: 54.0 / 49.2 / 51.3 / 59.9.
  int run = 1;
  while (run < 8 && static_cast<int64_t>(args.B) * nseg / (2 * run) >= 8192) run *= 2;
  const int64_t per_block = static_cast<int64_t>(kBlock / kWave) * run;
  int blocks = static_cast<int>((nseg + per_block - 1) / per_block);
  void* sum_args[] = {const_cast<VerifyArgs*>(&args), &blocks, &run};
  hipError_t rc = hipLaunchKernel(reinterpret_cast<const void*>(&verify_sum<BF16>),
                                  dim3(static_cast<uint32_t>(blocks) * static_cast<uint32_t>(args.B)), dim3(kBlock),
                                  sum_args, 0, stream);
  if (rc != hipSuccess) return rc;
  void* pick_args[] = {const_cast<VerifyArgs*>(&args)};
  return hipLaunchKernel(reinterpret_cast<const void*>(&verify_pick<BF16>), dim3(static_cast<uint32_t>(args.B)),
                         dim3(kWave), pick_args, 0, stream);
}

}  // namespace

int launch_verify(const VerifyArgs& args, bool bf16, hipStream_t stream) {
  const hipError_t rc = bf16 ? launch<true>(args, stream) : launch<false>(args, stream);
  return rc == hipSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}

}  // namespace kda
