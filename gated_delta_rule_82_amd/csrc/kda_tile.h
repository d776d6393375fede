// kda_tile.h - what the kernels that keep a state slab in registers share:
// streaming access to a state tile, element loads and stores, and the
// transpose-reduce over the lanes of a wave.  Included by the .hip sources
// only; everything has internal linkage.
#ifndef KDA_TILE_H_
#define KDA_TILE_H_

#include <hip/hip_runtime.h>

#include <cstdint>

#include "kda_device.h"

namespace kda {
namespace {

// ---------------------------------------------------------------------------
// memory
// ---------------------------------------------------------------------------

// The state is streamed through a raw buffer resource spanning exactly the
// tile: per-row offsets stay in scalar registers (one VGPR offset per lane),
// the hardware range check confines every access to the tile, and the
// cache-policy bit "nt" marks the data as touched once.
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
constexpr int kCachePolicyNT = 2;
constexpr int kRawBufferWord3 = 0x00020000;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t tile_resource(void* tile, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(tile, static_cast<short>(0), bytes, kRawBufferWord3);
}

// A lane moves its state in pieces of N consecutive values of one row: N = 4
// fp32 (16 bytes) or N = 4 / 8 bf16 (8 / 16 bytes), widened to fp32 on the
// way in and rounded to nearest-even on the way out.
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

template <bool SBF16, int N, int POLICY = kCachePolicyNT>
struct StateIO {
  static_assert(N == 4 || (SBF16 && N == 8), "state access width");
  static constexpr int kElem = SBF16 ? 2 : 4;
  __device__ static __forceinline__ void load(__amdgpu_buffer_rsrc_t r, int voff, int soff, float* x) {
    if constexpr (SBF16 && N == 8) {
      const u32x4 w = __builtin_amdgcn_raw_buffer_load_b128(r, voff, soff, POLICY);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[2 * e] = bf16_to_f32(w[e] & 0xffffu);
        x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
      }
    } else if constexpr (SBF16) {
      const u32x2 w = __builtin_amdgcn_raw_buffer_load_b64(r, voff, soff, POLICY);
      x[0] = bf16_to_f32(w.x & 0xffffu);
      x[1] = __uint_as_float(w.x & 0xffff0000u);
      x[2] = bf16_to_f32(w.y & 0xffffu);
      x[3] = __uint_as_float(w.y & 0xffff0000u);
    } else {
      const f32x4 w = __builtin_amdgcn_raw_buffer_load_b128(r, voff, soff, POLICY);
      x[0] = w.x;
      x[1] = w.y;
      x[2] = w.z;
      x[3] = w.w;
    }
  }
  __device__ static __forceinline__ void store(__amdgpu_buffer_rsrc_t r, int voff, int soff, const float* x) {
    if constexpr (SBF16 && N == 8) {
      u32x4 w;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = f32x2_to_bf16x2_rne(x[2 * e], x[2 * e + 1]);
      __builtin_amdgcn_raw_buffer_store_b128(w, r, voff, soff, POLICY);
    } else if constexpr (SBF16) {
      const u32x2 w = {f32x2_to_bf16x2_rne(x[0], x[1]), f32x2_to_bf16x2_rne(x[2], x[3])};
      __builtin_amdgcn_raw_buffer_store_b64(w, r, voff, soff, POLICY);
    } else {
      const f32x4 w = {x[0], x[1], x[2], x[3]};
      __builtin_amdgcn_raw_buffer_store_b128(w, r, voff, soff, POLICY);
    }
  }
};

template <int CPL>
__device__ __forceinline__ void load_f32(const float* p, float (&x)[CPL]) {
  if constexpr (CPL == 2) {
    const float2 w = *reinterpret_cast<const float2*>(p);
    x[0] = w.x;
    x[1] = w.y;
  } else {
    x[0] = p[0];
  }
}

template <bool BF16>
__device__ __forceinline__ float load_scalar(const void* base, int64_t off) {
  if constexpr (BF16) return bf16_to_f32(static_cast<const uint16_t*>(base)[off]);
  else return static_cast<const float*>(base)[off];
}

template <bool BF16>
__device__ __forceinline__ void store_scalar(void* base, int64_t off, float x) {
  if constexpr (BF16) static_cast<uint16_t*>(base)[off] = static_cast<uint16_t>(f32_to_bf16_rne(x));
  else static_cast<float*>(base)[off] = x;
}

// Two consecutive values at an even element offset.
template <bool BF16>
__device__ __forceinline__ void store_pair(void* base, int64_t off, float x0, float x1) {
  if constexpr (BF16) *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(base) + off) = f32x2_to_bf16x2_rne(x0, x1);
  else *reinterpret_cast<float2*>(static_cast<float*>(base) + off) = make_float2(x0, x1);
}

// N (1 or 2) consecutive elements of one row, kept in storage form until
// used, so that a load issued a token ahead is waited for only where its
// value is taken.
template <bool BF16, int N>
struct RawRun {
  static constexpr int W = (BF16 && N == 2) ? 1 : N;
  uint32_t w[W];
  __device__ __forceinline__ void load(const void* base, int64_t off) {
    if constexpr (BF16 && N == 2) {
      w[0] = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(base) + off);
    } else if constexpr (BF16) {
      w[0] = static_cast<const uint16_t*>(base)[off];
    } else if constexpr (N == 2) {
      const u32x2 x = *reinterpret_cast<const u32x2*>(static_cast<const float*>(base) + off);
      w[0] = x[0];
      w[1] = x[1];
    } else {
      w[0] = __float_as_uint(static_cast<const float*>(base)[off]);
    }
  }
  __device__ __forceinline__ void unpack(float (&x)[N]) const {
    if constexpr (BF16 && N == 2) {
      x[0] = bf16_to_f32(w[0] & 0xffffu);
      x[1] = __uint_as_float(w[0] & 0xffff0000u);
    } else if constexpr (BF16) {
      x[0] = bf16_to_f32(w[0]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = __uint_as_float(w[i]);
    }
  }
};

template <int N>
constexpr int log2_exact() {
  static_assert(N > 0 && (N & (N - 1)) == 0, "power of two");
  int l = 0;
  while ((1 << l) < N) ++l;
  return l;
}

// ---------------------------------------------------------------------------
// transpose-reduce over lane bits
// ---------------------------------------------------------------------------

// Exchange across lane bit BIT (partner lane ^ (1 << BIT)) with the cheapest
// instruction for that bit: a row swap for bits 5 and 4, DPP below.  Lanes
// with the bit clear keep `lo` + the partner's `lo`, the others `hi` + the
// partner's `hi`; with lo == hi it is a plain pairwise sum.
template <int BIT>
__device__ __forceinline__ float xchg_level(bool up, float lo, float hi) {
  if constexpr (BIT == 5) return swap32_add(lo, hi);
  else if constexpr (BIT == 4) return swap16_add(lo, hi);
  else return dpp_level<(1 << BIT)>(up, lo, hi);
}

// HALF-sized transpose levels on lane bits BIT, BIT-1, ...: each level keeps
// half of the values a lane carries and sums it with the partner's copy;
// after LEVELS levels (by default until one value is left) a lane carries
// HALF * 2 / 2^LEVELS values.
template <int HALF, int BIT, int LEVELS = 32>
__device__ __forceinline__ void transpose_levels(float* vals, int lane) {
  const bool up = ((lane >> BIT) & 1) != 0;
#pragma unroll
  for (int m = 0; m < HALF; ++m) vals[m] = xchg_level<BIT>(up, vals[m], vals[m + HALF]);
  if constexpr (HALF > 1 && LEVELS > 1) transpose_levels<HALF / 2, BIT - 1, LEVELS - 1>(vals, lane);
}

// Plain sums over lane bits HI down to LO (none when HI < LO).
template <int HI, int LO>
__device__ __forceinline__ float sum_levels(float x) {
  if constexpr (HI >= LO) {
    x = xchg_level<HI>(false, x, x);
    return sum_levels<HI - 1, LO>(x);
  } else {
    return x;
  }
}

}  // namespace
}  // namespace kda

#endif  // KDA_TILE_H_
