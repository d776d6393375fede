// kda_internal.h - what the argument checker hands to the kernel launcher.
#ifndef KDA_INTERNAL_H_
#define KDA_INTERNAL_H_

#include <cstdint>

#include "kda.h"

namespace kda {

// Validated, flattened arguments of one decode call (device pointers).
struct DecodeArgs {
  void* out;                    // [T, HV, dv]   bf16 or f32
  const void* q;                // [T, H, dk]    bf16 or f32
  const void* k;                // [T, H, dk]
  const void* v;                // [T, HV, dv]
  const float* raw_gate;        // [T, HV, dk]
  const float* beta_logits;     // [T, HV]
  const float* a_log;           // [HV]
  const float* dt_bias;         // [HV, dk]
  const int32_t* cu_seqlens;    // [B + 1]
  void* state_pool;             // [N, HV, dk, dv] or [N, HV, dv, dk], f32 or bf16
  const int32_t* state_indices; // [B]
  int32_t B, T, H, HV, G, N;
  int32_t gate_mode;            // enum kda_gate_mode
  float lower_bound, l2_eps, scale;
  // short convolution of the v stream (kda_decode_conv only; v is then the
  // pre-convolution x_v)
  const void* conv_w_v;         // [K, HV*dv] taps
  float* conv_win_v;            // [N, K-1, HV*dv] windows
  int32_t conv_k;               // K, 2..4
  int32_t conv_w_bf16;          // taps stored as bf16
};

// Arguments of the q/k convolution kernel of kda_decode_conv.
struct ConvQKArgs {
  const void* x[2];             // pre-convolution q, k [T, H, dk]
  const void* w[2];             // taps [K, H*dk]
  float* win[2];                // windows [N, K-1, H*dk]
  void* y[2];                   // convolved q, k [T, H, dk]
  const int32_t* cu_seqlens;
  const int32_t* state_indices;
  int32_t B, T, H, N;
  int32_t conv_k;
  int32_t w_bf16;
};

// The tokens a kda_gdr_decode or kda_decode_window call walks.
struct TokenStream {
  const void* q;                // [T, H, dk]    bf16 or f32 (unused by a replay)
  const void* k;                // [T, H, dk]
  const void* v;                // [T, HV, dv]
  const float* raw_gate;        // [T, HV, dk] (per channel) or [T, HV] (per head)
  const float* beta_logits;     // [T, HV]
  int32_t T;
};

// Validated, flattened arguments of one kda_gdr_decode or kda_decode_window
// call: the state advances through stream 0 and is written, then stream 1 is
// run from there and the state it ends with is dropped.  kda_gdr_decode has
// its tokens in stream 0, kda_decode_window the replay there and the window
// in stream 1.
struct WindowArgs {
  void* out;                    // [T, HV, dv] of the stream with outputs
  TokenStream src[2];
  const float* a_log;           // [HV]
  const float* dt_bias;         // [HV, dk] or [HV]
  const int32_t* cu_seqlens;    // [B + 1] of the stream with outputs
  const int32_t* begin;         // [B] first row of the replay   (window only)
  const int32_t* count;         // [B] tokens of the replay
  void* state_pool;
  const int32_t* state_indices;
  int32_t B, H, HV, G, N;
  int32_t gate_mode;
  float lower_bound, l2_eps, scale;
  int32_t window;               // 0: kda_gdr_decode, 1: kda_decode_window
};

// Enqueue the kernel of kda_gdr_decode / kda_decode_window.  Returns KDA_OK,
// KDA_ERR_UNSUPPORTED or KDA_ERR_LAUNCH.  Defined in kda_api.cpp, which
// picks the object of the gate's form: kda_window.hip is compiled once with
// KDA_WINDOW_CHANNEL 0 (one decay per head) and once with 1 (per channel).
int launch_window(const WindowArgs& args, int dk, int dv, bool qkv_bf16, bool state_bf16, int state_layout,
                  bool channel, hipStream_t stream);
template <bool CHANNEL>
int launch_window_gate(const WindowArgs& args, int dk, int dv, bool qkv_bf16, bool state_bf16,
                       int state_layout, hipStream_t stream);
template <>
int launch_window_gate<false>(const WindowArgs&, int, int, bool, bool, int, hipStream_t);
template <>
int launch_window_gate<true>(const WindowArgs&, int, int, bool, bool, int, hipStream_t);

// kda_verify, flattened.
struct VerifyArgs {
  int32_t* n_commit;            // [B]
  int32_t* next_token;          // [B]
  const void* target;           // [T, V] f32 or bf16
  const void* draft;            // [T, V], same dtype, or NULL: certain drafts
  const int32_t* tokens;        // [T]
  const float* u_accept;        // [T]
  const float* u_sample;        // [B]
  const int32_t* cu_seqlens;    // [B + 1]
  void* workspace;              // kda_verify's workspace
  int32_t B, T, V;
};
int launch_verify(const VerifyArgs& args, bool bf16, hipStream_t stream);

// Validated, flattened arguments of kda_ssm_decode and kda_ssm_prefill.
struct SsmArgs {
  void* out;                    // [T, HV, dv]  bf16 or f32
  const void* xbc;              // [T, C]       dtype of out
  const float* dt;              // [T, HV]
  const void* conv_w;           // [K, C]       f32 or bf16
  const void* conv_b;           // [C] or NULL, dtype of conv_w
  float* conv_win;              // [N, K-1, C]
  const float* a_log;           // [HV]
  const float* dt_bias;         // [HV]
  const float* d_skip;          // [HV] or NULL
  const int32_t* cu_seqlens;    // [B + 1]
  void* state_pool;             // [N, HV, dk, dv] or [N, HV, dv, dk]
  const int32_t* state_indices; // [B]
  float* workspace;             // kda_ssm_prefill only
  int32_t B, T, H, HV, G, N;
  int32_t C, K;
  int32_t w_bf16;               // dtype of conv_w and conv_b
};

// Enqueue kda_ssm_decode (kda_ssm_decode.hip) and kda_ssm_prefill
// (kda_ssm_prefill.hip, compiled once per dk and dv with KDA_SSM_DK and
// KDA_SSM_DV; kda_api.cpp picks the object).  Return codes as below.
int launch_ssm_decode(const SsmArgs& args, int dk, int dv, bool bf16, bool state_bf16, int state_layout,
                      hipStream_t stream);
template <int DK, int DV>
int launch_ssm_prefill_of(const SsmArgs& args, bool bf16, bool state_bf16, int state_layout, hipStream_t stream);
#define KDA_SSM_SIZES(X) X(32, 32) X(32, 64) X(32, 128) X(64, 32) X(64, 64) X(64, 128) X(128, 32) X(128, 64) X(128, 128)
#define KDA_SSM_DECLARE(DK, DV) \
  template <>                   \
  int launch_ssm_prefill_of<DK, DV>(const SsmArgs&, bool, bool, int, hipStream_t);
KDA_SSM_SIZES(KDA_SSM_DECLARE)
#undef KDA_SSM_DECLARE

// kda_norm_residual and kda_norm_gate, flattened (kda_norm.hip).
struct ResidualArgs {
  void* hidden_out;             // [rows, D]  bf16 or f32
  const void* hidden;
  void* normed;                 // [rows, D]  bf16 or f32
  const void* block_out;
  const float* weight;          // [D]
  const float* post_weight;     // [D] or NULL
  const float* scale;           // [D], [1] or NULL
  int32_t scale_per_channel;
  int64_t rows;
  int32_t D;
  float eps;
};
struct GateArgs {
  void* out;                    // [rows, D]  bf16 or f32
  const void* x;
  const void* gate;
  const float* weight;          // [groups, D]; row r takes r % groups
  int64_t rows;
  int32_t D, groups;
  int32_t silu;
  float eps;
};
int launch_norm_residual(const ResidualArgs& args, bool hidden_bf16, bool bf16, hipStream_t stream);
int launch_norm_gate(const GateArgs& args, bool gate_first, bool bf16, hipStream_t stream);

// The chunked gated delta rule (kda_gdr_prefill): DecodeArgs with raw_gate
// [T, HV] and dt_bias [HV].  Defined in kda_gdr_prefill.hip.
int launch_gdr_prefill(const DecodeArgs& args, int dk, int dv, bool qkv_bf16, bool state_bf16,
                       int state_layout, hipStream_t stream);

// Enqueue the decode kernel for (dk, dv, q/k/v dtype, state dtype, state
// layout) on `stream`.  Returns KDA_OK, KDA_ERR_UNSUPPORTED (no such
// specialization) or KDA_ERR_LAUNCH.  Defined in kda_decode.hip.
int launch_decode(const DecodeArgs& args, int dk, int dv, bool qkv_bf16, bool state_bf16,
                  int state_layout, bool conv_v, hipStream_t stream);

// Enqueue the chunked prefill kernel (dk, dv in {32, 64, 128}; matmul an
// enum kda_matmul).  Same return codes.  Defined in kda_api.cpp.
int launch_prefill(const DecodeArgs& args, int dk, int dv, bool qkv_bf16, bool state_bf16,
                   int state_layout, int matmul, hipStream_t stream);

// The same for one dk: kda_prefill.hip is compiled once per dk
// (KDA_PREFILL_DK = 32, 64, 128), each object defining its dk's
// specialization, so that the three compile in parallel; launch_prefill
// (kda_api.cpp) picks one.
template <int DK>
int launch_prefill_dk(const DecodeArgs& args, int dv, bool qkv_bf16, bool state_bf16, int state_layout,
                      int matmul, hipStream_t stream);
template <>
int launch_prefill_dk<32>(const DecodeArgs&, int, bool, bool, int, int, hipStream_t);
template <>
int launch_prefill_dk<64>(const DecodeArgs&, int, bool, bool, int, int, hipStream_t);
template <>
int launch_prefill_dk<128>(const DecodeArgs&, int, bool, bool, int, int, hipStream_t);

// Enqueue the q/k convolution kernel.  Same return codes.
int launch_conv_qk(const ConvQKArgs& args, int dk, bool x_bf16, hipStream_t stream);

}  // namespace kda

#endif  // KDA_INTERNAL_H_
