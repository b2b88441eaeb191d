// Internal launchers of the ternary linear library (not part of the C ABI).
// Every launcher assumes the host wrapper in api.cpp has already validated
// pointers, alignment and shapes; they only pick a configuration and launch.
#pragma once

#include <hip/hip_runtime.h>
#include <cstddef>
#include <cstdint>

namespace twl {

// Per-device facts the launchers need (cached by api.cpp).
struct DeviceInfo {
  int cu_count = 0;
};

hipError_t launch_rotate_quant(const uint16_t* x, const int8_t* sign, int64_t M, int64_t K,
                               int8_t* x_i8, float* a_scale, hipStream_t stream);
// The rotation alone: r [M, K] as bf16 bit patterns.
hipError_t launch_rotate_bf16(const uint16_t* x, const int8_t* sign, int64_t M, int64_t K,
                              uint16_t* r, hipStream_t stream);
// Exact-dequant bf16 reference linear: y = r_bf16 . (code * bf16(s))^T in fp32.
hipError_t launch_reference_bf16(const uint16_t* r, const uint8_t* packed, const uint16_t* s,
                                 int64_t M, int64_t N, int64_t K, float* y, hipStream_t stream);
// gate_up: bf16 [M, 2K]; rotates bf16(SiLU(gate) * up).
hipError_t launch_silu_mul_rotate_quant(const uint16_t* gate_up, const int8_t* sign, int64_t M,
                                        int64_t K, int8_t* x_i8, float* a_scale,
                                        hipStream_t stream);

hipError_t launch_pack(const int8_t* code, const uint16_t* s, int64_t N, int64_t K,
                       uint8_t* packed, int8_t* q, float* smax, int32_t* bad_codes,
                       hipStream_t stream);
// The same of 2 N rows, gate and up in turn.
hipError_t launch_pack_gated(const int8_t* code_gate, const uint16_t* s_gate, const int8_t* code_up,
                             const uint16_t* s_up, int64_t N, int64_t K, uint8_t* packed, int8_t* q,
                             float* smax, int32_t* bad_codes, hipStream_t stream);

// What the linear layer writes: fp32 y, the raw int32 accumulators, or y
// rounded to bf16 (round to nearest even).
// The gated kinds (ternary_gated_linear): rows of the weight are gate and up in
// turn, N = 2 I of them, and out [M, I] is SiLU(gate) * up of adjacent columns.
enum OutKind { kOutF32 = 0, kOutAcc = 1, kOutBf16 = 2, kOutGatedF32 = 3, kOutGatedBf16 = 4 };
constexpr bool is_gated(int kind) { return kind >= kOutGatedF32; }

// fp32 -> bf16 bits, round to nearest even (finite inputs).
__device__ __forceinline__ uint16_t f32_to_bf16_rne(float f) {
  const uint32_t u = __float_as_uint(f);
  return static_cast<uint16_t>((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
}

// SiLU(g) u = g u / (1 + e^-g), by the native exponential and reciprocal (1 ulp
// each).  The rounding of g log2(e) enters e^-g as |g| 2^-24 and the constant's own
// error (0.224 2^-24) as 0.224 |g| 2^-24, so the result is within (1.25 |g| + 8) 2^-24
// relative: below half a bf16 step by a factor of 900 at |g| = 50.  Where 1 + e^-g passes 2^126 (g below -87) the reciprocal is below the
// smallest normal number and comes out as 0.  Every kernel of ternary_gated_linear uses this
// form, so all of them give the same bits.
__device__ __forceinline__ float silu_mul(float g, float u) {
  const float e = __builtin_amdgcn_exp2f(g * -0x1.715476p+0f);
  return g * __builtin_amdgcn_rcpf(1.0f + e) * u;
}

// Stores one epilogue value v (y before rounding) or the accumulator s at
// element o of `out`, whose type follows `kind`.
__device__ __forceinline__ void store_out(void* out, size_t o, int kind, int32_t s, float v) {
  if (kind == kOutAcc)
    static_cast<int32_t*>(out)[o] = s;
  else if (kind == kOutBf16)
    static_cast<uint16_t*>(out)[o] = f32_to_bf16_rne(v);
  else
    static_cast<float*>(out)[o] = v;
}

hipError_t launch_gemm(const int8_t* x_i8, const float* a_scale, const uint8_t* packed,
                       const int8_t* q, const float* smax, int64_t M, int64_t N, int64_t K,
                       void* out, OutKind out_kind, void* workspace, size_t workspace_bytes,
                       const DeviceInfo& dev, hipStream_t stream);
size_t gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, const DeviceInfo& dev);
// The GEMM plan for this shape, as twl_plan_info reports it (info[0..7]).
void gemm_plan_info(int64_t M, int64_t N, int64_t K, const DeviceInfo& dev, int64_t* info);

// Decode kernels (M <= 24): kGemvAuto picks by M, kGemvDot4 / kGemvMfma force
// one.  When K is split across workgroups (gemv_workspace_bytes > 0) the
// kernel writes int32 partial sums to `part` (at least that many bytes).
enum GemvKind { kGemvAuto = 0, kGemvDot4 = 1, kGemvMfma = 2 };
hipError_t launch_gemv(const int8_t* x_i8, const float* a_scale, const uint8_t* packed,
                       const int8_t* q, const float* smax, int64_t M, int64_t N, int64_t K,
                       void* out, OutKind out_kind, void* part, size_t part_bytes, GemvKind kind,
                       const DeviceInfo& dev, hipStream_t stream);
size_t gemv_workspace_bytes(int64_t M, int64_t N, int64_t K, GemvKind kind, const DeviceInfo& dev);
// The decode plan for this shape, as twl_plan_info reports it (info[0..7]).
void gemv_plan_info(int64_t M, int64_t N, int64_t K, GemvKind kind, const DeviceInfo& dev, int64_t* info);

// The decode kernels for layers that the row-balanced kernel does not take (fewer than
// 16 rows a CU, or K above 33792; the dot4 or K-split MFMA kernel by M) up to
// their int32 partial sums: `part` gets [slices][M][N], slices being returned by
// gemv_part_slices, and holds that many.
int gemv_part_slices(int64_t M, int64_t N, int64_t K, const DeviceInfo& dev);
hipError_t launch_gemv_part(const int8_t* x_i8, const uint8_t* packed, const int8_t* q, int64_t M,
                            int64_t N, int64_t K, int32_t* part, const DeviceInfo& dev,
                            hipStream_t stream);

// ternary_gated_linear for decode batches (M <= 24) of a packed weight of N = 2 I
// interleaved rows: the row-balanced kernel with whole pairs of rows to a
// workgroup, or, where it does not apply, launch_gemv_part and a finishing kernel.
size_t gemv_gated_workspace_bytes(int64_t M, int64_t N, int64_t K, const DeviceInfo& dev);
hipError_t launch_gemv_gated(const int8_t* x_i8, const float* a_scale, const uint8_t* packed,
                             const int8_t* q, const float* smax, int64_t M, int64_t N, int64_t K,
                             void* out, OutKind out_kind, void* part, const DeviceInfo& dev,
                             hipStream_t stream);

// Fused decode: rotate_quant_act (silu: of bf16(SiLU(gate) * up), x being
// [gate | up] [M, 2K]) and the row-balanced decode kernel in one launch, which
// also writes x_i8 [M, K] and a_scale [M].  gemv_rot_applies tells whether the
// shape fits it; launch_gemv_rot returns hipErrorNotSupported otherwise.
bool gemv_rot_applies(int64_t M, int64_t N, int64_t K, const DeviceInfo& dev);
hipError_t launch_gemv_rot(const uint16_t* x, const int8_t* sign, bool silu, const uint8_t* packed,
                           const int8_t* q, const float* smax, int64_t M, int64_t N, int64_t K,
                           void* out, OutKind out_kind, int8_t* x_i8, float* a_scale,
                           const DeviceInfo& dev, hipStream_t stream);

// norm_rotate_quant_act (include/twl.h): every pointer but x and weight may be
// null; sign null leaves out the rotation (x_i8 and a_scale are then not
// written).  gate_stride: elements between the gate rows of two tokens (0: one
// row for all).
struct NormArgs {
  const uint16_t* x;
  const uint16_t* residual;
  const uint16_t* post_weight;
  const uint16_t* gate;
  const uint16_t* weight;
  const int8_t* sign;
  uint16_t* h;
  uint16_t* normed;
  int8_t* x_i8;
  float* a_scale;
  double branch_scale, eps;
  double inv_k;  // 1 / K, set by the launcher
  int64_t M, gate_stride;
  int K;
};
hipError_t launch_norm_rotate(NormArgs a, const DeviceInfo& dev, hipStream_t stream);

// lora_add (include/twl.h).  The caller sets the operands and sizes; the
// launcher plans the rest.  `part` holds lora_workspace_bytes.
struct LoraArgs {
  const void* y;
  const uint16_t* x;
  const int32_t* ids;
  const uint16_t* a;     // [n, R, K]
  const uint16_t* b;     // [n, N, R]
  const float* scale;    // [n]
  void* out;
  float* part;           // [slices][M][R]
  int64_t M;
  int N, K, R, n;
  int slices, shrink_ts;
  uint32_t shrink_tiles, shrink_passes;
  uint32_t expand_chunks, expand_tiles, expand_passes;
};
size_t lora_workspace_bytes(int64_t M, int K, int R, int64_t n, const DeviceInfo& dev);
hipError_t launch_lora(LoraArgs a, bool bf16, const DeviceInfo& dev, hipStream_t stream);

}  // namespace twl
