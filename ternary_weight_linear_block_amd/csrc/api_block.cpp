// C ABI of the block operators around the ternary linear layer (include/twl.h):
// argument validation and launches.  The same rules as api.cpp: nothing is
// allocated, nothing synchronises, every kernel goes to the caller's stream.
#include "api_common.h"

#include <algorithm>
#include <cmath>

namespace {

using namespace twl::api;

twl_status check_lora(int64_t M, int64_t K, int64_t R, int64_t n) {
  TWL_TRY(check_rows("M", M));
  TWL_TRY(check_rows("n_adapters", n));
  if (K <= 0 || K % 128 != 0 || K > TWL_MAX_K)
    return fail(TWL_ESHAPE, "K=%lld must be a positive multiple of 128 of at most %d", static_cast<long long>(K),
                TWL_MAX_K);
  if (R < 8 || R % 8 != 0 || R > TWL_LORA_MAX_R)
    return fail(TWL_ESHAPE, "R=%lld must be a multiple of 8 from 8 to %d", static_cast<long long>(R), TWL_LORA_MAX_R);
  return TWL_OK;
}

// Sizes of a gated pair of N x K projections (2 N packed rows).
twl_status check_gated(int64_t N, int64_t K) {
  TWL_TRY(check_rows("N", N));
  if (N > (int64_t{1} << 29)) return fail(TWL_ESHAPE, "N=%lld is too large", static_cast<long long>(N));
  return check_k(K);
}

// Whether this path runs a decode kernel at M tokens, and its workspace.
bool gated_decodes(int64_t M, int path) {
  return path == TWL_PATH_GEMV || (path == TWL_PATH_AUTO && M <= TWL_GEMV_MAX_M);
}

size_t gated_need(int64_t M, int64_t N, int64_t K, int path, const twl::DeviceInfo& dev) {
  return gated_decodes(M, path) ? twl::gemv_gated_workspace_bytes(M, 2 * N, K, dev)
                                : twl::gemm_workspace_bytes(M, 2 * N, K, dev);
}

}  // namespace

extern "C" {

twl_status twl_pack_ternary_gated(const int8_t* code_gate, const uint16_t* s_gate,
                                  const int8_t* code_up, const uint16_t* s_up, int64_t N, int64_t K,
                                  uint8_t* packed, int8_t* q, float* smax, int32_t* bad_codes,
                                  hipStream_t stream) {
  TWL_TRY(check_gated(N, K));
  if (N == 0) return ok();
  TWL_REQUIRE_PTR(code_gate);
  TWL_REQUIRE_PTR(s_gate);
  TWL_REQUIRE_PTR(code_up);
  TWL_REQUIRE_PTR(s_up);
  TWL_REQUIRE_PTR(packed);
  TWL_REQUIRE_PTR(q);
  TWL_REQUIRE_PTR(smax);
  if (bad_codes != nullptr && (reinterpret_cast<uintptr_t>(bad_codes) & 3u))
    return fail(TWL_EALIGN, "bad_codes is not 4-byte aligned");
  twl::DeviceInfo dev;
  TWL_TRY(current_device(&dev));
  return launched(twl::launch_pack_gated(code_gate, s_gate, code_up, s_up, N, K, packed, q, smax, bad_codes, stream),
                  "pack_ternary_gated");
}

size_t twl_gated_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  twl::DeviceInfo dev;
  if (M <= 0 || N <= 0 || check_rows("M", M) != TWL_OK || check_gated(N, K) != TWL_OK ||
      current_device(&dev) != TWL_OK)
    return 0;
  size_t need = gated_need(M, N, K, TWL_PATH_GEMM, dev);
  if (M <= TWL_GEMV_MAX_M) need = std::max(need, gated_need(M, N, K, TWL_PATH_GEMV, dev));
  return need;
}

twl_status twl_ternary_gated_linear(const int8_t* x_i8, const float* a_scale, const uint8_t* packed,
                                    const int8_t* q, const float* smax, int64_t M, int64_t N,
                                    int64_t K, void* out, int out_kind, int path, void* workspace,
                                    size_t workspace_bytes, hipStream_t stream) {
  TWL_TRY(check_rows("M", M));
  TWL_TRY(check_gated(N, K));
  if (path != TWL_PATH_AUTO && path != TWL_PATH_GEMM && path != TWL_PATH_GEMV)
    return fail(TWL_EINVAL, "path %d is not AUTO, GEMM or GEMV", path);
  if (out_kind != TWL_OUT_F32 && out_kind != TWL_OUT_BF16)
    return fail(TWL_EINVAL, "output kind %d is not fp32 or bf16", out_kind);
  if (path == TWL_PATH_GEMV && M > TWL_GEMV_MAX_M)
    return fail(TWL_ESHAPE, "the decode path takes M <= %d (got %lld)", TWL_GEMV_MAX_M, static_cast<long long>(M));
  if (M == 0 || N == 0) return ok();
  TWL_REQUIRE_PTR(x_i8);
  TWL_REQUIRE_PTR(a_scale);
  TWL_REQUIRE_PTR(packed);
  TWL_REQUIRE_PTR(q);
  TWL_REQUIRE_PTR(smax);
  TWL_REQUIRE_PTR(out);
  const size_t rows = static_cast<size_t>(M), n2 = 2 * static_cast<size_t>(N), k = static_cast<size_t>(K);
  const Range in[] = {{x_i8, rows * k, "x_i8"}, {a_scale, rows * 4, "a_scale"}, {packed, (n2 + 63) / 64 * 64 * (k / 4), "packed"},
                      {q, n2 * (k / 128), "q"}, {smax, n2 * 4, "smax"}, {out, rows * N * (out_kind == TWL_OUT_F32 ? 4 : 2), "out"}};
  for (int i = 0; i < 5; ++i)
    if (overlap(in[5], in[i])) return fail(TWL_EINVAL, "out overlaps %s", in[i].name);
  twl::DeviceInfo dev;
  TWL_TRY(current_device(&dev));
  const size_t need = gated_need(M, N, K, path, dev);
  TWL_TRY(check_workspace(need, workspace, workspace_bytes));
  const Range scratch = {need > 0 ? workspace : nullptr, need, "workspace"};
  for (const Range& i : in)
    if (overlap(scratch, i)) return fail(TWL_EINVAL, "workspace overlaps %s", i.name);
  const twl::OutKind kind = out_kind == TWL_OUT_BF16 ? twl::kOutGatedBf16 : twl::kOutGatedF32;
  if (gated_decodes(M, path))
    return launched(twl::launch_gemv_gated(x_i8, a_scale, packed, q, smax, M, 2 * N, K, out, kind, workspace, dev, stream),
                    "ternary_gated_linear (GEMV)");
  return launched(twl::launch_gemm(x_i8, a_scale, packed, q, smax, M, 2 * N, K, out, kind, workspace, workspace_bytes, dev,
                                   stream),
                  "ternary_gated_linear (GEMM)");
}

size_t twl_lora_workspace_bytes(int64_t M, int64_t K, int64_t R, int64_t n_adapters) {
  twl::DeviceInfo dev;
  if (check_lora(M, K, R, n_adapters) != TWL_OK || current_device(&dev) != TWL_OK) return 0;
  ok();
  return twl::lora_workspace_bytes(M, static_cast<int>(K), static_cast<int>(R), n_adapters, dev);
}

twl_status twl_lora_add(const void* y, const uint16_t* x, const int32_t* ids, const uint16_t* lora_a,
                        const uint16_t* lora_b, const float* scale, int64_t M, int64_t N, int64_t K,
                        int64_t R, int64_t n_adapters, int kind, void* out, void* workspace,
                        size_t workspace_bytes, hipStream_t stream) {
  TWL_TRY(check_lora(M, K, R, n_adapters));
  TWL_TRY(check_rows("N", N));
  // 64 rows of fp32 y and one adapter's B stay below 2^31 bytes (32-bit offsets)
  if (N > (int64_t{1} << 22)) return fail(TWL_ESHAPE, "N=%lld is too large", static_cast<long long>(N));
  if (kind != TWL_OUT_F32 && kind != TWL_OUT_BF16) return fail(TWL_EINVAL, "kind %d is not fp32 or bf16", kind);
  if (M == 0 || N == 0) return ok();
  TWL_REQUIRE_PTR(y);
  TWL_REQUIRE_PTR(ids);
  TWL_REQUIRE_PTR(out);
  if (n_adapters > 0) {
    TWL_REQUIRE_PTR(x);
    TWL_REQUIRE_PTR(lora_a);
    TWL_REQUIRE_PTR(lora_b);
    TWL_REQUIRE_PTR(scale);
  }
  twl::DeviceInfo dev;
  TWL_TRY(current_device(&dev));
  const size_t need = twl::lora_workspace_bytes(M, static_cast<int>(K), static_cast<int>(R), n_adapters, dev);
  TWL_TRY(check_workspace(need, workspace, workspace_bytes));
  const size_t rows = static_cast<size_t>(M), n = static_cast<size_t>(n_adapters);
  const size_t y_bytes = rows * N * (kind == TWL_OUT_F32 ? 4 : 2);
  const Range outs[] = {{out, y_bytes, "out"}, {need > 0 ? workspace : nullptr, need, "workspace"}};
  const Range in[] = {{y, y_bytes, "y"}, {x, n > 0 ? rows * K * 2 : 0, "x"}, {ids, rows * 4, "ids"},
                      {lora_a, n * R * K * 2, "lora_a"}, {lora_b, n * N * R * 2, "lora_b"}, {scale, n * 4, "scale"}};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 6; ++j)
      if (overlap(outs[i], in[j]) && !(i == 0 && j == 0 && out == y))
        return fail(TWL_EINVAL, "%s overlaps %s", outs[i].name, in[j].name);
  if (overlap(outs[0], outs[1])) return fail(TWL_EINVAL, "out overlaps workspace");
  twl::LoraArgs a = {};
  a.y = y;
  a.x = x;
  a.ids = ids;
  a.a = lora_a;
  a.b = lora_b;
  a.scale = scale;
  a.out = out;
  a.part = static_cast<float*>(workspace);
  a.M = M;
  a.N = static_cast<int>(N);
  a.K = static_cast<int>(K);
  a.R = static_cast<int>(R);
  a.n = static_cast<int>(n_adapters);
  return launched(twl::launch_lora(a, kind == TWL_OUT_BF16, dev, stream), "lora_add");
}

twl_status twl_norm_rotate_quant_act(const uint16_t* x, const uint16_t* residual,
                                     const uint16_t* post_weight, const uint16_t* gate,
                                     int64_t gate_stride, double branch_scale,
                                     const uint16_t* weight, double eps, const int8_t* sign,
                                     int64_t M, int64_t K, uint16_t* h, uint16_t* normed,
                                     int8_t* x_i8, float* a_scale, hipStream_t stream) {
  TWL_TRY(check_rows("M", M));
  TWL_TRY(check_k(K));
  if (!(eps > 0.0) || !std::isfinite(eps)) return fail(TWL_EINVAL, "eps=%g must be positive and finite", eps);
  if (!std::isfinite(branch_scale)) return fail(TWL_EINVAL, "branch_scale=%g must be finite", branch_scale);
  if (gate_stride != 0 && (gate_stride < K || gate_stride % 8 != 0 || gate_stride > (int64_t{1} << 30)))
    return fail(TWL_ESHAPE, "gate_stride=%lld must be 0 or a multiple of 8 from K=%lld to 2^30",
                static_cast<long long>(gate_stride), static_cast<long long>(K));
  const bool branch = residual != nullptr || post_weight != nullptr || gate != nullptr || branch_scale != 1.0;
  if (h != nullptr && !branch)
    return fail(TWL_EINVAL, "h is given, but no residual, post_weight, gate or branch_scale: it would be x");
  if (sign == nullptr) {
    if (x_i8 != nullptr || a_scale != nullptr) return fail(TWL_EINVAL, "x_i8 and a_scale need sign");
    if (M > 0 && normed == nullptr) return fail(TWL_EINVAL, "sign and normed are both NULL: no output");
  }
  if (M == 0) return ok();
  TWL_REQUIRE_PTR(x);
  TWL_REQUIRE_PTR(weight);
  TWL_OPTIONAL_PTR(residual);
  TWL_OPTIONAL_PTR(post_weight);
  TWL_OPTIONAL_PTR(gate);
  TWL_OPTIONAL_PTR(h);
  TWL_OPTIONAL_PTR(normed);
  if (sign != nullptr) {
    TWL_REQUIRE_PTR(sign);
    TWL_REQUIRE_PTR(x_i8);
    TWL_REQUIRE_PTR(a_scale);
  }
  // outputs may not overlap anything but h its own x or residual, element for
  // element (each lane reads what it overwrites first)
  const size_t rows = static_cast<size_t>(M), wide = rows * K * 2, table = static_cast<size_t>(K) * 2;
  const size_t gate_bytes = table + (rows - 1) * static_cast<size_t>(gate_stride) * 2;
  const Range out[] = {{h, wide, "h"}, {normed, wide, "normed"}, {x_i8, rows * K, "x_i8"}, {a_scale, rows * 4, "a_scale"}};
  const Range in[] = {{x, wide, "x"}, {residual, wide, "residual"}, {post_weight, table, "post_weight"},
                      {gate, gate_bytes, "gate"}, {weight, table, "weight"}, {sign, static_cast<size_t>(K), "sign"}};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 6; ++j)
      if (overlap(out[i], in[j]) && !(i == 0 && j < 2 && out[i].p == in[j].p))
        return fail(TWL_EINVAL, "%s overlaps %s", out[i].name, in[j].name);
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return fail(TWL_EINVAL, "%s overlaps %s", out[i].name, out[j].name);
  }
  twl::DeviceInfo dev;
  TWL_TRY(current_device(&dev));
  twl::NormArgs a = {};
  a.x = x;
  a.residual = residual;
  a.post_weight = post_weight;
  a.gate = gate;
  a.weight = weight;
  a.sign = sign;
  a.h = h;
  a.normed = normed;
  a.x_i8 = x_i8;
  a.a_scale = a_scale;
  a.branch_scale = branch_scale;
  a.eps = eps;
  a.M = M;
  a.gate_stride = gate_stride;
  a.K = static_cast<int>(K);
  return launched(twl::launch_norm_rotate(a, dev, stream), "norm_rotate_quant_act");
}

}  // extern "C"
