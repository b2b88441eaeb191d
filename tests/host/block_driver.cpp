// Host-only driver for the block operators' entry points (api_block.cpp), built with
// AddressSanitizer and UndefinedBehaviorSanitizer and run on the CPU.  The HIP
// runtime calls and the launchers are stubs, so a failing launch, a failing query
// and a device that is not gfx950 are forced from the host; what a launcher
// receives is checked too.  Exit status 0 when every check passes.
#include "twl.h"
#include "twl_internal.h"

#include <cstdio>
#include <cstring>
#include <limits>


namespace {
int g_failures = 0;
#define CHECK(cond)                                                    \
  do {                                                                 \
    if (!(cond)) {                                                     \
      std::printf("FAIL %s:%d: %s\n", __FILE__, __LINE__, #cond);      \
      ++g_failures;                                                    \
    }                                                                  \
  } while (0)

int g_device = 0;
hipError_t g_get_device = hipSuccess, g_launch = hipSuccess;
const char* g_arch[3] = {"gfx950", "gfx942:sramecc+:xnack-", "gfx950"};
int g_launches = 0;
twl::NormArgs g_norm;
twl::LoraArgs g_lora;
int64_t g_n = 0;
int g_kind = -1;
bool g_bf16 = false, g_decode = false;
size_t g_lora_ws = 0, g_gemm_ws = 0, g_gemv_ws = 0;
const void* g_ws = nullptr;
}  // namespace

extern "C" {
hipError_t hipGetDevice(int* dev) {
  *dev = g_device;
  return g_get_device;
}
hipError_t hipGetDeviceProperties(hipDeviceProp_t* prop, int dev) {
  std::memset(prop, 0, sizeof *prop);
  if (dev < 0 || dev >= 3) return hipErrorInvalidDevice;
  std::snprintf(prop->gcnArchName, sizeof prop->gcnArchName, "%s", g_arch[dev]);
  prop->multiProcessorCount = 256;
  return hipSuccess;
}
const char* hipGetErrorString(hipError_t) { return "stubbed HIP error"; }
}

namespace twl {
hipError_t launch_norm_rotate(NormArgs a, const DeviceInfo& dev, hipStream_t) {
  ++g_launches;
  g_norm = a;
  return dev.cu_count == 256 ? g_launch : hipErrorInvalidValue;
}
size_t lora_workspace_bytes(int64_t, int, int, int64_t n, const DeviceInfo&) { return n > 0 ? g_lora_ws : 0; }
hipError_t launch_lora(LoraArgs a, bool bf16, const DeviceInfo&, hipStream_t) {
  ++g_launches;
  g_lora = a;
  g_bf16 = bf16;
  return g_launch;
}
hipError_t launch_pack_gated(const int8_t*, const uint16_t*, const int8_t*, const uint16_t*, int64_t N, int64_t, uint8_t*,
                             int8_t*, float*, int32_t*, hipStream_t) {
  ++g_launches;
  g_n = N;
  return g_launch;
}
size_t gemm_workspace_bytes(int64_t, int64_t, int64_t, const DeviceInfo&) { return g_gemm_ws; }
size_t gemv_gated_workspace_bytes(int64_t, int64_t, int64_t, const DeviceInfo&) { return g_gemv_ws; }
hipError_t launch_gemm(const int8_t*, const float*, const uint8_t*, const int8_t*, const float*, int64_t, int64_t N, int64_t,
                       void*, OutKind kind, void* ws, size_t, const DeviceInfo&, hipStream_t) {
  ++g_launches;
  g_n = N;
  g_kind = kind;
  g_ws = ws;
  g_decode = false;
  return g_launch;
}
hipError_t launch_gemv_gated(const int8_t*, const float*, const uint8_t*, const int8_t*, const float*, int64_t, int64_t N,
                             int64_t, void*, OutKind kind, void* ws, const DeviceInfo&, hipStream_t) {
  ++g_launches;
  g_n = N;
  g_kind = kind;
  g_ws = ws;
  g_decode = true;
  return g_launch;
}
}  // namespace twl

namespace {
uint16_t* u16(uintptr_t a) { return reinterpret_cast<uint16_t*>(a); }
int8_t* i8(uintptr_t a) { return reinterpret_cast<int8_t*>(a); }
float* f32(uintptr_t a) { return reinterpret_cast<float*>(a); }
constexpr uintptr_t P(int i) { return 0x10000000ull * (i + 1); }

twl_status norm(const int8_t* sign = i8(P(5)), int64_t M = 4, double eps = 1e-6, double scale = 0.5) {
  return twl_norm_rotate_quant_act(u16(P(0)), u16(P(1)), u16(P(2)), u16(P(3)), 2048, scale, u16(P(4)), eps, sign, M, 1024,
                                   u16(P(6)), u16(P(7)), sign ? i8(P(8)) : nullptr, sign ? f32(P(9)) : nullptr, nullptr);
}
twl_status lora(int64_t M, int64_t n, void* ws, size_t bytes, int kind = TWL_OUT_BF16, int64_t N = 64) {
  return twl_lora_add(u16(P(0)), u16(P(1)), reinterpret_cast<int32_t*>(P(2)), u16(P(3)), u16(P(4)), f32(P(5)), M, N, 1024, 16,
                      n, kind, u16(P(6)), ws, bytes, nullptr);
}
twl_status gated(int64_t M, int path, int kind, void* ws, size_t bytes) {
  return twl_ternary_gated_linear(i8(P(0)), f32(P(1)), reinterpret_cast<uint8_t*>(P(2)), i8(P(3)), f32(P(4)), M, 100, 1024,
                                  u16(P(5)), kind, path, ws, bytes, nullptr);
}
}  // namespace

int main() {
  // norm: arguments as given, failures mapped
  CHECK(norm() == TWL_OK && g_launches == 1);
  CHECK(g_norm.M == 4 && g_norm.K == 1024 && g_norm.gate_stride == 2048 && g_norm.branch_scale == 0.5 && g_norm.eps == 1e-6);
  CHECK(g_norm.h == u16(P(6)) && g_norm.normed == u16(P(7)) && g_norm.x_i8 == i8(P(8)));
  CHECK(norm(nullptr) == TWL_OK && g_norm.sign == nullptr && g_norm.x_i8 == nullptr);
  CHECK(norm(i8(P(5)), 0) == TWL_OK && g_launches == 2);
  CHECK(norm(i8(P(5)), 4, -1.0) == TWL_EINVAL);
  CHECK(norm(i8(P(5)), 4, 1e-6, std::numeric_limits<double>::quiet_NaN()) == TWL_EINVAL);
  CHECK(norm(i8(P(5)), (int64_t{1} << 30) + 1) == TWL_ESHAPE);
  g_launch = hipErrorLaunchFailure;
  CHECK(norm() == TWL_EHIP);
  g_launch = hipSuccess;
  g_device = 1;
  CHECK(norm() == TWL_EDEVICE);
  g_device = 70;
  CHECK(norm() == TWL_EDEVICE);
  g_device = 0;
  g_get_device = hipErrorNoDevice;
  CHECK(norm() == TWL_EHIP && lora(4, 2, nullptr, 0) == TWL_EHIP && gated(4, 0, 2, nullptr, 0) == TWL_EHIP);
  CHECK(twl_lora_workspace_bytes(4, 1024, 16, 2) == 0 && twl_gated_workspace_bytes(4, 64, 1024) == 0);
  g_get_device = hipSuccess;
  // the largest sizes overflow nothing in the overlap checks
  CHECK(twl_norm_rotate_quant_act(u16(P(0)), nullptr, nullptr, u16(P(3)), int64_t{1} << 30, 1.0, u16(P(4)), 1e-6, i8(P(5)),
                                  int64_t{1} << 30, 65536, u16(P(6)), nullptr, i8(P(8)), f32(P(9)), nullptr) == TWL_EINVAL);

  // lora: the workspace rules
  g_launches = 0;
  g_lora_ws = 4096;
  CHECK(twl_lora_workspace_bytes(4, 1024, 16, 2) == 4096 && twl_lora_workspace_bytes(4, 1024, 12, 2) == 0);
  CHECK(lora(4, 2, nullptr, 0) == TWL_EINVAL && lora(4, 2, u16(P(7)), 4095) == TWL_EINVAL);
  CHECK(lora(4, 2, reinterpret_cast<char*>(P(7)) + 8, 8192) == TWL_EALIGN);
  CHECK(lora(4, 2, u16(P(1)), 8192) == TWL_EINVAL && lora(4, 2, u16(P(6)), 8192) == TWL_EINVAL);  // over x, over out
  CHECK(g_launches == 0);
  CHECK(lora(4, 2, u16(P(7)), 4096) == TWL_OK && g_launches == 1 && g_bf16 && g_lora.part == f32(P(7)) && g_lora.n == 2);
  CHECK(lora(4, 0, nullptr, 0, TWL_OUT_F32) == TWL_OK && !g_bf16 && g_lora.part == nullptr);
  CHECK(lora(0, 2, nullptr, 0) == TWL_OK && lora(4, 2, nullptr, 0, TWL_OUT_BF16, 0) == TWL_OK && g_launches == 2);
  CHECK(lora(4, 2, u16(P(7)), 4096, TWL_OUT_BF16, (int64_t{1} << 22) + 1) == TWL_ESHAPE);
  CHECK(lora(4, 2, u16(P(7)), 4096, TWL_OUT_ACC_I32) == TWL_EINVAL);

  // gated: kernel family by path and tokens, 2 N rows, kinds, workspaces
  g_launches = 0;
  g_gemm_ws = 1000;
  g_gemv_ws = 2000;
  CHECK(twl_gated_workspace_bytes(4, 100, 1024) == 2000 && twl_gated_workspace_bytes(25, 100, 1024) == 1000);
  CHECK(gated(4, TWL_PATH_AUTO, TWL_OUT_BF16, u16(P(6)), 1999) == TWL_EINVAL && g_launches == 0);
  CHECK(gated(4, TWL_PATH_AUTO, TWL_OUT_BF16, u16(P(6)), 2000) == TWL_OK);
  CHECK(g_decode && g_n == 200 && g_kind == twl::kOutGatedBf16 && g_ws == u16(P(6)));
  CHECK(gated(4, TWL_PATH_GEMM, TWL_OUT_F32, u16(P(6)), 1000) == TWL_OK && !g_decode && g_kind == twl::kOutGatedF32);
  CHECK(gated(25, TWL_PATH_AUTO, TWL_OUT_F32, u16(P(6)), 1000) == TWL_OK && !g_decode && g_n == 200);
  CHECK(gated(25, TWL_PATH_GEMV, TWL_OUT_F32, u16(P(6)), 4000) == TWL_ESHAPE);
  CHECK(gated(4, 0, TWL_OUT_F32, u16(P(2) + 50 * 1024), 4000) == TWL_EINVAL);  // over the last packed rows: 256 x K / 4
  CHECK(gated(4, 0, TWL_OUT_F32, u16(P(2) + 64 * 1024), 4000) == TWL_OK);
  CHECK(gated(4, 0, TWL_OUT_F32, u16(P(5) + 1584), 4000) == TWL_EINVAL);  // over out's end
  CHECK(gated(4, TWL_PATH_GEMV_MFMA, TWL_OUT_F32, u16(P(6)), 4000) == TWL_EINVAL);
  g_launch = hipErrorInvalidConfiguration;
  CHECK(gated(4, 0, TWL_OUT_F32, u16(P(6)), 4000) == TWL_EHIP);
  CHECK(lora(4, 2, u16(P(7)), 4096) == TWL_EHIP);
  g_launch = hipSuccess;
  CHECK(twl_pack_ternary_gated(i8(P(0)), u16(P(1)), i8(P(2)), u16(P(3)), 100, 1024, reinterpret_cast<uint8_t*>(P(4)), i8(P(5)),
                               f32(P(6)), nullptr, nullptr) == TWL_OK && g_n == 100);
  std::printf(g_failures == 0 ? "all checks passed\n" : "%d checks failed\n", g_failures);
  return g_failures != 0;
}
