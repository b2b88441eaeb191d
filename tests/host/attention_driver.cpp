// Host-only driver for the entry points of a block's attention half (api_attention.cpp),
// built with AddressSanitizer and UndefinedBehaviorSanitizer and run on the CPU.  The HIP
// runtime calls and the launchers are stubs, so a failing launch, a failing query
// and a device that is not gfx950 are forced from the host; what a launcher
// receives is checked too.  Exit status 0 when every check passes.
#include "api_common.h"
#include "attention_internal.h"

#include <cmath>
#include <cstdio>
#include <cstring>

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
const char* g_arch[2] = {"gfx950", "gfx942:sramecc+:xnack-"};
int g_launches = 0, g_d = 0;
bool g_f32 = false;
size_t g_int8_ws = 0, g_attn_ws = 0;
int64_t g_table_keys = 0;
twl::Int8Args g_int8;
twl::RopeArgs g_rope;
twl::AttnArgs g_attn;
}  // namespace

extern "C" {
hipError_t hipGetDevice(int* dev) {
  *dev = g_device;
  return g_get_device;
}
hipError_t hipGetDeviceProperties(hipDeviceProp_t* prop, int dev) {
  std::memset(prop, 0, sizeof *prop);
  if (dev < 0 || dev >= 2) return hipErrorInvalidDevice;
  std::snprintf(prop->gcnArchName, sizeof prop->gcnArchName, "%s", g_arch[dev]);
  prop->multiProcessorCount = 256;
  return hipSuccess;
}
const char* hipGetErrorString(hipError_t) { return "stubbed HIP error"; }
}

namespace twl {
size_t int8_workspace_bytes(int64_t, int64_t, int64_t, const DeviceInfo&) { return g_int8_ws; }
hipError_t launch_int8(Int8Args a, const DeviceInfo&, hipStream_t) {
  ++g_launches;
  g_int8 = a;
  return g_launch;
}
hipError_t launch_qk_rope(RopeArgs a, int D, bool f32, const DeviceInfo& dev, hipStream_t) {
  ++g_launches;
  g_rope = a;
  g_d = D;
  g_f32 = f32;
  return dev.cu_count == 256 ? g_launch : hipErrorInvalidValue;
}
size_t attention_workspace_bytes(int64_t, int64_t, int, int, int, int64_t table_keys, int, int, const DeviceInfo&) {
  g_table_keys = table_keys;
  return g_attn_ws;
}
hipError_t launch_attention(AttnArgs a, int D, const DeviceInfo&, hipStream_t) {
  ++g_launches;
  g_attn = a;
  g_d = D;
  return g_launch;
}
}  // namespace twl

namespace {
uint16_t* u16(uintptr_t a) { return reinterpret_cast<uint16_t*>(a); }
int8_t* i8(uintptr_t a) { return reinterpret_cast<int8_t*>(a); }
float* f32(uintptr_t a) { return reinterpret_cast<float*>(a); }
int32_t* i32(uintptr_t a) { return reinterpret_cast<int32_t*>(a); }
constexpr uintptr_t P(int i) { return 0x10000000ull * (i + 1); }

twl_status int8(void* ws = nullptr, size_t bytes = 0, int kind = TWL_OUT_BF16, int64_t M = 4) {
  return twl_int8_linear(i8(P(0)), f32(P(1)), i8(P(2)), f32(P(3)), kind == TWL_OUT_ACC_I32 ? nullptr : f32(P(4)), M, 96, 1008, u16(P(5)),
                         kind, ws, bytes, nullptr);
}
twl_status rope(int64_t M = 4, int64_t n_pages = 10, double eps = 1e-6) {
  return twl_qk_norm_rope(u16(P(0)), TWL_OUT_F32, 2048, u16(P(1)), nullptr, eps, f32(P(3)), 100, 64, 1, i32(P(4)), i32(P(5)), M, 4, 2,
                          128, u16(P(6)), u16(P(7)), u16(P(8)), n_pages, 16, nullptr);
}
twl_status attention(void* ws = nullptr, size_t bytes = 0, uintptr_t out = P(6), int64_t n_pages = 10, int64_t T = 4) {
  return twl_window_attention(u16(P(0)), u16(P(1)), u16(P(2)), i32(P(3)), i32(P(4)), i32(P(5)), 0.125, 100, 4, T, 2, 4, 2, 256, n_pages, 64,
                              8, u16(out), ws, bytes, nullptr);
}
bool says(const char* word) { return twl::api::g_last_error.find(word) != std::string::npos; }
}  // namespace

int main() {
  // int8_linear: arguments as given, the kinds, the workspace rules
  CHECK(int8() == TWL_OK && g_launches == 1);
  CHECK(g_int8.M == 4 && g_int8.N == 96 && g_int8.K == 1008 && g_int8.kind == twl::kOutBf16 && g_int8.bias == f32(P(4)));
  CHECK(g_int8.x == i8(P(0)) && g_int8.w == i8(P(2)) && g_int8.a_scale == f32(P(1)) && g_int8.w_scale == f32(P(3)));
  CHECK(int8(nullptr, 0, TWL_OUT_F32) == TWL_OK && g_int8.kind == twl::kOutF32);
  CHECK(int8(nullptr, 0, TWL_OUT_ACC_I32) == TWL_OK && g_int8.kind == twl::kOutAcc && g_int8.bias == nullptr);
  CHECK(int8(nullptr, 0, TWL_OUT_F32, 0) == TWL_OK && g_launches == 3);
  g_int8_ws = 4096;
  CHECK(twl_int8_workspace_bytes(4, 96, 1008) == 4096 && twl_int8_workspace_bytes(0, 96, 1008) == 0);
  CHECK(int8() == TWL_EINVAL && int8(u16(P(9)), 4095) == TWL_EINVAL && g_launches == 3);
  CHECK(int8(u16(P(9)), 4096) == TWL_OK && reinterpret_cast<uintptr_t>(g_int8.part) == P(9) && g_launches == 4);
  CHECK(int8(u16(P(9) + 8), 8192) == TWL_EALIGN);
  CHECK(int8(u16(P(2)), 4096) == TWL_EINVAL && says("workspace overlaps w_i8"));
  CHECK(int8(u16(P(5)), 4096) == TWL_EINVAL && says("workspace overlaps out"));
  g_int8_ws = 0;

  // qk_norm_rope
  g_launches = 0;
  CHECK(rope() == TWL_OK && g_launches == 1 && g_d == 128 && g_f32);
  CHECK(g_rope.M == 4 && g_rope.n_q == 4 && g_rope.n_kv == 2 && g_rope.rot == 64 && g_rope.n_pos == 100 && g_rope.interleaved == 1);
  CHECK(g_rope.stride == 2048 && g_rope.page_shift == 4 && g_rope.n_slots == 160 && g_rope.k_weight == nullptr);
  CHECK(g_rope.eps == 1e-6f);
  CHECK(rope(0) == TWL_OK && g_launches == 1);
  CHECK(rope(4, 0) == TWL_OK && g_rope.n_slots == 0);
  CHECK(rope(4, 10, 1.1754943508222875e-38) == TWL_OK && rope(4, 10, 1.17549e-38) == TWL_EINVAL);

  // window_attention: sizes, scale, workspace and overlaps
  g_launches = 0;
  CHECK(attention() == TWL_OK && g_launches == 1 && g_d == 256 && g_table_keys == 512);
  CHECK(g_attn.T == 4 && g_attn.B == 2 && g_attn.n_q == 4 && g_attn.n_kv == 2 && g_attn.page_shift == 6 && g_attn.n_pages == 10);
  CHECK(g_attn.table_pages == 8 && g_attn.window == 100 && g_attn.sinks == 4);
  CHECK(std::fabs(g_attn.scale_log2 - 0.125 * 1.4426950408889634) < 1e-7);
  CHECK(attention(nullptr, 0, P(6), 0) == TWL_OK && g_attn.n_pages == 0);
  CHECK(attention(nullptr, 0, P(6), 10, 0) == TWL_OK && g_launches == 2);
  CHECK(attention(nullptr, 0, P(0)) == TWL_EINVAL && says("out overlaps q"));
  CHECK(attention(nullptr, 0, P(1)) == TWL_EINVAL && says("out overlaps k_cache"));
  CHECK(attention(nullptr, 0, P(3)) == TWL_EINVAL && says("out overlaps page_table"));
  g_attn_ws = 1 << 20;
  CHECK(twl_attention_workspace_bytes(4, 2, 4, 2, 256, 64, 8, 100, 4) == 1 << 20 && twl_attention_workspace_bytes(0, 2, 4, 2, 256, 64, 8, 0, 0) == 0);
  CHECK(attention() == TWL_EINVAL && attention(u16(P(9)), (1 << 20) - 1) == TWL_EINVAL);
  CHECK(attention(u16(P(9)), 1 << 20) == TWL_OK && reinterpret_cast<uintptr_t>(g_attn.part) == P(9));
  CHECK(attention(u16(P(2)), 1 << 20) == TWL_EINVAL && says("workspace overlaps v_cache"));
  CHECK(attention(u16(P(6)), 1 << 20) == TWL_EINVAL && says("out overlaps workspace"));
  g_attn_ws = 0;

  // the largest sizes overflow nothing in the overlap checks
  CHECK(twl_window_attention(u16(P(0)), u16(P(1)), u16(P(2)), i32(P(3)), i32(P(4)), i32(P(5)), 1.0, 1 << 30, 1 << 30, 1 << 17, 4096, 1024,
                             1024, 256, (1 << 21) - 1, 1024, 1 << 20, u16(P(6)), nullptr, 0, nullptr) == TWL_EINVAL && says("overlaps"));
  CHECK(twl_int8_linear(i8(P(0)), f32(P(1)), i8(P(2)), f32(P(3)), f32(P(4)), 1 << 24, 512, 65536, u16(P(5)), TWL_OUT_F32, nullptr, 0,
                        nullptr) == TWL_EINVAL && says("overlaps"));
  CHECK(twl_qk_norm_rope(u16(P(0)), TWL_OUT_F32, 1 << 30, u16(P(1)), nullptr, 1e-6, f32(P(3)), 1 << 30, 256, 0, i32(P(4)), i32(P(5)),
                         1 << 15, 512, 256, 256, u16(P(6)), u16(P(7)), u16(P(8)), (1 << 21) - 1, 1024, nullptr) == TWL_EINVAL && says("overlaps"));

  // failures of the launch, the query and the device
  g_launch = hipErrorInvalidValue;
  CHECK(int8() == TWL_EHIP && rope() == TWL_EHIP && attention() == TWL_EHIP && says("window_attention"));
  g_launch = hipSuccess;
  g_launches = 0;
  g_device = 1;
  CHECK(int8() == TWL_EDEVICE && rope() == TWL_EDEVICE && attention() == TWL_EDEVICE);
  CHECK(twl_int8_workspace_bytes(4, 96, 1008) == 0);
  g_device = 0;
  g_get_device = hipErrorNoDevice;
  CHECK(int8() != TWL_OK && rope() != TWL_OK && attention() != TWL_OK && g_launches == 0);

  if (g_failures == 0) std::printf("all checks passed\n");
  return g_failures != 0;
}
