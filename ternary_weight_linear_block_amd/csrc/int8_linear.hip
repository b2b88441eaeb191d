// int8_linear: y = (sum_k x_i8 w_i8) a_scale[t] w_scale[n] + bias[n] on int8 MFMAs with
// int32 sums (include/twl.h).
#include "attention_internal.h"

#include <algorithm>

namespace twl {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));

// RT x 16 rows of w and MT x 16 tokens a workgroup, whose waves share K.
template <int RT, int MT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void int8_rows_kernel(Int8Args a) {
  __shared__ v4i part[WAVES][RT * MT][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, h = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * (16 * RT);
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * (16 * MT);
  const int8_t* wp[RT];
  const int8_t* xp[MT];
#pragma unroll
  for (int r = 0; r < RT; ++r) wp[r] = a.w + min(n0 + r * 16 + m, static_cast<int64_t>(a.N) - 1) * a.K;
#pragma unroll
  for (int t = 0; t < MT; ++t) xp[t] = a.x + min(t0 + t * 16 + m, static_cast<int64_t>(a.M) - 1) * a.K;
  v4i acc[RT][MT] = {};
  for (int k = wave * 64 + h * 16; k - h * 16 < a.K; k += 64 * WAVES) {
    v4i wf[RT], xf[MT];
    const bool in = k < a.K;  // K is a multiple of 16: a lane's 16 bytes are in range or none is
#pragma unroll
    for (int r = 0; r < RT; ++r) wf[r] = in ? *reinterpret_cast<const v4i*>(wp[r] + k) : v4i(0);
#pragma unroll
    for (int t = 0; t < MT; ++t) xf[t] = in ? *reinterpret_cast<const v4i*>(xp[t] + k) : v4i(0);
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[r][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[r], xf[t], acc[r][t], 0, 0, 0);
  }
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < MT; ++t) part[wave][r * MT + t][lane] = acc[r][t];
  __syncthreads();
  for (int f = wave; f < RT * MT; f += WAVES) {
    v4i s = part[0][f][lane];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) s += part[w][f][lane];
    const int64_t token = t0 + f % MT * 16 + m, n = n0 + f / MT * 16 + h * 4;
    if (token >= a.M) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (n + i >= a.N) continue;
      const int64_t o = token * a.N + n + i;
      if (a.kind == kOutAcc) {
        static_cast<int32_t*>(a.out)[o] = s[i];
        continue;
      }
      float v = static_cast<float>(s[i]) * a.a_scale[token] * a.w_scale[n + i];
      if (a.bias != nullptr) v += a.bias[n + i];
      if (a.kind == kOutBf16)
        static_cast<__bf16*>(a.out)[o] = static_cast<__bf16>(v);
      else
        static_cast<float*>(a.out)[o] = v;
    }
  }
}

}  // namespace

size_t int8_workspace_bytes(int64_t M, int64_t N, int64_t K, const DeviceInfo& dev) { return 0; }

hipError_t launch_int8(Int8Args a, const DeviceInfo& dev, hipStream_t stream) {
  const dim3 grid(static_cast<uint32_t>((static_cast<int64_t>(a.N) + 15) / 16), static_cast<uint32_t>((static_cast<int64_t>(a.M) + 31) / 32));
  int8_rows_kernel<1, 2, 4><<<grid, 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace twl
