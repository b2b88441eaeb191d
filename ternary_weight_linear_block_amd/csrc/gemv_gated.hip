// ternary_gated_linear for decode batches (M <= 24): out = SiLU(gate) * up of two
// ternary projections of one input.
//
// Mathematics: the rows of the packed weight are gate_0, up_0, gate_1, up_1, ...;
//   g = acc[t, 2 i] * a_scale[t] * smax[2 i] / 127,   u = the same of row 2 i + 1,
//   out[t, i] = g / (1 + e^-g) * u
// from the exact int32 acc of the linear layer's decode kernels.
//
// Wide layers run the row-balanced kernel (gemv_rows.h) with whole pairs of rows
// to a workgroup: both sums of a pair are then in its LDS and the product is
// formed there, in the same launch.  Layers it does not take (fewer than 16 rows a
// CU, or K above 33792 at any width) run the linear layer's dot4 or K-split kernel up
// to its int32 partial sums and the finishing kernel below, which takes the place of
// its reduce kernel.
//
// 2 x 17408 x 5120: 12 us for one token (46 MB, 3.9 TB/s, what the row-balanced
// kernel reaches for the plain layer of as many rows) and 16.7 us for 24, bound by
// the stream of the weights and, with 24 tokens, by the MFMA and LDS work of the
// two token tiles.
#include "gemv_rows.h"

#include <cstdio>
#include <cstdlib>

namespace twl {
namespace {

// Sum of the slices' partial sums of both rows of a pair, then the rescale and
// the product.  One thread a result, a row of workgroups a token.
__global__ __launch_bounds__(256) void gated_finish_kernel(const int32_t* __restrict__ part, int slices, int M, int N,
                                                           const float* __restrict__ a_scale,
                                                           const float* __restrict__ smax,
                                                           void* __restrict__ out, int out_kind) {
  const int pairs = N / 2, t = blockIdx.y;
  const int pr = blockIdx.x * 256 + threadIdx.x;  // pairs is at most 2^29
  if (pr >= pairs) return;
  int2 s = make_int2(0, 0);
  for (int sl = 0; sl < slices; ++sl) {
    const int2 v = *reinterpret_cast<const int2*>(part + (static_cast<size_t>(sl) * M + t) * N + 2 * pr);
    s.x += v.x;
    s.y += v.y;
  }
  const float g = static_cast<float>(s.x) * a_scale[t] * (smax[2 * pr] * (1.0f / 127.0f));
  const float u = static_cast<float>(s.y) * a_scale[t] * (smax[2 * pr + 1] * (1.0f / 127.0f));
  store_out(out, static_cast<size_t>(t) * pairs + pr, out_kind == kOutGatedBf16 ? kOutBf16 : kOutF32, 0, silu_mul(g, u));
}

}  // namespace

size_t gemv_gated_workspace_bytes(int64_t M, int64_t N, int64_t K, const DeviceInfo& dev) {
  if (M <= 0 || N <= 0 || K <= 0 || tuned_rows_plan(M, N, K, dev).slices > 0) return 0;
  return static_cast<size_t>(gemv_part_slices(M, N, K, dev)) * static_cast<size_t>(M) * static_cast<size_t>(N) * 4;
}

hipError_t launch_gemv_gated(const int8_t* x_i8, const float* a_scale, const uint8_t* packed,
                             const int8_t* q, const float* smax, int64_t M, int64_t N, int64_t K,
                             void* out, OutKind out_kind, void* part, const DeviceInfo& dev,
                             hipStream_t stream) {
  if (M < 1 || M > kXRows || N < 2 || N % 2 != 0) return hipErrorInvalidValue;
  const GemvPlan pl = tuned_rows_plan(M, N, K, dev);
  if (std::getenv("TWL_LOG"))
    std::fprintf(stderr, "[twl] gated gemv%s M=%lld N=%lld K=%lld\n", pl.slices > 0 ? "-rows" : " + finish",
                 static_cast<long long>(M), static_cast<long long>(N), static_cast<long long>(K));
  if (pl.slices > 0) {
    GemvArgs a = {};
    a.x = x_i8;
    a.a_scale = a_scale;
    a.packed = packed;
    a.q = q;
    a.smax = smax;
    a.out = out;
    a.N = static_cast<int>(N);
    a.K = static_cast<int>(K);
    a.G = static_cast<int>(K >> 7);
    a.n_rb = pl.n_rb;
    a.slices = 1;
    a.out_kind = out_kind;
    if (pl.nw * 64 > 512) return hipErrorInvalidValue;
    return launch_rows<false, true>(a, static_cast<int>(M), pl, stream);
  }
  const hipError_t e = launch_gemv_part(x_i8, packed, q, M, N, K, static_cast<int32_t*>(part), dev, stream);
  if (e != hipSuccess) return e;
  const dim3 grid(static_cast<unsigned>((N / 2 + 255) / 256), static_cast<unsigned>(M));
  hipLaunchKernelGGL(gated_finish_kernel, grid, dim3(256), 0, stream, static_cast<const int32_t*>(part),
                     gemv_part_slices(M, N, K, dev), static_cast<int>(M), static_cast<int>(N), a_scale, smax, out,
                     static_cast<int>(out_kind));
  return hipGetLastError();
}

}  // namespace twl
