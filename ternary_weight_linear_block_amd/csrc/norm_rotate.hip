// norm_rotate_quant_act: the step between two blocks of a pre-norm (and
// post-norm) transformer, fused with the ternary linear's input rotation.
//
// Mathematics, per token (all of it in fp64 up to the two bf16 roundings):
//   b = x                                            the block's output
//   b = b * post_weight / sqrt(mean(b^2) + eps)      RMSNorm after the block (optional)
//   b = b * gate * branch_scale                      (optional, per channel or per element)
//   h = bf16(residual + b)                           the new residual stream
//   n = bf16(h * weight / sqrt(mean(h^2) + eps))     RMSNorm before the next block
//   x_i8, a_scale = rotate_quant_act(n)              rotate_block.h, unchanged
// n is rounded to bf16 because that is what an unfused pipeline stores, what
// adapters beside the projection read, and what rotate_quant_act takes: the
// int8 result equals rotate_quant_act(n) bit for bit.  The sums and products are
// fp64 because a value next to a bf16 rounding border would otherwise round
// either way with the order of the sum; an element costs about 17 fp64
// operations, which the memory time covers.
//
// One workgroup per token, wave w owns the 1024-blocks w, w + nw, ... in the
// rotation's first layout (lane = 16 consecutive elements), so a row is read
// once and stays in registers as packed bf16 through both norms and the
// rotation; the statistics meet in LDS (waves in order, so the sums do not
// depend on timing).
#include "rotate_block.h"

#include <algorithm>

namespace twl {
namespace {

using rot::kBlock;
using rot::kWaveBufWords;

constexpr int kMaxNormWaves = 16;

__device__ __forceinline__ double lo_f64(uint32_t w) { return static_cast<double>(__uint_as_float(w << 16)); }
__device__ __forceinline__ double hi_f64(uint32_t w) { return static_cast<double>(__uint_as_float(w & 0xFFFF0000u)); }

__device__ __forceinline__ uint32_t pack_bf16(double lo, double hi) {
  return f32_to_bf16_rne(static_cast<float>(lo)) |
         (static_cast<uint32_t>(f32_to_bf16_rne(static_cast<float>(hi))) << 16);
}

// 16 consecutive bf16 of one lane
struct Row16 {
  uint32_t w[8];
};

__device__ __forceinline__ Row16 load16(const uint16_t* p) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint4 b = *reinterpret_cast<const uint4*>(p + 8);
  return Row16{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}

__device__ __forceinline__ void store16(uint16_t* p, const Row16& r) {
  *reinterpret_cast<uint4*>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
  *reinterpret_cast<uint4*>(p + 8) = make_uint4(r.w[4], r.w[5], r.w[6], r.w[7]);
}

// Sum of squares of a lane's elements.  The empty asm afterwards makes the packed
// words opaque: without it the compiler keeps their fp64 copies (32 registers a
// block) from here to their next use and spills.
__device__ __forceinline__ double sum_squares(Row16& r) {
  double s = 0.0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const double a = lo_f64(r.w[e]), b = hi_f64(r.w[e]);
    s += a * a;
    s += b * b;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) asm volatile("" : "+v"(r.w[e]));
  return s;
}

// Sum over the workgroup, waves added in order; `slots` holds one double a wave.
__device__ __forceinline__ double block_sum(double s, double* slots, int wave, int lane, int nw) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) s += __shfl_xor(s, m);
  if (lane == 0) slots[wave] = s;
  __syncthreads();
  double t = slots[0];
  for (int w = 1; w < nw; ++w) t += slots[w];
  return t;
}

// ROT: rotate and quantise; else only h and n are written.
template <int BPW, bool ROT>
__global__ __launch_bounds__(1024) void norm_rotate_kernel(NormArgs a) {
  extern __shared__ float wbuf_all[];  // ROT: nw x kWaveBufWords
  // two sets, alternated by token: a wave may write its slot of the next token
  // while another still reads this one's
  __shared__ double post_slots[2][kMaxNormWaves];
  __shared__ double pre_slots[2][kMaxNormWaves];
  __shared__ float max_slots[2][kMaxNormWaves];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nw = blockDim.x >> 6;
  const int K = a.K, nblocks = K / kBlock;
  const bool branch = a.residual != nullptr || a.post_weight != nullptr || a.gate != nullptr || a.branch_scale != 1.0;
  float* wb = wbuf_all + wave * kWaveBufWords;
  int par = 0;
  for (int64_t t = blockIdx.x; t < a.M; t += gridDim.x, par ^= 1) {
    const size_t row = static_cast<size_t>(t) * K;
    Row16 v[BPW];
#pragma unroll
    for (int i = 0; i < BPW; ++i) {
      const int b = wave + i * nw;
      v[i] = b < nblocks ? load16(a.x + row + b * kBlock + lane * 16) : Row16{};
    }
    if (branch) {
      double inv = 1.0;
      if (a.post_weight != nullptr) {
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < BPW; ++i) s += sum_squares(v[i]);
        inv = 1.0 / sqrt(block_sum(s, post_slots[par], wave, lane, nw) / K + a.eps);
      }
#pragma unroll
      for (int i = 0; i < BPW; ++i) {
        const int b = wave + i * nw;
        if (b >= nblocks) continue;
        if (BPW > 1) __builtin_amdgcn_sched_barrier(0);  // one block's operands at a time: no spills
        const int k0 = b * kBlock + lane * 16;
        Row16 pw{}, gt{}, rs{};
        if (a.post_weight != nullptr) pw = load16(a.post_weight + k0);
        if (a.gate != nullptr) gt = load16(a.gate + static_cast<size_t>(t) * a.gate_stride + k0);
        if (a.residual != nullptr) rs = load16(a.residual + row + k0);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          double lo = lo_f64(v[i].w[e]), hi = hi_f64(v[i].w[e]);
          if (a.post_weight != nullptr) {
            lo = lo * inv * lo_f64(pw.w[e]);
            hi = hi * inv * hi_f64(pw.w[e]);
          }
          if (a.gate != nullptr) {
            lo *= lo_f64(gt.w[e]);
            hi *= hi_f64(gt.w[e]);
          }
          lo *= a.branch_scale;
          hi *= a.branch_scale;
          if (a.residual != nullptr) {
            lo += lo_f64(rs.w[e]);
            hi += hi_f64(rs.w[e]);
          }
          v[i].w[e] = pack_bf16(lo, hi);
        }
        if (a.h != nullptr) store16(a.h + row + k0, v[i]);
      }
    }
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < BPW; ++i) s += sum_squares(v[i]);
    const double inv = 1.0 / sqrt(block_sum(s, pre_slots[par], wave, lane, nw) / K + a.eps);
    float r[ROT ? BPW : 1][16];
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < BPW; ++i) {
      const int b = wave + i * nw;
      if (b >= nblocks) continue;
      if (BPW > 1) __builtin_amdgcn_sched_barrier(0);
      const int k0 = b * kBlock + lane * 16;
      const Row16 w = load16(a.weight + k0);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v[i].w[e] = pack_bf16(lo_f64(v[i].w[e]) * inv * lo_f64(w.w[e]), hi_f64(v[i].w[e]) * inv * hi_f64(w.w[e]));
      if (a.normed != nullptr) store16(a.normed + row + k0, v[i]);
      if constexpr (ROT) {
        const uint4 sg = *reinterpret_cast<const uint4*>(a.sign + k0);
        rot::BlockIn in = {{}, {}, {sg.x, sg.y, sg.z, sg.w}};
#pragma unroll
        for (int e = 0; e < 8; ++e) in.x[e] = v[i].w[e];
        rot::rotate_loaded<false>(in, lane, wb, r[i]);
#pragma unroll
        for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(r[i][e]));
      }
    }
    if constexpr (ROT) {
#pragma unroll
      for (int m = 32; m >= 1; m >>= 1) amax = fmaxf(amax, __shfl_xor(amax, m));
      if (lane == 0) max_slots[par][wave] = amax;
      __syncthreads();
      float tmax = max_slots[par][0];
      for (int w = 1; w < nw; ++w) tmax = fmaxf(tmax, max_slots[par][w]);
      const rot::TokenQuant tq = rot::token_quant(tmax);
      if (threadIdx.x == 0) a.a_scale[t] = tq.scale;
#pragma unroll
      for (int i = 0; i < BPW; ++i) {
        const int b = wave + i * nw;
        if (b >= nblocks) continue;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *reinterpret_cast<uint32_t*>(a.x_i8 + row + b * kBlock + 256 * c + 4 * lane) = rot::quant_run(r[i], c, tq);
      }
    }
  }
}

template <int BPW, bool ROT>
hipError_t launch_bpw(const NormArgs& a, hipStream_t stream) {
  const int nblocks = a.K / kBlock;
  const int nw = (nblocks + BPW - 1) / BPW;
  const size_t lds = ROT ? static_cast<size_t>(nw) * kWaveBufWords * sizeof(float) : 0;
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(norm_rotate_kernel<BPW, ROT>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds));
    if (e != hipSuccess) return e;
  }
  // one workgroup a token, up to the grid limit; past it workgroups take several
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(a.M, 1 << 20));
  hipLaunchKernelGGL((norm_rotate_kernel<BPW, ROT>), dim3(grid), dim3(64 * nw), lds, stream, a);
  return hipGetLastError();
}

template <bool ROT>
hipError_t launch_rot(const NormArgs& a, hipStream_t stream) {
  const int nblocks = a.K / kBlock;  // 1 .. 64 (validated by the caller)
  if (nblocks <= 16) return launch_bpw<1, ROT>(a, stream);
  if (nblocks <= 32) return launch_bpw<2, ROT>(a, stream);
  return launch_bpw<4, ROT>(a, stream);
}

}  // namespace

hipError_t launch_norm_rotate(const NormArgs& a, hipStream_t stream) {
  if (a.M == 0) return hipSuccess;
  return a.sign != nullptr ? launch_rot<true>(a, stream) : launch_rot<false>(a, stream);
}

}  // namespace twl
