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
// int8 result equals rotate_quant_act(n) bit for bit.  The sums are fp64 and every
// product exact or fp64, because a value next to a bf16 rounding border would
// otherwise round either way with the order of the sum (fp64 runs at the rate of
// fp32 here: 4 cycles a wave, conversions too).
//
// Wave w of a workgroup owns the 1024-blocks w, w + nw, ... of a row, so a row is
// read once and stays in registers as packed bf16 through both norms and the
// rotation (which takes it through LDS into its own first layout); the
// statistics meet in LDS (waves in order, so the sums do not depend on timing).
// Workgroups stay and take every gridDim.x-th token; with one block a wave the
// next token's rows are loaded while this one is computed.
//
// 8192 tokens of 5120 with everything: 115 us, 4.0 TB/s of the 461 MB that have to
// move (a copy reaches 5.15): the fp64 and rotation instructions, 2300 cycles a
// block, take as long as the memory and overlap it in part.  333 tokens of 17408,
// the norm alone: 12.8 us, the instructions of the CUs that have two tokens.  One
// token of 5120: 5.5 us, two rounds of loads, three barriers and the rotation in
// turn.
#include "rotate_block.h"

#include <algorithm>
#include <atomic>

namespace twl {
namespace {

using rot::kBlock;
using rot::kWaveBufWords;

constexpr int kMaxNormWaves = 16;

__device__ __forceinline__ double lo_f64(uint32_t w) { return static_cast<double>(__uint_as_float(w << 16)); }
__device__ __forceinline__ double hi_f64(uint32_t w) { return static_cast<double>(__uint_as_float(w & 0xFFFF0000u)); }

typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

// fp64 -> fp32 -> bf16, both to nearest even (v_cvt_pk_bf16_f32)
__device__ __forceinline__ uint32_t pack_bf16(double lo, double hi) {
  const v2f f = {static_cast<float>(lo), static_cast<float>(hi)};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, v2bf));
}

// One lane's 16 bf16 of a 1024-block: elements 8 lane .. + 7 and 512 + 8 lane .. + 7,
// so that a load or store of the wave covers 1024 consecutive bytes.
struct Row16 {
  uint32_t w[8];
};

__device__ __forceinline__ Row16 load16(const uint16_t* block, int lane) {
  const uint4 a = *reinterpret_cast<const uint4*>(block + 8 * lane);
  const uint4 b = *reinterpret_cast<const uint4*>(block + 512 + 8 * lane);
  return Row16{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}

__device__ __forceinline__ void store16(uint16_t* block, int lane, const Row16& r) {
  *reinterpret_cast<uint4*>(block + 8 * lane) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
  *reinterpret_cast<uint4*>(block + 512 + 8 * lane) = make_uint4(r.w[4], r.w[5], r.w[6], r.w[7]);
}

// The same 16 values a lane as the rotation wants them, elements 16 lane .. + 15,
// through the wave's transpose buffer (idle between two rotations).
__device__ __forceinline__ Row16 consecutive(const Row16& r, int lane, float* wb) {
  uint4* buf = reinterpret_cast<uint4*>(wb);
  rot::wave_lds_sync();
  // 16-byte units, one spare after every eight: the reads hit different banks
  const auto at = [](int unit) { return unit + (unit >> 3); };
  buf[at(lane)] = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
  buf[at(64 + lane)] = make_uint4(r.w[4], r.w[5], r.w[6], r.w[7]);
  rot::wave_lds_sync();
  const uint4 a = buf[at(2 * lane)], b = buf[at(2 * lane + 1)];
  return Row16{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}

// Makes the packed words opaque to the compiler, which otherwise keeps fp64 copies
// of them (32 registers a block) from one use to the next, or over the whole token
// loop, and spills.
__device__ __forceinline__ void opaque(Row16& r) {
#pragma unroll
  for (int e = 0; e < 8; ++e) asm volatile("" : "+v"(r.w[e]));
}

// Sum of squares of a lane's elements.
__device__ __forceinline__ double sum_squares(Row16& r) {
  double s = 0.0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const double a = lo_f64(r.w[e]), b = hi_f64(r.w[e]);
    s = __builtin_fma(a, a, s);
    s = __builtin_fma(b, b, s);
  }
  opaque(r);
  return s;
}

// The product of a row's element and its norm weight, both bf16, is exact in fp32
// unless it leaves fp32's range.  So a row whose norm factor f = 1 / sqrt(mean + eps)
// lies outside 2^-12 .. 2^8 is first multiplied by the power of two next below f
// (exact but for elements 2^-126 below 1 / f) and its factor divided by it.  Then the
// product passes 2^128 only where the normed value passes 2^116, and where it falls
// below 2^-126, to a multiple of 2^-149, the value is off by 2^-9 of a step of bf16's
// denormals at most.  A gate, which nothing bounds, is multiplied in fp64.  All of them
// in fp64 cost an instruction more an element: 333 tokens of 17408 13.7 instead of
// 13.0 us, 2048 of 17408 with everything 106.9 instead of 102.6 (gate in fp32: 100.7).
__device__ __forceinline__ bool in_range(double f) { return f >= 0x1p-12 && f <= 0x1p8; }

template <int BPW, class Rows>
__device__ __forceinline__ double to_range(Rows& in, double f) {
  const int e = __builtin_amdgcn_frexp_exp(f) - 1;
#pragma unroll
  for (int i = 0; i < BPW; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t& w = in[i].x.w[k];
      w = pack_bf16(ldexp(lo_f64(w), e), ldexp(hi_f64(w), e));
    }
  return ldexp(f, -e);
}

// row_ror:n of a wave's four rows of 16 lanes
template <int N>
__device__ __forceinline__ uint32_t row_ror(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x120 + N, 0xF, 0xF, true));
}

template <int N>
__device__ __forceinline__ double row_ror(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint64_t lo = row_ror<N>(static_cast<uint32_t>(b)), hi = row_ror<N>(static_cast<uint32_t>(b >> 32));
  return __builtin_bit_cast(double, (hi << 32) | lo);
}

__device__ __forceinline__ double read_lane(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(b), lane);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(b >> 32), lane);
  return __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);
}

// Sum over the workgroup, waves added in order; `slots` holds one double a wave.
// Lane rotations and lane reads instead of LDS shuffles: a tenth of their latency.
__device__ __forceinline__ double block_sum(double s, double* slots, int wave, int lane, int nw) {
  s += row_ror<8>(s);
  s += row_ror<4>(s);
  s += row_ror<2>(s);
  s += row_ror<1>(s);
  s = (read_lane(s, 0) + read_lane(s, 16)) + (read_lane(s, 32) + read_lane(s, 48));
  if (nw == 1) return s;
  if (lane == 0) slots[wave] = s;
  __syncthreads();
  double t = slots[0];
  for (int w = 1; w < nw; ++w) t += slots[w];
  return t;
}

// fmaxf over the wave of non-negative values, which order like their bits.
__device__ __forceinline__ float wave_max(float m) {
  uint32_t u = __float_as_uint(m);
  u = max(u, row_ror<8>(u));
  u = max(u, row_ror<4>(u));
  u = max(u, row_ror<2>(u));
  u = max(u, row_ror<1>(u));
  const uint32_t a = max(__builtin_amdgcn_readlane(u, 0), __builtin_amdgcn_readlane(u, 16));
  const uint32_t b = max(__builtin_amdgcn_readlane(u, 32), __builtin_amdgcn_readlane(u, 48));
  return __uint_as_float(max(a, b));
}

// One lane's operands of a block that change with the token.
struct TokenIn {
  Row16 x, residual, gate;
};

// One lane's operands of a block that do not.
struct Tables {
  Row16 weight, post, gate;
  uint4 sign;
};

// ROT: rotate and quantise; else only h and n are written.  BRANCH: any of
// post_weight, gate, branch_scale and residual is there.
// AHEAD (one block a wave): the next token's rows are loaded while this one is
// computed, from where its own operands have been used (loaded at its start they
// cost 16 registers more: 4096 tokens of 9216 106 instead of 103 us; not ahead 114).
// WAVES: waves a SIMD that the registers have to leave room for.
template <int BPW, bool ROT, bool BRANCH, bool AHEAD, int MAXT, int WAVES>
__global__ __launch_bounds__(MAXT) __attribute__((amdgpu_waves_per_eu(WAVES)))
void norm_rotate_kernel(NormArgs a) {
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
  const bool post = BRANCH && a.post_weight != nullptr, gated = BRANCH && a.gate != nullptr;
  const bool token_gate = gated && a.gate_stride != 0, residual = BRANCH && a.residual != nullptr;
  float* wb = wbuf_all + wave * kWaveBufWords;
  static_assert(!AHEAD || BPW == 1, "one block a wave");

  // a wave's block past the last re-reads it (no branch around loads) and is not used
  const auto k_of = [&](int i) { return min(wave + i * nw, nblocks - 1) * kBlock; };
  const auto load_x = [&](int64_t t, int i, TokenIn& in) { in.x = load16(a.x + static_cast<size_t>(t) * K + k_of(i), lane); };
  const auto load_branch = [&](int64_t t, int i, TokenIn& in) {
    if (residual) in.residual = load16(a.residual + static_cast<size_t>(t) * K + k_of(i), lane);
    if (token_gate) in.gate = load16(a.gate + static_cast<size_t>(t) * a.gate_stride + k_of(i), lane);
  };
  const auto load_branch_tables = [&](int i, Tables& tab) {
    if (post) tab.post = load16(a.post_weight + k_of(i), lane);
    if (gated && !token_gate) tab.gate = load16(a.gate + k_of(i), lane);
  };
  const auto load_tables = [&](int i, Tables& tab) {
    tab.weight = load16(a.weight + k_of(i), lane);
    if (ROT) tab.sign = *reinterpret_cast<const uint4*>(a.sign + k_of(i) + 16 * lane);
  };

  int64_t t = blockIdx.x;  // the grid is at most M
  TokenIn next = {};
  if (AHEAD) {
    load_x(t, 0, next);
    load_branch(t, 0, next);
  }
  int par = 0;
  for (; t < a.M; t += gridDim.x, par ^= 1) {
    const size_t row = static_cast<size_t>(t) * K;
    TokenIn in[BPW];
    Tables tab[BPW];
    if (AHEAD) {
      in[0] = next;
      tab[0] = Tables{};
      load_branch_tables(0, tab[0]);
    } else {
#pragma unroll
      for (int i = 0; i < BPW; ++i) {
        in[i] = TokenIn{};
        tab[i] = Tables{};
        load_x(t, i, in[i]);
        // two blocks' operands fit the registers ahead of the first sum, four do not
        if (BPW <= 2) {
          load_branch(t, i, in[i]);
          load_branch_tables(i, tab[i]);
        }
      }
    }
    if (BRANCH) {
      double factor = a.branch_scale;
      if (post) {
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < BPW; ++i)
          if (wave + i * nw < nblocks) s += sum_squares(in[i].x);
        const double mean = block_sum(s, post_slots[par], wave, lane, nw) * a.inv_k;
        double f = rsqrt(mean + a.eps);
        if (!in_range(f)) f = to_range<BPW>(in, f);
        factor *= f;
      }
#pragma unroll
      for (int i = 0; i < BPW; ++i) {
        if (BPW > 1) __builtin_amdgcn_sched_barrier(0);  // one block's fp64 values at a time: no spills
        if (BPW > 2) {
          load_branch(t, i, in[i]);
          load_branch_tables(i, tab[i]);
        }
        const Row16& gate = token_gate ? in[i].gate : tab[i].gate;
        Row16& v = in[i].x;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          // eight elements, one uniform branch an operand (branches inside the
          // element loop leave a wave waiting for each result in turn)
          float p[8];
          double b[8];
          const auto each = [&](const Row16& r, auto f) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint32_t w = r.w[4 * half + e / 2];
              f(e, __uint_as_float(e % 2 == 0 ? w << 16 : w & 0xFFFF0000u));
            }
          };
          each(v, [&](int e, float x) { p[e] = x; });
          if (post) each(tab[i].post, [&](int e, float w) { p[e] *= w; });
#pragma unroll
          for (int e = 0; e < 8; ++e) b[e] = static_cast<double>(p[e]);
          if (gated) each(gate, [&](int e, float g) { b[e] *= static_cast<double>(g); });
          if (residual) {
            each(in[i].residual, [&](int e, float x) { b[e] = __builtin_fma(b[e], factor, static_cast<double>(x)); });
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) b[e] *= factor;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) v.w[4 * half + e] = pack_bf16(b[2 * e], b[2 * e + 1]);
        }
        if (a.h != nullptr && wave + i * nw < nblocks) store16(a.h + row + k_of(i), lane, v);
      }
    }
    if (BPW <= 2) {
#pragma unroll
      for (int i = 0; i < BPW; ++i) load_tables(i, tab[i]);
    }
    if (AHEAD) {
      const int64_t tn = std::min<int64_t>(t + gridDim.x, a.M - 1);
      load_x(tn, 0, next);
      load_branch(tn, 0, next);
    }
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < BPW; ++i)
      if (wave + i * nw < nblocks) s += sum_squares(in[i].x);
    const double mean = block_sum(s, pre_slots[par], wave, lane, nw) * a.inv_k;
    double inv = rsqrt(mean + a.eps);
    if (!in_range(inv)) inv = to_range<BPW>(in, inv);
    float r[ROT ? BPW : 1][16];
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < BPW; ++i) {
      if (BPW > 1) __builtin_amdgcn_sched_barrier(0);
      if (wave + i * nw >= nblocks) continue;
      if (BPW > 2) load_tables(i, tab[i]);
      Row16& v = in[i].x;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t x = v.w[e], w = tab[i].weight.w[e];
        const float lo = __uint_as_float(x << 16) * __uint_as_float(w << 16);  // exact
        const float hi = __uint_as_float(x & 0xFFFF0000u) * __uint_as_float(w & 0xFFFF0000u);
        v.w[e] = pack_bf16(static_cast<double>(lo) * inv, static_cast<double>(hi) * inv);
      }
      if (a.normed != nullptr) store16(a.normed + row + k_of(i), lane, v);
      if constexpr (ROT) {
        const Row16 c = consecutive(v, lane, wb);
        const uint32_t sg[4] = {tab[i].sign.x, tab[i].sign.y, tab[i].sign.z, tab[i].sign.w};
        rot::BlockIn b = {};  // signs applied here, two bf16 at a time
#pragma unroll
        for (int e = 0; e < 8; ++e)
          b.x[e] = c.w[e] ^ (__builtin_amdgcn_perm(0u, sg[e / 2], e % 2 == 0 ? 0x010C000Cu : 0x030C020Cu) & 0x80008000u);
        rot::rotate_loaded<false, false>(b, lane, wb, r[i]);
#pragma unroll
        for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(r[i][e]));
      }
    }
    if constexpr (ROT) {
      float tmax = wave_max(amax);
      if (nw > 1) {
        if (lane == 0) max_slots[par][wave] = tmax;
        __syncthreads();
        for (int w = 0; w < nw; ++w) tmax = fmaxf(tmax, max_slots[par][w]);
      }
      const rot::TokenQuant tq = rot::token_quant_unscaled(tmax);
      if (threadIdx.x == 0) a.a_scale[t] = tq.scale;
      // run c of a lane's four runs of 4 consecutive elements, as one dword
      const auto store_all = [&](auto run) {
#pragma unroll
        for (int i = 0; i < BPW; ++i) {
          const int b = wave + i * nw;
          if (b >= nblocks) continue;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            *reinterpret_cast<uint32_t*>(a.x_i8 + row + b * kBlock + 256 * c + 4 * lane) = run(&r[i][4 * c]);
        }
      };
      // the test is hoisted out of the element loop (one branch per token)
      if (tq.markstein)
        store_all([&](const float* w) { return rot::quant_run_markstein(w, tq); });
      else
        store_all([&](const float* w) {
          uint32_t word = 0;
#pragma unroll
          for (int d = 0; d < 4; ++d) word |= rot::quant_byte(rot::quotient_unscaled(w[d], tq)) << (8 * d);
          return word;
        });
    }
  }
}

template <int BPW, bool ROT, bool BRANCH, bool AHEAD, int MAXT, int WAVES>
hipError_t launch_form(const NormArgs& a, const DeviceInfo& dev, hipStream_t stream) {
  const int nblocks = a.K / kBlock;
  const int nw = (nblocks + BPW - 1) / BPW;
  if (nw > kMaxNormWaves || 64 * nw > MAXT) return hipErrorInvalidValue;
  const size_t lds = ROT ? static_cast<size_t>(nw) * kWaveBufWords * sizeof(float) : 0;
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(norm_rotate_kernel<BPW, ROT, BRANCH, AHEAD, MAXT, WAVES>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds));
    if (e != hipSuccess) return e;
  }
  // as many workgroups as are resident at once, so that all of them take the same
  // number of tokens, one more at most
  // (asked once for each number of waves: the query costs as much as a launch)
  static std::atomic<int> resident_of[kMaxNormWaves + 1];
  int per_cu = resident_of[nw].load(std::memory_order_relaxed);
  if (per_cu == 0) {
    const hipError_t e = hipOccupancyMaxActiveBlocksPerMultiprocessor(
        &per_cu, norm_rotate_kernel<BPW, ROT, BRANCH, AHEAD, MAXT, WAVES>, 64 * nw, lds);
    if (e != hipSuccess) return e;
    resident_of[nw].store(std::max(1, per_cu), std::memory_order_relaxed);
  }
  const int64_t resident = static_cast<int64_t>(std::max(1, dev.cu_count)) * std::max(1, per_cu);
  hipLaunchKernelGGL((norm_rotate_kernel<BPW, ROT, BRANCH, AHEAD, MAXT, WAVES>), dim3(static_cast<unsigned>(std::min(a.M, resident))),
                     dim3(64 * nw), lds, stream, a);
  return hipGetLastError();
}

template <bool ROT, bool BRANCH>
hipError_t launch_blocks(const NormArgs& a, const DeviceInfo& dev, hipStream_t stream) {
  const int nblocks = a.K / kBlock;  // 1 .. 64 (validated by the caller)
  // One block a wave up to 16, the next token's rows ahead: a token's latency is
  // lowest (5120: 5.8 us, two blocks a wave 6.7), and many tokens keep the memory
  // busiest (each call followed by one that reads x_i8, both: 8192 tokens of 5120
  // with everything 216 us, two blocks a wave without rows ahead 232, with them and
  // half the waves 226; 4096 of 12288 256 against 291).  The exception is the norm alone,
  // whose few operands leave the registers to two blocks a wave: 8192 of 8192 240 ->
  // 233 us, of 5120 159 -> 146.
  if constexpr (!BRANCH) {
    if (nblocks <= 8 && a.M > 3 * dev.cu_count) return launch_form<2, ROT, false, false, 256, 3>(a, dev, stream);
  }
  if (nblocks <= 16) return launch_form<1, ROT, BRANCH, true, 1024, 4>(a, dev, stream);
  // two up to 24 (17408: one token 9.6 us, 2048 109; four a wave 14.5 and 149), then
  // four, in more registers (28672: 98 us against 106) while 12 waves hold the row
  if (nblocks <= 24) return launch_form<2, ROT, BRANCH, false, 768, 3>(a, dev, stream);
  if (nblocks <= 48) return launch_form<4, ROT, BRANCH, false, 768, 3>(a, dev, stream);
  return launch_form<4, ROT, BRANCH, false, 1024, 4>(a, dev, stream);
}

}  // namespace

hipError_t launch_norm_rotate(NormArgs a, const DeviceInfo& dev, hipStream_t stream) {
  if (a.M == 0) return hipSuccess;
  a.inv_k = 1.0 / a.K;
  const bool branch = a.residual != nullptr || a.post_weight != nullptr || a.gate != nullptr || a.branch_scale != 1.0;
  if (a.sign != nullptr) return branch ? launch_blocks<true, true>(a, dev, stream) : launch_blocks<true, false>(a, dev, stream);
  return branch ? launch_blocks<false, true>(a, dev, stream) : launch_blocks<false, false>(a, dev, stream);
}

}  // namespace twl
