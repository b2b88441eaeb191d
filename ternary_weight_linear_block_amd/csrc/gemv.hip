// Decode ternary linear (M <= 24 tokens): two HBM-streaming kernels over the
// packed 2-bit weights, a VALU int8 dot-product GEMV for the smallest batches
// and a matrix-core variant for the rest.
//
// Method ([P1] "Ternary-Bonsai-2-27B on 2x RTX 5070 with vLLM TP=2", section 4
// for the arithmetic, section 5 for the prior art): the same exact int32
// accumulator as the prefill GEMM,
//   acc[t,n] = sum_k x_i8[t,k] * code[n,k] * q[n, k/128],
//   y[t,n]   = acc[t,n] * a_scale[t] * smax[n] / 127.
// The pages tried a dp4a decode GEMV on their GPU (section 5 table: 2.1x as a
// kernel, +2% end to end, rejected because its error grew); here both decode
// kernels are bit-exact with the GEMM because all compute the same integer sum.
//
// gfx950 mapping (both kernels)
//   * A workgroup holds one 64-row block and one K range; each wave takes a
//     run of at most GMAX consecutive 128-groups of that range and issues the
//     loads of its whole run up front (up to GMAX x 2 KB per wave in flight),
//     so the memory system sees the matrix as one burst instead of a
//     latency-bound sequence of small reads.  In the tiled weight layout a
//     wave's group is one contiguous 2 KB tile, read with two 1 KB loads.
//   * Per packed word: 1 shift, 4 ANDs, 4 byte-permutes against tables built
//     from {-q, +q, 0} give the 16 int8 weights code * q.
//   * The waves' partial sums meet in LDS through integer atomics (exact).
//     Streaming is bound per CU (about 22 GB/s each, measured), so every CU
//     needs an equal share: when there are too few row blocks, K is also split
//     across workgroups ("slices"), each slice writes its int32 partial sums to
//     the workspace and a second kernel adds them in slice order and rescales.
// dot4 kernel (gemv_kernel): lane l owns row n0 + l; one half-wave swap
//   (v_permlane32_swap) gives each lane its row's 8 words, then 4 v_dot4 per
//   word and token, with the activations read at wave-uniform addresses
//   through the constant address space (scalar loads, one copy per wave).
//   Its VALU work grows with M: it is used for M < 4 on layers too narrow
//   for the row-balanced kernel.
// MFMA kernels: the tokens padded to 32 form the B operand of
//   v_mfma_i32_32x32x32_i8 (in gemv_rows_kernel at up to 16 tokens: padded to
//   16, v_mfma_i32_16x16x64_i8; above 16 tokens, where 16-row subtiles pad the
//   rows less, two 16-token operands of that instruction) and the unpacked
//   weights the A operand, which makes the work nearly independent of M.
//   gemv_rows_kernel gives every CU an equal contiguous range of rows over all
//   of K (no partial sums leave the workgroup) and is used at every M whenever
//   each CU gets at least 16 rows;
//   gemv_mfma_kernel keeps the 64-row-block split with K slices (4 <= M <= 24)
//   for layers with fewer rows per CU.
#include "gemv_rows.h"

#include <algorithm>
#include <cstdio>
#include <cstdlib>

namespace twl {
namespace {

constexpr int kMaxWaves = 16;

// Activations are read at wave-uniform addresses; reading them through the
// constant address space makes them scalar loads (one copy in SGPRs for the
// whole wave) instead of 64 identical vector loads.
typedef __attribute__((address_space(4))) const u32x4 const_u32x4;

// v_permlane32_swap_b32 exchanges lanes 32..63 of its first operand with lanes
// 0..31 of its second: applied to each dword of two 16-byte values it moves
// lo's upper-lane half into hi's lower lanes and back.
__device__ __forceinline__ void swap_halves(uint4& lo, uint4& hi) {
  auto r0 = __builtin_amdgcn_permlane32_swap(lo.x, hi.x, false, false);
  auto r1 = __builtin_amdgcn_permlane32_swap(lo.y, hi.y, false, false);
  auto r2 = __builtin_amdgcn_permlane32_swap(lo.z, hi.z, false, false);
  auto r3 = __builtin_amdgcn_permlane32_swap(lo.w, hi.w, false, false);
  lo = make_uint4(r0[0], r1[0], r2[0], r3[0]);
  hi = make_uint4(r0[1], r1[1], r2[1], r3[1]);
}

// MT is the exact number of tokens (1 .. 24).  A workgroup of nw waves covers
// one 64-row block and one K slice; its waves split the slice's groups as
// evenly as possible, at most GMAX each.  Static LDS: MT x 64 ints for the
// cross-wave sums.
template <int MT, int GMAX>
__global__ __launch_bounds__(1024) void gemv_kernel(GemvArgs a) {
  __shared__ int red[MT * 64];
  const int lane = threadIdx.x & 63;
  // wave index as a scalar: everything derived from it (the K range, the
  // activation addresses) is then known to be wave-uniform
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nw = blockDim.x >> 6;
  const int rb = blockIdx.x % a.n_rb;
  const int slice = blockIdx.x / a.n_rb;
  const int n0 = rb * 64;
  const int N = a.N, K = a.K, G = a.G;

  for (int i = threadIdx.x; i < MT * 64; i += blockDim.x) red[i] = 0;
  __syncthreads();

  const int s_lo = (slice * G) / a.slices;
  const int s_n = ((slice + 1) * G) / a.slices - s_lo;
  const int g0 = s_lo + (wave * s_n) / nw;
  const int ng = s_lo + ((wave + 1) * s_n) / nw - g0;   // 0 .. GMAX

  if (ng > 0) {
    // The group's weights are one contiguous 2 KB tile (64 rows x 32 bytes;
    // rows past N are code-0 padding), read with two 1 KB loads: in load A
    // lane l < 32 takes bytes 0-15 of row l and lane l >= 32 bytes 16-31 of
    // row l - 32; load B the same for rows 32..63.  One half-swap (lanes
    // 32..63 of A with lanes 0..31 of B) then leaves lane l with bytes 0-15
    // (A) and 16-31 (B) of its own row n0 + l.
    const int hsel = lane >> 5;
    const int rlo = lane & 31;
    const uint8_t* srcA = a.packed + static_cast<size_t>(rb) * G * 2048 + rlo * 32 + hsel * 16;
    const uint8_t* srcB = srcA + 1024;
    const int8_t* qrow = a.q + static_cast<size_t>(min(n0 + lane, N - 1)) * G;

    // all of this wave's groups in flight at once (slots past ng re-read the
    // last group, which is already on its way: no extra HBM traffic)
    uint4 dA[GMAX], dB[GMAX];
#pragma unroll
    for (int j = 0; j < GMAX; ++j) {
      const size_t g = static_cast<size_t>(g0 + min(j, ng - 1));
      dA[j] = *reinterpret_cast<const uint4*>(srcA + g * 2048);
      dB[j] = *reinterpret_cast<const uint4*>(srcB + g * 2048);
    }
    int qv[GMAX];
#pragma unroll
    for (int j = 0; j < GMAX; ++j) qv[j] = qrow[g0 + min(j, ng - 1)];

    // small M: two accumulator chains per token so consecutive dot4s do not
    // wait on each other
    constexpr int NA = MT <= 4 ? 2 : 1;
    int acc[NA][MT];
#pragma unroll
    for (int c = 0; c < NA; ++c)
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[c][t] = 0;

#pragma unroll
    for (int j = 0; j < GMAX; ++j) {
      if (j != 0 && j >= ng) continue;   // ng >= 1: group 0 always runs
      uint4 lo = dA[j], hi = dB[j];
      swap_halves(lo, hi);
      const uint32_t words[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
      const QTables tab = make_tables(qv[j]);
      const int8_t* xg = a.x + static_cast<size_t>(g0 + j) * 128;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        const v4i wq = unpack16(words[w], tab);
        const int wq0 = wq.x, wq1 = wq.y, wq2 = wq.z, wq3 = wq.w;
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          const u32x4 xv = *(const const_u32x4*)(xg + static_cast<size_t>(t) * K + 16 * w);
          int s = acc[w % NA][t];
          s = __builtin_amdgcn_sdot4(wq0, static_cast<int>(xv.x), s, false);
          s = __builtin_amdgcn_sdot4(wq1, static_cast<int>(xv.y), s, false);
          s = __builtin_amdgcn_sdot4(wq2, static_cast<int>(xv.z), s, false);
          s = __builtin_amdgcn_sdot4(wq3, static_cast<int>(xv.w), s, false);
          acc[w % NA][t] = s;
        }
      }
    }
    // exact cross-wave reduction (integer LDS atomics, order independent)
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      int s = acc[0][t];
#pragma unroll
      for (int c = 1; c < NA; ++c) s += acc[c][t];
      atomicAdd(&red[t * 64 + lane], s);
    }
  }
  __syncthreads();

  const int n = n0 + lane;
  auto finish = [&](int t, int s) {
    const size_t o = static_cast<size_t>(t) * N + n;
    const float v = a.out_kind == kOutAcc
                        ? 0.0f
                        : static_cast<float>(s) * a.a_scale[t] * (a.smax[n] * (1.0f / 127.0f));
    store_out(a.out, o, a.out_kind, s, v);
  };
  if (a.slices == 1) {
    if (n < N)
      for (int t = wave; t < MT; t += nw) finish(t, red[t * 64 + lane]);
    return;
  }

  // K is split across workgroups: this slice's partial sums go to the
  // workspace; gemv_reduce_kernel adds the slices in order and rescales.  (A
  // last-arriver scheme inside this kernel needs device-scope fences, which
  // write back the L2 on this multi-XCD part and were measured to cost far
  // more than the second launch.)
  if (n < N)
    for (int t = wave; t < MT; t += nw)
      a.part[(static_cast<size_t>(slice) * MT + t) * N + n] = red[t * 64 + lane];
}

// Decode with the matrix cores (M = 2 .. 32 tokens, padded to 32).  Same
// work split as gemv_kernel (one 64-row block and one K slice per workgroup,
// a run of at most GMAX groups per wave), but each group is 8 MFMAs
// v_mfma_i32_32x32x32_i8: A = the unpacked weights of 32 rows x 32 k
// (subtile s = rows 32 s .. 32 s + 31 of the block, k-step t), B = 32 k x 32
// tokens of x_i8.  The k values of a (lane half h, k-step t) pair only have to
// agree between A and B: lane half h at k-step t covers k = 16 (4 h + t) ..
// +15 of the group, so a lane's weights for the whole group are the 16
// contiguous packed bytes [16 h, 16 h + 16) of its row (one load per subtile,
// no lane exchange), and its activations are the 64 contiguous bytes
// [64 h, 64 h + 64) of token row j of the group.  Columns j >= M re-read row
// M - 1 and are never reduced.
template <int GMAX, int MAXT>
__global__ __launch_bounds__(MAXT) void gemv_mfma_kernel(GemvArgs a, int M) {
  __shared__ int red[64 * kRedStride];
  typedef int v16i __attribute__((ext_vector_type(16)));
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nw = blockDim.x >> 6;
  const int rb = blockIdx.x % a.n_rb;
  const int slice = blockIdx.x / a.n_rb;
  const int n0 = rb * 64;
  const int N = a.N, K = a.K, G = a.G;

  for (int i = threadIdx.x; i < 64 * kRedStride; i += blockDim.x) red[i] = 0;
  __syncthreads();

  const int s_lo = (slice * G) / a.slices;
  const int s_n = ((slice + 1) * G) / a.slices - s_lo;
  const int g0 = s_lo + (wave * s_n) / nw;
  const int ng = s_lo + ((wave + 1) * s_n) / nw - g0;   // 0 .. GMAX

  if (ng > 0) {
    const int j = lane & 31;   // A: weight row in the subtile; B: token column
    const int h = lane >> 5;   // lane half
    const uint8_t* srcA = a.packed + static_cast<size_t>(rb) * G * 2048 + j * 32 + h * 16;
    const uint8_t* srcB = srcA + 1024;
    const int8_t* qrowA = a.q + static_cast<size_t>(min(n0 + j, N - 1)) * G;
    const int8_t* qrowB = a.q + static_cast<size_t>(min(n0 + 32 + j, N - 1)) * G;
    const int8_t* xrow = a.x + static_cast<size_t>(min(j, M - 1)) * K + h * 64;

    uint4 dA[GMAX], dB[GMAX];
    v4i xv[GMAX][4];
#pragma unroll
    for (int jj = 0; jj < GMAX; ++jj) {
      const size_t g = static_cast<size_t>(g0 + min(jj, ng - 1));
      dA[jj] = *reinterpret_cast<const uint4*>(srcA + g * 2048);
      dB[jj] = *reinterpret_cast<const uint4*>(srcB + g * 2048);
#pragma unroll
      for (int t = 0; t < 4; ++t) xv[jj][t] = *reinterpret_cast<const v4i*>(xrow + g * 128 + 16 * t);
    }
    int qa[GMAX], qb[GMAX];
#pragma unroll
    for (int jj = 0; jj < GMAX; ++jj) {
      qa[jj] = qrowA[g0 + min(jj, ng - 1)];
      qb[jj] = qrowB[g0 + min(jj, ng - 1)];
    }

    v16i acc0 = {}, acc1 = {};
#pragma unroll
    for (int jj = 0; jj < GMAX; ++jj) {
      if (jj != 0 && jj >= ng) continue;   // ng >= 1: group 0 always runs
      const QTables ta = make_tables(qa[jj]);
      const QTables tb = make_tables(qb[jj]);
      const uint32_t wa[4] = {dA[jj].x, dA[jj].y, dA[jj].z, dA[jj].w};
      const uint32_t wb[4] = {dB[jj].x, dB[jj].y, dB[jj].z, dB[jj].w};
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        acc0 = __builtin_amdgcn_mfma_i32_32x32x32_i8(unpack16(wa[t], ta), xv[jj][t], acc0, 0, 0, 0);
        acc1 = __builtin_amdgcn_mfma_i32_32x32x32_i8(unpack16(wb[t], tb), xv[jj][t], acc1, 0, 0, 0);
      }
    }
    // exact cross-wave reduction.  32x32 accumulator layout: lane (j, h) holds
    // column j (token) and, in register r, row 8 (r / 4) + 4 h + (r % 4)
    if (j < M) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int row = 8 * (r >> 2) + 4 * h + (r & 3);
        atomicAdd(&red[row * kRedStride + j], acc0[r]);
        atomicAdd(&red[(32 + row) * kRedStride + j], acc1[r]);
      }
    }
  }
  __syncthreads();

  const int n = n0 + lane;
  if (n >= N) return;
  for (int t = wave; t < M; t += nw) {
    const int s = red[lane * kRedStride + t];
    const size_t o = static_cast<size_t>(t) * N + n;
    if (a.slices > 1)
      a.part[static_cast<size_t>(slice) * M * N + o] = s;
    else
      store_out(a.out, o, a.out_kind, s,
                a.out_kind == kOutAcc ? 0.0f
                                      : static_cast<float>(s) * a.a_scale[t] * (a.smax[n] * (1.0f / 127.0f)));
  }
}

// Sum of the slices' partial sums in slice order, then the rescale.
__global__ __launch_bounds__(256) void gemv_reduce_kernel(const int32_t* __restrict__ part,
                                                          int slices, int M, int N,
                                                          const float* __restrict__ a_scale,
                                                          const float* __restrict__ smax,
                                                          void* __restrict__ out, int out_kind) {
  const size_t total = static_cast<size_t>(M) * N;
  const size_t stride = static_cast<size_t>(gridDim.x) * blockDim.x;
  for (size_t i = static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += stride) {
    int s = 0;
    for (int sl = 0; sl < slices; ++sl) s += part[static_cast<size_t>(sl) * total + i];
    float v = 0.0f;
    if (out_kind != kOutAcc) {
      const int t = static_cast<int>(i / static_cast<size_t>(N));
      const int n = static_cast<int>(i - static_cast<size_t>(t) * N);
      v = static_cast<float>(s) * a_scale[t] * (smax[n] * (1.0f / 127.0f));
    }
    store_out(out, i, out_kind, s, v);
  }
}

// From this many tokens on, the matrix-core kernel beats the dot4 kernel
// (measured on both decode shapes: at 4 tokens they are about even, at 8 the
// MFMA kernel is 1.3-1.6x faster, at 24 2.6-3.5x).
constexpr int kMfmaMinM = 4;

constexpr int kGmaxChoices[] = {2, 3, 5, 9};

// Streaming cost model (measured on MI355X): each CU moves about 22 GB/s, so
// the busiest CU's bytes set the time; splitting K over several workgroups per
// row block evens the CUs out but costs a second launch (about 3.5 us).
constexpr double kCuBytesPerUs = 22.0e3;
constexpr double kReduceUs = 3.5;

GemvPlan make_plan_for(int64_t M, int64_t N, int64_t K, const DeviceInfo& dev, bool mfma) {
  const int G = static_cast<int>(K >> 7);
  const int cus = std::max(1, dev.cu_count);
  GemvPlan best;
  best.slices = 0;  // none found yet
  double best_t = 1e30;
  for (int slices = 1; slices <= 32 && slices <= G; ++slices) {
    GemvPlan p;
    p.mfma = mfma;
    p.n_rb = static_cast<int>((N + 63) / 64);
    p.slices = slices;
    const int per_slice = (G + slices - 1) / slices;
    // two or three groups per wave keeps many waves in flight; at most 16
    // waves, at most 9 groups each (MFMA kernel, for its register budget: at
    // most 3 groups with 16 waves, 5 with 8)
    p.nw = std::min(kMaxWaves, std::max(1, per_slice / 2));
    int gw = (per_slice + p.nw - 1) / p.nw;
    if (mfma && gw > 3 && p.nw > 8) {
      p.nw = 8;
      gw = (per_slice + p.nw - 1) / p.nw;
    }
    if (gw > (mfma ? 5 : 9)) continue;
    for (int c : kGmaxChoices)
      if (c >= gw) { p.gmax = c; break; }
    const int64_t wgs = static_cast<int64_t>(p.n_rb) * slices;
    const double per_cu = static_cast<double>((wgs + cus - 1) / cus) * 64.0 * per_slice * 32.0;
    // partial sums: written once, read once by the reduce kernel (~4 TB/s)
    const double part_us = slices > 1 ? 2.0 * slices * static_cast<double>(M) * N * 4 / 4.0e6 : 0.0;
    const double t = per_cu / kCuBytesPerUs + (slices > 1 ? kReduceUs + part_us : 0.0);
    if (t < best_t - 1e-9) { best_t = t; best = p; }
  }
  return best;
}

// The plan of the kernels for narrow layers: the K-split matrix-core kernel where
// wanted and it applies, else the dot4 kernel.  Always returns a valid plan for
// 1 <= M <= 24 and K <= the library's limit: the dot4 kernel takes up to 16
// waves x 9 groups x 32 slices.
GemvPlan make_narrow_plan(int64_t M, int64_t N, int64_t K, bool want_mfma, const DeviceInfo& dev) {
  if (want_mfma && M <= 32) {
    const GemvPlan p = make_plan_for(M, N, K, dev, true);
    if (p.slices > 0) return p;
  }
  return make_plan_for(M, N, K, dev, false);
}

// Automatic choice: the row-balanced matrix-core kernel whenever its plan
// applies (at every M), else the dot4 kernel below kMfmaMinM tokens and the
// K-split matrix-core kernel from there on.
GemvPlan make_plan(int64_t M, int64_t N, int64_t K, GemvKind kind, const DeviceInfo& dev) {
  if (kind != kGemvDot4 && M <= kXRows) {
    const GemvPlan r = tuned_rows_plan(M, N, K, dev);
    if (r.slices > 0) return r;
  }
  return make_narrow_plan(M, N, K, kind == kGemvMfma || (kind == kGemvAuto && M >= kMfmaMinM), dev);
}

hipError_t launch_mfma(GemvArgs a, int M, const GemvPlan& pl, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(pl.n_rb * pl.slices));
  const dim3 block(64 * pl.nw);
  switch (pl.gmax) {
    case 2: hipLaunchKernelGGL((gemv_mfma_kernel<2, 1024>), grid, block, 0, stream, a, M); break;
    case 3: hipLaunchKernelGGL((gemv_mfma_kernel<3, 1024>), grid, block, 0, stream, a, M); break;
    default: hipLaunchKernelGGL((gemv_mfma_kernel<5, 512>), grid, block, 0, stream, a, M); break;
  }
  return hipGetLastError();
}

template <int MT>
hipError_t launch_mt(GemvArgs a, const GemvPlan& pl, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(pl.n_rb * pl.slices));
  const dim3 block(64 * pl.nw);
  switch (pl.gmax) {
    case 2: hipLaunchKernelGGL((gemv_kernel<MT, 2>), grid, block, 0, stream, a); break;
    case 3: hipLaunchKernelGGL((gemv_kernel<MT, 3>), grid, block, 0, stream, a); break;
    case 5: hipLaunchKernelGGL((gemv_kernel<MT, 5>), grid, block, 0, stream, a); break;
    default: hipLaunchKernelGGL((gemv_kernel<MT, 9>), grid, block, 0, stream, a); break;
  }
  return hipGetLastError();
}

// One of the kernels for narrow layers, as the plan says.
hipError_t launch_narrow(const GemvArgs& a, int64_t M, const GemvPlan& pl, hipStream_t stream) {
  if (pl.mfma) {
    if (M > 32 || pl.nw * 64 > (pl.gmax <= 3 ? 1024 : 512)) return hipErrorInvalidValue;
    return launch_mfma(a, static_cast<int>(M), pl, stream);
  }
  switch (static_cast<int>(M)) {
    case 1: return launch_mt<1>(a, pl, stream);
    case 2: return launch_mt<2>(a, pl, stream);
    case 3: return launch_mt<3>(a, pl, stream);
    case 4: return launch_mt<4>(a, pl, stream);
    case 5: return launch_mt<5>(a, pl, stream);
    case 6: return launch_mt<6>(a, pl, stream);
    case 7: return launch_mt<7>(a, pl, stream);
    case 8: return launch_mt<8>(a, pl, stream);
    case 9: return launch_mt<9>(a, pl, stream);
    case 10: return launch_mt<10>(a, pl, stream);
    case 11: return launch_mt<11>(a, pl, stream);
    case 12: return launch_mt<12>(a, pl, stream);
    case 13: return launch_mt<13>(a, pl, stream);
    case 14: return launch_mt<14>(a, pl, stream);
    case 15: return launch_mt<15>(a, pl, stream);
    case 16: return launch_mt<16>(a, pl, stream);
    case 17: return launch_mt<17>(a, pl, stream);
    case 18: return launch_mt<18>(a, pl, stream);
    case 19: return launch_mt<19>(a, pl, stream);
    case 20: return launch_mt<20>(a, pl, stream);
    case 21: return launch_mt<21>(a, pl, stream);
    case 22: return launch_mt<22>(a, pl, stream);
    case 23: return launch_mt<23>(a, pl, stream);
    case 24: return launch_mt<24>(a, pl, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

void gemv_plan_info(int64_t M, int64_t N, int64_t K, GemvKind kind, const DeviceInfo& dev, int64_t* info) {
  const GemvPlan pl = make_plan(M, N, K, kind, dev);
  const bool rows = pl.rows_ns > 0;
  info[0] = rows ? 2 : (pl.mfma ? 4 : 3);
  info[1] = rows ? (N + pl.rows_wgs - 1) / pl.rows_wgs : 64;
  info[2] = 0;
  info[3] = pl.slices;
  info[4] = rows ? pl.rows_wgs : static_cast<int64_t>(pl.n_rb) * pl.slices;
  info[5] = pl.nw;
  info[6] = pl.slices > 1 ? 1 : 0;
  info[7] = pl.slices > 1 ? static_cast<int64_t>(pl.slices) * M * N * 4 : 0;
}

size_t gemv_workspace_bytes(int64_t M, int64_t N, int64_t K, GemvKind kind, const DeviceInfo& dev) {
  if (M <= 0 || N <= 0 || K <= 0) return 0;
  const GemvPlan pl = make_plan(M, N, K, kind, dev);
  if (pl.slices <= 1) return 0;
  return static_cast<size_t>(pl.slices) * static_cast<size_t>(M) * static_cast<size_t>(N) * 4;
}

hipError_t launch_gemv(const int8_t* x_i8, const float* a_scale, const uint8_t* packed,
                       const int8_t* q, const float* smax, int64_t M, int64_t N, int64_t K,
                       void* out, OutKind out_kind, void* part, size_t part_bytes, GemvKind kind,
                       const DeviceInfo& dev, hipStream_t stream) {
  if (M == 0 || N == 0) return hipSuccess;
  const GemvPlan pl = make_plan(M, N, K, kind, dev);
  if (pl.slices <= 0 || (kind == kGemvMfma && !pl.mfma)) return hipErrorInvalidValue;
  if (pl.slices > 1 && (part == nullptr || part_bytes < gemv_workspace_bytes(M, N, K, kind, dev)))
    return hipErrorInvalidValue;
  if (std::getenv("TWL_LOG")) {
    // the row kernel's form: subtiles, token operands, groups of loads in
    // flight per wave (as launch_rows_ns dispatches them) and early issue
    char form[96] = "";
    if (pl.rows_ns > 0) {
      const int depth = pl.gmax == 3 ? 3 : (pl.gmax == 5 || (pl.gmax == 17 && pl.rows_early)) ? pl.rows_p : 5;
      std::snprintf(form, sizeof(form), ", %d-row subtiles x%d%s, %d in flight%s", pl.rows_rs, pl.rows_ns,
                    pl.rows_th == 2 ? " (two 16-token operands)" : "", depth, pl.rows_early ? ", early" : "");
    }
    std::fprintf(stderr, "[twl] gemv%s M=%lld N=%lld K=%lld -> <= %d groups/wave, %d waves/WG, %d slices, grid=%d%s\n",
                 pl.rows_ns > 0 ? "-rows" : (pl.mfma ? "-mfma" : ""), static_cast<long long>(M),
                 static_cast<long long>(N), static_cast<long long>(K), pl.gmax, pl.nw, pl.slices,
                 pl.rows_ns > 0 ? pl.rows_wgs : pl.n_rb * pl.slices, form);
  }
  GemvArgs a = {};
  a.x = x_i8;
  a.a_scale = a_scale;
  a.packed = packed;
  a.q = q;
  a.smax = smax;
  a.out = out;
  a.part = static_cast<int32_t*>(part);
  a.N = static_cast<int>(N);
  a.K = static_cast<int>(K);
  a.G = static_cast<int>(K >> 7);
  a.n_rb = pl.n_rb;
  a.slices = pl.slices;
  a.out_kind = out_kind;
  hipError_t e = hipErrorInvalidValue;
  if (pl.rows_ns > 0) {
    if (M > kXRows || pl.nw * 64 > 512) return hipErrorInvalidValue;  // x slots hold kXRows tokens
    e = launch_rows<false>(a, static_cast<int>(M), pl, stream);
  } else {
    e = launch_narrow(a, M, pl, stream);
  }
  if (e != hipSuccess || pl.slices <= 1) return e;
  const size_t total = static_cast<size_t>(M) * static_cast<size_t>(N);
  const unsigned blocks = static_cast<unsigned>(std::min<size_t>((total + 255) / 256, 4096));
  hipLaunchKernelGGL(gemv_reduce_kernel, dim3(blocks), dim3(256), 0, stream, a.part, pl.slices,
                     static_cast<int>(M), a.N, a_scale, smax, out, a.out_kind);
  return hipGetLastError();
}

int gemv_part_slices(int64_t M, int64_t N, int64_t K, const DeviceInfo& dev) {
  return make_narrow_plan(M, N, K, M >= kMfmaMinM, dev).slices;
}

hipError_t launch_gemv_part(const int8_t* x_i8, const uint8_t* packed, const int8_t* q, int64_t M,
                            int64_t N, int64_t K, int32_t* part, const DeviceInfo& dev,
                            hipStream_t stream) {
  const GemvPlan pl = make_narrow_plan(M, N, K, M >= kMfmaMinM, dev);
  if (pl.slices <= 0) return hipErrorInvalidValue;
  GemvArgs a = {};
  a.x = x_i8;
  a.packed = packed;
  a.q = q;
  a.out = part;  // one slice: the accumulators themselves
  a.part = part;
  a.N = static_cast<int>(N);
  a.K = static_cast<int>(K);
  a.G = static_cast<int>(K >> 7);
  a.n_rb = pl.n_rb;
  a.slices = pl.slices;
  a.out_kind = kOutAcc;
  return launch_narrow(a, M, pl, stream);
}

// The fused decode kernel applies when the row-balanced plan does with one
// round of workgroups and the whole rotation fits the workgroup: at most
// kRotMaxM tokens of at most kRotMaxK, and at most 2 1024-blocks per wave
// (kRotBlocksPerWave = 3 for a single token).  Measured against the two
// launches (µs): 5120 -> 17408 9.7 / 12.0 at M = 1, 10.5 / 11.6 at M = 2,
// but 11.8 / 11.5 at M = 3 and 12.3 / 12.0 at M = 4 (three rounds of
// rotation per wave); 5120 -> 5120 7.4 / 8.5 at M = 1, 9.3 / 8.4 at M = 3;
// 5120 -> 34816 (two rounds of workgroups, each rotating again) 18.0 / 14.5
// at M = 1.
bool gemv_rot_applies(int64_t M, int64_t N, int64_t K, const DeviceInfo& dev) {
  if (M < 1 || M > kRotMaxM || K > kRotMaxK || N < 1) return false;
  const GemvPlan pl = make_rows_plan(N, K, dev);
  if (pl.slices <= 0 || pl.rows_ns <= 0 || pl.gmax > 17 || pl.nw * 64 > 512 || pl.nw > (K >> 7))
    return false;
  if (pl.rows_wgs > dev.cu_count) return false;
  const int64_t rounds = M == 1 ? kRotBlocksPerWave : 2;
  return M * (K >> 10) <= rounds * pl.nw;
}

hipError_t launch_gemv_rot(const uint16_t* x, const int8_t* sign, bool silu, const uint8_t* packed,
                           const int8_t* q, const float* smax, int64_t M, int64_t N, int64_t K,
                           void* out, OutKind out_kind, int8_t* x_i8, float* a_scale,
                           const DeviceInfo& dev, hipStream_t stream) {
  if (!gemv_rot_applies(M, N, K, dev)) return hipErrorNotSupported;
  // 16-row subtiles and v_mfma_i32_16x16x64_i8, tokens padded to 16, as the
  // two-step path uses at these batch sizes
  GemvPlan pl = make_rows_plan(N, K, dev);
  pl.rows_rs = 16;
  pl.rows_ns = static_cast<int>((N + pl.rows_wgs - 1) / pl.rows_wgs + 15) / 16;
  if (std::getenv("TWL_LOG"))
    std::fprintf(stderr, "[twl] gemv-rows+rotation M=%lld N=%lld K=%lld silu=%d -> <= %d groups/wave, %d waves/WG, grid=%d\n",
                 static_cast<long long>(M), static_cast<long long>(N), static_cast<long long>(K),
                 silu ? 1 : 0, pl.gmax, pl.nw, pl.rows_wgs);
  GemvArgs a = {};
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
  a.xb = x;
  a.sign = sign;
  a.x_i8_out = x_i8;
  a.a_scale_out = a_scale;
  a.silu = silu ? 1 : 0;
  return launch_rows<true>(a, static_cast<int>(M), pl, stream);
}

}  // namespace twl
