// The row-balanced matrix-core decode kernel (M <= 24 tokens), its plan and its
// launches.  Shared by gemv.hip (the linear layer, with and without the fused
// rotation) and gemv_gated.hip (the gated pair of projections).
#pragma once

#include "rotate_block.h"

#include <algorithm>
#include <type_traits>

namespace twl {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i_t __attribute__((ext_vector_type(16)));

// The 16 int8 weights {code * q} of one packed word (16 codes), as the four
// dwords of a dot4 operand (dword i = codes 4i .. 4i+3 of the word).  Fields
// at bits 0-1 / 4-5 of each byte are selectors {0,1,2} into ta = [-q, +q, 0,
// 0]; fields at bits 2-3 / 6-7, masked in place, are selectors {0,4,8}: byte 0
// of tb1 (-q), byte 0 of tb0 (+q), or the sign fill of tb1's byte 1, which is
// 0.  9 VALU operations per 16 codes.
struct QTables {
  uint32_t ta, tb0, tb1;
};

__device__ __forceinline__ QTables make_tables(int qv) {
  const uint32_t neg = static_cast<uint32_t>(-qv) & 0xFFu;
  const uint32_t pos = static_cast<uint32_t>(qv) & 0xFFu;
  return QTables{neg | (pos << 8), pos, neg};
}

__device__ __forceinline__ v4i unpack16(uint32_t w, const QTables& t) {
  const uint32_t w4 = w >> 4;
  v4i b;
  b.x = static_cast<int>(__builtin_amdgcn_perm(0u, t.ta, w & 0x03030303u));
  b.y = static_cast<int>(__builtin_amdgcn_perm(t.tb0, t.tb1, w & 0x0C0C0C0Cu));
  b.z = static_cast<int>(__builtin_amdgcn_perm(0u, t.ta, w4 & 0x03030303u));
  b.w = static_cast<int>(__builtin_amdgcn_perm(t.tb0, t.tb1, w4 & 0x0C0C0C0Cu));
  return b;
}

struct GemvArgs {
  const int8_t* x;
  const float* a_scale;
  const uint8_t* packed;
  const int8_t* q;
  const float* smax;
  void* out;          // y [M,N] (fp32 or bf16) or int32 acc [M,N]
  int32_t* part;      // [slices][M][N] int32 partial sums when slices > 1
  int N, K, G;        // G = K / 128
  int n_rb;           // 64-row blocks
  int slices;         // workgroups per row block (K split across workgroups)
  int out_kind;       // OutKind
  // fused rotation (gemv_rows_kernel with ROT): the kernel quantises its own
  // activations from bf16 x [M, K] (with silu, [gate | up] [M, 2K]) and writes
  // x_i8 [M, K] and a_scale [M] from workgroup 0
  const uint16_t* xb;
  const int8_t* sign;
  int8_t* x_i8_out;
  float* a_scale_out;
  int silu;
};

// Direct global->LDS loads for the activations of the row-balanced kernel.
// Three 1 KB instructions (lane i writes LDS[lds + 1024 k + 16 i]) at address
// sbase (wave-uniform, SGPR pair) + voff_k (per lane).  Issued from inline asm
// so that the compiler does not drain vmcnt before every LDS read; the kernel
// waits for them itself.  The LDS reads of the slot being refilled are
// complete first (lgkmcnt(0)).
// `n` (1 .. 3, wave-uniform) instructions are issued: tokens 8 n .. 23 of a
// slot are not loaded when M <= 8 n.
__device__ __forceinline__ void dma16xn(int n, const void* sbase, uint32_t v0, uint32_t v1, uint32_t v2,
                                        uint32_t lds0, uint32_t lds1, uint32_t lds2) {
  if (n >= 3)
    asm volatile(
        "s_waitcnt lgkmcnt(0)\n\t"
        "s_mov_b32 m0, %3\n\tglobal_load_lds_dwordx4 %0, %6\n\t"
        "s_mov_b32 m0, %4\n\tglobal_load_lds_dwordx4 %1, %6\n\t"
        "s_mov_b32 m0, %5\n\tglobal_load_lds_dwordx4 %2, %6"
        :: "v"(v0), "v"(v1), "v"(v2), "s"(lds0), "s"(lds1), "s"(lds2), "s"(sbase) : "memory", "m0");
  else if (n == 2)
    asm volatile(
        "s_waitcnt lgkmcnt(0)\n\t"
        "s_mov_b32 m0, %2\n\tglobal_load_lds_dwordx4 %0, %4\n\t"
        "s_mov_b32 m0, %3\n\tglobal_load_lds_dwordx4 %1, %4"
        :: "v"(v0), "v"(v1), "s"(lds0), "s"(lds1), "s"(sbase) : "memory", "m0");
  else
    asm volatile(
        "s_waitcnt lgkmcnt(0)\n\t"
        "s_mov_b32 m0, %1\n\tglobal_load_lds_dwordx4 %0, %2"
        :: "v"(v0), "s"(lds0), "s"(sbase) : "memory", "m0");
}

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  // gfx9 s_waitcnt: vmcnt[3:0] + vmcnt_hi[15:14], expcnt[6:4], lgkmcnt[11:8]
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

__device__ __forceinline__ const void* sgpr_ptr(const void* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
  return reinterpret_cast<const void*>((static_cast<uint64_t>(hi) << 32) | lo);
}

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
      (const __attribute__((address_space(3))) char*)(p)));
}

// 16-byte chunk swizzle inside a 128-byte LDS row (distinct chunks for any 8
// consecutive rows, so the column-wise 16-byte reads hit distinct banks).
__device__ __forceinline__ int chunk_swizzle(int row) { return (row ^ (row >> 3)) & 7; }

// Wait until at most `later` groups of PER loads each are outstanding (a
// constant once the caller's loop is unrolled; later <= 4).
template <int PER>
__device__ __forceinline__ void wait_groups_after(int later) {
  switch (later) {
    case 1: wait_vmcnt<PER>(); break;
    case 2: wait_vmcnt<2 * PER>(); break;
    case 3: wait_vmcnt<3 * PER>(); break;
    case 4: wait_vmcnt<4 * PER>(); break;
    default: wait_vmcnt<0>(); break;
  }
}

constexpr int kRedStride = 40;  // [n][m] int32 sums: 64 rows, 32 tokens, padded

// Row-balanced matrix-core decode (M <= 24 tokens, N >= 16 rows per CU).
// Streaming is bound per CU, so each workgroup takes an equal contiguous range
// of rows [r0, r1) (any length up to RS NS) over the whole of K: every CU
// streams the same number of bytes and no partial sums leave the workgroup.
// The rows form NS subtiles of RS rows, the A operand of the MFMA (rows past
// r1 are computed and dropped):
//   RS = 32 (17..24 tokens): v_mfma_i32_32x32x32_i8, lane (j, h) = (row or
//     token j = lane % 32, half h = lane / 32); per 128-k group a lane holds
//     16 packed bytes of its row (k = 64 h .. 64 h + 63), four MFMAs;
//   RS = 16 (up to 16 tokens): v_mfma_i32_16x16x64_i8, lane (j, h) = (row or
//     token j = lane % 16, quarter h = lane / 16); per group a lane holds 8
//     packed bytes (k = 32 h .. 32 h + 31), two MFMAs.  Tokens pad to 16
//     instead of 32 and rows to a multiple of 16.
// Integer sums are exact, so A and B only have to agree on which k each
// (lane group, byte) covers.  The waves split K into runs of at
// most GMAX groups and keep P groups of loads in flight: group jj + P is issued
// as soon as group jj has been consumed (EARLY: as soon as group jj has
// landed, into a (P + 1)-th buffer and activation slot, before group jj is
// computed), so the stream and the unpack / MFMA work overlap.  Loads are
// issued unconditionally (slots past the wave's run re-read its last group)
// so that the compiler's vmcnt waits stay static.
// The activations of a group (at most kXRows tokens x 128 bytes) go to LDS
// by direct loads with 8 lanes per 128-byte row, so each 1 KB load touches 16
// cache lines; read as MFMA operands (16 bytes of one token per lane) they
// would touch 64 per instruction, and the address unit, not HBM, would bound
// the kernel.  Each wave owns P slots (P + 1 with EARLY), one per group in
// flight.
constexpr int kXRows = 24;              // the decode paths take M <= 24
// Word 3 of a raw buffer resource on gfx9-family parts: 32-bit data format
// (DATA_FORMAT = 4 in bits 15..18), no swizzle, no index stride, so the
// range check is a plain byte count.
constexpr int kRawBufferWord3 = 0x00020000;
// cache-policy operand of the buffer loads: nontemporal (the weights are read
// once per call)
constexpr int kCacheNonTemporal = 2;
constexpr int kXSlot = kXRows * 128;    // bytes per group slot
constexpr int kRowsMaxWaves = 8;
// Fused rotation (ROT): at most kRotMaxM tokens of at most kRotMaxK, each wave
// rotating at most kRotBlocksPerWave 1024-blocks; all of x_i8 then stays in
// LDS, rows padded by 16 bytes (so that the tokens' 16-byte reads fall on
// different banks).
constexpr int kRotMaxM = 2;
constexpr int kRotMaxK = 17408;
constexpr int kRotBlocksPerWave = 3;
constexpr int kRotXBytes = kRotMaxM * (kRotMaxK + 16);
// Up to this many tokens the row-balanced kernel uses 16-row subtiles and
// v_mfma_i32_16x16x64_i8 (the tokens are one 16-wide operand); above, 32-row
// subtiles and v_mfma_i32_32x32x32_i8.  Measured 0.1-0.7 us faster per call
// on the decode layers at M = 1, 8 and 16 (5120 -> 17408: 8.62 -> 8.48 us at
// M = 1, 11.10 -> 10.60 at M = 16; 17408 -> 5120: 10.50 -> 9.76 at M = 1).
constexpr int kRows16MaxM = 16;

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
template <int NS, int RS>
struct RowGroup {
  // RS = 32: 16 packed bytes of row 32 s + j, half h; RS = 16: 8 bytes of row 16 s + j, quarter h
  typename std::conditional<RS == 32, uint4, uint2>::type w[NS];
};

// ROT: the workgroup first rotates and quantises the M <= kRotMaxM tokens
// itself (every workgroup, redundantly: at most kRotBlocksPerWave blocks per
// wave), while its first P groups of weights are already in flight; x_i8 then
// stays in LDS for the whole K and no activation is loaded per group.  The
// rotation and the quantiser are those of rotate_quant_act (rotate_block.h),
// so x_i8, a_scale and y equal the two-step result bit for bit.
//
// TH = 2 (16-row subtiles, more than 16 tokens): the tokens form two 16-wide
// B operands (tokens 0-15 and 16-31), so each unpacked weight operand feeds
// two v_mfma_i32_16x16x64_i8 and the rows of a workgroup pad to a multiple
// of 16, not 32.
//
// GATED: the rows are those of two projections in turn (gate, up, gate, ...), a
// workgroup takes whole pairs, and the epilogue writes SiLU(gate) * up of each
// pair, [M, N / 2], straight from the sums in LDS.
template <int NS, int GMAX, int P, int MAXT, bool ROT = false, int RS = 32, bool EARLY = false, int TH = 1,
          bool GATED = false>
__global__ __launch_bounds__(MAXT) void gemv_rows_kernel(GemvArgs a, int M) {
  static_assert(P >= 1 && P <= GMAX, "prefetch depth");
  static_assert(TH == 1 || (TH == 2 && RS == 16 && !ROT), "token halves");
  static_assert(MAXT <= 64 * kRowsMaxWaves, "x slots are sized for 8 waves");
  static_assert(RS == 32 || RS == 16, "subtile rows");
  typedef typename std::conditional<RS == 32, v16i_t, v4i>::type acc_t;
  __shared__ int red[RS * NS * kRedStride];
  // per-wave group slots, or (ROT) all of x_i8: token t at t * (K + 16)
  // EARLY: group jj + P is issued as soon as group jj has landed, before
  // group jj is computed, into a (P + 1)-th buffer and slot
  constexpr int NB = EARLY ? P + 1 : P;
  __shared__ __attribute__((aligned(1024))) int8_t xs[ROT ? kRotXBytes : kRowsMaxWaves * NB * kXSlot];
  __shared__ float rot_buf[ROT ? kRowsMaxWaves * rot::kWaveBufWords : 1];  // rotation transposes
  __shared__ unsigned tok_max[kRotMaxM];  // ROT: absmax bits of each token
  __shared__ float row_scale[32];        // a_scale of the tokens
  __shared__ float col_scale[RS * NS];   // smax of the rows
  // QLDS: the workgroup's rows of q (R x G bytes, contiguous in q, G <= 8
  // GMAX) staged in LDS by coalesced loads, instead of per-lane gathers of
  // the lane's rows (measured, µs: 5120 <- 17408 9.58 -> 8.78 at M = 1 and
  // 13.61 -> 13.18 at M = 24, 5120 -> 17408 8.49 -> 8.25 at M = 1; with
  // 32-row subtiles on 5-group waves, one group in flight, the barrier that
  // publishes the staged rows cost more than it saved: 11.83 -> 12.12 at M =
  // 24 on 5120 -> 17408, so those keep the gathers; the fused kernels
  // publish the rows with the barriers their rotation already has)
  constexpr bool QLDS = GMAX <= 17 && (ROT || !(GMAX == 5 && RS == 32));
  __shared__ __attribute__((aligned(16))) int8_t qs[QLDS ? RS * NS * GMAX * 8 : 4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nw = blockDim.x >> 6;
  const int N = a.N, K = a.K, G = a.G;
  // rows of this workgroup: an even share of N (gridDim.x shares)
  constexpr int kUnit = GATED ? 2 : 1;  // rows that stay together
  const int r0 = kUnit * static_cast<int>((static_cast<int64_t>(blockIdx.x) * (N / kUnit)) / gridDim.x);
  const int r1 = kUnit * static_cast<int>((static_cast<int64_t>(blockIdx.x + 1) * (N / kUnit)) / gridDim.x);
  const int R = r1 - r0;  // 1 .. 32 NS (checked by the planner)

  for (int i = threadIdx.x; i < RS * NS * kRedStride; i += blockDim.x) red[i] = 0;
  if (ROT && threadIdx.x < kRotMaxM) tok_max[threadIdx.x] = 0u;
  __syncthreads();

  const int g0 = (wave * G) / nw;
  const int ng = ((wave + 1) * G) / nw - g0;  // 0 .. GMAX

  // the epilogue's scales, loaded by the last wave now and used after the
  // main loop, so that their latency hides behind the weight stream (clamped
  // indices and no per-lane branch: a divergent load here made the compiler
  // wait for it before the stream was issued)
  const bool scale_wave = wave == nw - 1 && a.out_kind != kOutAcc;
  float sc_row = 0.0f, sc_col0 = 0.0f, sc_col1 = 0.0f;
  if (scale_wave) {
    if (!ROT) sc_row = a.a_scale[min(lane, M - 1)];
    sc_col0 = a.smax[r0 + min(lane, R - 1)];
    sc_col1 = a.smax[r0 + min(lane + 64, R - 1)];
  }

  if (ng > 0) {
    const int j = lane & (RS - 1), h = lane / RS;
    // lanes past the last row of this workgroup re-read that row: the same
    // cache lines, so no bytes beyond the workgroup's own rows are fetched
    // weights through a buffer resource: its base is the workgroup's first
    // row block and its range the row blocks the workgroup's rows touch (at
    // most three of G x 2 KB; a load outside it would return zeros instead of
    // reading another workgroup's rows).  A load then takes its lane offset
    // from a VGPR and the group's offset from an SGPR: no address arithmetic
    // per load.
    const int rb0 = r0 >> 6;
    const __amdgpu_buffer_rsrc_t wres = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(a.packed) + static_cast<size_t>(rb0) * G * 2048, 0,
        (((r1 - 1) >> 6) - rb0 + 1) * G * 2048, kRawBufferWord3);
    uint32_t wbase[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int n = min(r0 + RS * s + j, r1 - 1);
      wbase[s] = static_cast<uint32_t>(((n >> 6) - (r0 >> 6)) * G * 2048 + (n & 63) * 32 + h * (RS == 32 ? 16 : 8));
    }
    // ROT: this wave's blocks of x (block bi = wave + i nw of the M x K/1024
    // blocks is token bi / nblk, block bi % nblk), loaded first: waits complete
    // in issue order, so behind the q and weight loads the rotation would wait
    // for those too
    const int nblk = K >> 10;
    const int nbt = ROT ? M * nblk : 0;  // <= kRotBlocksPerWave * nw (checked by the host)
    rot::BlockIn rin[ROT ? kRotBlocksPerWave : 1];
    if (ROT) {
      // no branch around the loads (a join with loads in flight makes the
      // compiler wait for them): slots past the last block re-load it
#pragma unroll
      for (int i = 0; i < kRotBlocksPerWave; ++i) {
        const int bi = min(wave + i * nw, nbt - 1);
        const int t = bi / nblk, b = bi - t * nblk;
        rin[i] = rot::load_block_rt(a.xb + static_cast<size_t>(t) * (a.silu ? 2 * K : K), a.sign,
                                    a.silu ? K : 0, b, lane);
      }
      __builtin_amdgcn_sched_barrier(0);  // all of them ahead of the q and weight loads
    }
    // q of this lane's rows for all of the wave's groups: QD dwords from the
    // 4-aligned start q[n, g0 & ~3] (rows of q are G bytes, G % 8 == 0, so no
    // dword straddles a row end; dwords past the row end are clamped), loaded
    // once up front instead of one byte gather per group
    // (held in vector registers: as a plain array the compiler may move it to
    // LDS, which then waits on the loads before the other groups are issued)
    constexpr int QD = GMAX / 4 + 2;
    constexpr int QV = QD <= 4 ? 4 : (QD <= 8 ? 8 : 16);
    static_assert(QD <= QV, "q dwords");
    typedef uint32_t qvec __attribute__((ext_vector_type(QV)));
    const int qa = g0 & ~3, qsh = g0 & 3;
    const int qd_last = (G - qa) / 4 - 1;
    qvec qw[QLDS ? 1 : NS];  // indexed by constants only (unrolled), so kept in registers
    // QLDS: dwords t, t + MAXT, ... of the workgroup's R x G bytes of q (from
    // q[r0, 0]: G % 8 == 0, so dword aligned), clamped so that every slot
    // loads (no branch around loads in flight), issued ahead of the weights
    // and written to LDS once the first group has landed (fused: before the
    // rotation's first barrier)
    constexpr int QI = QLDS ? (RS * NS * GMAX * 2 + MAXT - 1) / MAXT : 1;
    const int qdw = R * G / 4;
    uint32_t qr[QI];
    if constexpr (QLDS) {
      const uint32_t* qsrc = reinterpret_cast<const uint32_t*>(a.q + static_cast<size_t>(r0) * G);
#pragma unroll
      for (int i = 0; i < QI; ++i) qr[i] = qsrc[min(static_cast<int>(threadIdx.x) + i * MAXT, qdw - 1)];
    } else {
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const int n = min(r0 + RS * s + j, r1 - 1);
        const uint32_t* qrow = reinterpret_cast<const uint32_t*>(a.q + static_cast<size_t>(n) * G + qa);
        qvec v = {};
#pragma unroll
        for (int d = 0; d < QD; ++d) v[d] = qrow[min(d, qd_last)];
        qw[s] = v;
      }
    }
    // q[n, g0 + jj]: QLDS, one byte of the staged rows; else byte qsh + jj of
    // the lane's run (jj is a constant once unrolled): a 64-bit shift of two
    // dwords picked by constant indices
    const auto qbyte = [&](int s, int jj) {
      if constexpr (QLDS) {
        return static_cast<int>(qs[min(RS * s + j, R - 1) * G + g0 + min(jj, ng - 1)]);
      } else {
        const qvec& v = qw[s];
        const uint64_t w = (static_cast<uint64_t>(v[(jj >> 2) + 1]) << 32) | v[jj >> 2];
        return static_cast<int>(static_cast<int8_t>(w >> (8 * (qsh + (jj & 3)))));
      }
    };
    // activation DMA: instruction i, lane l -> LDS row r = 8 i + l / 8 (token
    // min(r, M - 1)), LDS chunk l % 8 holding global chunk (l % 8) ^ swizzle(r);
    // xi = ceil(M / 8) instructions per group
    const int xi = (M + 7) >> 3;
    uint32_t xoff[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int r = 8 * i + (lane >> 3);
      // 24-bit multiply (tokens < 24, K <= 2^16): a 32-bit result, so the
      // compiler does not form a 64-bit multiply-add whose unused high half
      // could be a register still waiting on a load
      xoff[i] = __umul24(static_cast<uint32_t>(min(r, M - 1)), static_cast<uint32_t>(K)) +
                static_cast<uint32_t>(16 * ((lane & 7) ^ chunk_swizzle(r)));
    }
    const void* xbase = sgpr_ptr(a.x);
    const uint32_t xs_wave = lds_addr(xs) + static_cast<uint32_t>(wave * NB * kXSlot);
    // this lane's operand row in a slot (tokens past kXRows are never reduced)
    const int jr = min(j, kXRows - 1);

    // per group: NS weight loads (VGPR), then the xi activation DMAs; the
    // activation wait below counts on exactly this order.  The weights are
    // read once per call: nontemporal loads (measured 2-3% faster)
    RowGroup<NS, RS> buf[NB];
    auto issue = [&](RowGroup<NS, RS>& d, int jj) {
      const int g = g0 + min(jj, ng - 1);
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        if constexpr (RS == 32) {
          const u32x4 t = __builtin_amdgcn_raw_buffer_load_b128(wres, wbase[s], g * 2048, kCacheNonTemporal);
          d.w[s] = make_uint4(t.x, t.y, t.z, t.w);
        } else {
          const u32x2 t = __builtin_amdgcn_raw_buffer_load_b64(wres, wbase[s], g * 2048, kCacheNonTemporal);
          d.w[s] = make_uint2(t.x, t.y);
        }
      }
      if (!ROT) {
        const uint32_t slot = __builtin_amdgcn_readfirstlane(xs_wave + (jj % NB) * kXSlot);
        const uint32_t gx = static_cast<uint32_t>(g) * 128;
        dma16xn(xi, xbase, xoff[0] + gx, xoff[1] + gx, xoff[2] + gx, slot, slot + 1024, slot + 2048);
      }
    };
#pragma unroll
    for (int jj = 0; jj < P; ++jj) issue(buf[jj], jj);

    if (ROT) {
      // Every wave has groups here (the planner keeps nw <= G), so all of them
      // reach the two barriers.
      float* wb = rot_buf + wave * rot::kWaveBufWords;
      float rv[kRotBlocksPerWave][16];
#pragma unroll
      for (int i = 0; i < kRotBlocksPerWave; ++i) {
        const int bi = wave + i * nw;
        if (bi < nbt) {
          const int t = bi / nblk;
          if (a.silu)
            rot::rotate_loaded<true>(rin[i], lane, wb, rv[i]);
          else
            rot::rotate_loaded<false>(rin[i], lane, wb, rv[i]);
          float m = 0.0f;
#pragma unroll
          for (int e = 0; e < 16; ++e) m = fmaxf(m, fabsf(rv[i][e]));
#pragma unroll
          for (int sh = 32; sh >= 1; sh >>= 1) m = fmaxf(m, __shfl_xor(m, sh));
          // non-negative floats order like their bit patterns
          if (lane == 0) atomicMax(&tok_max[t], __float_as_uint(m));
        }
      }
      if constexpr (QLDS) {
        // the staged q rows, published by the barriers of the rotation
#pragma unroll
        for (int i = 0; i < QI; ++i) {
          const int d = static_cast<int>(threadIdx.x) + i * MAXT;
          if (d < qdw) reinterpret_cast<uint32_t*>(qs)[d] = qr[i];
        }
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kRotBlocksPerWave; ++i) {
        const int bi = wave + i * nw;
        if (bi < nbt) {
          const int t = bi / nblk, b = bi - t * nblk;
          const rot::TokenQuant tq = rot::token_quant(__uint_as_float(tok_max[t]));
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t word = rot::quant_run(rv[i], c, tq);
            const int k = b * rot::kBlock + 256 * c + 4 * lane;
            *reinterpret_cast<uint32_t*>(xs + t * (K + 16) + k) = word;
            if (blockIdx.x == 0) *reinterpret_cast<uint32_t*>(a.x_i8_out + static_cast<size_t>(t) * K + k) = word;
          }
        }
      }
      if (wave == 0 && lane < M) {
        const float sc = rot::token_quant(__uint_as_float(tok_max[lane])).scale;
        row_scale[lane] = sc;
        if (blockIdx.x == 0) a.a_scale_out[lane] = sc;
      }
      __syncthreads();
    }

    acc_t acc[NS];
    acc_t acc2[TH == 2 ? NS : 1];  // TH = 2: tokens 16 .. 31
#pragma unroll
    for (int s = 0; s < NS; ++s) acc[s] = acc_t{0};
#pragma unroll
    for (int s = 0; s < (TH == 2 ? NS : 1); ++s) acc2[s] = acc_t{0};
#pragma unroll
    for (int jj = 0; jj < GMAX; ++jj) {
      RowGroup<NS, RS>& d = buf[jj % NB];
      // this group's activation DMAs are done once at most the loads of the
      // groups issued after it are outstanding (NS + xi per group; counting
      // NS + 1 only makes the wait stricter)
      if (!ROT) wait_groups_after<NS + 1>(min(P - 1, GMAX - 1 - jj));
      asm volatile("" ::: "memory");
      if (EARLY && jj + P < GMAX) issue(buf[(jj + P) % NB], jj + P);
      if (QLDS && !ROT && jj == 0) {
        // the q loads were issued before the weights, so they have landed;
        // every wave has groups (the planner keeps nw <= G), so all reach
        // the barrier
#pragma unroll
        for (int i = 0; i < QI; ++i) {
          const int d = static_cast<int>(threadIdx.x) + i * MAXT;
          if (d < qdw) reinterpret_cast<uint32_t*>(qs)[d] = qr[i];
        }
        __syncthreads();
      }
      if (jj == 0 || jj < ng) {
        // k-chunks (16 bytes) of the group this lane supplies: RS = 32, chunk
        // 4 h + t for MFMA t = 0..3; RS = 16, chunk 2 h + t for MFMA t = 0, 1
        constexpr int NT = RS == 32 ? 4 : 2;
        v4i xv[NT];
        v4i xv2[TH == 2 ? NT : 1];
        if (ROT) {
          const int8_t* xr = xs + min(j, M - 1) * (K + 16) + (g0 + min(jj, ng - 1)) * 128 + 16 * NT * h;
#pragma unroll
          for (int t = 0; t < NT; ++t) xv[t] = *reinterpret_cast<const v4i*>(xr + 16 * t);
        } else {
          const int8_t* xr = xs + (wave * NB + jj % NB) * kXSlot + jr * 128;
#pragma unroll
          for (int t = 0; t < NT; ++t)
            xv[t] = *reinterpret_cast<const v4i*>(xr + 16 * ((NT * h + t) ^ chunk_swizzle(jr)));
          if constexpr (TH == 2) {
            const int jr2 = min(j + 16, kXRows - 1);
            const int8_t* xr2 = xs + (wave * NB + jj % NB) * kXSlot + jr2 * 128;
#pragma unroll
            for (int t = 0; t < NT; ++t)
              xv2[t] = *reinterpret_cast<const v4i*>(xr2 + 16 * ((NT * h + t) ^ chunk_swizzle(jr2)));
          }
        }
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          const QTables tab = make_tables(qbyte(s, jj));
          if constexpr (RS == 32) {
            const uint32_t wv[4] = {d.w[s].x, d.w[s].y, d.w[s].z, d.w[s].w};
#pragma unroll
            for (int t = 0; t < 4; ++t)
              acc[s] = __builtin_amdgcn_mfma_i32_32x32x32_i8(unpack16(wv[t], tab), xv[t], acc[s], 0, 0, 0);
          } else {
            const uint32_t wv[2] = {d.w[s].x, d.w[s].y};
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const v4i wop = unpack16(wv[t], tab);
              acc[s] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wop, xv[t], acc[s], 0, 0, 0);
              if constexpr (TH == 2) acc2[s] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wop, xv2[t], acc2[s], 0, 0, 0);
            }
          }
        }
      }
      if (!EARLY && jj + P < GMAX) issue(d, jj + P);
    }
    // exact cross-wave reduction; lane (j, h) holds token j and, in register
    // r, row 8 (r / 4) + 4 h + (r % 4) of each subtile
    if (j < M) {
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int r = 0; r < (RS == 32 ? 16 : 4); ++r) {
          // RS = 32: register r holds row 8 (r / 4) + 4 h + (r % 4); RS = 16: row 4 h + r
          const int row = RS * s + (RS == 32 ? 8 * (r >> 2) + 4 * h + (r & 3) : 4 * h + r);
          atomicAdd(&red[row * kRedStride + j], acc[s][r]);
        }
    }
    if (TH == 2 && j + 16 < M) {
#pragma unroll
      for (int s = 0; s < (TH == 2 ? NS : 1); ++s)
#pragma unroll
        for (int r = 0; r < 4; ++r) atomicAdd(&red[(RS * s + 4 * h + r) * kRedStride + j + 16], acc2[s][r]);
    }
  }
  if (scale_wave) {
    if (!ROT && lane < M) row_scale[lane] = sc_row;
    if (lane < R) col_scale[lane] = sc_col0;
    if (lane + 64 < R) col_scale[lane + 64] = sc_col1;
  }
  __syncthreads();

  if constexpr (GATED) {
    const int pairs = R / 2;
    const auto value = [&](int t, int rr) {
      return static_cast<float>(red[rr * kRedStride + t]) * row_scale[t] * (col_scale[rr] * (1.0f / 127.0f));
    };
    for (int i = threadIdx.x; i < M * pairs; i += blockDim.x) {
      const int t = i / pairs, pr = i - t * pairs;
      const size_t o = static_cast<size_t>(t) * (N / 2) + r0 / 2 + pr;
      store_out(a.out, o, a.out_kind == kOutGatedBf16 ? kOutBf16 : kOutF32, 0,
                silu_mul(value(t, 2 * pr), value(t, 2 * pr + 1)));
    }
    return;
  }
  for (int i = threadIdx.x; i < M * R; i += blockDim.x) {
    const int t = i / R, rr = i - t * R;
    const int sum = red[rr * kRedStride + t];
    const size_t o = static_cast<size_t>(t) * N + r0 + rr;
    store_out(a.out, o, a.out_kind, sum,
              a.out_kind == kOutAcc ? 0.0f
                                    : static_cast<float>(sum) * row_scale[t] * (col_scale[rr] * (1.0f / 127.0f)));
  }
}

struct GemvPlan {
  int gmax = 2;    // compile-time bound on groups per wave
  int nw = 1;      // waves per workgroup
  int slices = 1;  // workgroups per 64-row block (K split across workgroups)
  int n_rb = 1;
  bool mfma = false;
  // row-balanced MFMA kernel: `rows_wgs` workgroups of an even share of N
  int rows_ns = 0;   // subtiles of rows_rs rows per workgroup (0: not this kernel)
  int rows_rs = 32;
  int rows_wgs = 0;
  int rows_p = 2;    // groups of loads in flight per wave when gmax is 5 or 17
  bool rows_early = false;  // issue a group's successor before computing it
  int rows_th = 1;   // 2: 16-row subtiles with the tokens as two 16-wide operands
};

constexpr int kRowsGmaxChoices[] = {3, 5, 9, 17, 33};

// Row-balanced plan: an even share of rows for every CU (a multiple of the CU
// count of workgroups), at most 3 subtiles of 32 rows each, the whole of K
// split over the waves.  Every workgroup reads all of x_i8 (M x K bytes, by
// coalesced direct loads into LDS) next to its R x K / 4 bytes of weights; the
// plan is taken when each workgroup has at least 16 rows.  Measured against
// the K-split kernel and its second launch: 17408 -> 5120 (20 rows per CU)
// 10.1 against 12.1 us at M = 4, 13.6 against 15.2 us at M = 24; and, for
// these shapes, faster than the dot4 kernel from M = 1 on.
GemvPlan make_rows_plan(int64_t N, int64_t K, const DeviceInfo& dev) {
  GemvPlan p;
  p.slices = 0;
  const int cus = std::max(1, dev.cu_count);
  const int G = static_cast<int>(K >> 7);
  const int64_t per_round = static_cast<int64_t>(cus) * 96;
  const int64_t rounds = (N + per_round - 1) / per_round;
  const int64_t wgs = rounds * cus;
  if (N < 16 * wgs) return p;
  const int64_t rmax = (N + wgs - 1) / wgs;
  p.rows_ns = static_cast<int>((rmax + 31) / 32);
  p.rows_wgs = static_cast<int>(wgs);
  p.n_rb = static_cast<int>((N + 63) / 64);
  p.mfma = true;
  p.slices = 1;
  p.nw = std::min(8, std::max(1, G));
  const int gw = (G + p.nw - 1) / p.nw;
  p.gmax = 0;
  for (int c : kRowsGmaxChoices)
    if (c >= gw) { p.gmax = c; break; }
  if (p.gmax == 0) p.slices = 0;
  return p;
}

// make_rows_plan with the subtile form and the loads in flight chosen for M tokens
// (slices = 0 where the row-balanced kernel does not apply).
GemvPlan tuned_rows_plan(int64_t M, int64_t N, int64_t K, const DeviceInfo& dev) {
  GemvPlan r = make_rows_plan(N, K, dev);
  if (r.slices > 0 && M <= kRows16MaxM) {
    // 16-row subtiles and v_mfma_i32_16x16x64_i8: tokens padded to 16, not
    // 32, and the rows of a workgroup to a multiple of 16
    const int64_t rmax = (N + r.rows_wgs - 1) / r.rows_wgs;
    r.rows_rs = 16;
    r.rows_ns = static_cast<int>((rmax + 15) / 16);
  } else if (r.slices > 0 && r.gmax == 5) {
    // more than 16 tokens on 5-group waves: 16-row subtiles with two
    // 16-token operands where they pad the rows less than 32-row subtiles
    // (68 rows: 80, not 96), each unpacked weight operand feeding two
    // MFMAs.  Measured against the 32-row form, one group in flight and
    // issued early in both (µs, alternating on one box, bit-identical y):
    // 5120 -> 17408 10.43 -> 10.09 at M = 24, 10.20 -> 9.82 at M = 17;
    // 5120 -> 34816 17.32 -> 16.31 at M = 24, 17.23 -> 15.66 at M = 20.
    // Deeper prefetch was slower (three groups early: 10.80 and 20.18 at
    // M = 24; two, not early: 10.81 and 16.76).
    const int64_t rmax = (N + r.rows_wgs - 1) / r.rows_wgs;
    const int ns16 = static_cast<int>((rmax + 15) / 16);
    if (ns16 * 16 < r.rows_ns * 32 && ns16 <= 6) {
      r.rows_rs = 16;
      r.rows_ns = ns16;
      r.rows_th = 2;
    }
  }
  if (r.slices > 0) {
    // Loads in flight per wave, measured (µs, alternating on one box):
    // - 5-group waves (K = 5120) keep two by default (the workgroup then
    //   needs 65 KB of LDS, so two share a CU where N needs two rounds of
    //   workgroups, 5120 -> 34816).
    // - With 32-row subtiles (17..24 tokens) one group in flight, the next
    //   issued as soon as it has landed, before it is computed ("early"),
    //   is faster: 10.59 -> 9.66 on 5120 -> 17408, 16.94 -> 15.96 on
    //   5120 -> 34816, 6.57 -> 6.45 on 5120 -> 5120 at M = 24.
    // - With one round of workgroups and 16-row subtiles: all five, not
    //   early, on one subtile (4096 rows: 4.21 against 4.28 us with three
    //   early at M = 1); three, early, on two (5120 -> 5120, 20 rows: 5.22
    //   -> 5.00 at M = 1, 6.08 -> 5.67 at M = 16, against all five);
    //   with more subtiles two, early, up to 8 tokens and one above
    //   (5120 -> 17408: 8.23 -> 7.86 at M = 1, 8.57 -> 8.21 at M = 8,
    //   8.88 -> 8.42 at M = 12, 9.19 -> 8.65 at M = 16, against three).
    // - Two rounds of workgroups (5120 -> 34816) with 16-row subtiles keep
    //   two up to 8 tokens (one early: 11.43 -> 11.64 at M = 1) and one,
    //   early, above (14.20 -> 13.58 at M = 16).
    // - 17-group waves (K = 17408) keep five; with 16-row subtiles three
    //   early are faster (5120 <- 17408: 9.71 -> 9.49 at M = 1, 9.79 ->
    //   9.60 at M = 8), with 32-row subtiles slower (13.36 -> 15.08).
    const bool one_round = r.rows_wgs <= dev.cu_count;
    if (r.gmax == 5) {
      if (r.rows_rs == 32 || r.rows_th == 2) {
        r.rows_p = 1;
        r.rows_early = true;
      } else if (one_round) {
        r.rows_p = r.rows_ns == 1 ? 5 : r.rows_ns == 2 ? 3 : (M <= 8 ? 2 : 1);
        r.rows_early = r.rows_ns > 1;
      } else if (M > 8) {
        r.rows_p = 1;
        r.rows_early = true;
      }
    } else if (r.gmax == 17 && r.rows_rs == 16 && one_round) {
      r.rows_p = 3;
      r.rows_early = true;
    }
  }
  return r;
}

template <int NS, int MAXT, bool ROT = false, int RS = 32, bool GATED = false>
hipError_t launch_rows_ns(GemvArgs a, int M, const GemvPlan& pl, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(pl.rows_wgs));
  const dim3 block(64 * pl.nw);
  // the kernel stages q with MAXT threads (nw = 8 whenever K >= 1024)
  if (64 * pl.nw != MAXT) return hipErrorInvalidValue;
  // groups of loads in flight per wave, within the register budget: the
  // plan's rows_p and rows_early for 5- and 17-group waves, else 5 (3 for
  // 3-group waves)
  constexpr int PM = 5;
  switch (pl.gmax) {
    case 3: hipLaunchKernelGGL((gemv_rows_kernel<NS, 3, 3, MAXT, ROT, RS, false, 1, GATED>),
                               grid, block, 0, stream, a, M); break;
    case 5:
      if constexpr (!ROT) {
        if (pl.rows_early) {
          if (pl.rows_p == 1) {
            hipLaunchKernelGGL((gemv_rows_kernel<NS, 5, 1, MAXT, false, RS, true, 1, GATED>),
                               grid, block, 0, stream, a, M);
            break;
          }
          if constexpr (RS == 16) {
            if (pl.rows_p == 2) {
              hipLaunchKernelGGL((gemv_rows_kernel<NS, 5, 2, MAXT, false, RS, true, 1, GATED>),
                                 grid, block, 0, stream, a, M);
              break;
            }
            if (pl.rows_p == 3) {
              hipLaunchKernelGGL((gemv_rows_kernel<NS, 5, 3, MAXT, false, RS, true, 1, GATED>),
                                 grid, block, 0, stream, a, M);
              break;
            }
          }
          return hipErrorInvalidValue;
        }
        if constexpr (RS == 16 && NS == 1) {
          if (pl.rows_p == 5) {
            hipLaunchKernelGGL((gemv_rows_kernel<NS, 5, 5, MAXT, false, RS, false, 1, GATED>),
                               grid, block, 0, stream, a, M);
            break;
          }
        }
      }
      // the fused kernels (their x_i8 fills the LDS) on at most two subtiles:
      // two groups, early (5120 -> 5120: 7.24 -> 7.00 us at M = 1, 8.23 ->
      // 7.97 at M = 2; one early, or two early on more subtiles, was slower)
      if constexpr (ROT && NS <= 2) {
        hipLaunchKernelGGL((gemv_rows_kernel<NS, 5, 2, MAXT, ROT, RS, true, 1, GATED>), grid, block, 0, stream, a, M);
        break;
      }
      // two groups in flight, not early: two rounds of workgroups up to 8
      // tokens, and the other fused kernels
      hipLaunchKernelGGL((gemv_rows_kernel<NS, 5, 2, MAXT, ROT, RS, false, 1, GATED>), grid, block, 0, stream, a, M);
      break;
    case 9: hipLaunchKernelGGL((gemv_rows_kernel<NS, 9, PM, MAXT, ROT, RS, false, 1, GATED>),
                               grid, block, 0, stream, a, M); break;
    case 17:
      if constexpr (!ROT && RS == 16) {
        if (pl.rows_early && pl.rows_p == 3) {
          hipLaunchKernelGGL((gemv_rows_kernel<NS, 17, 3, MAXT, false, RS, true, 1, GATED>),
                             grid, block, 0, stream, a, M);
          break;
        }
      }
      hipLaunchKernelGGL((gemv_rows_kernel<NS, 17, PM, MAXT, ROT, RS, false, 1, GATED>),
                         grid, block, 0, stream, a, M);
      break;
    case 33:
      // K > kRotMaxK: never planned with ROT
      if (ROT) return hipErrorInvalidValue;
      hipLaunchKernelGGL((gemv_rows_kernel<NS, 33, PM, MAXT, false, RS, false, 1, GATED>),
                         grid, block, 0, stream, a, M);
      break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

// 16-row subtiles with two 16-token operands (TH = 2): 5-group waves, one
// group in flight, its successor issued early (as for 32-row subtiles).
template <int NS, bool GATED>
hipError_t launch_rows_halves(GemvArgs a, int M, const GemvPlan& pl, hipStream_t stream) {
  if (pl.nw != 8 || pl.gmax != 5 || !pl.rows_early || pl.rows_p != 1) return hipErrorInvalidValue;
  hipLaunchKernelGGL((gemv_rows_kernel<NS, 5, 1, 512, false, 16, true, 2, GATED>), dim3(static_cast<unsigned>(pl.rows_wgs)),
                     dim3(512), 0, stream, a, M);
  return hipGetLastError();
}

template <bool ROT, bool GATED = false>
hipError_t launch_rows(GemvArgs a, int M, const GemvPlan& pl, hipStream_t stream) {
  if constexpr (!ROT) {
    if (pl.rows_rs == 16 && pl.rows_th == 2) {
      switch (pl.rows_ns) {
        case 1: return launch_rows_halves<1, GATED>(a, M, pl, stream);
        case 2: return launch_rows_halves<2, GATED>(a, M, pl, stream);
        case 3: return launch_rows_halves<3, GATED>(a, M, pl, stream);
        case 4: return launch_rows_halves<4, GATED>(a, M, pl, stream);
        case 5: return launch_rows_halves<5, GATED>(a, M, pl, stream);
        case 6: return launch_rows_halves<6, GATED>(a, M, pl, stream);
        default: return hipErrorInvalidValue;
      }
    }
  }
  if (pl.rows_rs == 16) {
    switch (pl.rows_ns) {
      case 1: return launch_rows_ns<1, 512, ROT, 16, GATED>(a, M, pl, stream);
      case 2: return launch_rows_ns<2, 512, ROT, 16, GATED>(a, M, pl, stream);
      case 3: return launch_rows_ns<3, 512, ROT, 16, GATED>(a, M, pl, stream);
      case 4: return launch_rows_ns<4, 512, ROT, 16, GATED>(a, M, pl, stream);
      case 5: return launch_rows_ns<5, 512, ROT, 16, GATED>(a, M, pl, stream);
      case 6: return launch_rows_ns<6, 512, ROT, 16, GATED>(a, M, pl, stream);
      default: return hipErrorInvalidValue;
    }
  }
  if constexpr (ROT) {
    return hipErrorInvalidValue;  // the fused kernels use 16-row subtiles
  } else {
    switch (pl.rows_ns) {
      case 1: return launch_rows_ns<1, 512, false, 32, GATED>(a, M, pl, stream);
      case 2: return launch_rows_ns<2, 512, false, 32, GATED>(a, M, pl, stream);
      case 3: return launch_rows_ns<3, 512, false, 32, GATED>(a, M, pl, stream);
      default: return hipErrorInvalidValue;
    }
  }
}

}  // namespace
}  // namespace twl
