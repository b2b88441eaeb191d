// lora_add: low-rank adapters of many requests beside a shared projection.
//
// Mathematics, for token t with adapter a = ids[t] (none when a is outside
// 0 .. n-1: then out[t] = y[t]):
//   v[t, r]   = sum_k x[t, k] A[a, r, k]
//   out[t, n] = y[t, n] + sum_r (scale[a] v[t, r]) B[a, n, r]
//
// A decode batch of small adapters takes one kernel, a token and a share of n to a
// workgroup (lora_token_kernel).  All else takes two, both on
// v_mfma_f32_16x16x32_bf16 with the adapter's rows as the first operand and 16
// tokens as the second, so that a lane's results are consecutive ranks (or n) of one
// token:
//   shrink  a workgroup takes 16 consecutive tokens and a slice of K, its waves
//           split the slice; their sums meet in LDS (in wave order) and the slice's
//           sum goes to the workspace, fp32 [slices][M][R].
//   expand  a workgroup takes 16 or 64 consecutive tokens and a range of n; it adds
//           the slices in order, scales, and splits v into two bf16 terms (three for
//           fp32 y), v = hi + lo (+ lo2) with hi = bf16(v), lo = bf16(v - hi): the
//           remainder is at most 2^-16 (2^-24) of v, where a single bf16 would cost
//           2^-8, as much as the rounding of a bf16 y.
// Tokens keep their order: a tile finds its distinct adapters with ballots over
// the ids and makes one pass for each, storing only that adapter's tokens.  So no
// sort precedes the kernels, batches in request order (the usual one) make one or
// two passes, and an adapter that holds NaN reaches its own tokens only.  With few
// tokens the passes of a tile go to different workgroups.
#include "twl_internal.h"

#include <algorithm>
#include <type_traits>

namespace twl {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef unsigned int v4u __attribute__((ext_vector_type(4)));

// With 32 tokens four waves, whose LDS leaves three workgroups a CU (eight: 4096
// tokens of rank 64 117 us instead of 110); with 16 eight, each with less of K (500
// tokens of K = 17408 25.3 us, four 26.7; 1000 tokens of rank 16 17.5 and 16.3).
constexpr int shrink_waves(int ts) { return ts == 1 ? 8 : 4; }
constexpr int kExpandWaves = 4;
constexpr int kLdsBytes = 160 * 1024;  // of a CU

__device__ __forceinline__ v8bf load8(const uint16_t* p) { return *reinterpret_cast<const v8bf*>(p); }

// The distinct adapters of a tile of up to 64 consecutive tokens, one pass each,
// in the order of their first token.  All of it is wave-uniform but `id`.
struct Passes {
  int id;          // lane l: adapter of token l of the tile, -1 for none
  uint64_t rest;   // tokens whose adapter has not had its pass

  __device__ __forceinline__ Passes(const int32_t* ids, int64_t t0, int tokens, int64_t M, int n, int lane) {
    const int64_t t = t0 + lane;
    const bool in = lane < tokens && t < M;
    const int v = ids[in ? t : M - 1];
    id = in && v >= 0 && v < n ? v : -1;
    rest = __ballot(id >= 0);
  }
  __device__ __forceinline__ bool next(int& adapter, uint64_t& tokens) {
    if (rest == 0) return false;
    adapter = __builtin_amdgcn_readlane(id, __builtin_ctzll(rest));
    tokens = __ballot(id == adapter);
    rest &= ~tokens;
    return true;
  }
};

// Workgroups are dispatched to the XCDs in turn: work item of workgroup `bid` of
// `total` such that each XCD gets a contiguous range of the items, whose neighbours
// share an adapter's rows in its L2 (4096 tokens of rank 64 on 17408: 110 us, with
// the items in order 126).  Workgroups of later passes stand behind all of the first
// passes', so that those without a pass cost little (between them: 135 against 114).
__device__ __forceinline__ int xcd_item(int bid, int total) {
  constexpr int kXcds = 8;
  const int per = total / kXcds, rem = total % kXcds, xcd = bid % kXcds;
  return xcd * per + min(xcd, rem) + bid / kXcds;
}

typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

// two fp32 -> two bf16, to nearest even (v_cvt_pk_bf16_f32)
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const v2f f = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, v2bf));
}

// LDS operations of one wave execute in order; this only keeps the compiler from
// moving the reads of other lanes' data above the writes, or the next writes above
// these reads.
__device__ __forceinline__ void wave_lds_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Work item (p, slice, tile): passes p, p + passes, ... of 16 TS tokens over one
// slice of K.  RT: 16-row fragments of the rank.
//
// A load straight into the operand's layout (lane = 16 bytes of one of 16 rows)
// touches 64 cache lines an instruction, and the address unit bounds the kernel
// (4096 tokens of 5120, rank 64: 59 us).  So a wave loads 64 k of its rows with 8
// lanes a row and 8 rows an instruction, and turns them over in LDS of its own
// (16-byte units swizzled by row, no bank conflicts): no barrier before the sums
// meet.  The next 64 k are on their way while these are multiplied; two units at
// once cost the LDS of other workgroups (400 tokens of 16 adapters, rank 16, both
// kernels: 41.5 against 36.3 us).
//
// 25 us for 4096 tokens of 5120 and rank 64, 1.7 TB/s of x: still the address unit
// (half of the time busy), which A passes through once for 32 tokens; 13 us for 500
// tokens of 17408, 2.7 TB/s of x and A.
template <int RT, int TS>
__global__ __launch_bounds__(64 * shrink_waves(TS)) void lora_shrink_kernel(LoraArgs a) {
  constexpr int kShrinkWaves = shrink_waves(TS);
  constexpr int TM = 16 * TS;
  constexpr int kStride = 16 * RT + 4;  // floats of a token's row of sums, padded
  constexpr int G = 2 * (TS + RT);      // groups of 8 rows: x, then A
  constexpr int kStage = G * 1024, kSums = TM * kStride * 4;
  __shared__ __attribute__((aligned(16))) char lds[kShrinkWaves * (kStage > kSums ? kStage : kSums)];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int j = lane & 15, q = lane >> 4;
  const uint32_t items = a.slices * a.shrink_tiles;
  const int p = blockIdx.x / items;
  const uint32_t item = xcd_item(blockIdx.x - p * items, items);
  const int slice = item / a.shrink_tiles, tile = item - slice * a.shrink_tiles;
  const int64_t t0 = static_cast<int64_t>(tile) * TM;
  const int K = a.K, R = a.R;
  // this wave's 64-k units
  const uint32_t units = K / 64, parts = a.slices * kShrinkWaves, part = slice * kShrinkWaves + wave;
  const int u0 = static_cast<int>(units * part / parts), u1 = static_cast<int>(units * (part + 1) / parts);  // <= 2^10 parts
  char* stage = lds + wave * kStage;
  float* sums = reinterpret_cast<float*>(lds);  // [wave][token][rank], when the staging is done

  const int r8 = lane >> 3, c8 = lane & 7;  // row of a group and 16-byte unit of this lane's loads
  const char* xb = reinterpret_cast<const char*>(a.x + static_cast<size_t>(t0) * K);
  const int rows = static_cast<int>(std::min<int64_t>(TM, a.M - t0));
  uint32_t off[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int r = g < 2 * TS ? min(8 * g + r8, rows - 1) : min(8 * (g - 2 * TS) + r8, R - 1);
    off[g] = static_cast<uint32_t>(r) * static_cast<uint32_t>(2 * K) + 16 * c8;
  }
  const int put = r8 * 128 + 16 * (c8 ^ r8);
  const auto get = [&](int frag, int s) {  // fragment frag (x, then A), k step s of the unit
    const int at = (2 * frag + (j >> 3)) * 1024 + (j & 7) * 128 + 16 * ((4 * s + q) ^ (j & 7));
    return *reinterpret_cast<const v8bf*>(stage + at);
  };

  v4u raw[G];
  const auto load = [&](int g0, int g1, const char* base, int u) {  // a unit past the last re-reads it and is not multiplied
#pragma unroll
    for (int g = 0; g < G; ++g)
      if (g >= g0 && g < g1) raw[g] = *reinterpret_cast<const v4u*>(base + off[g] + 128 * max(min(u, u1 - 1), 0));
  };
  constexpr int kAll = 2 * TS;  // groups of x
  Passes passes(a.ids, t0, TM, a.M, a.n, lane);
  int adapter;
  uint64_t tokens;
  for (int skip = p; passes.next(adapter, tokens); --skip) {
    if (skip != 0) continue;
    skip = a.shrink_passes;
    const char* ab = reinterpret_cast<const char*>(a.a + static_cast<size_t>(adapter) * R * K);
    v4f acc[TS][RT];
#pragma unroll
    for (int h = 0; h < TS; ++h)
#pragma unroll
      for (int f = 0; f < RT; ++f) acc[h][f] = v4f{0};
    load(0, kAll, xb, u0);
    load(kAll, G, ab, u0);
    for (int u = u0; u < u1; ++u) {
      wave_lds_sync();  // the previous unit has been read
#pragma unroll
      for (int g = 0; g < G; ++g) *reinterpret_cast<v4u*>(stage + g * 1024 + put) = raw[g];
      load(0, kAll, xb, u + 1);
      load(kAll, G, ab, u + 1);
      wave_lds_sync();
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        v8bf xv[TS];
#pragma unroll
        for (int h = 0; h < TS; ++h) xv[h] = get(h, s);
#pragma unroll
        for (int f = 0; f < RT; ++f) {
          const v8bf av = get(TS + f, s);
#pragma unroll
          for (int h = 0; h < TS; ++h) acc[h][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, xv[h], acc[h][f], 0, 0, 0);
        }
      }
    }
    // lane (j, q) holds ranks 16 f + 4 q .. + 3 of token 16 h + j
    __syncthreads();  // every wave is past its staging
#pragma unroll
    for (int h = 0; h < TS; ++h)
#pragma unroll
      for (int f = 0; f < RT; ++f)
        *reinterpret_cast<v4f*>(sums + (wave * TM + 16 * h + j) * kStride + 16 * f + 4 * q) = acc[h][f];
    __syncthreads();
    for (int e = threadIdx.x; e < TM * (R / 4); e += 64 * kShrinkWaves) {
      const int tok = e / (R / 4), r = 4 * (e % (R / 4));
      if (!((tokens >> tok) & 1)) continue;
      v4f sum = *reinterpret_cast<const v4f*>(sums + tok * kStride + r);
#pragma unroll
      for (int w = 1; w < kShrinkWaves; ++w) sum += *reinterpret_cast<const v4f*>(sums + (w * TM + tok) * kStride + r);
      *reinterpret_cast<v4f*>(a.part + (static_cast<size_t>(slice) * a.M + t0 + tok) * R + r) = sum;
    }
    __syncthreads();  // the sums have been read: the next pass stages over them
  }
}

// Loads and stores through a buffer resource: a lane whose offset is kOutside reads
// zeros and writes nothing, so no branch stands around them (behind a branch the
// compiler cannot count what is in flight and waits for all of it).  Ranges stay
// below 2^31 bytes.
constexpr int kRawBufferWord3 = 0x00020000;  // 32-bit data format, no swizzle: a byte count as range
constexpr uint32_t kOutside = 0x80000000u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, size_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, static_cast<int>(bytes), kRawBufferWord3);
}

// One wave's 16 tokens x 64 n of y, in y's type: pieces of 16 bytes, 8 (fp32: 16)
// lanes a token, where rows are 4-byte aligned (the memory instructions ask for no
// more); bf16 rows of odd N in pieces of one n, for which 1855 tokens of 9216 -> 5955,
// rank 64, take 41 us, with 5954 n 37 and 5952 (16-byte aligned) 34.
template <bool BF16, int PIECE>
struct Out {
  static constexpr int kSize = BF16 ? 2 : 4;
  static constexpr int kItems = 16 * kSize / PIECE;  // instructions
  static constexpr int kEach = PIECE / kSize;        // elements of a piece
  static constexpr int kLanes = 64 / kEach;          // lanes a token
  static_assert(PIECE == 16 || (BF16 && PIECE == 2), "pieces");
  typedef typename std::conditional<PIECE == 16, v4u, uint16_t>::type Raw;
  Raw raw[kItems];

  static __device__ __forceinline__ int token(int i, int lane) { return (64 * i + lane) / kLanes; }
  static __device__ __forceinline__ int column(int lane) { return kEach * (lane % kLanes); }

  static __device__ __forceinline__ Raw load(__amdgpu_buffer_rsrc_t buf, uint32_t at) {
    if constexpr (PIECE == 16) return __builtin_amdgcn_raw_buffer_load_b128(buf, at, 0, 0);
    else return __builtin_amdgcn_raw_buffer_load_b16(buf, at, 0, 0);
  }
  static __device__ __forceinline__ void store(Raw v, __amdgpu_buffer_rsrc_t buf, uint32_t at) {
    if constexpr (PIECE == 16) __builtin_amdgcn_raw_buffer_store_b128(v, buf, at, 0, 0);
    else __builtin_amdgcn_raw_buffer_store_b16(v, buf, at, 0, 0);
  }

  // adds d[0 ..] to item i
  __device__ __forceinline__ Raw sum(int i, const float* d) const {
    Raw w;
    if constexpr (PIECE == 2) {
      w = static_cast<uint16_t>(pack_bf16(__uint_as_float(static_cast<uint32_t>(raw[i]) << 16) + d[0], 0.0f));
    } else if constexpr (BF16) {
      const v4f lo = *reinterpret_cast<const v4f*>(d), hi = *reinterpret_cast<const v4f*>(d + 4);
      const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = pack_bf16(__uint_as_float(raw[i][e] << 16) + v[2 * e], __uint_as_float(raw[i][e] & 0xFFFF0000u) + v[2 * e + 1]);
    } else {
      const v4f v = *reinterpret_cast<const v4f*>(d);
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(__uint_as_float(raw[i][e]) + v[e]);
    }
    return w;
  }
};

// The same element by element, for the last columns of rows that are no whole number
// of pieces: out = y + d (d in LDS, a row of kStride floats a token; null: nothing) of
// the tokens of `tokens`, one token an instruction, lane = one n.  at: byte offset of
// the first token's element of this lane; row: bytes of a row.
template <bool BF16, int kStride>
__device__ __forceinline__ void finish_columns(__amdgpu_buffer_rsrc_t y, __amdgpu_buffer_rsrc_t out, const float* d,
                                               uint32_t tokens, uint32_t at, uint32_t row, bool in, int lane) {
#pragma unroll 1
  for (int t = 0; t < 16; ++t) {
    const uint32_t o = in && ((tokens >> t) & 1) != 0 ? at + t * row : kOutside;
    if constexpr (BF16) {
      uint16_t v = __builtin_amdgcn_raw_buffer_load_b16(y, o, 0, 0);
      if (d != nullptr)
        v = static_cast<uint16_t>(pack_bf16(__uint_as_float(static_cast<uint32_t>(v) << 16) + d[t * kStride + lane], 0.0f));
      __builtin_amdgcn_raw_buffer_store_b16(v, out, o, 0, 0);
    } else {
      uint32_t v = __builtin_amdgcn_raw_buffer_load_b32(y, o, 0, 0);
      if (d != nullptr) v = __float_as_uint(__uint_as_float(v) + d[t * kStride + lane]);
      __builtin_amdgcn_raw_buffer_store_b32(v, out, o, 0, 0);
    }
  }
}

// LDS-only workgroup barrier: this wave's LDS operations have completed, then the
// waves meet (loads and stores in flight are not waited for).
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Work item (p, chunk, tile): passes p, p + passes, ... of 16 WT tokens over an even
// share of the ranges of 64 WN n, WN = 4 / WT.  A wave has 16 tokens x 64 n: with
// WT = 4 the waves share B's 64 rows, with WT = 1 (few tokens) each has its own.
// RS: 32-rank steps.
//
// As in the shrink kernel nothing is read or written in the matrix layout, whose
// lanes lie a row of y apart: B's 64 rows are one piece of memory, copied to LDS in
// order, and the products go through LDS to where y's 16-byte pieces are.  v stays
// in registers; the next range's B and the next two's y are on their way while one
// is computed.
//
// 85 us for 4096 tokens of rank 64 on 17408, bf16: 3.4 TB/s of y in and out, and as
// many bytes of B from L2 again; what is left is the wait for ids, partial sums and
// first operands (16 us when no second pass runs beside them).
constexpr int kOutStride = 64 + 4;  // floats of a token's products in LDS, padded

struct ExpandLds {
  int row;    // bf16 of a row of v or B, padded
  int bufs;   // buffers of B: shared ones alternate (one barrier a range)
  int b, vd;  // bytes: B; v's terms before the loop, then the products
  constexpr ExpandLds(int wt, int rs, bool bf16)
      : row(32 * rs + 8), bufs(wt > 1 ? 2 : 1), b(bufs * (kExpandWaves / wt) * 64 * row * 2),
        vd(std::max((bf16 ? 2 : 3) * 16 * wt * row * 2, kExpandWaves * 16 * kOutStride * 4)) {}
};

template <int WT, int RS, bool BF16, int PIECE>
__global__ __launch_bounds__(64 * kExpandWaves) void lora_expand_kernel(LoraArgs a) {
  using Y = Out<BF16, PIECE>;
  constexpr ExpandLds L(WT, RS, BF16);
  constexpr int TM = 16 * WT, WN = kExpandWaves / WT, TERMS = BF16 ? 2 : 3;
  constexpr int kStride = L.row, NB = L.bufs;
  constexpr int BL = 4 * RS / WT;  // 16-byte loads a lane for 64 rows of B of full rank
  constexpr int kSize = BF16 ? 2 : 4;
  static_assert(BL >= 1, "loads of B");
  __shared__ __attribute__((aligned(16))) uint16_t b_lds[NB][WN][64 * kStride];
  static_assert(sizeof(b_lds) == L.b, "what the launcher counts");
  __shared__ __attribute__((aligned(16))) char vd_lds[L.vd];
  uint16_t* vt = reinterpret_cast<uint16_t*>(vd_lds);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wt = wave % WT, wn = wave / WT;
  const int j = lane & 15, q = lane >> 4;
  const uint32_t items = a.expand_chunks * a.expand_tiles;
  const int p = blockIdx.x / items;
  const uint32_t item = xcd_item(blockIdx.x - p * items, items);
  const int chunk = item / a.expand_tiles, tile = item - chunk * a.expand_tiles;
  const int64_t t0 = static_cast<int64_t>(tile) * TM;
  const int N = a.N, R = a.R;
  const int step = 64 * WN, ranges = (N + step - 1) / step;
  // this wave's 64 n of the chunk's ranges: n_lo, n_lo + step, ... below n_hi
  const int n_lo = static_cast<int>(static_cast<int64_t>(ranges) * chunk / a.expand_chunks) * step + 64 * wn;
  const int n_hi = min(N, static_cast<int>(static_cast<int64_t>(ranges) * (chunk + 1) / a.expand_chunks) * step);
  const int n_end = n_hi + 64 * wn;  // every wave goes round as often as the first
  float* dw = reinterpret_cast<float*>(vd_lds) + wave * 16 * kOutStride;
  const int col = Y::column(lane);
  const size_t tile_bytes = static_cast<size_t>(std::min<int64_t>(TM, a.M - t0)) * N * kSize;
  const size_t tile_at = static_cast<size_t>(t0) * N * kSize;
  const __amdgpu_buffer_rsrc_t y_buf = buffer_of(static_cast<const char*>(a.y) + tile_at, tile_bytes);
  const __amdgpu_buffer_rsrc_t out_buf = buffer_of(static_cast<char*>(a.out) + tile_at, tile_bytes);

  Passes passes(a.ids, t0, TM, a.M, a.n, lane);
  // byte offset in the tile of this lane's piece i at n = 0 for the wave's tokens of
  // `tokens`, kOutside for others (adding n leaves it outside: rows stay below 2^30)
  const auto piece = [&](uint64_t tokens, int i) {
    const int t = 16 * wt + Y::token(i, lane);
    return ((tokens >> t) & 1) != 0 ? static_cast<uint32_t>(t * N + col) * kSize : kOutside;
  };
  // ranges below n_vec are whole pieces, the row's last may go element by element
  const int n_vec = N % Y::kEach == 0 ? n_hi : min(n_hi, N & ~63);
  const auto at = [&](uint32_t piece0, int nb) { return nb + col < n_vec ? piece0 + static_cast<uint32_t>(nb) * kSize : kOutside; };
  const auto finish = [&](const float* d, uint64_t tokens, int nb) {
    finish_columns<BF16, kOutStride>(y_buf, out_buf, d, static_cast<uint32_t>(tokens >> (16 * wt)),
                                     static_cast<uint32_t>(16 * wt * N + nb + lane) * kSize, static_cast<uint32_t>(N) * kSize,
                                     nb + lane < N, lane);
  };

  // tokens without an adapter: copied with the tile's first pass, or here if it has none
  uint64_t none = a.out != a.y && p == 0 ? __ballot(passes.id < 0 && lane < TM && t0 + lane < a.M) : 0;
  if (passes.rest == 0) {
    for (int nb = n_lo; nb < n_hi; nb += 4 * step) {
      typename Y::Raw y[4][Y::kItems];
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int i = 0; i < Y::kItems; ++i) y[u][i] = Y::load(y_buf, at(piece(none, i), nb + u * step));
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int i = 0; i < Y::kItems; ++i) Y::store(y[u][i], out_buf, at(piece(none, i), nb + u * step));
      for (int u = 0; u < 4; ++u)
        if (nb + u * step >= n_vec && nb + u * step < n_hi)
          finish(nullptr, none, nb + u * step);
    }
    return;
  }
  // the 16-byte pieces of 64 rows of B, R / 8 a row, by their place in memory: where
  // this lane's go in LDS
  const int pieces = 8 * R, first_piece = 64 * wt + lane;
  uint32_t b_at[BL];
#pragma unroll
  for (int l = 0; l < BL; ++l) {
    const uint32_t c = first_piece + 64 * WT * l, r = c / (static_cast<uint32_t>(R) / 8u);
    b_at[l] = r * kStride + 8 * (c - r * (R / 8));
  }
  if (R < 32 * RS) {  // the columns past the rank stay zero: v is zero there, B has to be finite
    for (uint32_t e = threadIdx.x; e < sizeof(b_lds) / 16; e += 64 * kExpandWaves)
      reinterpret_cast<v4u*>(&b_lds[0][0][0])[e] = v4u{0, 0, 0, 0};
    lds_barrier();
  }
  int adapter;
  uint64_t tokens;
  for (int skip = p; passes.next(adapter, tokens); --skip) {
    if (skip != 0) continue;
    skip = a.expand_passes;
    const __amdgpu_buffer_rsrc_t b_buf =
        buffer_of(a.b + static_cast<size_t>(adapter) * N * R, static_cast<size_t>(N) * R * 2);
    v4u braw[BL];
    const auto load_b = [&](int nb) {  // rows past the adapter's end are zeros
#pragma unroll
      for (int l = 0; l < BL; ++l) {
        const int c = first_piece + 64 * WT * l;
        braw[l] = __builtin_amdgcn_raw_buffer_load_b128(b_buf, nb < n_hi && c < pieces ? 2u * nb * R + 16u * c : kOutside, 0, 0);
      }
    };
    const uint64_t written = tokens | none;
    uint32_t own[Y::kItems];
    bool copied[Y::kItems];  // this token takes nothing from the adapter
#pragma unroll
    for (int i = 0; i < Y::kItems; ++i) {
      own[i] = piece(written, i);
      copied[i] = ((none >> (16 * wt + Y::token(i, lane))) & 1) != 0;
    }
    const auto load_y = [&](Y& y, int nb) {
#pragma unroll
      for (int i = 0; i < Y::kItems; ++i) y.raw[i] = Y::load(y_buf, at(own[i], nb));
    };
    Y even, odd;
    load_b(n_lo);
    load_y(even, n_lo);
    load_y(odd, n_lo + step);
    const float scale = a.scale[adapter];
    lds_barrier();  // the previous pass's products have been read
    for (int e = threadIdx.x; e < TM * 8 * RS; e += 64 * kExpandWaves) {
      const int tok = e / (8 * RS), r = 4 * (e % (8 * RS));
      v4f v = {0.0f, 0.0f, 0.0f, 0.0f};
      if (r < R && ((tokens >> tok) & 1)) {
        const float* src = a.part + static_cast<size_t>(t0 + tok) * R + r;
        const size_t next = static_cast<size_t>(a.M) * R;
        for (int s = 0; s < a.slices; s += 8) {  // eight loads in flight, added in order
          v4f part[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) part[u] = *reinterpret_cast<const v4f*>(src + min(s + u, a.slices - 1) * next);
#pragma unroll
          for (int u = 0; u < 8; ++u)
            if (s + u < a.slices) v += part[u];
        }
        v *= scale;
      }
#pragma unroll
      for (int term = 0; term < TERMS; ++term) {
        const uint2 b = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
        v -= v4f{__uint_as_float(b.x << 16), __uint_as_float(b.x & 0xFFFF0000u), __uint_as_float(b.y << 16),
                 __uint_as_float(b.y & 0xFFFF0000u)};
        *reinterpret_cast<uint2*>(vt + (term * TM + tok) * kStride + r) = b;
      }
    }
    lds_barrier();
    v8bf v[TERMS][RS];
#pragma unroll
    for (int term = 0; term < TERMS; ++term)
#pragma unroll
      for (int s = 0; s < RS; ++s) v[term][s] = load8(vt + (term * TM + 16 * wt + j) * kStride + 32 * s + 8 * q);
    lds_barrier();  // v's place takes the products
    const auto range = [&](Y& y, int nb, int buf) {
      uint16_t* bw = b_lds[WT > 1 ? buf : 0][wn];
      if (WT == 1) wave_lds_sync();  // the previous range's B has been read
#pragma unroll
      for (int l = 0; l < BL; ++l)
        if (first_piece + 64 * WT * l < pieces) *reinterpret_cast<v4u*>(bw + b_at[l]) = braw[l];
      load_b(nb + step);
      if (WT == 1) wave_lds_sync();
      else lds_barrier();
      v4f acc[4] = {v4f{0}, v4f{0}, v4f{0}, v4f{0}};
#pragma unroll
      for (int s = 0; s < RS; ++s) {
        v8bf w[4];
#pragma unroll
        for (int f = 0; f < 4; ++f) w[f] = load8(bw + (16 * f + j) * kStride + 32 * s + 8 * q);
#pragma unroll
        for (int term = 0; term < TERMS; ++term)
#pragma unroll
          for (int f = 0; f < 4; ++f) acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[f], v[term][s], acc[f], 0, 0, 0);
      }
      // lane (j, q) holds n = nb + 16 f + 4 q .. + 3 of token j
      wave_lds_sync();  // the previous products have been read
#pragma unroll
      for (int f = 0; f < 4; ++f) *reinterpret_cast<v4f*>(dw + j * kOutStride + 16 * f + 4 * q) = acc[f];
      wave_lds_sync();
#pragma unroll
      for (int i = 0; i < Y::kItems; ++i) {
        const typename Y::Raw sum = y.sum(i, dw + Y::token(i, lane) * kOutStride + col);
        Y::store(copied[i] ? y.raw[i] : sum, out_buf, at(own[i], nb));
      }
      load_y(y, nb + 2 * step);
    };
    for (int nb = n_lo; nb < n_end; nb += 2 * step) {
      range(even, nb, 0);
      if (nb + step < n_end) range(odd, nb + step, 1);
    }
    // the products of the wave's last range are still there
    const int nb = n_lo + (n_end - n_lo - 1) / step * step;
    if (n_end > n_lo && nb >= n_vec && nb < n_hi) {
      finish(dw, tokens, nb);
      finish(nullptr, none, nb);
    }
    none = 0;
  }
}

// Decode: both products of one token over one share of n, in one launch.
//
// A workgroup computes all of its token's v: thread = 8 k of every row of A, eight
// rows in flight and the next eight behind them, fp32 sums by v_dot2_f32_bf16, lanes
// by exchanges, waves in LDS in order.  Then thread = one n: R products with v in
// fp32.  Every workgroup of a token reads its A again (from L2), which costs less
// than a second launch and its latencies as long as A is small.
//
// 6.2 us for one token of rank 16 on 5120 x 5120 (two kernels: 8.0), 9.1 us for 24
// tokens of 32 adapters on 5120 x 17408 (12.0): ids, A, the sums and B in turn, and
// 1 us at least for each eight rows.
constexpr int kTokenThreads = 1024;
constexpr int kTokenR = 24;     // largest rank
constexpr int kTokenSteps = 4;  // of eight rows of 8192 k

// lanes exchanged by a DPP control: 0x128 l ^ 8, 0x141 l ^ 7, 0x4E l ^ 2, 0xB1 l ^ 1
template <int CTRL>
__device__ __forceinline__ float from(float s) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(s), CTRL, 0xF, 0xF, true));
}

// Sums of eight values over each 16 lanes, halved at each exchange: lane l gets that
// of value (l >> 1) & 7 (a sum of each over all lanes, 32 exchanges instead of 8,
// costs 0.3 us more for two times eight rows).
__device__ __forceinline__ float add_row16(const float (&v)[8], int lane) {
  float w[4], u[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = ((lane & 8) != 0 ? v[i + 4] : v[i]) + from<0x128>((lane & 8) != 0 ? v[i] : v[i + 4]);
#pragma unroll
  for (int i = 0; i < 2; ++i) u[i] = ((lane & 4) != 0 ? w[i + 2] : w[i]) + from<0x141>((lane & 4) != 0 ? w[i] : w[i + 2]);
  const float z = ((lane & 2) != 0 ? u[1] : u[0]) + from<0x4E>((lane & 2) != 0 ? u[0] : u[1]);
  return z + from<0xB1>(z);
}

template <bool BF16>
__device__ __forceinline__ float load_y(const void* y, size_t at) {
  if constexpr (BF16) return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(y)[at]) << 16);
  else return static_cast<const float*>(y)[at];
}

template <bool BF16>
__device__ __forceinline__ void store_y(void* out, size_t at, float v) {
  if constexpr (BF16) static_cast<uint16_t*>(out)[at] = static_cast<uint16_t>(pack_bf16(v, 0.0f));
  else static_cast<float*>(out)[at] = v;
}

template <bool BF16>
__global__ __launch_bounds__(kTokenThreads) void lora_token_kernel(LoraArgs a) {
  constexpr int kGroups = kTokenThreads / 16;  // of lanes whose sums meet in LDS
  __shared__ float part[kTokenR][kGroups + 1];
  __shared__ __attribute__((aligned(16))) float v_lds[kTokenR];
  const int tid = threadIdx.x, lane = tid & 63;
  const uint32_t item = xcd_item(blockIdx.x, gridDim.x);
  const uint32_t t = item / a.expand_chunks, chunk = item - t * a.expand_chunks;
  const int N = a.N, K = a.K, R = a.R;
  const int units = (N + 63) / 64;
  const int n_lo = 64 * static_cast<int>(static_cast<int64_t>(units) * chunk / a.expand_chunks);
  const int n_hi = min(N, 64 * static_cast<int>(static_cast<int64_t>(units) * (chunk + 1) / a.expand_chunks));
  const size_t row = static_cast<size_t>(t) * N;
  const int n0 = min(n_lo + tid, N - 1);
  const float y0 = load_y<BF16>(a.y, row + n0);
  const int id = __builtin_amdgcn_readfirstlane(a.ids[t]);
  if (id < 0 || id >= a.n) {
    if (a.out == a.y) return;
    typedef typename std::conditional<BF16, uint16_t, uint32_t>::type Bits;
    for (int n = n_lo + tid; n < n_hi; n += kTokenThreads)
      static_cast<Bits*>(a.out)[row + n] = static_cast<const Bits*>(a.y)[row + n];
    return;
  }
  const uint16_t* b = a.b + static_cast<size_t>(id) * N * R;
  const uint16_t* at = a.a + static_cast<size_t>(id) * R * K;
  const uint16_t* x = a.x + static_cast<size_t>(t) * K;
  const int pieces = K / 8, rounds = (pieces + kTokenThreads - 1) / kTokenThreads;
  const float scale = a.scale[id];

  // eight rows of A and x at this thread's piece; a piece past the end is zeros of x
  struct Step {
    v4u a[8], x;
  };
  const auto load = [&](Step& s, int r0, int round) {
    const int p = tid + round * kTokenThreads, k = 8 * min(p, pieces - 1);
    s.x = *reinterpret_cast<const v4u*>(x + k);
#pragma unroll
    for (int r = 0; r < 8; ++r) s.a[r] = *reinterpret_cast<const v4u*>(at + static_cast<size_t>(min(r0 + r, R - 1)) * K + k);
    if (p >= pieces) s.x = v4u{0, 0, 0, 0};
  };
  Step cur, next;
  load(cur, 0, 0);
  v4u b0[kTokenR / 8];  // the first n's row of B
#pragma unroll
  for (int p = 0; p < kTokenR / 8; ++p) b0[p] = *reinterpret_cast<const v4u*>(b + static_cast<size_t>(n0) * R + 8 * min(p, R / 8 - 1));
  float acc[8] = {};
  int r0 = 0, round = 0;
  const int steps = (R / 8) * rounds;
  for (int i = 0; i < steps; ++i) {
    const bool last = round + 1 == rounds;
    const int rn = last ? r0 + 8 : r0, roundn = last ? 0 : round + 1;
    load(next, rn, roundn);
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t w = cur.a[r][e], v = cur.x[e];  // a bit_cast of the elements themselves takes the first
        acc[r] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(v2bf, w), __builtin_bit_cast(v2bf, v), acc[r], false);
      }
    if (last) {
      const float s = add_row16(acc, lane);
      if ((lane & 1) == 0) part[r0 + ((lane >> 1) & 7)][tid >> 4] = s;
#pragma unroll
      for (int r = 0; r < 8; ++r) acc[r] = 0.0f;
    }
    cur = next;
    r0 = rn;
    round = roundn;
  }
  __syncthreads();
  if (tid < 8 * R) {
    const int r = tid >> 3, g = tid & 7;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kGroups / 8; ++i) s += part[r][8 * i + g];
    s += __shfl_xor(s, 1);
    s += __shfl_xor(s, 2);
    s += __shfl_xor(s, 4);
    if (g == 0) v_lds[r] = scale * s;
  }
  __syncthreads();
  for (int n = n_lo + tid; n < n_hi; n += kTokenThreads) {
    const bool ahead = n == n_lo + tid;
    float s = 0.0f;
    const auto add = [&](const v4u& w, int p) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s = __builtin_fmaf(v_lds[8 * p + 2 * e], __uint_as_float(w[e] << 16), s);
        s = __builtin_fmaf(v_lds[8 * p + 2 * e + 1], __uint_as_float(w[e] & 0xFFFF0000u), s);
      }
    };
#pragma unroll
    for (int p = 0; p < kTokenR / 8; ++p) {
      if (8 * p >= R) break;
      add(ahead ? b0[p] : *reinterpret_cast<const v4u*>(b + static_cast<size_t>(n) * R + 8 * p), p);
    }
    store_y<BF16>(a.out, row + n, (ahead ? y0 : load_y<BF16>(a.y, row + n)) + s);
  }
}

template <int WT, int RS>
hipError_t launch_expand(const LoraArgs& a, bool bf16, unsigned grid, hipStream_t stream) {
  const dim3 g(grid), b(64 * kExpandWaves);
  if (!bf16) hipLaunchKernelGGL((lora_expand_kernel<WT, RS, false, 16>), g, b, 0, stream, a);
  else if (a.N % 2 == 0) hipLaunchKernelGGL((lora_expand_kernel<WT, RS, true, 16>), g, b, 0, stream, a);
  else hipLaunchKernelGGL((lora_expand_kernel<WT, RS, true, 2>), g, b, 0, stream, a);
  return hipGetLastError();
}

int ceil_div(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

// Tokens up to which every pass of a tile of 16 has a workgroup of its own: each
// token may have its own adapter.  200 tokens of 8 adapters in any order, rank 64,
// 5120 -> 17408: 42 us, and 45 with four workgroups a tile of 64; of four requests,
// 5120 -> 5120: 13.5 and 16 us.
constexpr int kSplitPassesM = 256;

// Workgroups that share a tile's passes (pass p, p + passes, ...).  Larger batches
// have few adapters a tile, and a workgroup without a pass costs its launch: 4096
// tokens of 24 requests take 109 us with four, 127 with one (a tile in which one
// request ends and the next begins takes twice as long); 1500 tokens of 16 adapters
// in any order 112, and 136 with two; but 1000 tokens of rank 16 17 us with four and
// 21.5 with eight.  Eight cost nothing where y is large: the 4096 tokens above 109,
// and 337 instead of 500 us with 200 of them in decode, each with an adapter of its
// own.  The border, 4 x 10^7 elements of y, lies between those (7 x 10^7) and 4096 x
// 5120 (2 x 10^7, rank 128: 89.1 us with either); 1500 x 5120 (8 x 10^6) takes 32.5
// with four and 33.8 with eight in request order, 111.7 and 107.9 in any order.
int passes_of(const LoraArgs& a, int tokens) {
  const int share = a.M <= kSplitPassesM ? 16 : a.M * a.N >= 40000000 ? 8 : 4;
  return static_cast<int>(std::min<int64_t>({share, a.M, std::max(1, a.n), tokens}));
}

// Tiles of 32 tokens (each row of A read once for two fragments of tokens) where
// there are enough of them and the ranks' rows leave LDS for it: 4096 tokens of rank
// 64 110 us, in tiles of 16 122; 1000 tokens 44 and 38.  Slices of K that give every
// CU a workgroup (two of the smaller ones of 32 tokens), a wave at least one 64-k
// unit: half as many take 118 us for 4096 tokens and 31 instead of 25 for 500 of
// K = 17408, twice as many 114 and 31, for their sums are read again in every range
// of n.
void plan_shrink(LoraArgs& a, const DeviceInfo& dev) {
  const int cus = std::max(1, dev.cu_count);
  a.shrink_ts = a.M > 4 * static_cast<int64_t>(cus) && a.R <= 64 ? 2 : 1;
  a.shrink_tiles = ceil_div(a.M, 16 * a.shrink_ts);
  a.shrink_passes = passes_of(a, 16 * a.shrink_ts);
  const int64_t busy = a.M <= kSplitPassesM ? std::min<int64_t>(a.M, std::max(1, a.n)) : a.shrink_tiles;
  const int64_t want = a.shrink_ts == 1 ? cus : 2 * cus;
  a.slices = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((want + busy - 1) / busy, a.K / 64 / shrink_waves(a.shrink_ts))));
}

// Whether lora_token_kernel runs, which needs no workspace: every token has a
// workgroup and A is a few steps of loads.  Measured on either side, one token (M = 6
// for 10240) and 24 of 32 adapters, two kernels in brackets: rank 24, 5120 -> 5120, 7.4
// (8.1) and 8.6 (10.1) us; rank 16, 10240 -> 2000, two rounds, 8.5 (8.8) and 8.9
// (10.2); but rank 32, 5120 -> 5120, 8.8 (7.9) and 10.9 (10.4); rank 16, 17408 ->
// 5120, three rounds, 10.7 (9.5) and 12.7 (11.7).  200 tokens of rank 16, 5120 ->
// 5120: 13.2 (20.3).
bool one_launch(const LoraArgs& a, const DeviceInfo& dev) {
  return a.n > 0 && a.M <= std::min(kSplitPassesM, std::max(1, dev.cu_count)) &&
         a.R <= kTokenR && a.R / 8 * ceil_div(a.K, 8 * kTokenThreads) <= kTokenSteps;
}

template <int TS>
hipError_t launch_shrink(const LoraArgs& a, unsigned grid, hipStream_t stream) {
  const dim3 g(grid), b(64 * shrink_waves(TS));
  if (a.R <= 16) hipLaunchKernelGGL((lora_shrink_kernel<1, TS>), g, b, 0, stream, a);
  else if (a.R <= 32) hipLaunchKernelGGL((lora_shrink_kernel<2, TS>), g, b, 0, stream, a);
  else if (a.R <= 64) hipLaunchKernelGGL((lora_shrink_kernel<4, TS>), g, b, 0, stream, a);
  else if constexpr (TS == 1) hipLaunchKernelGGL((lora_shrink_kernel<8, TS>), g, b, 0, stream, a);
  else return hipErrorInvalidValue;  // not planned
  return hipGetLastError();
}

}  // namespace

size_t lora_workspace_bytes(int64_t M, int K, int R, int64_t n, const DeviceInfo& dev) {
  if (M <= 0 || n <= 0) return 0;
  LoraArgs a = {};
  a.M = M;
  a.K = K;
  a.R = R;
  a.n = static_cast<int>(n);
  if (one_launch(a, dev)) return 0;
  plan_shrink(a, dev);
  return static_cast<size_t>(a.slices) * static_cast<size_t>(M) * R * sizeof(float);
}

hipError_t launch_lora(LoraArgs a, bool bf16, const DeviceInfo& dev, hipStream_t stream) {
  if (a.M == 0 || a.N == 0) return hipSuccess;
  const int cus = std::max(1, dev.cu_count);
  if (one_launch(a, dev)) {
    // a round of workgroups, of 256 n at least
    a.expand_chunks = static_cast<uint32_t>(std::min<int64_t>(cus / a.M, ceil_div(a.N, 256)));
    const dim3 g(static_cast<unsigned>(a.M * a.expand_chunks)), b(kTokenThreads);
    if (bf16) hipLaunchKernelGGL(lora_token_kernel<true>, g, b, 0, stream, a);
    else hipLaunchKernelGGL(lora_token_kernel<false>, g, b, 0, stream, a);
    return hipGetLastError();
  }
  plan_shrink(a, dev);
  const int64_t shrink_grid = static_cast<int64_t>(a.shrink_tiles) * a.shrink_passes * a.slices;
  // 64 tokens a workgroup read B once, 16 tokens and 256 n make more workgroups of
  // smaller tiles: the first where B is large against y or the grid is many times
  // the card (4096 tokens of rank 64 on 17408: 109 against 134 us; 500 of rank 64 on
  // 5120: 27.4 and 29.9), else the second (2048 tokens of rank 32 on 5120: 22.7
  // against 20.9 us, 1000 of rank 16: 19.0 and 17.7)
  const bool large = a.R > 32 || static_cast<int64_t>(ceil_div(a.M, 64)) * ceil_div(a.N, 64) >= 16 * cus;
  const int WT = a.M > kSplitPassesM && large ? 4 : 1;
  const int RS = a.R <= 32 ? 1 : a.R <= 64 ? 2 : 4;
  a.expand_tiles = ceil_div(a.M, 16 * WT);
  a.expand_passes = passes_of(a, 16 * WT);
  // Ranges of n a workgroup.  Each workgroup sums the slices of its tokens and waits
  // for its first operands, so few long ones are better, as long as they fill the
  // card: first passes take half of the workgroups that can be resident (the other
  // half is for the passes behind them; all of them: 4096 tokens of rank 128 on 5120
  // 96 against 89 us, 2048 of rank 32 24 against 21; a quarter: 108 and 22).
  // And where the slices' bytes outweigh y's, as many as level them while two of
  // three CUs have a workgroup (500 tokens, K = 17408, N = 5120: 25 us, 27.6 with
  // one for every CU).
  const ExpandLds lds(WT, RS, bf16);
  const int64_t resident = static_cast<int64_t>(std::min(4, kLdsBytes / (lds.b + lds.vd))) * cus;
  const int64_t ranges = ceil_div(a.N, 256 / WT);
  const int64_t groups = static_cast<int64_t>(a.expand_tiles) * (a.M <= kSplitPassesM ? a.expand_passes : 1);
  const int64_t limit = std::max<int64_t>(1, resident / 2 / groups);
  const int64_t y_bytes = 2 * (256 / WT) * (bf16 ? 2 : 4), slice_bytes = static_cast<int64_t>(a.slices) * a.R * 4;
  const int64_t each = std::max((ranges + limit / 2) / limit, std::min(slice_bytes / y_bytes, ranges * groups * 3 / (2 * cus)));
  a.expand_chunks = static_cast<uint32_t>(ceil_div(ranges, static_cast<int>(std::max<int64_t>(1, each))));
  const int64_t expand_grid = static_cast<int64_t>(a.expand_tiles) * a.expand_passes * a.expand_chunks;
  if (shrink_grid > 0x7FFFFFFF || expand_grid > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  if (a.n > 0) {  // without adapters there is only the copy below
    const unsigned sg = static_cast<unsigned>(shrink_grid);
    const hipError_t e = a.shrink_ts == 2 ? launch_shrink<2>(a, sg, stream) : launch_shrink<1>(a, sg, stream);
    if (e != hipSuccess) return e;
  }
  const unsigned eg = static_cast<unsigned>(expand_grid);
  if (WT == 1)
    return RS == 1 ? launch_expand<1, 1>(a, bf16, eg, stream)
           : RS == 2 ? launch_expand<1, 2>(a, bf16, eg, stream) : launch_expand<1, 4>(a, bf16, eg, stream);
  return RS == 1 ? launch_expand<4, 1>(a, bf16, eg, stream)
         : RS == 2 ? launch_expand<4, 2>(a, bf16, eg, stream) : launch_expand<4, 4>(a, bf16, eg, stream);
}

}  // namespace twl
