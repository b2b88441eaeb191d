// int8_linear: y = (sum_k x_i8 w_i8) a_scale[t] w_scale[n] + bias[n] on int8 MFMAs with
// int32 sums (include/twl.h).
#include "attention_internal.h"

#include <algorithm>
#include <type_traits>

namespace twl {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kGroup = 8;  // rows of tiles in an XCD's order
constexpr int kXcds = 8;   // workgroups are dispatched to the XCDs round robin

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

__device__ __forceinline__ void wait_lgkm0() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// Workgroup barrier without the fence of __syncthreads: each wave waits for its own loads.
__device__ __forceinline__ void bare_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Direct global->LDS load of 16 bytes a lane from sbase + voff to lds_base + 16 * lane
// (inline asm for the reasons given in gemm_i8.hip; M0 is set in the same statement).
__device__ __forceinline__ void dma16(const void* sbase, uint32_t voff, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(voff), "s"(sbase), "s"(lds_base) : "memory", "m0");
}

__device__ __forceinline__ const void* sgpr_ptr(const void* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
  return reinterpret_cast<const void*>((static_cast<uint64_t>(hi) << 32) | lo);
}

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) char*)(p)));
}

// LDS operations of one wave execute in order; the fences keep the compiler to it.
__device__ __forceinline__ void lds_wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ uint32_t bf16_bits(float v) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}

// y of a sum: three roundings in the order that include/twl.h states, and the bias's.
__device__ __forceinline__ float scaled(int32_t acc, float a, float w, bool has_bias, float bias) {
  const float y = static_cast<float>(acc) * a * w;
  return has_bias ? y + bias : y;
}

template <int KIND>
__device__ __forceinline__ void store_one(void* out, int64_t o, int32_t v) {
  if (KIND == kOutBf16)
    static_cast<uint16_t*>(out)[o] = static_cast<uint16_t>(bf16_bits(__int_as_float(v)));
  else
    static_cast<int32_t*>(out)[o] = v;
}

// Four results (fp32 bits or sums) to columns of a row, where N is a multiple of 4.
template <int KIND>
__device__ __forceinline__ void store_four(void* out, int64_t o, v4i v) {
  if (KIND == kOutBf16)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + o) =
        make_uint2(bf16_bits(__int_as_float(v[0])) | bf16_bits(__int_as_float(v[1])) << 16,
                   bf16_bits(__int_as_float(v[2])) | bf16_bits(__int_as_float(v[3])) << 16);
  else
    *reinterpret_cast<v4i*>(static_cast<int32_t*>(out) + o) = v;
}

// 32 rows of W results from a wave's LDS rows of `stride` words to out [M, N] at (row0,
// col0): 16 bytes a lane where rows are aligned to it (8 for bf16 with N % 8 == 4), else
// one by one.
template <int KIND, int W>
__device__ __forceinline__ void store_rows(void* out, int M, int N, int row0, int col0, const int32_t* tr, int stride, int lane) {
  if (KIND == kOutBf16 && (N & 7) == 0) {
    const int c = lane % (W / 8) * 8;
#pragma unroll
    for (int r = lane / (W / 8); r < 32; r += 512 / W) {
      const v4i a = *reinterpret_cast<const v4i*>(tr + r * stride + c), b = *reinterpret_cast<const v4i*>(tr + r * stride + c + 4);
      if (row0 + r >= M || col0 + c >= N) continue;
      v4i p;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int lo = e < 2 ? a[2 * e] : b[2 * e - 4], hi = e < 2 ? a[2 * e + 1] : b[2 * e - 3];
        p[e] = static_cast<int>(bf16_bits(__int_as_float(lo)) | bf16_bits(__int_as_float(hi)) << 16);
      }
      *reinterpret_cast<v4i*>(static_cast<uint16_t*>(out) + static_cast<int64_t>(row0 + r) * N + col0 + c) = p;
    }
  } else if ((N & 3) == 0) {
    const int c = lane % (W / 4) * 4;
#pragma unroll
    for (int r = lane / (W / 4); r < 32; r += 256 / W) {
      const v4i v = *reinterpret_cast<const v4i*>(tr + r * stride + c);
      if (row0 + r < M && col0 + c < N) store_four<KIND>(out, static_cast<int64_t>(row0 + r) * N + col0 + c, v);
    }
  } else {
    const int c = lane % W;
#pragma unroll 4
    for (int r = lane / W; r < 32; r += 64 / W)
      if (row0 + r < M && col0 + c < N) store_one<KIND>(out, static_cast<int64_t>(row0 + r) * N + col0 + c, tr[r * stride + c]);
  }
}

// ---------------------------------------------------------------------------------
// Few tokens: 16 RT rows of w and 16 MT tokens a workgroup, whose waves share K.  The
// weights go from memory into MFMA operands as they lie: a lane loads 16 bytes of row
// lane % 16; U steps of 128 bytes of each row are in flight in a wave.
//
// Bound by the stream of w (at M <= 32 each byte is used by at most 64 operations, a sixth of what
// the MFMAs do in its time): no LDS, no barrier before the end, only loads that are
// deep enough.  1 token 5120 -> 7168 9.6 us (3.8 TB/s; too short to reach the rate of a copy, 5.1), 24 tokens
// 5120 -> 65536 73 us (4.6 TB/s).  Whole cache lines by four lanes instead of half ones: 24 tokens
// 17408 -> 5120 44 -> 32 us.

template <int RT, int MT, int WAVES, int U, int KIND>
__global__ __launch_bounds__(64 * WAVES) void int8_rows_kernel(Int8Args a) {
  __shared__ v4i part[WAVES][RT * MT][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, h = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * (16 * RT);
  const int t0 = static_cast<int>(blockIdx.y) * (16 * MT);
  const int8_t* wp[RT];
  const int8_t* xp[MT];
#pragma unroll
  for (int r = 0; r < RT; ++r) wp[r] = a.w + min(n0 + r * 16 + m, static_cast<int64_t>(a.N) - 1) * a.K + h * 32;
#pragma unroll
  for (int t = 0; t < MT; ++t) xp[t] = a.x + static_cast<int64_t>(min(t0 + t * 16 + m, a.M - 1)) * a.K + h * 32;
  v4i acc[RT][MT] = {};
  // steps of 128 bytes: a lane's two products take bytes 32 h .. + 31 of each row, so that four
  // lanes touch a whole cache line at once
  const int whole = a.K / 128, steps = (a.K + 127) / 128;
  int s = steps * wave / WAVES;
  const int end = steps * (wave + 1) / WAVES, full = min(end, whole);
  v4i wf[U][2][RT], xf[U][2][MT];
  auto multiply = [&] {
    __builtin_amdgcn_sched_barrier(0);  // all loads first
#pragma unroll
    for (int u = 0; u < 2 * U; ++u)
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[r][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[u / 2][u % 2][r], xf[u / 2][u % 2][t], acc[r][t], 0, 0, 0);
  };
  for (; s + U <= full; s += U) {
#pragma unroll
    for (int u = 0; u < 2 * U; ++u) {
#pragma unroll
      for (int r = 0; r < RT; ++r) wf[u / 2][u % 2][r] = *reinterpret_cast<const v4i*>(wp[r] + (s + u / 2) * 128 + u % 2 * 16);
#pragma unroll
      for (int t = 0; t < MT; ++t) xf[u / 2][u % 2][t] = *reinterpret_cast<const v4i*>(xp[t] + (s + u / 2) * 128 + u % 2 * 16);
    }
    multiply();
  }
  while (s < end) {  // what is left in one go: bytes past the end repeat the row's start with x as 0
#pragma unroll
    for (int u = 0; u < 2 * U; ++u) {
      const int k = (s + u / 2) * 128 + u % 2 * 16;
      const bool in = s + u / 2 < end && k + h * 32 < a.K;  // K is a multiple of 16: all of a lane's bytes or none
#pragma unroll
      for (int r = 0; r < RT; ++r) wf[u / 2][u % 2][r] = *reinterpret_cast<const v4i*>(wp[r] + (in ? k : -h * 32));
#pragma unroll
      for (int t = 0; t < MT; ++t) xf[u / 2][u % 2][t] = in ? *reinterpret_cast<const v4i*>(xp[t] + k) : v4i(0);
    }
    multiply();
    s += U;
  }
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < MT; ++t) part[wave][r * MT + t][lane] = acc[r][t];
  __syncthreads();
  for (int f = wave; f < RT * MT; f += WAVES) {
    v4i sum = part[0][f][lane];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) sum += part[w][f][lane];
    const int token = t0 + f % MT * 16 + m;
    const int64_t n = n0 + f / MT * 16 + h * 4;
    if (token >= a.M) continue;
    const float as = KIND == kOutAcc ? 0.0f : a.a_scale[token];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (n + i >= a.N) continue;
      const int64_t o = static_cast<int64_t>(token) * a.N + n + i;
      store_one<KIND>(a.out, o, KIND == kOutAcc ? sum[i] : __float_as_int(scaled(sum[i], as, a.w_scale[n + i], a.bias != nullptr, a.bias != nullptr ? a.bias[n + i] : 0.0f)));
    }
  }
}

// ---------------------------------------------------------------------------------
// Many tokens: a tile of BM tokens x BN channels a workgroup of WM x WN waves, on 32x32x32 MFMAs; stages of
// 128 of K go to LDS by direct loads, STAGES of them in flight.
//
// Bound by the MFMAs: 4096 tokens 5120 -> 17408 342 to 376 us, 1.94 to 2.13 POP/s, 8192^3 467 us, 2.35 (the library's
// product of that size 2.15).  To get there from 392 us: loads of a stage issued one by one among its products, not in
// one go; a stage's buffer handed on as soon as its last operands are in registers; operands read a
// step ahead, across the barrier.  Without gain: a prefetch of w into L2, stages of 64, four waves of 64 x 64.

template <int BM_, int BN_, int WM_, int WN_, int SK_, int STAGES_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, SK = SK_, STAGES = STAGES_;
  static constexpr int WAVES = WM * WN, THREADS = 64 * WAVES;
  static constexpr int RM = BM / WM / 32, RN = BN / WN / 32;  // 32 x 32 fragments of a wave
  static constexpr int ROWS = 1024 / SK, CHUNKS = SK / 16;    // rows of a load instruction, 16-byte chunks of a row
  static constexpr int BYTES = (BM + BN) * SK;                // a stage of x and w: SK of K
  static constexpr int LOADS = (BM + BN) / ROWS / WAVES;      // load instructions of a wave and stage
  static constexpr int TR = RN * 32 + 8;                      // words of a row of the output transpose (the lane halves' rows on other banks)
  static constexpr int PIPE = STAGES * BYTES;                 // the pipeline's buffers; the scales lie behind them
  static constexpr int LDS = PIPE + (BM + 2 * BN) * 4;
  static_assert((BM + BN) % (ROWS * WAVES) == 0 && BM % ROWS == 0 && BM % (32 * WM) == 0 && BN % (32 * WN) == 0, "whole fragments and loads");
  static_assert(WAVES * 32 * TR * 4 <= PIPE && LDS <= 160 * 1024, "the output transpose fits the pipeline's buffers");
  static_assert((STAGES - 1) * LOADS < 64, "vmcnt range");

  // Place of a row's 16-byte chunk: reads of one chunk of 8 adjacent rows (and of the even
  // or odd ones of 16) meet distinct banks.
  __device__ static __forceinline__ int place(int row, int chunk) { return chunk ^ (SK == 128 ? (row ^ (row >> 3)) & 7 : (row >> 2) & 3); }
};

template <class T, int KIND>
__global__ __launch_bounds__(T::THREADS) void int8_gemm_kernel(Int8Args a) {
  __shared__ __attribute__((aligned(16))) char smem[T::LDS];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l32 = lane & 31, half = lane >> 5;
  const int wm = wave / T::WN, wn = wave % T::WN;
  // workgroups go round the XCDs: give each of them adjacent tiles
  const int total = a.tiles_m * a.tiles_n * a.splits;
  const int per = total / kXcds, rem = total % kXcds, xcd = blockIdx.x % kXcds;
  const int lin = xcd * per + min(xcd, rem) + static_cast<int>(blockIdx.x / kXcds);
  const int split = lin % a.splits, tile = lin / a.splits;
  // in an XCD, kGroup rows of tiles at a time: what runs together shares x and w in its L2
  const int group = tile / (kGroup * a.tiles_n) * kGroup, wide = min(kGroup, a.tiles_m - group), in = tile - group * a.tiles_n;
  const int m0 = (group + in % wide) * T::BM, n0 = in / wide * T::BN;

  const uint32_t lds = lds_addr(smem);
  const void* xbase = sgpr_ptr(a.x + static_cast<int64_t>(m0) * a.K);
  const void* wbase = sgpr_ptr(a.w + static_cast<int64_t>(n0) * a.K);
  // a load instruction brings ROWS rows of SK bytes, 16-byte chunks XOR-swizzled by row; the
  // first BM rows of a stage are x's, then w's.  Rows past the last repeat it.
  uint32_t off[T::LOADS];
#pragma unroll
  for (int i = 0; i < T::LOADS; ++i) {
    const int row = (i * T::WAVES + wave) * T::ROWS + lane / T::CHUNKS;
    const bool is_x = (i * T::WAVES + wave) * T::ROWS < T::BM;
    const int r = is_x ? min(row, a.M - 1 - m0) : min(row - T::BM, a.N - 1 - n0);
    off[i] = static_cast<uint32_t>(r) * a.K + T::place(row, lane % T::CHUNKS) * 16;
  }
  const int all = (a.K + T::SK - 1) / T::SK;  // this split's stages of K: [first, last)
  const int first = static_cast<int>(static_cast<int64_t>(all) * split / a.splits);
  const int stages = static_cast<int>(static_cast<int64_t>(all) * (split + 1) / a.splits) - first;
  auto load_one = [&](int s, int i) {
    const bool is_x = (i * T::WAVES + wave) * T::ROWS < T::BM;
    uint32_t o = off[i] + (first + s) * T::SK;
    if (first + s == all - 1) {  // chunks past K bring the row's start; x's are cleared before their use
      const int row = (i * T::WAVES + wave) * T::ROWS + lane / T::CHUNKS;
      const int k = (first + s) * T::SK + T::place(row, lane % T::CHUNKS) * 16;
      if (k >= a.K) o -= k;
    }
    dma16(is_x ? xbase : wbase, o, lds + s % T::STAGES * T::BYTES + (i * T::WAVES + wave) * 1024);
  };
  auto load = [&](int s) {
#pragma unroll
    for (int i = 0; i < T::LOADS; ++i) load_one(s, i);
  };
  // the tile's scales, read here so that nothing waits for them at the end
  float* rs = reinterpret_cast<float*>(smem + T::PIPE);
  float* cs = rs + T::BM;
  float* bs = cs + T::BN;
  if (KIND != kOutAcc) {
    for (int i = threadIdx.x; i < T::BM; i += T::THREADS) rs[i] = a.a_scale[min(m0 + i, a.M - 1)];
    for (int i = threadIdx.x; i < T::BN; i += T::THREADS) {
      const int n = min(n0 + i, a.N - 1);
      cs[i] = a.w_scale[n];
      bs[i] = a.bias != nullptr ? a.bias[n] : 0.0f;
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // written before the first barrier below
  }
  v16i acc[T::RM][T::RN] = {};
#pragma unroll
  for (int s = 0; s < T::STAGES; ++s)
    if (s < stages) load(s);

  // Fragments of k-step k of a stage: lane half h takes chunk h CHUNKS / 2 + k of its rows.  They are
  // read a step ahead; the last step of a stage runs behind the barrier that ends the
  // stage, beside the first reads of the next one.
  const int arow = wm * T::RM * 32 + l32, brow = T::BM + wn * T::RN * 32 + l32;
  struct Frags {
    v4i a[T::RM], b[T::RN];
  } f[4];
  auto read = [&](Frags& g, int s, int k) {
    const char* stage = smem + s % T::STAGES * T::BYTES;
#pragma unroll
    for (int r = 0; r < T::RM; ++r) g.a[r] = *reinterpret_cast<const v4i*>(stage + (arow + 32 * r) * T::SK + T::place(arow + 32 * r, half * (T::CHUNKS / 2) + k) * 16);
#pragma unroll
    for (int r = 0; r < T::RN; ++r) g.b[r] = *reinterpret_cast<const v4i*>(stage + (brow + 32 * r) * T::SK + T::place(brow + 32 * r, half * (T::CHUNKS / 2) + k) * 16);
  };
  auto multiply = [&](const Frags& g) {
#pragma unroll
    for (int i = 0; i < T::RM; ++i)
#pragma unroll
      for (int j = 0; j < T::RN; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(g.a[i], g.b[j], acc[i][j], 0, 0, 0);
  };
  // The same, with loads [from, to) of a stage among the products: issued in one go they
  // would keep the waves from their products while the address unit takes them.
  auto multiply_and_load = [&](const Frags& g, int s, int from, int to) {
#pragma unroll
    for (int i = 0; i < T::RM; ++i)
#pragma unroll
      for (int j = 0; j < T::RN; ++j) {
        const int m = i * T::RN + j, lo = from + (to - from) * m / (T::RM * T::RN), hi = from + (to - from) * (m + 1) / (T::RM * T::RN);
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(g.a[i], g.b[j], acc[i][j], 0, 0, 0);
        // the operand (named, not read) keeps what follows behind this product
        if (lo < hi) asm volatile("" : "+v"(acc[i][j]));
#pragma unroll
        for (int l = lo; l < hi; ++l) load_one(s, l);
      }
  };
  // Stage s has landed: this wave's loads of it are done, then everyone's; the tail of K is cleared.
  auto arrive = [&](int s, int after) {  // after: stages whose loads were issued behind those of s
    if (after >= T::STAGES - 1)
      wait_vmcnt<(T::STAGES - 1) * T::LOADS>();
    else if (after == T::STAGES - 2)
      wait_vmcnt<(T::STAGES - 2) * T::LOADS>();
    else
      wait_vmcnt<0>();
    bare_barrier();
    if (first + s == all - 1 && a.K % T::SK != 0) {
      for (int c = threadIdx.x; c < T::BM * T::CHUNKS; c += T::THREADS) {
        const int row = c / T::CHUNKS;
        if ((first + s) * T::SK + T::place(row, c % T::CHUNKS) * 16 >= a.K) *reinterpret_cast<v4i*>(smem + s % T::STAGES * T::BYTES + c * 16) = 0;
      }
      __syncthreads();
    }
  };
  arrive(0, min(stages, T::STAGES) - 1);
  read(f[0], 0, 0);
  // Memory operations before this stay before those after it: the compiler would move each
  // read next to its use.
  auto issued = [] { asm volatile("" ::: "memory"); };
  auto step = [&](int s, auto loads) {
    constexpr bool LOAD = decltype(loads)::value;
    read(f[1], s, 1);
    issued();
    multiply(f[0]);
    read(f[2], s, 2);
    read(f[3], s, 3);
    issued();
    multiply(f[1]);
    // the stage is in registers: its buffer takes the loads of a later one
    wait_lgkm0();
    bare_barrier();
    if constexpr (LOAD) {
      multiply_and_load(f[2], s + T::STAGES, 0, T::LOADS / 2);
      wait_vmcnt<(T::STAGES - 2) * T::LOADS + T::LOADS / 2>();
      bare_barrier();
      read(f[0], s + 1, 0);
      issued();
      multiply_and_load(f[3], s + T::STAGES, T::LOADS / 2, T::LOADS);
    } else {
      multiply(f[2]);
      if (s + 1 < stages) {
        arrive(s + 1, stages - 2 - s);
        read(f[0], s + 1, 0);
      }
      multiply(f[3]);
    }
  };
  int s = 0;
  for (; s + T::STAGES < stages; ++s) step(s, std::true_type());
  for (; s < stages; ++s) step(s, std::false_type());
  bare_barrier();  // every wave's reads are done: the buffers are free

  // Lane: channel l32 of a fragment, register r: token 8 (r / 4) + 4 half + r % 4.  32 tokens at
  // a time go through the wave's part of LDS and leave along the rows.
  int32_t* tr = reinterpret_cast<int32_t*>(smem) + wave * 32 * T::TR;
  void* out = a.splits == 1 ? a.out : a.part + static_cast<int64_t>(split) * a.M * a.N;
  const int col = wn * T::RN * 32;
  const bool has_bias = a.bias != nullptr;
#pragma unroll
  for (int i = 0; i < T::RM; ++i) {
    const int row = wm * T::RM * 32 + i * 32;
    lds_wave_sync();
#pragma unroll
    for (int r = 0; r < 16; r += 4) {
      const int rr = 8 * (r >> 2) + 4 * half;
      const v4f rows = *reinterpret_cast<const v4f*>(rs + row + rr);
#pragma unroll
      for (int j = 0; j < T::RN; ++j) {
        const float c = cs[col + j * 32 + l32], b = bs[col + j * 32 + l32];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          tr[(rr + e) * T::TR + j * 32 + l32] =
              KIND == kOutAcc ? acc[i][j][r + e] : __float_as_int(scaled(acc[i][j][r + e], rows[e], c, has_bias, b));
      }
    }
    lds_wave_sync();
    store_rows<KIND, T::RN * 32>(out, a.M, a.N, m0 + row, n0 + col, tr, T::TR, lane);
  }
}

// The splits' sums joined: four outputs a lane where N allows it, else one.
template <int KIND>
__global__ __launch_bounds__(256) void int8_reduce_kernel(Int8Args a) {
  const int64_t plane = static_cast<int64_t>(a.M) * a.N;
  const int per = (a.N & 3) == 0 ? 4 : 1;
  const int64_t o = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * per;
  if (o >= plane) return;
  const int token = static_cast<int>(o / a.N), n = static_cast<int>(o - static_cast<int64_t>(token) * a.N);
  const float as = KIND == kOutAcc ? 0.0f : a.a_scale[token];
  if (per == 4) {
    v4i sum = *reinterpret_cast<const v4i*>(a.part + o);
    for (int s = 1; s < a.splits; ++s) sum += *reinterpret_cast<const v4i*>(a.part + s * plane + o);
    v4i v = sum;
    if (KIND != kOutAcc) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[e] = __float_as_int(scaled(sum[e], as, a.w_scale[n + e], a.bias != nullptr, a.bias != nullptr ? a.bias[n + e] : 0.0f));
    }
    store_four<KIND>(a.out, o, v);
    return;
  }
  int32_t sum = a.part[o];
  for (int s = 1; s < a.splits; ++s) sum += a.part[s * plane + o];
  store_one<KIND>(a.out, o, KIND == kOutAcc ? sum : __float_as_int(scaled(sum, as, a.w_scale[n], a.bias != nullptr, a.bias != nullptr ? a.bias[n] : 0.0f)));
}

// The tiles, largest first.  Many tokens want the largest (its loads and LDS reads are the
// fewest for a product), as long as whole rounds of workgroups fill the device.
using Tile0 = Tile<256, 256, 2, 4, 128, 2>;
using Tile1 = Tile<192, 256, 2, 4, 128, 2>;
using Tile2 = Tile<256, 128, 4, 2, 128, 3>;
using Tile3 = Tile<128, 128, 2, 4, 128, 3>;
using Tile4 = Tile<64, 128, 2, 2, 128, 3>;  // two workgroups a CU, as the next
using Tile5 = Tile<64, 64, 2, 2, 128, 4>;
struct TileCost {
  int bm, bn;
  float fixed, stage, least;  // us a workgroup and a stage of one, alone on its CU or as the CU's share; and at least
};
// measured at K = 5120, bf16 output, 80 to 2176 workgroups
constexpr TileCost kTiles[] = {{256, 256, 8.0f, 1.55f, 1.55f}, {192, 256, 7.0f, 1.27f, 1.27f}, {256, 128, 5.0f, 1.03f, 1.0f},
                               {128, 128, 3.0f, 0.66f, 0.65f}, {64, 128, 2.0f, 0.42f, 0.66f},  {64, 64, 2.0f, 0.27f, 0.33f}};
constexpr int kRowsMax = 32;  // tokens of the rows kernel

struct Plan {
  int rt, mt;  // rows kernel: its RT and MT; rt = 0: a tile kernel
  int tile, splits;
};

Plan make_plan(int64_t M, int64_t N, int64_t K, const DeviceInfo& dev) {
  Plan p = {};
  p.splits = 1;
  if (M <= kRowsMax) {
    // Two tokens tiles double the operands loaded beside the weights, which wider row tiles
    // share; narrow layers want the workgroups.  us, RT = 1 / 2 / 4: 24 tokens 5120 -> 65536
    // 112 / 86 / 73, 24 tokens 17408 -> 5120 43 / 32 / 48, 16 tokens 5120 -> 5120 12.3 / 10.8 / 16, 1 token
    // 5120 -> 17408 20 / 22 / 26, 1 token 5120 -> 1024 5.7 / 7.8 / 12.
    p.mt = M <= 16 ? 1 : 2;
    p.rt = N < 16 * dev.cu_count || M <= 4 ? 1 : p.mt == 1 || N < 128 * dev.cu_count ? 2 : 4;
    return p;
  }
  // The plan of least time: rounds of workgroups by the table, a second kernel and the
  // sums' traffic (4 TB/s) where K is split, into parts of at least 4 stages.
  const int64_t stages = (K + 127) / 128;
  float best = 0.0f;
  for (int t = 0; t < 6; ++t) {
    const TileCost& c = kTiles[t];
    const int64_t tiles = ((M + c.bm - 1) / c.bm) * ((N + c.bn - 1) / c.bn);
    for (int splits = 1; splits <= 8 && (splits == 1 || stages / splits >= 4); splits *= 2) {
      if (splits > 1 && tiles * splits > 2 * dev.cu_count) break;
      const float share = static_cast<float>((tiles * splits + dev.cu_count - 1) / dev.cu_count);  // workgroups of the fullest CU
      const float depth = static_cast<float>((stages + splits - 1) / splits);
      float us = share * c.fixed + depth * std::max(c.least, share * c.stage);
      if (splits > 1) us += 4.0f + 2.0f * splits * static_cast<float>(M * N) * 4.0f / 4e6f;
      if (best == 0.0f || us < best) {
        best = us;
        p.tile = t;
        p.splits = splits;
      }
    }
  }
  return p;
}

template <int RT, int MT, int WAVES, int U, int KIND>
hipError_t launch_rows(const Int8Args& a, hipStream_t stream) {
  const dim3 grid(static_cast<uint32_t>((static_cast<int64_t>(a.N) + 16 * RT - 1) / (16 * RT)), static_cast<uint32_t>((a.M + 16 * MT - 1) / (16 * MT)));
  int8_rows_kernel<RT, MT, WAVES, U, KIND><<<grid, 64 * WAVES, 0, stream>>>(a);
  return hipGetLastError();
}

template <class T, int KIND>
hipError_t launch_tiles(Int8Args a, hipStream_t stream) {
  a.tiles_m = (a.M + T::BM - 1) / T::BM;
  a.tiles_n = (a.N + T::BN - 1) / T::BN;
  const uint32_t blocks = static_cast<uint32_t>(a.tiles_m) * a.tiles_n * a.splits;
  if (a.splits == 1) {
    int8_gemm_kernel<T, KIND><<<blocks, T::THREADS, 0, stream>>>(a);
    return hipGetLastError();
  }
  int8_gemm_kernel<T, kOutAcc><<<blocks, T::THREADS, 0, stream>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t items = static_cast<int64_t>(a.M) * a.N / ((a.N & 3) == 0 ? 4 : 1);
  int8_reduce_kernel<KIND><<<static_cast<uint32_t>((items + 255) / 256), 256, 0, stream>>>(a);
  return hipGetLastError();
}

template <int KIND>
hipError_t launch_kind(Int8Args a, const DeviceInfo& dev, hipStream_t stream) {
  const Plan p = make_plan(a.M, a.N, a.K, dev);
  a.splits = p.splits;
  if (p.rt > 0) {
    if (p.rt == 1) return p.mt == 1 ? launch_rows<1, 1, 4, 2, KIND>(a, stream) : launch_rows<1, 2, 4, 2, KIND>(a, stream);
    if (p.rt == 2) return p.mt == 1 ? launch_rows<2, 1, 4, 2, KIND>(a, stream) : launch_rows<2, 2, 4, 2, KIND>(a, stream);
    return launch_rows<4, 2, 8, 1, KIND>(a, stream);
  }
  switch (p.tile) {
    case 0: return launch_tiles<Tile0, KIND>(a, stream);
    case 1: return launch_tiles<Tile1, KIND>(a, stream);
    case 2: return launch_tiles<Tile2, KIND>(a, stream);
    case 3: return launch_tiles<Tile3, KIND>(a, stream);
    case 4: return launch_tiles<Tile4, KIND>(a, stream);
    default: return launch_tiles<Tile5, KIND>(a, stream);
  }
}

}  // namespace

size_t int8_workspace_bytes(int64_t M, int64_t N, int64_t K, const DeviceInfo& dev) {
  const Plan p = make_plan(M, N, K, dev);
  return p.splits == 1 ? 0 : static_cast<size_t>(p.splits) * M * N * sizeof(int32_t);
}

hipError_t launch_int8(Int8Args a, const DeviceInfo& dev, hipStream_t stream) {
  if (a.kind == kOutAcc) return launch_kind<kOutAcc>(a, dev, stream);
  if (a.kind == kOutBf16) return launch_kind<kOutBf16>(a, dev, stream);
  return launch_kind<kOutF32>(a, dev, stream);
}

}  // namespace twl
