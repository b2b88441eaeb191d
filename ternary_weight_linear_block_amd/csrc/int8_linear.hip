// int8_linear: y = (sum_k x_i8 w_i8) a_scale[t] w_scale[n] + bias[n] on int8 MFMAs with
// int32 sums (include/twl.h).
#include "attention_internal.h"

#include <algorithm>

namespace twl {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));

constexpr int kStageK = 128;  // k of a pipeline stage
constexpr int kXcds = 8;      // workgroups are dispatched to the XCDs round robin

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

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

// Swizzle of a 128-byte row's 16-byte chunks: reads of one chunk of 8 adjacent rows (and
// of the even or odd ones of 16) meet distinct banks.
__device__ __forceinline__ int swizzle(int row) { return (row ^ (row >> 3)) & 7; }

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

// A 32 x 32 fragment of results (fp32 bits or sums) from a wave's LDS rows of `stride`
// words to out [M, N] at (row0, col0): 16 bytes a lane where rows are aligned to it (8
// for bf16 with N % 8 == 4), else one by one along the row.
template <int KIND>
__device__ __forceinline__ void store_fragment(void* out, int M, int N, int row0, int col0, const int32_t* tr, int stride, int lane) {
  if (KIND == kOutBf16 && (N & 7) == 0) {
    const int c = 8 * (lane & 3), col = col0 + c;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int rr = 16 * k + (lane >> 2);
      const v4i a = *reinterpret_cast<const v4i*>(tr + rr * stride + c), b = *reinterpret_cast<const v4i*>(tr + rr * stride + c + 4);
      if (row0 + rr >= M || col >= N) continue;
      v4i p;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int lo = e < 2 ? a[2 * e] : b[2 * e - 4], hi = e < 2 ? a[2 * e + 1] : b[2 * e - 3];
        p[e] = static_cast<int>(bf16_bits(__int_as_float(lo)) | bf16_bits(__int_as_float(hi)) << 16);
      }
      *reinterpret_cast<v4i*>(static_cast<uint16_t*>(out) + static_cast<int64_t>(row0 + rr) * N + col) = p;
    }
  } else if ((N & 3) == 0) {
    const int c = 4 * (lane & 7), col = col0 + c;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int rr = 8 * k + (lane >> 3);
      const v4i v = *reinterpret_cast<const v4i*>(tr + rr * stride + c);
      if (row0 + rr >= M || col >= N) continue;
      const int64_t o = static_cast<int64_t>(row0 + rr) * N + col;
      if (KIND == kOutBf16)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + o) =
            make_uint2(bf16_bits(__int_as_float(v[0])) | bf16_bits(__int_as_float(v[1])) << 16,
                       bf16_bits(__int_as_float(v[2])) | bf16_bits(__int_as_float(v[3])) << 16);
      else
        *reinterpret_cast<v4i*>(static_cast<int32_t*>(out) + o) = v;
    }
  } else {
    const int col = col0 + (lane & 31);
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int rr = 2 * r + (lane >> 5);
      if (row0 + rr < M && col < N) store_one<KIND>(out, static_cast<int64_t>(row0 + rr) * N + col, tr[rr * stride + (lane & 31)]);
    }
  }
}

// ---------------------------------------------------------------------------------
// Few tokens: 16 RT rows of w and 16 MT tokens a workgroup, whose waves share K.  The
// weights go from memory into MFMA operands as they lie: a lane loads 16 bytes of row
// lane % 16, four lanes 64 bytes of a row; U steps of 64 bytes are in flight in a wave.

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
  for (int r = 0; r < RT; ++r) wp[r] = a.w + min(n0 + r * 16 + m, static_cast<int64_t>(a.N) - 1) * a.K + h * 16;
#pragma unroll
  for (int t = 0; t < MT; ++t) xp[t] = a.x + static_cast<int64_t>(min(t0 + t * 16 + m, a.M - 1)) * a.K + h * 16;
  v4i acc[RT][MT] = {};
  const int whole = a.K / 64, steps = (a.K + 63) / 64;
  int s = steps * wave / WAVES;
  const int end = steps * (wave + 1) / WAVES, full = min(end, whole);
  for (; s + U <= full; s += U) {
    v4i wf[U][RT], xf[U][MT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int r = 0; r < RT; ++r) wf[u][r] = *reinterpret_cast<const v4i*>(wp[r] + (s + u) * 64);
#pragma unroll
      for (int t = 0; t < MT; ++t) xf[u][t] = *reinterpret_cast<const v4i*>(xp[t] + (s + u) * 64);
    }
    __builtin_amdgcn_sched_barrier(0);  // all loads first
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[r][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[u][r], xf[u][t], acc[r][t], 0, 0, 0);
  }
  for (; s < end; ++s) {
    v4i wf[RT], xf[MT];
    const bool in = s * 64 + h * 16 < a.K;  // K is a multiple of 16: a lane's 16 bytes are in range or none is
#pragma unroll
    for (int r = 0; r < RT; ++r) wf[r] = in ? *reinterpret_cast<const v4i*>(wp[r] + s * 64) : v4i(0);
#pragma unroll
    for (int t = 0; t < MT; ++t) xf[t] = in ? *reinterpret_cast<const v4i*>(xp[t] + s * 64) : v4i(0);
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
// Many tokens: a tile of BM tokens x BN channels a workgroup of WM x WN waves.

template <int BM_, int BN_, int WM_, int WN_, int STAGES_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, STAGES = STAGES_;
  static constexpr int WAVES = WM * WN, THREADS = 64 * WAVES;
  static constexpr int RM = BM / WM / 32, RN = BN / WN / 32;  // 32 x 32 fragments of a wave
  static constexpr int BYTES = (BM + BN) * kStageK;           // a stage of x and w
  static constexpr int LOADS = (BM + BN) / 8 / WAVES;         // load instructions (8 rows each) of a wave and stage
  static constexpr int TR = 36;                               // words of a row of the output transpose
  static_assert((BM + BN) / 8 % WAVES == 0 && BM % (32 * WM) == 0 && BN % (32 * WN) == 0, "whole fragments and loads");
  static_assert(WAVES * 32 * TR * 4 <= STAGES * BYTES, "the output transpose fits the pipeline's buffers");
  static constexpr int LDS = STAGES * BYTES + (BM + 2 * BN) * 4;
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
  const int m0 = tile % a.tiles_m * T::BM, n0 = tile / a.tiles_m * T::BN;

  const uint32_t lds = lds_addr(smem);
  const void* xbase = sgpr_ptr(a.x + static_cast<int64_t>(m0) * a.K);
  const void* wbase = sgpr_ptr(a.w + static_cast<int64_t>(n0) * a.K);
  // a load instruction brings 8 rows of 128 bytes, 16-byte chunks XOR-swizzled by row; the
  // first BM rows of a stage are x's, then w's.  Rows past the last repeat it.
  uint32_t off[T::LOADS];
#pragma unroll
  for (int i = 0; i < T::LOADS; ++i) {
    const int row = (i * T::WAVES + wave) * 8 + (lane >> 3);
    const bool is_x = (i * T::WAVES + wave) * 8 < T::BM;
    const int r = is_x ? min(row, a.M - 1 - m0) : min(row - T::BM, a.N - 1 - n0);
    off[i] = static_cast<uint32_t>(r) * a.K + ((lane & 7) ^ swizzle(row)) * 16;
  }
  const int all = (a.K + kStageK - 1) / kStageK;  // this split's stages of K: [first, last)
  const int first = static_cast<int>(static_cast<int64_t>(all) * split / a.splits);
  const int stages = static_cast<int>(static_cast<int64_t>(all) * (split + 1) / a.splits) - first;
  auto load = [&](int s) {
    const uint32_t base = lds + s % T::STAGES * T::BYTES;
#pragma unroll
    for (int i = 0; i < T::LOADS; ++i) {
      const bool is_x = (i * T::WAVES + wave) * 8 < T::BM;
      uint32_t o = off[i] + (first + s) * kStageK;
      if (first + s == all - 1) {  // chunks past K bring the row's start; x's are cleared before their use
        const int row = (i * T::WAVES + wave) * 8 + (lane >> 3);
        const int k = (first + s) * kStageK + ((lane & 7) ^ swizzle(row)) * 16;
        if (k >= a.K) o -= k;
      }
      dma16(is_x ? xbase : wbase, o, base + (i * T::WAVES + wave) * 1024);
    }
  };
  v16i acc[T::RM][T::RN] = {};
#pragma unroll
  for (int s = 0; s < T::STAGES - 1; ++s)
    if (s < stages) load(s);

  int arow[T::RM], brow[T::RN];
#pragma unroll
  for (int r = 0; r < T::RM; ++r) arow[r] = wm * T::RM * 32 + r * 32 + l32;
#pragma unroll
  for (int r = 0; r < T::RN; ++r) brow[r] = T::BM + wn * T::RN * 32 + r * 32 + l32;

  for (int s = 0; s < stages; ++s) {
    if (s + T::STAGES - 1 <= stages)
      wait_vmcnt<(T::STAGES - 2) * T::LOADS>();
    else
      wait_vmcnt<0>();
    bare_barrier();
    const char* stage = smem + s % T::STAGES * T::BYTES;
    if (first + s == all - 1 && a.K % kStageK != 0) {
      for (int c = threadIdx.x; c < T::BM * 8; c += T::THREADS) {
        const int row = c >> 3;
        if ((first + s) * kStageK + ((c & 7) ^ swizzle(row)) * 16 >= a.K) *reinterpret_cast<v4i*>(smem + s % T::STAGES * T::BYTES + c * 16) = 0;
      }
      __syncthreads();
    }
    if (s + T::STAGES - 1 < stages) load(s + T::STAGES - 1);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v4i af[T::RM], bf[T::RN];
#pragma unroll
      for (int r = 0; r < T::RM; ++r) af[r] = *reinterpret_cast<const v4i*>(stage + arow[r] * 128 + ((half * 4 + k) ^ swizzle(arow[r])) * 16);
#pragma unroll
      for (int r = 0; r < T::RN; ++r) bf[r] = *reinterpret_cast<const v4i*>(stage + brow[r] * 128 + ((half * 4 + k) ^ swizzle(brow[r])) * 16);
#pragma unroll
      for (int i = 0; i < T::RM; ++i)
#pragma unroll
        for (int j = 0; j < T::RN; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(af[i], bf[j], acc[i][j], 0, 0, 0);
    }
  }
  bare_barrier();  // every wave's reads are done (its products waited for them): the buffers are free

  // Lane: channel l32 of a fragment, register r: token 8 (r / 4) + 4 half + r % 4.
  float* rs = reinterpret_cast<float*>(smem + T::STAGES * T::BYTES);
  float* cs = rs + T::BM;
  float* bs = cs + T::BN;
  if (KIND != kOutAcc) {
    for (int i = threadIdx.x; i < T::BM; i += T::THREADS) rs[i] = a.a_scale[min(m0 + i, a.M - 1)];
    for (int i = threadIdx.x; i < T::BN; i += T::THREADS) {
      const int n = min(n0 + i, a.N - 1);
      cs[i] = a.w_scale[n];
      bs[i] = a.bias != nullptr ? a.bias[n] : 0.0f;
    }
    __syncthreads();
  }
  int32_t* tr = reinterpret_cast<int32_t*>(smem) + wave * 32 * T::TR;
  void* out = a.splits == 1 ? a.out : a.part + static_cast<int64_t>(split) * a.M * a.N;
#pragma unroll
  for (int j = 0; j < T::RN; ++j) {
    const int col0 = wn * T::RN * 32 + j * 32;
    const float c = KIND == kOutAcc ? 0.0f : cs[col0 + l32], b = KIND == kOutAcc ? 0.0f : bs[col0 + l32];
#pragma unroll
    for (int i = 0; i < T::RM; ++i) {
      const int row0 = wm * T::RM * 32 + i * 32;
      lds_wave_sync();
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int rr = 8 * (r >> 2) + 4 * half + (r & 3);
        int32_t v = acc[i][j][r];
        if (KIND != kOutAcc) {
          v = __float_as_int(scaled(v, rs[row0 + rr], c, a.bias != nullptr, b));
        }
        tr[rr * T::TR + l32] = v;
      }
      lds_wave_sync();
      store_fragment<KIND>(out, a.M, a.N, m0 + row0, n0 + col0, tr, T::TR, lane);
    }
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
    if (KIND == kOutBf16)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + o) =
          make_uint2(bf16_bits(__int_as_float(v[0])) | bf16_bits(__int_as_float(v[1])) << 16,
                     bf16_bits(__int_as_float(v[2])) | bf16_bits(__int_as_float(v[3])) << 16);
    else
      *reinterpret_cast<v4i*>(static_cast<int32_t*>(a.out) + o) = v;
    return;
  }
  int32_t sum = a.part[o];
  for (int s = 1; s < a.splits; ++s) sum += a.part[s * plane + o];
  store_one<KIND>(a.out, o, KIND == kOutAcc ? sum : __float_as_int(scaled(sum, as, a.w_scale[n], a.bias != nullptr, a.bias != nullptr ? a.bias[n] : 0.0f)));
}

struct Plan {
  int rows_rt, rows_mt;  // rows kernel: its RT and MT; rt = 0: the tile kernel
  int tile, splits;
};

// tiles of the tile kernel
using TileL = Tile<256, 256, 2, 4, 2>;
using TileM = Tile<128, 128, 2, 2, 4>;
using TileS = Tile<64, 64, 1, 2, 4>;
constexpr int kBM[3] = {256, 128, 64}, kBN[3] = {256, 128, 64};

Plan make_plan(int64_t M, int64_t N, int64_t K, const DeviceInfo& dev) {
  Plan p = {};
  p.splits = 1;
  if (M <= 32) {
    p.rows_mt = M <= 16 ? 1 : 2;
    p.rows_rt = N >= 16 * 4 * 4 * dev.cu_count ? 4 : N >= 16 * 2 * 4 * dev.cu_count ? 2 : 1;
    return p;
  }
  auto tiles = [&](int t) { return ((M + kBM[t] - 1) / kBM[t]) * ((N + kBN[t] - 1) / kBN[t]); };
  p.tile = tiles(0) >= dev.cu_count ? 0 : tiles(1) >= dev.cu_count ? 1 : 2;
  const int64_t stages = (K + kStageK - 1) / kStageK;
  if (tiles(p.tile) < dev.cu_count)
    p.splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(dev.cu_count / tiles(p.tile), stages / 4)));
  return p;
}

template <int RT, int MT, int KIND>
hipError_t launch_rows(const Int8Args& a, hipStream_t stream) {
  const dim3 grid(static_cast<uint32_t>((static_cast<int64_t>(a.N) + 16 * RT - 1) / (16 * RT)), static_cast<uint32_t>((a.M + 16 * MT - 1) / (16 * MT)));
  int8_rows_kernel<RT, MT, 8, RT == 1 ? 8 : 8 / RT, KIND><<<grid, 512, 0, stream>>>(a);
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
  if (p.rows_rt > 0) {
    if (p.rows_mt == 1) return p.rows_rt == 1 ? launch_rows<1, 1, KIND>(a, stream) : p.rows_rt == 2 ? launch_rows<2, 1, KIND>(a, stream) : launch_rows<4, 1, KIND>(a, stream);
    return p.rows_rt == 1 ? launch_rows<1, 2, KIND>(a, stream) : p.rows_rt == 2 ? launch_rows<2, 2, KIND>(a, stream) : launch_rows<4, 2, KIND>(a, stream);
  }
  if (p.tile == 0) return launch_tiles<TileL, KIND>(a, stream);
  if (p.tile == 1) return launch_tiles<TileM, KIND>(a, stream);
  return launch_tiles<TileS, KIND>(a, stream);
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
