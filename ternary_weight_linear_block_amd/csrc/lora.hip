// lora_add: low-rank adapters of many requests beside a shared projection.
//
// Mathematics, for token t with adapter a = ids[t] (none when a is outside
// 0 .. n-1: then out[t] = y[t]):
//   v[t, r]   = sum_k x[t, k] A[a, r, k]
//   out[t, n] = y[t, n] + sum_r (scale[a] v[t, r]) B[a, n, r]
//
// Two kernels, both on v_mfma_f32_16x16x32_bf16 with the adapter's rows as the
// first operand and 16 tokens as the second, so that a lane's results are
// consecutive ranks (or consecutive n) of one token:
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

constexpr int kShrinkWaves = 8;
constexpr int kExpandWaves = 4;
constexpr int kChunk = 32 * kExpandWaves;  // n of one round of an expand workgroup

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

// Workgroup (tile, slice, p): passes p, p + passes, ... of 16 tokens over one
// slice of K.  RT: 16-row fragments of the rank.
template <int RT>
__global__ __launch_bounds__(64 * kShrinkWaves) void lora_shrink_kernel(LoraArgs a) {
  constexpr int kStride = 16 * RT + 4;  // floats of a token's row, padded
  __shared__ __attribute__((aligned(16))) float red[kShrinkWaves][16 * kStride];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int j = lane & 15, q = lane >> 4;
  const int tile = blockIdx.x % a.shrink_tiles;
  const int rest = blockIdx.x / a.shrink_tiles;
  const int p = rest % a.shrink_passes, slice = rest / a.shrink_passes;
  const int64_t t0 = static_cast<int64_t>(tile) * 16;
  const int K = a.K, R = a.R;
  // this wave's 32-k steps
  const int steps = K / 32, parts = a.slices * kShrinkWaves, part = slice * kShrinkWaves + wave;
  const int s0 = static_cast<int>(static_cast<int64_t>(steps) * part / parts);
  const int s1 = static_cast<int>(static_cast<int64_t>(steps) * (part + 1) / parts);
  const uint16_t* xr = a.x + std::min<int64_t>(t0 + j, a.M - 1) * K + 8 * q;

  Passes passes(a.ids, t0, 16, a.M, a.n, lane);
  int adapter;
  uint64_t tokens;
  for (int i = 0; passes.next(adapter, tokens); ++i) {
    if (i % a.shrink_passes != p) continue;
    const uint16_t* ar[RT];
#pragma unroll
    for (int f = 0; f < RT; ++f)
      ar[f] = a.a + (static_cast<size_t>(adapter) * R + min(16 * f + j, R - 1)) * K + 8 * q;
    v4f acc[RT];
#pragma unroll
    for (int f = 0; f < RT; ++f) acc[f] = v4f{0};
    const auto run = [&](int s, auto count) {  // `count` steps from s, all their loads in flight together
      constexpr int U = decltype(count)::value;
      v8bf xv[U], av[U][RT];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        xv[u] = load8(xr + 32 * (s + u));
#pragma unroll
        for (int f = 0; f < RT; ++f) av[u][f] = load8(ar[f] + 32 * (s + u));
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int f = 0; f < RT; ++f)
          acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av[u][f], xv[u], acc[f], 0, 0, 0);
    };
    constexpr int U = RT <= 2 ? 8 : RT == 4 ? 4 : 2;
    int s = s0;
    for (; s + U <= s1; s += U) run(s, std::integral_constant<int, U>());
    for (; s < s1; ++s) run(s, std::integral_constant<int, 1>());
    // lane (j, q) holds ranks 16 f + 4 q .. + 3 of token j
    __syncthreads();  // the previous pass has been read
#pragma unroll
    for (int f = 0; f < RT; ++f) *reinterpret_cast<v4f*>(&red[wave][j * kStride + 16 * f + 4 * q]) = acc[f];
    __syncthreads();
    for (int e = threadIdx.x; e < 16 * (R / 4); e += 64 * kShrinkWaves) {
      const int tok = e / (R / 4), r = 4 * (e % (R / 4));
      if (!((tokens >> tok) & 1)) continue;
      v4f sum = *reinterpret_cast<const v4f*>(&red[0][tok * kStride + r]);
#pragma unroll
      for (int w = 1; w < kShrinkWaves; ++w) sum += *reinterpret_cast<const v4f*>(&red[w][tok * kStride + r]);
      *reinterpret_cast<v4f*>(a.part + (static_cast<size_t>(slice) * a.M + t0 + tok) * R + r) = sum;
    }
  }
}

// 8 consecutive outputs of one token, n0 .. n0 + 7.  VEC: rows are 16-byte aligned
// (N % 8 == 0), so the eight are inside the row together.
template <bool BF16, bool VEC>
struct Out8 {
  float v[8];

  __device__ __forceinline__ void load(const void* y, size_t row, int n0, int N) {
    if constexpr (VEC) {
      if (n0 >= N) return;
      if constexpr (BF16) {
        const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(y) + row + n0);
        const uint32_t d[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[2 * e] = __uint_as_float(d[e] << 16);
          v[2 * e + 1] = __uint_as_float(d[e] & 0xFFFF0000u);
        }
      } else {
        const v4f lo = *reinterpret_cast<const v4f*>(static_cast<const float*>(y) + row + n0);
        const v4f hi = *reinterpret_cast<const v4f*>(static_cast<const float*>(y) + row + n0 + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[e] = lo[e];
          v[4 + e] = hi[e];
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (n0 + e < N)
          v[e] = BF16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(y)[row + n0 + e]) << 16)
                      : static_cast<const float*>(y)[row + n0 + e];
    }
  }

  __device__ __forceinline__ void store(void* out, size_t row, int n0, int N) const {
    if constexpr (VEC) {
      if (n0 >= N) return;
      if constexpr (BF16) {
        uint32_t d[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          d[e] = f32_to_bf16_rne(v[2 * e]) | (static_cast<uint32_t>(f32_to_bf16_rne(v[2 * e + 1])) << 16);
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + row + n0) = make_uint4(d[0], d[1], d[2], d[3]);
      } else {
        *reinterpret_cast<v4f*>(static_cast<float*>(out) + row + n0) = v4f{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<v4f*>(static_cast<float*>(out) + row + n0 + 4) = v4f{v[4], v[5], v[6], v[7]};
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (n0 + e < N) {
          if (BF16)
            static_cast<uint16_t*>(out)[row + n0 + e] = f32_to_bf16_rne(v[e]);
          else
            static_cast<float*>(out)[row + n0 + e] = v[e];
        }
    }
  }
};

// Workgroup (chunk, tile, p): passes p, p + passes, ... of 16 TT tokens over
// `expand_rounds` ranges of kChunk n.  RS: 32-rank steps.
template <int TT, int RS, bool BF16, bool VEC>
__global__ __launch_bounds__(64 * kExpandWaves) void lora_expand_kernel(LoraArgs a) {
  constexpr int TM = 16 * TT, TERMS = BF16 ? 2 : 3;
  constexpr int kStride = 32 * RS + 8;  // bf16 of a token's row, padded
  __shared__ __attribute__((aligned(16))) uint16_t vt[TERMS][TM * kStride];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int j = lane & 15, q = lane >> 4;
  const int chunk = blockIdx.x % a.expand_chunks;
  const int rest = blockIdx.x / a.expand_chunks;
  const int p = rest % a.expand_passes, tile = rest / a.expand_passes;
  const int64_t t0 = static_cast<int64_t>(tile) * TM;
  const int N = a.N, R = a.R;
  const int n_lo = chunk * a.expand_rounds * kChunk + 32 * wave;
  const int n_hi = min(N, (chunk + 1) * a.expand_rounds * kChunk);

  Passes passes(a.ids, t0, TM, a.M, a.n, lane);
  if (a.out != a.y && p == 0) {
    // tokens without an adapter
    const uint64_t tokens = __ballot(passes.id < 0 && lane < TM && t0 + lane < a.M);
#pragma unroll
    for (int tt = 0; tt < TT; ++tt)
      if ((tokens >> (16 * tt + j)) & 1) {
        const size_t row = static_cast<size_t>(t0 + 16 * tt + j) * N;
        for (int nb = n_lo; nb < n_hi; nb += kChunk) {
          Out8<BF16, VEC> o;
          o.load(a.y, row, nb + 8 * q, N);
          o.store(a.out, row, nb + 8 * q, N);
        }
      }
  }
  int adapter;
  uint64_t tokens;
  for (int i = 0; passes.next(adapter, tokens); ++i) {
    if (i % a.expand_passes != p) continue;
    const float scale = a.scale[adapter];
    __syncthreads();  // the previous pass has been read
    for (int e = threadIdx.x; e < TM * (32 * RS / 4); e += 64 * kExpandWaves) {
      const int tok = e / (32 * RS / 4), r = 4 * (e % (32 * RS / 4));
      v4f v = {0.0f, 0.0f, 0.0f, 0.0f};
      if (r < R && ((tokens >> tok) & 1)) {
        const float* src = a.part + static_cast<size_t>(t0 + tok) * R + r;
        for (int s = 0; s < a.slices; ++s) v += *reinterpret_cast<const v4f*>(src + static_cast<size_t>(s) * a.M * R);
        v *= scale;
      }
#pragma unroll
      for (int term = 0; term < TERMS; ++term) {
        uint16_t b[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          b[c] = f32_to_bf16_rne(v[c]);
          v[c] -= __uint_as_float(static_cast<uint32_t>(b[c]) << 16);
        }
        *reinterpret_cast<uint2*>(&vt[term][tok * kStride + r]) =
            make_uint2(b[0] | (static_cast<uint32_t>(b[1]) << 16), b[2] | (static_cast<uint32_t>(b[3]) << 16));
      }
    }
    __syncthreads();
    for (int nb = n_lo; nb < n_hi; nb += kChunk) {
      // fragment f row i of the first operand is n = nb + 8 (i / 4) + 4 f + i % 4, so
      // that lane (j, q) ends up with n = nb + 8 q .. + 7 of token j
      v8bf w[2][RS];
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const int n = min(nb + 8 * (j >> 2) + 4 * f + (j & 3), N - 1);
        const uint16_t* br = a.b + (static_cast<size_t>(adapter) * N + n) * R;
#pragma unroll
        for (int s = 0; s < RS; ++s) w[f][s] = load8(br + min(32 * s + 8 * q, R - 8));
      }
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) {
        if (((tokens >> (16 * tt)) & 0xFFFF) == 0) continue;
        const bool mine = (tokens >> (16 * tt + j)) & 1;
        const size_t row = static_cast<size_t>(t0 + 16 * tt + j) * N;
        Out8<BF16, VEC> o;
        if (mine) o.load(a.y, row, nb + 8 * q, N);
        v4f acc[2] = {v4f{0}, v4f{0}};
#pragma unroll
        for (int s = 0; s < RS; ++s)
#pragma unroll
          for (int term = 0; term < TERMS; ++term) {
            const v8bf v = load8(&vt[term][(16 * tt + j) * kStride + 32 * s + 8 * q]);
#pragma unroll
            for (int f = 0; f < 2; ++f) acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[f][s], v, acc[f], 0, 0, 0);
          }
        if (mine) {
#pragma unroll
          for (int e = 0; e < 8; ++e) o.v[e] += acc[e >> 2][e & 3];
          o.store(a.out, row, nb + 8 * q, N);
        }
      }
    }
  }
}

template <int TT, int RS>
hipError_t launch_expand(const LoraArgs& a, bool bf16, unsigned grid, hipStream_t stream) {
  const dim3 g(grid), b(64 * kExpandWaves);
  const bool vec = a.N % 8 == 0;
  if (bf16 && vec) hipLaunchKernelGGL((lora_expand_kernel<TT, RS, true, true>), g, b, 0, stream, a);
  else if (bf16) hipLaunchKernelGGL((lora_expand_kernel<TT, RS, true, false>), g, b, 0, stream, a);
  else if (vec) hipLaunchKernelGGL((lora_expand_kernel<TT, RS, false, true>), g, b, 0, stream, a);
  else hipLaunchKernelGGL((lora_expand_kernel<TT, RS, false, false>), g, b, 0, stream, a);
  return hipGetLastError();
}

int ceil_div(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

// Tokens up to which a tile's passes go to different workgroups: every token may
// have an adapter of its own, as in decode.
constexpr int kSplitPassesM = 64;

// Workgroups of K slices: enough to give every CU one, a wave at least four
// 32-k steps.
void plan_shrink(LoraArgs& a, const DeviceInfo& dev) {
  a.shrink_tiles = ceil_div(a.M, 16);
  a.shrink_passes = a.M <= kSplitPassesM ? static_cast<int>(std::min<int64_t>({16, a.M, std::max(1, a.n)})) : 1;
  const int want = ceil_div(std::max(1, dev.cu_count), static_cast<int64_t>(a.shrink_tiles) * a.shrink_passes);
  a.slices = std::max(1, std::min(want, a.K / 32 / (4 * kShrinkWaves)));
}

}  // namespace

size_t lora_workspace_bytes(int64_t M, int K, int R, int64_t n, const DeviceInfo& dev) {
  if (M <= 0 || n <= 0) return 0;
  LoraArgs a = {};
  a.M = M;
  a.K = K;
  a.R = R;
  a.n = static_cast<int>(n);
  plan_shrink(a, dev);
  return static_cast<size_t>(a.slices) * static_cast<size_t>(M) * R * sizeof(float);
}

hipError_t launch_lora(LoraArgs a, bool bf16, const DeviceInfo& dev, hipStream_t stream) {
  if (a.M == 0 || a.N == 0) return hipSuccess;
  plan_shrink(a, dev);
  const int64_t shrink_grid = static_cast<int64_t>(a.shrink_tiles) * a.shrink_passes * a.slices;
  // 64 tokens a workgroup (each reads its adapters' B once for four fragments of
  // tokens) where that still gives every CU a workgroup
  const int rounds_all = ceil_div(a.N, kChunk);
  const int TT = static_cast<int64_t>(ceil_div(a.M, 64)) * rounds_all >= dev.cu_count && a.M > kSplitPassesM ? 4 : 1;
  a.expand_passes = a.M <= kSplitPassesM ? static_cast<int>(std::min<int64_t>({16, a.M, std::max(1, a.n)})) : 1;
  const int64_t tiles = ceil_div(a.M, 16 * TT);
  // several ranges of n a workgroup, which share the sum over the slices, where
  // that leaves four workgroups a CU
  a.expand_rounds = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(16, tiles * rounds_all / (4 * std::max(1, dev.cu_count)))));
  a.expand_chunks = ceil_div(rounds_all, a.expand_rounds);
  const int64_t expand_grid = tiles * a.expand_passes * a.expand_chunks;
  if (shrink_grid > 0x7FFFFFFF || expand_grid > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  const dim3 g(static_cast<unsigned>(shrink_grid)), b(64 * kShrinkWaves);
  if (a.n == 0) ;  // no adapter at all: only the copy below
  else if (a.R <= 16) hipLaunchKernelGGL(lora_shrink_kernel<1>, g, b, 0, stream, a);
  else if (a.R <= 32) hipLaunchKernelGGL(lora_shrink_kernel<2>, g, b, 0, stream, a);
  else if (a.R <= 64) hipLaunchKernelGGL(lora_shrink_kernel<4>, g, b, 0, stream, a);
  else hipLaunchKernelGGL(lora_shrink_kernel<8>, g, b, 0, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const unsigned eg = static_cast<unsigned>(expand_grid);
  if (TT == 1)
    return a.R <= 32 ? launch_expand<1, 1>(a, bf16, eg, stream)
           : a.R <= 64 ? launch_expand<1, 2>(a, bf16, eg, stream) : launch_expand<1, 4>(a, bf16, eg, stream);
  return a.R <= 32 ? launch_expand<4, 1>(a, bf16, eg, stream)
         : a.R <= 64 ? launch_expand<4, 2>(a, bf16, eg, stream) : launch_expand<4, 4>(a, bf16, eg, stream);
}

}  // namespace twl
