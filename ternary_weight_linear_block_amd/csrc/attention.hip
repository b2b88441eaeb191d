// window_attention: causal attention over the pages of a cache with a sliding window
// and a few first tokens that stay visible (include/twl.h).
//
//   o = sum_j p_j v_j / sum_j p_j,   p_j = 2^(s_j - m),  s_j = scale log2(e) q k_j
//
// over the keys j that the query at position p sees: j <= p and (p - j < window or
// j < sinks).  One pass: m is the running maximum, and what was summed before is
// multiplied by 2^(m_old - m_new).
#include "attention_internal.h"

#include <algorithm>

namespace twl {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v4bf __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));

// Start of a running maximum: finite, so that differences of two of them are numbers;
// a masked score is -infinity and its weight exactly 0.
constexpr float kNoMax = -1e30f;

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) char*)(p)));
}

// Direct global->LDS load of 16 bytes a lane to lds_base + 16 * lane (see gemm_i8.hip).
__device__ __forceinline__ void dma16(const void* src, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %1\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "s"(lds_base) : "memory", "m0");
}

// The same from a wave-uniform address plus a lane's offset.
__device__ __forceinline__ void dma16(const void* base, uint32_t offset, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(offset), "s"(base), "s"(lds_base) : "memory", "m0");
}

__device__ __forceinline__ void wait_vm0() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Four elements of one column from four rows: within 16 lanes, lane l gives the address
// of elements 4 (l % 4) .. + 3 of row l / 4 and receives column l of rows 0 .. 3.
__device__ __forceinline__ v4bf read_tr(uint32_t addr) {
  return __builtin_bit_cast(v4bf, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                      reinterpret_cast<__attribute__((address_space(3))) v4s*>(addr)));
}

// One sequence's share of a workgroup's tile of `rows` packed rows (a row: a new token
// and one of the g query heads of a key head, row = token * g + head).
struct Tile {
  int seq, q0, n;     // sequence, its first new token in q, its new tokens
  int row0;           // first packed row in the sequence
  int kv;             // context length
  int seen;           // keys that the page table holds, at most kv
};

// The sequence of tile `tile`: sequence b owns the tiles from floor(q_start[b] g / rows) + b,
// which leaves it at least ceil(n g / rows) of them.  False for a tile without rows.
__device__ __forceinline__ bool find_tile(const AttnArgs& a, int tile, int rows, int lane, Tile* t) {
  int count = 0;
  for (int base = 0; base < a.B; base += 64) {
    const int b = base + lane;
    bool before = false;
    if (b < a.B) {
      const int64_t q0 = min(max(a.q_start[b], 0), a.T);
      before = q0 * a.group / rows + b <= tile;
    }
    const int here = __popcll(__ballot(before));
    count += here;
    if (here < 64) break;
  }
  if (count == 0) return false;
  const int b = count - 1;
  t->seq = b;
  t->q0 = min(max(a.q_start[b], 0), a.T);
  t->n = min(max(a.q_start[b + 1], t->q0), a.T) - t->q0;
  const int first = static_cast<int>(static_cast<int64_t>(t->q0) * a.group / rows) + b;
  t->row0 = (tile - first) * rows;
  t->kv = max(a.kv_len[b], 0);
  t->seen = a.n_pages > 0 ? static_cast<int>(min(static_cast<int64_t>(t->kv), static_cast<int64_t>(a.table_pages) << a.page_shift)) : 0;
  return t->row0 < t->n * a.group;
}

// The blocks of `size` keys that the rows of a tile see: `sink` blocks from key 0 and
// the blocks first .. first + total - sink - 1.
struct Blocks {
  int lo, hi, sink, first, total;
};

__device__ __forceinline__ Blocks find_blocks(const AttnArgs& a, const Tile& t, int rows, int size) {
  Blocks k;
  const int i0 = t.row0 / a.group, i1 = (min(t.row0 + rows, t.n * a.group) - 1) / a.group;
  const int p0 = t.kv - t.n + i0, p1 = t.kv - t.n + i1;
  k.hi = max(min(t.seen, p1 + 1), 0);
  k.lo = a.window > 0 ? min(max(p0 - a.window + 1, 0), k.hi) : 0;
  k.first = k.lo / size;
  k.sink = (min(min(a.sinks, k.first * size), k.hi) + size - 1) / size;
  k.total = k.sink + (k.hi + size - 1) / size - k.first;
  return k;
}

// Splits of a tile's blocks that do work: at most a.splits, each of kSplitBlocks or more.
constexpr int kSmallRows = 16, kSmallKeys = 32, kSmallWaves = 4, kSplitBlocks = 2 * kSmallWaves;
constexpr int kLargeSplitBlocks = 4;

__device__ __forceinline__ int large_splits(const AttnArgs& a, int total) {
  return max(1, min(a.large_splits, total / kLargeSplitBlocks));
}

// Workgroup barriers: alone, and behind this wave's LDS operations.
__device__ __forceinline__ void bare_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  bare_barrier();
}

__device__ __forceinline__ const void* sgpr_ptr(const void* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
  return reinterpret_cast<const void*>((static_cast<uint64_t>(hi) << 32) | lo);
}

// The value of the lane 32 on (or back).
__device__ __forceinline__ float other_half(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(threadIdx.x & 32 ? r[0] : r[1]);
}

__device__ __forceinline__ float add_pair(v2bf pair, float sum) {
  return __builtin_amdgcn_fdot2_f32_bf16(pair, v2bf{static_cast<__bf16>(1.0f), static_cast<__bf16>(1.0f)}, sum, false);
}

__device__ __forceinline__ int active_splits(const AttnArgs& a, int total) {
  return max(1, min(a.splits, total / kSplitBlocks));
}

// Few rows (decode, drafted tokens): one tile of 16 packed rows a workgroup, its waves
// (and a.splits workgroups) take the blocks of 32 keys in turn and join their sums.
//
// S^T = K Q^T on 16x16x32 MFMAs: a lane holds row lane % 16 and, with the rows of K
// taken in the order below, the scores of keys 8 (lane / 16) .. + 7 of a block, which
// is where O^T = V^T P^T wants its P.  V^T comes from the wave's own LDS by transposing reads.
template <int D>
__global__ __launch_bounds__(256) void attention_small_kernel(AttnArgs a) {
  constexpr int C = D / 32;                 // steps of 32 along D
  constexpr int DT = D / 16;                // tiles of 16 along D
  constexpr int ROW = 2 * D;                // bytes of a key
  constexpr int VBYTES = kSmallKeys * ROW;  // a wave's block of V; later its 16 x D sums in fp32
  __shared__ __attribute__((aligned(16))) char smem[kSmallWaves * VBYTES];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, h = lane >> 4;
  const int head = blockIdx.x % a.n_kv;
  const int split = blockIdx.x / a.n_kv % a.splits;
  Tile t;
  if (!find_tile(a, blockIdx.x / a.n_kv / a.splits, kSmallRows, lane, &t) || t.n * a.group > a.small_rows) return;
  const Blocks k = find_blocks(a, t, kSmallRows, kSmallKeys);
  const int splits = active_splits(a, k.total);
  if (split >= splits) return;
  const int from = static_cast<int>(static_cast<int64_t>(k.total) * split / splits);
  const int to = static_cast<int>(static_cast<int64_t>(k.total) * (split + 1) / splits);

  // this lane's row
  const int row = t.row0 + m;
  const bool real = row < t.n * a.group;
  const int token = min(row, t.n * a.group - 1) / a.group, qh = head * a.group + min(row, t.n * a.group - 1) % a.group;
  const int p = t.kv - t.n + token;
  const int64_t out_row = static_cast<int64_t>(t.q0 + token) * a.n_q + qh;
  v8bf q[C];
#pragma unroll
  for (int c = 0; c < C; ++c) q[c] = *reinterpret_cast<const v8bf*>(a.q + out_row * D + c * 32 + h * 8);

  const int32_t* table = a.page_table + static_cast<int64_t>(t.seq) * a.table_pages;
  const int page_mask = (1 << a.page_shift) - 1;
  char* vmem = smem + wave * VBYTES;
  const uint32_t vbase = lds_addr(vmem);

  v4f o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d) o[d] = 0.0f;
  float mx = kNoMax, sum = 0.0f;

  for (int i = from + wave; i < to; i += kSmallWaves) {
    const int key0 = (i < k.sink ? i : i - k.sink + k.first) * kSmallKeys;
    // the block lies in one page, or in two of 16 keys
    const int e0 = key0 >> a.page_shift, e1 = (key0 + 16) >> a.page_shift;
    int pg0 = table[min(e0, a.table_pages - 1)], pg1 = table[min(e1, a.table_pages - 1)];
    const bool bad0 = pg0 < 0 || pg0 >= a.n_pages, bad1 = pg1 < 0 || pg1 >= a.n_pages;
    if (bad0) pg0 = 0;
    if (bad1) pg1 = 0;
    const int64_t at0 = ((static_cast<int64_t>(pg0) * a.n_kv + head) << a.page_shift) + (key0 & page_mask);
    const int64_t at1 = ((static_cast<int64_t>(pg1) * a.n_kv + head) << a.page_shift) + ((key0 + 16) & page_mask);
    // V, 1 KB an instruction; a row's 32-byte units are XOR-swizzled by the key
#pragma unroll
    for (int n = 0; n < VBYTES / 1024; ++n) {
      const int byte = n * 1024 + lane * 16;
      const int key = byte / ROW, unit = (byte % ROW) / 32;
      const int swz = D == 64 ? key & 3 : (key & 3) | (key >> 1 & 4);
      const int64_t at = key < 16 ? at0 + key : at1 + (key - 16);
      dma16(reinterpret_cast<const char*>(a.v) + at * ROW + (unit ^ swz) * 32 + (byte & 16), vbase + n * 1024);
    }
    v4f s0 = 0.0f, s1 = 0.0f;
    const int64_t at = m < 8 ? at0 + (m >> 2) * 8 + (m & 3) : at1 + (m >> 2) * 8 + (m & 3) - 16;
    const uint16_t* kp = a.k + at * D + h * 8;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const v8bf k0 = *reinterpret_cast<const v8bf*>(kp + c * 32);
      const v8bf k1 = *reinterpret_cast<const v8bf*>(kp + 4 * D + c * 32);
      s0 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k0, q[c], s0, 0, 0, 0);
      s1 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k1, q[c], s1, 0, 0, 0);
    }
    float s[8] = {s0[0], s0[1], s0[2], s0[3], s1[0], s1[1], s1[2], s1[3]};
    // keys past the last, before the window or in a page that is none
    const bool border = bad0 || bad1 || key0 + kSmallKeys - 1 > min(k.hi - 1, t.kv - t.n + t.row0 / a.group) ||
                        (a.window > 0 && key0 < t.kv - a.window);
    float top = mx;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      s[e] *= a.scale_log2;
      if (border) {
        const int j = key0 + 8 * h + e;
        const bool sees = j <= p && j < t.seen && (a.window == 0 || p - j < a.window || j < a.sinks) && !(h < 2 ? bad0 : bad1);
        s[e] = sees ? s[e] : -__builtin_inff();
      }
      top = fmaxf(top, s[e]);
    }
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    const float alpha = __builtin_amdgcn_exp2f(mx - top);
    mx = top;
    float part = 0.0f;
    v8bf pr;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      pr[e] = static_cast<__bf16>(__builtin_amdgcn_exp2f(s[e] - top));
      part += static_cast<float>(pr[e]);  // the weights as the product has them: their rounding divides out in part
    }
    sum = sum * alpha + part;
#pragma unroll
    for (int d = 0; d < DT; ++d) o[d] *= alpha;
    wait_vm0();
    if (border) {
      // what no row sees may hold anything: its weight 0 must meet a number
      const int key = lane >> 1;
      const int j = key0 + key;
      const bool dead = j >= k.hi || (j < k.lo && j >= a.sinks) || (key < 16 ? bad0 : bad1);
      if (dead)
#pragma unroll
        for (int c = 0; c < ROW / 32; ++c)
          *reinterpret_cast<v4f*>(vmem + key * ROW + (lane & 1) * (ROW / 2) + c * 16) = 0.0f;
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      v4bf half[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int key = h * 8 + e * 4 + (m >> 2);
        const int swz = D == 64 ? key & 3 : (key & 3) | (key >> 1 & 4);
        half[e] = read_tr(vbase + key * ROW + (d ^ swz) * 32 + (m & 3) * 8);
      }
      const v8bf vt = __builtin_shufflevector(half[0], half[1], 0, 1, 2, 3, 4, 5, 6, 7);
      o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vt, pr, o[d], 0, 0, 0);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the reads are done before the next block lands
  }

  // join the waves: every wave's maximum, sum and O^T through LDS
  __shared__ float stat[2][kSmallWaves][16];
  sum += __shfl_xor(sum, 16);
  sum += __shfl_xor(sum, 32);
  if (h == 0) {
    stat[0][wave][m] = mx;
    stat[1][wave][m] = sum;
  }
  __syncthreads();
  float top = kNoMax, all = 0.0f;
#pragma unroll
  for (int w = 0; w < kSmallWaves; ++w) top = fmaxf(top, stat[0][w][m]);
#pragma unroll
  for (int w = 0; w < kSmallWaves; ++w) all += stat[1][w][m] * __builtin_amdgcn_exp2f(stat[0][w][m] - top);
  const float mine = __builtin_amdgcn_exp2f(mx - top);
  v4f* mem = reinterpret_cast<v4f*>(vmem);
#pragma unroll
  for (int d = 0; d < DT; ++d) mem[d * 64 + lane] = o[d] * mine;  // lane: row m, d * 16 + h * 4 .. + 3
  __syncthreads();
  const bool whole = splits == 1;
  const float inv = whole && all > 0.0f ? 1.0f / all : 0.0f;
#pragma unroll
  for (int u = 0; u < DT / kSmallWaves; ++u) {
    const int d = u * kSmallWaves + wave;
    v4f v = 0.0f;
#pragma unroll
    for (int w = 0; w < kSmallWaves; ++w) v += reinterpret_cast<const v4f*>(smem + w * VBYTES)[d * 64 + lane];
    if (!real) continue;
    if (whole)
      *reinterpret_cast<v4bf*>(a.out + out_row * D + d * 16 + h * 4) = __builtin_convertvector(v * inv, v4bf);
    else
      *reinterpret_cast<v4f*>(a.part + (static_cast<int64_t>(split) * a.T * a.n_q + out_row) * D + d * 16 + h * 4) = v;
  }
  if (!whole && real && wave == 0 && h == 0) {
    float* ml = a.part + static_cast<int64_t>(a.max_splits) * a.T * a.n_q * D + (static_cast<int64_t>(split) * a.T * a.n_q + out_row) * 2;
    ml[0] = top;
    ml[1] = all;
  }
}

// Many rows: a tile of 32 WAVES packed rows a workgroup, 32 of them a wave, whose waves
// share each block of KT x 32 keys in LDS (two buffers, loaded a block ahead).
//
// S^T = K Q^T and O^T = V^T P^T on 32x32x16 MFMAs: a lane holds one row (lane % 32) in both,
// so that maximum, sum and factors are a lane's own (and its partner's, 32 lanes on), and
// the scores' registers are the operand of the second product as they lie: registers 8 a .. 8 a + 7
// of a 32-key tile are keys 16 a + 4 (lane / 32) .. + 3 and 8 more on, and the transposing reads
// of V take the keys in that order.
//
// The maximum that weights refer to follows the scores' only when a row's grows by more than
// 2^8 (weights stay below 2^8, sums far below fp32's range): most blocks leave O as it is.
template <int D, int WAVES>
struct Large {
  static constexpr int KT = D == 256 ? 1 : 2, KEYS = 32 * KT, ROWS = 32 * WAVES;
  static constexpr int ROW = 2 * D, CHUNKS = D / 8;             // bytes and 16-byte chunks of a key
  static constexpr int RPI = 1024 / ROW;                        // keys of a load instruction
  static constexpr int LOADS = KEYS / RPI / WAVES;              // load instructions of a wave for K, and for V
  static constexpr int TILE = KEYS * ROW;                       // bytes of a block's K
  static_assert(KEYS % (RPI * WAVES) == 0, "whole loads");

  // K: chunks of 16 adjacent keys on distinct banks; V: the 64-byte units of four adjacent keys.
  __device__ static __forceinline__ int k_place(int key, int chunk) { return chunk ^ (D == 64 ? (key ^ (key >> 3 & 3)) & 7 : key & 15); }
  __device__ static __forceinline__ int v_turn(int key) { return D == 64 ? key >> 1 & 1 : key & 3; }
};

template <int D, int WAVES>
__global__ __launch_bounds__(64 * WAVES, D == 256 ? 1 : 2) void attention_large_kernel(AttnArgs a) {
  using L = Large<D, WAVES>;
  constexpr int KT = L::KT, KEYS = L::KEYS, ROW = L::ROW, DS = D / 16, DT = D / 32;
  __shared__ __attribute__((aligned(16))) char smem[4 * L::TILE];  // K, V of two blocks
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l32 = lane & 31, half = lane >> 5;
  const int head = blockIdx.x % a.n_kv, split = blockIdx.x / a.n_kv % a.large_splits;
  // the last tiles of a sequence see the most keys: they start first
  const int tile = static_cast<int>(gridDim.x / (a.n_kv * a.large_splits)) - 1 - static_cast<int>(blockIdx.x / a.n_kv / a.large_splits);
  Tile t;
  if (!find_tile(a, tile, L::ROWS, lane, &t) || t.n * a.group <= a.small_rows) return;
  const Blocks k = find_blocks(a, t, L::ROWS, KEYS);
  const int splits = large_splits(a, k.total);
  if (split >= splits) return;
  const int from = static_cast<int>(static_cast<int64_t>(k.total) * split / splits);
  const int to = static_cast<int>(static_cast<int64_t>(k.total) * (split + 1) / splits);

  // this wave's rows, this lane's row
  const int rows = t.n * a.group, first_row = t.row0 + wave * 32;
  const int row = min(first_row + l32, rows - 1), token = row / a.group;
  const int p = t.kv - t.n + token;
  const int p_low = t.kv - t.n + min(first_row, rows - 1) / a.group, p_high = first_row < rows ? t.kv - t.n + min(first_row + 31, rows - 1) / a.group : -1;
  const int64_t out_row = static_cast<int64_t>(t.q0 + token) * a.n_q + head * a.group + row % a.group;
  const float scale = a.scale_log2 == 0.0f ? 1.0f : __builtin_fabsf(a.scale_log2);
  v8bf q[DS];
#pragma unroll
  for (int c = 0; c < DS; ++c) {
    v8s bits = *reinterpret_cast<const v8s*>(a.q + out_row * D + c * 16 + half * 8);
    if (a.scale_log2 < 0.0f) bits ^= static_cast<short>(0x8000);
    if (a.scale_log2 == 0.0f) bits = 0;
    q[c] = __builtin_bit_cast(v8bf, bits);
  }

  const int32_t* table = a.page_table + static_cast<int64_t>(t.seq) * a.table_pages;
  const int page_mask = (1 << a.page_shift) - 1;
  const uint32_t lds = lds_addr(smem);
  uint32_t k_off[L::LOADS], v_off[L::LOADS];
#pragma unroll
  for (int i = 0; i < L::LOADS; ++i) {
    const int key = (i * WAVES + wave) * L::RPI + lane / L::CHUNKS, chunk = lane % L::CHUNKS;
    k_off[i] = lane / L::CHUNKS * ROW + L::k_place(key, chunk) * 16;
    v_off[i] = lane / L::CHUNKS * ROW + (chunk ^ L::v_turn(key) * 4) * 16;
  }
  auto key_of = [&](int i) { return (i < k.sink ? i : i - k.sink + k.first) * KEYS; };
  // the pages of block i's keys, one a lane
  auto pages = [&](int i) { return table[min((key_of(min(i, to - 1)) + lane % KEYS) >> a.page_shift, a.table_pages - 1)]; };
  auto load = [&](int i, int page_ids) {
    const int key0 = key_of(i);
#pragma unroll
    for (int n = 0; n < L::LOADS; ++n) {
      const int key = (n * WAVES + wave) * L::RPI;  // a load's keys lie in one page
      int page = __builtin_amdgcn_readlane(page_ids, key);
      if (page < 0 || page >= a.n_pages) page = 0;
      const int64_t at = ((((static_cast<int64_t>(page) * a.n_kv + head) << a.page_shift) + ((key0 + key) & page_mask))) * ROW;
      const uint32_t to_lds = lds + (i & 1) * 2 * L::TILE + key * ROW;
      dma16(sgpr_ptr(reinterpret_cast<const char*>(a.k) + at), k_off[n], to_lds);
      dma16(sgpr_ptr(reinterpret_cast<const char*>(a.v) + at), v_off[n], to_lds + L::TILE);
    }
  };

  v16f o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d) o[d] = 0.0f;
  float mx = kNoMax, sum = 0.0f;
  const int kx = L::k_place(l32, half) * 16;                    // XOR a step's 32 bytes: the lane's chunk of its key
  const int vkey = 4 * half + (lane >> 2 & 3);                  // the lane's key of a transposing read, of 8
  const uint32_t k_read = lds + l32 * ROW, v_read = lds + L::TILE + vkey * ROW + (lane >> 4 & 1) * 32 + (lane & 3) * 8;

  int ids = 0, next_ids = 0;
  if (from < to) {
    ids = pages(from);
    next_ids = pages(from + 1);
    load(from, ids);
  }
  for (int i = from; i < to; ++i) {
    const int key0 = key_of(i);
    const uint64_t none = __ballot(ids < 0 || ids >= a.n_pages);  // lanes of keys whose page is none
    wait_vm0();
    lds_barrier();
    ids = next_ids;
    if (i + 1 < to) load(i + 1, ids);
    next_ids = pages(i + 2);
    if (none != 0 || key0 + KEYS > k.hi || (key0 < k.lo && key0 + KEYS > a.sinks)) {
      // what no row of the tile sees may hold anything: its weight 0 must meet a number
      char* v = smem + (i & 1) * 2 * L::TILE + L::TILE;
      for (int c = threadIdx.x; c < L::TILE / 16; c += 64 * WAVES) {
        const int key = c / L::CHUNKS, j = key0 + key;
        if (j >= k.hi || (j < k.lo && j >= a.sinks) || (none >> key & 1)) *reinterpret_cast<v4f*>(v + c * 16) = 0.0f;
      }
      lds_barrier();
    }
    // blocks that none of the wave's rows sees
    if (key0 > p_high || (a.window > 0 && key0 >= a.sinks && key0 + KEYS <= p_low - a.window + 1)) continue;

    const uint32_t kb = k_read + (i & 1) * 2 * L::TILE, vb = v_read + (i & 1) * 2 * L::TILE;
    v16f s[KT];
#pragma unroll
    for (int x = 0; x < KT; ++x) s[x] = 0.0f;
#pragma unroll
    for (int c = 0; c < DS; ++c)
#pragma unroll
      for (int x = 0; x < KT; ++x) {
        const v8bf kf = *reinterpret_cast<const __attribute__((address_space(3))) v8bf*>(kb + (kx ^ c * 32) + x * 32 * ROW);
        s[x] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, q[c], s[x], 0, 0, 0);
      }
    if (none != 0 || key0 + KEYS - 1 > p_low || key0 + KEYS > t.seen || (a.window > 0 && key0 <= p_high - a.window)) {
#pragma unroll
      for (int x = 0; x < KT; ++x)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int key = x * 32 + 8 * (r >> 2) + 4 * half + (r & 3), j = key0 + key;
          const bool sees = j <= p && j < t.seen && (a.window == 0 || p - j < a.window || j < a.sinks) && !(none >> key & 1);
          s[x][r] = sees ? s[x][r] : -__builtin_inff();
        }
    }
    float top = s[0][0];
#pragma unroll
    for (int x = 0; x < KT; ++x)
#pragma unroll
      for (int r = 0; r < 16; ++r) top = fmaxf(top, s[x][r]);
    top = fmaxf(top, other_half(top)) * scale;
    if (__any(top > mx + 8.0f)) {
      const float now = fmaxf(mx, top), alpha = __builtin_amdgcn_exp2f(mx - now);
      mx = now;
      sum *= alpha;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[d] *= alpha;
    }
    v8bf w[KT][2];
#pragma unroll
    for (int x = 0; x < KT; ++x)
#pragma unroll
      for (int r = 0; r < 16; r += 2) {
        v2bf pair;
        pair[0] = static_cast<__bf16>(__builtin_amdgcn_exp2f(__builtin_fmaf(s[x][r], scale, -mx)));
        pair[1] = static_cast<__bf16>(__builtin_amdgcn_exp2f(__builtin_fmaf(s[x][r + 1], scale, -mx)));
        sum = add_pair(pair, sum);  // the weights as the product has them
        w[x][r >> 3][r & 7] = pair[0];
        w[x][r >> 3][(r & 7) + 1] = pair[1];
      }
#pragma unroll
    for (int x = 0; x < KT; ++x)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          const uint32_t at = vb + (d ^ L::v_turn(lane >> 2 & 3)) * 64 + (x * 32 + e * 16) * ROW;
          const v4bf lo = read_tr(at), hi = read_tr(at + 8 * ROW);
          o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7), w[x][e], o[d], 0, 0, 0);
        }
  }

  sum += other_half(sum);
  const bool whole = splits == 1;
  const float inv = !whole ? 1.0f : sum > 0.0f ? 1.0f / sum : 0.0f;
  if (first_row + l32 >= rows) return;
  // registers 4 r .. 4 r + 3 of O^T: elements d * 32 + 8 r + 4 half .. + 3 of the lane's row
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int r = 0; r < 16; r += 4) {
      const v4f v = v4f{o[d][r], o[d][r + 1], o[d][r + 2], o[d][r + 3]} * inv;
      const int64_t at = d * 32 + 2 * r + 4 * half;
      if (whole)
        *reinterpret_cast<v4bf*>(a.out + out_row * D + at) = __builtin_convertvector(v, v4bf);
      else
        *reinterpret_cast<v4f*>(a.part + (static_cast<int64_t>(split) * a.T * a.n_q + out_row) * D + at) = v;
    }
  if (!whole && half == 0) {
    float* ml = a.part + static_cast<int64_t>(a.max_splits) * a.T * a.n_q * D + (static_cast<int64_t>(split) * a.T * a.n_q + out_row) * 2;
    ml[0] = mx;
    ml[1] = sum;
  }
}

// The splits of every row of a tile joined: a wave a row.
template <int D>
__global__ __launch_bounds__(256) void attention_join_kernel(AttnArgs a) {
  constexpr int PER = D / 64;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int head = blockIdx.x % a.n_kv, quarter = blockIdx.x / a.n_kv % 4;
  Tile t;
  if (!find_tile(a, blockIdx.x / a.n_kv / 4, kSmallRows, lane, &t)) return;
  int splits;
  if (t.n * a.group <= a.small_rows) {
    splits = active_splits(a, find_blocks(a, t, kSmallRows, kSmallKeys).total);
  } else {
    Tile large = t;
    large.row0 = t.row0 / a.large_rows * a.large_rows;
    splits = large_splits(a, find_blocks(a, large, a.large_rows, a.large_keys).total);
  }
  const int row = t.row0 + quarter * 4 + wave;
  if (splits == 1 || row >= t.n * a.group) return;
  const int64_t rows = static_cast<int64_t>(a.T) * a.n_q;
  const int64_t out_row = static_cast<int64_t>(t.q0 + row / a.group) * a.n_q + head * a.group + row % a.group;
  const float* ml = a.part + a.max_splits * rows * D + out_row * 2;
  float top = kNoMax;
  for (int s = 0; s < splits; ++s) top = fmaxf(top, ml[s * rows * 2]);
  float all = 0.0f, acc[PER] = {};
  for (int s = 0; s < splits; ++s) {
    const float w = __builtin_amdgcn_exp2f(ml[s * rows * 2] - top);
    all += ml[s * rows * 2 + 1] * w;
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] += a.part[(s * rows + out_row) * D + lane * PER + e] * w;
  }
  const float inv = all > 0.0f ? 1.0f / all : 0.0f;
#pragma unroll
  for (int e = 0; e < PER; ++e)
    *reinterpret_cast<__bf16*>(a.out + out_row * D + lane * PER + e) = static_cast<__bf16>(acc[e] * inv);
}

int64_t tiles_of(const AttnArgs& a, int rows) { return static_cast<int64_t>(a.T) * a.group / rows + a.B; }

// Sequences of more packed rows than this take the kernel for many rows (where the call may hold any).
constexpr int kSmallMost = 64;

// What a call launches.  The lengths are on the device: a call of few rows for its sequences
// runs the kernel for few rows alone, whatever the lengths; others run both, and each
// sequence's length says which one takes it.
struct Plan {
  bool small, large;
  int waves, small_rows, splits, large_splits, max_splits;
};

Plan make_plan(int64_t T, int64_t B, int group, int n_kv, int D, int64_t table_keys, int window, int sinks, const DeviceInfo& dev) {
  Plan p = {};
  const bool few = T * group <= kSmallMost * B || T * group <= kSmallMost;
  p.small = few || B > 1;
  p.large = !few;
  p.small_rows = few ? 1 << 30 : B == 1 ? 0 : kSmallMost;
  // few rows: workgroups that share a tile's keys, enough to fill the device and none of less
  // than kSplitBlocks blocks of what the table can hold
  int64_t keys = table_keys;
  if (window > 0) keys = std::min<int64_t>(keys, static_cast<int64_t>(window) + sinks + kSmallRows + 2 * kSmallKeys);
  const int64_t most = std::max<int64_t>(1, (keys + kSmallKeys - 1) / kSmallKeys / kSplitBlocks);
  const int64_t tiles = std::max<int64_t>(1, std::min(T, T * group / kSmallRows + std::min(B, T))) * n_kv;
  p.splits = !p.small ? 1 : static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(most, 32), 2 * dev.cu_count / tiles)));
  // many rows: 256 a workgroup where that still fills the device, else 128, and splits below that
  const int64_t rows = T * group * n_kv;
  p.waves = D < 256 && rows / 256 >= 2 * dev.cu_count ? 8 : 4;
  const int64_t large_tiles = std::max<int64_t>(1, rows / (32 * p.waves));
  p.large_splits = !p.large ? 1 : static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(table_keys / 512, 16), dev.cu_count / large_tiles)));
  p.max_splits = std::max(p.splits, p.large_splits);
  return p;
}

template <int D, int WAVES>
hipError_t launch_large(AttnArgs& a, hipStream_t stream) {
  using L = Large<D, WAVES>;
  a.large_rows = L::ROWS;
  a.large_keys = L::KEYS;
  attention_large_kernel<D, WAVES><<<static_cast<uint32_t>(tiles_of(a, L::ROWS)) * a.n_kv * a.large_splits, 64 * WAVES, 0, stream>>>(a);
  return hipGetLastError();
}

template <int D>
hipError_t launch_d(AttnArgs a, const Plan& p, hipStream_t stream) {
  a.large_rows = a.large_keys = 32;
  if (p.large) {
    const hipError_t e = p.waves == 8 && D < 256 ? launch_large<D, D < 256 ? 8 : 4>(a, stream) : launch_large<D, 4>(a, stream);
    if (e != hipSuccess) return e;
  }
  const uint32_t tiles = static_cast<uint32_t>(tiles_of(a, kSmallRows)) * a.n_kv;
  if (p.small) {
    attention_small_kernel<D><<<tiles * a.splits, 256, 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.max_splits == 1) return hipSuccess;
  attention_join_kernel<D><<<tiles * 4, 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

size_t attention_workspace_bytes(int64_t T, int64_t B, int n_q, int n_kv, int D, int64_t table_keys, int window, int sinks,
                                 const DeviceInfo& dev) {
  const int splits = make_plan(T, B, n_q / n_kv, n_kv, D, table_keys, window, sinks, dev).max_splits;
  return splits == 1 ? 0 : static_cast<size_t>(splits) * T * n_q * (D + 2) * sizeof(float);
}

hipError_t launch_attention(AttnArgs a, int D, const DeviceInfo& dev, hipStream_t stream) {
  a.group = a.n_q / a.n_kv;
  const Plan p = make_plan(a.T, a.B, a.group, a.n_kv, D, static_cast<int64_t>(a.table_pages) << a.page_shift, a.window, a.sinks, dev);
  a.splits = p.splits;
  a.large_splits = p.large_splits;
  a.max_splits = p.max_splits;
  a.small_rows = p.small_rows;
  if (D == 64) return launch_d<64>(a, p, stream);
  if (D == 128) return launch_d<128>(a, p, stream);
  return launch_d<256>(a, p, stream);
}

}  // namespace twl
