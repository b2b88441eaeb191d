// window_attention: causal attention over the pages of a cache with a sliding window
// and a few first tokens that stay visible (include/twl.h).
//
//   o = sum_j p_j v_j / sum_j p_j,   p_j = 2^(s_j - m),  s_j = scale log2(e) q k_j
//
// over the keys j that the query at position p sees: j <= p and (p - j < window or
// j < sinks).  One pass: m is the running maximum, and what was summed before is
// multiplied by 2^(m_old - m_new).
//
// Scores, maxima and sums are fp32.  The weights p are rounded to bf16, the type of the values that
// they meet in the second product (what the rounding leaves would take a product of its own, half
// as many again); the sum adds the rounded ones.  Against 64 bits outputs are off by 1.7 to 2.0e-3 of
// their norm, where weights in fp32 leave 1.6 to 1.7e-3, the rounding of the outputs alone.
#include "attention_internal.h"

#include <algorithm>
#include <type_traits>

namespace twl {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v4bf __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));

// Start of a running maximum: finite, so that differences of two of them are numbers, and
// below every score; a masked score is -infinity and its weight exactly 0.
constexpr float kNoMax = -3.4028235e38f;

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) char*)(p)));
}

// Direct global->LDS load of 16 bytes a lane, from a wave-uniform address plus a lane's offset to
// lds_base + 16 * lane (see gemm_i8.hip).
__device__ __forceinline__ void dma16(const void* base, uint32_t offset, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(offset), "s"(base), "s"(lds_base) : "memory", "m0");
}

// Waits for this wave's loads, of either kind.  The builtin, not inline asm: the compiler then
// knows that its own loads have landed and does not wait for them again behind later ones.
__device__ __forceinline__ void wait_vm0() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x7 << 4 | 0xF << 8);  // vmcnt 0, the others as they are
  asm volatile("" ::: "memory");
}

// Four elements of one column from four rows: within 16 lanes, lane l gives the address
// of elements 4 (l % 4) .. + 3 of row l / 4 and receives column l of rows 0 .. 3.
__device__ __forceinline__ v4bf read_tr(uint32_t addr) {
  return __builtin_bit_cast(v4bf, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                      reinterpret_cast<__attribute__((address_space(3))) v4s*>(addr)));
}

// Longest context (a table holds no more): positions, windows and their sums stay within 32 bits.
constexpr int kMostKeys = 1 << 30;

// One sequence's share of a workgroup's tile of `rows` packed rows (a row: a new token
// and one of the g query heads of a key head, row = token * g + head).
struct Tile {
  int seq, q0, n;     // sequence, its first new token in q, its new tokens
  int row0;           // first packed row in the sequence
  int kv;             // context length
  int seen;           // keys that the page table holds, at most kv
};

__device__ __forceinline__ void set_sequence(const AttnArgs& a, int seq, int start, int end, int kv, Tile* t) {
  t->seq = seq;
  t->q0 = min(max(start, 0), a.T);
  t->n = min(max(end, t->q0), a.T) - t->q0;
  t->kv = min(max(kv, 0), kMostKeys);
  t->seen = a.n_pages > 0 ? static_cast<int>(min(static_cast<int64_t>(t->kv), static_cast<int64_t>(a.table_pages) << a.page_shift)) : 0;
}

// The last sequence whose start, scaled by `before(start, b)`, is not beyond what is looked
// for: each lane looks at one sequence, and what the found one needs comes with it.
template <class Before>
__device__ __forceinline__ bool find_sequence(const AttnArgs& a, int lane, Tile* t, Before before) {
  bool found = false;
  for (int base = 0; base < a.B; base += 64) {
    const int b = min(base + lane, a.B - 1);
    const int start = a.q_start[b], end = a.q_start[b + 1], kv = a.kv_len[b];
    const int q0 = min(max(start, 0), a.T);
    const int here = __popcll(__ballot(base + lane < a.B && before(q0, b)));
    if (here > 0) {
      found = true;
      set_sequence(a, base + here - 1, __builtin_amdgcn_readlane(start, here - 1), __builtin_amdgcn_readlane(end, here - 1),
                   __builtin_amdgcn_readlane(kv, here - 1), t);
    }
    if (here < 64) break;
  }
  return found;
}

// The sequence of tile `tile`: sequence b owns the tiles from floor(q_start[b] g / rows) + b,
// which leaves it at least ceil(n g / rows) of them.  False for a tile without rows (and, where
// starts decrease, for one before its sequence).
__device__ __forceinline__ bool find_tile(const AttnArgs& a, int tile, int rows, int lane, Tile* t) {
  auto first = [&](int q0, int b) { return static_cast<int>(static_cast<int64_t>(q0) * a.group / rows) + b; };
  if (!find_sequence(a, lane, t, [&](int q0, int b) { return first(q0, b) <= tile; })) return false;
  t->row0 = (tile - first(t->q0, t->seq)) * rows;
  return t->row0 >= 0 && t->row0 < t->n * a.group;
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
constexpr int kLargeSplitBlocks = 2;

// Sequences of more packed rows than this take the kernel for many rows (where the call may hold any); the
// kernel for few rows then has kShortTiles tiles for each sequence.
constexpr int kSmallMost = 64, kShortTiles = kSmallMost / kSmallRows;
constexpr int kAllRows = 1 << 30;  // small_rows where the kernel for few rows takes all sequences

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

// The larger, and the sum, of a lane's value and that of the lane 32 on (or back).
__device__ __forceinline__ float max_halves(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float add_halves(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
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
//
// Bound by the stream of keys and values: 24 tokens of up to 16384 keys of 256, 924 MB, 187 us, 4.9 TB/s, 96%
// of a copy; short contexts by a chain of trips to memory (lengths, pages, keys), 6 us and the join's 4.  A wave's
// next block is in flight, keys to registers and values to LDS, while it works on one (before, 232 us); waves
// take blocks of their own, so that no barrier stands between the loads and the end.
template <int D>
__global__ __launch_bounds__(256) void attention_small_kernel(AttnArgs a) {
  constexpr int C = D / 32;                 // steps of 32 along D
  constexpr int DT = D / 16;                // tiles of 16 along D
  constexpr int ROW = 2 * D;                // bytes of a key
  constexpr int VBYTES = kSmallKeys * ROW;  // a block of V; a wave has two, and later 16 x D sums in fp32 in the first
  __shared__ __attribute__((aligned(16))) char smem[kSmallWaves * 2 * VBYTES];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, h = lane >> 4;
  const int head = blockIdx.x % a.n_kv;
  const int split = blockIdx.x / a.n_kv % a.splits;
  Tile t;
  const int tile = blockIdx.x / a.n_kv / a.splits;
  if (a.small_rows == kAllRows) {
    if (!find_tile(a, tile, kSmallRows, lane, &t)) return;
  } else {
    const int b = tile / kShortTiles;
    set_sequence(a, b, a.q_start[b], a.q_start[b + 1], a.kv_len[b], &t);
    t.row0 = tile % kShortTiles * kSmallRows;
    if (t.row0 >= t.n * a.group || t.n * a.group > a.small_rows) return;
  }
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
  char* vmem = smem + wave * 2 * VBYTES;
  const uint32_t vbase = lds_addr(vmem);

  // The wave's blocks: from + wave, four on each time.  A lane holds the page of 16 keys of one
  // of the next 32 of them.
  const int count = (to - from - wave + kSmallWaves - 1) / kSmallWaves;
  auto key_of = [&](int it) {
    const int i = from + wave + min(it, count - 1) * kSmallWaves;
    return (i < k.sink ? i : i - k.sink + k.first) * kSmallKeys;
  };
  auto pages = [&](int it) { return table[min((key_of(it + (lane >> 1)) + (lane & 1) * 16) >> a.page_shift, a.table_pages - 1)]; };
  struct Keys {
    v8bf k[2][C];
  } cur, next;
  int ids = 0;
  // a block's page ids; the keys 0 .. 15 and 16 .. 31 lie in a page each (or in one)
  auto page_of = [&](int it, int sub) { return __builtin_amdgcn_readlane(ids, (it & 31) * 2 + sub); };
  auto is_none = [&](int page) { return page < 0 || page >= a.n_pages; };
  // V to LDS, 1 KB an instruction (a row's 32-byte units XOR-swizzled by the key), K to registers
  auto load = [&](int it, Keys& to_k) {
    if ((it & 31) == 0) ids = pages(it);
    const int key0 = key_of(it), pg0 = page_of(it, 0), pg1 = page_of(it, 1);
    const int64_t at0 = ((static_cast<int64_t>(is_none(pg0) ? 0 : pg0) * a.n_kv + head) << a.page_shift) + (key0 & page_mask);
    const int64_t at1 = ((static_cast<int64_t>(is_none(pg1) ? 0 : pg1) * a.n_kv + head) << a.page_shift) + ((key0 + 16) & page_mask);
#pragma unroll
    for (int n = 0; n < VBYTES / 1024; ++n) {
      const int byte = n * 1024 + lane * 16;
      const int key = byte / ROW, unit = (byte % ROW) / 32;
      const int swz = D == 64 ? key & 3 : (key & 3) | (key >> 1 & 4);
      const char* base = reinterpret_cast<const char*>(a.v) + (n * 1024 / ROW < 16 ? at0 : at1 - 16) * ROW;  // an instruction's keys lie in one page
      dma16(sgpr_ptr(base), key * ROW + (unit ^ swz) * 32 + (byte & 16), vbase + (it & 1) * VBYTES + n * 1024);
    }
    const int64_t at = m < 8 ? at0 + (m >> 2) * 8 + (m & 3) : at1 + (m >> 2) * 8 + (m & 3) - 16;
    const uint16_t* kp = a.k + at * D + h * 8;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      to_k.k[0][c] = *reinterpret_cast<const v8bf*>(kp + c * 32);
      to_k.k[1][c] = *reinterpret_cast<const v8bf*>(kp + 4 * D + c * 32);
    }
  };

  v4f o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d) o[d] = 0.0f;
  float mx = kNoMax, sum = 0.0f;

  if (count > 0) load(0, next);
  for (int it = 0; it < count; ++it) {
    const int key0 = key_of(it);
    const bool bad0 = is_none(page_of(it, 0)), bad1 = is_none(page_of(it, 1));
    wait_vm0();
    cur = next;
    if (it + 1 < count) load(it + 1, next);
    v4f s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      s0 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(cur.k[0][c], q[c], s0, 0, 0, 0);
      s1 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(cur.k[1][c], q[c], s1, 0, 0, 0);
    }
    float s[8] = {s0[0], s0[1], s0[2], s0[3], s1[0], s1[1], s1[2], s1[3]};
    // keys past the last, before the window or in a page that is none
    const bool border = bad0 || bad1 || key0 + kSmallKeys - 1 > min(k.hi - 1, t.kv - t.n + t.row0 / a.group) ||
                        (a.window > 0 && key0 < t.kv - a.window);
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] *= a.scale_log2;
    if (border) {
      const bool none = h < 2 ? bad0 : bad1;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int j = key0 + 8 * h + e;
        const bool hidden = (j > p) | (j >= t.seen) | ((a.window > 0) & (p - j >= a.window) & (j >= a.sinks)) | none;
        s[e] = hidden ? -__builtin_inff() : s[e];
      }
    }
    float top = mx;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmaxf(top, s[e]);
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
    char* v = vmem + (it & 1) * VBYTES;
    if (border) {
      // what no row sees may hold anything: its weight 0 must meet a number
      const int key = lane >> 1;
      const int j = key0 + key;
      const bool dead = j >= k.hi || (j < k.lo && j >= a.sinks) || (key < 16 ? bad0 : bad1);
      if (dead)
#pragma unroll
        for (int c = 0; c < ROW / 32; ++c)
          *reinterpret_cast<v4f*>(v + key * ROW + (lane & 1) * (ROW / 2) + c * 16) = 0.0f;
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      v4bf half[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int key = h * 8 + e * 4 + (m >> 2);
        const int swz = D == 64 ? key & 3 : (key & 3) | (key >> 1 & 4);
        half[e] = read_tr(vbase + (it & 1) * VBYTES + key * ROW + (d ^ swz) * 32 + (m & 3) * 8);
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
    for (int w = 0; w < kSmallWaves; ++w) v += reinterpret_cast<const v4f*>(smem + w * 2 * VBYTES)[d * 64 + lane];
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

// Many rows: a tile of 128 packed rows a workgroup, 32 of them a wave, whose waves share
// each block of 64 keys in LDS (two buffers, loaded a block ahead).
//
// S^T = K Q^T and O^T = V^T P^T on 32x32x16 MFMAs: a lane holds one row (lane % 32) in both,
// so that maximum, sum and factors are a lane's own (and its partner's, 32 lanes on), and
// the scores' registers are the operand of the second product as they lie: registers 8 a .. 8 a + 7
// of a 32-key tile are keys 16 a + 4 (lane / 32) .. + 3 and 8 more on, and the transposing reads
// of V take the keys in that order.
//
// The maximum that weights refer to follows the scores' only when a row's grows by more than
// 2^8 (weights stay below 2^8, sums far below fp32's range): most blocks leave O as it is.
//
// Bound by the MFMAs and, in the shadow of which they must lie, a block's exponentials and maxima.  Heads
// of 64 and 128: two or three workgroups share a CU, so that one has its products while another has its
// exponentials; 8192 tokens of 40 heads of 128, window 4096: 506 to 561 us, 0.92 to 1.02 PFLOP/s (the library's
// product of 8192^3 in bf16: 1.40; the clock falls as the calls go on).  Heads of 256 (O takes 128 registers): one,
// with all of it between a wave's own products; 4096 causal tokens of 20 heads 215 us, 800 TFLOP/s (one after the
// other: 243).  What a tile costs beside its blocks, 12 us with two on a CU and 17 alone, is a chain of waits: its
// sequence, pages, first keys, stores.
template <int D>
struct Large {
  static constexpr int WAVES = 4, ROWS = 32 * WAVES;
  static constexpr int KT = 2, KEYS = 32 * KT;                  // tiles of 32 keys of a block
  static constexpr int ROW = 2 * D, CHUNKS = D / 8;             // bytes and 16-byte chunks of a key
  static constexpr int RPI = 1024 / ROW;                        // keys of a load instruction
  static constexpr int LOADS = KEYS / RPI / WAVES;              // load instructions of a wave for K, and for V
  static constexpr int TILE = KEYS * ROW;                       // bytes of a block's K
  static_assert(KEYS % (RPI * WAVES) == 0, "whole loads");

  // K: chunks of 16 adjacent keys on distinct banks; V: the 64-byte units of four adjacent keys.
  __device__ static __forceinline__ int k_place(int key, int chunk) { return chunk ^ (D == 64 ? (key ^ (key >> 3 & 3)) & 7 : key & 15); }
  __device__ static __forceinline__ int v_turn(int key) { return D == 64 ? key >> 1 & 1 : key & 3; }
};

template <int D>
__global__ __launch_bounds__(64 * Large<D>::WAVES, D < 256 ? 2 : 1) void attention_large_kernel(AttnArgs a) {
  using L = Large<D>;
  constexpr int KT = L::KT, KEYS = L::KEYS, ROW = L::ROW, DS = D / 16, DT = D / 32;
  constexpr bool WIDE = D == 256;
  __shared__ __attribute__((aligned(16))) char smem[4 * L::TILE];  // K of two blocks, V of two
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

  // Blocks of which every row of the wave sees every key (none to mask), and those of which some row
  // of the tile sees each (none to clean), as ranges of the tile's blocks; sinks' blocks are in neither.
  const int p_low = t.kv - t.n + min(first_row, rows - 1) / a.group, p_high = t.kv - t.n + min(first_row + 31, rows - 1) / a.group;
  auto block_of = [&](int b) { return max(b - k.first, 0) + k.sink; };  // the place of keys b KEYS .. in the tile's blocks
  const int calm_from = block_of(a.window > 0 ? (max(p_high - a.window + 1, 0) + KEYS - 1) / KEYS : 0);
  const int calm_to = block_of(max(min(p_low + 1, t.seen), 0) / KEYS);
  const int whole_from = block_of((k.lo + KEYS - 1) / KEYS), whole_to = block_of(k.hi / KEYS);

  const int32_t* table = a.page_table + static_cast<int64_t>(t.seq) * a.table_pages;
  const int page_mask = (1 << a.page_shift) - 1;
  const uint32_t lds = lds_addr(smem);
  uint32_t k_off[L::LOADS], v_off[L::LOADS];
#pragma unroll
  for (int i = 0; i < L::LOADS; ++i) {
    const int key = (i * L::WAVES + wave) * L::RPI + lane / L::CHUNKS, chunk = lane % L::CHUNKS;
    k_off[i] = lane / L::CHUNKS * ROW + L::k_place(key, chunk) * 16;
    v_off[i] = lane / L::CHUNKS * ROW + (chunk ^ L::v_turn(key) * 4) * 16;
  }
  auto key_of = [&](int i) { return (i < k.sink ? i : i - k.sink + k.first) * KEYS; };
  // A block's keys, one a lane: the byte offset of each in the caches, and the lanes of those whose page is none.
  auto pages = [&](int i) { return table[min((key_of(min(i, to - 1)) + lane % KEYS) >> a.page_shift, a.table_pages - 1)]; };
  struct Where {
    uint32_t lo, hi;
    uint64_t none;
  };
  auto where = [&](int i, int page) {
    Where w;
    const bool bad = page < 0 || page >= a.n_pages;
    w.none = __ballot(bad);
    const uint64_t at = (static_cast<uint64_t>(static_cast<uint32_t>(bad ? 0 : page)) * static_cast<uint32_t>(a.n_kv << a.page_shift) +
                         static_cast<uint32_t>((head << a.page_shift) + ((key_of(i) + lane % KEYS) & page_mask))) * ROW;
    w.lo = static_cast<uint32_t>(at);
    w.hi = static_cast<uint32_t>(at >> 32);
    return w;
  };
  auto load_one = [&](const Where& w, const uint16_t* cache, const uint32_t (&off)[L::LOADS], uint32_t to_lds, int n) {
    const int key = (n * L::WAVES + wave) * L::RPI;  // a load's keys lie in one page
    const uint64_t at = static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(w.hi, key))) << 32 |
                        static_cast<uint32_t>(__builtin_amdgcn_readlane(w.lo, key));
    dma16(reinterpret_cast<const char*>(cache) + at, off[n], to_lds + key * ROW);
  };
  auto load = [&](const Where& w, const uint16_t* cache, const uint32_t (&off)[L::LOADS], uint32_t to_lds) {
#pragma unroll
    for (int n = 0; n < L::LOADS; ++n) load_one(w, cache, off, to_lds, n);
  };

  const int kx = L::k_place(l32, half) * 16;                    // XOR a step's 32 bytes: the lane's chunk of its key
  const int vkey = 4 * half + (lane >> 2 & 3);                  // the lane's key of a transposing read, of 8
  // (the swizzles turn over 256 bytes: what lies 256 on has the same address but for that)
  constexpr int KR = DS < 8 ? DS : 8, VR = DT < 4 ? DT : 4;
  uint32_t k_read[KR], v_read[VR];
#pragma unroll
  for (int c = 0; c < KR; ++c) k_read[c] = lds + l32 * ROW + (kx ^ c * 32);
#pragma unroll
  for (int d = 0; d < VR; ++d)
    v_read[d] = lds + 2 * L::TILE + vkey * ROW + (lane >> 4 & 1) * 32 + (lane & 3) * 8 + (d ^ L::v_turn(lane >> 2 & 3)) * 64;

  v16f o[DT], s[KT];
  v8bf w[KT][2];
#pragma unroll
  for (int d = 0; d < DT; ++d) o[d] = 0.0f;
  float mx = scale > 1.0f ? kNoMax / scale : kNoMax, sum = 0.0f;  // the maximum, not scaled yet

  // Operand of product n of a block's scores, and of its second product, in buffer `odd`.
  auto read_k = [&](int odd, int n) {
    return *reinterpret_cast<const __attribute__((address_space(3))) v8bf*>(k_read[n / KT % KR] + odd * L::TILE + n / KT / KR * 256 + n % KT * 32 * ROW);
  };
  auto read_v = [&](int odd, int n) {
    const uint32_t at = v_read[n % DT % VR] + n % DT / VR * 256 + odd * L::TILE + (n / (2 * DT) * 32 + n / DT % 2 * 16) * ROW;
    const v4bf lo = read_tr(at), hi = read_tr(at + 8 * ROW);
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  // O of a wave alone on its SIMD lies in accumulation registers, 128 beside the 240 of all else, which the
  // compiler does not do by itself (it moved parts of it to and fro, 298 us for 4096 tokens).  It does not know
  // what the instruction is either.  Its operands come from LDS loads, for which the compiler waits, and from
  // before a barrier.  12 states must pass between the instruction and another's use of O: `drain` (20) behind the
  // last product of a block, `settle` around other operations on O.  Two must pass between an operation that writes O
  // and the instruction: add_last has them, since the compiler copies O right before the last block's products.
  // The build checks the distances in what the compiler made (codegen.py).
  auto add_values = [&](v16f& acc, v8bf v, v8bf p) {
    asm volatile("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(v), "v"(p));
  };
  auto add_last = [&](v16f& acc, v8bf v, v8bf p) {
    asm volatile("s_nop 1\n\tv_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(v), "v"(p));
  };
  auto drain = [] { asm volatile("s_nop 15\n\ts_nop 3" ::: "memory"); };
  auto settle = [](v16f& acc) { asm volatile("s_nop 15\n\ts_nop 15" : "+a"(acc)); };
  // The scores of the block in buffer `odd` and the second product of the one before it, in turn
  // (their chains of products are apart), operands read AHEAD products before.
  constexpr int N = DS * KT, AHEAD = WIDE ? 3 : 2;
  auto products = [&](int odd) {
    v8bf kf[AHEAD], vf[AHEAD];
#pragma unroll
    for (int x = 0; x < KT; ++x) s[x] = 0.0f;
#pragma unroll
    for (int n = 0; n < AHEAD; ++n) {
      kf[n] = read_k(odd, n);
      vf[n] = read_v(1 - odd, n);
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      __builtin_amdgcn_sched_barrier(0);
      s[n % KT] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[n % AHEAD], q[n / KT], s[n % KT], 0, 0, 0);
      o[n % DT] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[n % AHEAD], w[n / (2 * DT)][n / DT % 2], o[n % DT], 0, 0, 0);
      if (n + AHEAD < N) {
        kf[n % AHEAD] = read_k(odd, n + AHEAD);
        vf[n % AHEAD] = read_v(1 - odd, n + AHEAD);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  // The scores of block i that a row does not see become -infinity: the keys that the lane's row sees as
  // bits, of which an element takes its own (two operations each; the tests for each element took 11).
  auto mask = [&](v16f (&s)[KT], int i, uint64_t none) {
    if (none == 0 && i >= calm_from && i < calm_to) return;
    const int key0 = key_of(i), last = min(p, t.seen - 1) - key0;
    uint64_t seen = last < 0 ? 0 : ~uint64_t{0} >> (63 - min(last, 63));
    if (a.window > 0) {
      const int first = p - a.window + 1 - key0, sinks = a.sinks - key0;
      const uint64_t near = first > 63 ? 0 : ~uint64_t{0} << max(first, 0), sunk = sinks <= 0 ? 0 : ~uint64_t{0} >> (64 - min(sinks, 64));
      seen &= near | sunk;
    }
    seen = (seen & ~none) >> 4 * half;  // element (x, r) is key x * 32 + 8 (r / 4) + r % 4 behind key0 + 4 half
#pragma unroll
    for (int x = 0; x < KT; ++x) {
      const int bits = static_cast<int>(seen >> x * 32);
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const uint32_t keep = __builtin_amdgcn_sbfe(bits, 8 * (r >> 2) + (r & 3), 1);
        s[x][r] = __uint_as_float((keep & __float_as_uint(s[x][r])) | (~keep & __float_as_uint(-__builtin_inff())));
      }
    }
  };
  // Block i's scores to weights.
  auto weigh = [&](int i, uint64_t none) {
    mask(s, i, none);
    float tops[4];  // chains of their own: a dependent operation waits twice as long as the next one
#pragma unroll
    for (int c = 0; c < 4; ++c) tops[c] = s[c % KT][c];
#pragma unroll
    for (int x = 0; x < KT; ++x)
#pragma unroll
      for (int r = 0; r < 16; r += 2) tops[r / 2 % 4] = fmaxf(fmaxf(tops[r / 2 % 4], s[x][r]), s[x][r + 1]);
    float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
    top = max_halves(top);
    // s scale - mx scale in one operation: exact but for the rounding of mx scale.  Of the weights under one maximum
    // that is a common factor, which divides out; those before and after a move of the maximum differ by the two
    // roundings, half an ulp of a scaled score each (2 in the exponent at 2^26), which is no more than a score in fp32
    // leaves open itself.  Beyond 2^26 the difference comes first.
    float factor = scale, shift = mx * scale;
    if (__any(((top - mx) * scale > 8.0f) | (__builtin_fabsf(shift) > 0x1p26f))) {
      const float now = fmaxf(mx, top), alpha = __builtin_amdgcn_exp2f((mx - now) * scale);
      mx = now;
      shift = mx * scale;
      sum *= alpha;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[d] *= alpha;
      if (__any(__builtin_fabsf(shift) > 0x1p26f)) {
#pragma unroll
        for (int x = 0; x < KT; ++x)
#pragma unroll
          for (int r = 0; r < 16; ++r) s[x][r] = (s[x][r] - mx) * scale;
        factor = 1.0f;
        shift = 0.0f;
      }
    }
    float sums[2] = {sum, 0.0f};
#pragma unroll
    for (int x = 0; x < KT; ++x)
#pragma unroll
      for (int r = 0; r < 16; r += 2) {
        v2bf pair;
        pair[0] = static_cast<__bf16>(__builtin_amdgcn_exp2f(__builtin_fmaf(s[x][r], factor, -shift)));
        pair[1] = static_cast<__bf16>(__builtin_amdgcn_exp2f(__builtin_fmaf(s[x][r + 1], factor, -shift)));
        sums[r / 2 & 1] = add_pair(pair, sums[r / 2 & 1]);  // the weights as the product has them
        w[x][r >> 3][r & 7] = pair[0];
        w[x][r >> 3][(r & 7) + 1] = pair[1];
      }
    sum = sums[0] + sums[1];
  };
  // What no row of the tile sees of block i's values may hold anything: its weight 0 must meet a number.
  auto clean = [&](int i, int odd, uint64_t none) {
    if (none == 0 && i >= whole_from && i < whole_to) return;
    const int key0 = key_of(i);
    char* v = smem + (2 + odd) * L::TILE;
    for (int c = threadIdx.x; c < L::TILE / 16; c += 64 * L::WAVES) {
      const int key = c / L::CHUNKS, j = key0 + key;
      if (j >= k.hi || (j < k.lo && j >= a.sinks) || (none >> key & 1)) *reinterpret_cast<v4f*>(v + c * 16) = 0.0f;
    }
    lds_barrier();
  };

  if (from < to) {
    if constexpr (WIDE) {
      // One wave a SIMD: a block's weights are formed between the products of the next one's scores and
      // of the previous one's values, none of which wait for them.
      // at[x]: block i + x's keys (x = 0, 1, 2), last: the lanes without a page of block i - 1, ids: the pages of block i + 3
      Where at[3] = {where(from, pages(from)), where(from + 1, pages(from + 1)), where(from + 2, pages(from + 2))};
      uint64_t last = 0;
      int ids = pages(from + 3);
      load(at[0], a.k, k_off, lds);
      for (int c = threadIdx.x; c < L::TILE / 16; c += 64 * L::WAVES) *reinterpret_cast<v4f*>(smem + 3 * L::TILE + c * 16) = 0.0f;  // no values yet
      wait_vm0();
      lds_barrier();
      load(at[1], a.k, k_off, lds + L::TILE);
      v16f sc[2][KT];
      v8bf wt[2][KT][2] = {};
#pragma unroll
      for (int x = 0; x < KT; ++x) sc[0][x] = 0.0f;
#pragma unroll
      for (int n = 0; n < N; ++n) sc[0][n % KT] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(read_k(0, n), q[n / KT], sc[0][n % KT], 0, 0, 0);
#pragma unroll
      for (int d = 0; d < DT; ++d) settle(o[d]);
      // Block i, whose buffers are `odd`.
      auto step = [&](int i, int odd) {
        wait_vm0();
        lds_barrier();
        const Where keys = at[2], values = at[0];
        if (i > from) clean(i - 1, 1 - odd, last);
        mask(sc[odd], i, at[0].none);
        v8bf kf[AHEAD], vf[AHEAD];
#pragma unroll
        for (int n = 0; n < AHEAD; ++n) {
          kf[n] = read_k(1 - odd, n);
          vf[n] = read_v(1 - odd, n);
        }
        __builtin_amdgcn_sched_barrier(0);
        last = at[0].none;
        at[0] = at[1];
        at[1] = at[2];
        at[2] = where(i + 3, ids);
        ids = pages(i + 4);
#pragma unroll
        for (int x = 0; x < KT; ++x) sc[1 - odd][x] = 0.0f;
        // of the N pairs of products, the first T come with the maximum, the next 16 KT / 2 with two weights each
        constexpr int T = 4 * KT;
        static_assert(T + 1 + 8 * KT <= N && 4 * L::LOADS == N, "a place for each");
        float tops[2] = {mx, mx}, old = mx, alpha = 1.0f, sums[2];
#pragma unroll
        for (int n = 0; n < N; ++n) {
          __builtin_amdgcn_sched_barrier(0);
          sc[1 - odd][n % KT] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[n % AHEAD], q[n / KT], sc[1 - odd][n % KT], 0, 0, 0);
          // what one product hides comes behind each of the two
          if (n + AHEAD < N) kf[n % AHEAD] = read_k(1 - odd, n + AHEAD);
          const int x = n < T ? n / 4 : n <= T + 8 * KT ? (n - T - 1) / 8 : 0, r = n < T ? n % 4 * 4 : (n - T - 1) % 8 * 2;
          const v16f& now = sc[odd][x];
          v2bf pair;
          if (n < T) {
            tops[0] = fmaxf(fmaxf(tops[0], now[r]), now[r + 1]);
            tops[1] = fmaxf(fmaxf(tops[1], now[r + 2]), now[r + 3]);
          } else if (n == T) {
            const float top = max_halves(fmaxf(tops[0], tops[1]));
            mx = (top - mx) * scale > 8.0f ? top : mx;
          } else if (n <= T + 8 * KT) {
            pair[0] = static_cast<__bf16>(__builtin_amdgcn_exp2f((now[r] - mx) * scale));
          }
          __builtin_amdgcn_sched_barrier(0);
          add_values(o[n % DT], vf[n % AHEAD], wt[1 - odd][n / (2 * DT)][n / DT % 2]);
          if (n + AHEAD < N) vf[n % AHEAD] = read_v(1 - odd, n + AHEAD);
          // loads among the products: in one go behind the barrier they would keep the waves from them while the
          // address unit takes them (the last blocks' keys once more where there are no further)
          if (n % 4 == 1)
            load_one(values, a.v, v_off, lds + (2 + odd) * L::TILE, n / 4);
          else if (n % 4 == 3)
            load_one(keys, a.k, k_off, lds + odd * L::TILE, n / 4);
          if (n == T) {
            alpha = __builtin_amdgcn_exp2f((old - mx) * scale);
            sums[0] = sum * alpha;
            sums[1] = 0.0f;
          } else if (n > T && n <= T + 8 * KT) {
            pair[1] = static_cast<__bf16>(__builtin_amdgcn_exp2f((now[r + 1] - mx) * scale));
            asm volatile("" : "+v"(pair));  // formed here, not behind the products
            sums[n & 1] = add_pair(pair, sums[n & 1]);
            wt[odd][x][r >> 3][r & 7] = pair[0];
            wt[odd][x][r >> 3][(r & 7) + 1] = pair[1];
          }
        }
        __builtin_amdgcn_sched_barrier(0);
        drain();  // copies of O that the compiler makes on its way out of here find it whole
        __builtin_amdgcn_sched_barrier(0);
        sum = sums[0] + sums[1];
        if (i > from && __any(mx != old)) {  // (before the first there is nothing)
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            settle(o[d]);
            o[d] *= alpha;
            settle(o[d]);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      };
      auto finish = [&](int odd) {  // the last block's values
        wait_vm0();
        lds_barrier();
        clean(to - 1, odd, last);
#pragma unroll
        for (int n = 0; n < N; ++n) add_last(o[n % DT], read_v(odd, n), wt[odd][n / (2 * DT)][n / DT % 2]);
        drain();
#pragma unroll
        for (int d = 0; d < DT; ++d) settle(o[d]);
      };
      int i = from;
      for (; i + 1 < to; i += 2) {
        step(i, 0);
        step(i + 1, 1);
      }
      if (i < to) {
        step(i, 0);
        finish(0);
      } else {
        finish(1);
      }
    } else {
      // here: block i's keys, then: block i + 1's, ids: the pages of block i + 2
      Where here = where(from, pages(from)), then = where(from + 1, pages(from + 1));
      int ids = pages(from + 2);
      load(here, a.k, k_off, lds);
      wait_vm0();
      bare_barrier();
      load(then, a.k, k_off, lds + L::TILE);  // the last block once more where there is none
      load(here, a.v, v_off, lds + 2 * L::TILE);
#pragma unroll
      for (int x = 0; x < KT; ++x) s[x] = 0.0f;
#pragma unroll
      for (int n = 0; n < N; ++n) s[n % KT] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(read_k(0, n), q[n / KT], s[n % KT], 0, 0, 0);
      // Block i, whose buffers are `odd`: its weights, then its second product beside the next one's scores
      // (of the last, what the buffer holds: they are not used).
      auto step = [&](int i, int odd) {
        weigh(i, here.none);
        wait_vm0();
        lds_barrier();
        const uint64_t none = here.none;
        here = then;
        then = where(i + 2, ids);
        ids = pages(i + 3);
        if (i + 2 < to) load(then, a.k, k_off, lds + odd * L::TILE);
        if (i + 1 < to) load(here, a.v, v_off, lds + (3 - odd) * L::TILE);
        clean(i, odd, none);
        products(1 - odd);
      };
      for (int i = from; i < to; i += 2) {
        step(i, 0);
        if (i + 1 >= to) break;
        step(i + 1, 1);
      }
      wait_vm0();
    }
  }

  sum = add_halves(sum);
  const bool whole = splits == 1;
  const float inv = !whole ? 1.0f : sum > 0.0f ? 1.0f / sum : 0.0f;
  // Out through the wave's quarter of LDS, so that stores are whole rows: registers 4 r .. 4 r + 3 of O^T are
  // elements d * 32 + 8 r + 4 half .. + 3 of the lane's row, which alone would be 16 bytes of 32 rows a store.
  bare_barrier();  // the buffers are free
  char* mem = smem + wave * L::TILE;
  auto leave = [&](auto* to, auto type) {
    typedef decltype(type) piece;                                   // four elements
    constexpr int ROWB = D / 4 * sizeof(piece), CH = ROWB / 16, TURN = CH < 16 ? CH - 1 : 15;
    static_assert(32 * ROWB <= L::TILE, "a quarter holds the wave's rows");
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int r = 0; r < 16; r += 4) {
        const v4f v = v4f{o[d][r], o[d][r + 1], o[d][r + 2], o[d][r + 3]} * inv;
        const int byte = (d * 8 + r / 2 + half) * static_cast<int>(sizeof(piece));
        *reinterpret_cast<piece*>(mem + l32 * ROWB + ((byte / 16) ^ (l32 & TURN)) * 16 + byte % 16) = __builtin_convertvector(v, piece);
      }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int j = 0; j < 32 * CH / 64; ++j) {
      const int r = (j * 64 + lane) / CH, c = lane % CH;
      const v4f v = *reinterpret_cast<const v4f*>(mem + r * ROWB + (c ^ (r & TURN)) * 16);
      const int64_t at = static_cast<int64_t>(__shfl(static_cast<int>(out_row), r)) * ROWB + c * 16;
      if (first_row + r < rows) *reinterpret_cast<v4f*>(reinterpret_cast<char*>(to) + at) = v;
    }
  };
  if (whole) {
    leave(a.out, v4bf());
    return;
  }
  const int64_t plane = static_cast<int64_t>(a.T) * a.n_q;
  leave(a.part + split * plane * D, v4f());
  if (half == 0 && first_row + l32 < rows) {
    float* ml = a.part + a.max_splits * plane * D + (split * plane + out_row) * 2;
    ml[0] = mx * scale;
    ml[1] = sum;
  }
}

// The splits of a row joined, eight splits a wave, so that one wait (2 us for sums that another XCD
// wrote) covers them all: a wave a row for up to eight splits (WAVES = 1; the calls with many rows),
// else a workgroup of four waves.  One wave for all splits, eight at a time, took 17 us for 64 of
// them, this 4; more than 32 splits were no faster (32768 keys: 34.9 us with 64, 34.1 with 32).
constexpr int kMostSplits = 32;

template <int D, int WAVES>
__global__ __launch_bounds__(256) void attention_join_kernel(AttnArgs a) {
  constexpr int PER = D / 64;
  typedef std::conditional_t<PER == 1, float, float __attribute__((ext_vector_type(PER == 1 ? 2 : PER)))> vec;
  __shared__ vec joined[4][64];
  const int lane = threadIdx.x & 63, wave_id = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wave = wave_id % WAVES;
  const int64_t rows = static_cast<int64_t>(a.T) * a.n_q, out_row = static_cast<int64_t>(blockIdx.x) * (4 / WAVES) + wave_id / WAVES;
  if (out_row >= rows) return;
  // lane s: maximum and sum of split s; and the sums of the wave's first splits: loaded before it is
  // known how many there are, which the lengths say (what was not written is not used)
  const float* ml = a.part + a.max_splits * rows * D + (min(lane, a.max_splits - 1) * rows + out_row) * 2;
  const float m_loaded = ml[0], l_loaded = ml[1];
  const float* part = a.part + out_row * D + lane * PER;
  vec v[8];
#pragma unroll
  for (int s = 0; s < 8; ++s) v[s] = wave * 8 + s < a.max_splits ? *reinterpret_cast<const vec*>(part + (wave * 8 + s) * rows * D) : vec(0.0f);
  Tile t;
  const int token = static_cast<int>(out_row / a.n_q), qh = static_cast<int>(out_row % a.n_q);
  if (!find_sequence(a, lane, &t, [&](int q0, int) { return q0 <= token; }) || token >= t.q0 + t.n) return;
  const int row = (token - t.q0) * a.group + qh % a.group;
  int splits;
  if (t.n * a.group <= a.small_rows) {
    t.row0 = row / kSmallRows * kSmallRows;
    splits = active_splits(a, find_blocks(a, t, kSmallRows, kSmallKeys).total);
  } else {
    t.row0 = row / a.large_rows * a.large_rows;
    splits = large_splits(a, find_blocks(a, t, a.large_rows, a.large_keys).total);
  }
  if (splits == 1) return;
  const float m = lane < splits ? m_loaded : kNoMax, l = lane < splits ? l_loaded : 0.0f;
  float top = m;
#pragma unroll
  for (int x = 1; x < 64; x *= 2) top = fmaxf(top, __shfl_xor(top, x));
  const float mine = __builtin_amdgcn_exp2f(m - top);
  float all = l * mine;
#pragma unroll
  for (int x = 1; x < 64; x *= 2) all += __shfl_xor(all, x);
  vec acc = 0.0f;
#pragma unroll
  for (int s = 0; s < 8; ++s)
    if (wave * 8 + s < splits) acc += v[s] * __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(mine), wave * 8 + s));
  if constexpr (WAVES > 1) {
    joined[wave][lane] = acc;
    __syncthreads();
    if (wave != 0) return;
    acc = joined[0][lane] + joined[1][lane] + joined[2][lane] + joined[3][lane];
  }
  acc *= all > 0.0f ? 1.0f / all : 0.0f;
  if constexpr (PER == 1) {
    *reinterpret_cast<__bf16*>(a.out + out_row * D + lane) = static_cast<__bf16>(acc);
  } else {
    typedef __bf16 bvec __attribute__((ext_vector_type(PER == 1 ? 2 : PER)));
    *reinterpret_cast<bvec*>(a.out + out_row * D + lane * PER) = __builtin_convertvector(acc, bvec);
  }
}

int64_t tiles_of(const AttnArgs& a, int rows) { return static_cast<int64_t>(a.T) * a.group / rows + a.B; }

// What a call launches.  The lengths are on the device: a call of few rows for its sequences
// runs the kernel for few rows alone, whatever the lengths; others run both, and each
// sequence's length says which one takes it.  What the sizes do not say costs time: keys
// are counted by the table's width, rows by all of T.  So a prompt under a wide table gets splits that
// do not pay (512 tokens 36 us, 19 under a table of 512), and single tokens beside a chunk get few splits
// (8 of 32768 keys and a chunk of 512 tokens 432 us, apart 198 and 68).
struct Plan {
  bool small, large;
  int small_rows, splits, large_splits, max_splits;
};

Plan make_plan(int64_t T, int64_t B, int group, int n_kv, int D, int64_t table_keys, int window, int sinks, const DeviceInfo& dev) {
  Plan p = {};
  // Keys of a tile, at most: whole blocks of what its tokens (rows / group and one more) see.
  auto reach = [&](int rows, int size) {
    const int64_t keys = window == 0 ? table_keys : std::min<int64_t>(table_keys, static_cast<int64_t>(window) + sinks + rows / group + 1 + 2 * size);
    return (keys + size - 1) / size * size;
  };
  const int64_t keys = reach(kSmallRows, kSmallKeys);
  // Few rows: workgroups that share a tile's keys, enough to fill the device (several times over, for lengths
  // that differ: 24 tokens of up to 16384 keys of 256 took 227 us with one workgroup a CU, 203 with two, 188 with
  // four, 199 with eight) and none of less than kSplitBlocks blocks of what the table can hold.
  // Where more than 16 query heads share a key head, a token has several tiles (9 tokens of 512 heads on one of 128, 9000
  // keys: 48 us, 155 where one was counted; 24 of 128 heads, 8192 keys 51 and 101).
  const int64_t wide = (group + kSmallRows - 1) / kSmallRows;
  const int64_t tiles = std::max<int64_t>(1, std::min(T * wide, T * group / kSmallRows + std::min(B, T))) * n_kv;
  const int64_t most = std::min<int64_t>(std::max<int64_t>(1, keys / kSmallKeys / kSplitBlocks),
                                         std::min<int64_t>(kMostSplits, (1 << 23) / (B * n_kv)));  // the grid stays below 2^24 workgroups
  p.splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(most, (D == 64 ? 12 : D == 128 ? 8 : 4) * dev.cu_count / tiles)));
  // Many rows: where the tiles leave workgroups' places free (two a CU, one for D = 256), splits, if what
  // they save (a block of keys takes 1.7 us where few workgroups run) is more than the second
  // kernel and the sums' way through memory (4 TB/s).  us with the splits chosen and without: 512 of 16384 keys
  // 185 and 333, 200 of 4000 43 and 91, 2 x 2430 tokens of 2 heads of 64 36 and 45; 512 tokens of 40 heads 19 without, 35 with 3.
  const int64_t large_tiles = std::max<int64_t>(1, T * group * n_kv / 128), places = (D < 256 ? 2 : 1) * dev.cu_count;
  const int64_t blocks = reach(128, 64) / 64;
  float large_us = 0.0f;
  for (int64_t n = 1; n == 1 || (n <= std::min<int64_t>(kMostSplits, blocks / kLargeSplitBlocks) && n * large_tiles <= places); ++n) {
    float us = 1.7f * static_cast<float>((blocks + n - 1) / n) * static_cast<float>((n * large_tiles + places - 1) / places);
    if (n > 1) us += 4.0f + static_cast<float>(n * T) * static_cast<float>(n_kv * group * (D + 2)) * 8.0f / 4e6f;
    if (n > 1 && us >= large_us) continue;
    large_us = us;
    p.large_splits = static_cast<int>(n);
  }
  // Which of the two: the kernel for few rows reads a tile's keys for 16 rows instead of 128 (25000 keys a us
  // for all tiles of D = 128), but has its keys shared by four waves and needs no second launch in a batch.
  // us, few and many: 2 x 28 tokens of 56 keys of 256 8 and 20, 10 x 111 of 223 10 and 18; 200 tokens of 4000
  // keys 87 and 43, 512 causal tokens 26 and 19.  A round of workgroups that waits for places (four a CU, two, one by D) adds 4 us.
  const float small_us = std::max(static_cast<float>(tiles * keys) * static_cast<float>(D) / 128.0f / 25000.0f, static_cast<float>(keys) * 0.01f / static_cast<float>(p.splits)) +
                         (p.splits > 1 ? 4.0f : 0.0f) + 4.0f * static_cast<float>(tiles * p.splits / ((D == 64 ? 4 : D == 128 ? 2 : 1) * dev.cu_count));
  const bool few = T * group <= kSmallMost * B || small_us < large_us + (B > 1 ? 4.0f : 0.0f);
  p.small = few || B > 1;
  p.large = !few;
  p.small_rows = few ? kAllRows : B == 1 ? 0 : kSmallMost;
  if (!p.small) p.splits = 1;
  if (!p.large) p.large_splits = 1;
  p.max_splits = std::max(p.splits, p.large_splits);
  return p;
}

template <int D>
hipError_t launch_d(AttnArgs a, const Plan& p, hipStream_t stream) {
  using L = Large<D>;
  a.large_rows = L::ROWS;
  a.large_keys = L::KEYS;
  if (p.large) {
    attention_large_kernel<D><<<static_cast<uint32_t>(tiles_of(a, L::ROWS)) * a.n_kv * a.large_splits, 64 * L::WAVES, 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (p.small) {
    // beside the other kernel, tiles by sequence: those of all rows, nearly all without work, took 7 us of
    // five chunks' 107
    const uint32_t tiles = static_cast<uint32_t>(p.large ? static_cast<int64_t>(a.B) * kShortTiles : tiles_of(a, kSmallRows)) * a.n_kv;
    attention_small_kernel<D><<<tiles * a.splits, 256, 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.max_splits == 1) return hipSuccess;
  const uint32_t rows = static_cast<uint32_t>(a.T) * a.n_q;
  if (a.max_splits <= 8)
    attention_join_kernel<D, 1><<<(rows + 3) / 4, 256, 0, stream>>>(a);
  else
    attention_join_kernel<D, 4><<<rows, 256, 0, stream>>>(a);
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
