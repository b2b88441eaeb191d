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
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v4bf __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));

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
  if (!find_tile(a, blockIdx.x / a.n_kv / a.splits, kSmallRows, lane, &t)) return;
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
    float* ml = a.part + static_cast<int64_t>(a.splits) * a.T * a.n_q * D + (static_cast<int64_t>(split) * a.T * a.n_q + out_row) * 2;
    ml[0] = top;
    ml[1] = all;
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
  const int splits = active_splits(a, find_blocks(a, t, kSmallRows, kSmallKeys).total);
  const int row = t.row0 + quarter * 4 + wave;
  if (splits == 1 || row >= t.n * a.group) return;
  const int64_t rows = static_cast<int64_t>(a.T) * a.n_q;
  const int64_t out_row = static_cast<int64_t>(t.q0 + row / a.group) * a.n_q + head * a.group + row % a.group;
  const float* ml = a.part + a.splits * rows * D + out_row * 2;
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

// Workgroups that share a tile's keys: enough to fill the device where there are few
// tiles, and none of less than kSplitBlocks blocks of what the table can hold.
int plan_splits(int64_t T, int64_t B, int group, int n_kv, int64_t table_keys, int window, int sinks, const DeviceInfo& dev) {
  const int64_t tiles = std::max<int64_t>(1, std::min(T, T * group / kSmallRows + std::min(B, T))) * n_kv;
  int64_t keys = table_keys;
  if (window > 0) keys = std::min<int64_t>(keys, static_cast<int64_t>(window) + sinks + kSmallRows + 2 * kSmallKeys);
  const int64_t most = std::max<int64_t>(1, (keys + kSmallKeys - 1) / kSmallKeys / kSplitBlocks);
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(most, 32), 2 * dev.cu_count / tiles)));
}

template <int D>
hipError_t launch_small(const AttnArgs& a, hipStream_t stream) {
  const uint32_t tiles = static_cast<uint32_t>(tiles_of(a, kSmallRows)) * a.n_kv;
  attention_small_kernel<D><<<tiles * a.splits, 256, 0, stream>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  attention_join_kernel<D><<<tiles * 4, 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

size_t attention_workspace_bytes(int64_t T, int64_t B, int n_q, int n_kv, int D, int64_t table_keys, int window, int sinks,
                                 const DeviceInfo& dev) {
  const int splits = plan_splits(T, B, n_q / n_kv, n_kv, table_keys, window, sinks, dev);
  return splits == 1 ? 0 : static_cast<size_t>(splits) * T * n_q * (D + 2) * sizeof(float);
}

hipError_t launch_attention(AttnArgs a, int D, const DeviceInfo& dev, hipStream_t stream) {
  a.group = a.n_q / a.n_kv;
  a.splits = plan_splits(a.T, a.B, a.group, a.n_kv, static_cast<int64_t>(a.table_pages) << a.page_shift, a.window, a.sinks, dev);
  if (D == 64) return launch_small<64>(a, stream);
  if (D == 128) return launch_small<128>(a, stream);
  return launch_small<256>(a, stream);
}

}  // namespace twl
