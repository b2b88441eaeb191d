// qk_norm_rope: RMSNorm of every query and key head of a fused projection's output,
// the position rotation, queries to a dense tensor, keys and values to the pages of
// a cache (include/twl.h).
//
//   n = x / sqrt(mean(x^2) + eps) w                    per head of D elements, fp32
//   (a, b) -> (a c - b s, b c + a s)                   pairs of the first `rot` elements
//
// A head's D <= 256 squares are summed in fp32 (relative error below 2^-20, against
// the 2^-9 of the one rounding to bf16 at the end).
//
// Split: a wave takes 512 elements of a token's row at a time, 8 a lane, so that a head
// is D / 8 adjacent lanes and a lane keeps its place in the head: weights, cosines and sines
// are loaded once for all of a wave's P pieces, whose own loads go out first.
// The partner of a pair lies rot / 16 lanes away (or in the lane itself where pairs are
// adjacent).  Every access is 16 bytes a lane; heads of the cache are whole runs of
// 2 D bytes.
//
// Bound by memory where there are many tokens: 8192 of 40 + 8 + 8 heads of 128, 239 MB, 52 us, 4.6 TB/s, where
// a copy reaches 5.1; few tokens take 2.8 to 3.5 us, one trip to memory behind another (positions, then angles).
// Before that, 105 us with one piece a wave whose loads waited for its position, sums through LDS
// exchanges and a divide and square root written out: now loads first, sums by lane moves, the native
// reciprocal root (1 ulp, against the 2^-9 of the rounding).
#include "attention_internal.h"

namespace twl {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v8f __attribute__((ext_vector_type(8)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, false));
}

// Sum over L adjacent lanes (8, 16 or 32), in each of them: within quads, between quads by
// mirrors of 8 and 16 lanes, between rows of 16 by an exchange.
template <int L>
__device__ __forceinline__ float sum_lanes(float v) {
  v += dpp<0xB1>(v);   // lane ^ 1
  v += dpp<0x4E>(v);   // lane ^ 2
  v += dpp<0x141>(v);  // 7 - lane of 8
  if (L >= 16) v += dpp<0x140>(v);  // 15 - lane of 16
  if (L >= 32) v += __shfl_xor(v, 16);
  return v;
}

template <int D, bool F32, int P>
__global__ __launch_bounds__(256) void qk_rope_kernel(RopeArgs a) {
  constexpr int L = D / 8;          // lanes of a head
  constexpr int HEADS = 512 / D;    // heads of a piece
  const int lane = threadIdx.x & 63;
  const uint32_t item = __builtin_amdgcn_readfirstlane(blockIdx.x * 4u + (threadIdx.x >> 6));
  const uint32_t token = item / a.parts, part = item % a.parts;
  if (token >= a.M) return;
  const int li = lane % L, d0 = li * 8;
  const int heads = a.n_q + 2 * a.n_kv, first = static_cast<int>(part) * (P * HEADS) + lane / L;
  // the rows' pieces: bf16 as they lie, fp32 in two halves
  v8bf raw[F32 ? 1 : P];
  v8f x[P];
  const int64_t row = static_cast<int64_t>(token) * a.stride + d0;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int head = min(first + i * HEADS, heads - 1);
    if (F32)
      x[i] = *reinterpret_cast<const v8f*>(static_cast<const float*>(a.qkv) + row + head * D);
    else
      raw[F32 ? 0 : i] = *reinterpret_cast<const v8bf*>(static_cast<const uint16_t*>(a.qkv) + row + head * D);
  }
  int pos = 0;
  if (a.rot > 0) {
    pos = a.positions[token];
    if (pos < 0 || pos >= a.n_pos) return;  // padding: nothing of this token is written
  }
  const int64_t slot = a.slots != nullptr ? a.slots[token] : static_cast<int64_t>(token);
  const bool keep = slot >= 0 && slot < a.n_slots;

  v8f wq = 1.0f, wk = 1.0f;
  if (a.q_weight != nullptr) wq = __builtin_convertvector(*reinterpret_cast<const v8bf*>(a.q_weight + d0), v8f);
  if (a.k_weight != nullptr) wk = __builtin_convertvector(*reinterpret_cast<const v8bf*>(a.k_weight + d0), v8f);
  // the lane's eight cosines and sines; identity outside the rotated part
  v8f c = 1.0f, s = 0.0f;
  const int half = a.rot / 2;
  const bool turns = d0 < a.rot;
  int partner = lane;
  if (turns) {
    const float* angles = a.cos_sin + static_cast<int64_t>(pos) * a.rot;
    if (a.interleaved) {
      const v4f c4 = *reinterpret_cast<const v4f*>(angles + d0 / 2), s4 = *reinterpret_cast<const v4f*>(angles + half + d0 / 2);
      c = __builtin_shufflevector(c4, c4, 0, 0, 1, 1, 2, 2, 3, 3);
      s = __builtin_shufflevector(s4, s4, 0, 0, 1, 1, 2, 2, 3, 3);
#pragma unroll
      for (int i = 0; i < 8; i += 2) s[i] = -s[i];
    } else {
      const bool low = d0 < half;
      const int at = low ? d0 : d0 - half;
      c = *reinterpret_cast<const v8f*>(angles + at);
      s = *reinterpret_cast<const v8f*>(angles + half + at);
      if (low) s = -s;
      partner = low ? lane + half / 8 : lane - half / 8;
    }
  }
  const int64_t page = slot >> a.page_shift, off = slot & ((1 << a.page_shift) - 1);
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int head = first + i * HEADS;
    if (!F32) x[i] = __builtin_convertvector(raw[F32 ? 0 : i], v8f);
    const bool is_q = head < a.n_q, is_v = head >= a.n_q + a.n_kv;
    float sum = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(x[i][e], x[i][e], sum);
    const float r = __builtin_amdgcn_rsqf(sum_lanes<L>(sum) * (1.0f / D) + a.eps);
    const bool norm = is_q ? a.q_weight != nullptr : a.k_weight != nullptr;
    v8f n = x[i];
    if (norm) n = x[i] * r * (is_q ? wq : wk);
    v8f other;
    if (a.interleaved) {
      other = __builtin_shufflevector(n, n, 1, 0, 3, 2, 5, 4, 7, 6);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) other[e] = __shfl(n[e], partner);
    }
    v8f y;
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = __builtin_fmaf(n[e], c[e], other[e] * s[e]);
    if (!turns) y = n;
    if (is_v) y = x[i];
    const v8bf out = __builtin_convertvector(y, v8bf);
    if (head >= heads) continue;
    if (is_q) {
      *reinterpret_cast<v8bf*>(a.q + (static_cast<int64_t>(token) * a.n_q + head) * D + d0) = out;
    } else if (keep) {
      const int h = is_v ? head - a.n_q - a.n_kv : head - a.n_q;
      const int64_t at = (((page * a.n_kv + h) << a.page_shift) + off) * D + d0;
      *reinterpret_cast<v8bf*>((is_v ? a.v_cache : a.k_cache) + at) = out;
    }
  }
}

template <int D, int P>
hipError_t launch_p(RopeArgs a, bool f32, hipStream_t stream) {
  const int64_t pieces = ((a.n_q + 2 * a.n_kv) * static_cast<int64_t>(D) + 511) / 512;
  a.parts = static_cast<uint32_t>((pieces + P - 1) / P);
  const uint32_t blocks = static_cast<uint32_t>((static_cast<int64_t>(a.M) * a.parts + 3) / 4);
  if (f32)
    qk_rope_kernel<D, true, P><<<blocks, 256, 0, stream>>>(a);
  else
    qk_rope_kernel<D, false, P><<<blocks, 256, 0, stream>>>(a);
  return hipGetLastError();
}

// Few tokens spread their pieces over waves; where there are more than the device holds at once, two
// pieces a wave share the token's loads (8192 tokens of 40 + 8 + 8 heads of 128, us: one piece 64.6, two 55.0,
// four 56.5, eight 56.1; 1000 tokens 11.2 to 11.4 with any).
template <int D>
hipError_t launch_d(const RopeArgs& a, bool f32, const DeviceInfo& dev, hipStream_t stream) {
  const int64_t pieces = ((a.n_q + 2 * a.n_kv) * static_cast<int64_t>(D) + 511) / 512;
  if (a.M * pieces >= 16 * 4 * static_cast<int64_t>(dev.cu_count)) return launch_p<D, 2>(a, f32, stream);
  return launch_p<D, 1>(a, f32, stream);
}

}  // namespace

hipError_t launch_qk_rope(RopeArgs a, int D, bool f32, const DeviceInfo& dev, hipStream_t stream) {
  if (D == 64) return launch_d<64>(a, f32, dev, stream);
  if (D == 128) return launch_d<128>(a, f32, dev, stream);
  return launch_d<256>(a, f32, dev, stream);
}

}  // namespace twl
