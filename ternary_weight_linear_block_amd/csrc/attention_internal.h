// Internal launchers of the attention half of a block (api_attention.cpp validates
// first, as api.cpp does for twl_internal.h's).
#pragma once

#include "twl_internal.h"

namespace twl {

// int8_linear (include/twl.h): out [M, N] of `kind` (kOutF32, kOutBf16, kOutAcc).
struct Int8Args {
  const int8_t* x;
  const float* a_scale;
  const int8_t* w;
  const float* w_scale;
  const float* bias;  // or null
  void* out;
  int32_t* part;      // holds int8_workspace_bytes
  int M, N, K;
  int kind;
  int tiles_m, tiles_n, splits;  // set by the launcher
};
size_t int8_workspace_bytes(int64_t M, int64_t N, int64_t K, const DeviceInfo& dev);
hipError_t launch_int8(Int8Args a, const DeviceInfo& dev, hipStream_t stream);

// qk_norm_rope (include/twl.h).  stride: elements between the rows of qkv.
struct RopeArgs {
  const void* qkv;
  const uint16_t* q_weight;  // or null
  const uint16_t* k_weight;  // or null
  const float* cos_sin;
  const int32_t* positions;
  const int32_t* slots;      // or null: token t goes to slot t
  uint16_t* q;
  uint16_t* k_cache;
  uint16_t* v_cache;
  int64_t stride, n_slots;
  float eps;
  uint32_t M, parts;         // parts: waves that share a token (set by the launcher)
  int n_q, n_kv, rot, n_pos, page_shift, interleaved;
};
hipError_t launch_qk_rope(RopeArgs a, int D, bool f32, const DeviceInfo& dev, hipStream_t stream);

// window_attention (include/twl.h).  The caller sets everything up to sinks.
struct AttnArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  const int32_t* page_table;
  const int32_t* q_start;
  const int32_t* kv_len;
  uint16_t* out;
  float* part;               // holds attention_workspace_bytes
  float scale_log2;          // scale * log2(e)
  int T, B, n_q, n_kv, page_shift, n_pages, table_pages, window, sinks;
  int group, splits, large_splits, max_splits;  // set by the launcher, as what follows
  int small_rows, large_rows, large_keys;
};
size_t attention_workspace_bytes(int64_t T, int64_t B, int n_q, int n_kv, int D, int64_t table_keys, int window, int sinks,
                                 const DeviceInfo& dev);
hipError_t launch_attention(AttnArgs a, int D, const DeviceInfo& dev, hipStream_t stream);

}  // namespace twl
