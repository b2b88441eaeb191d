// C ABI of the attention half of a block (include/twl.h): argument validation and
// launches.  The same rules as api.cpp: nothing is allocated, nothing synchronises,
// every kernel goes to the caller's stream.
#include "api_common.h"
#include "attention_internal.h"

#include <cfloat>
#include <cmath>

namespace {

using namespace twl::api;

twl_status check_int8(int64_t M, int64_t N, int64_t K) {
  TWL_TRY(check_rows("M", M));
  TWL_TRY(check_rows("N", N));
  if (K <= 0 || K % 16 != 0 || K > TWL_MAX_K)
    return fail(TWL_ESHAPE, "K=%lld must be a positive multiple of 16 of at most %d", static_cast<long long>(K), TWL_MAX_K);
  if (M > TWL_INT8_MAX_ROWS || N > TWL_INT8_MAX_ROWS || M * N > TWL_INT8_MAX_OUT)
    return fail(TWL_ESHAPE, "M=%lld, N=%lld: at most 2^24 each and 2^33 together", static_cast<long long>(M), static_cast<long long>(N));
  return TWL_OK;
}

twl_status check_heads(int64_t n_q, int64_t n_kv, int64_t D) {
  if (D != 64 && D != 128 && D != 256) return fail(TWL_ESHAPE, "head size %lld is not 64, 128 or 256", static_cast<long long>(D));
  if (n_kv < 1 || n_q < n_kv || n_q % n_kv != 0 || n_q > TWL_MAX_HEADS)
    return fail(TWL_ESHAPE, "n_q=%lld must be a multiple of n_kv=%lld of at most %d", static_cast<long long>(n_q),
                static_cast<long long>(n_kv), TWL_MAX_HEADS);
  return TWL_OK;
}

// log2 of a page size that is a power of two from `least` to 1024, or -1.
int page_shift(int64_t page, int64_t least) {
  if (page < least || page > 1024 || (page & (page - 1)) != 0) return -1;
  return __builtin_ctzll(static_cast<unsigned long long>(page));
}

twl_status check_pages(int64_t n_pages, int64_t page, int64_t least) {
  TWL_TRY(check_rows("n_pages", n_pages));
  if (page_shift(page, least) < 0)
    return fail(TWL_ESHAPE, "page size %lld is not a power of two from %lld to 1024", static_cast<long long>(page),
                static_cast<long long>(least));
  if (n_pages * page > (int64_t{1} << 31) - 1)  // slots are int32
    return fail(TWL_ESHAPE, "%lld pages of %lld tokens: at most 2^31 - 1 slots", static_cast<long long>(n_pages),
                static_cast<long long>(page));
  return TWL_OK;
}

twl_status check_attention(int64_t T, int64_t B, int64_t n_q, int64_t n_kv, int64_t D, int64_t page, int64_t table_pages,
                           int64_t window, int64_t sinks) {
  TWL_TRY(check_rows("T", T));
  TWL_TRY(check_rows("B", B));
  TWL_TRY(check_rows("table_pages", table_pages));
  TWL_TRY(check_heads(n_q, n_kv, D));
  TWL_TRY(check_pages(0, page, 16));
  TWL_TRY(check_rows("window", window));
  TWL_TRY(check_rows("sinks", sinks));
  if (T * n_q > (int64_t{1} << 27) || B > TWL_MAX_SEQUENCES || B * n_kv > (int64_t{1} << 22))
    return fail(TWL_ESHAPE, "T=%lld, B=%lld: at most 2^27 rows T n_q, %d sequences and 2^22 of B n_kv", static_cast<long long>(T),
                static_cast<long long>(B), TWL_MAX_SEQUENCES);
  if (table_pages * page > (int64_t{1} << 30))
    return fail(TWL_ESHAPE, "table_pages=%lld of %lld tokens: at most 2^30 tokens", static_cast<long long>(table_pages),
                static_cast<long long>(page));
  return TWL_OK;
}

}  // namespace

extern "C" {

size_t twl_int8_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  twl::DeviceInfo dev;
  if (check_int8(M, N, K) != TWL_OK || current_device(&dev) != TWL_OK) return 0;
  ok();
  return M == 0 || N == 0 ? 0 : twl::int8_workspace_bytes(M, N, K, dev);
}

twl_status twl_int8_linear(const int8_t* x_i8, const float* a_scale, const int8_t* w_i8, const float* w_scale,
                           const float* bias, int64_t M, int64_t N, int64_t K, void* out, int out_kind, void* workspace,
                           size_t workspace_bytes, hipStream_t stream) {
  TWL_TRY(check_int8(M, N, K));
  if (out_kind != TWL_OUT_F32 && out_kind != TWL_OUT_BF16 && out_kind != TWL_OUT_ACC_I32)
    return fail(TWL_EINVAL, "output kind %d is not fp32, bf16 or int32", out_kind);
  const bool scaled = out_kind != TWL_OUT_ACC_I32;
  if (!scaled && bias != nullptr) return fail(TWL_EINVAL, "the int32 sums take no bias");
  if (M == 0 || N == 0) return ok();
  TWL_REQUIRE_PTR(x_i8);
  TWL_REQUIRE_PTR(w_i8);
  TWL_REQUIRE_PTR(out);
  if (scaled) {
    TWL_REQUIRE_PTR(a_scale);
    TWL_REQUIRE_PTR(w_scale);
    TWL_OPTIONAL_PTR(bias);
  }
  const size_t m = static_cast<size_t>(M), n = static_cast<size_t>(N), k = static_cast<size_t>(K);
  const Range in[] = {{x_i8, m * k, "x_i8"}, {a_scale, scaled ? m * 4 : 0, "a_scale"}, {w_i8, n * k, "w_i8"},
                      {w_scale, scaled ? n * 4 : 0, "w_scale"}, {bias, n * 4, "bias"},
                      {out, m * n * (out_kind == TWL_OUT_BF16 ? 2 : 4), "out"}};
  for (int i = 0; i < 5; ++i)
    if (overlap(in[5], in[i])) return fail(TWL_EINVAL, "out overlaps %s", in[i].name);
  twl::DeviceInfo dev;
  TWL_TRY(current_device(&dev));
  const size_t need = twl::int8_workspace_bytes(M, N, K, dev);
  TWL_TRY(check_workspace(need, workspace, workspace_bytes));
  const Range scratch = {need > 0 ? workspace : nullptr, need, "workspace"};
  for (const Range& i : in)
    if (overlap(scratch, i)) return fail(TWL_EINVAL, "workspace overlaps %s", i.name);
  twl::Int8Args a = {};
  a.x = x_i8;
  a.a_scale = a_scale;
  a.w = w_i8;
  a.w_scale = w_scale;
  a.bias = bias;
  a.out = out;
  a.part = static_cast<int32_t*>(workspace);
  a.M = static_cast<int>(M);
  a.N = static_cast<int>(N);
  a.K = static_cast<int>(K);
  a.kind = out_kind == TWL_OUT_F32 ? twl::kOutF32 : out_kind == TWL_OUT_BF16 ? twl::kOutBf16 : twl::kOutAcc;
  return launched(twl::launch_int8(a, dev, stream), "int8_linear");
}

twl_status twl_qk_norm_rope(const void* qkv, int kind, int64_t row_stride, const uint16_t* q_weight,
                            const uint16_t* k_weight, double eps, const float* cos_sin, int64_t n_pos, int64_t rot,
                            int interleaved, const int32_t* positions, const int32_t* slots, int64_t M, int64_t n_q,
                            int64_t n_kv, int64_t D, uint16_t* q, uint16_t* k_cache, uint16_t* v_cache, int64_t n_pages,
                            int64_t page, hipStream_t stream) {
  TWL_TRY(check_rows("M", M));
  TWL_TRY(check_heads(n_q, n_kv, D));
  TWL_TRY(check_pages(n_pages, page, 1));
  const int64_t width = (n_q + 2 * n_kv) * D;
  if (kind != TWL_OUT_F32 && kind != TWL_OUT_BF16) return fail(TWL_EINVAL, "kind %d is not fp32 or bf16", kind);
  if (row_stride < width || row_stride % 8 != 0 || row_stride > (int64_t{1} << 30))
    return fail(TWL_ESHAPE, "row_stride=%lld must be a multiple of 8 from %lld to 2^30", static_cast<long long>(row_stride),
                static_cast<long long>(width));
  if (!(static_cast<float>(eps) >= FLT_MIN) || !std::isfinite(static_cast<float>(eps)))
    return fail(TWL_EINVAL, "eps=%g must be at least 2^-126 and finite as fp32", eps);
  if (rot < 0 || rot > D || rot % 16 != 0)
    return fail(TWL_ESHAPE, "rot=%lld must be a multiple of 16 of at most %lld", static_cast<long long>(rot), static_cast<long long>(D));
  TWL_TRY(check_rows("n_pos", n_pos));
  if (interleaved != 0 && interleaved != 1) return fail(TWL_EINVAL, "interleaved=%d is not 0 or 1", interleaved);
  if (M > (int64_t{1} << 26) / (width / 512 + 1)) return fail(TWL_ESHAPE, "M=%lld is too large", static_cast<long long>(M));
  if (M == 0) return ok();
  TWL_REQUIRE_PTR(qkv);
  TWL_REQUIRE_PTR(q);
  TWL_REQUIRE_PTR(k_cache);
  TWL_REQUIRE_PTR(v_cache);
  TWL_OPTIONAL_PTR(q_weight);
  TWL_OPTIONAL_PTR(k_weight);
  TWL_OPTIONAL_PTR(slots);
  if (rot > 0) {
    TWL_REQUIRE_PTR(cos_sin);
    TWL_REQUIRE_PTR(positions);
  }
  const size_t m = static_cast<size_t>(M), d = static_cast<size_t>(D);
  const size_t cache = static_cast<size_t>(n_pages) * page * n_kv * d * 2;
  const Range out[] = {{q, m * n_q * d * 2, "q"}, {k_cache, cache, "k_cache"}, {v_cache, cache, "v_cache"}};
  const Range in[] = {{qkv, ((m - 1) * row_stride + width) * (kind == TWL_OUT_F32 ? 4 : 2), "qkv"},
                      {q_weight, d * 2, "q_weight"}, {k_weight, d * 2, "k_weight"},
                      {rot > 0 ? cos_sin : nullptr, static_cast<size_t>(n_pos) * rot * 4, "cos_sin"},
                      {rot > 0 ? positions : nullptr, m * 4, "positions"}, {slots, m * 4, "slots"}};
  for (int i = 0; i < 3; ++i) {
    for (const Range& j : in)
      if (overlap(out[i], j)) return fail(TWL_EINVAL, "%s overlaps %s", out[i].name, j.name);
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return fail(TWL_EINVAL, "%s overlaps %s", out[i].name, out[j].name);
  }
  twl::DeviceInfo dev;
  TWL_TRY(current_device(&dev));
  twl::RopeArgs a = {};
  a.qkv = qkv;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.cos_sin = cos_sin;
  a.positions = positions;
  a.slots = slots;
  a.q = q;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.stride = row_stride;
  a.n_slots = n_pages * page;
  a.eps = static_cast<float>(eps);
  a.M = static_cast<uint32_t>(M);
  a.n_q = static_cast<int>(n_q);
  a.n_kv = static_cast<int>(n_kv);
  a.rot = static_cast<int>(rot);
  a.n_pos = static_cast<int>(n_pos);
  a.page_shift = page_shift(page, 1);
  a.interleaved = interleaved;
  return launched(twl::launch_qk_rope(a, static_cast<int>(D), kind == TWL_OUT_F32, dev, stream), "qk_norm_rope");
}

size_t twl_attention_workspace_bytes(int64_t T, int64_t B, int64_t n_q, int64_t n_kv, int64_t D, int64_t page,
                                     int64_t table_pages, int64_t window, int64_t sinks) {
  twl::DeviceInfo dev;
  if (check_attention(T, B, n_q, n_kv, D, page, table_pages, window, sinks) != TWL_OK || current_device(&dev) != TWL_OK) return 0;
  ok();
  if (T == 0 || B == 0) return 0;
  return twl::attention_workspace_bytes(T, B, static_cast<int>(n_q), static_cast<int>(n_kv), static_cast<int>(D), table_pages * page,
                                        static_cast<int>(window), static_cast<int>(sinks), dev);
}

twl_status twl_window_attention(const uint16_t* q, const uint16_t* k_cache, const uint16_t* v_cache, const int32_t* page_table,
                                const int32_t* q_start, const int32_t* kv_len, double scale, int64_t window, int64_t sinks,
                                int64_t T, int64_t B, int64_t n_q, int64_t n_kv, int64_t D, int64_t n_pages, int64_t page,
                                int64_t table_pages, uint16_t* out, void* workspace, size_t workspace_bytes,
                                hipStream_t stream) {
  TWL_TRY(check_attention(T, B, n_q, n_kv, D, page, table_pages, window, sinks));
  TWL_TRY(check_pages(n_pages, page, 16));
  if (!std::isfinite(scale) || !std::isfinite(static_cast<float>(scale * 1.4426950408889634)))
    return fail(TWL_EINVAL, "scale=%g must be finite", scale);
  if (T == 0 || B == 0) return ok();
  TWL_REQUIRE_PTR(q);
  TWL_REQUIRE_PTR(q_start);
  TWL_REQUIRE_PTR(kv_len);
  TWL_REQUIRE_PTR(out);
  const bool keys = n_pages > 0 && table_pages > 0;
  if (keys) {
    TWL_REQUIRE_PTR(k_cache);
    TWL_REQUIRE_PTR(v_cache);
    TWL_REQUIRE_PTR(page_table);
  }
  twl::DeviceInfo dev;
  TWL_TRY(current_device(&dev));
  const size_t need = twl::attention_workspace_bytes(T, B, static_cast<int>(n_q), static_cast<int>(n_kv), static_cast<int>(D),
                                                     table_pages * page, static_cast<int>(window), static_cast<int>(sinks), dev);
  TWL_TRY(check_workspace(need, workspace, workspace_bytes));
  const size_t rows = static_cast<size_t>(T) * n_q * D * 2, cache = static_cast<size_t>(n_pages) * page * n_kv * D * 2;
  const Range outs[] = {{out, rows, "out"}, {need > 0 ? workspace : nullptr, need, "workspace"}};
  const Range in[] = {{q, rows, "q"}, {k_cache, cache, "k_cache"}, {v_cache, cache, "v_cache"},
                      {page_table, static_cast<size_t>(B) * table_pages * 4, "page_table"},
                      {q_start, (static_cast<size_t>(B) + 1) * 4, "q_start"}, {kv_len, static_cast<size_t>(B) * 4, "kv_len"}};
  for (const Range& o : outs)
    for (const Range& i : in)
      if (overlap(o, i)) return fail(TWL_EINVAL, "%s overlaps %s", o.name, i.name);
  if (overlap(outs[0], outs[1])) return fail(TWL_EINVAL, "out overlaps workspace");
  twl::AttnArgs a = {};
  a.q = q;
  a.k = k_cache;
  a.v = v_cache;
  a.page_table = page_table;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.out = out;
  a.part = static_cast<float*>(workspace);
  a.scale_log2 = static_cast<float>(scale * 1.4426950408889634);
  a.T = static_cast<int>(T);
  a.B = static_cast<int>(B);
  a.n_q = static_cast<int>(n_q);
  a.n_kv = static_cast<int>(n_kv);
  a.page_shift = page_shift(page, 16);
  a.n_pages = keys ? static_cast<int>(n_pages) : 0;
  a.table_pages = static_cast<int>(table_pages);
  a.window = static_cast<int>(window);
  a.sinks = static_cast<int>(sinks);
  return launched(twl::launch_attention(a, static_cast<int>(D), dev, stream), "window_attention");
}

}  // extern "C"
