// The C ABI of the serving operators: argument validation and dispatch.  Every
// check runs on the host before any work is enqueued.
#include <cfloat>
#include <cmath>

#include "sa_internal.cuh"

using namespace sa;

namespace {

constexpr int64_t kInt32 = INT32_MAX;

bool aligned(const void* p, uintptr_t n) { return (uintptr_t)p % n == 0; }

sa_status check_window(int64_t window, int64_t sinks, float scale) {
  if (window < 0 || sinks < 0) return set_error(SA_ERR_INVALID_ARG, "window and sinks must be non-negative");
  if (window > kInt32 || sinks > kInt32) return set_error(SA_ERR_UNSUPPORTED, "window and sinks must fit 31 bits");
  if (!(scale >= 0.f) || std::isinf(scale)) return set_error(SA_ERR_INVALID_ARG, "scale must be finite and >= 0");
  return SA_OK;
}

sa_status check_window_shape(const sa_window_shape* s) {
  if (!s) return set_error(SA_ERR_INVALID_ARG, "shape is NULL");
  if (s->B <= 0 || s->Hq <= 0 || s->Hkv <= 0 || s->Nq <= 0 || s->Nk <= 0 || s->d <= 0)
    return set_error(SA_ERR_INVALID_ARG, "shape sizes must be positive");
  if (s->Hq % s->Hkv != 0) return set_error(SA_ERR_INVALID_ARG, "Hq must be a multiple of Hkv");
  if (s->dtype != SA_BF16 && s->dtype != SA_FP32) return set_error(SA_ERR_INVALID_ARG, "unknown dtype");
  if (s->Nq > kInt32 / 2 || s->Nk > kInt32 / 2 || s->B > kInt32 / 2 || s->Hq > 65535 || s->Nq * s->Hq > kInt32)
    return set_error(SA_ERR_UNSUPPORTED, "sizes too large");
  const int es = s->dtype == SA_BF16 ? 2 : 4;
  if (s->d > 256 || s->d * es % 16 != 0)
    return set_error(SA_ERR_UNSUPPORTED, "sa_window_attn needs d <= 256 and d * elem_size a multiple of 16");
  return SA_OK;
}

bool on_tensor_cores(const sa_window_shape& s) { return s.dtype == SA_BF16 && (s.d == 64 || s.d == 128); }

// Which of the two tensor-core kernels takes a shape.  The decode kernel splits
// every row tile's keys over the GPU: its time goes with the 16-row tiles of all
// kv heads times the keys, 5.7e-5 us each (d = 64: 3.6e-5), and 4 us more of launch
// and join.  The prefill kernel's goes with the waves of its 256-row units times
// the 128-key tiles, 1.9 us each (1.6).  So it wins above 260 (350) - 70,000 / keys
// row tiles a wave.  32 query and 8 kv heads of 128, decode and prefill us: over
// 4096 keys 128 tokens 69 and 70, 256 tokens 128 and 71; over 512 keys 32 tokens 12.6
// and 14.5, 64 tokens 14.8 and 14.6, 128 tokens 19.6 and 14.7.  Heads of 64, 4096
// keys: 128 tokens 46 and 58, 192 tokens 66 and 60.  24 heads of 128 of their own, 4
// sequences of 4096 keys: 32 tokens 56 and 58, 64 tokens 100 and 58.  (A causal
// prompt over itself is charged all of its keys, of which its units see half.)
bool prefill_wins(const sa_window_shape& s, int64_t window, int64_t sinks) {
  const int64_t group = s.Hq / s.Hkv, tiles = ceil_div(s.Nq, 128);
  const int64_t units = s.B * (group % 2 == 0 ? s.Hq / 2 * tiles : s.Hq * ceil_div(tiles, 2));
  const int64_t keys = window > 0 ? min64(s.Nk, window + sinks + s.Nq) : s.Nk;
  return s.B * s.Hkv * ceil_div(s.Nq * group, 16) + 70000 / keys > (s.d == 64 ? 350 : 260) * ceil_div(units, 148);
}

sa_status check_kv4(const sa_kv4_desc* d) {
  if (!d) return set_error(SA_ERR_INVALID_ARG, "the cache description is NULL");
  if (d->num_pages <= 0 || d->Hkv <= 0) return set_error(SA_ERR_INVALID_ARG, "cache sizes must be positive");
  if (d->page != 16 && d->page != 32 && d->page != 64 && d->page != 128)
    return set_error(SA_ERR_UNSUPPORTED, "page must be 16, 32, 64 or 128");
  if (d->d != 64 && d->d != 128) return set_error(SA_ERR_UNSUPPORTED, "the 4-bit cache needs d = 64 or 128");
  if (d->num_pages > kInt32 / d->page || d->Hkv > 65535)
    return set_error(SA_ERR_UNSUPPORTED, "num_pages * page must fit 31 bits, Hkv 16 bits");
  return SA_OK;
}

size_t kv4_size(const sa_kv4_desc& d) { return (size_t)d.num_pages * d.Hkv * (d.page / 16) * 18 * d.d; }

// Elements that a strided [..] block spans, last axis of `row` contiguous elements.
int64_t span(const int64_t* strides, const int64_t* sizes, int n, int64_t row) {
  int64_t e = row;
  for (int i = 0; i < n; ++i) e += (sizes[i] - 1) * strides[i];
  return e;
}

// No two rows of `row` elements share one: each stride, from the smallest up,
// steps over everything that the smaller ones reach.
bool disjoint_rows(const int64_t* strides, const int64_t* sizes, int n, int64_t row) {
  int64_t reach = row;
  bool used[4] = {};
  for (int k = 0; k < n; ++k) {
    int at = -1;
    for (int i = 0; i < n; ++i)
      if (!used[i] && (at < 0 || strides[i] < strides[at])) at = i;
    used[at] = true;
    if (sizes[at] <= 1) continue;
    if (strides[at] < reach) return false;
    reach += (sizes[at] - 1) * strides[at];
  }
  return true;
}

sa_status kv4_attn(int32_t stall, const void* q, int64_t T, int64_t Hq, const int64_t q_strides[2], const int32_t* cu_q,
                   int64_t B, const void* cache, const sa_kv4_desc* desc, const int32_t* table, int64_t max_blocks,
                   const int32_t* kv_len, int64_t window, int64_t sinks, float scale, void* out, float* lse,
                   int32_t* status, void* ws, size_t ws_bytes, void* stream) {
  if (sa_status e = check_kv4(desc)) return e;
  if (sa_status e = check_window(window, sinks, scale)) return e;
  if (T < 0 || B < 0 || max_blocks < 0 || Hq <= 0) return set_error(SA_ERR_INVALID_ARG, "negative size");
  if (Hq % desc->Hkv != 0) return set_error(SA_ERR_INVALID_ARG, "Hq must be a multiple of Hkv");
  if (T > kInt32 / 2 || B > kInt32 / 2 || Hq > 65535 || T * Hq > kInt32 || max_blocks > kInt32 / 2 / desc->page)
    return set_error(SA_ERR_UNSUPPORTED, "sizes too large");
  if (T == 0 || B == 0) return SA_OK;   // no row
  if (max_blocks == 0) return set_error(SA_ERR_INVALID_ARG, "max_blocks must be positive");
  if (!q || !q_strides || !cu_q || !cache || !table || !kv_len || !out)
    return set_error(SA_ERR_INVALID_ARG, "NULL argument to sa_kv4_attn");
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(cache, 16))
    return set_error(SA_ERR_INVALID_ARG, "q, out and the cache must be 16-byte aligned");
  if (q_strides[0] < 0 || q_strides[1] < 0 || q_strides[0] % 8 || q_strides[1] % 8)
    return set_error(SA_ERR_INVALID_ARG, "q strides must be non-negative multiples of 8 elements");
  const int64_t sizes[2] = {T, Hq};
  const size_t qb = 2 * span(q_strides, sizes, 2, desc->d), ob = (size_t)T * Hq * desc->d * 2, lb = (size_t)T * Hq * 4;
  if (ranges_overlap(out, ob, q, qb) || ranges_overlap(out, ob, cache, kv4_size(*desc)) ||
      (lse && (ranges_overlap(lse, lb, q, qb) || ranges_overlap(lse, lb, cache, kv4_size(*desc)) ||
               ranges_overlap(lse, lb, out, ob))))
    return set_error(SA_ERR_INVALID_ARG, "out and lse must overlap neither q, the cache nor each other");
  const size_t need = sa_kv4_attn_workspace(desc, Hq);
  if (!ws || ws_bytes < need || !aligned(ws, 256))
    return set_error(SA_ERR_WORKSPACE, "sa_kv4_attn needs %zu bytes of 256-byte aligned workspace", need);
  if (sa_status e = check_device()) return e;
  if (!is_sm100()) return set_error(SA_ERR_UNSUPPORTED, "sa_kv4_attn needs an sm_100 device");
  Kv4AttnArgs a{q, cache, cu_q, table, kv_len, out, lse, status, *desc, T, Hq, B, max_blocks,
                {q_strides[0], q_strides[1]}, window, sinks,
                scale > 0.f ? scale : 1.0f / std::sqrt((float)desc->d), ws, stall};
  return launch_kv4_attn(a, static_cast<cudaStream_t>(stream));
}

}  // namespace

extern "C" {

size_t sa_window_attn_workspace(const sa_window_shape* shape) {
  if (check_window_shape(shape) != SA_OK) return 0;
  return on_tensor_cores(*shape) ? decode_ws_bytes(shape->d) : 256;
}

sa_status sa_window_attn(const void* q, const void* k, const void* v, const sa_window_shape* shape, int64_t window,
                         int64_t sinks, const int32_t* q_len, const int32_t* kv_len, float scale, void* out,
                         float* lse, int32_t* status, void* ws, size_t ws_bytes, int32_t flags, void* stream) {
  if (sa_status e = check_window_shape(shape)) return e;
  if (!q || !k || !v || !out) return set_error(SA_ERR_INVALID_ARG, "NULL tensor argument");
  if (sa_status e = check_window(window, sinks, scale)) return e;
  const sa_window_shape& s = *shape;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16))
    return set_error(SA_ERR_INVALID_ARG, "q, k, v and out must be 16-byte aligned");
  const size_t es = s.dtype == SA_BF16 ? 2 : 4;
  const size_t qb = (size_t)(s.B * s.Hq * s.Nq * s.d) * es, kb = (size_t)(s.B * s.Hkv * s.Nk * s.d) * es;
  const size_t lb = (size_t)(s.B * s.Hq * s.Nq) * 4;
  if (ranges_overlap(out, qb, q, qb) || ranges_overlap(out, qb, k, kb) || ranges_overlap(out, qb, v, kb) ||
      (lse && (ranges_overlap(lse, lb, q, qb) || ranges_overlap(lse, lb, k, kb) || ranges_overlap(lse, lb, v, kb) ||
               ranges_overlap(lse, lb, out, qb))))
    return set_error(SA_ERR_INVALID_ARG, "out and lse must overlap neither q, k, v nor each other");
  const size_t need = sa_window_attn_workspace(shape);
  if (!ws || ws_bytes < need || !aligned(ws, 256))
    return set_error(SA_ERR_WORKSPACE, "sa_window_attn needs %zu bytes of 256-byte aligned workspace", need);
  if (flags != 0 && flags != SA_FLAG_FORCE_SIMT && flags != SA_FLAG_FORCE_DECODE && flags != SA_FLAG_FORCE_PREFILL)
    return set_error(SA_ERR_INVALID_ARG, "unknown flags");
  if (flags > SA_FLAG_FORCE_SIMT && !on_tensor_cores(s))
    return set_error(SA_ERR_UNSUPPORTED, "no tensor-core kernel for this shape");
  if (sa_status e = check_device()) return e;
  if (!is_sm100()) return set_error(SA_ERR_UNSUPPORTED, "sa_window_attn needs an sm_100 device");
  WindowArgs a{q, k, v, out, lse, q_len, kv_len, status, s, window, sinks,
               scale > 0.f ? scale : 1.0f / std::sqrt((float)s.d), ws};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!on_tensor_cores(s) || flags == SA_FLAG_FORCE_SIMT) return launch_window_simt(a, st);
  return flags == SA_FLAG_FORCE_PREFILL || (flags == 0 && prefill_wins(s, window, sinks)) ? launch_window_tc(a, st) : launch_window_decode(a, st);
}

size_t sa_kv4_bytes(const sa_kv4_desc* desc) { return check_kv4(desc) == SA_OK ? kv4_size(*desc) : 0; }

sa_status sa_kv4_append(const void* k, const void* v, int64_t T, const int64_t k_strides[2],
                        const int64_t v_strides[2], const int32_t* slots, const sa_kv4_desc* desc, void* cache,
                        int32_t* status, void* stream) {
  if (sa_status e = check_kv4(desc)) return e;
  if (T < 0 || T > kInt32) return set_error(SA_ERR_INVALID_ARG, "T must lie in 0 .. 2^31 - 1");
  if (!cache || !k_strides || !v_strides || (T > 0 && (!k || !v || !slots)))
    return set_error(SA_ERR_INVALID_ARG, "NULL argument to sa_kv4_append");
  const int64_t sizes[2] = {T, desc->Hkv};
  for (int i = 0; i < 2; ++i)
    if (k_strides[i] < 0 || v_strides[i] < 0 || k_strides[i] % 4 || v_strides[i] % 4)
      return set_error(SA_ERR_INVALID_ARG, "strides must be non-negative multiples of 4 elements");
  if (!aligned(k, 8) || !aligned(v, 8) || !aligned(cache, 16))
    return set_error(SA_ERR_INVALID_ARG, "k and v must be 8-byte, the cache 16-byte aligned");
  if (T == 0) return SA_OK;
  if (ranges_overlap(k, 2 * span(k_strides, sizes, 2, desc->d), cache, kv4_size(*desc)) ||
      ranges_overlap(v, 2 * span(v_strides, sizes, 2, desc->d), cache, kv4_size(*desc)))
    return set_error(SA_ERR_INVALID_ARG, "k and v must not overlap the cache");
  if (sa_status e = check_device()) return e;
  return launch_kv4_append(k, v, T, k_strides, v_strides, slots, *desc, cache, status,
                           static_cast<cudaStream_t>(stream));
}

sa_status sa_kv4_read(const void* cache, const sa_kv4_desc* desc, const int32_t* slots, int64_t T, void* k, void* v,
                      int32_t* status, void* stream) {
  if (sa_status e = check_kv4(desc)) return e;
  if (T < 0 || T > kInt32) return set_error(SA_ERR_INVALID_ARG, "T must lie in 0 .. 2^31 - 1");
  if (!cache || (T > 0 && (!k || !v || !slots))) return set_error(SA_ERR_INVALID_ARG, "NULL argument to sa_kv4_read");
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(cache, 16))
    return set_error(SA_ERR_INVALID_ARG, "k, v and the cache must be 16-byte aligned");
  if (T == 0) return SA_OK;
  const size_t bytes = (size_t)T * desc->Hkv * desc->d * 2;
  if (ranges_overlap(k, bytes, cache, kv4_size(*desc)) || ranges_overlap(v, bytes, cache, kv4_size(*desc)) ||
      ranges_overlap(k, bytes, v, bytes))
    return set_error(SA_ERR_INVALID_ARG, "k and v must overlap neither the cache nor each other");
  if (sa_status e = check_device()) return e;
  return launch_kv4_read(cache, *desc, slots, T, k, v, status, static_cast<cudaStream_t>(stream));
}

size_t sa_kv4_attn_workspace(const sa_kv4_desc* desc, int64_t Hq) {
  if (check_kv4(desc) != SA_OK || Hq <= 0 || Hq % desc->Hkv) return 0;
  return decode_ws_bytes(desc->d);
}

sa_status sa_kv4_attn(const void* q, int64_t T, int64_t Hq, const int64_t q_strides[2], const int32_t* cu_q,
                      int64_t B, const void* cache, const sa_kv4_desc* desc, const int32_t* table,
                      int64_t max_blocks, const int32_t* kv_len, int64_t window, int64_t sinks, float scale,
                      void* out, float* lse, int32_t* status, void* ws, size_t ws_bytes, void* stream) {
  return kv4_attn(-1, q, T, Hq, q_strides, cu_q, B, cache, desc, table, max_blocks, kv_len, window, sinks, scale, out,
                  lse, status, ws, ws_bytes, stream);
}

// Not part of the interface: sa_kv4_attn with a wait that runs out, for its test.  The
// copies of block `stall` are never reported whole, the limit is 10 ms instead of 2 s,
// and the status word gets SA_ERR_TIMEOUT.
sa_status sa_kv4_attn_stalled(int32_t stall, const void* q, int64_t T, int64_t Hq, const int64_t q_strides[2],
                              const int32_t* cu_q, int64_t B, const void* cache, const sa_kv4_desc* desc,
                              const int32_t* table, int64_t max_blocks, const int32_t* kv_len, int64_t window,
                              int64_t sinks, float scale, void* out, float* lse, int32_t* status, void* ws,
                              size_t ws_bytes, void* stream) {
  return kv4_attn(stall, q, T, Hq, q_strides, cu_q, B, cache, desc, table, max_blocks, kv_len, window, sinks, scale, out,
                  lse, status, ws, ws_bytes, stream);
}

sa_status sa_rope_frequencies(const sa_rope_scaling* desc, uint64_t* freqs, float* magnitude) {
  if (!desc || !freqs || !magnitude) return set_error(SA_ERR_INVALID_ARG, "NULL argument to sa_rope_frequencies");
  const int32_t rot_dim = desc->rot_dim, scaling = desc->scaling;
  const double factor = desc->factor, beta_fast = desc->beta_fast, beta_slow = desc->beta_slow;
  const int64_t original_len = desc->original_len;
  const double base = desc->base;
  if (rot_dim < 2 || rot_dim % 2 || rot_dim > 1024) return set_error(SA_ERR_INVALID_ARG, "rot_dim must be even, 2 .. 1024");
  if (!(base > 1.0) || std::isinf(base)) return set_error(SA_ERR_INVALID_ARG, "base must be above 1 and finite");
  if (scaling < SA_ROPE_SCALE_NONE || scaling > SA_ROPE_SCALE_YARN)
    return set_error(SA_ERR_INVALID_ARG, "unknown scaling");
  if (scaling != SA_ROPE_SCALE_NONE && (!(factor >= 1.0) || std::isinf(factor)))
    return set_error(SA_ERR_INVALID_ARG, "factor must be at least 1 and finite");
  const double two_pi = 6.283185307179586476925286766559;
  double lo = 0, hi = 0;
  *magnitude = 1.f;
  if (scaling == SA_ROPE_SCALE_YARN) {
    if (original_len < 1 || !(beta_slow > 0) || !(beta_fast >= beta_slow) || std::isinf(beta_fast))
      return set_error(SA_ERR_INVALID_ARG, "yarn needs original_len >= 1 and beta_fast >= beta_slow > 0");
    // The pair that turns `turns` times over original_len positions.
    auto pair = [&](double turns) {
      return rot_dim * std::log((double)original_len / (turns * two_pi)) / (2 * std::log(base));
    };
    lo = std::fmax(0.0, std::floor(pair(beta_fast)));
    hi = std::fmin(rot_dim - 1.0, std::ceil(pair(beta_slow)));
    *magnitude = (float)(0.1 * std::log(factor) + 1.0);
  }
  // In 64 bits of mantissa: a frequency is then off by less than 4 units of 2^-64 turns, and
  // the angle of a position of 2^31 by less than 3e-9 rad (53 bits would leave 3e-7).
  static_assert(LDBL_MANT_DIG >= 64, "the frequencies need a long double of 64 bits");
  long double b = base;
  if (scaling == SA_ROPE_SCALE_NTK && rot_dim > 2) b *= std::pow((long double)factor, (long double)rot_dim / (rot_dim - 2));
  for (int i = 0; i < rot_dim / 2; ++i) {
    long double w = std::pow(b, -2.0L * i / rot_dim);
    if (scaling == SA_ROPE_SCALE_LINEAR) w /= factor;
    if (scaling == SA_ROPE_SCALE_YARN) {
      const long double r = std::fmin(1.0L, std::fmax(0.0L, (i - (long double)lo) / std::fmax((long double)hi - lo, 1e-3L)));
      w = w * (1 - r) + w / factor * r;
    }
    // w <= 1: below 2^62 in units of 2^-64 turns
    freqs[i] = (uint64_t)std::llround(std::ldexp(w / 6.283185307179586476925286766559005768L, 64));
  }
  return SA_OK;
}

sa_status sa_rope(const void* q, void* q_out, const void* k, void* k_out, const int32_t* pos,
                  const uint64_t* freqs, const sa_rope_desc* desc, void* stream) {
  if (!desc) return set_error(SA_ERR_INVALID_ARG, "the description is NULL");
  const sa_rope_desc& d = *desc;
  if (d.B < 0 || d.N < 0 || d.Hq < 0 || d.Hk < 0 || d.d <= 0) return set_error(SA_ERR_INVALID_ARG, "negative size");
  if (d.dtype != SA_BF16 && d.dtype != SA_FP32) return set_error(SA_ERR_INVALID_ARG, "unknown dtype");
  if (d.layout != SA_ROPE_HALF && d.layout != SA_ROPE_INTERLEAVED)
    return set_error(SA_ERR_INVALID_ARG, "layout must be SA_ROPE_HALF or SA_ROPE_INTERLEAVED");
  if (d.rot_dim < 2 || d.rot_dim % 2 || d.rot_dim > d.d)
    return set_error(SA_ERR_INVALID_ARG, "rot_dim must be even, at least 2 and at most d");
  if (d.inverse != 0 && d.inverse != 1) return set_error(SA_ERR_INVALID_ARG, "inverse must be 0 or 1");
  if (!std::isfinite(d.magnitude)) return set_error(SA_ERR_INVALID_ARG, "magnitude must be finite");
  if (d.d > 1024 || d.Hq + d.Hk > 65535 || d.N > kInt32 || (d.N > 0 && d.B > kInt32 / d.N))
    return set_error(SA_ERR_UNSUPPORTED, "sizes too large");
  if (d.B == 0 || d.N == 0 || d.Hq + d.Hk == 0) return SA_OK;
  if (!pos || !freqs || (d.Hq > 0 && (!q || !q_out)) || (d.Hk > 0 && (!k || !k_out)))
    return set_error(SA_ERR_INVALID_ARG, "NULL argument to sa_rope");
  if (d.pos_stride < 0) return set_error(SA_ERR_INVALID_ARG, "pos_stride must be non-negative");
  const size_t es = d.dtype == SA_BF16 ? 2 : 4;
  if (!aligned(q, es) || !aligned(q_out, es) || !aligned(k, es) || !aligned(k_out, es) || !aligned(freqs, 8) ||
      !aligned(pos, 4))
    return set_error(SA_ERR_INVALID_ARG, "misaligned tensor");
  const int64_t* st[4] = {d.q_strides, d.q_out_strides, d.k_strides, d.k_out_strides};
  const void* ptr[4] = {q, q_out, k, k_out};
  size_t bytes[4];
  for (int i = 0; i < 4; ++i) {
    const int64_t H = i < 2 ? d.Hq : d.Hk, sizes[3] = {d.B, d.N, H};
    bytes[i] = 0;
    if (H == 0) continue;
    for (int j = 0; j < 3; ++j) {
      if (st[i][j] < 0) return set_error(SA_ERR_INVALID_ARG, "strides must be non-negative");
    }
    if ((i & 1) && !disjoint_rows(st[i], sizes, 3, d.d))
      return set_error(SA_ERR_INVALID_ARG, "the rows of an output overlap one another");
    bytes[i] = es * span(st[i], sizes, 3, d.d);
  }
  auto clash = [&](int a, int b) { return bytes[a] && bytes[b] && ranges_overlap(ptr[a], bytes[a], ptr[b], bytes[b]); };
  for (int i = 0; i < 2; ++i) {
    const int a = 2 * i, b = 2 * i + 1;
    bool same = ptr[a] == ptr[b];
    const int64_t sizes[3] = {d.B, d.N, i ? d.Hk : d.Hq};
    for (int j = 0; j < 3; ++j) same = same && (sizes[j] == 1 || st[a][j] == st[b][j]);
    if (!same && clash(a, b)) return set_error(SA_ERR_INVALID_ARG, "an output overlaps its input (in place needs equal strides)");
  }
  // The other tensor's rows may lie between this one's (a packed q, k, v
  // row), so only equal starts are refused here.
  if (d.Hq > 0 && d.Hk > 0 && (q_out == k_out || q_out == k || k_out == q))
    return set_error(SA_ERR_INVALID_ARG, "q and k must not share their buffers");
  if (sa_status e = check_device()) return e;
  return launch_rope(q, q_out, k, k_out, pos, freqs, d, static_cast<cudaStream_t>(stream));
}

sa_status sa_cache_plan(const int32_t* kv_len, const int32_t* q_len, const sa_plan_desc* desc, int32_t* table,
                        int32_t* free_list, const int32_t* free_in, int32_t* free_out, int32_t* new_len,
                        int32_t* cu_q, int32_t* slots, int32_t* positions, int32_t* status, void* stream) {
  if (!desc) return set_error(SA_ERR_INVALID_ARG, "the description is NULL");
  const sa_plan_desc& d = *desc;
  if (d.B <= 0 || d.max_blocks <= 0 || d.num_pages <= 0 || d.max_tokens < 0)
    return set_error(SA_ERR_INVALID_ARG, "B, max_blocks and num_pages must be positive, max_tokens non-negative");
  if (d.page != 16 && d.page != 32 && d.page != 64 && d.page != 128)
    return set_error(SA_ERR_UNSUPPORTED, "page must be 16, 32, 64 or 128");
  if (d.B > 18000 || d.num_pages > kInt32 / d.page || d.max_blocks > kInt32 / d.page || d.max_tokens > kInt32)
    return set_error(SA_ERR_UNSUPPORTED, "B must be at most 18000, pages and tokens must fit 31 bits");
  if (!kv_len || !q_len || !table || !free_list || !free_in || !free_out || !new_len || !cu_q ||
      (d.max_tokens > 0 && (!slots || !positions)))
    return set_error(SA_ERR_INVALID_ARG, "NULL argument to sa_cache_plan");
  // Every block of the kernel reads the inputs, while others already write.
  const void* ptr[10] = {kv_len, q_len, free_in, table, free_list, free_out, new_len, cu_q, slots, positions};
  const int64_t n[10] = {d.B, d.B, 1, d.B * d.max_blocks, d.num_pages, 1, d.B, d.B + 1, d.max_tokens, d.max_tokens};
  for (int i = 0; i < 10; ++i) {
    if (!aligned(ptr[i], 4)) return set_error(SA_ERR_INVALID_ARG, "misaligned array");
    for (int j = i + 1; j < 10; ++j)
      if (j >= 3 && ptr[i] && ptr[j] && ranges_overlap(ptr[i], 4 * n[i], ptr[j], 4 * n[j]))
        return set_error(SA_ERR_INVALID_ARG, "an output of sa_cache_plan overlaps another array");
  }
  if (sa_status e = check_device()) return e;
  return launch_plan(kv_len, q_len, d, table, free_list, free_in, free_out, new_len, cu_q, slots, positions, status,
                     static_cast<cudaStream_t>(stream));
}

}  // extern "C"
