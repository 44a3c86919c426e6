// The Python binding of the serving operators: argument checks and marshalling
// in compiled code.  A decode step makes its calls for kernels of 4 us; the
// same checks in Python took 6 to 9 us a call, here 1 to 2.
//
// The entry points themselves come from libsparseattn.so: Python loads it and
// hands their addresses to bind(), so that this module links against torch only.
#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include <optional>
#include <string>

#include "sparse_attn.h"

namespace {

using at::Tensor;
using Maybe = std::optional<Tensor>;

struct Entry {
  decltype(&sa_window_attn) window_attn;
  decltype(&sa_kv4_append) kv4_append;
  decltype(&sa_kv4_read) kv4_read;
  decltype(&sa_kv4_attn) kv4_attn;
  decltype(&sa_rope) rope;
  decltype(&sa_cache_plan) cache_plan;
} entry;

void bind(const py::dict& at) {
  auto get = [&](const char* name, auto& fn) {
    fn = reinterpret_cast<std::remove_reference_t<decltype(fn)>>(at[name].cast<uintptr_t>());
  };
  get("sa_window_attn", entry.window_attn);
  get("sa_kv4_append", entry.kv4_append);
  get("sa_kv4_read", entry.kv4_read);
  get("sa_kv4_attn", entry.kv4_attn);
  get("sa_rope", entry.rope);
  get("sa_cache_plan", entry.cache_plan);
}

[[noreturn]] void refuse(const std::string& what) { throw py::value_error(what); }
void need(bool ok, const char* what) {
  if (!ok) refuse(what);
}

// t is a CUDA tensor of this dtype, shape and device.
void same(const Tensor& t, at::ScalarType dtype, at::IntArrayRef shape, const char* name, c10::Device dev,
          bool contiguous = true) {
  if (t.defined() && t.scalar_type() == dtype && t.device() == dev && dev.is_cuda() && t.sizes() == shape &&
      (!contiguous || t.is_contiguous()))
    return;
  const std::string n = name;
  if (!t.defined() || t.scalar_type() != dtype) refuse(n + " must be a " + c10::toString(dtype) + " tensor");
  if (t.device() != dev || !dev.is_cuda()) refuse(n + " must be on the same CUDA device as the other tensors");
  if (t.sizes() != shape) {
    std::string a, b;
    for (int64_t x : shape) a += std::to_string(x) + ", ";
    for (int64_t x : t.sizes()) b += std::to_string(x) + ", ";
    refuse(n + " must have shape (" + a + "), not (" + b + ")");
  }
  refuse(n + " must be contiguous");
}
const int32_t* index(const Tensor& t, int64_t n, const char* name, c10::Device dev) {
  same(t, at::kInt, {n}, name, dev);
  return static_cast<const int32_t*>(t.data_ptr());
}
int32_t* index(const Maybe& t, int64_t n, const char* name, c10::Device dev) {
  return t ? const_cast<int32_t*>(index(*t, n, name, dev)) : nullptr;
}
// Element strides {token, head} of a bf16 [T, H, d] tensor with contiguous channels.
struct Rows {
  int64_t strides[2];
  Rows(const Tensor& t, const char* name, int64_t T, int64_t H, int64_t d, c10::Device dev) {
    same(t, at::kBFloat16, {T, H, d}, name, dev, false);
    if (t.stride(2) != 1 && d != 1) refuse(std::string("the channels of ") + name + " must be contiguous");
    strides[0] = t.stride(0);
    strides[1] = t.stride(1);
  }
};
int32_t dtype_code(const Tensor& t) {
  if (t.scalar_type() == at::kBFloat16) return SA_BF16;
  if (t.scalar_type() == at::kFloat) return SA_FP32;
  refuse(std::string("unsupported dtype ") + c10::toString(t.scalar_type()));
}
struct Ws {
  void* ptr;
  size_t bytes;
  Ws(const Tensor& ws, c10::Device dev) : ptr(ws.data_ptr()), bytes(ws.nbytes()) {
    need(ws.is_contiguous() && ws.device() == dev, "ws must be a contiguous tensor on the other tensors' device");
  }
};

// The C ABI's scale has 32 bits, and 0 there means 1 / sqrt(d).
float scale32(double scale) {
  const float s = (float)scale;
  need(s != 0.f || scale == 0.0, "scale must be 0 or a number that 32 bits hold");
  return s;
}

// call(stream) with `dev` current, on the given stream or the device's current one.
template <class F>
int on(c10::Device dev, std::optional<uintptr_t> stream, F call) {
  need(entry.rope != nullptr, "the library has not been loaded");
  const c10::cuda::OptionalCUDAGuard guard(dev);
  return call(stream ? reinterpret_cast<void*>(*stream) : c10::cuda::getCurrentCUDAStream(dev.index()).stream());
}

using Stream = std::optional<uintptr_t>;

int window_attn(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& out, const Maybe& lse, int64_t window,
                int64_t sinks, const Maybe& q_len, const Maybe& kv_len, double scale, const Maybe& status,
                const Tensor& ws, int32_t flags, Stream stream) {
  const float sc = scale32(scale);
  need(q.dim() == 4 && k.dim() == 4, "q and k must have four axes");
  const auto dev = q.device();
  const auto dt = q.scalar_type();
  const sa_window_shape s{q.size(0), q.size(1), k.size(1), q.size(2), k.size(2), q.size(3), dtype_code(q), 0};
  same(q, dt, {s.B, s.Hq, s.Nq, s.d}, "q", dev);
  same(k, dt, {s.B, s.Hkv, s.Nk, s.d}, "k", dev);
  same(v, dt, {s.B, s.Hkv, s.Nk, s.d}, "v", dev);
  same(out, dt, {s.B, s.Hq, s.Nq, s.d}, "out", dev);
  if (lse) same(*lse, at::kFloat, {s.B, s.Hq, s.Nq}, "lse", dev);
  const int32_t *ql = index(q_len, s.B, "q_len", dev), *kl = index(kv_len, s.B, "kv_len", dev);
  int32_t* st = index(status, 1, "status", dev);
  const Ws w(ws, dev);
  return on(dev, stream, [&](void* cs) {
    return entry.window_attn(q.data_ptr(), k.data_ptr(), v.data_ptr(), &s, window, sinks, ql, kl, sc,
                             out.data_ptr(), lse ? static_cast<float*>(lse->data_ptr()) : nullptr, st, w.ptr, w.bytes,
                             flags, cs);
  });
}

// The cache: pages uint8 [num_pages, Hkv, page / 16, 18 d], which KV4Cache has checked.
sa_kv4_desc describe(const Tensor& pages, int64_t page, int64_t d) {
  same(pages, at::kByte, {pages.size(0), pages.size(1), page / 16, 18 * d}, "pages", pages.device());
  return {pages.size(0), pages.size(1), (int32_t)page, (int32_t)d};
}

int kv4_append(const Tensor& k, const Tensor& v, const Tensor& slots, const Tensor& pages, int64_t page, int64_t d,
               const Maybe& status, Stream stream) {
  const auto dev = pages.device();
  const sa_kv4_desc desc = describe(pages, page, d);
  need(k.dim() == 3, "k must have three axes");
  const int64_t T = k.size(0);
  const Rows ks(k, "k", T, desc.Hkv, d, dev), vs(v, "v", T, desc.Hkv, d, dev);
  const int32_t* at = index(slots, T, "slots", dev);
  int32_t* st = index(status, 1, "status", dev);
  return on(dev, stream, [&](void* cs) {
    return entry.kv4_append(k.data_ptr(), v.data_ptr(), T, ks.strides, vs.strides, at, &desc, pages.data_ptr(), st, cs);
  });
}

int kv4_read(const Tensor& pages, int64_t page, int64_t d, const Tensor& slots, const Tensor& k, const Tensor& v,
             const Maybe& status, Stream stream) {
  const auto dev = pages.device();
  const sa_kv4_desc desc = describe(pages, page, d);
  need(k.dim() == 3, "k must have three axes");
  const int64_t T = k.size(0);
  same(k, at::kBFloat16, {T, desc.Hkv, d}, "k", dev);
  same(v, at::kBFloat16, {T, desc.Hkv, d}, "v", dev);
  const int32_t* at = index(slots, T, "slots", dev);
  int32_t* st = index(status, 1, "status", dev);
  return on(dev, stream, [&](void* cs) {
    return entry.kv4_read(pages.data_ptr(), &desc, at, T, k.data_ptr(), v.data_ptr(), st, cs);
  });
}

int kv4_attn(const Tensor& q, const Tensor& pages, int64_t page, int64_t d, const Tensor& table, const Tensor& kv_len,
             const Tensor& out, const Maybe& lse, const Tensor& cu_q, int64_t window, int64_t sinks, double scale,
             const Maybe& status, const Tensor& ws, Stream stream) {
  const float sc = scale32(scale);
  const auto dev = pages.device();
  const sa_kv4_desc desc = describe(pages, page, d);
  need(q.dim() == 3 && table.dim() == 2, "q must have three axes and table two");
  const int64_t T = q.size(0), Hq = q.size(1), B = table.size(0), blocks = table.size(1);
  const Rows qs(q, "q", T, Hq, d, dev);
  same(table, at::kInt, {B, blocks}, "table", dev);
  same(out, at::kBFloat16, {T, Hq, d}, "out", dev);
  if (lse) same(*lse, at::kFloat, {T, Hq}, "lse", dev);
  const int32_t *cu = index(cu_q, B + 1, "cu_q", dev), *kl = index(kv_len, B, "kv_len", dev);
  int32_t* st = index(status, 1, "status", dev);
  const Ws w(ws, dev);
  return on(dev, stream, [&](void* cs) {
    return entry.kv4_attn(q.data_ptr(), T, Hq, qs.strides, cu, B, pages.data_ptr(), &desc,
                          static_cast<const int32_t*>(table.data_ptr()), blocks, kl, window, sinks, sc,
                          out.data_ptr(), lse ? static_cast<float*>(lse->data_ptr()) : nullptr, st, w.ptr, w.bytes, cs);
  });
}

// Strides {batch, token, head} of a [T, H, d] or [B, N, H, d] tensor.
void rope_strides(const Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType dt, c10::Device dev,
                  int64_t* s) {
  same(t, dt, shape, name, dev, false);
  const int64_t n = t.dim();
  if (t.stride(n - 1) != 1 && shape[n - 1] != 1)
    refuse(std::string("the channels of ") + name + " must be contiguous");
  s[0] = n == 4 ? t.stride(0) : 0;
  s[1] = t.stride(n - 3);
  s[2] = t.stride(n - 2);
}

int rope(const Tensor& freqs, int32_t rot_dim, int32_t layout, double magnitude, const Tensor& pos, const Tensor& q,
         const Tensor& q_out, const Maybe& k, const Maybe& k_out, bool inverse, Stream stream) {
  const auto dev = q.device();
  const auto dt = q.scalar_type();
  const int64_t n = q.dim();
  need(n == 3 || n == 4, "q must have three or four axes");
  need(k.has_value() == k_out.has_value(), "k and k_out go together");
  sa_rope_desc d{};
  d.B = n == 4 ? q.size(0) : 1;
  d.N = q.size(n - 3);
  d.Hq = q.size(n - 2);
  d.d = q.size(n - 1);
  rope_strides(q, "q", q.sizes(), dt, dev, d.q_strides);
  rope_strides(q_out, "q_out", q.sizes(), dt, dev, d.q_out_strides);
  if (k) {
    need(k->dim() == n, "q and k must have as many axes");
    d.Hk = k->size(n - 2);
    auto shape = q.sizes().vec();
    shape[n - 2] = d.Hk;
    rope_strides(*k, "k", shape, dt, dev, d.k_strides);
    rope_strides(*k_out, "k_out", shape, dt, dev, d.k_out_strides);
  }
  const bool batched = n == 4 && pos.dim() == 2;
  same(pos, at::kInt, batched ? q.sizes().slice(0, 2) : q.sizes().slice(n - 3, 1), "pos", dev, false);
  need(d.N <= 1 || pos.stride(-1) == 1, "the positions of a sequence must be contiguous");
  need(freqs.device() == dev && freqs.scalar_type() == at::kLong && freqs.is_contiguous() && freqs.numel() >= rot_dim / 2,
       "the frequencies must be a Rope's, on the tensors' device");
  d.pos_stride = batched ? pos.stride(0) : 0;
  d.rot_dim = rot_dim;
  d.layout = layout;
  d.dtype = dtype_code(q);
  d.inverse = inverse;
  d.magnitude = (float)magnitude;
  return on(dev, stream, [&](void* cs) {
    return entry.rope(q.data_ptr(), q_out.data_ptr(), k ? k->data_ptr() : nullptr, k ? k_out->data_ptr() : nullptr,
                      static_cast<const int32_t*>(pos.data_ptr()), static_cast<const uint64_t*>(freqs.data_ptr()), &d, cs);
  });
}

int cache_plan(const Tensor& kv_len, const Tensor& q_len, const Tensor& table, const Tensor& free_list,
               const Tensor& free_count, int64_t page, const Tensor& new_len, const Tensor& cu_q, const Tensor& slots,
               const Tensor& positions, const Tensor& free_count_out, const Maybe& status, Stream stream) {
  const auto dev = table.device();
  need(table.dim() == 2, "table must have two axes");
  const sa_plan_desc d{table.size(0), table.size(1), free_list.numel(), slots.numel(), (int32_t)page, 0};
  same(table, at::kInt, {d.B, d.max_blocks}, "table", dev);
  auto out = [&](const Tensor& t, int64_t n, const char* name) { return const_cast<int32_t*>(index(t, n, name, dev)); };
  const int32_t *kl = index(kv_len, d.B, "kv_len", dev), *ql = index(q_len, d.B, "q_len", dev),
                *fin = index(free_count, 1, "free_count", dev);
  int32_t *fl = out(free_list, d.num_pages, "free_list"), *fout = out(free_count_out, 1, "free_count_out"),
          *nl = out(new_len, d.B, "new_len"), *cu = out(cu_q, d.B + 1, "cu_q"), *sl = out(slots, d.max_tokens, "slots"),
          *po = out(positions, d.max_tokens, "positions"), *st = index(status, 1, "status", dev);
  return on(dev, stream, [&](void* cs) {
    return entry.cache_plan(kl, ql, &d, static_cast<int32_t*>(table.data_ptr()), fl, fin, fout, nl, cu, sl, po, st, cs);
  });
}

}  // namespace

PYBIND11_MODULE(_serve, m) {
  m.attr("built_for_torch") = BUILT_FOR_TORCH;
  m.def("bind", &bind);
  m.def("window_attn", &window_attn);
  m.def("kv4_append", &kv4_append);
  m.def("kv4_read", &kv4_read);
  m.def("kv4_attn", &kv4_attn);
  m.def("rope", &rope);
  m.def("cache_plan", &cache_plan);
}
