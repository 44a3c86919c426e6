// Rotary positions: y = mag * R(p) x on the first rot_dim channels of every
// head, the other channels copied.  Pair i turns by the angle p * w_i:
//   (y1, y2) = mag * (x1 cos - x2 sin, x2 cos + x1 sin),
// its two channels either i and i + rot_dim / 2 ("half") or 2 i and 2 i + 1
// ("interleaved").  The transposed rotation (angle negated) is the gradient.
//
// The angle of a far position needs more bits than a float has: p = 10^6 with
// w = 1 would be off by 0.03 rad.  Frequencies are therefore held as turns per
// position in 64-bit fixed point (f = w / 2 pi * 2^64, good to a few units): p * f
// modulo 2^64 is the fraction of a turn (below 5e-9 rad off at 2^31), one integer
// multiply, and its top 32 bits are split into quarter turns and a rest for
// sincospif (2.5e-8 rad).
//
// Bound by HBM: x read once, y written once.  A CTA takes TOK tokens: it
// computes their cos and sin once into shared memory (one pair per thread) and
// all heads of q and k use them, so the trigonometry is 1 / (Hq + Hk) of the
// pairs and one launch serves both tensors.  16,411 tokens, 32 + 8 heads of 128 in
// bf16: 59.5 us on the GPU, 5.6 TB/s; through the call, on inputs that change, 63.
#include <cmath>

#include "sa_internal.cuh"

namespace sa {
namespace {

constexpr int kRopeThreads = 256;

struct RopeArgs {
  const void* x[2];
  void* y[2];
  int64_t xs[2][3], ys[2][3];   // element strides: batch, token, head
  int32_t heads[2];
  int32_t heads_all;
  int32_t copy[2];              // the channels past rot_dim need copying (not in place)
  const int32_t* pos;
  int64_t pos_sb;
  const uint64_t* freqs;
  int64_t tokens, N;            // B * N tokens in all, N per batch entry
  int32_t d, rot, inverse;
  float mag;
  int32_t items;                // vector items of one head (pairs of vectors, then copies)
  int32_t pair_items;
  uint64_t items_inv;           // ceil(2^40 / items): exact quotients, as numbers times items stay below 2^40
};

// VEC elements as they lie in memory, and as floats.
template <typename T, int VEC> struct Pack;
template <> struct Pack<uint16_t, 8> {
  using Raw = uint4;
  static __device__ __forceinline__ Raw load(const uint16_t* p) { return *reinterpret_cast<const uint4*>(p); }
  static __device__ __forceinline__ void open(const Raw& r, float* f) { unpack16(r, uint16_t{}, f); }
  static __device__ __forceinline__ Raw close(const float* f) {
    uint4 u;
    uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<uint32_t*>(&h);
    }
    return u;
  }
  static __device__ __forceinline__ void store(uint16_t* p, const Raw& r) { *reinterpret_cast<uint4*>(p) = r; }
};
template <> struct Pack<float, 4> {
  using Raw = float4;
  static __device__ __forceinline__ Raw load(const float* p) { return *reinterpret_cast<const float4*>(p); }
  static __device__ __forceinline__ void open(const Raw& r, float* f) { *reinterpret_cast<float4*>(f) = r; }
  static __device__ __forceinline__ Raw close(const float* f) { return *reinterpret_cast<const float4*>(f); }
  static __device__ __forceinline__ void store(float* p, const Raw& r) { *reinterpret_cast<float4*>(p) = r; }
};
// Any alignment: an element, or a pair, at a time.
template <typename T, int N> struct Few {
  struct Raw { T v[N]; };
  static __device__ __forceinline__ float one(uint16_t v) { return bf16_to_f32(v); }
  static __device__ __forceinline__ float one(float v) { return v; }
  static __device__ __forceinline__ Raw load(const T* p) {
    Raw r;
#pragma unroll
    for (int i = 0; i < N; ++i) r.v[i] = p[i];
    return r;
  }
  static __device__ __forceinline__ void open(const Raw& r, float* f) {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = one(r.v[i]);
  }
  static __device__ __forceinline__ Raw close(const float* f) {
    Raw r;
#pragma unroll
    for (int i = 0; i < N; ++i) Elem<T>::store(&r.v[i], f[i]);
    return r;
  }
  static __device__ __forceinline__ void store(T* p, const Raw& r) {
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = r.v[i];
  }
};
template <typename T> struct Pack<T, 2> : Few<T, 2> {};
template <typename T> struct Pack<T, 1> : Few<T, 1> {};

// One item: the vector pair (HALF) or vector of a head's rotated channels, or a
// vector of those that do not turn.
template <typename T, int VEC, bool HALF>
struct Item {
  static constexpr int W = VEC < 2 ? 2 : VEC;   // interleaved: whole pairs
  using PV = Pack<T, VEC>;
  using PW = Pack<T, W>;
  T* y;
  const float2* c;
  typename PV::Raw u, v;   // HALF: the pairs' first and second channels; else u: copied channels
  typename PW::Raw w;      // interleaved pairs
  int kind;                // 0: nothing, 1: turn, 2: copy
  __device__ __forceinline__ void load(const T* x, int half) {
    if (kind == 2 || (HALF && kind == 1)) u = PV::load(x);
    if (HALF && kind == 1) v = PV::load(x + half);
    if (!HALF && kind == 1) w = PW::load(x);
  }
  __device__ __forceinline__ void store(int half) {
    if (kind == 2) PV::store(y, u);
    if (kind != 1) return;
    if constexpr (HALF) {
      float a[VEC], b[VEC];
      PV::open(u, a);
      PV::open(v, b);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float2 t = c[e];
        const float p = a[e] * t.x - b[e] * t.y, q = b[e] * t.x + a[e] * t.y;
        a[e] = p;
        b[e] = q;
      }
      PV::store(y, PV::close(a));
      PV::store(y + half, PV::close(b));
    } else {
      float a[W];
      PW::open(w, a);
#pragma unroll
      for (int e = 0; e < W; e += 2) {
        const float2 t = c[e >> 1];
        const float p = a[e] * t.x - a[e + 1] * t.y, q = a[e + 1] * t.x + a[e] * t.y;
        a[e] = p;
        a[e + 1] = q;
      }
      PW::store(y, PW::close(a));
    }
  }
};

// x and y may be the same buffer (in place), so loads are plain loads and a
// thread reads all channels of its pairs before it writes them.
template <typename T, int VEC, bool HALF, int TOK>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  extern __shared__ float2 cs[];   // [TOK][rot / 2]
  __shared__ int64_t at[TOK][4];   // the tokens' places in q, q_out, k, k_out
  const int half = a.rot >> 1;
  const int64_t t0 = (int64_t)blockIdx.x * TOK;
  const int nt = (int)min64(TOK, a.tokens - t0);
  if (threadIdx.x < nt * 4) {
    const int tt = threadIdx.x >> 2, z = threadIdx.x & 3;
    const int64_t t = t0 + tt, b = t / a.N, n = t - b * a.N;
    const int64_t* s = z & 1 ? a.ys[z >> 1] : a.xs[z >> 1];
    at[tt][z] = b * s[0] + n * s[1];
  }
  __syncthreads();
  const int per_tok = a.heads_all * a.items, all = nt * per_tok;
  // Item i, its loads under way.
  auto item = [&](int i) {
    Item<T, VEC, HALF> m;
    m.kind = 0;
    if (i >= all) return m;
    int tt = 0;
#pragma unroll
    for (int x = 1; x < TOK; ++x) tt += i >= x * per_tok;
    const int r = i - tt * per_tok;
    int h = (int)(((uint64_t)r * a.items_inv) >> 40);   // r / items
    const int it = r - h * a.items;
    const int which = h >= a.heads[0];
    if (which) h -= a.heads[0];
    const bool turns = it < a.pair_items;
    if (!turns && !a.copy[which]) return m;
    const int ch = turns ? it * (HALF ? VEC : Item<T, VEC, HALF>::W) : a.rot + (it - a.pair_items) * VEC;
    m.kind = turns ? 1 : 2;
    m.y = static_cast<T*>(a.y[which]) + at[tt][2 * which + 1] + h * a.ys[which][2] + ch;
    m.c = cs + tt * half + (HALF ? ch : ch >> 1);
    m.load(static_cast<const T*>(a.x[which]) + at[tt][2 * which] + h * a.xs[which][2] + ch, half);
    return m;
  };
  // The first item's loads run while the angles are computed, each next one's
  // while one is turned and stored (items do not overlap, in place either).
  Item<T, VEC, HALF> m = item(threadIdx.x);
  for (int i = threadIdx.x; i < nt * half; i += kRopeThreads) {
    const int tt = i / half, f = i - tt * half;
    const int64_t t = t0 + tt, b = t / a.N;
    const int64_t p = a.pos[b * a.pos_sb + (t - b * a.N)];
    const uint64_t phase = (uint64_t)p * a.freqs[f];
    // The nearest quarter turn and the rest in [-1/4, 1/4) half turns: the
    // rest's rounding to 24 bits is then at most 2^-27 half turns, 2.4e-8 rad.
    const int32_t top = (int32_t)(phase >> 32);
    const uint32_t quarter = ((uint32_t)top + 0x20000000u) >> 30;
    float s, c;
    sincospif((float)(int32_t)((uint32_t)top - (quarter << 30)) * 0x1p-31f, &s, &c);
    if (quarter & 1) {
      const float x = c;
      c = -s;
      s = x;
    }
    if (quarter & 2) {
      c = -c;
      s = -s;
    }
    cs[i] = make_float2(c * a.mag, a.inverse ? -s * a.mag : s * a.mag);
  }
  __syncthreads();
  for (int i = threadIdx.x + kRopeThreads; m.kind || i - kRopeThreads < all; i += kRopeThreads) {
    const Item<T, VEC, HALF> next = item(i);
    m.store(half);
    m = next;
  }
}

template <typename T, int VEC, bool HALF, int TOK>
sa_status launch_tok(RopeArgs& a, cudaStream_t st) {
  a.pair_items = HALF ? a.rot / 2 / VEC : a.rot / (VEC < 2 ? 2 : VEC);
  a.items = a.pair_items + (a.d - a.rot) / VEC;
  a.items_inv = (1ull << 40) / a.items + 1;
  const int64_t ctas = ceil_div(a.tokens, TOK);
  if (ctas > 2147483647) return set_error(SA_ERR_UNSUPPORTED, "too many tokens");
  rope_kernel<T, VEC, HALF, TOK><<<(unsigned)ctas, kRopeThreads, (size_t)TOK * (a.rot / 2) * sizeof(float2), st>>>(a);
  return check_launch("rope_kernel");
}

template <typename T, int VEC>
sa_status launch_vec(RopeArgs& a, bool half, cudaStream_t st) {
  // Four tokens a CTA share the launch and the barrier once they fill the
  // GPU; below that one token a CTA spreads a decode step over the SMs.
  if (a.tokens >= 148 * 16) return half ? launch_tok<T, VEC, true, 4>(a, st) : launch_tok<T, VEC, false, 4>(a, st);
  return half ? launch_tok<T, VEC, true, 1>(a, st) : launch_tok<T, VEC, false, 1>(a, st);
}

}  // namespace

sa_status launch_rope(const void* q, void* q_out, const void* k, void* k_out, const int32_t* pos,
                      const uint64_t* freqs, const sa_rope_desc& d, cudaStream_t st) {
  RopeArgs a{};
  a.x[0] = q;
  a.y[0] = q_out;
  a.x[1] = k;
  a.y[1] = k_out;
  const int es = d.dtype == SA_BF16 ? 2 : 4;
  const int vec = 16 / es;
  bool wide = d.d % vec == 0 && d.rot_dim % vec == 0 && (d.layout == SA_ROPE_INTERLEAVED || (d.rot_dim / 2) % vec == 0);
  auto fits = [&](const void* p, const int64_t* s) {
    if ((uintptr_t)p % 16) wide = false;
    for (int i = 0; i < 3; ++i)
      if (s[i] % vec) wide = false;
  };
  fits(q, d.q_strides);
  fits(q_out, d.q_out_strides);
  if (k) {
    fits(k, d.k_strides);
    fits(k_out, d.k_out_strides);
  }
  for (int i = 0; i < 3; ++i) {
    a.xs[0][i] = d.q_strides[i];
    a.ys[0][i] = d.q_out_strides[i];
    a.xs[1][i] = d.k_strides[i];
    a.ys[1][i] = d.k_out_strides[i];
  }
  a.heads[0] = (int32_t)d.Hq;
  a.heads[1] = k ? (int32_t)d.Hk : 0;
  a.heads_all = a.heads[0] + a.heads[1];
  a.copy[0] = q != q_out;
  a.copy[1] = k != k_out;
  a.pos = pos;
  a.pos_sb = d.pos_stride;
  a.freqs = freqs;
  a.tokens = d.B * d.N;
  a.N = d.N;
  a.d = (int32_t)d.d;
  a.rot = d.rot_dim;
  a.inverse = d.inverse;
  a.mag = d.magnitude;
  const bool half = d.layout == SA_ROPE_HALF;
  if (d.dtype == SA_BF16) return wide ? launch_vec<uint16_t, 8>(a, half, st) : launch_vec<uint16_t, 1>(a, half, st);
  return wide ? launch_vec<float, 4>(a, half, st) : launch_vec<float, 1>(a, half, st);
}

}  // namespace sa
