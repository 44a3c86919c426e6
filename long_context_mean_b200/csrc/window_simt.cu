// Attention with a sliding window and first tokens that stay visible, on the
// CUDA cores: fp32, and bf16 head widths that have no tensor-core kernel.
//
// Mathematics: row i at position p = n_k - n_q + i sees key j iff j <= p, j < n_k
// and (window == 0 or p - j < window or j < sinks); o = sum 2^(c (s_j - m)) v_j / l
// with c = scale log2 e, the running maximum m of the raw scores and the running
// sum l.  The difference s_j - m is taken before the scaling, so its rounding is
// relative to the difference, not to the scores.
//
// Bound by the fp32 pipes (4 d flops a pair; there is no fp32 tensor-core
// instruction).  One CTA takes 64 rows of one query head and walks the tiles of
// 64 keys that some of its rows see.  A thread owns 8 rows times 4 keys of S and
// 8 rows times 4 (d / 64) channels of O in registers: 12 shared-memory vectors
// feed 128 multiply-adds, which keeps shared memory below the fp32 pipes' time
// (4 x 4 has 8 vectors for 64 and is bound by shared memory).
#include "sa_internal.cuh"

namespace sa {
namespace {

constexpr int kRows = 64, kKeys = 64, kThreads = 128;
constexpr float kLog2e = 1.4426950408889634f;

struct SimtArgs {
  const void* q;
  const void* k;
  const void* v;
  void* out;
  float* lse;
  const int32_t* q_len;
  const int32_t* kv_len;
  int32_t* status;
  int64_t Nq, Nk, window, sinks, row_tiles;
  int32_t Hq, Hkv, d;
  float scale;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Rows [r0, r0 + 64) of a [n][d] array as floats to shared memory, row stride
// d + 4 (float4 reads of neighbouring rows then meet no bank twice); rows that
// live() leaves out come as zeros.
template <typename T, class Live>
__device__ __forceinline__ void load_tile(float* dst, const T* src, int64_t r0, int d, Live live) {
  constexpr int V = 16 / sizeof(T);
  const int per = d / V;
  for (int i = threadIdx.x; i < 64 * per; i += kThreads) {
    const int r = i / per, c = (i - r * per) * V;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (live(r0 + r)) w = __ldg(reinterpret_cast<const uint4*>(src + (r0 + r) * d + c));
    float f[V];
    unpack16(w, T{}, f);
#pragma unroll
    for (int e = 0; e < V; e += 4) *reinterpret_cast<float4*>(dst + r * (d + 4) + c + e) = *reinterpret_cast<float4*>(f + e);
  }
}

// CW: 64-channel column blocks of O (d <= 64 CW).
template <typename T, int CW>
__global__ void __launch_bounds__(kThreads) window_simt_kernel(const __grid_constant__ SimtArgs a) {
  extern __shared__ __align__(16) float smf[];
  const int d = a.d, ds = d + 4;
  float* qs = smf;
  float* ks = qs + kRows * ds;
  float* vs = ks + kKeys * ds;
  float* ps = vs + kKeys * ds;   // [64][68]
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t bh = blockIdx.x / a.row_tiles, row0 = (blockIdx.x - bh * a.row_tiles) * kRows;
  const int64_t b = bh / a.Hq, h = bh - b * a.Hq;
  int64_t n_q = a.q_len ? a.q_len[b] : a.Nq, n_k = a.kv_len ? a.kv_len[b] : a.Nk;
  if (n_q < 0 || n_q > a.Nq || n_k < 0 || n_k > a.Nk) {
    if (threadIdx.x == 0) raise_status(a.status, SA_ERR_INVALID_ARG);
    n_q = max64(0, min64(n_q, a.Nq));
    n_k = max64(0, min64(n_k, a.Nk));
  }
  if (row0 >= n_q) return;
  const T* q = static_cast<const T*>(a.q) + bh * a.Nq * d;
  const int64_t kvh = b * a.Hkv + h / (a.Hq / a.Hkv);
  const T* k = static_cast<const T*>(a.k) + kvh * a.Nk * d;
  const T* v = static_cast<const T*>(a.v) + kvh * a.Nk * d;

  const int64_t first = n_k - n_q + row0;                          // position of the tile's first row
  const int64_t last = n_k - n_q + min64(n_q, row0 + kRows) - 1;   // and of its last
  const int64_t hi = min64(n_k, last + 1);
  const int64_t lo = min64(a.window > 0 ? max64(0, first - a.window + 1) : 0, max64(hi, 0));
  const int64_t n_sink = min64(a.sinks, lo);
  const int64_t sink_tiles = ceil_div_d(n_sink, kKeys), t_lo = max64(sink_tiles, lo / kKeys);
  const int64_t tiles = hi <= 0 ? 0 : sink_tiles + max64(0, ceil_div_d(hi, kKeys) - t_lo);

  load_tile<T>(qs, q, row0, d, [&](int64_t r) { return r < n_q; });
  float o[8][4 * CW], m[8], l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int e = 0; e < 4 * CW; ++e) o[i][e] = 0.f;
  }
  const float c2 = a.scale * kLog2e;
  for (int64_t t = 0; t < tiles; ++t) {
    const int64_t k0 = (t < sink_tiles ? t : t_lo + (t - sink_tiles)) * kKeys;
    auto live = [&](int64_t j) { return j < hi && (j >= lo || j < n_sink); };
    __syncthreads();
    load_tile<T>(ks, k, k0, d, live);
    load_tile<T>(vs, v, k0, d, live);
    __syncthreads();
    float s[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
    for (int c = 0; c < d; c += 4) {
      float4 kk[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) kk[j] = *reinterpret_cast<const float4*>(ks + (tx + 16 * j) * ds + c);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 x = *reinterpret_cast<const float4*>(qs + (ty * 8 + i) * ds + c);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          s[i][j] = fmaf(x.x, kk[j].x, fmaf(x.y, kk[j].y, fmaf(x.z, kk[j].z, fmaf(x.w, kk[j].w, s[i][j]))));
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t p = first + ty * 8 + i;
      float mx = m[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t key = k0 + tx + 16 * j;
        if (!(key <= p && key < n_k && (a.window == 0 || p - key < a.window || key < a.sinks))) s[i][j] = -INFINITY;
        mx = fmaxf(mx, s[i][j]);
      }
#pragma unroll
      for (int w = 1; w < 16; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      const float ref = mx == -INFINITY ? 0.f : mx;
      const float corr = ex2((m[i] - ref) * c2);
      m[i] = mx;
      l[i] *= corr;
#pragma unroll
      for (int e = 0; e < 4 * CW; ++e) o[i][e] *= corr;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float pr = ex2((s[i][j] - ref) * c2);
        l[i] += pr;
        ps[(ty * 8 + i) * 68 + tx + 16 * j] = pr;
      }
    }
    __syncwarp();   // a row's P is written and read by the same half warp
#pragma unroll 2
    for (int j = 0; j < kKeys; j += 4) {
      float4 pr[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) pr[i] = *reinterpret_cast<const float4*>(ps + (ty * 8 + i) * 68 + j);
#pragma unroll
      for (int w = 0; w < CW; ++w) {
        const int ch = tx * 4 + 64 * w;
        if (ch >= d) break;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float4 vv = *reinterpret_cast<const float4*>(vs + (j + x) * ds + ch);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float px = x == 0 ? pr[i].x : x == 1 ? pr[i].y : x == 2 ? pr[i].z : pr[i].w;
            o[i][4 * w] = fmaf(px, vv.x, o[i][4 * w]);
            o[i][4 * w + 1] = fmaf(px, vv.y, o[i][4 * w + 1]);
            o[i][4 * w + 2] = fmaf(px, vv.z, o[i][4 * w + 2]);
            o[i][4 * w + 3] = fmaf(px, vv.w, o[i][4 * w + 3]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int w = 1; w < 16; w <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
    const int64_t row = row0 + ty * 8 + i;
    if (row >= n_q) continue;
    const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];   // no visible key: zeros; NaN stays
    T* dst = static_cast<T*>(a.out) + (bh * a.Nq + row) * d;
#pragma unroll
    for (int w = 0; w < CW; ++w)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (tx * 4 + 64 * w < d) Elem<T>::store(dst + tx * 4 + 64 * w + e, o[i][4 * w + e] * inv);
    if (tx == 0 && a.lse) a.lse[bh * a.Nq + row] = l[i] == 0.f ? -INFINITY : fmaf(m[i], a.scale, logf(l[i]));
  }
}

template <typename T, int CW>
sa_status launch(const SimtArgs& a, int64_t heads, cudaStream_t st) {
  const size_t smem = (size_t)(3 * 64 * (a.d + 4) + 64 * 68) * sizeof(float);
  if (cudaFuncSetAttribute(window_simt_kernel<T, CW>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
      cudaSuccess)
    return set_error(SA_ERR_CUDA, "cudaFuncSetAttribute(window_simt_kernel) failed");
  const int64_t ctas = heads * a.row_tiles;
  if (ctas > INT32_MAX) return set_error(SA_ERR_UNSUPPORTED, "too many rows");
  window_simt_kernel<T, CW><<<(unsigned)ctas, kThreads, smem, st>>>(a);
  return check_launch("window_simt_kernel");
}

template <typename T>
sa_status launch_type(const SimtArgs& a, int64_t heads, cudaStream_t st) {
  if (a.d <= 64) return launch<T, 1>(a, heads, st);
  if (a.d <= 128) return launch<T, 2>(a, heads, st);
  return launch<T, 4>(a, heads, st);
}

}  // namespace

sa_status launch_window_simt(const WindowArgs& x, cudaStream_t st) {
  const sa_window_shape& s = x.shape;
  const SimtArgs a{x.q, x.k, x.v, x.out, x.lse, x.q_len, x.kv_len, x.status, s.Nq, s.Nk, x.window, x.sinks,
                   ceil_div(s.Nq, kRows), (int32_t)s.Hq, (int32_t)s.Hkv, (int32_t)s.d, x.scale};
  return s.dtype == SA_FP32 ? launch_type<float>(a, s.B * s.Hq, st) : launch_type<uint16_t>(a, s.B * s.Hq, st);
}

}  // namespace sa
