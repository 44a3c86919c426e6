// Attention with a sliding window and first tokens that stay visible, on the
// CUDA cores: fp32, and bf16 head widths that have no tensor-core kernel.
//
// Mathematics: row i at position p = n_k - n_q + i sees key j iff j <= p, j < n_k
// and (window == 0 or p - j < window or j < sinks); o = sum 2^(c (s_j - m)) v_j / l
// with c = scale log2 e, the running maximum m of the raw scores and the running
// sum l.  The difference s_j - m is taken before the scaling, so its rounding is
// relative to the difference, not to the scores.
//
// Bound by the fp32 pipes (4 d flops a pair; three tf32 or six bf16 products of
// the legacy tensor instructions would take as long).  One CTA takes 16 rows of
// one query head; its W warps take every W-th tile of 32 keys that some of the rows
// see, each with its own running maximum, sum and O, and join them at the end: no
// block barrier in the loop, and few rows still use several warps.  A lane owns 4
// rows times 4 keys of S and 4 rows times d / 8 channels of O in registers, rows and
// keys interleaved so that a warp's 4 row groups and 8 key groups each read one
// wavefront of shared memory: 8 wavefronts feed 64 multiply-adds a lane.  K and then
// V of a tile go through one buffer a warp; 16 warps an SM (d = 64) cover its
// latency.  2 x 1000 rows, 8 heads, d = 64, window 256: 57 us (64 x 64 tiles of a
// block, and 32 x 32 tiles with 8 rows a lane and two buffers, 80: 8 warps an SM
// leave the pipes idle half the time).
#include "sa_internal.cuh"

namespace sa {
namespace {

constexpr int kKeys = 32, kPs = kKeys + 4;
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

// Two fp32 numbers in one register pair: one instruction for two multiply-adds.
__device__ __forceinline__ uint64_t two(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 split(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// 16 bytes of a row to shared memory as floats (zeros where !on), from `at` to `to`:
// fp32 by an asynchronous copy, which the caller waits for.
template <typename T>
__device__ __forceinline__ void move16(uint32_t to, const T* at, bool on) {
  if constexpr (sizeof(T) == 4) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(at), "r"(on ? 16 : 0) : "memory");
  } else {
    uint4 w = make_uint4(0, 0, 0, 0);
    if (on) w = __ldg(reinterpret_cast<const uint4*>(at));
    float f[8];
    unpack16(w, T{}, f);
#pragma unroll
    for (int e = 0; e < 8; e += 4)
      asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to + 4 * e), "f"(f[e]), "f"(f[e + 1]), "f"(f[e + 2]),
                   "f"(f[e + 3])
                   : "memory");
  }
}
// Rows r0 .. r0 + n - 1 of a [..][d] array as floats to shared memory, row stride
// d + 4 (16-byte reads of neighbouring rows then meet no bank twice), by threads i0,
// i0 + step, ..; rows that live() leaves out (of those relative to r0) come as zeros.
// all: none is left out.  Where whole rows make a step, a thread keeps its
// column and nothing is computed but two addresses: the general walk took a
// third of the kernel's instructions.
template <typename T, class Live>
__device__ __forceinline__ void load_rows(float* dst, const T* src, int64_t r0, int n, int d, int i0, int step, bool all,
                                          Live live) {
  constexpr int V = 16 / sizeof(T);
  const int per = d / V, dr = step / per, dc = step - dr * per;
  int r = i0 / per, c = i0 - r * per;
  const T* at = src + r0 * d + (int64_t)i0 * V;   // (rows follow one another)
  uint32_t to = (uint32_t)__cvta_generic_to_shared(dst + r * (d + 4)) + c * V * 4;
  const uint32_t dto = (step * V + dr * 4) * 4;   // 4 floats of padding a row
  if (all && dc == 0) {
#pragma unroll 4
    for (; r < n; r += dr) {
      move16<T>(to, at, true);
      at += step * V;
      to += dto;
    }
  } else {
    for (; r < n;) {
      const bool on = live(r);
      move16<T>(to, on ? at : src, on);
      at += step * V;
      to += dto;
      r += dr;
      c += dc;
      if (c >= per) {
        c -= per;
        ++r;
        to += 16;
      }
    }
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}
__device__ __forceinline__ void wait_rows() {
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncwarp();
}

// RT: rows of a lane, every fourth of the tile's; CW: blocks of 32 channels (d <= 32 CW); W: warps.
template <typename T, int RT, int CW, int W>
__global__ void __launch_bounds__(32 * W, (CW <= 2 ? 16 : CW == 4 ? 12 : 8) / W) window_simt_kernel(const __grid_constant__ SimtArgs a) {
  constexpr int ROWS = 4 * RT, kThreads = 32 * W;
  extern __shared__ __align__(16) float smf[];
  const int d = a.d, ds = d + 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tx = lane & 7, ty = lane >> 3;
  float* qs = smf;
  float* const ks = qs + ROWS * ds + warp * (kKeys * ds + ROWS * kPs);   // this warp's K, then V, and P
  float* const ps = ks + kKeys * ds;
  const int64_t bh = blockIdx.x / a.row_tiles, row0 = (blockIdx.x - bh * a.row_tiles) * ROWS;
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

  const int64_t first = n_k - n_q + row0;                         // position of the tile's first row
  const int64_t last = n_k - n_q + min64(n_q, row0 + ROWS) - 1;   // and of its last
  const int64_t hi = max64(0, min64(n_k, last + 1));
  const int64_t lo = min64(a.window > 0 ? max64(0, first - a.window + 1) : 0, hi);
  const int64_t n_sink = min64(a.sinks, lo);
  const int sink_tiles = (int)ceil_div_d(n_sink, kKeys);
  const int64_t t_lo = max64(sink_tiles, lo / kKeys);
  const int tiles = (int)(sink_tiles + max64(0, ceil_div_d(hi, kKeys) - t_lo));
  auto key0 = [&](int t) { return (t < sink_tiles ? t : t_lo + (t - sink_tiles)) * kKeys; };
  // The tile's rows of K or V, zeros for keys that no row sees.
  auto load_tile = [&](const T* src, int64_t k0) {
    const int a1 = (int)min64(n_sink - k0, kKeys), b0 = (int)min64(lo - k0, kKeys), b1 = (int)min64(hi - k0, kKeys);
    load_rows<T>(ks, src, k0, kKeys, d, lane, 32, b1 == kKeys && (b0 <= 0 || a1 == kKeys),
                 [&](int r) { return r < b1 && (r >= b0 || r < a1); });
  };

  load_rows<T>(qs, q, row0, ROWS, d, threadIdx.x, kThreads, row0 + ROWS <= n_q, [&](int r) { return row0 + r < n_q; });
  if (warp < tiles) load_tile(k, key0(warp));
  wait_rows();
  __syncthreads();   // (Q; the only one before the join)
  uint64_t o[RT][2 * CW];   // channel pairs
  float m[RT], l[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int e = 0; e < 2 * CW; ++e) o[i][e] = 0;
  }
  const float c2 = a.scale * kLog2e;
  for (int t = warp; t < tiles; t += W) {
    const int64_t k0 = key0(t);
    if (t != warp) wait_rows();
    uint64_t s2[RT][4];   // sums over even and odd channels
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s2[i][j] = 0;
#pragma unroll 2
    for (int c = 0; c < d; c += 4) {
      ulonglong2 kk[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) kk[j] = *reinterpret_cast<const ulonglong2*>(ks + (tx + 8 * j) * ds + c);
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(qs + (ty + 4 * i) * ds + c);
#pragma unroll
        for (int j = 0; j < 4; ++j) s2[i][j] = fma2(x.x, kk[j].x, s2[i][j]);
#pragma unroll
        for (int j = 0; j < 4; ++j) s2[i][j] = fma2(x.y, kk[j].y, s2[i][j]);
      }
    }
    __syncwarp();
    load_tile(v, k0);
    const bool whole = k0 + kKeys - 1 <= first && (a.window == 0 || last - k0 < a.window || k0 + kKeys <= a.sinks);
    // (positions relative to the tile; a valid row's is below n_k)
    const int p0 = (int)(first - k0) + ty, c_s = (int)min64(a.sinks - k0, kKeys);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      float s[4], mx = m[i];
      const int c_hi = p0 + 4 * i, c_lo = a.window ? c_hi - (int)a.window + 1 : 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = split(s2[i][j]);
        s[j] = f.x + f.y;
        const int x = tx + 8 * j;
        if (!whole && (x > c_hi || (x < c_lo && x >= c_s))) s[j] = -INFINITY;
        mx = fmaxf(mx, s[j]);
      }
#pragma unroll
      for (int w = 1; w < 8; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      const float ref = mx == -INFINITY ? 0.f : mx;
      if (__any_sync(0xffffffffu, mx != m[i])) {
        const float corr = ex2((m[i] - ref) * c2);
        const uint64_t corr2 = two(corr, corr);
        l[i] *= corr;
#pragma unroll
        for (int e = 0; e < 2 * CW; ++e) o[i][e] = mul2(o[i][e], corr2);
      }
      m[i] = mx;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float pr = ex2((s[j] - ref) * c2);
        l[i] += pr;
        ps[(ty + 4 * i) * kPs + tx + 8 * j] = pr;
      }
    }
    wait_rows();   // V, and P
#pragma unroll 2
    for (int j = 0; j < kKeys; j += 4) {
      float4 pr[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i) pr[i] = *reinterpret_cast<const float4*>(ps + (ty + 4 * i) * kPs + j);
#pragma unroll
      for (int w = 0; w < CW; ++w) {
        const int ch = tx * 4 + 32 * w;
        if (ch >= d) break;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const ulonglong2 vv = *reinterpret_cast<const ulonglong2*>(ks + (j + x) * ds + ch);
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            const float px = x == 0 ? pr[i].x : x == 1 ? pr[i].y : x == 2 ? pr[i].z : pr[i].w;
            const uint64_t p2 = two(px, px);
            o[i][2 * w] = fma2(p2, vv.x, o[i][2 * w]);
            o[i][2 * w + 1] = fma2(p2, vv.y, o[i][2 * w + 1]);
          }
        }
      }
    }
    __syncwarp();
    if (t + W < tiles) load_tile(k, key0(t + W));
  }
  // Each warp's part over its K and P: O [ROWS][d + 4] and, behind it, m and l.
  __syncwarp();
#pragma unroll
  for (int i = 0; i < RT; ++i) {
#pragma unroll
    for (int w = 1; w < 8; w <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
#pragma unroll
    for (int w = 0; w < CW; ++w)
      if (tx * 4 + 32 * w < d)
        *reinterpret_cast<ulonglong2*>(ks + (ty + 4 * i) * ds + tx * 4 + 32 * w) = make_ulonglong2(o[i][2 * w], o[i][2 * w + 1]);
    if (tx == 0) {
      ps[ty + 4 * i] = m[i];
      ps[ROWS + ty + 4 * i] = l[i];
    }
  }
  __syncthreads();
  const int stride = kKeys * ds + ROWS * kPs;   // from one warp's part to the next
  const float* part = smf + ROWS * ds;
  for (int i = threadIdx.x; i < ROWS * (d / 4); i += kThreads) {
    const int r = i / (d / 4), ch = (i - r * (d / 4)) * 4;
    const int64_t row = row0 + r;
    if (row >= n_q) continue;
    const float* ml = part + kKeys * ds + r;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < W; ++w) top = fmaxf(top, ml[w * stride]);
    const float ref = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float g = ex2((ml[w * stride] - ref) * c2);
      const float4 x = *reinterpret_cast<const float4*>(part + w * stride + r * ds + ch);
      sum = fmaf(g, ml[w * stride + ROWS], sum);
      y.x = fmaf(g, x.x, y.x);
      y.y = fmaf(g, x.y, y.y);
      y.z = fmaf(g, x.z, y.z);
      y.w = fmaf(g, x.w, y.w);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;   // no visible key: zeros; NaN stays
    T* dst = static_cast<T*>(a.out) + (bh * a.Nq + row) * d + ch;
    Elem<T>::store(dst, y.x * inv);
    Elem<T>::store(dst + 1, y.y * inv);
    Elem<T>::store(dst + 2, y.z * inv);
    Elem<T>::store(dst + 3, y.w * inv);
    if (ch == 0 && a.lse) a.lse[bh * a.Nq + row] = sum == 0.f ? -INFINITY : fmaf(top, a.scale, logf(sum));
  }
}

template <typename T, int RT, int CW, int W>
sa_status launch(SimtArgs& a, int64_t heads, cudaStream_t st) {
  constexpr int ROWS = 4 * RT, kThreads = 32 * W;
  static_assert(ROWS <= kKeys, "a warp's part of O lies over its K");
  const size_t smem = (size_t)(ROWS * (a.d + 4) + W * (kKeys * (a.d + 4) + ROWS * kPs)) * sizeof(float);
  if (cudaFuncSetAttribute(window_simt_kernel<T, RT, CW, W>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
      cudaSuccess)
    return set_error(SA_ERR_CUDA, "cudaFuncSetAttribute(window_simt_kernel) failed");
  a.row_tiles = ceil_div(a.Nq, ROWS);
  const int64_t ctas = heads * a.row_tiles;
  if (ctas > INT32_MAX) return set_error(SA_ERR_UNSUPPORTED, "too many rows");
  window_simt_kernel<T, RT, CW, W><<<(unsigned)ctas, kThreads, smem, st>>>(a);
  return check_launch("window_simt_kernel");
}

// Two warps share a query tile; four where there are too few tiles for the GPU.
template <typename T, int RT, int CW>
sa_status launch_warps(SimtArgs& a, int64_t heads, cudaStream_t st) {
  return heads * ceil_div(a.Nq, 4 * RT) >= 148 * 4 ? launch<T, RT, CW, 2>(a, heads, st) : launch<T, RT, CW, 4>(a, heads, st);
}

template <typename T>
sa_status launch_type(SimtArgs& a, int64_t heads, cudaStream_t st) {
  if (a.d <= 32) return launch_warps<T, 4, 1>(a, heads, st);
  if (a.d <= 64) return launch_warps<T, 4, 2>(a, heads, st);
  if (a.d <= 128) return launch_warps<T, 4, 4>(a, heads, st);
  return launch_warps<T, 4, 8>(a, heads, st);
}

}  // namespace

sa_status launch_window_simt(const WindowArgs& x, cudaStream_t st) {
  const sa_window_shape& s = x.shape;
  SimtArgs a{x.q,  x.k,      x.v,     x.out, x.lse,          x.q_len,         x.kv_len,     x.status, s.Nq,
             s.Nk, x.window >= s.Nk ? 0 : x.window, x.sinks, 0, (int32_t)s.Hq, (int32_t)s.Hkv, (int32_t)s.d, x.scale};
  return s.dtype == SA_FP32 ? launch_type<float>(a, s.B * s.Hq, st) : launch_type<uint16_t>(a, s.B * s.Hq, st);
}

}  // namespace sa
