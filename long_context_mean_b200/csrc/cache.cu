// The paged 4-bit cache: block tables and slot maps from request lengths, and
// the rows' quantisation, storing and reading back.
//
// Codes: 32 neighbouring channels of one token and head share one bf16 scale
// s = bf16(amax / 7); the code of x is rint(x / s) in [-7, 7], held as code + 8
// in 4 bits.  x and s have 8 significant bits, so x / s rounded to 24 bits
// falls on the same side of every rounding border as the exact quotient: the
// codes are those of exact arithmetic.  A group with an infinity or a NaN gets
// a NaN scale, so that it reads back as NaN.
//
// A subtile is 16 tokens of one head, 576 * d / 32 bytes in one piece, in the
// order in which the attention kernel's matrix fragments are filled:
//   K codes   [token][q4][g][j]      channel 32 g + 8 q4 + j, 4 bits each
//   V codes   [p][c8][t4][g][hi][i]  channel 32 g + 4 c8 + i, token 8 p + 2 t4 + hi
//   K scales  [token][g], V scales [p][t4][g][hi]
// so a lane fills its operands with 16-byte shared-memory loads, and a V word
// holds two tokens whose codes meet in one register without a permute.
#include "sa_internal.cuh"

namespace sa {
namespace {

// ---------------------------------------------------------------------------
// Append and read
// ---------------------------------------------------------------------------
struct RowArgs {
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* ko;
  uint16_t* vo;
  int64_t ks[2], vs[2];     // element strides: token, head
  const int32_t* slots;
  uint8_t* cache;
  int32_t* status;
  int64_t T, slots_all;
  int32_t H, lg_page;
};

template <int G>
struct Place {   // byte offsets of four channels 4 c4 .. 4 c4 + 3 of a token
  int64_t base;
  int k, v, ks, vs;
  __device__ __forceinline__ Place(int64_t slot, int lg_page, int H, int h, int c4) {
    const int64_t page = slot >> lg_page;
    const int in = (int)(slot & ((1 << lg_page) - 1)), t = in & 15;
    base = (((page * H + h) << (lg_page - 4)) + (in >> 4)) * (576 * G);
    const int g = c4 >> 3, r = c4 & 7, p = t >> 3, t4 = (t & 7) >> 1, hi = t & 1;
    k = t * 16 * G + (r >> 1) * 4 * G + g * 4 + (r & 1) * 2;
    v = 256 * G + p * 128 * G + (r * 4 + t4) * 4 * G + g * 4 + hi * 2;
    ks = 512 * G + t * 2 * G + g * 2;
    vs = 544 * G + p * 16 * G + t4 * 4 * G + g * 4 + hi * 2;
  }
};

__device__ __forceinline__ uint32_t abs_max4(uint2 x) {
  return max(max(x.x & 0x7FFFu, (x.x >> 16) & 0x7FFFu), max(x.y & 0x7FFFu, (x.y >> 16) & 0x7FFFu));
}
// Scale of a group from the largest |x| (as bf16 bits, equal in the group's 8 lanes).
__device__ __forceinline__ uint16_t group_scale(uint32_t amax_bits) {
  if (amax_bits >= 0x7F80u) return 0x7FC0u;
  return f32_to_bf16_rne(__fdiv_rn(__uint_as_float(amax_bits << 16), 7.0f));
}
__device__ __forceinline__ uint32_t code4(uint2 x, uint16_t scale) {
  const float s = bf16_to_f32(scale);
  if (!(s > 0.f)) return 0x8888u;   // zero or NaN scale
  const uint32_t w[2] = {x.x, x.y};
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float f = __uint_as_float((i & 1) ? (w[i >> 1] & 0xFFFF0000u) : (w[i >> 1] << 16));
    // (a subnormal scale is coarse: the quotient may pass 7, hence the clamp)
    const int q = max(-7, min(7, __float2int_rn(__fdiv_rn(f, s))));
    r |= (uint32_t)(q + 8) << (4 * i);
  }
  return r;
}
__device__ __forceinline__ uint2 values4(uint32_t codes, uint16_t scale) {
  const float s = bf16_to_f32(scale);
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float a = (float)((int)((codes >> (8 * i)) & 15u) - 8) * s;
    const float b = (float)((int)((codes >> (8 * i + 4)) & 15u) - 8) * s;
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    w[i] = *reinterpret_cast<uint32_t*>(&h);
  }
  return make_uint2(w[0], w[1]);
}

// One thread per (token, head, 4 channels); 8 neighbouring lanes share a
// group.  WRITE: quantise and store; otherwise read back.
template <int G, bool WRITE>
__global__ void __launch_bounds__(256) kv4_rows_kernel(const __grid_constant__ RowArgs a) {
  constexpr int C4 = 8 * G;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int c4 = (int)(i % C4);
  const int64_t th = i / C4;
  const int64_t t = th / a.H;
  const int h = (int)(th - t * a.H);
  const bool in = t < a.T;   // a group's 8 lanes agree
  const int64_t slot = in ? a.slots[t] : -1;
  const bool live = slot >= 0 && slot < a.slots_all;
  if (in && !live && slot != -1) raise_status(a.status, SA_ERR_INVALID_ARG);
  const Place<G> at(live ? slot : 0, a.lg_page, a.H, h, c4);
  uint8_t* p = a.cache + at.base;
  if constexpr (WRITE) {
    uint2 k = make_uint2(0, 0), v = k;
    if (live) {
      k = __ldg(reinterpret_cast<const uint2*>(a.k + t * a.ks[0] + h * a.ks[1] + c4 * 4));
      v = __ldg(reinterpret_cast<const uint2*>(a.v + t * a.vs[0] + h * a.vs[1] + c4 * 4));
    }
    uint32_t m = abs_max4(k), n = abs_max4(v);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      n = max(n, __shfl_xor_sync(0xffffffffu, n, o));
    }
    const uint16_t sk = group_scale(m), sv = group_scale(n);
    if (!live) return;
    *reinterpret_cast<uint16_t*>(p + at.k) = (uint16_t)code4(k, sk);
    *reinterpret_cast<uint16_t*>(p + at.v) = (uint16_t)code4(v, sv);
    if ((c4 & 7) == 0) {
      *reinterpret_cast<uint16_t*>(p + at.ks) = sk;
      *reinterpret_cast<uint16_t*>(p + at.vs) = sv;
    }
  } else {
    if (!live) return;
    const uint2 k = values4(*reinterpret_cast<const uint16_t*>(p + at.k), *reinterpret_cast<const uint16_t*>(p + at.ks));
    const uint2 v = values4(*reinterpret_cast<const uint16_t*>(p + at.v), *reinterpret_cast<const uint16_t*>(p + at.vs));
    *reinterpret_cast<uint2*>(a.ko + t * a.ks[0] + h * a.ks[1] + c4 * 4) = k;
    *reinterpret_cast<uint2*>(a.vo + t * a.vs[0] + h * a.vs[1] + c4 * 4) = v;
  }
}

int log2i(int64_t x) {
  int r = 0;
  while ((1LL << r) < x) ++r;
  return r;
}

template <bool WRITE>
sa_status launch_rows(RowArgs& a, const sa_kv4_desc& d, cudaStream_t st) {
  const int64_t threads = a.T * d.Hkv * (d.d / 4);
  const int64_t ctas = ceil_div(threads, 256);
  if (ctas == 0) return SA_OK;
  if (ctas > 2147483647) return set_error(SA_ERR_UNSUPPORTED, "too many rows");
  a.H = (int32_t)d.Hkv;
  a.lg_page = log2i(d.page);
  a.slots_all = d.num_pages * d.page;
  if (d.d == 128)
    kv4_rows_kernel<4, WRITE><<<(unsigned)ctas, 256, 0, st>>>(a);
  else
    kv4_rows_kernel<2, WRITE><<<(unsigned)ctas, 256, 0, st>>>(a);
  return check_launch("kv4_rows_kernel");
}

// ---------------------------------------------------------------------------
// Block tables and slot maps
// ---------------------------------------------------------------------------
// Every CTA scans the requests' lengths by itself (three running sums: tokens,
// fresh pages, released pages) and then takes its share of the outputs, so the
// CTAs exchange nothing and one launch does it all.  The page that a fresh
// block takes is a position on the free stack, and a position above the old top
// is a released page, read from the ended request's row of the table; rows of
// ended requests and entries below a request's held blocks are never written.
constexpr int kPlanThreads = 512;

struct PlanArgs {
  const int32_t* kv_len;
  const int32_t* q_len;
  int32_t* table;
  int32_t* free_list;
  const int32_t* free_in;
  int32_t* free_out;
  int32_t* new_len;
  int32_t* cu_q;
  int32_t* slots;
  int32_t* positions;
  int32_t* status;
  int64_t max_tokens;
  int32_t B, max_blocks, num_pages, lg_page, per;   // per: requests per thread
};

__device__ __forceinline__ int blocks_of(int64_t n, int lg) { return (int)((n + (1 << lg) - 1) >> lg); }

// Largest i in [0, n) with pre[i] <= x (pre ascending, pre[0] = 0).
__device__ __forceinline__ int find(const int32_t* pre, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ PlanArgs a) {
  extern __shared__ int32_t sm[];
  int32_t* tok = sm;                 // [B + 1] running sums
  int32_t* fresh = tok + a.B + 1;
  int32_t* gone = fresh + a.B + 1;
  __shared__ int64_t part[3][kPlanThreads / 32];
  __shared__ int32_t bad, bad_code;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    bad = 0;
    bad_code = 0;
  }
  __syncthreads();
  const int b0 = min(a.B, tid * a.per), b1 = min(a.B, b0 + a.per);
  int64_t s[3] = {0, 0, 0};
  for (int b = b0; b < b1; ++b) {
    const int64_t old = a.kv_len[b], add = a.q_len[b];
    const int64_t most = (int64_t)a.max_blocks << a.lg_page;
    if (old < 0 || add < -1 || old > most) {
      atomicExch(&bad, 1);
      atomicCAS(&bad_code, 0, SA_ERR_INVALID_ARG);
      continue;
    }
    if (add > 0 && old + add > most) {
      atomicExch(&bad, 1);
      atomicCAS(&bad_code, 0, SA_ERR_CAPACITY);
      continue;
    }
    const int held = blocks_of(old, a.lg_page);
    if (add < 0) {
      s[2] += held;
    } else {
      s[0] += add;
      s[1] += blocks_of(old + add, a.lg_page) - held;
    }
  }
  // exclusive scan over the threads
  int64_t x[3];
#pragma unroll
  for (int c = 0; c < 3; ++c) {
    int64_t v = s[c];
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (lane == 31) part[c][warp] = v;
    x[c] = v - s[c];
  }
  __syncthreads();
  int64_t total[3] = {0, 0, 0};
#pragma unroll
  for (int c = 0; c < 3; ++c)
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      if (w == warp) x[c] += total[c];
      total[c] += part[c][w];
    }
  const int64_t count = *a.free_in;
  if (tid == 0) {
    int code = 0;
    if (count < 0 || count > a.num_pages) code = SA_ERR_INVALID_ARG;
    else if (count + total[2] > a.num_pages) code = SA_ERR_INVALID_ARG;   // more pages than there are
    else if (total[1] > count + total[2]) code = SA_ERR_CAPACITY;
    else if (total[0] > a.max_tokens) code = SA_ERR_CAPACITY;
    if (code && !bad) {
      bad = 1;
      bad_code = code;
    }
  }
  __syncthreads();
  const int64_t gtid = (int64_t)blockIdx.x * kPlanThreads + tid, gsize = (int64_t)gridDim.x * kPlanThreads;
  if (bad) {   // nothing is planned and nothing changes hands
    if (gtid == 0) {
      raise_status(a.status, bad_code);
      *a.free_out = (int32_t)count;
    }
    for (int64_t b = gtid; b <= a.B; b += gsize) {
      a.cu_q[b] = 0;
      if (b < a.B) a.new_len[b] = a.kv_len[b];
    }
    for (int64_t t = gtid; t < a.max_tokens; t += gsize) {
      a.slots[t] = -1;
      a.positions[t] = 0;
    }
    return;
  }
  for (int b = b0; b < b1; ++b) {
    tok[b] = (int32_t)x[0];
    fresh[b] = (int32_t)x[1];
    gone[b] = (int32_t)x[2];
    const int64_t old = a.kv_len[b], add = a.q_len[b];
    const int held = blocks_of(old, a.lg_page);
    if (add < 0) {
      x[2] += held;
    } else {
      x[0] += add;
      x[1] += blocks_of(old + add, a.lg_page) - held;
    }
  }
  if (tid == 0) {
    tok[a.B] = (int32_t)total[0];
    fresh[a.B] = (int32_t)total[1];
    gone[a.B] = (int32_t)total[2];
  }
  __syncthreads();
  const int n_tok = (int)total[0], n_fresh = (int)total[1], n_gone = (int)total[2];
  const int64_t top = count + n_gone;
  auto released = [&](int r) {   // the r-th released page
    const int b = find(gone, a.B, r);
    return a.table[(int64_t)b * a.max_blocks + (r - gone[b])];
  };
  auto taken = [&](int f) -> int32_t {   // the page of the f-th fresh block
    const int64_t at = top - 1 - f;
    const int32_t page = at >= count ? released((int)(at - count)) : a.free_list[at];
    if (page < 0 || page >= a.num_pages) {
      raise_status(a.status, SA_ERR_INVALID_ARG);
      return -1;
    }
    return page;
  };
  for (int64_t t = gtid; t < a.max_tokens; t += gsize) {
    int32_t slot = -1, pos = 0;
    if (t < n_tok) {
      const int b = find(tok, a.B, (int)t);
      const int64_t old = a.kv_len[b];
      pos = (int32_t)(old + (t - tok[b]));
      const int blk = pos >> a.lg_page, held = blocks_of(old, a.lg_page);
      int32_t page = blk < held ? a.table[(int64_t)b * a.max_blocks + blk] : taken(fresh[b] + blk - held);
      if (page < 0 || page >= a.num_pages) {
        raise_status(a.status, SA_ERR_INVALID_ARG);
        page = -1;
      }
      if (page >= 0) slot = (page << a.lg_page) + (pos & ((1 << a.lg_page) - 1));
    }
    a.slots[t] = slot;
    a.positions[t] = pos;
  }
  for (int64_t f = gtid; f < n_fresh; f += gsize) {
    const int b = find(fresh, a.B, (int)f);
    const int held = blocks_of(a.kv_len[b], a.lg_page);
    a.table[(int64_t)b * a.max_blocks + held + (f - fresh[b])] = taken((int)f);
  }
  for (int64_t r = gtid; r < n_gone; r += gsize) {
    const int32_t page = released((int)r);
    if (page < 0 || page >= a.num_pages) raise_status(a.status, SA_ERR_INVALID_ARG);
    a.free_list[count + r] = page;
  }
  for (int64_t b = gtid; b <= a.B; b += gsize) {
    a.cu_q[b] = tok[b];
    if (b < a.B) a.new_len[b] = a.q_len[b] < 0 ? 0 : a.kv_len[b] + a.q_len[b];
  }
  if (gtid == 0) *a.free_out = (int32_t)(top - n_fresh);
}

}  // namespace

sa_status launch_kv4_append(const void* k, const void* v, int64_t T, const int64_t* ks, const int64_t* vs,
                            const int32_t* slots, const sa_kv4_desc& d, void* cache, int32_t* status, cudaStream_t st) {
  RowArgs a{};
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  for (int i = 0; i < 2; ++i) {
    a.ks[i] = ks[i];
    a.vs[i] = vs[i];
  }
  a.slots = slots;
  a.cache = static_cast<uint8_t*>(cache);
  a.status = status;
  a.T = T;
  return launch_rows<true>(a, d, st);
}

sa_status launch_kv4_read(const void* cache, const sa_kv4_desc& d, const int32_t* slots, int64_t T, void* k, void* v,
                          int32_t* status, cudaStream_t st) {
  RowArgs a{};
  a.ko = static_cast<uint16_t*>(k);
  a.vo = static_cast<uint16_t*>(v);
  a.ks[0] = a.vs[0] = d.Hkv * d.d;
  a.ks[1] = a.vs[1] = d.d;
  a.slots = slots;
  a.cache = const_cast<uint8_t*>(static_cast<const uint8_t*>(cache));
  a.status = status;
  a.T = T;
  return launch_rows<false>(a, d, st);
}

size_t plan_smem(int64_t B) { return (size_t)3 * (B + 1) * sizeof(int32_t); }

sa_status launch_plan(const int32_t* kv_len, const int32_t* q_len, const sa_plan_desc& d, int32_t* table,
                      int32_t* free_list, const int32_t* free_in, int32_t* free_out, int32_t* new_len, int32_t* cu_q,
                      int32_t* slots, int32_t* positions, int32_t* status, cudaStream_t st) {
  PlanArgs a{kv_len,    q_len,   table,  free_list, free_in,       free_out,
             new_len,   cu_q,    slots,  positions, status,        d.max_tokens,
             (int32_t)d.B, (int32_t)d.max_blocks, (int32_t)d.num_pages, log2i(d.page),
             (int32_t)ceil_div(d.B, kPlanThreads)};
  const size_t smem = plan_smem(d.B);
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return set_error(SA_ERR_CUDA, "cudaFuncSetAttribute(plan_kernel) failed");
  // One CTA per 2048 outputs: every CTA repeats the scan, so more of them only
  // pay once there is that much to write.
  const int64_t want = ceil_div(max64(d.max_tokens, d.B), 4 * kPlanThreads);
  plan_kernel<<<(unsigned)min64(want, 148), kPlanThreads, smem, st>>>(a);
  return check_launch("plan_kernel");
}

}  // namespace sa
