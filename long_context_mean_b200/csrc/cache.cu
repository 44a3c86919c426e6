// The paged 4-bit cache: block tables and slot maps from request lengths, and
// the rows' quantisation, storing and reading back.
//
// Codes: 32 neighbouring channels of one token and head share one bf16 scale
// s = bf16(amax / 7); the code of x is rint(x / s) in [-7, 7], held as code + 8
// in 4 bits; the codes are those of exact arithmetic (code8).  A group with an
// infinity or a NaN gets a NaN scale, so that it reads back as NaN.
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
  int32_t H, lg_page, each;
  int32_t wide;             // the rows lie on 16-byte boundaries (else 8)
};
__device__ __forceinline__ uint4 load8(const uint16_t* p) {
  const uint2 a = __ldg(reinterpret_cast<const uint2*>(p)), b = __ldg(reinterpret_cast<const uint2*>(p + 4));
  return make_uint4(a.x, a.y, b.x, b.y);
}

// Byte offsets of a token's 8 channels 8 cc .. 8 cc + 7.
template <int G>
struct Place {
  int64_t base;
  int k, v, ks, vs;   // K's 4 bytes; V's first 2 bytes (tokens of a pair lie side by side, the next 4 channels 16 G on)
  __device__ __forceinline__ Place(int slot, int lg_page, int H, int h, int cc) {
    const int in = slot & ((1 << lg_page) - 1), t = in & 15;
    base = ((((int64_t)(slot >> lg_page) * H + h) << (lg_page - 4)) + (in >> 4)) * (576 * G);
    const int g = cc >> 2, q4 = cc & 3, p = t >> 3, t4 = (t & 7) >> 1, hi = t & 1;
    k = t * 16 * G + q4 * 4 * G + g * 4;
    v = 256 * G + p * 128 * G + (2 * q4 * 4 + t4) * 4 * G + g * 4 + hi * 2;
    ks = 512 * G + t * 2 * G + g * 2;
    vs = 544 * G + p * 16 * G + t4 * 4 * G + g * 4 + hi * 2;
  }
};

// The largest |x| of 8 values as bf16 bits, of the even and the odd ones.
__device__ __forceinline__ uint32_t abs_max8(const uint4& x) {
  constexpr uint32_t M = 0x7FFF7FFFu;
  return __vmaxu2(__vmaxu2(x.x & M, x.y & M), __vmaxu2(x.z & M, x.w & M));
}
// Scale of a group from the largest |x| (as bf16 bits, equal in the group's 4 lanes).
__device__ __forceinline__ uint16_t group_scale(uint32_t amax_bits) {
  // (A product: amax / 7 is never a tie of bf16, whose odd 9-bit numbers times 7 do
  // not fit amax's 8 bits, and at least 2^-12 relative away from one.)
  if (amax_bits >= 0x7F80u) return 0x7FC0u;
  return f32_to_bf16_rne(__uint_as_float(amax_bits << 16) * (1.0f / 7.0f));
}
__device__ __forceinline__ float reciprocal(float x) {   // to an ulp, for normal results
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// rint(x / s) + 8 of 8 values, 4 bits each, without dividing each: x and s have 8
// significant bits, so a quotient of 1/2 or more that is not a half integer is at
// least 1 / 2040 away from one, and x times 1 / s is off by 2^-20 at most.
// Rounded to multiples of 2^-12 it is therefore a half integer exactly where the
// true quotient is, and on the same side of it elsewhere.
__device__ __forceinline__ uint32_t code8(const uint4& x, uint16_t scale) {
  const float s = bf16_to_f32(scale);
  if (!(s > 0.f)) return 0x88888888u;   // zero or NaN scale
  float f[8];
  unpack16(x, uint16_t{}, f);
  float inv;
  if (s < 0x1p-60f) {
    // Room for the reciprocal; a subnormal scale is coarse, and the quotient may pass 7.
    const float up = s * 0x1p64f, top = 7.f * up;
    inv = reciprocal(up);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = fminf(fmaxf(f[i] * 0x1p64f, -top), top);
  } else {
    inv = reciprocal(s);
  }
  // 1.5 2^11: multiples of 2^-12; 1.5 2^23 + 8: integers, with code + 8 in the low
  // bits.  The words w = 16 w + bits gather the codes and 8 times kOne's bits.
  constexpr float kGrid = 0x1.8p11f, kOne = 0x1.8p23f + 8.f;
  constexpr uint32_t kBits = 0x4B400000u * 0x11111111u;
  uint32_t w = 0;
#pragma unroll
  for (int i = 7; i >= 0; --i) w = w * 16 + __float_as_uint((fmaf(f[i], inv, kGrid) - kGrid) + kOne);
  return w - kBits;
}
// The 8 values of a word of codes, rounded to bf16: 128 + nibble by an AND-OR, two
// channels a register, less 136, times the scale.
__device__ __forceinline__ uint4 values8(uint32_t codes, uint16_t scale) {
  const uint32_t s2 = scale * 0x00010001u;
  uint32_t v[4];   // channels i and i + 4
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x = ((codes >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
    const __nv_bfloat162 c = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&x), __floats2bfloat162_rn(136.f, 136.f));
    const __nv_bfloat162 y = __hmul2(c, *reinterpret_cast<const __nv_bfloat162*>(&s2));
    v[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
  return make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410), __byte_perm(v[0], v[1], 0x7632),
                    __byte_perm(v[2], v[3], 0x7632));
}

// A warp takes two neighbouring tokens (half warps) and 16 of their chunks of 8
// channels; 4 neighbouring lanes share a group.  Where the two tokens are a pair
// of the cache too (slots 2 n and 2 n + 1, as in every run of tokens), their V
// codes and scales, which lie side by side, are exchanged between the halves and move
// as 4 bytes, and with 16-byte rows on the other side one access a lane is left of
// each.  The bytes alone would take 13 us for 16,411 tokens of 8 heads of 128; bound
// by the instructions of the rounding and packing (86% and 73% of the issue slots):
// 21 us to store, 17 us to read.  WRITE: quantise and store; otherwise read back.
// A warp walks a.each blocks of chunks of its tokens.
template <int G, bool WRITE>
__global__ void __launch_bounds__(256) kv4_rows_kernel(const __grid_constant__ RowArgs a) {
  constexpr int CH = 4 * G, HEADS = 16 / CH;   // heads of a block of 16 chunks
  const int lane = threadIdx.x & 31, half = lane >> 4;
  const uint32_t per = (uint32_t)((a.H + HEADS - 1) / HEADS + a.each - 1) / a.each;   // warps of two tokens
  const uint32_t warp = blockIdx.x * 8 + (threadIdx.x >> 5), pair_no = warp / per;
  const int64_t t = (int64_t)pair_no * 2 + half;
  int h = (int)(warp - pair_no * per) * a.each * HEADS + (lane & 15) / CH;
  const int cc = lane & (CH - 1);
  const int slot = t < a.T ? a.slots[t] : -1;
  const bool live = slot >= 0 && slot < a.slots_all;
  if (!live && slot != -1) raise_status(a.status, SA_ERR_INVALID_ARG);
  const int mate = __shfl_xor_sync(0xffffffffu, live ? slot : -2, 16);
  const bool pair = live && mate == slot + (half ? -1 : 1) && (slot & 1) == half;
  if (pair_no * 2 >= a.T) return;   // (whole warps)
  const Place<G> at(live ? slot : 0, a.lg_page, a.H, h, cc);
  constexpr int NEXT = 16 * G;   // V's next 4 channels
  uint8_t* p = a.cache + at.base;
  const uint8_t* p_in = p;
  // The first half warp moves the pair's first 4 channels of V, the second the next 4.
  const int at_v = pair && half ? at.v - 2 + NEXT : at.v;
  const uint16_t *k_in = a.k + t * a.ks[0] + h * a.ks[1] + cc * 8, *v_in = a.v + t * a.vs[0] + h * a.vs[1] + cc * 8;
  uint16_t *k_out = a.ko + t * a.ks[0] + h * a.ks[1] + cc * 8, *v_out = a.vo + t * a.vs[0] + h * a.vs[1] + cc * 8;
  // Each block's loads run while the one before is worked on.
  uint4 k2 = make_uint4(0, 0, 0, 0), v2 = k2;   // WRITE
  uint32_t kc2 = 0, mine2 = 0;                  // read
  uint16_t sk2 = 0, sv2r = 0;
  auto fetch = [&](int head) {
    if (!(live && head < a.H)) return;
    if constexpr (WRITE) {
      k2 = a.wide ? __ldg(reinterpret_cast<const uint4*>(k_in)) : load8(k_in);
      v2 = a.wide ? __ldg(reinterpret_cast<const uint4*>(v_in)) : load8(v_in);
      k_in += HEADS * a.ks[1];
      v_in += HEADS * a.vs[1];
    } else {
      kc2 = __ldg(reinterpret_cast<const uint32_t*>(p_in + at.k));
      sk2 = __ldg(reinterpret_cast<const uint16_t*>(p_in + at.ks));
      sv2r = __ldg(reinterpret_cast<const uint16_t*>(p_in + at.vs));
      if (pair)
        mine2 = __ldg(reinterpret_cast<const uint32_t*>(p_in + at_v));
      else
        mine2 = __ldg(reinterpret_cast<const uint16_t*>(p_in + at.v)) |
                (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(p_in + at.v + NEXT)) << 16;
      p_in += (int64_t)HEADS * (576 * G) << (a.lg_page - 4);
    }
  };
  fetch(h);
#pragma unroll 2
  for (int i = 0; i < a.each; ++i) {
    const bool on = live && h < a.H;   // a group's 4 lanes, and a pair's two, agree
    if constexpr (WRITE) {
      const uint4 k = k2, v = v2;
      if (i + 1 < a.each) fetch(h + HEADS);
      uint32_t m = abs_max8(k), n = abs_max8(v);
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
        n = __vmaxu2(n, __shfl_xor_sync(0xffffffffu, n, o));
      }
      const uint16_t sk = group_scale(max(m & 0xFFFFu, m >> 16)), sv = group_scale(max(n & 0xFFFFu, n >> 16));
      const uint32_t kc = code8(k, sk), vc = code8(v, sv);
      const uint32_t got = __shfl_xor_sync(0xffffffffu, half ? vc & 0xFFFFu : vc >> 16, 16);
      const uint32_t sv2 = __shfl_xor_sync(0xffffffffu, (uint32_t)sv, 16);
      if (on) {
        *reinterpret_cast<uint32_t*>(p + at.k) = kc;
        if ((cc & 3) == 0) *reinterpret_cast<uint16_t*>(p + at.ks) = sk;
        if (pair) {
          *reinterpret_cast<uint32_t*>(p + at_v) = half ? got | (vc & 0xFFFF0000u) : (vc & 0xFFFFu) | got << 16;
          if ((cc & 3) == 0 && !half) *reinterpret_cast<uint32_t*>(p + at.vs) = sv | sv2 << 16;
        } else {
          *reinterpret_cast<uint16_t*>(p + at.v) = (uint16_t)vc;
          *reinterpret_cast<uint16_t*>(p + at.v + NEXT) = (uint16_t)(vc >> 16);
          if ((cc & 3) == 0) *reinterpret_cast<uint16_t*>(p + at.vs) = sv;
        }
      }
      p += (int64_t)HEADS * (576 * G) << (a.lg_page - 4);
    } else {
      const uint32_t kc = kc2, mine = mine2;
      const uint16_t sk = sk2, sv = sv2r;
      if (i + 1 < a.each) fetch(h + HEADS);
      const uint32_t got = __shfl_xor_sync(0xffffffffu, half ? mine & 0xFFFFu : mine >> 16, 16);
      if (on) {
        const uint32_t vc = !pair ? mine : half ? got | (mine & 0xFFFF0000u) : (mine & 0xFFFFu) | got << 16;
        *reinterpret_cast<uint4*>(k_out) = values8(kc, sk);
        *reinterpret_cast<uint4*>(v_out) = values8(vc, sv);
      }
      k_out += HEADS * a.ks[1];
      v_out += HEADS * a.vs[1];
    }
    h += HEADS;
  }
}

int log2i(int64_t x) {
  int r = 0;
  while ((1LL << r) < x) ++r;
  return r;
}

template <bool WRITE>
sa_status launch_rows(RowArgs& a, const sa_kv4_desc& d, cudaStream_t st) {
  // Once two warps an SM sub-partition are there, a warp walks several heads.
  const int64_t blocks = ceil_div(d.Hkv * (d.d / 8), 16), pairs = ceil_div(a.T, 2);
  a.each = (int32_t)max64(1, min64(min64(blocks, 4), pairs * blocks / (148 * 8)));
  const int64_t ctas = ceil_div(pairs * ceil_div(blocks, a.each), 8);
  if (ctas == 0) return SA_OK;
  if (ctas > 2147483647 / 8) return set_error(SA_ERR_UNSUPPORTED, "too many rows");
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
constexpr int32_t kNone = INT32_MAX;   // no error

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
  __shared__ int32_t bad;   // the lowest code of what is wrong, whichever thread finds it first
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) bad = kNone;
  __syncthreads();
  const int64_t count = *a.free_in;   // (with the lengths, not after them)
  const int b0 = min(a.B, tid * a.per), b1 = min(a.B, b0 + a.per);
  int64_t s[3] = {0, 0, 0};
  for (int b = b0; b < b1; ++b) {
    const int64_t old = a.kv_len[b], add = a.q_len[b];
    const int64_t most = (int64_t)a.max_blocks << a.lg_page;
    if (old < 0 || add < -1 || old > most) {
      atomicMin(&bad, SA_ERR_INVALID_ARG);
      continue;
    }
    if (add > 0 && old + add > most) {
      atomicMin(&bad, SA_ERR_CAPACITY);
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
  if (tid == 0) {
    int code = kNone;
    if (count < 0 || count > a.num_pages) code = SA_ERR_INVALID_ARG;
    else if (count + total[2] > a.num_pages) code = SA_ERR_INVALID_ARG;   // more pages than there are
    else if (total[1] > count + total[2]) code = SA_ERR_CAPACITY;
    else if (total[0] > a.max_tokens) code = SA_ERR_CAPACITY;
    bad = min(bad, code);
  }
  __syncthreads();
  const int64_t gtid = (int64_t)blockIdx.x * kPlanThreads + tid, gsize = (int64_t)gridDim.x * kPlanThreads;
  auto refuse = [&](int32_t code) {   // nothing is planned and nothing changes hands
    if (gtid == 0) {
      raise_status(a.status, code);
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
  };
  if (bad != kNone) return refuse(bad);
  bool wrong = false;   // a page is outside the cache
  auto look = [&](int32_t page) { wrong |= page < 0 || page >= a.num_pages; };
  int32_t filled = 0;   // the page of a block that is filled up, looked at after the next load or the barrier
  for (int b = b0; b < b1; ++b) {
    tok[b] = (int32_t)x[0];
    fresh[b] = (int32_t)x[1];
    gone[b] = (int32_t)x[2];
    const int64_t old = a.kv_len[b], add = a.q_len[b];
    const int held = blocks_of(old, a.lg_page);
    look(filled);
    if (add > 0 && (old & ((1 << a.lg_page) - 1))) filled = a.table[(int64_t)b * a.max_blocks + held - 1];
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
    return at >= count ? released((int)(at - count)) : a.free_list[at];
  };
  // Every page that changes hands or takes a token is looked at before anything is
  // written: released ones, the free ones that are taken, blocks that are filled
  // up.  Each CTA looks at all of them (no CTA writes what another looks at: entries
  // above the old top of the stack, and blocks that no request holds yet).
  // A thread takes a run of the released ones: one search, and loads side by side
  // (a search for each took 2 us more).
  for (int64_t i = top - n_fresh + tid; i < count; i += kPlanThreads) look(a.free_list[i]);
  const int run = (n_gone + kPlanThreads - 1) / kPlanThreads;
  for (int i = min(n_gone, tid * run), end = min(n_gone, i + run); i < end;) {
    const int b = find(gone, a.B, i), to = min(end, gone[b + 1]);
    const int32_t* row = a.table + (int64_t)b * a.max_blocks;
    const int from = gone[b];
#pragma unroll 8
    for (; i < to; ++i) look(row[i - from]);
  }
  look(filled);
  if (__syncthreads_or(wrong)) return refuse(SA_ERR_INVALID_ARG);
  // All outputs in one index space, so that their chains of loads run side by
  // side: released pages, fresh blocks, requests, tokens.
  const int64_t e1 = n_gone, e2 = e1 + n_fresh, e3 = e2 + a.B + 1, e4 = e3 + a.max_tokens;
  for (int64_t i = gtid; i < e4; i += gsize) {
    if (i < e1) {
      a.free_list[count + i] = released((int)i);
    } else if (i < e2) {
      const int f = (int)(i - e1), b = find(fresh, a.B, f);
      const int held = blocks_of(a.kv_len[b], a.lg_page);
      a.table[(int64_t)b * a.max_blocks + held + (f - fresh[b])] = taken(f);
    } else if (i < e3) {
      const int b = (int)(i - e2);
      a.cu_q[b] = tok[b];
      if (b < a.B) a.new_len[b] = a.q_len[b] < 0 ? 0 : a.kv_len[b] + a.q_len[b];
    } else {
      const int64_t t = i - e3;
      int32_t slot = -1, pos = 0;
      if (t < n_tok) {
        const int b = find(tok, a.B, (int)t);
        const int old = a.kv_len[b];
        pos = old + ((int)t - tok[b]);
        const int blk = pos >> a.lg_page, held = blocks_of(old, a.lg_page);
        const int32_t page = blk < held ? a.table[(int64_t)b * a.max_blocks + blk] : taken(fresh[b] + blk - held);
        slot = (page << a.lg_page) + (pos & ((1 << a.lg_page) - 1));
      }
      a.slots[t] = slot;
      a.positions[t] = pos;
    }
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
  a.wide = (uintptr_t)k % 16 == 0 && (uintptr_t)v % 16 == 0;
  for (int i = 0; i < 2; ++i) a.wide = a.wide && ks[i] % 8 == 0 && vs[i] % 8 == 0;
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
  // Every CTA repeats the scan, which costs the others nothing; how many pages are
  // released and taken is not known here, so some CTAs are there for them (256
  // requests of up to 16,000 tokens: 5.9 us, 1.6 of them the look at the pages;
  // without it 4.3, with one CTA 9.2).
  const int64_t want = max64(8, ceil_div(max64(d.max_tokens, d.B), 2 * kPlanThreads));
  plan_kernel<<<(unsigned)min64(want, 148), kPlanThreads, smem, st>>>(a);
  return check_launch("plan_kernel");
}

}  // namespace sa
