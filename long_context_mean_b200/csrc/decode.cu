// Attention of few query rows over long key ranges (single tokens, short
// runs of tokens): the 4-bit paged cache (KV4) and contiguous bf16 K, V.
//
// Mathematics: for the rows of one kv head (its group of query heads times
// the sequence's new tokens), o = sum_j 2^(s_j - m) v_j / l with s_j the score in
// log2 units, m the running maximum and l the running sum; a key range can be
// cut anywhere and the parts (m, l, o) joined afterwards.
//
// Bound by HBM: K and V are read once (KV4: 144 bytes per token and kv head at
// d = 128), everything else is small.  So:
//  * the work of the whole batch (every sequence, kv head and row tile times its
//    16 * SUBS-token tiles) is one line of tiles, cut into equal pieces, one per
//    CTA, whatever the lengths: a ragged batch and one long sequence fill the
//    GPU alike; a unit counts as some tiles more than it has (COST).  Lengths are
//    read on the device; a piece may hold several units (sequence, row tile, kv
//    head) and a unit several pieces.  Units that lie in one piece are finished
//    there; parts of others go to the workspace and join_kernel adds them up in
//    a fixed order (no atomics).
//  * each warp streams its own tiles through its own ring of stages (bulk
//    copies for the cache's subtiles, cp.async for rows; no block barrier in
//    the loop) and multiplies with mma.sync m16n8k16: the
//    16 side is the tokens (K) or channels (V), the 8 side the query rows, so a
//    group of 8 rows wastes nothing.  (tcgen05 wants its operands in shared
//    memory: the widened codes would have to be written there, 4 times the bytes
//    that arrive.)
//  * KV4, bound by the instructions that widen the codes: a nibble under a mask is
//    an fp16 (K) or bf16 (V) number already (below), five instructions for 8 codes;
//    a product takes K's offset 8 off, a subtraction V's; K's scales multiply the
//    32-channel partial scores in fp32, V's scales multiply P.  16 sequences of 8,000
//    to 30,000 tokens, 312 MB: 68 us (4.6 TB/s); nibbles widened to bf16 integers by
//    shift, AND-OR and subtraction took 108, 8-bit operands (converted back to
//    fp16 by the compiler) 165.  Contiguous bf16, 48 single tokens over up to 4352
//    keys of 8 heads, 513 MB: 84 us (6.1 TB/s).
//  * times here are the GPU's alone, over the same inputs again; through the call, on
//    inputs that change, those 48 tokens take 88 us, and 16 sequences of 4 to 131,072
//    tokens 105 where they take 97.
// Rounding: P (and P times the V scale) is rounded to bf16 for the second
// product; sums, maxima and outputs are fp32.
#include <cuda_fp16.h>

#include "sa_internal.cuh"

namespace sa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kWorkers = 444;      // 148 SMs * 3 CTAs
constexpr int kMinTiles = 4;       // tiles a piece holds at least: one per warp
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kJoinThreads = 256;
// The reference maximum moves (and O with it) only when a score passes it by
// 2^8: with every new maximum a fifth of the tiles would rescale 64 numbers.
constexpr float kRescale = 8.f;
constexpr unsigned long long kWaitNs = 2000000000ull, kTestWaitNs = 10000000ull;

// What a worker leaves for join_kernel.
struct Piece {
  int32_t last;          // the piece that ends the unit which begins in this one and goes on past it; 0: none
  int32_t b, row0, kvh, n_q, q0;  // that unit, as join_kernel needs it
};

struct DecodeArgs {
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  const uint8_t* cache;          // KV4
  const uint16_t* k;             // bf16, [B][Hkv][Nk][d]
  const uint16_t* v;
  const int32_t* table;
  const int32_t* kv_len;         // nullable (bf16): Nk
  const int32_t* q_len;          // nullable
  const int32_t* cu_q;           // nullable
  int32_t* status;
  Piece* pieces;
  float* part_ml;                // [kWorkers][2][rows][2]
  float* part_o;                 // [kWorkers][2][rows][d]
  int64_t q_sb, q_st, q_sh;      // element strides of q: sequence, token, head
  int64_t o_sb, o_st, o_sh;      // of out (lse: the same / d)
  int64_t T, Nq, Nk;             // packed tokens; tokens and keys per sequence at most
  int64_t max_blocks;
  int32_t num_pages, page_bytes, window, sinks;
  int32_t B, Hkv, group, lg_page;
  float scale_log2;
  int32_t stall;                 // test hook: this block's copies are never reported whole; -1: none
  unsigned long long wait_ns;    // limit of every wait
};

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
// 16 bytes to shared memory; zeros where !live (nothing is read then).
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool live) {
  const int n = live ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
// mbarriers of a warp's stages (arrivals: the fetching lanes) and bulk copies.
__device__ __forceinline__ void bar_init(uint32_t bar, int n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, int bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, int bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(ok)
               : "r"(bar), "r"(parity)
               : "memory");
  return ok != 0;
}
__device__ __forceinline__ unsigned long long clock_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
// Bounded wait for a copy in flight (a copy always arrives, so the bound only
// keeps a broken device from holding the kernel).  False where the time ran out,
// here (then the block's abort flag is set and the status raised) or in
// another warp's wait.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int32_t* abort, unsigned long long limit,
                                         int32_t* status) {
  if (bar_try(bar, parity)) return true;
  const unsigned long long t0 = clock_ns();
  for (;;) {
    if (bar_try(bar, parity)) return true;
    if (*abort) return false;
    if (clock_ns() - t0 > limit) {
      *abort = 1;
      raise_status(status, SA_ERR_TIMEOUT);
      return false;
    }
  }
}
__device__ __forceinline__ void mma16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816z(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {   // d = a b
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// The same on fp16 operands, d = a b + c.
__device__ __forceinline__ void mma16816h(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1, float c0, float c1, float c2, float c3) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack2bf(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack2h(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t sub2bf(uint32_t a, uint32_t b) {
  __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t mul2bf(uint32_t a, uint32_t b) {
  __nv_bfloat162 r = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}
// One unit: a sequence's row tile on one kv head, and the tiles it visits.
// (Tokens and keys of a sequence fit 30 bits.)
struct Unit {
  int32_t b, n_k, n_q, q0;         // sequence, its keys and rows' tokens, first packed token
  int32_t lo, n_sink;              // keys [0, n_sink) and [lo, n_k) are visited
  int32_t sink_tiles, t_lo;        // the sinks' tiles, then those from t_lo on
  int32_t row0, kvh;
};

// Sequence b as the whole batch sees it: tokens, keys, row tiles and tiles.
template <int TOK, int ROWS>
__device__ __forceinline__ void sequence(const DecodeArgs& a, int b, Unit& u, int& row_tiles, int& tiles) {
  const int T = (int)a.T, Nq = (int)a.Nq, Nk = (int)a.Nk;
  u.b = b;
  bool bad = false;
  if (a.cu_q) {
    int c0 = a.cu_q[b], c1 = a.cu_q[b + 1];
    bad = c0 < 0 || c1 < c0 || c1 > T;
    c0 = max(0, min(c0, T));
    c1 = max(c0, min(c1, T));
    u.q0 = c0;
    u.n_q = c1 - c0;
  } else {
    u.q0 = 0;
    const int n = a.q_len ? a.q_len[b] : Nq;
    u.n_q = max(0, min(n, Nq));
    bad = n != u.n_q;
  }
  const int n = a.kv_len ? a.kv_len[b] : Nk;
  u.n_k = max(0, min(n, Nk));
  if (bad || n != u.n_k) raise_status(a.status, SA_ERR_INVALID_ARG);
  const int first = u.n_k - u.n_q;    // position of the first row
  u.lo = min(a.window > 0 ? max(0, first - a.window + 1) : 0, u.n_k);
  u.n_sink = min(a.sinks, u.lo);
  // whole tiles; the window's tiles start behind the sinks' tiles
  u.sink_tiles = (u.n_sink + TOK - 1) / TOK;
  u.t_lo = max(u.sink_tiles, u.lo / TOK);
  tiles = max(1, u.sink_tiles + max(0, (u.n_k + TOK - 1) / TOK - u.t_lo));
  row_tiles = u.n_q > 0 ? (u.n_q * a.group + ROWS - 1) / ROWS : 0;
}
__device__ __forceinline__ int tile_at(const Unit& u, int i) { return i < u.sink_tiles ? i : u.t_lo + (i - u.sink_tiles); }

// ---------------------------------------------------------------------------
// Formats: how a tile is fetched and multiplied
// ---------------------------------------------------------------------------
// Both give scores s[SUBS][NQ][4] of 16-token subtiles (accumulator layout: rows =
// tokens lane / 4 and + 8, columns = query rows 2 (lane % 4), + 1) and take P back
// as B operands.
template <int D>
struct Kv4 {
  static constexpr int G = D / 32, SUBS = 4, TOK = 16 * SUBS, SUB_BYTES = 576 * G, STAGE = SUBS * SUB_BYTES;
  // 64 tokens a tile, two stages a warp, 12 warps an SM: 68 us on the case above;
  // 48 tokens 70, 32 tokens with three or four stages 78, with 16 warps 76.
  static constexpr int STAGES = 2, TILES = D / 16;
  static constexpr int CTAS = 3;
  // What a unit costs beside its tiles, in tiles (its lengths, queries and output
  // are a chain of memory latencies): without it a piece of many one-token
  // sequences takes longest, and the batch nearly twice the time: 16 sequences of 4
  // to 131,072 tokens take 97 us with 8.
  static constexpr int COST = 8;
  // Channel of accumulator tile j's row lane / 4 (+ 8 where half).
  static __device__ __forceinline__ int channel(int j, int half, int r) { return 32 * (j >> 1) + 4 * r + 2 * (j & 1) + half; }
  // A row of q in fp16: its values times 2^x, with 2^x chosen so that the
  // largest lies in [2^14, 2^15): bf16's 8 bits fit fp16's 11, exact down to
  // 2^-31 of the largest.  `off` holds - 8 2^-24 times the groups' sums in three
  // bf16 parts each, as the columns of one product with the tokens' scales
  // (k = group, + 4 the second part, + 8 the third); `unit` is the factor
  // scale log2(e) 2^(24 - x) of this lane's scores.
  struct Q {
    uint32_t part[4 * G], off[2];
    float unit[2];
  };
  static __device__ __forceinline__ void load_q(const uint16_t* p, bool live, int lane, float scale_log2, Q& q) {
    const int q4 = lane & 3;
    uint4 w[G];
    uint32_t top = 0;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      w[g] = make_uint4(0, 0, 0, 0);
      if (live) w[g] = *reinterpret_cast<const uint4*>(p + 32 * g + 8 * q4);
      const uint32_t x[4] = {w[g].x, w[g].y, w[g].z, w[g].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) top = max(top, max(x[e] & 0x7FFFu, (x[e] >> 16) & 0x7FFFu));
    }
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int x = min(127, 141 - (int)(top >> 7));
    const float up = __uint_as_float((uint32_t)(127 + x) << 23);
    const float unit = fmaxf(scale_log2 * 0x1p24f / up, 1.17549435e-38f);   // (0 times a masked -inf would be NaN)
#pragma unroll
    for (int c = 0; c < 2; ++c) q.unit[c] = __shfl_sync(0xffffffffu, unit, (2 * q4 + c) * 4);
    float lead[2] = {0.f, 0.f};   // the sums of groups 2 (q4 % 2), + 1
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float f[8];
      unpack16(w[g], uint16_t{}, f);
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        f[e] *= up;
        sum += f[e];
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      if (g >> 1 == (q4 & 1)) lead[g & 1] = sum * -0x1p-21f;
      // pairs (e, e + 4); the odd ones meet codes at 16 times their value
#pragma unroll
      for (int e = 0; e < 4; ++e) q.part[4 * g + e] = pack2h(f[e] * (e & 1 ? 0.0625f : 1.f), f[e + 4] * (e & 1 ? 0.0625f : 1.f));
    }
    uint32_t b[3];
#pragma unroll
    for (int n = 0; n < 3; ++n) {
      b[n] = pack2bf(lead[0], lead[1]);
      lead[0] -= __uint_as_float(b[n] << 16);
      lead[1] -= __uint_as_float(b[n] & 0xFFFF0000u);
    }
    q.off[0] = q4 < 2 ? b[0] : b[1];
    q.off[1] = q4 < 2 ? b[2] : 0u;
  }
  // Lane s < SUBS looks up and fetches subtile s: one bulk copy of its bytes,
  // which the stage's mbarrier counts.  A subtile that no row sees is left
  // out: its stage holds old bytes, whose scores are masked and whose scales are
  // replaced by zero.
  static constexpr bool kBulk = true;
  static constexpr int32_t kSkip = INT32_MIN;
  // The unit's place in the tables and the cache, in subtiles of 16 tokens.
  const int32_t* row;
  const uint8_t* base;
  int32_t lo, n_sink, n;
  int32_t page = kSkip, sub = 0;   // table entry and number of this lane's subtile that is fetched next
  __device__ __forceinline__ void start(const DecodeArgs& a, const Unit& u, int lane) {
    row = a.table + (int64_t)u.b * a.max_blocks;
    base = a.cache + ((int64_t)u.kvh << (a.lg_page - 4)) * SUB_BYTES;
    lo = u.lo >> 4;
    n_sink = (u.n_sink + 15) >> 4;
    n = lane < SUBS ? (u.n_k + 15) >> 4 : 0;
  }
  __device__ __forceinline__ void look(const DecodeArgs& a, int tile, int lane) {
    sub = tile * SUBS + lane;
    page = kSkip;
    if (sub < n && (sub >= lo || sub < n_sink)) page = max(-1, row[sub >> (a.lg_page - 4)]);
  }
  __device__ __forceinline__ void fetch(const DecodeArgs& a, const Unit&, int, uint32_t dst, uint32_t bar, int lane) {
    if (lane >= SUBS) return;
    const bool seen = page != kSkip;
    bar_expect(bar, seen ? SUB_BYTES : 0);
    if (!seen) return;
    int pg = page;
    if ((uint32_t)pg >= (uint32_t)a.num_pages) {   // the sequence's result is not defined, the access stays inside
      raise_status(a.status, SA_ERR_INVALID_ARG);
      pg = 0;
    }
    const int in = sub & ((1 << (a.lg_page - 4)) - 1);
    bulk_load(dst + lane * SUB_BYTES, base + (int64_t)pg * a.page_bytes + in * SUB_BYTES, SUB_BYTES, bar);
  }
  // A code + 8 in the low bits of a half word is the fp16 subnormal
  // (code + 8) 2^-24, and one nibble higher 16 times that: K's operands take a mask
  // each and a shift for two, and the offset 8 goes into the accumulator.
  template <int NQ>
  static __device__ __forceinline__ void scores(const uint8_t* st, int s, const Q* q, int lane, float (*out)[4]) {
    const uint8_t* p = st + s * SUB_BYTES;
    uint32_t w0[G], w1[G];
    ld<G>(p + lane * 4 * G, w0);
    ld<G>(p + 128 * G + lane * 4 * G, w1);
    uint32_t s0[G / 2], s1[G / 2];
    ld<G / 2>(p + 512 * G + (lane >> 2) * 2 * G, s0);
    ld<G / 2>(p + 512 * G + ((lane >> 2) + 8) * 2 * G, s1);
    // (G = 2: the columns of groups 2 and 3 are zero)
    const uint32_t t0 = lane & 1 ? s0[G / 2 - 1] : s0[0], t1 = lane & 1 ? s1[G / 2 - 1] : s1[0];
#pragma unroll
    for (int n = 0; n < NQ; ++n) mma16816z(out[n], t0, t1, t0, t1, q[n].off[0], q[n].off[1]);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      constexpr uint32_t L = 0x000F000Fu, H = 0x00F000F0u;
      const uint32_t y0 = w0[g] >> 8, y1 = w1[g] >> 8;
      const float f0 = __uint_as_float(g & 1 ? s0[g >> 1] & 0xFFFF0000u : s0[g >> 1] << 16);
      const float f1 = __uint_as_float(g & 1 ? s1[g >> 1] & 0xFFFF0000u : s1[g >> 1] << 16);
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        float c[4];
        mma16816h(c, w0[g] & L, w1[g] & L, w0[g] & H, w1[g] & H, q[n].part[4 * g], q[n].part[4 * g + 1], 0.f, 0.f, 0.f, 0.f);
        mma16816h(c, y0 & L, y1 & L, y0 & H, y1 & H, q[n].part[4 * g + 2], q[n].part[4 * g + 3], c[0], c[1], c[2], c[3]);
        out[n][0] = fmaf(c[0], f0, out[n][0]);
        out[n][1] = fmaf(c[1], f0, out[n][1]);
        out[n][2] = fmaf(c[2], f1, out[n][2]);
        out[n][3] = fmaf(c[3], f1, out[n][3]);
      }
    }
  }
  // A code + 8 in the low bits of a bf16 is (code + 8) 2^-133, one nibble
  // higher 16 times that (bf16's subnormals and first binade are linear): masks
  // again, and an exact subtraction of the offset (by products with a constant - 8
  // instead: 72 us where this takes 68, and sums of 8 w that cancel).  P comes times
  // 2^kShift, which keeps the products far from fp32's smallest numbers.
  static constexpr float kShift = 64.f;
  static __device__ __forceinline__ float gain(int half) { return half ? 0x1p65f : 0x1p69f; }   // 2^(133 - kShift), / 16
  // p: P as B operands (tokens 2 (lane % 4), + 1 and + 8, + 9).  keep: one bit per
  // token of the subtile whose V counts; a scale of any other token is
  // whatever the slot holds (possibly NaN) and is replaced by 0.
  template <int NQ>
  static __device__ __forceinline__ void accumulate(const uint8_t* st, int s, const uint32_t (*p)[2], uint32_t keep, int lane, float (*o)[TILES][4]) {
    const uint8_t* b = st + s * SUB_BYTES;
    uint32_t v0[G], v1[G], s0[G], s1[G];
    ld<G>(b + 256 * G + lane * 4 * G, v0);
    ld<G>(b + 384 * G + lane * 4 * G, v1);
    ld<G>(b + 544 * G + (lane & 3) * 4 * G, s0);
    ld<G>(b + 560 * G + (lane & 3) * 4 * G, s1);
    if (keep != 0xFFFFu) {
      const uint32_t k0 = keep >> (2 * (lane & 3)), k1 = k0 >> 8;
      const uint32_t m0 = ((k0 & 1) ? 0x0000FFFFu : 0u) | ((k0 & 2) ? 0xFFFF0000u : 0u);
      const uint32_t m1 = ((k1 & 1) ? 0x0000FFFFu : 0u) | ((k1 & 2) ? 0xFFFF0000u : 0u);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        s0[g] &= m0;
        s1[g] &= m1;
      }
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      constexpr uint32_t L = 0x000F000Fu, H = 0x00F000F0u, L8 = 0x00080008u, H8 = 0x00800080u;
      const uint32_t y0 = v0[g] >> 8, y1 = v1[g] >> 8;
      const uint32_t a0 = sub2bf(v0[g] & L, L8), a1 = sub2bf(v0[g] & H, H8), a2 = sub2bf(v1[g] & L, L8), a3 = sub2bf(v1[g] & H, H8);
      const uint32_t c0 = sub2bf(y0 & L, L8), c1 = sub2bf(y0 & H, H8), c2 = sub2bf(y1 & L, L8), c3 = sub2bf(y1 & H, H8);
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const uint32_t p0 = mul2bf(p[n][0], s0[g]), p1 = mul2bf(p[n][1], s1[g]);
        mma16816(o[n][2 * g], a0, a1, a2, a3, p0, p1);
        mma16816(o[n][2 * g + 1], c0, c1, c2, c3, p0, p1);
      }
    }
  }
  template <int N>
  static __device__ __forceinline__ void ld(const uint8_t* p, uint32_t* w) {
    if constexpr (N == 4) *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(p);
    else if constexpr (N == 2) *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(p);
    else *w = *reinterpret_cast<const uint32_t*>(p);
  }
};

// Contiguous bf16 K and V.  Rows are swizzled in shared memory so that both
// operand reads are 16-byte loads without bank conflicts: chunk c (8 channels) of
// K token t lies at c ^ 4 (t & 1), of V token t at c ^ 2 ((t >> 1) & 3).
template <int D>
struct Bf16 {
  static constexpr int SUBS = 1, TOK = 16, STAGE = TOK * D * 4, STAGES = 3;
  static constexpr int TILES = D / 16, CH = D / 8;   // CH: chunks of a row
  static constexpr float kShift = 0.f;
  static __device__ __forceinline__ float gain(int) { return 1.f; }
  static constexpr int CTAS = 2;
  static constexpr int COST = 8;
  static __device__ __forceinline__ int channel(int j, int half, int r) { return D == 128 ? 64 * half + 8 * r + j : 8 * r + 4 * half + j; }
  struct Q {
    uint32_t part[D / 8];
    float unit[2];
  };
  static __device__ __forceinline__ void load_q(const uint16_t* p, bool live, int lane, float scale_log2, Q& q) {
#pragma unroll
    for (int c = 0; c < CH / 4; ++c) {
      uint4 w = make_uint4(0, 0, 0, 0);
      if (live) w = *reinterpret_cast<const uint4*>(p + (4 * c + (lane & 3)) * 8);
      q.part[4 * c] = w.x;
      q.part[4 * c + 1] = w.y;
      q.part[4 * c + 2] = w.z;
      q.part[4 * c + 3] = w.w;
    }
    q.unit[0] = q.unit[1] = scale_log2;
  }
  static constexpr bool kBulk = false;
  __device__ __forceinline__ void start(const DecodeArgs&, const Unit&, int) {}
  __device__ __forceinline__ void look(const DecodeArgs&, int, int) {}
  __device__ __forceinline__ void fetch(const DecodeArgs& a, const Unit& u, int tile, uint32_t dst, uint32_t, int lane) {
    const int t0 = tile * TOK;
    const int64_t base = ((int64_t)u.b * a.Hkv + u.kvh) * a.Nk;
#pragma unroll
    for (int i = 0; i < TOK * CH / 32; ++i) {
      const int e = i * 32 + lane, t = e / CH, c = e % CH;
      const int key = t0 + t;
      // keys that no row of the unit sees are not read: they come as zeros
      const bool live = key < u.n_k && (key >= u.lo || key < u.n_sink);
      const int64_t at = (base + (live ? key : 0)) * D + c * 8;
      cp16(dst + t * D * 2 + (c ^ ((t & 1) << 2)) * 16, a.k + at, live);
      cp16(dst + TOK * D * 2 + t * D * 2 + (c ^ (((t >> 1) & 3) << 1)) * 16, a.v + at, live);
    }
  }
  template <int NQ>
  static __device__ __forceinline__ void scores(const uint8_t* st, int, const Q* q, int lane, float (*out)[4]) {
    const int r = lane >> 2, q4 = lane & 3;
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) out[n][e] = 0.f;
#pragma unroll
    for (int c = 0; c < CH / 4; ++c) {
      const int ch = (4 * c + q4) ^ ((r & 1) << 2);   // rows r and r + 8 have the same parity
      const uint4 x = *reinterpret_cast<const uint4*>(st + r * D * 2 + ch * 16);
      const uint4 y = *reinterpret_cast<const uint4*>(st + (r + 8) * D * 2 + ch * 16);
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        mma16816(out[n], x.x, y.x, x.y, y.y, q[n].part[4 * c], q[n].part[4 * c + 1]);
        mma16816(out[n], x.z, y.z, x.w, y.w, q[n].part[4 * c + 2], q[n].part[4 * c + 3]);
      }
    }
  }
  template <int NQ>
  static __device__ __forceinline__ void accumulate(const uint8_t* st, int, const uint32_t (*p)[2], uint32_t, int lane, float (*o)[TILES][4]) {
    const int r = lane >> 2, t4 = lane & 3;
    const uint8_t* b = st + TOK * D * 2;
    uint4 w[4][D / 64];   // tokens 2 t4, + 1, + 8, + 9
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 2 * t4 + (i & 1) + 8 * (i >> 1);
#pragma unroll
      for (int h = 0; h < D / 64; ++h)
        w[i][h] = *reinterpret_cast<const uint4*>(b + t * D * 2 + ((r + 8 * h) ^ (((t >> 1) & 3) << 1)) * 16);
    }
    auto word = [&](int i, int h, int x) { return reinterpret_cast<const uint32_t*>(&w[i][h])[x]; };
    // the pair (token, token + 1) of channel x of chunk h
    auto pair = [&](int i, int h, int x) {
      return __byte_perm(word(i, h, x >> 1), word(i + 1, h, x >> 1), (x & 1) ? 0x7632 : 0x5410);
    };
#pragma unroll
    for (int j = 0; j < TILES; ++j) {
      const int h1 = D == 128 ? 1 : 0, x1 = D == 128 ? j : 4 + j;
      const uint32_t a0 = pair(0, 0, j), a1 = pair(0, h1, x1), a2 = pair(2, 0, j), a3 = pair(2, h1, x1);
#pragma unroll
      for (int n = 0; n < NQ; ++n) mma16816(o[n][j], a0, a1, a2, a3, p[n][0], p[n][1]);
    }
  }
};

// Row R of the sequence's n_q * group rows on kv head kvh: its token and query head.
__device__ __forceinline__ int64_t row_off(const DecodeArgs& a, const Unit& u, int R, int64_t sb, int64_t st, int64_t sh) {
  const int i = R / a.group, h = u.kvh * a.group + R % a.group;
  return (a.cu_q ? (u.q0 + i) * st : u.b * sb + i * st) + h * sh;
}

// o (unnormalised, relative to m) of 8 channels of row R, to its place.
template <int D>
__device__ __forceinline__ void finish_row(const DecodeArgs& a, const Unit& u, int R, int c8, float m, float l, const float* o) {
  const int64_t off = row_off(a, u, R, a.o_sb, a.o_st, a.o_sh);
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);   // no visible key: zeros; NaN stays
  uint4 w;
  uint32_t* p = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = pack2bf(o[2 * i] * inv, o[2 * i + 1] * inv);
  *reinterpret_cast<uint4*>(a.out + off + c8 * 8) = w;
  if (c8 == 0 && a.lse) a.lse[off / D] = (m + log2f(l)) * kLn2;   // log2f(0) = -inf
}

template <class F, int D, int NQ>
__global__ void __launch_bounds__(kThreads, NQ == 1 ? F::CTAS : 2) decode_kernel(const __grid_constant__ DecodeArgs a) {
  constexpr int ROWS = 8 * NQ, TOK = F::TOK;
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ int64_t scan[kWarps];
  __shared__ int64_t found_off;
  __shared__ int found_b;
  __shared__ float wm[kWarps][ROWS], wl[kWarps][ROWS];
  __shared__ __align__(8) uint64_t bars[kWarps][F::STAGES];
  __shared__ volatile int32_t abort;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = lane >> 2, t4 = lane & 3;
  if (F::kBulk && tid < kWarps * F::STAGES) {
    bar_init(smem_addr(&bars[0][0] + tid), F::SUBS + ((int)blockIdx.x == a.stall));
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid == 0) abort = 0;

  // Where this piece of the line of tiles starts.
  const int per_thread = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(a.B, tid * per_thread), b1 = min(a.B, b0 + per_thread);
  int64_t sum = 0;
  for (int b = b0; b < b1; ++b) {
    Unit u;
    int rt, tl;
    sequence<TOK, ROWS>(a, b, u, rt, tl);
    sum += (int64_t)rt * a.Hkv * (F::COST + tl);
  }
  int64_t inc = sum;
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) scan[warp] = inc;
  if (tid == 0) found_b = a.B;
  __syncthreads();
  int64_t before = 0, W = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += scan[w];
    W += scan[w];
  }
  const int64_t per = max64(kMinTiles, (W + gridDim.x - 1) / gridDim.x);
  const int64_t start = min64(W, blockIdx.x * per), end = min64(W, start + per);
  int64_t pos = before + inc - sum;
  if (start < end && start >= pos && start < pos + sum) {
    for (int b = b0; b < b1; ++b) {
      Unit u;
      int rt, tl;
      sequence<TOK, ROWS>(a, b, u, rt, tl);
      const int64_t n = (int64_t)rt * a.Hkv * (F::COST + tl);
      if (start < pos + n) {
        found_b = b;
        found_off = start - pos;
        break;
      }
      pos += n;
    }
  }
  __syncthreads();
  Piece piece{};
  int b = found_b;
  int64_t off = found_off;

  F f;
  const uint32_t ring = smem_addr(sm) + warp * (F::STAGES * F::STAGE);
  const uint8_t* ring_p = sm + warp * (F::STAGES * F::STAGE);
  const uint32_t bar = smem_addr(&bars[warp][0]);
  int in = 0, out = 0;        // the stages that are filled and read next
  uint32_t phase = 0;         // of the stage that is read next
  int64_t at = start;
  while (at < end && b < a.B) {
    Unit u;
    int rt, tl;
    sequence<TOK, ROWS>(a, b, u, rt, tl);
    const int64_t whole = (int64_t)rt * a.Hkv * (F::COST + tl);
    if (off >= whole) {   // next sequence
      off -= whole;
      ++b;
      continue;
    }
    const int cost = F::COST + tl, unit = (int)(off / cost);
    const int x0 = (int)(off - (int64_t)unit * cost), x1 = (int)min64(cost, x0 + (end - at));
    const int i0 = max(0, x0 - F::COST), i1 = max(0, x1 - F::COST);   // the unit's tiles in this piece
    at += x1 - x0;
    off += x1 - x0;
    if (i1 == 0) continue;   // its tiles begin in the next piece
    u.kvh = unit % a.Hkv;
    u.row0 = (unit / a.Hkv) * ROWS;
    const int rows_all = u.n_q * a.group;

    const int first = i0 + warp;
    const int mine = first < i1 ? (i1 - first + kWarps - 1) / kWarps : 0;
    int sent = 0;
    f.start(a, u, lane);
    int next = tile_at(u, first);   // the tile that is fetched next
    if (mine > 0) f.look(a, next, lane);
    auto send = [&]() {
      if (sent < mine) {
        f.fetch(a, u, next, ring + in * F::STAGE, bar + in * 8, lane);
        in = in + 1 == F::STAGES ? 0 : in + 1;
        ++sent;
        next = tile_at(u, first + sent * kWarps);
        if (sent < mine) f.look(a, next, lane);
      }
      if (!F::kBulk) cp_commit();
    };
#pragma unroll
    for (int s = 0; s < F::STAGES - 1; ++s) send();

    typename F::Q q[NQ];
    int qpos[NQ][2];   // positions of this lane's columns (query rows)
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int R = u.row0 + 8 * n + r;
      const bool live = R < rows_all;
      F::load_q(a.q + row_off(a, u, live ? R : 0, a.q_sb, a.q_st, a.q_sh), live, lane, a.scale_log2, q[n]);
#pragma unroll
      for (int c = 0; c < 2; ++c) qpos[n][c] = u.n_k - u.n_q + min(rows_all - 1, u.row0 + 8 * n + 2 * t4 + c) / a.group;
    }
    const int p_min = u.n_k - u.n_q + u.row0 / a.group;
    const int p_max = u.n_k - u.n_q + min(rows_all - 1, u.row0 + ROWS - 1) / a.group;

    float o[NQ][F::TILES][4], m[NQ][2], l[NQ][2];   // m: log2 units
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
#pragma unroll
      for (int j = 0; j < F::TILES; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][j][e] = 0.f;
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
    }

    for (int i = 0; i < mine; ++i) {
      if constexpr (F::kBulk) {
        if (!__all_sync(0xffffffffu, bar_wait(bar + out * 8, phase, &abort, a.wait_ns, a.status))) {
          // A wait has run out: nothing more is fetched, and what is under way lands first.
          const unsigned long long t0 = clock_ns();
          for (; i < sent; ++i) {
            while (!bar_try(bar + out * 8, phase) && clock_ns() - t0 < a.wait_ns) {}
            if (++out == F::STAGES) {
              out = 0;
              phase ^= 1;
            }
          }
          break;
        }
      } else {
        cp_wait<F::STAGES - 2>();
        __syncwarp();
      }
      const uint8_t* st = ring_p + out * F::STAGE;
      send();
      if (++out == F::STAGES) {
        out = 0;
        phase ^= 1;
      }
      const int t0 = tile_at(u, first + i * kWarps) * TOK;
      float s[F::SUBS][NQ][4];
#pragma unroll
      for (int x = 0; x < F::SUBS; ++x) F::template scores<NQ>(st, x, q, lane, s[x]);
      const bool all = t0 + TOK - 1 <= p_min && t0 + TOK <= u.n_k &&
                       (a.window == 0 || p_max - t0 < a.window || t0 + TOK <= a.sinks);
      uint32_t keep[F::SUBS];
#pragma unroll
      for (int x = 0; x < F::SUBS; ++x) keep[x] = 0xFFFFu;
      if (!all) {
#pragma unroll
        for (int x = 0; x < F::SUBS; ++x) {
#pragma unroll
          for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = t0 + 16 * x + r + 8 * (e >> 1), p = qpos[n][e & 1];
              const bool see = key < u.n_k && key <= p && (a.window == 0 || p - key < a.window || key < a.sinks);
              if (!see) s[x][n][e] = -INFINITY;
            }
          // tokens that some row of the unit may see
          const int k0 = t0 + 16 * x + (lane & 15);
          keep[x] = __ballot_sync(0xffffffffu, k0 < u.n_k && (k0 >= u.lo || k0 < u.n_sink)) & 0xFFFFu;
        }
      }
      bool moved = false;
      float corr[NQ][2], ref[NQ][2];
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float x = fmaxf(s[0][n][c], s[0][n][c + 2]);
#pragma unroll
          for (int y = 1; y < F::SUBS; ++y) x = fmaxf(x, fmaxf(s[y][n][c], s[y][n][c + 2]));
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
          x *= q[n].unit[c];   // (positive)
          const float mn = x > m[n][c] + kRescale ? x : m[n][c];   // m = -inf: any score is above
          ref[n][c] = mn == -INFINITY ? 0.f : mn;
          corr[n][c] = ex2f(m[n][c] - ref[n][c]);
          moved |= mn != m[n][c];
          m[n][c] = mn;
        }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          l[n][0] *= corr[n][0];
          l[n][1] *= corr[n][1];
#pragma unroll
          for (int j = 0; j < F::TILES; ++j) {
            o[n][j][0] *= corr[n][0];
            o[n][j][1] *= corr[n][1];
            o[n][j][2] *= corr[n][0];
            o[n][j][3] *= corr[n][1];
          }
        }
      }
#pragma unroll
      for (int x = 0; x < F::SUBS; ++x) {
        uint32_t p[NQ][2];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          float e[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) e[y] = ex2f(fmaf(s[x][n][y], q[n].unit[y & 1], F::kShift - ref[n][y & 1]));
          l[n][0] += e[0] + e[2];
          l[n][1] += e[1] + e[3];
          p[n][0] = transpose8(pack2bf(e[0], e[1]));
          p[n][1] = transpose8(pack2bf(e[2], e[3]));
        }
        F::template accumulate<NQ>(st, x, p, keep[x], lane, o);
      }
    }
    if (!F::kBulk) cp_wait<0>();

    // Join the four warps' parts in shared memory (over the rings).
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[n][c] += __shfl_xor_sync(0xffffffffu, l[n][c], d);
        l[n][c] *= exp2f(-F::kShift);
        if (r == 0) {
          wm[warp][8 * n + 2 * t4 + c] = m[n][c];
          wl[warp][8 * n + 2 * t4 + c] = l[n][c];
        }
      }
    __syncthreads();
    const bool begins = i0 == 0, ends = i1 == tl;
    const int64_t slot = (int64_t)blockIdx.x * 2 + (begins ? 1 : 0);
    // (no wait lies between this barrier and the next, so all threads see the same)
    if (F::kBulk && abort) {
      // The rows of this piece's units stay as they were; those of the unit that
      // goes through it become NaN.
      if (!begins && tid < ROWS) *reinterpret_cast<float2*>(a.part_ml + (slot * ROWS + tid) * 2) = make_float2(-INFINITY, NAN);
      break;
    }
    float* os = reinterpret_cast<float*>(sm);   // [warp][ROWS][D + 4]
    constexpr int OS = D + 4;
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int j = 0; j < F::TILES; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          os[(warp * ROWS + 8 * n + 2 * t4 + (e & 1)) * OS + F::channel(j, e >> 1, r)] = o[n][j][e] * F::gain(e >> 1);
    __syncthreads();
    for (int e = tid; e < ROWS * (D / 8); e += kThreads) {
      const int row = e / (D / 8), c8 = e % (D / 8);
      float mx = wm[0][row];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, wm[w][row]);
      const float rf = mx == -INFINITY ? 0.f : mx;
      float acc[8] = {}, ls = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float g = ex2f(wm[w][row] - rf);
        ls += g * wl[w][row];
        const float* src = os + (w * ROWS + row) * OS + c8 * 8;
#pragma unroll
        for (int x = 0; x < 8; ++x) acc[x] += g * src[x];
      }
      const int R = u.row0 + row;
      if (R >= rows_all) continue;
      if (begins && ends) {
        finish_row<D>(a, u, R, c8, mx, ls, acc);
      } else {
        float* dst = a.part_o + (slot * ROWS + row) * D + c8 * 8;
        *reinterpret_cast<float4*>(dst) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        *reinterpret_cast<float4*>(dst + 4) = make_float4(acc[4], acc[5], acc[6], acc[7]);
        if (c8 == 0) *reinterpret_cast<float2*>(a.part_ml + (slot * ROWS + row) * 2) = make_float2(mx, ls);
      }
    }
    if (begins && !ends) {
      piece.last = blockIdx.x + (int)((cost - x1 + per - 1) / per);   // every piece but the last one holds `per` tiles
      piece.b = u.b;
      piece.row0 = u.row0;
      piece.kvh = u.kvh;
      piece.n_q = u.n_q;
      piece.q0 = u.q0;
    }
    // The rings are filled next by the async proxy, after these generic accesses.
    if (F::kBulk) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
  }
  if (tid == 0) a.pieces[blockIdx.x] = piece;
}

// Adds up the parts of the unit that begins in piece blockIdx.x and ends in a
// later one.  The parts are dealt to groups of threads, one thread 8 channels
// of a row, and the groups' sums joined in order: a long sequence alone has some
// 40 parts a unit, and one thread after another would wait for each.  Launched
// as a dependent of decode_kernel: it waits for that grid's writes.
template <class F, int D, int NQ>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ DecodeArgs a) {
  constexpr int ROWS = 8 * NQ, C8 = D / 8, BATCH = 6;
  __shared__ float part[kJoinThreads][11];   // m, l and 8 sums of a thread
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Piece p = a.pieces[blockIdx.x];
  if (p.last == 0) return;
  Unit u{};
  u.b = p.b;
  u.q0 = p.q0;
  u.n_q = p.n_q;
  u.row0 = p.row0;
  u.kvh = p.kvh;
  const int rows = min(ROWS, u.n_q * a.group - u.row0), items = rows * C8;
  const int groups = kJoinThreads / items, item = threadIdx.x % items, g = threadIdx.x / items;
  const int row = item / C8, c8 = item % C8;
  float m = -INFINITY, l = 0.f, acc[8] = {};
  auto add = [&](float pm, float pl, const float* v) {
    const float mn = fmaxf(m, pm), rf = mn == -INFINITY ? 0.f : mn;
    const float x = ex2f(m - rf), y = ex2f(pm - rf);
    l = l * x + pl * y;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = acc[i] * x + v[i] * y;
    m = mn;
  };
  if (g < groups) {
    for (int w0 = blockIdx.x + g; w0 <= p.last; w0 += BATCH * groups) {
      float2 ml[BATCH];
      float v[BATCH][8];
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const int w = w0 + i * groups;
        ml[i] = make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
        if (w <= p.last) {
          const int64_t at = ((int64_t)w * 2 + (w == (int)blockIdx.x ? 1 : 0)) * ROWS + row;
          ml[i] = *reinterpret_cast<const float2*>(a.part_ml + at * 2);
          *reinterpret_cast<float4*>(v[i]) = *reinterpret_cast<const float4*>(a.part_o + at * D + c8 * 8);
          *reinterpret_cast<float4*>(v[i] + 4) = *reinterpret_cast<const float4*>(a.part_o + at * D + c8 * 8 + 4);
        }
      }
#pragma unroll
      for (int i = 0; i < BATCH; ++i) add(ml[i].x, ml[i].y, v[i]);
    }
    float* d = part[threadIdx.x];
    d[0] = m;
    d[1] = l;
#pragma unroll
    for (int i = 0; i < 8; ++i) d[2 + i] = acc[i];
  }
  __syncthreads();
  if (g != 0) return;
  for (int k = 1; k < groups; ++k) {
    const float* d = part[k * items + item];
    add(d[0], d[1], d + 2);
  }
  finish_row<D>(a, u, u.row0 + row, c8, m, l, acc);
}

size_t ws_bytes(int64_t rows, int64_t d) {
  return align_up(kWorkers * sizeof(Piece), 256) + align_up((size_t)kWorkers * 2 * rows * 2 * sizeof(float), 256) +
         (size_t)kWorkers * 2 * rows * d * sizeof(float);
}

// A window that reaches past every key is none; so no position minus window
// leaves 31 bits.
void set_window(DecodeArgs& a, int64_t window, int64_t sinks) {
  a.window = window >= a.Nk ? 0 : (int32_t)window;
  a.sinks = (int32_t)min64(sinks, a.Nk);
}

template <class F, int D, int NQ>
sa_status launch(DecodeArgs& a, int64_t max_tiles, void* ws, cudaStream_t st) {
  constexpr int ROWS = 8 * NQ;
  constexpr int smem_ring = kWarps * F::STAGES * F::STAGE, smem_join = kWarps * ROWS * (D + 4) * 4;
  constexpr int smem = smem_ring > smem_join ? smem_ring : smem_join;
  char* w = static_cast<char*>(ws);
  a.pieces = reinterpret_cast<Piece*>(w);
  w += align_up(kWorkers * sizeof(Piece), 256);
  a.part_ml = reinterpret_cast<float*>(w);
  w += align_up((size_t)kWorkers * 2 * ROWS * 2 * sizeof(float), 256);
  a.part_o = reinterpret_cast<float*>(w);
  if (cudaFuncSetAttribute(decode_kernel<F, D, NQ>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return set_error(SA_ERR_CUDA, "cudaFuncSetAttribute(decode_kernel) failed");
  const int workers = NQ == 1 ? 148 * F::CTAS : 148 * 2;
  const int grid = (int)max64(1, min64(workers, ceil_div(max_tiles, kMinTiles)));
  decode_kernel<F, D, NQ><<<grid, kThreads, smem, st>>>(a);
  if (sa_status e = check_launch("decode_kernel")) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, join_kernel<F, D, NQ>, a) != cudaSuccess)
    return check_launch("join_kernel");
  return SA_OK;
}

template <template <int> class F>
sa_status launch_format(DecodeArgs& a, int64_t d, int nq, int64_t max_tiles, void* ws, cudaStream_t st) {
  if (d == 128)
    return nq == 1 ? launch<F<128>, 128, 1>(a, max_tiles, ws, st) : launch<F<128>, 128, 2>(a, max_tiles, ws, st);
  return nq == 1 ? launch<F<64>, 64, 1>(a, max_tiles, ws, st) : launch<F<64>, 64, 2>(a, max_tiles, ws, st);
}

}  // namespace

size_t decode_ws_bytes(int64_t d) { return ws_bytes(16, d); }

sa_status launch_kv4_attn(const Kv4AttnArgs& x, cudaStream_t st) {
  DecodeArgs a{};
  a.q = static_cast<const uint16_t*>(x.q);
  a.out = static_cast<uint16_t*>(x.out);
  a.lse = x.lse;
  a.cache = static_cast<const uint8_t*>(x.cache);
  a.table = x.table;
  a.kv_len = x.kv_len;
  a.cu_q = x.cu_q;
  a.status = x.status;
  a.q_sb = a.q_st = x.q_strides[0];
  a.q_sh = x.q_strides[1];
  a.o_sb = a.o_st = x.Hq * x.desc.d;
  a.o_sh = x.desc.d;
  a.T = x.T;
  a.Nq = 1;
  a.Nk = x.max_blocks * x.desc.page;
  a.max_blocks = x.max_blocks;
  a.num_pages = (int32_t)x.desc.num_pages;
  a.page_bytes = (int32_t)(x.desc.Hkv * (x.desc.page / 16) * 18 * x.desc.d);
  set_window(a, x.window, x.sinks);
  a.B = (int32_t)x.B;
  a.Hkv = (int32_t)x.desc.Hkv;
  a.group = (int32_t)(x.Hq / x.desc.Hkv);
  while ((1LL << a.lg_page) < x.desc.page) ++a.lg_page;
  a.scale_log2 = x.scale * kLog2e;
  a.stall = x.stall;
  a.wait_ns = x.stall >= 0 ? kTestWaitNs : kWaitNs;
  // Two column tiles (16 rows) a unit where the average sequence has more than 8 rows.
  const int nq = x.T * a.group > 8 * x.B ? 2 : 1;
  const int64_t row_tiles = ceil_div(x.T * a.group, 8 * nq) + x.B;
  const int64_t max_tiles = row_tiles * a.Hkv * ceil_div(a.Nk, Kv4<128>::TOK);
  return launch_format<Kv4>(a, x.desc.d, nq, max_tiles, x.ws, st);
}

sa_status launch_window_decode(const WindowArgs& x, cudaStream_t st) {
  DecodeArgs a{};
  a.q = static_cast<const uint16_t*>(x.q);
  a.k = static_cast<const uint16_t*>(x.k);
  a.v = static_cast<const uint16_t*>(x.v);
  a.out = static_cast<uint16_t*>(x.out);
  a.lse = x.lse;
  a.kv_len = x.kv_len;
  a.q_len = x.q_len;
  a.status = x.status;
  const sa_window_shape& s = x.shape;
  a.q_st = a.o_st = s.d;
  a.q_sh = a.o_sh = s.Nq * s.d;
  a.q_sb = a.o_sb = s.Hq * s.Nq * s.d;
  a.Nq = s.Nq;
  a.Nk = s.Nk;
  set_window(a, x.window, x.sinks);
  a.B = (int32_t)s.B;
  a.Hkv = (int32_t)s.Hkv;
  a.group = (int32_t)(s.Hq / s.Hkv);
  a.scale_log2 = x.scale * kLog2e;
  const int nq = s.Nq * a.group > 8 ? 2 : 1;
  int64_t keys = s.Nk;
  if (x.window > 0) keys = min64(keys, x.window + x.sinks + s.Nq + 2 * Bf16<128>::TOK);
  const int64_t max_tiles = s.B * ceil_div(s.Nq * a.group, 8 * nq) * a.Hkv * ceil_div(keys, Bf16<128>::TOK);
  return launch_format<Bf16>(a, s.d, nq, max_tiles, x.ws, st);
}

}  // namespace sa
