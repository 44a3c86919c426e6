// Prefill attention with a sliding window and first tokens that stay visible,
// exact to the token, on the sm_100a tensor cores (bf16, d in {64, 128}).
//
// Mathematics: row i of a sequence sits at position p = n_k - n_q + i and sees key
// j iff j <= p, j < n_k and (window == 0 or p - j < window or j < sinks);
// o = sum 2^(c s_j - m) v_j / l with c = scale log2 e, an online maximum m and the
// sum l of the same rows.  Only the 128-key tiles that hold a visible pair of a
// unit are visited: the sinks' tiles and the window's.  Tiles that every row sees
// whole take no mask.
//
// Bound by the tensor cores and the exponentials alike: a 128 x 128 tile of S
// and its product with V take 1024 clocks of tcgen05.mma, its 16,384
// exponentials 1024 clocks of the special-function units.  So:
//  * persistent CTAs, one per SM; a unit is two 128-row query tiles that share
//    every K and V tile: two query heads of one kv head where the group is even,
//    two neighbouring row blocks of one head otherwise.  While the softmax of one
//    tile runs, the tensor cores work on the other.
//  * tiles of 128 keys: the S product of 128 x 64 x 16 steps would read 6 KB of
//    shared memory in 32 clocks of mma, above the 128 bytes a clock that an SM
//    has; 128 x 128 x 16 reads 8 KB in 64.
//  * warp 0 loads Q and one ring of K and V tiles by TMA, warp 1 issues the
//    products (S = Q K^T into TMEM, O += P V with P from TMEM over its S), four
//    warps per query tile do the softmax, one thread a row.  The products of one
//    query tile are issued in order P V(t), S(t + 1), so S may overwrite P without
//    a barrier, and S(t + 1)'s arrival tells that P V(t) is done.
//  * O is rescaled only when a row's maximum grows by more than 2^8.
// 16,384 rows, 32/8 heads of 128, window 4096, 128 sinks: 855 us, 1155 TFLOP/s of
// visible pairs, some 3100 clocks for two tiles of 2048 clocks of mma; three padded
// prompts of up to 2777 rows, window 1024: 99 us over the same inputs again, 111 on inputs
// that change; a unit of ten tiles there pays its start and its output.
// Roundings: P is rounded to bf16 for the second product (l sums the unrounded
// values); everything else is fp32.
// V rows that no row of the unit sees (behind a sequence of a padded batch,
// before the window) are zeroed in shared memory before the product reads them,
// so that no NaN in them meets a weight of zero.
// Waits are bounded as in the block-sparse kernel: on expiry SA_ERR_TIMEOUT is
// raised, every role stops issuing, drains what it issued and leaves.
#include "sa_internal.cuh"
#include "tc_ptx.cuh"

namespace sa {
namespace {

constexpr int kTile = 128;                 // keys of a tile, rows of a query tile
constexpr int kThreads = 384;              // 4 helper warps, 2 x 4 softmax warps
constexpr int kStages = 4;                 // K and V tiles in flight (five are no faster)
constexpr int kOutBytes = 4096;            // a softmax warp's stage of output rows
constexpr float kRescale = 8.0f;           // log2 units
constexpr unsigned long long kWaitNs = 2000000000ull;

template <int D>
struct Cfg {
  static constexpr int CHUNKS = D / 64;               // 128-byte columns of a row
  static constexpr int TILE_BYTES = kTile * D * 2;
  static constexpr int CHUNK_BYTES = kTile * 128;
  static constexpr int OFF_KV = 2 * TILE_BYTES;
  static constexpr int OFF_OUT = OFF_KV + kStages * TILE_BYTES;   // 8 warps' output stages
  static constexpr int OFF_CTL = OFF_OUT + 8 * kOutBytes;
  static constexpr int SMEM = OFF_CTL + 1024;
};
static_assert(Cfg<128>::SMEM <= 227 * 1024, "shared memory above the 227 KB a CTA may use");

// A query tile of a unit.  Its tiles of keys, by their number kt (128 keys
// each): some row sees some key of kt < sink or from <= kt < to; every row sees
// every key where kt < whole_to and (kt >= whole_from or kt < whole_sink).
struct Rows {
  int32_t bh, row0, first, last;   // head of the batch, first row, positions of the first and last row
  int32_t live, sink, from, to, whole_sink, whole_from, whole_to;
};
// One unit; the producer derives it and the other roles read it from the ring.
struct Unit {
  int32_t n;                       // tiles of keys that it visits; -1: no unit is left
  int32_t sink_tiles, t_lo;        // the sinks' tiles, then from t_lo on
  int32_t n_q, n_k, kvh;
  int32_t lo, hi, n_sink;          // keys that some row sees: [0, n_sink) and [lo, hi)
  Rows rows[2];
  __device__ __forceinline__ int tile(int t) const { return t < sink_tiles ? t : t_lo + t - sink_tiles; }
};
__device__ __forceinline__ bool active(const Rows& r, int kt) { return kt < r.sink || (kt >= r.from && kt < r.to); }

struct Ctl {
  uint64_t q_full[2], q_empty[2];
  uint64_t kv_full[kStages], kv_empty[kStages];
  uint64_t s_full[2], p_half[2], p_full[2], o_full[2], o_free[2];
  uint64_t u_full[4], u_empty[4];
  uint64_t mma_done;
  unsigned long long wait_ns;
  uint32_t tmem_base;
  volatile uint32_t abort;
  Unit ring[4];
};
static_assert(sizeof(Ctl) <= 1024, "control block too large");

struct Params {
  uint16_t* out;
  float* lse;
  const int32_t* q_len;
  const int32_t* kv_len;
  int32_t* status;
  int32_t* counter;        // next unit past the first of each CTA
  int32_t B, Hq, Hkv, Nq, Nk, window, sinks;
  int32_t by_heads;        // the two query tiles are heads (else row blocks)
  int32_t pairs;           // units of one row block over the batch
  int32_t num_units;
  float scale_log2;
};

__device__ __forceinline__ void unit_at(const Params& p, int i, Unit& u) {
  const int blocks = p.num_units / p.pairs;
  const int qb = blocks - 1 - i / p.pairs, pair = i % p.pairs;   // the latest rows have the most keys
  const int per = p.by_heads ? p.Hq / 2 : p.Hq;
  const int b = pair / per, h = (pair % per) * (p.by_heads ? 2 : 1);
  int n_q = p.q_len ? p.q_len[b] : p.Nq, n_k = p.kv_len ? p.kv_len[b] : p.Nk;
  if (n_q < 0 || n_q > p.Nq || n_k < 0 || n_k > p.Nk) {
    raise_status(p.status, SA_ERR_INVALID_ARG);
    n_q = max(0, min(n_q, p.Nq));
    n_k = max(0, min(n_k, p.Nk));
  }
  u.n_q = n_q;
  u.n_k = n_k;
  u.kvh = b * p.Hkv + h / (p.Hq / p.Hkv);
  int hi = 0, lo = 0;
  for (int w = 0; w < 2; ++w) {
    Rows& r = u.rows[w];
    r.bh = b * p.Hq + h + (p.by_heads ? w : 0);
    r.row0 = (p.by_heads ? qb : 2 * qb + w) * kTile;
    r.live = r.row0 < n_q;
    r.first = n_k - n_q + r.row0;
    r.last = n_k - n_q + min(n_q, r.row0 + kTile) - 1;
    const int to = r.live ? max(0, r.last + 1) : 0, from = p.window ? max(0, r.first - p.window + 1) : 0;
    if (w == 0) lo = from;
    hi = max(hi, to);
    r.sink = (min(p.sinks, to) + kTile - 1) / kTile;
    r.from = from / kTile;
    r.to = (to + kTile - 1) / kTile;
    r.whole_sink = p.sinks / kTile;
    r.whole_from = p.window ? (max(0, r.last - p.window + 1) + kTile - 1) / kTile : 0;
    r.whole_to = max(0, r.first + 1) / kTile;
  }
  u.hi = hi;
  u.lo = min(lo, hi);
  u.n_sink = min(p.sinks, u.lo);
  u.sink_tiles = (u.n_sink + kTile - 1) / kTile;
  u.t_lo = max(u.sink_tiles, u.lo / kTile);
  u.n = hi > 0 ? u.sink_tiles + max(0, (hi + kTile - 1) / kTile - u.t_lo) : 0;
}

template <int D>
__device__ void producer(const CUtensorMap* tmQ, const CUtensorMap* tmK, const CUtensorMap* tmV, const Params& p,
                         Ctl* c, uint32_t sb) {
  using C = Cfg<D>;
  uint32_t it = 0, nq[2] = {0, 0};
  int i = blockIdx.x;
  auto load = [&](const CUtensorMap* map, int key, int head) {
    const int s = it % kStages;
    if (!mbar_wait(&c->kv_empty[s], ((it / kStages) & 1) ^ 1, c, p.status)) return false;
    mbar_expect_tx(&c->kv_full[s], C::TILE_BYTES);
#pragma unroll
    for (int x = 0; x < C::CHUNKS; ++x)
      tma_load_3d(sb + C::OFF_KV + s * C::TILE_BYTES + x * C::CHUNK_BYTES, map, 64 * x, key, head, &c->kv_full[s]);
    ++it;
    return true;
  };
  bool ok = true;
  for (uint32_t j = 0; ok; ++j) {
    const int slot = j & 3;
    if (!(ok = mbar_wait(&c->u_empty[slot], ((j >> 2) & 1) ^ 1, c, p.status))) break;
    Unit& u = c->ring[slot];
    const bool some = i < p.num_units;
    if (some)
      unit_at(p, i, u);
    else
      u.n = -1;
    mbar_arrive(&c->u_full[slot]);
    if (!some) break;
    // the next unit: the CTAs' first ones are their own numbers
    i = p.num_units > (int)gridDim.x ? (int)gridDim.x + atomicAdd(p.counter, 1) : p.num_units;
    const int n = u.n, kvh = u.kvh;
    for (int t = 0; t < n && ok; ++t) {
      const int k0 = u.tile(t) * kTile;
      if (!(ok = load(tmK, k0, kvh))) break;
      if (t == 0) {
        for (int w = 0; w < 2 && ok; ++w) {
          if (!u.rows[w].live) continue;
          if (!(ok = mbar_wait(&c->q_empty[w], (nq[w] & 1) ^ 1, c, p.status))) break;
          ++nq[w];
          mbar_expect_tx(&c->q_full[w], C::TILE_BYTES);
#pragma unroll
          for (int x = 0; x < C::CHUNKS; ++x)
            tma_load_3d(sb + w * C::TILE_BYTES + x * C::CHUNK_BYTES, tmQ, 64 * x, u.rows[w].row0, u.rows[w].bh,
                        &c->q_full[w]);
        }
        if (!ok) break;
      }
      ok = load(tmV, k0, kvh);
    }
  }
  // The copies issued last have landed before the CTA may exit.
  for (int w = 0; w < 2; ++w)
    if (nq[w] > 0) mbar_drain(&c->q_full[w], (nq[w] - 1) & 1, c->wait_ns);
  for (uint32_t j = it > (uint32_t)kStages ? it - kStages : 0; j < it; ++j)
    mbar_drain(&c->kv_full[j % kStages], (j / kStages) & 1, c->wait_ns);
}

// The whole warp runs this, so that addresses and descriptors are uniform, and
// one elected lane issues.  (A single lane that built every descriptor anew
// took 85 to 110 clocks a product, whose mma takes 64.)
template <int D>
__device__ void mma_issuer(const Params& p, Ctl* c, uint32_t sb, uint32_t tm) {
  using C = Cfg<D>;
  constexpr uint32_t idesc_s = make_idesc(kTile, kTile, 0), idesc_pv = make_idesc(kTile, D, 1);
  // Descriptors differ in their start address (16-byte units in the low bits) only.
  const uint64_t q_desc = desc_sw128(sb, 16, 1024), k_desc = desc_sw128(sb + C::OFF_KV, 16, 1024),
                 v_desc = desc_sw128(sb + C::OFF_KV, C::CHUNK_BYTES, 1024);
  uint32_t ks = 0, kph = 0;                           // stage and phase of the next K tile
  uint32_t nq[2] = {0, 0}, np[2] = {0, 0};            // units and tiles so far of each query tile
  const bool leader = elect_one();
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, c, p.status));
    if (ok) tc_fence_after();
    return ok;
  };
  auto commit = [&](uint64_t* bar) {
    if (leader) umma_commit(bar);
  };
  auto next = [](uint32_t& s, uint32_t& ph) {
    if (++s == kStages) {
      s = 0;
      ph ^= 1;
    }
  };
  auto qk = [&](int w, uint32_t s) {
    if (leader) {
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        constexpr uint32_t chunk = C::CHUNK_BYTES / 16;
        const uint32_t at = (kk >> 2) * chunk + (kk & 3) * 2;
        umma_ss(tm + 256 * w + 128, q_desc + (w * (C::TILE_BYTES / 16) + at), k_desc + (s * (C::TILE_BYTES / 16) + at),
                idesc_s, kk > 0 ? 1u : 0u);
      }
      umma_commit(&c->s_full[w]);
    }
    __syncwarp();
  };
  // Bit w: query tile w is active in tile t of the unit.
  auto flags = [](const Unit& u, int t) {
    const int kt = u.tile(t);
    const uint32_t f = (active(u.rows[0], kt) ? 1u : 0u) | (active(u.rows[1], kt) ? 2u : 0u);
    return __shfl_sync(0xffffffffu, f, 0);
  };
  for (uint32_t j = 0;; ++j) {
    const int slot = j & 3;
    if (!wait(&c->u_full[slot], (j >> 2) & 1)) break;
    const Unit& u = c->ring[slot];
    const int n = __shfl_sync(0xffffffffu, u.n, 0);
    if (n < 0) break;
    bool some[2] = {false, false};                    // O holds a product of this unit
    if (n > 0) {
      if (!wait(&c->kv_full[ks], kph)) break;
      for (int w = 0; w < 2; ++w) {
        if (!u.rows[w].live) continue;
        if (!wait(&c->q_full[w], nq[w] & 1)) break;
        ++nq[w];
        if (active(u.rows[w], u.tile(0))) qk(w, ks);
      }
      if (!ok) break;
      commit(&c->kv_empty[ks]);
      next(ks, kph);
    }
    // The tensor cores hold two or three products in their queue, so whatever this
    // warp does between two batches has to be short: tiles are looked up one
    // ahead, and V and the next K are waited for before P.
    uint32_t act = n > 0 ? flags(u, 0) : 0, act1 = n > 1 ? flags(u, 1) : 0;
    for (int t = 0; t < n; ++t) {
      const uint32_t vs = ks, vph = kph;
      next(ks, kph);
      if (!wait(&c->kv_full[vs], vph)) break;
      if (t + 1 < n && !wait(&c->kv_full[ks], kph)) break;
      uint32_t act2 = 0;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        if (act >> w & 1) {
          if (!some[w] && !wait(&c->o_free[w], ((nq[w] - 1) & 1) ^ 1)) break;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!wait(h ? &c->p_full[w] : &c->p_half[w], np[w] & 1)) break;
            if (leader) {
#pragma unroll
              for (int kk = 4 * h; kk < 4 * h + 4; ++kk)
                umma_ts(tm + 256 * w, tm + 256 * w + 128 + kk * 8, v_desc + (vs * (C::TILE_BYTES / 16) + kk * 128),
                        idesc_pv, some[w] || kk > 0 ? 1u : 0u);
            }
            __syncwarp();
          }
          if (!ok) break;
          if (act1 >> w & 1) qk(w, ks);
          ++np[w];
          some[w] = true;
        } else if (act1 >> w & 1) {
          qk(w, ks);
        }
        if (t + 2 < n) {
          if (w == 0) act2 = flags(u, t + 2);
        } else if (t + 1 == n && u.rows[w].live) {
          // Before the other query tile's last product, which waits for that one's P
          // (one wait a unit, so that the barrier's phases and the units go together).
          if (!some[w] && !wait(&c->o_free[w], ((nq[w] - 1) & 1) ^ 1)) break;
          commit(&c->q_empty[w]);
          commit(&c->o_full[w]);
        }
      }
      if (!ok) break;
      commit(&c->kv_empty[vs]);
      if (t + 1 < n) {
        commit(&c->kv_empty[ks]);
        next(ks, kph);
      }
      act = act1;
      act1 = act2;
    }
    if (!ok) break;
    __syncwarp();
    if (leader) mbar_arrive(&c->u_empty[slot]);
  }
  // Every tensor operation issued here has completed before TMEM is released.
  if (leader) {
    umma_commit(&c->mma_done);
    mbar_drain(&c->mma_done, 0, c->wait_ns);
  }
  __syncwarp();
}

// Bits x < n.
__device__ __forceinline__ uint32_t below(int n) { return n >= 32 ? ~0u : (1u << max(n, 0)) - 1; }

// Query tile w: thread (quarter wq, lane) owns row 32 wq + lane.
template <int D>
__device__ void softmax_rows(const Params& p, Ctl* c, uint8_t* smem, uint32_t tm, int w, int wq, int lane) {
  using C = Cfg<D>;
  const int row = wq * 32 + lane;
  const uint32_t to = tm + 256 * w + ((uint32_t)(wq * 32) << 16), ts = to + 128;
  const uint32_t stage = smem_u32(smem) + C::OFF_OUT + (4 * w + wq) * kOutBytes;
  const float sc = p.scale_log2;
  uint32_t it0 = 0, ns = 0, no = 0;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, c, p.status));
  };
  auto arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  for (uint32_t j = 0;; ++j) {
    const int slot = j & 3;
    if (!wait(&c->u_full[slot], (j >> 2) & 1)) return;
    const Unit& u = c->ring[slot];
    const Rows& rows = u.rows[w];
    const int n = u.n;
    if (n < 0) return;
    float m = -INFINITY, l = 0.f;       // the reference maximum (log2 units) and the sum relative to it
    for (int t = 0; t < n; ++t) {
      const int kt = u.tile(t);
      if (!active(rows, kt)) continue;
      const bool whole = kt < rows.whole_to && (kt >= rows.whole_from || kt < rows.whole_sink);
      const int k0 = kt * kTile;
      if (!whole && (k0 + kTile > u.hi || (k0 < u.lo && k0 + kTile > u.n_sink))) {
        // V rows that no row of the unit sees
        const uint32_t itv = it0 + 2 * t + 1;
        if (!wait(&c->kv_full[itv % kStages], (itv / kStages) & 1)) return;
        const int key = k0 + row;
        if (key >= u.hi || (key < u.lo && key >= u.n_sink)) {
          // the swizzle moves 16-byte pieces within a row's 128 bytes: the whole row is
          // zeroed, neighbouring lanes in other banks (in one, the padded prompts take 6% longer)
          uint4* v = reinterpret_cast<uint4*>(smem + C::OFF_KV + (itv % kStages) * C::TILE_BYTES + row * 128);
#pragma unroll
          for (int x = 0; x < C::CHUNKS; ++x)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[x * (C::CHUNK_BYTES / 16) + (e ^ (row & 7))] = make_uint4(0, 0, 0, 0);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      if (!wait(&c->s_full[w], ns & 1)) return;
      ++ns;
      tc_fence_after();
      float s[kTile];
#pragma unroll
      for (int x = 0; x < kTile / 32; ++x) tmem_ld32(ts + x * 32, s + x * 32);
      tmem_wait_ld();
      if (!whole) {
        // (a valid row's position is below n_k)
        // One bit a key (comparisons for every key took 2% of the 16,384 rows' time,
        // 6% of the padded prompts').
        const int c_hi = rows.first + row - k0, c_lo = p.window ? c_hi - p.window + 1 : 0, c_s = p.sinks - k0;
#pragma unroll
        for (int x = 0; x < kTile; x += 32) {
          const uint32_t see = below(c_hi + 1 - x) & (~below(c_lo - x) | below(c_s - x));
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (!(see >> e & 1)) s[x + e] = -INFINITY;
        }
      }
      float mx[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) mx[x] = fmaxf(s[x], s[x + 4]);
#pragma unroll
      for (int x = 8; x < kTile; x += 8)
#pragma unroll
        for (int y = 0; y < 4; ++y) mx[y] = max3(mx[y], s[x + y], s[x + y + 4]);
      const float top = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * sc;
      float corr = 1.f;
      bool moved = false;
      if (top > m + kRescale) {         // (m = -inf: any score is above)
        moved = m != -INFINITY;         // (a row that saw nothing so far has O = 0)
        corr = ex2(m - top);
        m = top;
      }
      // O's rescale first: S(t)'s arrival tells that P V of the tile before is done.
      if (__any_sync(0xffffffffu, moved)) {
        const float f = moved ? corr : 1.f;
#pragma unroll 1
        for (int x = 0; x < D / 16; ++x) {
          float o[16];
          tmem_ld16(to + x * 16, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] *= f;
          tmem_st16(to + x * 16, reinterpret_cast<const uint32_t*>(o));
        }
      }
      const float ref = m == -INFINITY ? 0.f : m;
      const uint64_t sc2 = pack2(sc, sc), neg2 = pack2(-ref, -ref);
      uint64_t acc[2] = {pack2(0.f, 0.f), pack2(0.f, 0.f)};
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float a, b;
          unpack2(ffma2(pack2(s[32 * x + 2 * e], s[32 * x + 2 * e + 1]), sc2, neg2), a, b);
          a = ex2(a);
          b = ex2(b);
          acc[e & 1] = fadd2(acc[e & 1], pack2(a, b));
          pk[e] = pack_bf16(a, b);
        }
        tmem_st16(ts + 16 * x, pk);
        if (x & 1) {
          tmem_wait_st();
          tc_fence_before();
          arrive(x == 1 ? &c->p_half[w] : &c->p_full[w]);
        }
      }
      float a, b;
      unpack2(fadd2(acc[0], acc[1]), a, b);
      l = l * corr + (a + b);
    }
    it0 += 2 * n;
    const int base = rows.row0 + wq * 32, r = base + lane, live = rows.live, bh = rows.bh, n_q = u.n_q;
    const bool valid = r < n_q;
    const int64_t at = (int64_t)bh * p.Nq + r;
    arrive(&c->u_empty[slot]);
    if (!live) continue;
    if (n > 0) {
      if (!wait(&c->o_full[w], no & 1)) return;
      ++no;
      tc_fence_after();
    }
    // O / l through shared memory: a lane holds a row of TMEM, and 16-byte stores
    // of 32 rows would touch 32 lines each (5 us a unit where its tiles take 20 to
    // 60); from the stage a store writes 4 rows of 128 bytes.
    const float inv = 1.f / l;
    const uint32_t mine = stage + lane * 128;
#pragma unroll 1
    for (int x = 0; x < D / 64; ++x) {
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float o[32];
        if (n > 0) {
          tmem_ld32(to + x * 64 + y * 32, o);
          tmem_wait_ld();
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint4 v = make_uint4(0, 0, 0, 0);   // a row that sees no key
          if (l != 0.f) {
            v.x = pack_bf16(o[8 * e + 0] * inv, o[8 * e + 1] * inv);
            v.y = pack_bf16(o[8 * e + 2] * inv, o[8 * e + 3] * inv);
            v.z = pack_bf16(o[8 * e + 4] * inv, o[8 * e + 5] * inv);
            v.w = pack_bf16(o[8 * e + 6] * inv, o[8 * e + 7] * inv);
          }
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(mine + (((4 * y + e) ^ (lane & 7)) << 4)), "r"(v.x),
                       "r"(v.y), "r"(v.z), "r"(v.w)
                       : "memory");
        }
      }
      if (n > 0 && x == D / 64 - 1) {
        tc_fence_before();
        arrive(&c->o_free[w]);
      }
      __syncwarp();
      const int row4 = lane >> 3, chunk = lane & 7;
      uint16_t* dst = p.out + ((int64_t)bh * p.Nq + base + row4) * D + x * 64 + chunk * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint4 v;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "r"(stage + (4 * i + row4) * 128 + ((chunk ^ ((4 * i + row4) & 7)) << 4))
                     : "memory");
        if (base + 4 * i + row4 < n_q) *reinterpret_cast<uint4*>(dst + (int64_t)4 * i * D) = v;
      }
      __syncwarp();
    }
    if (valid && p.lse) p.lse[at] = l != 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    window_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Params p) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // The base has to lie on the swizzle's 1024-byte boundary, as it does without
  // static shared memory (there is no room for a slack).
  uint8_t* smem = smem_raw;
  const uint32_t sb = smem_u32(smem);
  if (sb % 1024 != 0) {
    raise_status(p.status, SA_ERR_CUDA);
    return;
  }
  Ctl* c = reinterpret_cast<Ctl*>(smem + C::OFF_CTL);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int w = 0; w < 2; ++w) {
      mbar_init(&c->q_full[w], 1);
      mbar_init(&c->q_empty[w], 1);
      mbar_init(&c->s_full[w], 1);
      mbar_init(&c->p_half[w], 4);    // one lane of each softmax warp
      mbar_init(&c->p_full[w], 4);
      mbar_init(&c->o_full[w], 1);
      mbar_init(&c->o_free[w], 4);
    }
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&c->kv_full[s], 1);
      mbar_init(&c->kv_empty[s], 1);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&c->u_full[s], 1);
      mbar_init(&c->u_empty[s], 9);   // the MMA lane and one lane of each softmax warp
    }
    mbar_init(&c->mma_done, 1);
    c->wait_ns = kWaitNs;
    c->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&c->tmem_base)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c->tmem_base;

  // 384 x 168 registers at launch; 256 x 200 + 128 x 96 fit in them.
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    if (warp == 0 && lane == 0) producer<D>(&tmQ, &tmK, &tmV, p, c, sb);
    if (warp == 1) mma_issuer<D>(p, c, sb, tmem);
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    softmax_rows<D>(p, c, smem, tmem, (warp - 4) >> 2, warp & 3, lane);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

// 3-D map over [heads][N][D] bf16, box [1][128][64], 128-byte swizzle.
bool make_map(CUtensorMap* m, const void* base, int64_t heads, int64_t N, int D) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)N, (cuuint64_t)heads};
  cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)N * D * 2};
  cuuint32_t box[3] = {64, kTile, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
sa_status launch(const WindowArgs& x, cudaStream_t st) {
  using C = Cfg<D>;
  const sa_window_shape& s = x.shape;
  CUtensorMap mq, mk, mv;
  if (!make_map(&mq, x.q, s.B * s.Hq, s.Nq, D) || !make_map(&mk, x.k, s.B * s.Hkv, s.Nk, D) ||
      !make_map(&mv, x.v, s.B * s.Hkv, s.Nk, D))
    return set_error(SA_ERR_CUDA, "cuTensorMapEncodeTiled failed (driver entry point unavailable or bad map)");
  Params p{};
  p.out = static_cast<uint16_t*>(x.out);
  p.lse = x.lse;
  p.q_len = x.q_len;
  p.kv_len = x.kv_len;
  p.status = x.status;
  p.counter = static_cast<int32_t*>(x.ws);
  p.B = (int32_t)s.B;
  p.Hq = (int32_t)s.Hq;
  p.Hkv = (int32_t)s.Hkv;
  p.Nq = (int32_t)s.Nq;
  p.Nk = (int32_t)s.Nk;
  // a window that reaches past every key is none; so no position minus window leaves 31 bits
  p.window = x.window >= s.Nk ? 0 : (int32_t)x.window;
  p.sinks = (int32_t)min64(x.sinks, s.Nk);
  p.by_heads = (s.Hq / s.Hkv) % 2 == 0;
  const int64_t tiles = ceil_div(s.Nq, kTile);
  const int64_t pairs = s.B * (p.by_heads ? s.Hq / 2 : s.Hq), units = pairs * (p.by_heads ? tiles : ceil_div(tiles, 2));
  if (units > INT32_MAX / 2) return set_error(SA_ERR_UNSUPPORTED, "too many rows");
  p.pairs = (int32_t)pairs;
  p.num_units = (int32_t)units;
  p.scale_log2 = x.scale * kLog2e;
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (cudaFuncSetAttribute(window_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
    return set_error(SA_ERR_CUDA, "cudaFuncSetAttribute(window_tc_kernel) failed");
  if (units > sms && cudaMemsetAsync(p.counter, 0, sizeof(int32_t), st) != cudaSuccess)
    return set_error(SA_ERR_CUDA, "cudaMemsetAsync(work counter) failed");
  window_tc_kernel<D><<<(unsigned)min64(units, sms), kThreads, C::SMEM, st>>>(mq, mk, mv, p);
  return check_launch("window_tc_kernel");
}

}  // namespace

sa_status launch_window_tc(const WindowArgs& a, cudaStream_t st) {
  return a.shape.d == 128 ? launch<128>(a, st) : launch<64>(a, st);
}

}  // namespace sa
