// seq_sm100.cu -- tcgen05 / TMA forward of sequence attention (causal sliding
// window with sink tokens; bf16, head_dim up to 128, in kernels for 64 and 128).
//
// One pass over a query tile's visible key tiles with a running maximum and sum.
// An item is one head's pair of 128-query tiles (or a single tile where pairs
// would leave SMs idle): both tiles read the same key and value tiles, and
// while one tile's softmax runs on the exp unit the other's products run on the
// tensor pipe. Per key tile and query tile
//   S = Q K^T (fp32 in TMEM), P = 2^(c S - m) in registers, P as bf16 over S's
//   columns, O += P V with A = P from TMEM.
// The running maximum m of a row moves only when a tile raises it by more than
// 2^8, so O is rescaled in TMEM (by the softmax threads) a few times per row
// at most. P is rounded to bf16 (off by 2^-8 of each term at most; terms of
// either sign average out), or split in two where a row has few keys
// (kFewKeys); the row sum takes the unrounded fp32 values.
//
// TMEM: per query tile a ring of NB S buffers of KT keys, and O. With two or three
// buffers the next S is there when a softmax step ends; steps of 64 keys make
// room for them (a single 128-key buffer: 579 us against 505, at the time, for
// 16384 tokens, 16 heads x 128, window 4096; 61 us against 49 for two ragged
// 4096-token sequences, 16 heads x 64, window 512).
//
// Warps: 0-3 and 4-7 one softmax warpgroup per query tile (thread = row), 8
// the TMA producer, 9 issues S and owns TMEM, 10 issues O += P V. Keys and
// values have ring slots of their own, so S starts before V has landed.
//
// Bound: per 128 x 128 tile of a head the tensor pipe needs 8 hd cycles (S and
// O at 8192 FLOP per cycle and SM) and the exp unit 1024 (16 per cycle), so
// head_dim 128 is bound by both alike, head_dim 64 by the exp unit. Measured: 437 us
// for the first case above (1100 TFLOP/s), 44 us for the second. The tensor cores are
// then busy for 71% of the time, with what S costs because N = 64 (both operands come
// from shared memory; the products themselves are 52%), the exp unit for 55%: a step
// goes through two products, the softmax and four barriers, each waiting for the
// one before, and TMEM has no room for more steps in flight. On the exp unit's
// side there is nothing to gain: a polynomial on the FMA pipe for a quarter to all
// of the exponentials, or two threads per row, left the time as it was; one warp
// that issues all products took 759 us, four (one for each product of a query
// tile) 470.
#include "seq_tc.cuh"

namespace swin {
namespace {

using namespace ptx;

constexpr int kSeqThreads = 384;
constexpr int kSeqProducer = 8, kSeqMma = 9, kSeqMma2 = 10;
constexpr float kSeqMove = 8.f;   // the running maximum moves by more than this (log2)

struct SeqMaps {
  CUtensorMap q, k, v;
};

// What an item is, for every role alike.
template <int KT>
struct SeqItem {
  int b, h, i0, n;       // first query, tokens of the sequence
  KeyTiles u, kt[2];     // key tiles of the whole item and of each query tile
  int steps;             // of the item (0: all padding)
  bool has[2];           // query tiles that are not all padding
  __device__ __forceinline__ bool needs(int w, int tile) const {
    return has[w] && tile <= kt[w].hi && (tile >= kt[w].lo || tile < kt[w].s);
  }
  __device__ __forceinline__ bool few(int w) const { return kt[w].count() * KT <= kFewKeys; }
};
template <int KT>
__device__ __forceinline__ SeqItem<KT> seq_item(const SeqParams& p, long long t, int nq) {
  SeqItem<KT> it;
  const int bh = p.B * p.H;
  const int per = (p.S + kRows * nq - 1) / (kRows * nq);
  const int r = (int)(t / bh), z = (int)(t - (long long)r * bh);
  it.b = z / p.H;
  it.h = z - it.b * p.H;
  it.i0 = (per - 1 - r) * kRows * nq;   // the longest rows first
  it.n = seq_len(p, it.b);
  it.steps = 0;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int i0 = it.i0 + w * kRows;
    it.has[w] = w < nq && i0 < it.n;
    it.kt[w] = seq_key_tiles(p, i0, min(it.n, i0 + kRows), KT);
  }
  if (it.has[0]) {
    it.u = seq_key_tiles(p, it.i0, min(it.n, it.i0 + kRows * nq), KT);
    it.steps = it.u.count();
  }
  return it;
}

template <int HD>
struct SeqFwdCfg {
  static constexpr int KT = 64;                 // keys of a step
  static constexpr int NB = HD > 64 ? 2 : 3;    // S buffers of a query tile
  static constexpr uint32_t kTileCols = NB * KT + HD;  // TMEM columns of a query tile
  static constexpr uint32_t kOCol = NB * KT;           // O behind the buffers
  static_assert(2 * kTileCols <= 512, "TMEM columns");
  static constexpr uint32_t kQTile = kRows * HD * 2;
  static constexpr uint32_t kSlot = KT * HD * 2;
  static constexpr int kQBufs = HD > 64 ? 1 : 2;
  static constexpr int kSlots = HD > 64 ? 8 : 16;       // ring of key / value tiles
  static constexpr uint32_t kRing = kQBufs * 2 * kQTile;
  static constexpr uint32_t kBars = kRing + kSlots * kSlot;
  static constexpr int kNumBars = 2 * kQBufs + 2 * kSlots + 6 * NB + 2 + 2 + 1;
  static constexpr uint32_t kFeedAt = kBars + (kNumBars * 8 + 15) / 16 * 16;
  static constexpr uint32_t kTotal = kFeedAt + sizeof(Feed<SeqItem<KT>>) + 16;   // TMEM address, abort
  static constexpr uint32_t kSmem = kTotal + 1024;
};

template <int HD>
__global__ void __launch_bounds__(kSeqThreads, 1)
    seq_fwd_kernel(const __grid_constant__ SeqParams p, const __grid_constant__ SeqMaps maps,
                   const int nq) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  using C = SeqFwdCfg<HD>;
  constexpr int NQ = C::kQBufs, NS = C::kSlots, NB = C::NB, KT = C::KT;
  constexpr uint32_t QB = C::kQTile, SB = C::kSlot;
  uint8_t* qbuf = smem;
  uint8_t* kv = smem + C::kRing;
  uint64_t* bars = (uint64_t*)(smem + C::kBars);
  uint64_t* q_full = bars;
  uint64_t* q_empty = q_full + NQ;
  uint64_t* kv_full = q_empty + NQ;
  uint64_t* kv_empty = kv_full + NS;
  uint64_t* s_full = kv_empty + NS;   // [2][NB] per query tile and buffer: S is there,
  uint64_t* p_full = s_full + 2 * NB; //   P is written,
  uint64_t* o_done = p_full + 2 * NB; //   O += P V is done
  uint64_t* o_empty = o_done + 2 * NB;   // [2] per query tile: O is read
  uint64_t* drain = o_empty + 2;      // [2]: one per MMA-issuing thread
  uint64_t* never = drain + 2;
  using Item = SeqItem<KT>;
  Feed<Item>* feed = (Feed<Item>*)(smem + C::kFeedAt);
  uint32_t* tmem_slot = (uint32_t*)(smem + C::kFeedAt + sizeof(Feed<Item>));
  volatile int* abort = (volatile int*)(tmem_slot + 1);

  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NQ; ++i) { mbar_init(&q_full[i], 1); mbar_init(&q_empty[i], 1); }
    for (int i = 0; i < NS; ++i) { mbar_init(&kv_full[i], 1); mbar_init(&kv_empty[i], 1); }
    for (int i = 0; i < 2 * NB; ++i) {
      mbar_init(&s_full[i], 1); mbar_init(&p_full[i], kWg); mbar_init(&o_done[i], 1);
    }
    for (int i = 0; i < 2; ++i) { mbar_init(&o_empty[i], kWg); mbar_init(&drain[i], 1); }
    mbar_init(never, 1);
    feed_init(feed, 2 + 8);   // the MMA and softmax warps
    abort[0] = abort[1] = 0;   // [1]: warps that recompute rows
    fence_mbar_init();
  }
  if (warp == kSeqProducer && lane == 0) {
    prefetch_tmap(&maps.q);
    prefetch_tmap(&maps.k);
    prefetch_tmap(&maps.v);
  }
  if (warp == kSeqMma) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  FeedRead<Item> rd{feed};

  if (warp == kSeqProducer) {
    if (lane == 0) {
      FeedWrite<Item> out{feed};
      long long t = blockIdx.x;
      bool more = true;
      Ring<NQ> rq;
      Ring<NS> rs;
      long long k = 0, e = 0;   // items with work, ring slots filled
      bool ok = true;
      do {
        const Item it = seq_item<KT>(p, t, nq);
        if (!out.put(it, true, abort, p.status)) break;
        if (it.steps) {
          const int kh = it.h / p.G;
          if (!seq_wait(&q_empty[rq.s], rq.parity ^ 1, abort, p.status)) break;
          mbar_arrive_expect_tx(&q_full[rq.s], nq * QB);
          for (int w = 0; w < nq; ++w)
            load_tokens<kRows, HD>(&maps.q, qbuf + (rq.s * 2 + w) * QB, it.h, it.i0 + w * kRows,
                                   it.b, &q_full[rq.s]);
          rq.next();
          ++k;
          for (int x = 0; x < it.steps && ok; ++x)
            for (int kvi = 0; kvi < 2; ++kvi, ++e, rs.next()) {
              if (!seq_wait(&kv_empty[rs.s], rs.parity ^ 1, abort, p.status)) {
                ok = false;
                break;
              }
              mbar_arrive_expect_tx(&kv_full[rs.s], SB);
              load_tokens<KT, HD>(kvi ? &maps.v : &maps.k, kv + rs.s * SB, kh, it.u.tile(x) * KT,
                                  it.b, &kv_full[rs.s]);
            }
        }
        // ask when the item's loads are out, not before: an early question hands
        // the next items out in order, whoever is busy
        more = ok && out.next(&t, abort, p.status);
      } while (more);
      if (!*abort) out.put(Item(), false, abort, p.status);
      if (*abort) {  // let copies and answers in flight land before the CTA leaves
        for (long long j = (e > NS ? e - NS : 0); j < e; ++j)
          mbar_drain(&kv_full[j % NS], (uint32_t)((j / NS) & 1), kTestLimitNs * 100);
        for (long long j = (k > NQ ? k - NQ : 0); j < k; ++j)
          mbar_drain(&q_full[j % NQ], (uint32_t)((j / NQ) & 1), kTestLimitNs * 100);
        out.drain();
      }
    }
  } else if (warp == kSeqMma) {
    // S = Q_w K^T of both query tiles, key tile by key tile. The whole warp walks
    // along and one elected lane issues.
    constexpr uint32_t idesc_s = idesc_bf16(kRows, KT, 0, 0);
    const uint32_t q0 = smem_u32(qbuf), k0 = smem_u32(kv);
    Ring<NQ> rq;
    Ring<NS> rs;
    Ring<NB> rb[2];   // S buffers of each query tile
    bool ok = true;
    while (ok) {
      const Item* item = rd.next(abort, p.status);
      if (!item) break;
      const Item it = *item;
      if (!it.steps) continue;
      if (!warp_wait(&q_full[rq.s], rq.parity, abort, p.status)) break;
      for (int x = 0; x < it.steps && ok; ++x) {
        const int tile = it.u.tile(x);
        ok = warp_wait(&kv_full[rs.s], rs.parity, abort, p.status);
        if (!ok) break;
        const uint64_t kd = kmajor_base(uniform(k0 + rs.s * SB));
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          if (!ok || !it.needs(w, tile)) continue;
          // the buffer's previous O += P V is done
          ok = warp_wait(&o_done[w * NB + rb[w].s], rb[w].parity ^ 1, abort, p.status);
          if (!ok) continue;
          tc_fence_after();
          const uint64_t qd = kmajor_base(uniform(q0 + (rq.s * 2 + w) * QB));
          const uint32_t to = uniform(tmem + w * C::kTileCols + rb[w].s * KT);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk)
              umma_ss(to, qd + kmajor_step<kRows>(kk), kd + kmajor_step<KT>(kk), idesc_s, kk > 0);
            umma_commit(&s_full[w * NB + rb[w].s]);
          }
          __syncwarp();
          rb[w].next();
        }
        if (ok && elect_one()) umma_commit(&kv_empty[rs.s]);
        __syncwarp();
        rs.next();
        rs.next();   // past the value tile
      }
      if (ok && elect_one()) umma_commit(&q_empty[rq.s]);
      __syncwarp();
      rq.next();
    }
    if (__any_sync(0xffffffffu, *abort) && elect_one()) {   // the lane that issued
      umma_commit(&drain[0]);
      mbar_drain(&drain[0], 0, kTestLimitNs * 100);
    }
  } else if (warp == kSeqMma2) {
    // O += P V of both query tiles, as soon as each P is written (all lanes walk
    // along: they zero the padding rows of a last value tile)
    constexpr uint32_t idesc_o = idesc_bf16(kRows, HD, 0, 1);
    const uint32_t v0 = smem_u32(kv);
    Ring<NS> rs;
    Ring<NB> rb[2];
    uint32_t items[2] = {0, 0};   // of a query tile so far
    bool ok = true;
    while (ok) {
      const Item* item = rd.next(abort, p.status);
      if (!item) break;
      const Item it = *item;
      if (!it.steps) continue;
      uint32_t on[2] = {0, 0};    // products add to O
      for (int x = 0; x < it.steps && ok; ++x) {
        const int tile = it.u.tile(x);
        rs.next();                // past the key tile
        if (!warp_wait(&kv_full[rs.s], rs.parity, abort, p.status)) {
          ok = false;
          break;
        }
        if ((tile + 1) * KT > it.n) {
          zero_rows<KT, HD>(kv + rs.s * SB, it.n - tile * KT);
          fence_proxy_async();
          __syncwarp();
        }
        const uint64_t v_s = mnmajor_base<KT, HD>(uniform(v0 + rs.s * SB));
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          if (!ok || !it.needs(w, tile)) continue;
          // a new item overwrites O: the previous item's epilogue has read it
          ok = (on[w] || warp_wait(&o_empty[w], (items[w] & 1) ^ 1, abort, p.status)) &&
               warp_wait(&p_full[w * NB + rb[w].s], rb[w].parity, abort, p.status);
          if (!ok) continue;
          tc_fence_after();
          const uint32_t a = uniform(tmem + w * C::kTileCols + rb[w].s * KT);
          const uint32_t o = uniform(tmem + w * C::kTileCols + C::kOCol);
          if (elect_one()) {
            if (it.few(w)) {
#pragma unroll
              for (int kk = 0; kk < KT / 16; ++kk) {
                umma_ts(o, a + kk * 8, v_s + mnmajor_step(kk), idesc_o, on[w] | (kk > 0));
                umma_ts(o, a + KT / 2 + kk * 8, v_s + mnmajor_step(kk), idesc_o, 1);
              }
            } else {
#pragma unroll
              for (int kk = 0; kk < KT / 16; ++kk)
                umma_ts(o, a + kk * 8, v_s + mnmajor_step(kk), idesc_o, on[w] | (kk > 0));
            }
            umma_commit(&o_done[w * NB + rb[w].s]);
          }
          __syncwarp();
          on[w] = 1;
          rb[w].next();
        }
        if (ok && elect_one()) umma_commit(&kv_empty[rs.s]);
        __syncwarp();
        rs.next();
      }
#pragma unroll
      for (int w = 0; w < 2; ++w) items[w] += it.has[w];
    }
    if (__any_sync(0xffffffffu, *abort) && elect_one()) {
      umma_commit(&drain[1]);
      mbar_drain(&drain[1], 0, kTestLimitNs * 100);
    }
  } else if (warp < 8) {
    // Softmax and epilogue of query tile w (thread = row = TMEM lane).
    const int w = warp >> 2, row = threadIdx.x & (kWg - 1);
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t base = tmem + lane_base + w * C::kTileCols, o_col = base + C::kOCol;
    const float2 sc = make_float2(p.scale_log2, p.scale_log2);
    // Waits name a round of a barrier by its parity; none can be mistaken here: a
    // buffer's next round needs this warp's P, its last one ended before S was
    // written again.
    uint64_t *sf = s_full + w * NB, *pf = p_full + w * NB, *od = o_done + w * NB;
    Ring<NB> rb, last;   // this product's buffer and the one before's
    while (const Item* item = rd.next(abort, p.status)) {
      const Item it = *item;
      const int i0 = it.i0 + w * kRows, i = i0 + row;
      const bool stored = w < nq && i < p.S, real = i < it.n;
      const long long orow = ((long long)it.b * p.S + i) * p.H + it.h;
      __nv_bfloat16* dst = (__nv_bfloat16*)p.out + orow * p.hd;
      if (p.test_timeout && it.steps) mbar_wait(never, 0, abort, p.status, kTestLimitNs);
      const KeyTiles kt = w ? it.kt[1] : it.kt[0];
      const bool has = w ? it.has[1] : it.has[0], few = w ? it.few(1) : it.few(0);
      const int steps = has ? kt.count() : 0;
      float m = -INFINITY, l = 0.f;
      for (int x = 0; x < steps; ++x) {
        const int k0 = kt.tile(x) * KT;
        const uint32_t s_col = base + rb.s * KT;
        seq_wait(&sf[rb.s], rb.parity, abort, p.status);
        tc_fence_after();
        float v[KT];
        float m0 = -INFINITY, m1 = m0, m2 = m0, m3 = m0;
        const bool plain =
            k0 + KT - 1 <= i0 && (i0 + kRows - 1 - k0 < p.window || k0 + KT <= p.sinks);
        const int hi = i - k0, lo = hi - p.window + 1, sk = p.sinks - k0;
        auto mask = [&](int c0) {
          const uint32_t see = column_mask(lo - c0, hi - c0, sk - c0);
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (!(see & (1u << c))) v[c0 + c] = -INFINITY;
        };
        auto top = [&](int c0) {
#pragma unroll
          for (int c = c0; c < c0 + 32; c += 8) {
            m0 = fmaxf(fmaxf(m0, v[c]), v[c + 1]);
            m1 = fmaxf(fmaxf(m1, v[c + 2]), v[c + 3]);
            m2 = fmaxf(fmaxf(m2, v[c + 4]), v[c + 5]);
            m3 = fmaxf(fmaxf(m3, v[c + 6]), v[c + 7]);
          }
        };
        // head_dim 128: the first half's maxima while the second half is on its way
        // (440 us against 480 for 16384 tokens, 16 heads, window 4096); at 64 both
        // halves at once (44 us against 46 for two sequences of 4096, window 512)
        __syncwarp();
        tmem_ld32(s_col, v);
        if constexpr (HD > 64) {
          tmem_wait_ld_regs(v);
          tmem_ld32(s_col + 32, v + 32);
          if (!plain) mask(0);
          top(0);
          tmem_wait_ld_regs(v + 32);
          if (!plain) mask(32);
        } else {
          tmem_ld32(s_col + 32, v + 32);
          tmem_wait_ld_regs(v);
          reg_fence32(v + 32);
          if (!plain) {
            mask(0);
            mask(32);
          }
          top(0);
        }
        top(32);
        const float mt = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3)) * p.scale_log2;
        const bool move = mt > m + kSeqMove;
        const float f = move ? ex2(m - mt) : 1.f;   // 0 while m = -inf
        if (move) {
          l *= f;
          m = mt;
        }
        if (x > 0 && __any_sync(0xffffffffu, move)) {
          // O is free of the previous product before it is scaled
          seq_wait(&od[last.s], last.parity, abort, p.status);
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < HD; c += 16) {
            float o[16];
            __syncwarp();
            tmem_ld16(o_col + c, o);
            tmem_wait_ld_regs16(o);
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] *= f;
            __syncwarp();
            tmem_st16u(o_col + c, reinterpret_cast<const uint32_t*>(o));
          }
        }
        // a row whose keys so far are all masked subtracts 0 (P = 0)
        const float mu = m == -INFINITY ? 0.f : m;
        const float2 nm = make_float2(-mu, -mu);
        float2 la = make_float2(0.f, 0.f), lb = la;
        if (few) {   // hi and lo parts, 16 columns at a time (registers)
#pragma unroll
          for (int c0 = 0; c0 < KT; c0 += 16) {
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int c = 0; c < 16; c += 2) {
              const float2 a = __ffma2_rn(make_float2(v[c0 + c], v[c0 + c + 1]), sc, nm);
              const float2 e = make_float2(ex2(a.x), ex2(a.y));
              la = __fadd2_rn(la, e);
              split_pair(e, hi[c / 2], lo[c / 2]);
            }
            __syncwarp();
            tmem_st8u(s_col + c0 / 2, hi);
            tmem_st8u(s_col + KT / 2 + c0 / 2, lo);
          }
        } else {
#pragma unroll
          for (int c0 = 0; c0 < KT; c0 += 32) {
            uint32_t pk[16];
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
              const float2 a = __ffma2_rn(make_float2(v[c0 + c], v[c0 + c + 1]), sc, nm);
              const float2 b = __ffma2_rn(make_float2(v[c0 + c + 2], v[c0 + c + 3]), sc, nm);
              const float2 ea = make_float2(ex2(a.x), ex2(a.y)), eb = make_float2(ex2(b.x), ex2(b.y));
              la = __fadd2_rn(la, ea);
              lb = __fadd2_rn(lb, eb);
              pk[c / 2] = pack_bf16(ea.x, ea.y);
              pk[c / 2 + 1] = pack_bf16(eb.x, eb.y);
            }
            __syncwarp();
            tmem_st16u(s_col + c0 / 2, pk);
          }
        }
        l += (la.x + la.y) + (lb.x + lb.y);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&pf[rb.s]);
        last = rb;
        rb.next();
      }
      if (!has) {   // padding: zeros
        if (w < nq) {
          uint4 z[8] = {};
#pragma unroll
          for (int c = 0; c < HD; c += 64)
            store_rows_clipped<8>(z, stored ? dst + c : nullptr, (p.hd - c) / 8);
          if (stored && p.lse) p.lse[orow] = 0.f;
        }
        continue;
      }
      seq_wait(&od[last.s], last.parity, abort, p.status);   // the last product
      tc_fence_after();
      const bool live = !*abort;
      const float inv = 1.f / l;
      bool bad = !(fabsf(inv) <= 3.4e38f);
#pragma unroll
      for (int c = 0; c < HD; c += 64) {
        float o[64];
        tmem_load_cols<64>(o_col + c, o);
        tmem_wait_ld_regs(o);
        reg_fence32(o + 32);
        if (c + 64 >= HD) {
          tc_fence_before();
          mbar_arrive(&o_empty[w]);
        }
        float2 odd = make_float2(0.f, 0.f);   // NaN once any entry is not finite
#pragma unroll
        for (int j = 0; j < 64; j += 2)
          odd = __ffma2_rn(make_float2(o[j], o[j + 1]), make_float2(0.f, 0.f), odd);
        bad |= !(odd.x + odd.y == 0.f);
        if (!real) {
#pragma unroll
          for (int j = 0; j < 64; ++j) o[j] = 0.f;
        }
        uint4 a[8];
        pack_chunks<8>(o, real ? inv : 0.f, a);
        store_rows_clipped<8>(a, stored && live ? dst + c : nullptr, (p.hd - c) / 8);
      }
      if (stored && live && p.lse) p.lse[orow] = real ? (m + __log2f(l)) / kSeqLog2e : 0.f;
      // a row whose sum is NaN has a NaN logit of its own: it is as it should be
      uint32_t fix = __ballot_sync(0xffffffffu, bad && real && live && l == l);
      if (fix) {
        if (lane == 0) atomicAdd((int*)abort + 1, 1);
        while (fix) {
          const int r = __ffs(fix) - 1;
          fix &= fix - 1;
          __syncwarp();
          fix_out_row<__nv_bfloat16>(p, it.b, it.h, i0 + (warp & 3) * 32 + r);
        }
        __syncwarp();
        if (lane == 0) atomicAdd((int*)abort + 1, -1);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kSeqMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int HD>
cudaError_t fwd_launch(const SeqParams& p, cudaStream_t st) {
  using C = SeqFwdCfg<HD>;
  SeqMaps maps;
  if (!encode_tokens(&maps.q, p.q, p, p.H, p.qs, kRows) ||
      !encode_tokens(&maps.k, p.k, p, p.K, p.ks, C::KT) ||
      !encode_tokens(&maps.v, p.v, p, p.K, p.ks, C::KT))
    return cudaErrorInvalidValue;
  static_assert(C::kSmem <= kSmemLimit, "shared memory");
  const cudaError_t e = allow_smem<seq_fwd_kernel<HD>>(C::kSmem);
  if (e != cudaSuccess) return e;
  // pairs of query tiles, unless they leave more than half of the SMs idle
  const long long tiles = (p.S + kRows - 1) / kRows, bh = (long long)p.B * p.H;
  const int nq = tiles > 1 && (tiles + 1) / 2 * bh > kSeqSms / 2 ? 2 : 1;
  const long long items = (tiles + nq - 1) / nq * bh;
  if (items > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  seq_fwd_kernel<HD><<<(unsigned)items, kSeqThreads, C::kSmem, st>>>(p, maps, nq);
  note_launch();
  return cudaGetLastError();
}

}  // namespace

bool seq_fast_supported(int dtype, int hd) {
  return dtype == SWIN_DTYPE_BF16 && hd <= 128;
}

cudaError_t seq_fast_forward(const SeqParams& p, cudaStream_t st) {
  return p.hd <= 64 ? fwd_launch<64>(p, st) : fwd_launch<128>(p, st);
}

}  // namespace swin
