// seq_bwd_sm100.cu -- tcgen05 / TMA backward of sequence attention (bf16,
// head_dim up to 128, in kernels for 64 and 128).
//
// Two kernels, because dQ sums over keys and dK, dV over queries, and a sum
// that crosses blocks would need atomics, whose order changes results:
//  * query side, item = (head, 128 queries): S = Q K^T, dP = dO V^T over the
//    visible keys in steps of 64, P = 2^(c S - L), dS = P (dP - D), dQ += dS K;
//  * key side, item = (128 keys, query heads, queries; DkvPlan): S^T = K Q^T,
//    dP^T = V dO^T over the queries in steps of 64 (thread = key), dV += P^T dO,
//    dK += dS^T Q.
// One kernel template runs both: a stationary pair of 128-row tiles (Q, dO or
// K, V), a streamed pair of 64-row tiles, two or three TMEM buffers of S | dP
// (64 + 64 columns) and the accumulators. P and dS are rounded to bf16 over their own
// columns and are the A operand of the gradient products from TMEM (off by
// 2^-8 of each term at most); sums are fp32 in TMEM.
//
// D_i = dO_i.o_i uses the stored, rounded o. Where a row sees few keys its dS is
// a small difference of dP and D and that rounding would show, so items of at
// most kFewKeys keys take D = sum_j P_ij dP_ij from a pass of their own
// first (and leave it for the key side): an error of 0.11 of the gradients' RMS
// in the first rows of a sequence becomes that of other rows. Longer rows would
// pay two more products per step for an error already below the outputs' own
// rounding.
//
// Warps: a softmax warpgroup per TMEM buffer, taking the steps in turn (thread =
// row); then the TMA producer, a warp that issues S and dP and owns TMEM, and one
// that issues the gradient products. Bound: the tensor pipe at head_dim 128 (per
// 128 x 64 step S and dP with N = 64, which read both operands from shared memory
// at 1.5 times the cost of N = 128, and one or two gradient products), the exp
// unit and the softmax warps' latencies at 64. Measured: 8192 causal tokens, 8
// heads x 128 (2 key heads), 476 us for the whole backward, 208 us of them the
// query side (tensor cores busy 73% of the time, 52% without what N = 64 loses) and
// 294 us the key side (64% and 47%) when profiled; two ragged sequences of 4096, 16 heads
// x 64, window 512: 132 us (58 and 74 when profiled).
#include "seq_tc.cuh"

namespace swin {
namespace {

using namespace ptx;

constexpr int kStep = 64;         // keys (queries) of a step
// TMEM: NB buffers of S | dP, then ND accumulators of HD columns (dQ) or 2 HD
// (dV, dK). Three buffers let a step's products start while the two softmax
// pairs work on those before; head_dim 128 leaves the key side two.
template <int HD, bool KEYS>
struct BwdTmem {
  static constexpr int NB = KEYS && HD > 64 ? 2 : 3;
  static constexpr int ND = KEYS || HD > 64 ? 1 : 2;
  static constexpr int NW = NB;                 // softmax warpgroups, one per buffer
  static constexpr int kSoft = 4 * NW;          // their warps; then producer and MMA warps
  static constexpr int kThreads = (kSoft + 3) * 32;
  static constexpr uint32_t kAccCol = NB * 2 * kStep;
  static constexpr uint32_t kAccCols = KEYS ? 2 * HD : HD;
  static_assert(kAccCol + ND * kAccCols <= 512, "TMEM columns");
};

struct BwdMaps {
  CUtensorMap a0, a1, b0, b1;   // stationary pair, streamed pair
};

// An item of either side, for every role alike: `steps` streamed tiles a pass.
template <bool KEYS>
struct BwdItem {
  DkvItem d;             // key side
  KeyTiles kt;           // query side: key steps
  int b, h, r0, n;       // query side: head and first query; key side: r0 = first key
  int steps, passes;
  // Whether the query rows of a step (key side: from `row`) see few keys (kFewKeys).
  __device__ __forceinline__ bool few(const SeqParams& p, int row) const {
    if constexpr (KEYS) return min(row + kStep, p.window + p.sinks) <= kFewKeys;
    else return passes == 2;
  }
};
// Walks an item's steps in order: first streamed token and query head of each (with
// what it needs of the item in registers).
template <bool KEYS>
struct StepWalk {
  int row, head, x;
  int i0, i1, s, lo;
  __device__ __forceinline__ explicit StepWalk(const BwdItem<KEYS>& it)
      : i0(KEYS ? it.d.i0 : 0), i1(KEYS ? it.d.i1 : 0), s(it.kt.s), lo(it.kt.lo * kStep) {
    head = KEYS ? it.d.h0 : it.h;
    start();
  }
  __device__ __forceinline__ void start() {
    x = 0;
    row = KEYS ? i0 : (s > 0 ? 0 : lo);
  }
  __device__ __forceinline__ void next() {
    ++x;
    row += kStep;
    if constexpr (KEYS) {
      if (row >= i1) {
        row = i0;
        ++head;
      }
    } else {
      if (x == s) row = lo;
    }
  }
};
template <bool KEYS>
__device__ __forceinline__ BwdItem<KEYS> bwd_item(const SeqParams& p, long long t) {
  BwdItem<KEYS> it;
  it.steps = 0;
  it.passes = 1;
  if constexpr (KEYS) {
    it.d = dkv_item(p, t);
    it.b = it.d.b;
    it.h = it.d.kh;
    it.n = it.d.n;
    it.r0 = it.d.tile * kRows;
    if (it.d.i0 < it.d.i1)
      it.steps = (it.d.i1 - it.d.i0 + kStep - 1) / kStep * (it.d.h1 - it.d.h0);
  } else {
    const int bh = p.B * p.H, tiles = (p.S + kRows - 1) / kRows;
    const int r = (int)(t / bh), z = (int)(t - (long long)r * bh);
    it.b = z / p.H;
    it.h = z - it.b * p.H;
    it.n = seq_len(p, it.b);
    it.r0 = (tiles - 1 - r) * kRows;   // the longest rows first
    if (it.r0 < it.n) {
      it.kt = seq_key_tiles(p, it.r0, min(it.n, it.r0 + kRows), kStep);
      it.steps = it.kt.count();
      it.passes = it.steps * kStep <= kFewKeys ? 2 : 1;
    }
  }
  return it;
}

template <int HD, bool KEYS>
struct BwdCfg {
  static constexpr uint32_t kTile = kRows * HD * 2;    // stationary tile
  static constexpr uint32_t kSub = kStep * HD * 2;     // streamed tile
  static constexpr int kABufs = HD > 64 ? 1 : 2;
  static constexpr int kStages = HD > 64 ? 4 : 6;
  static constexpr uint32_t kRing = kABufs * 2 * kTile;
  static constexpr uint32_t kLd = kRing + kStages * 2 * kSub;
  static constexpr uint32_t kXch = kLd + (KEYS ? kStages * kStep : kABufs * kRows) * 8;
  static constexpr uint32_t kBars = kXch + 3 * kRows * 4;
  static constexpr uint32_t kFeedAt = kBars + 8 * 40;
  static constexpr uint32_t kTotal = kFeedAt + sizeof(Feed<BwdItem<KEYS>>) + 16;
  static constexpr uint32_t kSmem = kTotal + 1024;
};

// NC fp32 columns (the first hd of them) of a row times `mul`, zero where !keep, to
// bf16 rows or fp32 partial rows (dst: this lane's row or nullptr); says whether
// any is not finite. Arrives on `empty` once the columns are in registers.
template <int NC>
__device__ __forceinline__ bool store_grad(uint32_t col, float mul, bool keep, void* dst,
                                           bool f32, int hd, uint64_t* empty) {
  float o[NC];
  __syncwarp();
#pragma unroll
  for (int c = 0; c < NC; c += 32) tmem_ld32(col + c, o + c);
  tmem_wait_ld_regs(o);
#pragma unroll
  for (int c = 32; c < NC; c += 32) reg_fence32(o + c);
  if (empty) {
    tc_fence_before();
    mbar_arrive(empty);
  }
  float2 odd = make_float2(0.f, 0.f);   // NaN once any entry is not finite
#pragma unroll
  for (int j = 0; j < NC; j += 2)
    odd = __ffma2_rn(make_float2(o[j], o[j + 1]), make_float2(0.f, 0.f), odd);
#pragma unroll
  for (int j = 0; j < NC; ++j) o[j] = keep ? o[j] * mul : 0.f;
  if (f32) {
#pragma unroll
    for (int c = 0; c < NC; c += 32) {
      uint4 a[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        a[j] = make_uint4(__float_as_uint(o[c + 4 * j]), __float_as_uint(o[c + 4 * j + 1]),
                          __float_as_uint(o[c + 4 * j + 2]), __float_as_uint(o[c + 4 * j + 3]));
      store_rows_clipped<8>(a, dst ? (float*)dst + c : nullptr, (hd - c) / 4);
    }
  } else {
    constexpr int W = 32;   // channels of a store round (64: 3% slower in all)
#pragma unroll
    for (int c = 0; c < NC; c += W) {
      uint4 a[W / 8];
      pack_chunks<W / 8>(o + c, 1.f, a);
      store_rows_clipped<W / 8>(a, dst ? (__nv_bfloat16*)dst + c : nullptr, (hd - c) / 8);
    }
  }
  return !(odd.x + odd.y == 0.f);
}

template <int HD, bool KEYS>
__global__ void __launch_bounds__(BwdTmem<HD, KEYS>::kThreads, 1)
    seq_bwd_kernel(const __grid_constant__ SeqParams p,
                   const __grid_constant__ BwdMaps maps) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  using C = BwdCfg<HD, KEYS>;
  using TM = BwdTmem<HD, KEYS>;
  constexpr int NA = C::kABufs, NS = C::kStages, NB = TM::NB, ND = TM::ND, NW = TM::NW;
  constexpr int kSoft = TM::kSoft, kBProducer = kSoft, kBMma = kSoft + 1, kBMma2 = kSoft + 2;
  constexpr uint32_t TB = C::kTile, SB = C::kSub;
  uint8_t* abuf = smem;
  uint8_t* ring = smem + C::kRing;
  float* lds = (float*)(smem + C::kLd);   // -L and -D: of a stage's queries, of a Q tile's
  float* xch = (float*)(smem + C::kXch);
  uint64_t* bars = (uint64_t*)(smem + C::kBars);
  uint64_t* a_full = bars;
  uint64_t* a_empty = a_full + NA;
  uint64_t* b_full = a_empty + NA;
  uint64_t* b_empty = b_full + NS;
  uint64_t* s_full = b_empty + NS;    // [NB] per TMEM buffer
  uint64_t* p_full = s_full + NB;
  uint64_t* g_done = p_full + NB;
  uint64_t* acc_full = g_done + NB;   // [ND] each
  uint64_t* acc_empty = acc_full + ND;
  uint64_t* drain = acc_empty + ND;   // [2]: one per MMA-issuing thread
  uint64_t* never = drain + 2;
  using Item = BwdItem<KEYS>;
  Feed<Item>* feed = (Feed<Item>*)(smem + C::kFeedAt);
  uint32_t* tmem_slot = (uint32_t*)(smem + C::kFeedAt + sizeof(Feed<Item>));
  volatile int* abort = (volatile int*)(tmem_slot + 1);
  static_assert(2 * NA + 2 * NS + 3 * NB + 2 * ND + 3 <= 40, "barriers");

  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    // a stationary pair is free once S and dP of its item are done and (query side)
    // the softmax warps have read its rows' L and D
    for (int i = 0; i < NA; ++i) {
      mbar_init(&a_full[i], 1);
      mbar_init(&a_empty[i], KEYS ? 1 : 1 + kSoft);
    }
    // a stage is free once the gradient products and (key side) the readers of
    // its (L, D) are done: the latter arrive before p_full, which those wait for
    for (int i = 0; i < NS; ++i) { mbar_init(&b_full[i], 1); mbar_init(&b_empty[i], 1); }
    for (int i = 0; i < NB; ++i) {
      mbar_init(&s_full[i], 1); mbar_init(&p_full[i], kWg); mbar_init(&g_done[i], 1);
    }
    for (int i = 0; i < ND; ++i) {
      mbar_init(&acc_full[i], 1); mbar_init(&acc_empty[i], 2 * kWg);
    }
    for (int i = 0; i < 2; ++i) mbar_init(&drain[i], 1);
    mbar_init(never, 1);
    feed_init(feed, 2 + kSoft);   // the MMA and softmax warps
    abort[0] = abort[1] = 0;   // [1]: warps that recompute rows
    fence_mbar_init();
  }
  if (warp == kBProducer && lane == 0) {
    prefetch_tmap(&maps.a0);
    prefetch_tmap(&maps.a1);
    prefetch_tmap(&maps.b0);
    prefetch_tmap(&maps.b1);
  }
  if (warp == kBMma) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // up to here the kernel before this one may still run; the next one's blocks may
  // set themselves up behind this one's in the same way
  grid_dep_wait();
  grid_dep_launch();
  FeedRead<Item> rd{feed};

  if (warp == kBProducer) {
    if (lane == 0) {
      Ring<NA> ra;
      Ring<NS> rb;
      long long k = 0, e = 0;   // items with work, stages filled
      FeedWrite<Item> out{feed};
      long long t = blockIdx.x;
      bool ok = true, more = true;
      do {
        const Item it = bwd_item<KEYS>(p, t);
        if (!out.put(it, true, abort, p.status)) break;
        if (it.steps) {
          uint8_t* a = abuf + ra.s * 2 * TB;
          uint64_t* af = &a_full[ra.s];
          if (!seq_wait(&a_empty[ra.s], ra.parity ^ 1, abort, p.status)) break;
          mbar_arrive_expect_tx(af, 2 * TB + (KEYS ? 0 : kRows * 8));
          load_tokens<kRows, HD>(&maps.a0, a, it.h, it.r0, it.b, af);
          load_tokens<kRows, HD>(&maps.a1, a + TB, it.h, it.r0, it.b, af);
          if constexpr (!KEYS) {   // rows of nl, nd are padded to whole tiles
            const long long at = ((long long)it.b * p.H + it.h) * p.ld_stride + it.r0;
            bulk_load(lds + ra.s * 2 * kRows, p.nl + at, kRows * 4, af);
            bulk_load(lds + ra.s * 2 * kRows + kRows, p.nd + at, kRows * 4, af);
          }
          ra.next();
          ++k;
          const int kh = it.h / p.G;
          for (int ps = 0; ps < it.passes && ok; ++ps) {
            for (StepWalk<KEYS> w(it); w.x < it.steps; w.next(), rb.next(), ++e) {
              if (!seq_wait(&b_empty[rb.s], rb.parity ^ 1, abort, p.status)) {
                ok = false;
                break;
              }
              uint64_t* bf = &b_full[rb.s];
              uint8_t* d = ring + rb.s * 2 * SB;
              const int h = KEYS ? w.head : kh;
              mbar_arrive_expect_tx(bf, 2 * SB + (KEYS ? kStep * 8 : 0));
              load_tokens<kStep, HD>(&maps.b0, d, h, w.row, it.b, bf);
              load_tokens<kStep, HD>(&maps.b1, d + SB, h, w.row, it.b, bf);
              if constexpr (KEYS) {
                const long long at = ((long long)it.b * p.H + h) * p.ld_stride + w.row;
                bulk_load(lds + rb.s * 2 * kStep, p.nl + at, kStep * 4, bf);
                bulk_load(lds + rb.s * 2 * kStep + kStep, p.nd + at, kStep * 4, bf);
              }
            }
          }
        }
        more = ok && out.next(&t, abort, p.status);   // (not earlier: see seq_fwd_kernel)
      } while (more);
      if (!*abort) out.put(Item(), false, abort, p.status);
      if (*abort) {
        out.drain();
        for (long long j = (e > NS ? e - NS : 0); j < e; ++j)
          mbar_drain(&b_full[j % NS], (uint32_t)((j / NS) & 1), kTestLimitNs * 100);
        for (long long j = (k > NA ? k - NA : 0); j < k; ++j)
          mbar_drain(&a_full[j % NA], (uint32_t)((j / NA) & 1), kTestLimitNs * 100);
      }
    }
  } else if (warp == kBMma) {
    // S = A0 B0^T and dP = A1 B1^T of each step (the whole warp walks along, one
    // elected lane issues)
    constexpr uint32_t idesc = idesc_bf16(kRows, kStep, 0, 0);
    Ring<NA> ra;
    Ring<NS> rb;
    Ring<NB> buf;    // TMEM buffers in turn
    const uint32_t as = smem_u32(abuf), bs = smem_u32(ring);
    bool ok = true;
    while (ok) {
      const Item* item = rd.next(abort, p.status);
      if (!item) break;
      const Item it = *item;
      if (!it.steps) continue;
      if (!warp_wait(&a_full[ra.s], ra.parity, abort, p.status)) break;
      const uint32_t a_at = uniform(as + ra.s * 2 * TB);
      const uint64_t a0 = kmajor_base(a_at), a1 = kmajor_base(a_at + TB);
      for (int x = it.steps * it.passes; x > 0; --x, rb.next(), buf.next()) {
        // the buffer is free once its previous gradient products are done
        ok = warp_wait(&b_full[rb.s], rb.parity, abort, p.status) &&
             warp_wait(&g_done[buf.s], buf.parity ^ 1, abort, p.status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t b_at = uniform(bs + rb.s * 2 * SB);
        const uint64_t b0 = kmajor_base(b_at), b1 = kmajor_base(b_at + SB);
        const uint32_t d = uniform(tmem + buf.s * 2 * kStep);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk)
            umma_ss(d, a0 + kmajor_step<kRows>(kk), b0 + kmajor_step<kStep>(kk), idesc, kk > 0);
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk)
            umma_ss(d + kStep, a1 + kmajor_step<kRows>(kk), b1 + kmajor_step<kStep>(kk), idesc,
                    kk > 0);
          umma_commit(&s_full[buf.s]);
        }
        __syncwarp();
      }
      if (ok && elect_one()) umma_commit(&a_empty[ra.s]);
      __syncwarp();
      ra.next();
    }
    if (__any_sync(0xffffffffu, *abort) && elect_one()) {   // the lane that issued
      umma_commit(&drain[0]);
      mbar_drain(&drain[0], 0, kTestLimitNs * 100);
    }
  } else if (warp == kBMma2) {
    // dQ += dS K, or dV += P^T dO and dK += dS^T Q (the lanes also zero the padding
    // rows of a last streamed pair)
    constexpr uint32_t idesc = idesc_bf16(kRows, HD, 0, 1);
    Ring<NS> rb;
    Ring<NB> buf;
    Ring<ND> acc;
    const uint32_t bs = smem_u32(ring);
    bool ok = true;
    while (ok) {
      const Item* item = rd.next(abort, p.status);
      if (!item) break;
      const Item it = *item;
      if (!it.steps) continue;
      uint32_t on = 0;   // products add to the accumulators
      for (int ps = 0; ps < it.passes && ok; ++ps) {
        const bool grads = ps == it.passes - 1;
        if (grads) ok = warp_wait(&acc_empty[acc.s], acc.parity ^ 1, abort, p.status);
        const uint32_t to = uniform(tmem + TM::kAccCol + acc.s * TM::kAccCols);
        for (StepWalk<KEYS> w(it); ok && w.x < it.steps; w.next(), rb.next(), buf.next()) {
          // (the stage has landed: S of this step was computed from it)
          ok = warp_wait(&p_full[buf.s], buf.parity, abort, p.status);
          if (!ok) break;
          if (grads && w.row + kStep > it.n) {
            zero_rows<kStep, HD>(ring + rb.s * 2 * SB, it.n - w.row);
            zero_rows<kStep, HD>(ring + rb.s * 2 * SB + SB, it.n - w.row);
            fence_proxy_async();
            __syncwarp();
          }
          tc_fence_after();
          const uint32_t b_at = uniform(bs + rb.s * 2 * SB);
          const uint64_t b0 = mnmajor_base<kStep, HD>(b_at), b1 = mnmajor_base<kStep, HD>(b_at + SB);
          const uint32_t d = uniform(tmem + buf.s * 2 * kStep);
          const bool few = it.few(p, w.row);
          if (elect_one()) {
            if (grads) {
              // A from TMEM: 16 elements of K are 8 columns; split, the 32 columns of
              // each half of the step hold its high parts, then its low ones
#pragma unroll
              for (int part = 0; part < 2; ++part) {
                if (part && !few) break;
#pragma unroll
                for (int kk = 0; kk < kStep / 16; ++kk) {
                  const uint32_t a = d + (few ? 32 * (kk >> 1) + 8 * (kk & 1) + 16 * part : 8 * kk);
                  const uint32_t add = on | (part > 0) | (kk > 0);
                  if constexpr (KEYS) {
                    umma_ts(to, a, b1 + mnmajor_step(kk), idesc, add);
                    umma_ts(to + HD, a + kStep, b0 + mnmajor_step(kk), idesc, add);
                  } else {
                    umma_ts(to, a, b0 + mnmajor_step(kk), idesc, add);
                  }
                }
              }
            }
            umma_commit(&b_empty[rb.s]);
            umma_commit(&g_done[buf.s]);
          }
          __syncwarp();
          on |= grads;
        }
      }
      if (ok && elect_one()) umma_commit(&acc_full[acc.s]);
      __syncwarp();
      acc.next();
    }
    if (__any_sync(0xffffffffu, *abort) && elect_one()) {
      umma_commit(&drain[1]);
      mbar_drain(&drain[1], 0, kTestLimitNs * 100);
    }
  } else if (warp < kSoft) {
    // Warpgroup wg takes the steps of buffer wg; thread = row (query or key) = TMEM lane.
    // Waits name a round of a barrier by its parity; none can be mistaken here:
    // S of a buffer's next step is not issued before P of this one is written.
    const int wg = warp >> 2, row = threadIdx.x & (kWg - 1);
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const float2 c2 = make_float2(p.scale_log2, p.scale_log2);
    Ring<NA> ra;
    Ring<NS> rb;
    Ring<NB> rbuf;
    Ring<ND> racc;
    for (;;) {
      const Item* item = rd.next(abort, p.status);
      // the warpgroups go on together
      if (named_sync_or(1, kSoft * 32, !item || *abort)) break;
      const Item& it = *item;
      const int r = it.r0 + row;
      const bool stored = r < p.S, real = r < it.n;
      if (p.test_timeout && it.steps) mbar_wait(never, 0, abort, p.status, kTestLimitNs);
      float nl = 0.f, nd = 0.f;
      if constexpr (!KEYS) {
        if (it.steps) {
          seq_wait(&a_full[ra.s], ra.parity, abort, p.status);
          nl = lds[ra.s * 2 * kRows + row];
          nd = lds[ra.s * 2 * kRows + kRows + row];
          __syncwarp();
          if (lane == 0) mbar_arrive(&a_empty[ra.s]);
          ra.next();
        }
      }
      float dsum = 0.f;
      StepWalk<KEYS> w(it);
      const int steps = it.steps, total = steps * it.passes, r0 = it.r0;
      const int i1 = KEYS ? it.d.i1 : 0;
      for (int x = 0; x < total; ++x, w.next(), rb.next(), rbuf.next()) {
        if (!KEYS && x == steps) {
          w.start();
          // D of the row: the warpgroups' parts, in order
          xch[wg * kRows + row] = dsum;
          named_sync(1, kSoft * 32);
          nd = xch[row];
#pragma unroll
          for (int y = 1; y < NW; ++y) nd += xch[y * kRows + row];
          nd = -nd;
          if (wg == 0 && real) p.nd[((long long)it.b * p.H + it.h) * p.ld_stride + r] = nd;
        }
        if (rbuf.s != wg) continue;
        const uint32_t s_col = tmem + lane_base + rbuf.s * 2 * kStep;
        const int c0 = w.row;   // first token of the step's columns
        seq_wait(&s_full[rbuf.s], rbuf.parity, abort, p.status);
        tc_fence_after();
        // visible columns of the row: lo .. hi, and below sk
        int lo, hi, sk = 0;
        bool plain;
        if constexpr (KEYS) {
          lo = r - c0;
          hi = i1 - 1;
          if (r >= p.sinks && p.window <= 0x7fffffff - r) hi = min(hi, r + p.window - 1);
          hi -= c0;
          plain = c0 >= r0 + kRows - 1 && c0 + kStep <= i1 &&
                  (c0 + kStep - 1 - r0 < p.window || r0 + kRows <= p.sinks);
        } else {
          hi = r - c0;
          lo = hi - p.window + 1;
          sk = p.sinks - c0;
          plain = c0 + kStep - 1 <= r0 &&
                  (r0 + kRows - 1 - c0 < p.window || c0 + kStep <= p.sinks);
        }
        const bool sums = !KEYS && x < total - steps;   // the pass for D
        const float4* lv = reinterpret_cast<const float4*>(lds + rb.s * 2 * kStep);
        const float4* dv = lv + kStep / 4;
        const float sub = sums ? 0.f : nd;
        const bool few = KEYS ? it.few(p, c0) : total > steps;
        // a half of the step's columns at a time (both halves in registers at once needs
        // two warpgroups of twice the registers: 150 us against 146 for the window 512
        // case above when it was tried)
#pragma unroll
        for (int h = 0; h < kStep; h += 32) {
          float v[32], g[32];
          __syncwarp();
          tmem_ld32(s_col + h, v);
          tmem_ld32(s_col + kStep + h, g);
          tmem_wait_ld_regs(v);
          reg_fence32(g);
          // P = 2^(c S - L) and dS = P (dP - D)
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            float4 l4 = make_float4(nl, nl, nl, nl), d4 = make_float4(sub, sub, sub, sub);
            if constexpr (KEYS) {   // of four queries
              l4 = lv[(h + j) / 4];
              d4 = dv[(h + j) / 4];
            }
            const float2 a = __ffma2_rn(make_float2(v[j], v[j + 1]), c2, make_float2(l4.x, l4.y));
            const float2 b = __ffma2_rn(make_float2(v[j + 2], v[j + 3]), c2, make_float2(l4.z, l4.w));
            v[j] = ex2(a.x);
            v[j + 1] = ex2(a.y);
            v[j + 2] = ex2(b.x);
            v[j + 3] = ex2(b.y);
            const float2 ga = __fadd2_rn(make_float2(g[j], g[j + 1]), make_float2(d4.x, d4.y));
            const float2 gb = __fadd2_rn(make_float2(g[j + 2], g[j + 3]), make_float2(d4.z, d4.w));
            g[j] = ga.x;
            g[j + 1] = ga.y;
            g[j + 2] = gb.x;
            g[j + 3] = gb.y;
          }
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float2 e = __fmul2_rn(make_float2(g[j], g[j + 1]), make_float2(v[j], v[j + 1]));
            g[j] = e.x;
            g[j + 1] = e.y;
          }
          if (!plain) {
            const uint32_t see = column_mask(lo - h, hi - h, sk - h);
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!(see & (1u << j))) {
                if constexpr (KEYS) v[j] = 0.f;
                g[j] = 0.f;
              }
          }
          if (sums) {
            float a0 = 0.f, a1 = 0.f;
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              a0 += g[j];
              a1 += g[j + 1];
            }
            dsum += a0 + a1;
          } else {
            // over columns that this half's loads have emptied
            if (few) {
              const uint32_t to = s_col + h;
              if constexpr (KEYS) split_to_columns(to, to + 16, v);
              split_to_columns(to + (KEYS ? kStep : 0), to + (KEYS ? kStep : 0) + 16, g);
            } else {
              const uint32_t to = s_col + h / 2;
              uint32_t pk[16];
              if constexpr (KEYS) {
                round_pairs(v, pk);
                __syncwarp();
                tmem_st16u(to, pk);
              }
              round_pairs(g, pk);
              __syncwarp();
              tmem_st16u(to + (KEYS ? kStep : 0), pk);
            }
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&p_full[rbuf.s]);
      }
      // epilogue: two warpgroups store half of the accumulator columns each (dV, dK)
      bool bad = false;
      if (wg < 2) {
        constexpr int NC = TM::kAccCols / 2;
        if (it.steps) {
          seq_wait(&acc_full[racc.s], racc.parity, abort, p.status);
          tc_fence_after();
        }
        const uint32_t acc = tmem + lane_base + TM::kAccCol + racc.s * TM::kAccCols + wg * NC;
        void* dst;
        bool f32 = false;
        float mul = p.scale;
        if constexpr (KEYS) {
          f32 = it.d.partial;
          if (f32) dst = (wg == 0 ? it.d.pv : it.d.pk) + row * it.d.row_stride;
          else
            dst = (__nv_bfloat16*)(wg == 0 ? p.dv : p.dk) +
                  ((long long)it.b * p.S + r) * p.ks + (long long)it.h * p.hd;
          if (wg == 0) mul = 1.f;
        } else {
          dst = (__nv_bfloat16*)p.dq + ((long long)it.b * p.S + r) * p.qs +
                (long long)it.h * p.hd + wg * NC;
        }
        if (!stored || *abort) dst = nullptr;
        // an item without steps has no products: its rows are zeros whatever TMEM holds
        bad = store_grad<NC>(acc, mul, real && it.steps, dst, f32, p.hd - (KEYS ? 0 : wg * NC),
                             it.steps ? &acc_empty[racc.s] : nullptr) && real && it.steps;
        // (a row whose L or D is NaN has a NaN of its own: it is as it should be)
        if (!KEYS && !(nl == nl && nd == nd)) bad = false;
      }
      if (it.steps) racc.next();
      if (named_sync_or(1, kSoft * 32, bad && !*abort)) {
        int* flags = (int*)xch;
        if (wg == 0) flags[row] = 0;
        named_sync(1, kSoft * 32);
        if (bad) flags[row] = 1;
        if (lane == 0) atomicAdd((int*)abort + 1, 1);
        named_sync(1, kSoft * 32);
        for (int y = warp; y < kRows; y += kSoft)
          if (flags[y]) {
            if constexpr (KEYS) fix_dkv_row<__nv_bfloat16>(p, it.d, it.r0 + y);
            else fix_dq_row<__nv_bfloat16>(p, it.b, it.h, it.r0 + y);
          }
        if (lane == 0) atomicAdd((int*)abort + 1, -1);
        named_sync(1, kSoft * 32);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kBMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int HD, bool KEYS>
cudaError_t bwd_launch(const SeqParams& p, const BwdMaps& maps, cudaStream_t st) {
  using C = BwdCfg<HD, KEYS>;
  static_assert(C::kSmem <= kSmemLimit, "shared memory");
  const cudaError_t e = allow_smem<seq_bwd_kernel<HD, KEYS>>(C::kSmem);
  if (e != cudaSuccess) return e;
  const long long items =
      KEYS ? p.plan.items : (long long)p.B * p.H * ((p.S + kRows - 1) / kRows);
  if (items > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch_dependent(seq_bwd_kernel<HD, KEYS>, dim3((unsigned)items),
                          BwdTmem<HD, KEYS>::kThreads, C::kSmem, st, p, maps);
}

}  // namespace

cudaError_t seq_fast_backward(const SeqParams& p, cudaStream_t st) {
  BwdMaps q, k;
  const long long os = (long long)p.H * p.hd;
  if (!encode_tokens(&q.a0, p.q, p, p.H, p.qs, kRows) ||
      !encode_tokens(&q.a1, p.dout, p, p.H, os, kRows) ||
      !encode_tokens(&q.b0, p.k, p, p.K, p.ks, kStep) ||
      !encode_tokens(&q.b1, p.v, p, p.K, p.ks, kStep) ||
      !encode_tokens(&k.a0, p.k, p, p.K, p.ks, kRows) ||
      !encode_tokens(&k.a1, p.v, p, p.K, p.ks, kRows) ||
      !encode_tokens(&k.b0, p.q, p, p.H, p.qs, kStep) ||
      !encode_tokens(&k.b1, p.dout, p, p.H, os, kStep))
    return cudaErrorInvalidValue;
  const cudaError_t e =
      p.hd <= 64 ? bwd_launch<64, false>(p, q, st) : bwd_launch<128, false>(p, q, st);
  if (e != cudaSuccess) return e;
  return p.hd <= 64 ? bwd_launch<64, true>(p, k, st) : bwd_launch<128, true>(p, k, st);
}

}  // namespace swin
