// seq_sm100.cu -- tcgen05 / TMA forward of sequence attention (causal sliding
// window with sink tokens; bf16, head_dim 64 or 128).
//
// One pass over a query tile's visible key tiles with a running maximum and sum.
// An item is one head's pair of 128-query tiles (or a single tile where pairs
// would leave SMs idle): both tiles read the same key and value tiles, so a
// pair halves the shared-memory traffic of TMA, and while one tile's softmax
// runs on the exp unit the other's products run on the tensor pipe. Per key
// tile and query tile
//   S = Q K^T (M = N = 128, fp32 in TMEM), P = 2^(c S - m) in registers,
//   P as bf16 over S's columns, O += P V with A = P from TMEM.
// The running maximum m of a row moves only when a tile raises it by more than
// 2^8, so O is rescaled in TMEM (by the softmax threads) a few times per row
// at most. P is rounded to bf16 (off by 2^-8 of each term at most; terms of
// either sign average out); the row sum takes the unrounded fp32 values.
//
// TMEM: query tile w owns columns 256 w ..: S / P in 128, O in the next hd.
// Warps: 0-3 and 4-7 one softmax warpgroup per query tile (thread = row), 8
// the TMA producer, 9 issues S and owns TMEM, 10 issues O += P V. Keys and
// values have a ring slot each, so S starts before V has landed. Persistent
// grid; items with the longest rows come first.
//
// Bound: per 128 x 128 tile of a head the tensor pipe needs 8 hd cycles (S and
// O at 8192 FLOP per cycle and SM) and the exp unit 1024 (16 per cycle), so
// head_dim 128 is bound by both alike, head_dim 64 by the exp unit.
#include "fast_common.cuh"
#include "seq_common.cuh"

namespace swin {
namespace {

using namespace ptx;

constexpr int kSeqThreads = 384;
constexpr int kSeqProducer = 8, kSeqMma = 9, kSeqMma2 = 10;
constexpr uint32_t kSeqOCol = 128;
constexpr float kSeqMove = 8.f;   // the running maximum moves by more than this (log2)

struct SeqMaps {
  CUtensorMap q, k, v;
};

template <int HD>
struct SeqFwdCfg {
  static constexpr uint32_t kTile = kRows * HD * 2;
  static constexpr int kQBufs = HD > 64 ? 1 : 2;
  static constexpr int kSlots = HD > 64 ? 4 : 8;   // ring of key / value tiles
  static constexpr uint32_t kBars = (kQBufs * 2 + kSlots) * kTile;
  static constexpr uint32_t kTotal = kBars + 8 * 48 + 16;
  static constexpr uint32_t kSmem = kTotal + 1024;
};

// What an item is, for every role alike.
struct SeqItem {
  int b, h, i0, n;       // first query, tokens of the sequence
  KeyTiles u;            // key tiles of the whole item
  int steps;             // of them (0: the item is all padding)
};
__device__ __forceinline__ SeqItem seq_item(const SeqParams& p, long long t, int nq) {
  SeqItem it;
  const int bh = p.B * p.H;
  const int per = (p.S + kRows * nq - 1) / (kRows * nq);
  const int r = (int)(t / bh), z = (int)(t - (long long)r * bh);
  it.b = z / p.H;
  it.h = z - it.b * p.H;
  it.i0 = (per - 1 - r) * kRows * nq;
  it.n = seq_len(p, it.b);
  it.steps = 0;
  if (it.i0 < it.n) {
    it.u = seq_key_tiles(p, it.i0, min(it.n, it.i0 + kRows * nq), kRows);
    it.steps = it.u.count();
  }
  return it;
}
// Key tiles of query tile w of the item; none if it is all padding.
__device__ __forceinline__ bool seq_sub(const SeqParams& p, const SeqItem& it, int w,
                                        KeyTiles& kt) {
  const int i0 = it.i0 + w * kRows;
  if (i0 >= it.n) return false;
  kt = seq_key_tiles(p, i0, min(it.n, i0 + kRows), kRows);
  return true;
}
__device__ __forceinline__ bool seq_needs(const KeyTiles& kt, int tile) {
  return tile <= kt.hi && (tile >= kt.lo || tile < kt.s);
}

// One [128 tokens][HD] tile of head h (channel halves of 64 as regions).
template <int HD>
__device__ __forceinline__ void load_rows(const CUtensorMap* m, uint8_t* dst, int h, int row,
                                          int b, uint64_t* bar) {
  using T = TileGeom<HD>;
#pragma unroll
  for (int hf = 0; hf < T::kHalves; ++hf)
    tma_load_4d(dst + hf * T::kHalfBytes, m, bar, hf * T::kBoxEl, h, row, b);
}

// Zeroes rows from .. 127 of a [128][HD] tile (a warp): what padding tokens
// hold must not meet a zero weight in a product (0 x NaN).
template <int HD>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int from) {
  using T = TileGeom<HD>;
  const int lane = threadIdx.x & 31;
  constexpr int C = T::kRowBytes / 16;
  for (int hf = 0; hf < T::kHalves; ++hf)
    for (int x = from * C + lane; x < kRows * C; x += 32)
      st_shared_v4(smem_u32(tile + hf * T::kHalfBytes + x * 16), 0u, 0u, 0u, 0u);
  fence_proxy_async();
  __syncwarp();
}

// A wait of a whole warp: every lane sees the phase, and all take the same way
// when the wait is given up.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                          int* status) {
  const bool ok = mbar_wait(bar, parity, abort, status, kWaitLimitNs);
  return __all_sync(0xffffffffu, ok);
}

template <int HD>
__global__ void __launch_bounds__(kSeqThreads, 1)
    seq_fwd_kernel(const __grid_constant__ SeqParams p, const __grid_constant__ SeqMaps maps,
                   const int nq, const long long n_items) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  using C = SeqFwdCfg<HD>;
  constexpr int NQ = C::kQBufs, NS = C::kSlots;
  constexpr uint32_t TB = C::kTile;
  uint8_t* qbuf = smem;
  uint8_t* kv = smem + NQ * 2 * TB;
  uint64_t* bars = (uint64_t*)(smem + C::kBars);
  uint64_t* q_full = bars;
  uint64_t* q_empty = q_full + NQ;
  uint64_t* kv_full = q_empty + NQ;
  uint64_t* kv_empty = kv_full + NS;
  uint64_t* s_full = kv_empty + NS;   // [2] per query tile
  uint64_t* p_full = s_full + 2;
  uint64_t* o_done = p_full + 2;
  uint64_t* t_empty = o_done + 2;
  uint64_t* drain = t_empty + 2;      // [2]: one per MMA-issuing thread
  uint64_t* never = drain + 2;
  uint32_t* tmem_slot = (uint32_t*)(smem + C::kBars + 8 * 48);
  volatile int* abort = (volatile int*)(tmem_slot + 1);
  static_assert(2 * NQ + 2 * NS + 8 + 3 <= 48, "barriers");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NQ; ++i) { mbar_init(&q_full[i], 1); mbar_init(&q_empty[i], 1); }
    for (int i = 0; i < NS; ++i) { mbar_init(&kv_full[i], 1); mbar_init(&kv_empty[i], 1); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1); mbar_init(&p_full[i], kWg);
      mbar_init(&o_done[i], 1); mbar_init(&t_empty[i], kWg);
      mbar_init(&drain[i], 1);
    }
    mbar_init(never, 1);
    *abort = 0;
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

  if (warp == kSeqProducer) {
    if (lane == 0) {
      long long k = 0, e = 0;   // items with work, ring slots filled
      bool ok = true;
      for (long long t = blockIdx.x; t < n_items && ok; t += gridDim.x) {
        const SeqItem it = seq_item(p, t, nq);
        if (!it.steps) continue;
        const int qs = (int)(k % NQ), kh = it.h / p.G;
        if (!mbar_wait(&q_empty[qs], (uint32_t)(((k / NQ) & 1) ^ 1), abort, p.status,
                       kWaitLimitNs))
          break;
        mbar_arrive_expect_tx(&q_full[qs], nq * TB);
        for (int w = 0; w < nq; ++w)
          load_rows<HD>(&maps.q, qbuf + (qs * 2 + w) * TB, it.h, it.i0 + w * kRows, it.b,
                        &q_full[qs]);
        ++k;
        for (int x = 0; x < it.steps && ok; ++x)
          for (int kvi = 0; kvi < 2; ++kvi, ++e) {
            const int s = (int)(e % NS);
            if (!mbar_wait(&kv_empty[s], (uint32_t)(((e / NS) & 1) ^ 1), abort, p.status,
                           kWaitLimitNs)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&kv_full[s], TB);
            load_rows<HD>(kvi ? &maps.v : &maps.k, kv + s * TB, kh, it.u.tile(x) * kRows, it.b,
                          &kv_full[s]);
          }
      }
      if (*abort) {  // let copies already in flight land before the CTA leaves
        for (long long j = (e > NS ? e - NS : 0); j < e; ++j)
          mbar_drain(&kv_full[j % NS], (uint32_t)((j / NS) & 1), kTestLimitNs * 100);
        for (long long j = (k > NQ ? k - NQ : 0); j < k; ++j)
          mbar_drain(&q_full[j % NQ], (uint32_t)((j / NQ) & 1), kTestLimitNs * 100);
      }
    }
  } else if (warp == kSeqMma) {
    if (lane == 0) {   // S = Q_w K^T of both query tiles, key tile by key tile
      constexpr uint32_t idesc_s = idesc_bf16(kRows, kRows, 0, 0);
      long long k = 0, e = 0;
      uint32_t ns[2] = {0, 0};   // products of a query tile so far
      bool ok = true;
      for (long long t = blockIdx.x; t < n_items && ok; t += gridDim.x) {
        const SeqItem it = seq_item(p, t, nq);
        if (!it.steps) continue;
        KeyTiles kt[2];
        bool has[2];
        for (int w = 0; w < 2; ++w) has[w] = w < nq && seq_sub(p, it, w, kt[w]);
        const int qs = (int)(k % NQ);
        if (!mbar_wait(&q_full[qs], (uint32_t)((k / NQ) & 1), abort, p.status, kWaitLimitNs))
          break;
        for (int x = 0; x < it.steps && ok; ++x, e += 2) {
          const int s = (int)(e % NS), tile = it.u.tile(x);
          if (!mbar_wait(&kv_full[s], (uint32_t)((e / NS) & 1), abort, p.status, kWaitLimitNs)) {
            ok = false;
            break;
          }
          const uint32_t k_s = smem_u32(kv + s * TB);
          for (int w = 0; w < 2; ++w) {
            if (!has[w] || !seq_needs(kt[w], tile)) continue;
            // S's columns are free once the previous O += P V of this tile is done
            if (!mbar_wait(&o_done[w], (ns[w] & 1) ^ 1, abort, p.status, kWaitLimitNs)) {
              ok = false;
              break;
            }
            ++ns[w];
            tc_fence_after();
            const uint32_t q_s = smem_u32(qbuf + (qs * 2 + w) * TB);
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk)
              umma_ss(tmem + w * 256, desc_kmajor_tile<HD>(q_s, kk), desc_kmajor_tile<HD>(k_s, kk),
                      idesc_s, kk);
            umma_commit(&s_full[w]);
          }
          if (ok) umma_commit(&kv_empty[s]);
        }
        if (ok) umma_commit(&q_empty[qs]);
        ++k;
      }
      if (*abort) {
        umma_commit(&drain[0]);
        mbar_drain(&drain[0], 0, kTestLimitNs * 100);
      }
    }
  } else if (warp == kSeqMma2) {
    // O += P V of both query tiles, as soon as each P is written (all lanes walk
    // along: they zero the padding rows of a last value tile)
    constexpr uint32_t idesc_o = idesc_bf16(kRows, HD, 0, 1);
    long long e = 0;
    uint32_t ns[2] = {0, 0}, done[2] = {0, 0};   // products, items of a query tile so far
    bool ok = true;
    for (long long t = blockIdx.x; t < n_items && ok; t += gridDim.x) {
      const SeqItem it = seq_item(p, t, nq);
      if (!it.steps) continue;
      KeyTiles kt[2];
      bool has[2], first[2] = {true, true};
      for (int w = 0; w < 2; ++w) has[w] = w < nq && seq_sub(p, it, w, kt[w]);
      for (int x = 0; x < it.steps && ok; ++x, e += 2) {
        const long long ev = e + 1;
        const int s = (int)(ev % NS), tile = it.u.tile(x);
        if (!warp_wait(&kv_full[s], (uint32_t)((ev / NS) & 1), abort, p.status)) {
          ok = false;
          break;
        }
        if ((tile + 1) * kRows > it.n) zero_rows<HD>(kv + s * TB, it.n - tile * kRows);
        const uint32_t v_s = smem_u32(kv + s * TB);
        for (int w = 0; w < 2; ++w) {
          if (!has[w] || !seq_needs(kt[w], tile)) continue;
          // a new item overwrites O: the previous item's epilogue has read it
          if ((first[w] && !warp_wait(&t_empty[w], (done[w] & 1) ^ 1, abort, p.status)) ||
              !warp_wait(&p_full[w], ns[w] & 1, abort, p.status)) {
            ok = false;
            break;
          }
          ++ns[w];
          tc_fence_after();
          if (lane == 0) {
            const uint32_t base = tmem + w * 256;
#pragma unroll
            for (int kk = 0; kk < kRows / 16; ++kk)
              umma_ts(base + kSeqOCol, base + kk * 8, desc_mnmajor_tile<HD>(v_s, kk), idesc_o,
                      (!first[w] || kk > 0) ? 1u : 0u);
            umma_commit(&o_done[w]);
          }
          __syncwarp();
          first[w] = false;
        }
        if (ok && lane == 0) umma_commit(&kv_empty[s]);
        __syncwarp();
      }
      for (int w = 0; w < 2; ++w) done[w] += has[w];
    }
    if (*abort && lane == 0) {
      umma_commit(&drain[1]);
      mbar_drain(&drain[1], 0, kTestLimitNs * 100);
    }
  } else if (warp < 8) {
    // Softmax and epilogue of query tile w (thread = row = TMEM lane).
    const int w = warp >> 2, row = threadIdx.x & (kWg - 1);
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lane_base + w * 256;
    const uint32_t o_col = s_col + kSeqOCol;
    uint32_t ns = 0;
    for (long long t = blockIdx.x; t < n_items && w < nq; t += gridDim.x) {
      if (*abort) break;
      const SeqItem it = seq_item(p, t, nq);
      const int i0 = it.i0 + w * kRows, i = i0 + row;
      const bool stored = i < p.S, real = i < it.n;
      const long long orow = ((long long)it.b * p.S + i) * p.H + it.h;
      __nv_bfloat16* dst = (__nv_bfloat16*)p.out + orow * HD;
      KeyTiles kt;
      if (!seq_sub(p, it, w, kt)) {   // padding: zeros
        float z[64];
#pragma unroll
        for (int c = 0; c < 64; ++c) z[c] = 0.f;
#pragma unroll
        for (int c = 0; c < HD; c += 64)
          store_rows_bf16<64>(z, 0.f, stored ? (const void*)(dst + c) : nullptr);
        if (stored && p.lse) p.lse[orow] = 0.f;
        continue;
      }
      if (p.test_timeout) mbar_wait(never, 0, abort, p.status, kTestLimitNs);
      float m = -INFINITY, l = 0.f;
      const int cnt = kt.count();
      for (int x = 0; x < cnt; ++x, ++ns) {
        const int k0 = kt.tile(x) * kRows;
        mbar_wait(&s_full[w], ns & 1, abort, p.status, kWaitLimitNs);
        tc_fence_after();
        float v[128];
        tmem_load_cols<128>(s_col, v);
        tmem_wait_ld();
        const bool plain = k0 + kRows - 1 <= i0 &&
                           (i0 + kRows - 1 - k0 < p.window || k0 + kRows <= p.sinks);
        if (!plain) {
          const int hi = i - k0, lo = hi - p.window + 1, sk = p.sinks - k0;
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (c > hi || (c < lo && c >= sk)) v[c] = -INFINITY;
        }
        float m0 = -INFINITY, m1 = m0, m2 = m0, m3 = m0;
#pragma unroll
        for (int c = 0; c < 128; c += 4) {
          m0 = fmaxf(m0, v[c]);
          m1 = fmaxf(m1, v[c + 1]);
          m2 = fmaxf(m2, v[c + 2]);
          m3 = fmaxf(m3, v[c + 3]);
        }
        const float mt = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3)) * p.scale_log2;
        const bool move = mt > m + kSeqMove;
        const float f = move ? ex2(m - mt) : 1.f;   // 0 while m = -inf
        if (move) {
          l *= f;
          m = mt;
        }
        if (x > 0 && __any_sync(0xffffffffu, move)) {
          // O is free of the previous product before it is scaled
          mbar_wait(&o_done[w], (ns & 1) ^ 1, abort, p.status, kWaitLimitNs);
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
        const float2 nm = make_float2(-mu, -mu), sc = make_float2(p.scale_log2, p.scale_log2);
        float2 la = make_float2(0.f, 0.f), lb = la;
#pragma unroll
        for (int c0 = 0; c0 < 128; c0 += 32) {
          uint32_t pk[16];
#pragma unroll
          for (int c = c0; c < c0 + 32; c += 4) {
            const float2 a = __ffma2_rn(make_float2(v[c], v[c + 1]), sc, nm);
            const float2 b = __ffma2_rn(make_float2(v[c + 2], v[c + 3]), sc, nm);
            const float2 ea = make_float2(ex2(a.x), ex2(a.y)), eb = make_float2(ex2(b.x), ex2(b.y));
            la = __fadd2_rn(la, ea);
            lb = __fadd2_rn(lb, eb);
            pk[(c - c0) / 2] = pack_bf16(ea.x, ea.y);
            pk[(c - c0) / 2 + 1] = pack_bf16(eb.x, eb.y);
          }
          __syncwarp();
          tmem_st16u(s_col + c0 / 2, pk);
        }
        l += (la.x + la.y) + (lb.x + lb.y);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&p_full[w]);
      }
      mbar_wait(&o_done[w], (ns & 1) ^ 1, abort, p.status, kWaitLimitNs);   // the last product
      tc_fence_after();
      const float inv = 1.f / l;
      bool bad = false;
#pragma unroll
      for (int c = 0; c < HD; c += 64) {
        float o[64];
        tmem_load_cols<64>(o_col + c, o);
        tmem_wait_ld();
        if (c + 64 >= HD) {
          tc_fence_before();
          mbar_arrive(&t_empty[w]);
        }
        float big = 0.f;   // fmaxf drops NaN, so sum the (finite) magnitudes' excess instead
#pragma unroll
        for (int j = 0; j < 64; ++j) {
          big += o[j] * 0.f;              // NaN once any entry is not finite
          o[j] = real ? o[j] * inv : 0.f;
        }
        bad |= big != 0.f;
        store_rows_bf16<64>(o, 1.f, stored && !*abort ? (const void*)(dst + c) : nullptr);
      }
      bad |= !(fabsf(inv) <= 3.4e38f);
      if (stored && !*abort && p.lse) p.lse[orow] = real ? (m + __log2f(l)) / kSeqLog2e : 0.f;
      uint32_t fix = __ballot_sync(0xffffffffu, bad && real && !*abort);
      while (fix) {
        const int r = __ffs(fix) - 1;
        fix &= fix - 1;
        __syncwarp();
        fix_out_row<__nv_bfloat16>(p, it.b, it.h, i0 + (warp & 3) * 32 + r);
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

// The map [hd, heads, S, B] of one operand, box [64, 1, rows, 1].
bool encode_tokens(CUtensorMap* m, const void* base, const SeqParams& p, int heads,
                   long long stride, int rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)p.hd, (cuuint64_t)heads, (cuuint64_t)p.S,
                              (cuuint64_t)p.B};
  const cuuint64_t strides[3] = {(cuuint64_t)p.hd * 2, (cuuint64_t)stride * 2,
                                 (cuuint64_t)stride * 2 * p.S};
  const cuuint32_t box[4] = {64, 1, (cuuint32_t)rows, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int HD>
cudaError_t fwd_launch(const SeqParams& p, const SeqMaps& maps, cudaStream_t st) {
  auto kernel = seq_fwd_kernel<HD>;
  const int smem = SeqFwdCfg<HD>::kSmem;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  // pairs of query tiles, unless they leave more than half of the SMs idle
  const int sms = num_sms();
  const long long tiles = (p.S + kRows - 1) / kRows, bh = (long long)p.B * p.H;
  const int nq = tiles > 1 && (tiles + 1) / 2 * bh > sms / 2 ? 2 : 1;
  const long long items = (tiles + nq - 1) / nq * bh;
  kernel<<<(unsigned)(items < sms ? items : sms), kSeqThreads, smem, st>>>(p, maps, nq, items);
  note_launch();
  return cudaGetLastError();
}

}  // namespace

bool seq_fast_supported(int dtype, int hd) {
  return dtype == SWIN_DTYPE_BF16 && (hd == 64 || hd == 128);
}

cudaError_t seq_fast_forward(const SeqParams& p, cudaStream_t st) {
  SeqMaps maps;
  if (!encode_tokens(&maps.q, p.q, p, p.H, p.qs, kRows) ||
      !encode_tokens(&maps.k, p.k, p, p.K, p.ks, kRows) ||
      !encode_tokens(&maps.v, p.v, p, p.K, p.ks, kRows))
    return cudaErrorInvalidValue;
  return p.hd == 64 ? fwd_launch<64>(p, maps, st) : fwd_launch<128>(p, maps, st);
}

}  // namespace swin
