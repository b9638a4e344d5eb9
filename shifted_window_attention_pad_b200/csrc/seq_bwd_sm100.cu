// seq_bwd_sm100.cu -- tcgen05 / TMA backward of sequence attention (bf16,
// head_dim 64 or 128).
//
// Two kernels, because dQ sums over keys and dK, dV over queries, and a sum
// that crosses blocks would need atomics, whose order changes results:
//  * query side, item = (head, 128 queries): S = Q K^T, dP = dO V^T over the
//    visible keys in steps of 64, P = 2^(c S - L), dS = P (dP - D), dQ += dS K;
//  * key side, item = (128 keys, query heads, queries; DkvPlan): S^T = K Q^T,
//    dP^T = V dO^T over the queries in steps of 64 (thread = key), dV += P^T dO,
//    dK += dS^T Q.
// One kernel template runs both: a stationary pair of 128-row tiles (Q, dO or
// K, V), a streamed pair of 64-row tiles, two TMEM buffers of S | dP (64 + 64
// columns) and the accumulators. P and dS are rounded to bf16 over their own
// columns and are the A operand of the gradient products from TMEM (off by
// 2^-8 of each term at most); sums are fp32 in TMEM.
//
// D_i = dO_i.o_i uses the stored, rounded o. Where a row sees few keys its dS is
// a small difference of dP and D and that rounding would show, so items of at
// most kTwoPass key steps take D = sum_j P_ij dP_ij from a pass of their own
// first (and leave it for the key side): an error of 0.11 of the gradients' RMS
// in the first rows of a sequence becomes that of other rows. Longer rows would
// pay two more products per step for an error already below the outputs' own
// rounding.
//
// Warps: 0-15 four softmax warpgroups, two per TMEM buffer, each 32 of the
// step's 64 columns; 16 the TMA producer; 17 issues S and dP and owns TMEM; 18
// issues the gradient products. Bound: the tensor pipe (per 128 x 64 step of
// head_dim 128: S and dP 384 cycles each, limited by shared-memory reads of
// both operands, 256 for each gradient product).
#include "fast_common.cuh"
#include "seq_common.cuh"

namespace swin {
namespace {

using namespace ptx;

constexpr int kStep = 64;         // keys (queries) of a step
constexpr int kSoft = 16;         // softmax warps
constexpr int kBProducer = 16, kBMma = 17, kBMma2 = 18;
constexpr int kBThreads = 19 * 32;
constexpr int kTwoPass = 6;
constexpr uint32_t kAccCol = 256;

struct BwdMaps {
  CUtensorMap a0, a1, b0, b1;   // stationary pair, streamed pair
};

template <int HD>
struct BwdCfg {
  static constexpr uint32_t kTile = kRows * HD * 2;    // stationary tile
  static constexpr uint32_t kSub = kStep * HD * 2;     // streamed tile
  static constexpr int kABufs = HD > 64 ? 1 : 2;
  static constexpr int kStages = HD > 64 ? 4 : 6;
  static constexpr uint32_t kRing = kABufs * 2 * kTile;
  static constexpr uint32_t kLd = kRing + kStages * 2 * kSub;
  static constexpr uint32_t kXch = kLd + kStages * kStep * 8;
  static constexpr uint32_t kBars = kXch + 4 * kRows * 4;
  static constexpr uint32_t kTotal = kBars + 8 * 40 + 16;
  static constexpr uint32_t kSmem = kTotal + 1024;
};

// Operands of 64-row tiles (channel halves of 64 as [64][64] regions).
template <int HD>
__device__ __forceinline__ uint64_t sub_kmajor(uint32_t base, int k16) {
  return smem_desc(base + (k16 >> 2) * (kStep * 128) + (k16 & 3) * 32, 16, 1024, kSwizzle128);
}
template <int HD>
__device__ __forceinline__ uint64_t sub_mnmajor(uint32_t base, int k16) {
  return smem_desc(base + k16 * 16 * 128, HD > 64 ? kStep * 128 : 1024, 1024, kSwizzle128);
}

template <int ROWS, int HD>
__device__ __forceinline__ void load_tokens(const CUtensorMap* m, uint8_t* dst, int h, int row,
                                            int b, uint64_t* bar) {
#pragma unroll
  for (int hf = 0; hf < HD / 64; ++hf)
    tma_load_4d(dst + hf * ROWS * 128, m, bar, hf * 64, h, row, b);
}

// Zeroes rows from .. 63 of a streamed tile (a warp; see seq_fwd_kernel).
template <int HD>
__device__ __forceinline__ void zero_sub_rows(uint8_t* tile, int from) {
  const int lane = threadIdx.x & 31;
  for (int hf = 0; hf < HD / 64; ++hf)
    for (int x = from * 8 + lane; x < kStep * 8; x += 32)
      st_shared_v4(smem_u32(tile + hf * kStep * 128 + x * 16), 0u, 0u, 0u, 0u);
}

__device__ __forceinline__ bool bwd_warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                              int* status) {
  const bool ok = mbar_wait(bar, parity, abort, status, kWaitLimitNs);
  return __all_sync(0xffffffffu, ok);
}

// An item of either side, for every role alike: `steps` streamed tiles a pass.
template <bool KEYS>
struct BwdItem {
  DkvItem d;             // key side
  KeyTiles kt;           // query side: key steps
  int b, h, r0, n;       // query side: head and first query; key side: r0 = first key
  int steps, passes, per;   // per: steps of one query head (key side)
  __device__ __forceinline__ int row(int x) const {   // first streamed token of step x
    if constexpr (KEYS) return d.i0 + (x % per) * kStep;
    else return kt.tile(x) * kStep;
  }
  __device__ __forceinline__ int head(int x) const {   // query head of step x
    if constexpr (KEYS) return d.h0 + x / per;
    else return h;
  }
};
template <bool KEYS>
__device__ __forceinline__ BwdItem<KEYS> bwd_item(const SeqParams& p, long long t) {
  BwdItem<KEYS> it;
  it.steps = 0;
  it.passes = 1;
  it.per = 1;
  if constexpr (KEYS) {
    it.d = dkv_item(p, t);
    it.b = it.d.b;
    it.h = it.d.kh;
    it.n = it.d.n;
    it.r0 = it.d.tile * kRows;
    if (it.d.i0 < it.d.i1) {
      it.per = (it.d.i1 - it.d.i0 + kStep - 1) / kStep;
      it.steps = it.per * (it.d.h1 - it.d.h0);
    }
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
      it.passes = it.steps <= kTwoPass ? 2 : 1;
    }
  }
  return it;
}

// NC fp32 columns of a row times `mul`, zero where !keep, to bf16 rows or fp32
// partial rows (dst: this lane's row or nullptr); says whether any is not finite.
template <int NC>
__device__ __forceinline__ bool store_grad(uint32_t col, float mul, bool keep, void* dst,
                                           bool f32) {
  bool bad = false;
#pragma unroll
  for (int c = 0; c < NC; c += 16) {
    float o[16];
    __syncwarp();
    tmem_ld16(col + c, o);
    tmem_wait_ld_regs16(o);
    float big = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      big += o[j] * 0.f;                    // NaN once any entry is not finite
      o[j] = keep ? o[j] * mul : 0.f;
    }
    bad |= big != 0.f;
    if (f32) {
      uint4 a[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        a[j] = make_uint4(__float_as_uint(o[4 * j]), __float_as_uint(o[4 * j + 1]),
                          __float_as_uint(o[4 * j + 2]), __float_as_uint(o[4 * j + 3]));
      store_rows_coalesced<4>(a, dst ? (const void*)((float*)dst + c) : nullptr);
    } else {
      store_rows_bf16<16>(o, 1.f, dst ? (const void*)((__nv_bfloat16*)dst + c) : nullptr);
    }
  }
  return bad;
}

template <int HD, bool KEYS>
__global__ void __launch_bounds__(kBThreads, 1)
    seq_bwd_kernel(const __grid_constant__ SeqParams p, const __grid_constant__ BwdMaps maps,
                   const long long n_items) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  using C = BwdCfg<HD>;
  constexpr int NA = C::kABufs, NS = C::kStages;
  constexpr uint32_t TB = C::kTile, SB = C::kSub;
  uint8_t* abuf = smem;
  uint8_t* ring = smem + C::kRing;
  float2* lds = (float2*)(smem + C::kLd);
  float* xch = (float*)(smem + C::kXch);
  uint64_t* bars = (uint64_t*)(smem + C::kBars);
  uint64_t* a_full = bars;
  uint64_t* a_empty = a_full + NA;
  uint64_t* b_full = a_empty + NA;
  uint64_t* b_empty = b_full + NS;
  uint64_t* s_full = b_empty + NS;    // [2] per TMEM buffer
  uint64_t* p_full = s_full + 2;
  uint64_t* g_done = p_full + 2;
  uint64_t* acc_full = g_done + 2;
  uint64_t* acc_empty = acc_full + 1;
  uint64_t* drain = acc_empty + 1;    // [2]: one per MMA-issuing thread
  uint64_t* never = drain + 2;
  uint32_t* tmem_slot = (uint32_t*)(smem + C::kBars + 8 * 40);
  volatile int* abort = (volatile int*)(tmem_slot + 1);
  static_assert(2 * NA + 2 * NS + 6 + 2 + 3 <= 40, "barriers");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NA; ++i) { mbar_init(&a_full[i], 1); mbar_init(&a_empty[i], 1); }
    // a stage is free once the gradient products and (key side) the readers of
    // its (L, D) are done: the latter arrive before p_full, which those wait for
    for (int i = 0; i < NS; ++i) { mbar_init(&b_full[i], 1); mbar_init(&b_empty[i], 1); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1); mbar_init(&p_full[i], 2 * kWg);
      mbar_init(&g_done[i], 1); mbar_init(&drain[i], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, 4 * kWg);
    mbar_init(never, 1);
    *abort = 0;
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

  if (warp == kBProducer) {
    if (lane == 0) {
      long long k = 0, e = 0;   // items with work, stages filled
      bool ok = true;
      for (long long t = blockIdx.x; t < n_items && ok; t += gridDim.x) {
        const BwdItem<KEYS> it = bwd_item<KEYS>(p, t);
        if (!it.steps) continue;
        const int as = (int)(k % NA);
        if (!mbar_wait(&a_empty[as], (uint32_t)(((k / NA) & 1) ^ 1), abort, p.status,
                       kWaitLimitNs))
          break;
        mbar_arrive_expect_tx(&a_full[as], 2 * TB);
        load_tokens<kRows, HD>(&maps.a0, abuf + as * 2 * TB, it.h, it.r0, it.b, &a_full[as]);
        load_tokens<kRows, HD>(&maps.a1, abuf + as * 2 * TB + TB, it.h, it.r0, it.b, &a_full[as]);
        ++k;
        for (int x = 0; x < it.steps * it.passes; ++x, ++e) {
          const int s = (int)(e % NS), u = x % it.steps, row = it.row(u);
          const int h = KEYS ? it.head(u) : it.h / p.G;
          if (!mbar_wait(&b_empty[s], (uint32_t)(((e / NS) & 1) ^ 1), abort, p.status,
                         kWaitLimitNs)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&b_full[s], 2 * SB + (KEYS ? kStep * 8 : 0));
          load_tokens<kStep, HD>(&maps.b0, ring + s * 2 * SB, h, row, it.b, &b_full[s]);
          load_tokens<kStep, HD>(&maps.b1, ring + s * 2 * SB + SB, h, row, it.b, &b_full[s]);
          if constexpr (KEYS)   // rows of p.ld are padded to whole steps
            bulk_load(lds + s * kStep, p.ld + ((long long)it.b * p.H + h) * p.ld_stride + row,
                      kStep * 8, &b_full[s]);
        }
      }
      if (*abort) {
        for (long long j = (e > NS ? e - NS : 0); j < e; ++j)
          mbar_drain(&b_full[j % NS], (uint32_t)((j / NS) & 1), kTestLimitNs * 100);
        for (long long j = (k > NA ? k - NA : 0); j < k; ++j)
          mbar_drain(&a_full[j % NA], (uint32_t)((j / NA) & 1), kTestLimitNs * 100);
      }
    }
  } else if (warp == kBMma) {
    if (lane == 0) {   // S = A0 B0^T and dP = A1 B1^T of each step
      constexpr uint32_t idesc = idesc_bf16(kRows, kStep, 0, 0);
      long long k = 0, e = 0;
      uint32_t nb[2] = {0, 0};
      bool ok = true;
      for (long long t = blockIdx.x; t < n_items && ok; t += gridDim.x) {
        const BwdItem<KEYS> it = bwd_item<KEYS>(p, t);
        if (!it.steps) continue;
        const int as = (int)(k % NA);
        if (!mbar_wait(&a_full[as], (uint32_t)((k / NA) & 1), abort, p.status, kWaitLimitNs))
          break;
        const uint32_t a0 = smem_u32(abuf + as * 2 * TB), a1 = a0 + TB;
        for (int x = 0; x < it.steps * it.passes; ++x, ++e) {
          const int s = (int)(e % NS), b = (int)(e & 1);
          // the buffer is free once its previous gradient products are done
          if (!mbar_wait(&b_full[s], (uint32_t)((e / NS) & 1), abort, p.status, kWaitLimitNs) ||
              !mbar_wait(&g_done[b], (nb[b] & 1) ^ 1, abort, p.status, kWaitLimitNs)) {
            ok = false;
            break;
          }
          ++nb[b];
          tc_fence_after();
          const uint32_t b0 = smem_u32(ring + s * 2 * SB), b1 = b0 + SB;
          const uint32_t d = tmem + b * 128;
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk)
            umma_ss(d, desc_kmajor_tile<HD>(a0, kk), sub_kmajor<HD>(b0, kk), idesc, kk);
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk)
            umma_ss(d + 64, desc_kmajor_tile<HD>(a1, kk), sub_kmajor<HD>(b1, kk), idesc, kk);
          umma_commit(&s_full[b]);
        }
        if (ok) umma_commit(&a_empty[as]);
        ++k;
      }
      if (*abort) {
        umma_commit(&drain[0]);
        mbar_drain(&drain[0], 0, kTestLimitNs * 100);
      }
    }
  } else if (warp == kBMma2) {
    // dQ += dS K, or dV += P^T dO and dK += dS^T Q (all lanes walk along: they
    // zero the padding rows of a last streamed pair)
    constexpr uint32_t idesc = idesc_bf16(kRows, HD, 0, 1);
    long long k = 0, e = 0;
    uint32_t nb[2] = {0, 0};
    bool ok = true;
    for (long long t = blockIdx.x; t < n_items && ok; t += gridDim.x) {
      const BwdItem<KEYS> it = bwd_item<KEYS>(p, t);
      if (!it.steps) continue;
      bool first = true;
      for (int x = 0; x < it.steps * it.passes; ++x, ++e) {
        const int s = (int)(e % NS), b = (int)(e & 1);
        const bool grads = x >= it.steps * (it.passes - 1);
        if (!bwd_warp_wait(&b_full[s], (uint32_t)((e / NS) & 1), abort, p.status)) {
          ok = false;
          break;
        }
        const int row = it.row(x % it.steps);
        if (grads && row + kStep > it.n) {
          zero_sub_rows<HD>(ring + s * 2 * SB, it.n - row);
          zero_sub_rows<HD>(ring + s * 2 * SB + SB, it.n - row);
          fence_proxy_async();
          __syncwarp();
        }
        if ((first && grads &&
             !bwd_warp_wait(acc_empty, (uint32_t)((k & 1) ^ 1), abort, p.status)) ||
            !bwd_warp_wait(&p_full[b], nb[b] & 1, abort, p.status)) {
          ok = false;
          break;
        }
        ++nb[b];
        tc_fence_after();
        if (lane == 0) {
          if (grads) {
            const uint32_t b0 = smem_u32(ring + s * 2 * SB), b1 = b0 + SB;
            const uint32_t d = tmem + b * 128;
            // A from TMEM: 16 elements of K are 8 columns; the two column halves
            // of a step sit 32 columns apart
#pragma unroll
            for (int kk = 0; kk < kStep / 16; ++kk) {
              const uint32_t a = d + 32 * (kk >> 1) + 8 * (kk & 1);
              const uint32_t acc = (!first || kk > 0) ? 1u : 0u;
              if constexpr (KEYS) {
                umma_ts(tmem + kAccCol, a, sub_mnmajor<HD>(b1, kk), idesc, acc);
                umma_ts(tmem + kAccCol + HD, a + 64, sub_mnmajor<HD>(b0, kk), idesc, acc);
              } else {
                umma_ts(tmem + kAccCol, a, sub_mnmajor<HD>(b0, kk), idesc, acc);
              }
            }
          }
          umma_commit(&b_empty[s]);
          umma_commit(&g_done[b]);
        }
        __syncwarp();
        if (grads) first = false;
      }
      if (ok && lane == 0) umma_commit(acc_full);
      __syncwarp();
      ++k;
    }
    if (*abort && lane == 0) {
      umma_commit(&drain[1]);
      mbar_drain(&drain[1], 0, kTestLimitNs * 100);
    }
  } else if (warp < kSoft) {
    // Warpgroup wg: buffer wg >> 1, columns 32 (wg & 1) .. of its steps; thread =
    // row (query or key) = TMEM lane.
    const int wg = warp >> 2, buf = wg >> 1, half = wg & 1;
    const int row = threadIdx.x & (kWg - 1);
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lane_base + buf * 128 + 32 * half;
    const float c = p.scale_log2;
    long long e = 0, k = 0;
    uint32_t nb = 0;
    for (long long t = blockIdx.x; t < n_items; t += gridDim.x) {
      if (named_sync_or(1, kSoft * 32, *abort)) break;
      const BwdItem<KEYS> it = bwd_item<KEYS>(p, t);
      const int r = it.r0 + row;
      const bool stored = r < p.S, real = r < it.n;
      if (p.test_timeout && it.steps) mbar_wait(never, 0, abort, p.status, kTestLimitNs);
      float2 ld = make_float2(0.f, 0.f);
      const long long ld_at = ((long long)it.b * p.H + it.h) * p.ld_stride + r;
      if constexpr (!KEYS) {
        if (real) ld = p.ld[ld_at];
      }
      float dsum = 0.f;
      for (int x = 0; x < it.steps * it.passes; ++x, ++e) {
        if (!KEYS && it.passes == 2 && x == it.steps) {
          // D of the row: the four warpgroups' parts, in order
          xch[wg * kRows + row] = dsum;
          named_sync(1, kSoft * 32);
          ld.y = (xch[row] + xch[kRows + row]) + (xch[2 * kRows + row] + xch[3 * kRows + row]);
          if (wg == 0 && real) p.ld[ld_at] = ld;
        }
        if ((int)(e & 1) != buf) continue;
        const int s = (int)(e % NS);
        const int c0 = it.row(x % it.steps) + 32 * half;   // first token of these columns
        mbar_wait(&s_full[buf], nb & 1, abort, p.status, kWaitLimitNs);
        ++nb;
        tc_fence_after();
        float v[32], g[32];
        __syncwarp();
        tmem_ld32(s_col, v);
        tmem_ld32(s_col + 64, g);
        tmem_wait_ld_regs(v);
        reg_fence32(g);
        // visible columns of the row: lo .. hi, and below sk
        int lo, hi, sk = 0;
        bool plain;
        if constexpr (KEYS) {
          lo = r - c0;
          const bool sink = r < p.sinks;
          hi = min(it.d.i1 - 1, sink ? 0x7fffffff : (p.window > 0x7fffffff - r ? 0x7fffffff : r + p.window - 1)) - c0;
          plain = c0 >= it.r0 + kRows - 1 && c0 + 32 <= it.d.i1 &&
                  (c0 + 31 - it.r0 < p.window || it.r0 + kRows <= p.sinks);
        } else {
          hi = r - c0;
          lo = hi - p.window + 1;
          sk = p.sinks - c0;
          plain = c0 + 31 <= it.r0 && (it.r0 + kRows - 1 - c0 < p.window || c0 + 32 <= p.sinks);
        }
        if constexpr (KEYS) {
          const float4* ldv = reinterpret_cast<const float4*>(lds + s * kStep + 32 * half);
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float4 q = ldv[j / 2];   // L, D of two queries
            const float2 a = __ffma2_rn(make_float2(v[j], v[j + 1]), make_float2(c, c),
                                        make_float2(-q.x, -q.z));
            v[j] = ex2(a.x);
            v[j + 1] = ex2(a.y);
            g[j] = g[j] - q.y;
            g[j + 1] = g[j + 1] - q.w;
          }
        } else {
          const float2 nl = make_float2(-ld.x, -ld.x);
          const float sub = it.passes == 2 && x < it.steps ? 0.f : ld.y;
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float2 a = __ffma2_rn(make_float2(v[j], v[j + 1]), make_float2(c, c), nl);
            v[j] = ex2(a.x);
            v[j + 1] = ex2(a.y);
            g[j] = g[j] - sub;
            g[j + 1] = g[j + 1] - sub;
          }
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) g[j] *= v[j];
        if (!plain) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (KEYS ? (j < lo || j > hi) : (j > hi || (j < lo && j >= sk))) {
              v[j] = 0.f;
              g[j] = 0.f;
            }
        }
        if (!KEYS && it.passes == 2 && x < it.steps) {
          float a0 = 0.f, a1 = 0.f;
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            a0 += g[j];
            a1 += g[j + 1];
          }
          dsum += a0 + a1;
        } else {
          uint32_t w[16];
          if constexpr (KEYS) {
#pragma unroll
            for (int j = 0; j < 16; ++j) w[j] = pack_bf16(v[2 * j], v[2 * j + 1]);
            __syncwarp();
            tmem_st16u(s_col, w);
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) w[j] = pack_bf16(g[2 * j], g[2 * j + 1]);
          __syncwarp();
          tmem_st16u(KEYS ? s_col + 64 : s_col, w);
          tmem_wait_st();
        }
        tc_fence_before();
        mbar_arrive(&p_full[buf]);
      }
      // epilogue: each warpgroup a quarter of the accumulator columns
      constexpr int NC = KEYS ? HD / 2 : HD / 4;
      if (it.steps) {
        mbar_wait(acc_full, (uint32_t)(k & 1), abort, p.status, kWaitLimitNs);
        tc_fence_after();
        ++k;
      }
      const uint32_t acc = tmem + lane_base + kAccCol + wg * NC;
      void* dst;
      bool f32 = false;
      float mul = p.scale;
      if constexpr (KEYS) {
        const int off = (wg & 1) * NC;   // dV, dV, dK, dK
        const long long at = ((long long)it.b * p.S + r) * p.ks + (long long)it.h * HD + off;
        f32 = it.d.partial;
        if (f32) dst = (wg < 2 ? it.d.pv : it.d.pk) + row * it.d.row_stride + off;
        else dst = (__nv_bfloat16*)(wg < 2 ? p.dv : p.dk) + at;
        if (wg < 2) mul = 1.f;
      } else {
        dst = (__nv_bfloat16*)p.dq + ((long long)it.b * p.S + r) * p.qs + (long long)it.h * HD +
              wg * NC;
      }
      if (!stored || *abort) dst = nullptr;
      // an item without steps has no products: its rows are zeros whatever TMEM holds
      const bool bad = store_grad<NC>(acc, mul, real && it.steps, dst, f32) && real && it.steps;
      if (it.steps) {
        tc_fence_before();
        mbar_arrive(acc_empty);
      }
      if (named_sync_or(1, kSoft * 32, bad && !*abort)) {
        int* flags = (int*)xch;
        if (wg == 0) flags[row] = 0;
        named_sync(1, kSoft * 32);
        if (bad) flags[row] = 1;
        named_sync(1, kSoft * 32);
        for (int y = warp; y < kRows; y += kSoft)
          if (flags[y]) {
            if constexpr (KEYS) fix_dkv_row<__nv_bfloat16>(p, it.d, it.r0 + y);
            else fix_dq_row<__nv_bfloat16>(p, it.b, it.h, it.r0 + y);
          }
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

// The map [hd, heads, S, B] of one operand, box [64, 1, rows, 1].
bool encode_rows(CUtensorMap* m, const void* base, const SeqParams& p, int heads,
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

template <int HD, bool KEYS>
cudaError_t bwd_launch(const SeqParams& p, const BwdMaps& maps, cudaStream_t st) {
  auto kernel = seq_bwd_kernel<HD, KEYS>;
  const int smem = BwdCfg<HD>::kSmem;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const long long items =
      KEYS ? p.plan.items : (long long)p.B * p.H * ((p.S + kRows - 1) / kRows);
  const int sms = num_sms();
  kernel<<<(unsigned)(items < sms ? items : sms), kBThreads, smem, st>>>(p, maps, items);
  note_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t seq_fast_backward(const SeqParams& p, cudaStream_t st) {
  BwdMaps q, k;
  const long long os = (long long)p.H * p.hd;
  if (!encode_rows(&q.a0, p.q, p, p.H, p.qs, kRows) ||
      !encode_rows(&q.a1, p.dout, p, p.H, os, kRows) ||
      !encode_rows(&q.b0, p.k, p, p.K, p.ks, kStep) ||
      !encode_rows(&q.b1, p.v, p, p.K, p.ks, kStep) ||
      !encode_rows(&k.a0, p.k, p, p.K, p.ks, kRows) ||
      !encode_rows(&k.a1, p.v, p, p.K, p.ks, kRows) ||
      !encode_rows(&k.b0, p.q, p, p.H, p.qs, kStep) ||
      !encode_rows(&k.b1, p.dout, p, p.H, os, kStep))
    return cudaErrorInvalidValue;
  const cudaError_t e =
      p.hd == 64 ? bwd_launch<64, false>(p, q, st) : bwd_launch<128, false>(p, q, st);
  if (e != cudaSuccess) return e;
  return p.hd == 64 ? bwd_launch<64, true>(p, k, st) : bwd_launch<128, true>(p, k, st);
}

}  // namespace swin
