// seq_common.cuh -- device pieces shared by the portable and the tcgen05
// kernels of sequence attention: which keys a query sees, the work items of
// the key-side backward, and the exact recomputation of single rows.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "seq.h"

namespace swin {
namespace {

__device__ __forceinline__ float seq_ld(const float* p) { return *p; }
__device__ __forceinline__ float seq_ld(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void seq_st(float* p, float x) { *p = x; }
__device__ __forceinline__ void seq_st(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

__device__ __forceinline__ int seq_len(const SeqParams& p, int b) {
  if (!p.lengths) return p.S;
  const int n = p.lengths[b];
  return n < 0 ? 0 : (n > p.S ? p.S : n);
}

__device__ __forceinline__ bool seq_visible(const SeqParams& p, int n, int i, int j) {
  return j <= i && i < n && (i - j < p.window || j < p.sinks);
}

// Key tiles of T keys that queries i0 .. i1 - 1 (i1 <= n, i0 < i1) can see:
// 0 .. s - 1 (sinks only) and lo .. hi, s <= lo.
struct KeyTiles {
  int s, lo, hi;
  __device__ int count() const { return s + hi - lo + 1; }
  __device__ int tile(int x) const { return x < s ? x : lo + x - s; }
};
__device__ __forceinline__ KeyTiles seq_key_tiles(const SeqParams& p, int i0, int i1, int T) {
  KeyTiles t;
  const int first = i0 - p.window + 1;
  t.lo = first > 0 ? first / T : 0;
  t.hi = (i1 - 1) / T;
  const int st = (p.sinks + T - 1) / T;
  t.s = st < t.lo ? st : t.lo;
  return t;
}

// One item of the key-side backward: keys tile * T .., query heads h0 .. h1 - 1
// of one kv head, queries i0 .. i1 - 1.
struct DkvItem {
  int b, kh, tile, h0, h1, i0, i1, n;
  bool partial;
  float *pk, *pv;        // partial: fp32 rows of hd, row_stride elements apart
  long long row_stride;
};
__device__ __forceinline__ DkvItem dkv_item(const SeqParams& p, long long id) {
  const DkvPlan& d = p.plan;
  const int nz = p.B * p.K * d.gs;
  const long long r = id / nz;
  const int z = (int)(id - r * nz);
  DkvItem it;
  const int gs = z % d.gs, bk = z / d.gs;
  it.kh = bk % p.K;
  it.b = bk / p.K;
  const int per = p.G / d.gs;
  it.h0 = it.kh * p.G + gs * per;
  it.h1 = it.h0 + per;
  it.n = seq_len(p, it.b);
  int chunk = 0;
  const bool sink = r < (long long)d.nst * d.qc;
  if (sink) {
    it.tile = (int)(r / d.qc);
    chunk = (int)(r - (long long)it.tile * d.qc);
  } else {
    it.tile = d.nst + (int)(r - (long long)d.nst * d.qc);
  }
  const int j0 = it.tile * d.T;
  it.i0 = j0;
  if (sink) {
    it.i0 = max(j0, chunk * d.ch);
    it.i1 = min(it.n, chunk == d.qc - 1 ? it.n : (chunk + 1) * d.ch);
  } else if (j0 < p.sinks) {
    it.i1 = it.n;
  } else {
    const long long e = (long long)j0 + d.T - 1 + p.window;
    it.i1 = e < it.n ? (int)e : it.n;
  }
  it.partial = sink || d.gs > 1;
  it.pk = it.pv = nullptr;
  it.row_stride = 0;
  if (sink) {
    const long long slot = ((long long)z * d.nst + it.tile) * d.qc + chunk;
    it.pk = p.sink_part + slot * 2 * d.T * p.hd;
    it.pv = it.pk + (long long)d.T * p.hd;
    it.row_stride = p.hd;
  } else if (d.gs > 1) {
    const long long all = (long long)p.B * p.S * p.K * p.hd;
    it.pk = p.main_part + gs * 2 * all + (((long long)it.b * p.S + j0) * p.K + it.kh) * p.hd;
    it.pv = it.pk + all;
    it.row_stride = (long long)p.K * p.hd;
  }
  return it;
}

// Bits lo .. hi of 32 columns and those below sk.
__device__ __forceinline__ uint32_t below(int n) {   // bits 0 .. n - 1
  return n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1u);
}
__device__ __forceinline__ uint32_t column_mask(int lo, int hi, int sk) {
  return below(hi + 1) & (~below(lo) | below(sk));
}

// ---- single rows, exactly --------------------------------------------------------
// A tile's products multiply masked entries by zero, and 0 x NaN (or 0 x inf) is
// NaN: a non-finite value of a token that a row does not see can spoil the
// row. The kernels therefore look at each result row, and one that is not
// finite is computed again here by one warp from its visible tokens alone
// (lanes across the channels, tokens one after another). A row that does see
// the value comes out non-finite again, as it should. Not inlined: it never
// runs on finite data.
constexpr int kFixT = 8;   // channels per lane, up to 256

template <typename E>
__device__ __forceinline__ void fix_load(float* r, const E* row, int hd) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int t = 0; t < kFixT; ++t) r[t] = lane + 32 * t < hd ? seq_ld(row + lane + 32 * t) : 0.f;
}
__device__ __forceinline__ float fix_dot(const float* a, const float* b) {
  float s = 0.f;
#pragma unroll
  for (int t = 0; t < kFixT; ++t) s = fmaf(a[t], b[t], s);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}
template <typename E>
__device__ __forceinline__ void fix_store(E* row, const float* r, float mul, int hd) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int t = 0; t < kFixT; ++t)
    if (lane + 32 * t < hd) seq_st(row + lane + 32 * t, r[t] * mul);
}

// Every channel of both is NaN already (all lanes agree): nothing can change it.
__device__ __forceinline__ bool fix_lost(const float* a, const float* b, int hd) {
  bool lost = true;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int t = 0; t < kFixT; ++t)
    if (lane + 32 * t < hd) lost &= a[t] != a[t] && b[t] != b[t];
  return __all_sync(0xffffffffu, lost);
}

template <typename E>
__device__ __noinline__ void fix_out_row(const SeqParams& p, int b, int h, int i) {
  const int kh = h / p.G;
  const E* kb = (const E*)p.k + (long long)b * p.S * p.ks + (long long)kh * p.hd;
  const E* vb = (const E*)p.v + (long long)b * p.S * p.ks + (long long)kh * p.hd;
  float q[kFixT], x[kFixT], acc[kFixT];
  fix_load(q, (const E*)p.q + ((long long)b * p.S + i) * p.qs + (long long)h * p.hd, p.hd);
#pragma unroll
  for (int t = 0; t < kFixT; ++t) acc[t] = 0.f;
  const int lo = max(0, i - p.window + 1);
  float m = -INFINITY, l = 0.f;
  for (int j = p.sinks > 0 ? 0 : lo; j <= i; ++j) {
    if (j >= p.sinks && j < lo) j = lo;
    fix_load(x, kb + (long long)j * p.ks, p.hd);
    const float a = fix_dot(q, x) * p.scale_log2;
    const float mn = a > m ? a : (a != a ? a : m);   // a NaN stays
    const float f = mn == -INFINITY ? 1.f : exp2f(m - mn);
    const float w = a == -INFINITY ? 0.f : exp2f(a - mn);
    m = mn;
    l = l * f + w;
    fix_load(x, vb + (long long)j * p.ks, p.hd);
#pragma unroll
    for (int t = 0; t < kFixT; ++t) acc[t] = fmaf(w, x[t], acc[t] * f);
    // (lse needs every key: only where it is NaN as well is there nothing left)
    if ((j & 15) == 15 && l != l && fix_lost(acc, acc, p.hd)) break;
  }
  const long long row = ((long long)b * p.S + i) * p.H + h;
  fix_store((E*)p.out + row * p.hd, acc, 1.f / l, p.hd);
  if (p.lse && (threadIdx.x & 31) == 0) p.lse[row] = (m + log2f(l)) / kSeqLog2e;
}

template <typename E>
__device__ __noinline__ void fix_dq_row(const SeqParams& p, int b, int h, int i) {
  const int kh = h / p.G;
  const E* kb = (const E*)p.k + (long long)b * p.S * p.ks + (long long)kh * p.hd;
  const E* vb = (const E*)p.v + (long long)b * p.S * p.ks + (long long)kh * p.hd;
  float q[kFixT], g[kFixT], x[kFixT], y[kFixT], acc[kFixT];
  fix_load(q, (const E*)p.q + ((long long)b * p.S + i) * p.qs + (long long)h * p.hd, p.hd);
  fix_load(g, (const E*)p.dout + (((long long)b * p.S + i) * p.H + h) * p.hd, p.hd);
#pragma unroll
  for (int t = 0; t < kFixT; ++t) acc[t] = 0.f;
  const long long la = ((long long)b * p.H + h) * p.ld_stride + i;
  const float nl = p.nl[la], nd = p.nd[la];
  const int lo = max(0, i - p.window + 1);
  for (int j = p.sinks > 0 ? 0 : lo; j <= i; ++j) {
    if (j >= p.sinks && j < lo) j = lo;
    fix_load(x, kb + (long long)j * p.ks, p.hd);
    fix_load(y, vb + (long long)j * p.ks, p.hd);
    const float w = exp2f(fix_dot(q, x) * p.scale_log2 + nl);
    const float ds = w * (fix_dot(g, y) + nd);
#pragma unroll
    for (int t = 0; t < kFixT; ++t) acc[t] = fmaf(ds, x[t], acc[t]);
    if ((j & 15) == 15 && fix_lost(acc, acc, p.hd)) break;
  }
  fix_store((E*)p.dq + ((long long)b * p.S + i) * p.qs + (long long)h * p.hd, acc, p.scale, p.hd);
}

// dk and dv of key j over the item's heads and queries, to the item's partial
// rows or to dk, dv.
template <typename E>
__device__ __noinline__ void fix_dkv_row(const SeqParams& p, const DkvItem& it, int j) {
  const long long at = ((long long)it.b * p.S + j) * p.ks + (long long)it.kh * p.hd;
  float k[kFixT], v[kFixT], x[kFixT], y[kFixT], ak[kFixT], av[kFixT];
  fix_load(k, (const E*)p.k + at, p.hd);
  fix_load(v, (const E*)p.v + at, p.hd);
#pragma unroll
  for (int t = 0; t < kFixT; ++t) ak[t] = av[t] = 0.f;
  bool lost = false;
  for (int h = it.h0; h < it.h1 && !lost; ++h)
    for (int i = max(it.i0, j); i < it.i1 && !lost; ++i) {
      if (!seq_visible(p, it.n, i, j)) break;
      fix_load(x, (const E*)p.q + ((long long)it.b * p.S + i) * p.qs + (long long)h * p.hd, p.hd);
      fix_load(y, (const E*)p.dout + (((long long)it.b * p.S + i) * p.H + h) * p.hd, p.hd);
      const long long la = ((long long)it.b * p.H + h) * p.ld_stride + i;
      const float w = exp2f(fix_dot(x, k) * p.scale_log2 + p.nl[la]);
      const float ds = w * (fix_dot(y, v) + p.nd[la]);
#pragma unroll
      for (int t = 0; t < kFixT; ++t) {
        ak[t] = fmaf(ds, x[t], ak[t]);
        av[t] = fmaf(w, y[t], av[t]);
      }
      lost = (i & 15) == 15 && fix_lost(ak, av, p.hd);
    }
  if (it.partial) {
    const long long r = (j - it.tile * p.plan.T) * it.row_stride;
    fix_store(it.pk + r, ak, p.scale, p.hd);
    fix_store(it.pv + r, av, 1.f, p.hd);
  } else {
    fix_store((E*)p.dk + at, ak, p.scale, p.hd);
    fix_store((E*)p.dv + at, av, 1.f, p.hd);
  }
}

}  // namespace
}  // namespace swin
