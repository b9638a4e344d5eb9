// seq_generic.cu -- portable kernels of sequence attention (sliding window with
// sink tokens): fp32 storage and every head size; also the (lse, D) rows and the
// sums of partials that both kernel families use.
//
// One pass over the visible key tiles with a running maximum and sum (forward);
// the backward recomputes P from lse, once by query tiles (dq) and once by key
// tiles (dk, dv), so no sum crosses blocks and results are repeatable. All
// arithmetic is fp32 FMA on tiles in shared memory: 256 threads as 16 x 16,
// each holding a (T/16) x (T/16) piece of the logits and (T/16) x (HD/16) of the
// accumulators, fed by 16-byte shared loads (rows padded by 4 floats, which
// keeps the 16 rows a quarter-warp reads on different banks). Bound by the FMA
// pipe and shared loads, not by memory: a tile of T keys is read once for T
// queries.
#include <math.h>

#include "seq_common.cuh"
#include "sm100_ptx.cuh"

namespace swin {
namespace {

constexpr int kThr = 256;


// rows row0 .. row0 + T - 1 (those below `rows` real, others zero) of hd channels
template <typename E, int HD, int T>
__device__ __forceinline__ void load_tile(float* dst, const E* src, long long stride, int rows,
                                          int hd) {
  constexpr int C = HD / 8;
  for (int x = threadIdx.x; x < T * C; x += kThr) {
    const int r = x / C, c = (x - r * C) * 8;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
    if (r < rows && c < hd) {
      const E* s = src + r * stride + c;
      if constexpr (sizeof(E) == 4) {
        a = *reinterpret_cast<const float4*>(s);
        b = *reinterpret_cast<const float4*>(s + 4);
      } else {
        const uint4 u = *reinterpret_cast<const uint4*>(s);
        a = make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u),
                        __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xFFFF0000u));
        b = make_float4(__uint_as_float(u.z << 16), __uint_as_float(u.z & 0xFFFF0000u),
                        __uint_as_float(u.w << 16), __uint_as_float(u.w & 0xFFFF0000u));
      }
    }
    float* d = dst + r * (HD + 4) + c;
    *reinterpret_cast<float4*>(d) = a;
    *reinterpret_cast<float4*>(d + 4) = b;
  }
}

// acc[r][c] = sum_d a[ty + 16 r][d] b[tx + 16 c][d]. What bounds these products are the
// reads of their operands from shared memory, two values per FMA of a thread's 4 x 4
// outputs: 17 to 20 of the FMA pipe's 70 TFLOP/s for 4096 tokens (packed FMAs instead
// of single ones: 583 us against 610 for the backward, the forward as it was).
template <int HD, int R>
__device__ __forceinline__ void tile_dots(float (&acc)[R][R], const float* a, const float* b,
                                          int ty, int tx) {
  float2 two[R][R];   // even and odd channels
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int c = 0; c < R; ++c) two[r][c] = make_float2(0.f, 0.f);
#pragma unroll 4
  for (int d = 0; d < HD; d += 4) {
    float4 x[R], y[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      x[r] = *reinterpret_cast<const float4*>(a + (ty + 16 * r) * (HD + 4) + d);
      y[r] = *reinterpret_cast<const float4*>(b + (tx + 16 * r) * (HD + 4) + d);
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < R; ++c) {
        two[r][c] = __ffma2_rn(make_float2(x[r].x, x[r].y), make_float2(y[c].x, y[c].y), two[r][c]);
        two[r][c] = __ffma2_rn(make_float2(x[r].z, x[r].w), make_float2(y[c].z, y[c].w), two[r][c]);
      }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int c = 0; c < R; ++c) acc[r][c] = two[r][c].x + two[r][c].y;
}

// Channels of a thread: NC = HD / 16 in runs of V.
template <int HD>
struct Cols {
  static constexpr int NC = HD / 16;
  static constexpr int V = NC < 4 ? NC : 4;
  __device__ static int col(int tx, int c) { return (c / V) * 16 * V + tx * V + c % V; }
};

// acc[r][c] += sum_k w[ty + 16 r][k] m[k][col c]
template <int HD, int R, int T>
__device__ __forceinline__ void tile_accum(float (&acc)[R][HD / 16], const float* w,
                                           const float* m, int ty, int tx) {
  using C = Cols<HD>;
#pragma unroll 2
  for (int k = 0; k < T; k += 4) {
    float4 x[R];
#pragma unroll
    for (int r = 0; r < R; ++r)
      x[r] = *reinterpret_cast<const float4*>(w + (ty + 16 * r) * (T + 4) + k);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float y[C::NC];
#pragma unroll
      for (int c = 0; c < C::NC; c += C::V) {
        const float* s = m + (k + u) * (HD + 4) + C::col(tx, c);
        if constexpr (C::V == 4) {
          const float4 f = *reinterpret_cast<const float4*>(s);
          y[c] = f.x; y[c + 1] = f.y; y[c + 2] = f.z; y[c + 3] = f.w;
        } else {
          const float2 f = *reinterpret_cast<const float2*>(s);
          y[c] = f.x; y[c + 1] = f.y;
        }
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float e = u == 0 ? x[r].x : (u == 1 ? x[r].y : (u == 2 ? x[r].z : x[r].w));
#pragma unroll
        for (int c = 0; c < C::NC; c += 2) {
          const float2 f = __ffma2_rn(make_float2(e, e), make_float2(y[c], y[c + 1]),
                                      make_float2(acc[r][c], acc[r][c + 1]));
          acc[r][c] = f.x;
          acc[r][c + 1] = f.y;
        }
      }
    }
  }
}

__device__ __forceinline__ float half_max(float v) {   // over the 16 threads of a row
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float half_sum(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Marks the tile's rows that hold a non-finite value (each thread's part of
// row ty + 16 r is acc[r][..]); flags is cleared by the caller before.
template <int R, int NC>
__device__ __forceinline__ void flag_rows(const float (&acc)[R][NC], int* flags, int ty) {
#pragma unroll
  for (int r = 0; r < R; ++r) {
    bool bad = false;
#pragma unroll
    for (int c = 0; c < NC; ++c) bad |= !(fabsf(acc[r][c]) <= 3.4028235e38f);
    if (bad) flags[ty + 16 * r] = 1;
  }
}

template <typename E, int HD, int T>
__global__ void __launch_bounds__(kThr) gen_fwd_kernel(const __grid_constant__ SeqParams p) {
  constexpr int R = T / 16, NC = HD / 16;
  using C = Cols<HD>;
  extern __shared__ float sm[];
  float* qs = sm;
  float* kv = qs + T * (HD + 4);
  float* ps = kv + T * (HD + 4);
  int* flags = (int*)(ps + T * (T + 4));
  const int ntile = (p.S + T - 1) / T;
  const long long bh = blockIdx.x / ntile;
  const int tile = ntile - 1 - (int)(blockIdx.x - bh * ntile);   // the longest rows first
  const int b = (int)(bh / p.H), h = (int)(bh - (long long)b * p.H), kh = h / p.G;
  const int n = seq_len(p, b), i0 = tile * T, stored = min(T, p.S - i0);
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  E* out = (E*)p.out + (((long long)b * p.S + i0) * p.H + h) * p.hd;
  const long long os = (long long)p.H * p.hd;
  float acc[R][NC], m[R], l[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) acc[r][c] = 0.f;
  }
  if (threadIdx.x < T) flags[threadIdx.x] = 0;
  if (i0 < n) {
    load_tile<E, HD, T>(qs, (const E*)p.q + ((long long)b * p.S + i0) * p.qs + (long long)h * p.hd,
                        p.qs, min(T, n - i0), p.hd);
    const E* kb = (const E*)p.k + (long long)b * p.S * p.ks + (long long)kh * p.hd;
    const E* vb = (const E*)p.v + (long long)b * p.S * p.ks + (long long)kh * p.hd;
    const KeyTiles kt = seq_key_tiles(p, i0, min(n, i0 + T), T);
    for (int x = 0; x < kt.count(); ++x) {
      const int j0 = kt.tile(x) * T;
      __syncthreads();
      load_tile<E, HD, T>(kv, kb + (long long)j0 * p.ks, p.ks, min(T, n - j0), p.hd);
      __syncthreads();
      float s[R][R];
      tile_dots<HD, R>(s, qs, kv, ty, tx);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int i = i0 + ty + 16 * r;
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < R; ++c) {
          s[r][c] = seq_visible(p, n, i, j0 + tx + 16 * c) ? s[r][c] * p.scale_log2 : -INFINITY;
          mx = fmaxf(mx, s[r][c]);
        }
        mx = fmaxf(m[r], half_max(mx));
        const float mu = mx == -INFINITY ? 0.f : mx;   // a row with no key yet: P = 0
        const float f = exp2f(m[r] - mu);
        m[r] = mx;
        l[r] *= f;
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[r][c] *= f;
#pragma unroll
        for (int c = 0; c < R; ++c) {
          const float w = exp2f(s[r][c] - mu);
          l[r] += w;
          ps[(ty + 16 * r) * (T + 4) + tx + 16 * c] = w;
        }
      }
      __syncthreads();
      load_tile<E, HD, T>(kv, vb + (long long)j0 * p.ks, p.ks, min(T, n - j0), p.hd);
      __syncthreads();
      tile_accum<HD, R, T>(acc, ps, kv, ty, tx);
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = ty + 16 * r;
    const float sum = half_sum(l[r]);
    if (row >= stored) continue;
    const bool real = i0 + row < n;
    const float inv = real ? 1.f / sum : 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      acc[r][c] = real ? acc[r][c] * inv : 0.f;
      if (C::col(tx, c) < p.hd) seq_st(out + row * os + C::col(tx, c), acc[r][c]);
    }
    if (p.lse && tx == 0)
      p.lse[((long long)b * p.S + i0 + row) * p.H + h] =
          real ? (m[r] + log2f(sum)) / kSeqLog2e : 0.f;
  }
  flag_rows<R, NC>(acc, flags, ty);
  __syncthreads();
  for (int row = threadIdx.x / 32; row < stored; row += kThr / 32)
    if (flags[row] && i0 + row < n) fix_out_row<E>(p, b, h, i0 + row);
}

template <typename E, int HD, int T>
__global__ void __launch_bounds__(kThr) gen_dq_kernel(const __grid_constant__ SeqParams p) {
  constexpr int R = T / 16, NC = HD / 16;
  using C = Cols<HD>;
  extern __shared__ float sm[];
  float* qs = sm;
  float* gs = qs + T * (HD + 4);
  float* ks = gs + T * (HD + 4);
  float* vs = ks + T * (HD + 4);
  float* ps = vs + T * (HD + 4);
  int* flags = (int*)(ps + T * (T + 4));
  const int ntile = (p.S + T - 1) / T;
  const long long bh = blockIdx.x / ntile;
  const int tile = ntile - 1 - (int)(blockIdx.x - bh * ntile);
  const int b = (int)(bh / p.H), h = (int)(bh - (long long)b * p.H), kh = h / p.G;
  const int n = seq_len(p, b), i0 = tile * T, stored = min(T, p.S - i0);
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  ptx::grid_dep_wait();
  float acc[R][NC];
  float2 ld[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int c = 0; c < NC; ++c) acc[r][c] = 0.f;
    const int i = i0 + ty + 16 * r;
    const long long la = bh * p.ld_stride + i;
    ld[r] = i < n ? make_float2(p.nl[la], p.nd[la]) : make_float2(0.f, 0.f);
  }
  if (threadIdx.x < T) flags[threadIdx.x] = 0;
  if (i0 < n) {
    const int rows = min(T, n - i0);
    load_tile<E, HD, T>(qs, (const E*)p.q + ((long long)b * p.S + i0) * p.qs + (long long)h * p.hd,
                        p.qs, rows, p.hd);
    load_tile<E, HD, T>(gs, (const E*)p.dout + (((long long)b * p.S + i0) * p.H + h) * p.hd,
                        (long long)p.H * p.hd, rows, p.hd);
    const E* kb = (const E*)p.k + (long long)b * p.S * p.ks + (long long)kh * p.hd;
    const E* vb = (const E*)p.v + (long long)b * p.S * p.ks + (long long)kh * p.hd;
    const KeyTiles kt = seq_key_tiles(p, i0, min(n, i0 + T), T);
    for (int x = 0; x < kt.count(); ++x) {
      const int j0 = kt.tile(x) * T;
      __syncthreads();
      load_tile<E, HD, T>(ks, kb + (long long)j0 * p.ks, p.ks, min(T, n - j0), p.hd);
      load_tile<E, HD, T>(vs, vb + (long long)j0 * p.ks, p.ks, min(T, n - j0), p.hd);
      __syncthreads();
      float s[R][R], dp[R][R];
      tile_dots<HD, R>(s, qs, ks, ty, tx);
      tile_dots<HD, R>(dp, gs, vs, ty, tx);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < R; ++c) {
          const bool see = seq_visible(p, n, i0 + ty + 16 * r, j0 + tx + 16 * c);
          const float w = exp2f(s[r][c] * p.scale_log2 + ld[r].x);
          ps[(ty + 16 * r) * (T + 4) + tx + 16 * c] = see ? w * (dp[r][c] + ld[r].y) : 0.f;
        }
      __syncthreads();
      tile_accum<HD, R, T>(acc, ps, ks, ty, tx);
    }
  }
  __syncthreads();
  E* dq = (E*)p.dq + ((long long)b * p.S + i0) * p.qs + (long long)h * p.hd;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = ty + 16 * r;
    if (row >= stored) continue;
#pragma unroll
    for (int c = 0; c < NC; ++c)
      if (C::col(tx, c) < p.hd)   // padding: zeros, whatever masked tokens hold
        seq_st(dq + row * p.qs + C::col(tx, c), i0 + row < n ? acc[r][c] * p.scale : 0.f);
  }
  flag_rows<R, NC>(acc, flags, ty);
  __syncthreads();
  for (int row = threadIdx.x / 32; row < stored; row += kThr / 32)
    if (flags[row] && i0 + row < n) fix_dq_row<E>(p, b, h, i0 + row);
}

template <typename E, int HD, int T>
__global__ void __launch_bounds__(kThr) gen_dkv_kernel(const __grid_constant__ SeqParams p) {
  constexpr int R = T / 16, NC = HD / 16;
  using C = Cols<HD>;
  extern __shared__ float sm[];
  float* ks = sm;
  float* vs = ks + T * (HD + 4);
  float* qs = vs + T * (HD + 4);
  float* gs = qs + T * (HD + 4);
  float* ps = gs + T * (HD + 4);
  float* ds = ps + T * (T + 4);
  float2* lds = (float2*)(ds + T * (T + 4));
  int* flags = (int*)(lds + T);
  const DkvItem it = dkv_item(p, blockIdx.x);
  ptx::grid_dep_wait();
  const int j0 = it.tile * T, stored = min(T, p.S - j0);
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  float ak[R][NC], av[R][NC];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int c = 0; c < NC; ++c) ak[r][c] = av[r][c] = 0.f;
  if (threadIdx.x < T) flags[threadIdx.x] = 0;
  if (it.i0 < it.i1) {
    const long long at = ((long long)it.b * p.S + j0) * p.ks + (long long)it.kh * p.hd;
    load_tile<E, HD, T>(ks, (const E*)p.k + at, p.ks, min(T, it.n - j0), p.hd);
    load_tile<E, HD, T>(vs, (const E*)p.v + at, p.ks, min(T, it.n - j0), p.hd);
    for (int h = it.h0; h < it.h1; ++h)
      for (int i0 = it.i0; i0 < it.i1; i0 += T) {
        const int rows = min(T, it.i1 - i0);
        __syncthreads();
        load_tile<E, HD, T>(qs,
                            (const E*)p.q + ((long long)it.b * p.S + i0) * p.qs + (long long)h * p.hd,
                            p.qs, rows, p.hd);
        load_tile<E, HD, T>(gs, (const E*)p.dout + (((long long)it.b * p.S + i0) * p.H + h) * p.hd,
                            (long long)p.H * p.hd, rows, p.hd);
        if (threadIdx.x < T) {
          const long long la = ((long long)it.b * p.H + h) * p.ld_stride + i0 + threadIdx.x;
          lds[threadIdx.x] = (int)threadIdx.x < rows ? make_float2(p.nl[la], p.nd[la])
                                                     : make_float2(0.f, 0.f);
        }
        __syncthreads();
        float s[R][R], dp[R][R];
        tile_dots<HD, R>(s, ks, qs, ty, tx);
        tile_dots<HD, R>(dp, vs, gs, ty, tx);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int c = 0; c < R; ++c) {
            const int i = i0 + tx + 16 * c;
            const float2 ld = lds[tx + 16 * c];
            const bool see = i < it.i1 && seq_visible(p, it.n, i, j0 + ty + 16 * r);
            const float w = exp2f(s[r][c] * p.scale_log2 + ld.x);
            ps[(ty + 16 * r) * (T + 4) + tx + 16 * c] = see ? w : 0.f;
            ds[(ty + 16 * r) * (T + 4) + tx + 16 * c] = see ? w * (dp[r][c] + ld.y) : 0.f;
          }
        __syncthreads();
        tile_accum<HD, R, T>(av, ps, gs, ty, tx);
        tile_accum<HD, R, T>(ak, ds, qs, ty, tx);
      }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = ty + 16 * r;
    if (row >= stored) continue;
    const long long at = ((long long)it.b * p.S + j0 + row) * p.ks + (long long)it.kh * p.hd;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int col = C::col(tx, c);
      if (col >= p.hd) continue;
      const bool real = j0 + row < it.n;   // padding: zeros, whatever masked tokens hold
      const float dk = real ? ak[r][c] * p.scale : 0.f, dv = real ? av[r][c] : 0.f;
      if (it.partial) {
        it.pk[row * it.row_stride + col] = dk;
        it.pv[row * it.row_stride + col] = dv;
      } else {
        seq_st((E*)p.dk + at + col, dk);
        seq_st((E*)p.dv + at + col, dv);
      }
    }
  }
  flag_rows<R, NC>(ak, flags, ty);
  flag_rows<R, NC>(av, flags, ty);
  __syncthreads();
  for (int row = threadIdx.x / 32; row < stored; row += kThr / 32)
    if (flags[row] && j0 + row < it.n) fix_dkv_row<E>(p, it, j0 + row);
}

// (-lse log2 e, -D), D = dO.o, of every row, [B][H][ld_stride]: `lanes` lanes per
// row (16 bytes of out and dout each at a time), so a warp reads whole lines.
// Bound by HBM (out and dout once).
template <typename E>
__global__ void __launch_bounds__(256) prep_kernel(const __grid_constant__ SeqParams p, int shift) {
  // (only blocks that fill an SM may come early: small ones would crowd on the first
  // SMs with room, 80 us against 65 for the portable backward of 544 tokens)
  if (p.plan.T == 128) ptx::grid_dep_launch();
  const int lanes = 1 << shift;
  const long long row = ((long long)blockIdx.x * 256 + threadIdx.x) >> shift;   // (b S + i) H + h
  const int lane = threadIdx.x & (lanes - 1);
  constexpr int V = 16 / sizeof(E);
  float d = 0.f;
  bool real = false;
  long long at = -1;
  if (row < (long long)p.B * p.S * p.H) {
    // (32-bit division where it fits: a 64-bit one is some hundred cycles)
    const long long tok = row >> 32 ? row / p.H : (long long)((uint32_t)row / (uint32_t)p.H);
    const int h = (int)(row - tok * p.H);
    const int b = (int)((uint32_t)tok / (uint32_t)p.S), i = (int)(tok - (long long)b * p.S);
    at = ((long long)b * p.H + h) * p.ld_stride + i;
    real = i < seq_len(p, b);
  }
  if (real) {
    const E* o = (const E*)p.o + row * p.hd;
    const E* g = (const E*)p.dout + row * p.hd;
#pragma unroll 4
    for (int c = lane * V; c < p.hd; c += lanes * V) {
      const uint4 uo = *reinterpret_cast<const uint4*>(o + c);
      const uint4 ug = *reinterpret_cast<const uint4*>(g + c);
      const E* eo = reinterpret_cast<const E*>(&uo);
      const E* eg = reinterpret_cast<const E*>(&ug);
#pragma unroll
      for (int e = 0; e < V; ++e) d = fmaf(seq_ld(eo + e), seq_ld(eg + e), d);
    }
  }
  for (int o = lanes / 2; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  if (lane == 0 && at >= 0) {
    p.nl[at] = real ? -p.lse_in[row] * kSeqLog2e : -INFINITY;
    p.nd[at] = -d;
  }
}

// dk, dv of every key row whose items left partials, summed in the order of the
// parts (query-head parts, then query chunks), 4 channels a thread.
template <typename E>
__global__ void __launch_bounds__(256) dkv_reduce_kernel(const __grid_constant__ SeqParams p) {
  const DkvPlan& d = p.plan;
  const uint32_t q4 = p.hd / 4;
  const long long x = (long long)blockIdx.x * 256 + threadIdx.x;
  // with gs == 1 only the sink tiles have partials
  const uint32_t rows = d.gs > 1 ? p.S : min(p.S, d.nst * d.T);
  const uint32_t per = p.K * q4;   // of a token
  const long long tok = x / per;
  if (tok >= (long long)p.B * rows) return;   // (nothing to wait for)
  const uint32_t y = (uint32_t)(x - tok * per);
  const int kh = y / q4, c = (int)(y - kh * q4) * 4;
  const int b = (int)((uint32_t)tok / rows), j = (int)((uint32_t)tok - b * rows);
  const int tile = j / d.T;
  ptx::grid_dep_wait();
  float4 k = make_float4(0.f, 0.f, 0.f, 0.f), v = k;
  auto add = [](float4& a, const float* s) {
    const float4 t = *reinterpret_cast<const float4*>(s);
    a.x += t.x; a.y += t.y; a.z += t.z; a.w += t.w;
  };
  for (int g = 0; g < d.gs; ++g) {
    if (tile < d.nst) {
      const long long z = ((long long)b * p.K + kh) * d.gs + g;
      for (int u = 0; u < d.qc; ++u) {
        const float* s = p.sink_part + ((z * d.nst + tile) * d.qc + u) * 2 * d.T * p.hd +
                         (long long)(j - tile * d.T) * p.hd + c;
        add(k, s);
        add(v, s + (long long)d.T * p.hd);
      }
    } else {
      const long long all = (long long)p.B * p.S * p.K * p.hd;
      const float* s = p.main_part + g * 2 * all + (((long long)b * p.S + j) * p.K + kh) * p.hd + c;
      add(k, s);
      add(v, s + all);
    }
  }
  const long long at = ((long long)b * p.S + j) * p.ks + (long long)kh * p.hd + c;
  if constexpr (sizeof(E) == 4) {
    *reinterpret_cast<float4*>((E*)p.dk + at) = k;
    *reinterpret_cast<float4*>((E*)p.dv + at) = v;
  } else {
    auto pack = [](float4 f) {
      __nv_bfloat162 h[2] = {__floats2bfloat162_rn(f.x, f.y), __floats2bfloat162_rn(f.z, f.w)};
      return *reinterpret_cast<uint2*>(h);
    };
    *reinterpret_cast<uint2*>((E*)p.dk + at) = pack(k);
    *reinterpret_cast<uint2*>((E*)p.dv + at) = pack(v);
  }
}

// `after`: behind another kernel of the same call.
template <auto Kernel>
cudaError_t go(long long grid, size_t smem, const SeqParams& p, cudaStream_t st, bool after) {
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const cudaError_t e = allow_smem<Kernel>(smem);
  if (e != cudaSuccess) return e;
  if (after) return launch_dependent(Kernel, dim3((unsigned)grid), kThr, smem, st, p);
  Kernel<<<(unsigned)grid, kThr, smem, st>>>(p);
  note_launch();
  return cudaGetLastError();
}

template <typename E, int HD, int T>
cudaError_t fwd(const SeqParams& p, cudaStream_t st) {
  const size_t smem = (2 * T * (HD + 4) + T * (T + 4) + T) * 4;
  return go<gen_fwd_kernel<E, HD, T>>((long long)p.B * p.H * ((p.S + T - 1) / T), smem, p, st,
                                      false);
}
template <typename E, int HD, int T>
cudaError_t bwd(const SeqParams& p, cudaStream_t st) {
  const size_t dq = (4 * T * (HD + 4) + T * (T + 4) + T) * 4;
  const size_t dkv = (4 * T * (HD + 4) + 2 * T * (T + 4) + 3 * T) * 4;
  const cudaError_t e =
      go<gen_dq_kernel<E, HD, T>>((long long)p.B * p.H * ((p.S + T - 1) / T), dq, p, st, true);
  if (e != cudaSuccess) return e;
  return go<gen_dkv_kernel<E, HD, T>>(p.plan.items, dkv, p, st, true);
}
template <typename E, int T>
cudaError_t run_hd(const SeqParams& p, bool back, cudaStream_t st) {
  if (p.hd <= 32) return back ? bwd<E, 32, T>(p, st) : fwd<E, 32, T>(p, st);
  if (p.hd <= 64) return back ? bwd<E, 64, T>(p, st) : fwd<E, 64, T>(p, st);
  return back ? bwd<E, 128, T>(p, st) : fwd<E, 128, T>(p, st);
}
template <typename E>
cudaError_t run_tile(const SeqParams& p, bool back, cudaStream_t st) {
  if (p.hd > 128) return back ? bwd<E, 256, 32>(p, st) : fwd<E, 256, 32>(p, st);
  return p.plan.T == 32 ? run_hd<E, 32>(p, back, st) : run_hd<E, 64>(p, back, st);
}

}  // namespace

// 64 x 64 tiles feed the FMA pipe better, 32 x 32 tiles give four times the blocks;
// the small ones are for work that would leave SMs without a block, for sequences
// that one of them holds (and for heads above 128, whose large tiles would not fit
// shared memory).
int seq_generic_tile(int B, int S, int H, int hd) {
  return hd > 128 || S <= 32 || (long long)B * H * ((S + 63) / 64) < kSeqSms ? 32 : 64;
}

DkvPlan make_dkv_plan(int B, int S, int K, int G, int hd, int window, int sinks, int T) {
  DkvPlan d;
  d.T = T;
  d.ntiles = (S + T - 1) / T;
  // Chunks of the sink tiles' queries: as many queries as a window tile has, four
  // tiles at least (eight of the tensor-core kernels', whose items cost some steps
  // besides) and at most 16 chunks; not for more than four sink tiles, which are
  // enough to fill the card by themselves.
  const int st = (sinks + T - 1) / T;
  d.nst = d.qc = d.ch = 0;
  if (st > 0 && st <= 4) {
    int ch = (S + 15) / 16;
    ch = ch < window + T ? window + T : ch;
    const int least = T == 128 ? 8 * T : 4 * T;
    ch = ch < least ? least : ch;
    ch = (int)(((long long)ch + T - 1) / T * T);
    if (ch < S) {
      d.nst = st < d.ntiles ? st : d.ntiles;
      d.ch = ch;
      d.qc = (S + ch - 1) / ch;
    }
  }
  // Parts of a group's query heads: the fewest that give the card four items
  // per SM.
  const long long tiles = (long long)d.nst * d.qc + d.ntiles - d.nst;
  d.gs = 1;
  for (int g = 1; g <= G; ++g)
    if (G % g == 0) {
      d.gs = g;
      if ((long long)B * K * g * tiles >= 4LL * kSeqSms) break;
    }
  d.items = (long long)B * K * d.gs * tiles;
  d.main_bytes = d.gs > 1 ? (size_t)2 * d.gs * B * S * K * hd * 4 : 0;
  d.sink_bytes = (size_t)2 * B * K * d.gs * d.nst * d.qc * T * hd * 4;
  return d;
}

cudaError_t seq_generic_forward(const SeqParams& p, int dtype, cudaStream_t st) {
  return dtype == SWIN_DTYPE_BF16 ? run_tile<__nv_bfloat16>(p, false, st)
                                  : run_tile<float>(p, false, st);
}

cudaError_t seq_generic_backward(const SeqParams& p, int dtype, cudaStream_t st) {
  return dtype == SWIN_DTYPE_BF16 ? run_tile<__nv_bfloat16>(p, true, st)
                                  : run_tile<float>(p, true, st);
}

cudaError_t seq_prep(const SeqParams& p, int dtype, cudaStream_t st) {
  // lanes of a row, a power of two: two chunks of 16 bytes of out and dout each (one: the
  // finding of places costs more; 165 us against 162.5 for a backward of 2 x 4096 tokens)
  int shift = 0;
  while (shift < 5 && (2 << shift) * (dtype == SWIN_DTYPE_BF16 ? 8 : 4) < p.hd) ++shift;
  const long long rows = (long long)p.B * p.S * p.H, grid = ((rows << shift) + 255) / 256;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if (dtype == SWIN_DTYPE_BF16)
    prep_kernel<__nv_bfloat16><<<(unsigned)grid, 256, 0, st>>>(p, shift);
  else
    prep_kernel<float><<<(unsigned)grid, 256, 0, st>>>(p, shift);
  note_launch();
  return cudaGetLastError();
}

cudaError_t seq_reduce(const SeqParams& p, int dtype, cudaStream_t st) {
  const DkvPlan& d = p.plan;
  if (d.gs == 1 && d.nst == 0) return cudaSuccess;
  const long long rows = d.gs > 1 ? p.S : (p.S < d.nst * d.T ? p.S : d.nst * d.T);
  const long long grid = ((long long)p.B * rows * p.K * (p.hd / 4) + 255) / 256;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const dim3 g((unsigned)grid);
  return dtype == SWIN_DTYPE_BF16
             ? launch_dependent(dkv_reduce_kernel<__nv_bfloat16>, g, 256, 0, st, p)
             : launch_dependent(dkv_reduce_kernel<float>, g, 256, 0, st, p);
}

}  // namespace swin
