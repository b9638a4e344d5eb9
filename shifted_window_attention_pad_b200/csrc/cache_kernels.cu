// cache_kernels.cu -- the paged key-value cache: appending tokens, attention of
// one token per sequence, and eviction by accumulated attention weight
// (declared in include/swin_seqattn.h).
#include <math.h>

#include "seq_common.cuh"
#include "sm100_ptx.cuh"

namespace swin {
namespace {

constexpr int kDecThr = 128;    // decode block: 4 warps
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ int cache_len(const CacheParams& p, int b) {
  const int n = p.lengths[b];
  return n < 0 ? 0 : (n > p.max_len ? (int)p.max_len : n);
}

// Row of position pos of sequence b in units of rows of one kv head:
// (page * K + kh) * ps + row; -1 (and the status word) for a bad page.
__device__ __forceinline__ long long cache_row(const CacheParams& p, const int* table, int b,
                                               int kh, int pos) {
  const int pg = pos / p.ps;
  const int id = table[(long long)b * p.mp + pg];
  if (id < 0 || id >= p.pages) {
    atomicExch(p.status, SWIN_ERR_INVALID_ARG);
    return -1;
  }
  return ((long long)id * p.K + kh) * p.ps + (pos - pg * p.ps);
}

// ---- append ------------------------------------------------------------------------
// A block takes kAppend x 256 chunks of 16 bytes of one sequence's new rows, channels
// fastest, four of K and of V in flight per thread. Bound by HBM (every new row
// read once and written once): 157 MB in 27 us.
constexpr int kAppend = 4;
template <typename E>
__global__ void __launch_bounds__(256)
    append_kernel(const __grid_constant__ CacheParams p, int blocks) {
  constexpr int V = 16 / sizeof(E);
  const int b = blockIdx.x / blocks;   // `blocks` blocks per sequence
  const uint32_t cpr = p.hd / V, per_tok = p.K * cpr;
  int cnt = p.T;
  if (p.counts) {
    cnt = p.counts[b];
    cnt = cnt < 0 ? 0 : (cnt > p.T ? p.T : cnt);
  }
  const int first = cache_len(p, b) - cnt;
  const uint32_t x0 = (blockIdx.x - b * blocks) * (256 * kAppend) + threadIdx.x;
  uint4 k[kAppend], v[kAppend];
  long long dst[kAppend];
#pragma unroll
  for (int u = 0; u < kAppend; ++u) {
    const uint32_t x = x0 + u * 256;
    const int t = x / per_tok, y = x - t * per_tok;
    const int kh = y / cpr, c = (y - kh * cpr) * V;
    dst[u] = -1;
    if (t >= cnt) continue;
    if (first + t < 0) {
      atomicExch(p.status, SWIN_ERR_INVALID_ARG);
      continue;
    }
    const long long row = cache_row(p, p.table, b, kh, first + t);
    if (row < 0) continue;
    const long long src = ((long long)b * p.T + t) * p.ks + (long long)kh * p.hd + c;
    dst[u] = row * p.hd + c;
    k[u] = *reinterpret_cast<const uint4*>((const E*)p.k_new + src);
    v[u] = *reinterpret_cast<const uint4*>((const E*)p.v_new + src);
  }
#pragma unroll
  for (int u = 0; u < kAppend; ++u)
    if (dst[u] >= 0) {
      *reinterpret_cast<uint4*>((E*)p.kc + dst[u]) = k[u];
      *reinterpret_cast<uint4*>((E*)p.vc + dst[u]) = v[u];
    }
}

// ---- decode ------------------------------------------------------------------------
// The visible positions of a sequence are numbered 0 .. n - 1: the sinks, then
// the window (vis_pos). They are cut into units of `unit`; the units of all
// sequences, kv heads and chunks of query heads form one list, and block c of
// C takes units c T / C .. (c + 1) T / C of the T there are, whatever the mix
// of lengths: every block gets the same number of bytes to read, which is what
// bounds the kernel: 599 MB of 64 sequences in 101 us (5.9 TB/s), two of up to 65536
// tokens with their logits in 27 us. A block that has all units of a (sequence, kv head,
// chunk) writes its output; pieces go to the workspace and join_kernel adds
// them in order. All of this is computed on the device from the lengths, so a
// captured graph follows them.
struct DecodePlan {
  int C, heads, nchunk, hds;     // blocks, query heads of a chunk, chunks, row of partials
  int unit;                      // visible positions of a work unit
  float* part;                   // [C][2][heads][hds]: m, l (hds - 2, hds - 1) and O
  float* lse2;                   // [B][H] of finished heads, log2 units
  float* logits;                 // weights: [B][H][vis_max], log2 units
  long long vis_max;
  long long* prefix;             // [B + 1] units before each sequence; NULL: small batch
};

// a / b, in 32 bits where both fit (a 64-bit division is some hundred cycles).
__device__ __forceinline__ long long quot(long long a, long long b) {
  return ((a | b) >> 32) ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}

struct Vis {
  int n, len, first, shift;      // positions < first are themselves, others + shift
};
__device__ __forceinline__ Vis vis_of(const CacheParams& p, int b) {
  Vis v;
  v.len = cache_len(p, b);
  const long long cap = (long long)p.window + p.sinks;
  v.n = v.len < cap ? v.len : (int)cap;
  v.shift = v.len - v.n;
  v.first = v.shift > 0 ? p.sinks : v.len;
  return v;
}
__device__ __forceinline__ int vis_pos(const Vis& v, int u) {
  return u < v.first ? u : u + v.shift;
}
__device__ __forceinline__ int units_of(const CacheParams& p, int unit, int b) {
  return (vis_of(p, b).n + unit - 1) / unit;
}

// Total units per (kv head, chunk) over the batch and, of them, those before
// sequence `b_stop` (block-wide; THR threads; `sh` holds 2 THR / 32 values).
template <int THR>
__device__ __forceinline__ void batch_units(const CacheParams& p, int unit, int b_stop,
                                            long long* sh, long long& before, long long& total) {
  long long bef = 0, tot = 0;
  for (int b = threadIdx.x; b < p.B; b += THR) {
    const int u = units_of(p, unit, b);
    tot += u;
    if (b < b_stop) bef += u;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    bef += __shfl_xor_sync(0xffffffffu, bef, o);
    tot += __shfl_xor_sync(0xffffffffu, tot, o);
  }
  if ((threadIdx.x & 31) == 0) {
    sh[threadIdx.x / 32] = bef;
    sh[THR / 32 + threadIdx.x / 32] = tot;
  }
  __syncthreads();
  before = total = 0;
#pragma unroll
  for (int w = 0; w < THR / 32; ++w) {
    before += sh[w];
    total += sh[THR / 32 + w];
  }
  __syncthreads();
}

// Units before every sequence of a batch that is too large for each block to add up
// the lengths itself. One block; each thread a contiguous run, as in find_place.
constexpr int kScanThr = 1024, kScanBatch = 1024;   // batches above take this kernel
__global__ void __launch_bounds__(kScanThr)
    units_scan_kernel(const __grid_constant__ CacheParams p, int unit, long long* prefix) {
  __shared__ long long sh[32];
  const int per = (p.B + kScanThr - 1) / kScanThr;
  const int b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
  long long sum = 0;
  for (int b = b0; b < b1; ++b) sum += units_of(p, unit, b);
  long long inc = sum;
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += t;
  }
  if (lane == 31) sh[warp] = inc;
  __syncthreads();
  for (int w = 0; w < warp; ++w) inc += sh[w];
  long long at = inc - sum;
  for (int b = b0; b < b1; ++b) {
    prefix[b] = at;
    at += units_of(p, unit, b);
  }
  if (threadIdx.x == kScanThr - 1) prefix[p.B] = inc;
}

// The block's place in the list of units: total units of the batch (per kv head and
// chunk), and the sequence that holds unit `start / kcn` of block c's first unit
// with the units before it. One pass over the lengths: each thread a contiguous run
// of sequences, an exclusive scan over threads (`sh` holds 7 values).
struct Place {
  long long total, start, end, before;
  int b;
};
__device__ __forceinline__ Place find_place(const CacheParams& p, const DecodePlan& d, int unit,
                                            int kcn, long long* sh) {
  const int C = d.C;
  if (d.prefix) {   // by bisection: the last sequence with prefix <= target
    Place pl;
    pl.total = d.prefix[p.B] * kcn;
    pl.start = quot((long long)blockIdx.x * pl.total, C);
    pl.end = quot((long long)(blockIdx.x + 1) * pl.total, C);
    const long long target = quot(pl.start, kcn);
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int mid = lo + (hi - lo) / 2;
      if (d.prefix[mid] <= target) lo = mid;
      else hi = mid;
    }
    pl.b = lo;
    pl.before = d.prefix[lo];
    return pl;
  }
  const int per = (p.B + kDecThr - 1) / kDecThr;
  const int b0 = threadIdx.x * per, b1 = min(p.B, b0 + per);
  long long sum = 0;
  for (int b = b0; b < b1; ++b) sum += units_of(p, unit, b);
  long long inc = sum;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += t;
  }
  if (lane == 31) sh[threadIdx.x / 32] = inc;
  __syncthreads();
  Place pl;
  pl.total = 0;
#pragma unroll
  for (int w = 0; w < kDecThr / 32; ++w) {
    if (w < (int)threadIdx.x / 32) inc += sh[w];
    pl.total += sh[w];
  }
  pl.total *= kcn;
  pl.start = quot((long long)blockIdx.x * pl.total, C);
  pl.end = quot((long long)(blockIdx.x + 1) * pl.total, C);
  const long long target = quot(pl.start, kcn);
  long long before = inc - sum;
  if (pl.start < pl.end && target >= before && target < inc) {
    int b = b0;
    for (;;) {
      const int u = units_of(p, unit, b);
      if (target < before + u) break;
      before += u;
      ++b;
    }
    sh[5] = b;
    sh[6] = before;
  }
  __syncthreads();
  pl.b = (int)sh[5];
  pl.before = sh[6];
  return pl;
}

struct Segment {
  int b, kh, h0, hc;        // query heads h0 .. h0 + hc - 1
  int u0, u1;               // units
  Vis vis;
  bool writes_new;          // this block writes the new token's row (first chunk of heads)
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool ok) {
  const int n = ok ? 16 : 0;   // 0 source bytes: zero fill, the address is not read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ uint32_t movm_t(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Where a warp's lane stands for position u of the segment: its row in the
// cache, -1 (nothing) or -2 (the new token).
__device__ __forceinline__ long long lane_row(const CacheParams& p, const Segment& s, int u) {
  if (u >= s.vis.n) return -1;
  const int pos = vis_pos(s.vis, u);
  if (p.k_new && pos == s.vis.len - 1) return -2;
  return cache_row(p, p.table, s.b, s.kh, pos);
}

// bf16, head_dim 32, 64 or 128, 8 NT query heads of one kv head at a time. Each
// warp runs alone over tiles of TK positions through a ring of ST cp.async
// stages (16-byte chunks, swizzled against bank conflicts); two blocks per SM, so
// that one streams while the other ends a sequence. Logits transposed,
// S^T = K Q^T, and O^T = V^T P^T, on mma.sync: the key and channel sides have
// 16 rows to give and the query heads are the 8-wide side, so the eight heads
// or fewer of a group fill a tile; P^T moves from the one product to the other
// through movmatrix. Arithmetic is a few per cent of the warp's time: the
// cache is read once, and its bytes bound the kernel.
template <int HD, int NT, int ST, int TK>
struct MmaCore {
  static constexpr int kHeads = 8 * NT, kUnit = 4 * TK;  // TK positions per warp and tile
  static constexpr int kCpr = HD / 8;                    // 16-byte chunks of a row
  static constexpr int kTileBytes = TK * HD * 2;         // one of K, V
  static constexpr int kWarpBytes = ST * 2 * kTileBytes + ST * 4;
  static constexpr size_t kRing = 4 * (size_t)((kWarpBytes + 127) / 128 * 128);
  static constexpr size_t kMerge = 4 * kHeads * (HD + 2) * sizeof(float);
  static constexpr size_t kSmem = kRing > kMerge ? kRing : kMerge;

  __device__ static uint32_t at(int row, int chunk) {
    const int x = HD >= 64 ? (row & 7) : ((row >> 1) & 3);
    return row * (HD * 2) + ((chunk ^ x) << 4);
  }

  // Leaves m, l and O of this warp in `res` ([heads][HD + 2]) after a
  // block-wide barrier (the ring is reused).
  __device__ static void run(const CacheParams& p, const DecodePlan& d, const Segment& s,
                             unsigned char* smem, float* res_all) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    unsigned char* mine = smem + warp * (kRing / 4);
    const uint32_t base = ptx::smem_u32(mine);
    uint32_t* vmask = (uint32_t*)(mine + ST * 2 * kTileBytes);
    const __nv_bfloat16* kc = (const __nv_bfloat16*)p.kc;
    const __nv_bfloat16* vc = (const __nv_bfloat16*)p.vc;
    const long long new_at = (long long)s.b * p.ks + (long long)s.kh * HD;

    uint32_t qf[NT][HD / 16][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int h = nt * 8 + lane / 4;
      const __nv_bfloat16* q = (const __nv_bfloat16*)p.q + (long long)s.b * p.qs +
                               (long long)(s.h0 + h) * HD + (lane & 3) * 2;
#pragma unroll
      for (int ks = 0; ks < HD / 16; ++ks) {
        qf[nt][ks][0] = h < s.hc ? *(const uint32_t*)(q + ks * 16) : 0u;
        qf[nt][ks][1] = h < s.hc ? *(const uint32_t*)(q + ks * 16 + 8) : 0u;
      }
    }
    float o[HD / 16][NT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int ct = 0; ct < HD / 16; ++ct)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[ct][nt][e] = 0.f;
    }

    // tiles warp, warp + 4, ... of the segment's TK-position tiles
    const int t_end = min(s.u1 * 4, (s.vis.n + TK - 1) / TK);
    const int t0 = s.u0 * 4 + warp;
    const int cnt = t0 < t_end ? (t_end - t0 + 3) / 4 : 0;
    auto row_of = [&](int tile) {   // lane r < TK: position r of the tile
      return lane < TK ? lane_row(p, s, tile * TK + lane) : -1ll;
    };
    long long row_next = cnt > 0 ? row_of(t0) : -1;
    auto issue = [&](int x) {   // tile x of this warp into stage x % ST
      if (x < cnt) {
        const int st = x % ST;
        const long long row = row_next;
        if (x + 1 < cnt) row_next = row_of(t0 + (x + 1) * 4);
        const uint32_t ok = __ballot_sync(0xffffffffu, row != -1);
        if (lane == 0) vmask[st] = ok;
        const uint32_t kb = base + st * 2 * kTileBytes, vb = kb + kTileBytes;
        constexpr int RPI = 32 / kCpr;   // rows per instruction
#pragma unroll
        for (int i = 0; i < TK / RPI; ++i) {
          const int r = i * RPI + lane / kCpr, c = lane % kCpr;
          const long long rr = __shfl_sync(0xffffffffu, row, r);
          const __nv_bfloat16* ks = kc + (rr >= 0 ? rr : 0) * HD + c * 8;
          const __nv_bfloat16* vs = vc + (rr >= 0 ? rr : 0) * HD + c * 8;
          if (rr == -2) {
            ks = (const __nv_bfloat16*)p.k_new + new_at + c * 8;
            vs = (const __nv_bfloat16*)p.v_new + new_at + c * 8;
          }
          cp_async16(kb + at(r, c), ks, rr != -1);
          cp_async16(vb + at(r, c), vs, rr != -1);
        }
      }
      cp_commit();
    };
#pragma unroll
    for (int x = 0; x < ST - 1; ++x) issue(x);
#pragma unroll 1
    for (int x = 0; x < cnt; ++x) {
      cp_wait<ST - 2>();
      __syncwarp();
      const int st = x % ST;
      const uint32_t kb = base + st * 2 * kTileBytes, vb = kb + kTileBytes;
      const uint32_t ok = vmask[st];
      float sacc[TK / 16][NT][4];
#pragma unroll
      for (int mt = 0; mt < TK / 16; ++mt) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) sacc[mt][nt][e] = 0.f;
#pragma unroll
        for (int ks = 0; ks < HD / 16; ++ks) {
          uint32_t a[4];
          ldm4(a, kb + at(mt * 16 + (lane & 15), 2 * ks + (lane >> 4)));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(sacc[mt][nt], a, qf[nt][ks][0], qf[nt][ks][1]);
        }
      }
      uint32_t pf[TK / 16][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int mt = 0; mt < TK / 16; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = mt * 16 + lane / 4 + (e >> 1) * 8;
            const float v = (ok >> key) & 1 ? sacc[mt][nt][e] * p.scale_log2 : -INFINITY;
            sacc[mt][nt][e] = v;
            mx[e & 1] = fmaxf(mx[e & 1], v);
          }
        if (d.logits) {
          const int u = (t0 + x * 4) * TK;
#pragma unroll
          for (int mt = 0; mt < TK / 16; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = mt * 16 + lane / 4 + (e >> 1) * 8;
              const int h = nt * 8 + (lane & 3) * 2 + (e & 1);
              if (h < s.hc && u + key < s.vis.n)
                d.logits[((long long)s.b * p.H + s.h0 + h) * d.vis_max + u + key] = sacc[mt][nt][e];
            }
        }
        float f[2], mu[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], w));
          mx[e] = fmaxf(mx[e], m[nt][e]);
          mu[e] = mx[e] == -INFINITY ? 0.f : mx[e];
          f[e] = ptx::ex2(m[nt][e] - mu[e]);
          m[nt][e] = mx[e];
          l[nt][e] *= f[e];
        }
        if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
          for (int ct = 0; ct < HD / 16; ++ct)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[ct][nt][e] *= f[e & 1];
        }
#pragma unroll
        for (int mt = 0; mt < TK / 16; ++mt) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            w[e] = ptx::ex2(sacc[mt][nt][e] - mu[e & 1]);
            l[nt][e & 1] += w[e];
          }
          // P in bf16 (off by 2^-8 at most, errors of many keys average out);
          // the sum takes the unrounded values
          pf[mt][nt][0] = movm_t(ptx::pack_bf16(w[0], w[1]));
          pf[mt][nt][1] = movm_t(ptx::pack_bf16(w[2], w[3]));
        }
      }
#pragma unroll
      for (int mt = 0; mt < TK / 16; ++mt)
#pragma unroll
        for (int ct = 0; ct < HD / 16; ++ct) {
          uint32_t a[4];
          ldm4t(a, vb + at(mt * 16 + (lane & 7) + (lane >> 4) * 8, 2 * ct + ((lane >> 3) & 1)));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(o[ct][nt], a, pf[mt][nt][0], pf[mt][nt][1]);
        }
      __syncwarp();   // the stage is read: the next issue may overwrite it
      issue(x + ST - 1);
    }
    cp_wait<0>();
    __syncthreads();
    float* res = res_all + warp * kHeads * (HD + 2);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[nt][e];
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
        float* r = res + (nt * 8 + (lane & 3) * 2 + e) * (HD + 2);
        if (lane < 4) {
          r[HD] = m[nt][e];
          r[HD + 1] = sum;
        }
#pragma unroll
        for (int ct = 0; ct < HD / 16; ++ct) {
          r[ct * 16 + lane / 4] = o[ct][nt][e];
          r[ct * 16 + lane / 4 + 8] = o[ct][nt][e + 2];
        }
      }
  }
};

// Any head size and type: lanes across the channels (HT per lane), R positions'
// rows in flight, up to four query heads. A unit is small (R positions per warp),
// so that short caches use many SMs. For fp32 its loads keep HBM busy; for narrow
// bf16 rows with many heads the dot products' shuffles bound it.
template <typename E, int HT>
struct LaneCore {
  static constexpr int R = HT <= 2 ? 8 : 4;
  static constexpr int kHeads = 4, kUnit = 4 * R;   // (decode_shape has the same)
  static constexpr size_t kSmem = 4 * kHeads * (32 * HT + 2) * sizeof(float);

  __device__ static void run(const CacheParams& p, const DecodePlan& d, const Segment& s,
                             unsigned char*, float* res_all) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const long long new_at = (long long)s.b * p.ks + (long long)s.kh * p.hd;
    float q[kHeads][HT], o[kHeads][HT], m[kHeads], l[kHeads];
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      m[h] = -INFINITY;
      l[h] = 0.f;
#pragma unroll
      for (int t = 0; t < HT; ++t) {
        o[h][t] = 0.f;
        q[h][t] = h < s.hc && lane + 32 * t < p.hd
                      ? seq_ld((const E*)p.q + (long long)s.b * p.qs +
                               (long long)(s.h0 + h) * p.hd + lane + 32 * t) * p.scale_log2
                      : 0.f;
      }
    }
    // runs of R positions: warp, warp + 4, ... of the segment's
    const int run_end = min(s.u1 * 4, (s.vis.n + R - 1) / R);
    int run = s.u0 * 4 + warp;
    auto row_at = [&](int x) {   // lane r < R: position r of run x
      return lane < R && x < run_end ? lane_row(p, s, x * R + lane) : -1ll;
    };
    long long row_next = row_at(run);
#pragma unroll 1
    for (; run < run_end; run += 4) {
      const long long row = row_next;
      float k[R][HT], v[R][HT];
      bool ok[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const long long rr = __shfl_sync(0xffffffffu, row, r);
        ok[r] = rr != -1;   // positions behind the last are -1 too
        const E* ks = rr == -2 ? (const E*)p.k_new + new_at : (const E*)p.kc + rr * p.hd;
        const E* vs = rr == -2 ? (const E*)p.v_new + new_at : (const E*)p.vc + rr * p.hd;
#pragma unroll
        for (int t = 0; t < HT; ++t) {
          const bool in = ok[r] && lane + 32 * t < p.hd;
          k[r][t] = in ? seq_ld(ks + lane + 32 * t) : 0.f;
          v[r][t] = in ? seq_ld(vs + lane + 32 * t) : 0.f;
        }
      }
      row_next = row_at(run + 4);
#pragma unroll
      for (int h = 0; h < kHeads; ++h) {
        if (h >= s.hc) break;
        float a[R], mx = m[h];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          a[r] = 0.f;
#pragma unroll
          for (int t = 0; t < HT; ++t) a[r] = fmaf(q[h][t], k[r][t], a[r]);
        }
#pragma unroll
        for (int w = 16; w > 0; w >>= 1)
#pragma unroll
          for (int r = 0; r < R; ++r) a[r] += __shfl_xor_sync(0xffffffffu, a[r], w);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          if (!ok[r]) a[r] = -INFINITY;
          mx = fmaxf(mx, a[r]);
        }
        if (d.logits && lane < R && run * R + lane < s.vis.n) {
          float x = a[0];
#pragma unroll
          for (int r = 1; r < R; ++r)
            if (lane == r) x = a[r];
          d.logits[((long long)s.b * p.H + s.h0 + h) * d.vis_max + run * R + lane] = x;
        }
        const float mu = mx == -INFINITY ? 0.f : mx;
        const float f = exp2f(m[h] - mu);
        m[h] = mx;
        l[h] *= f;
#pragma unroll
        for (int t = 0; t < HT; ++t) o[h][t] *= f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float w = exp2f(a[r] - mu);
          l[h] += w;
#pragma unroll
          for (int t = 0; t < HT; ++t) o[h][t] = fmaf(w, v[r][t], o[h][t]);
        }
      }
    }
    float* res = res_all + warp * kHeads * (p.hd + 2);
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      float* r = res + h * (p.hd + 2);
#pragma unroll
      for (int t = 0; t < HT; ++t)
        if (lane + 32 * t < p.hd) r[lane + 32 * t] = o[h][t];
      if (lane == 0) {
        r[p.hd] = m[h];
        r[p.hd + 1] = l[h];
      }
    }
  }
};

// l = 0 only where no position counted (an empty sequence, bad pages).
__device__ __forceinline__ float lse2_of(float m, float l) {
  return l == 0.f ? -INFINITY : m + log2f(l);
}

template <typename E, class Core>
__global__ void __launch_bounds__(kDecThr)
    decode_kernel(const __grid_constant__ CacheParams p, const __grid_constant__ DecodePlan d) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ long long sh[7];
  __shared__ float fac[4][Core::kHeads], sum_sh[Core::kHeads];
  float* res = (float*)smem;
  constexpr int kUnit = Core::kUnit;
  ptx::grid_dep_launch();   // join_kernel may start (and wait)
  const int kcn = p.K * d.nchunk, hw = p.hd + 2;
  const Place pl = find_place(p, d, kUnit, kcn, sh);
  long long cur = pl.start, before = pl.before;
  const long long start = pl.start, end = pl.end;
  int b = pl.b;
  while (cur < end) {
    Segment s;
    s.b = b;
    s.vis = vis_of(p, b);
    const int U = (s.vis.n + kUnit - 1) / kUnit;
    const long long rel = cur - before * kcn;
    if (U == 0 || rel >= (long long)U * kcn) {   // next sequence
      before += U;
      ++b;
      continue;
    }
    const int kc = (int)quot(rel, U);
    s.kh = kc / d.nchunk;
    const int chunk = kc - s.kh * d.nchunk;
    s.h0 = s.kh * p.G + chunk * d.heads;
    s.hc = min(d.heads, p.G - chunk * d.heads);
    s.u0 = (int)(rel - (long long)kc * U);
    s.u1 = (int)min((long long)U, s.u0 + (end - cur));
    Core::run(p, d, s, smem, res);
    __syncthreads();
    // the four warps' parts, in order
    const bool whole = s.u0 == 0 && s.u1 == U;
    const int slot = cur == start ? 0 : 1;
    float* part = d.part + ((long long)blockIdx.x * 2 + slot) * d.heads * d.hds;
    if ((int)threadIdx.x < s.hc) {
      const int h = threadIdx.x;
      float m[4], M = -INFINITY, L = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        m[w] = res[(w * Core::kHeads + h) * hw + p.hd];
        M = fmaxf(M, m[w]);
      }
      const float mu = M == -INFINITY ? 0.f : M;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        fac[w][h] = exp2f(m[w] - mu);
        L = fmaf(res[(w * Core::kHeads + h) * hw + p.hd + 1], fac[w][h], L);
      }
      sum_sh[h] = whole ? (L == 0.f ? 0.f : 1.f / L) : 1.f;
      if (whole) {
        const float z = lse2_of(M, L);
        if (p.lse) p.lse[(long long)s.b * p.H + s.h0 + h] = z * kLn2;
        d.lse2[(long long)s.b * p.H + s.h0 + h] = z;
      } else {
        part[h * d.hds + p.hd] = M;
        part[h * d.hds + p.hd + 1] = L;
      }
    }
    __syncthreads();
    E* out = (E*)p.out + ((long long)s.b * p.H + s.h0) * p.hd;
    for (int x = threadIdx.x; x < s.hc * p.hd; x += kDecThr) {
      const int h = x / p.hd, c = x - h * p.hd;
      float O = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) O = fmaf(res[(w * Core::kHeads + h) * hw + c], fac[w][h], O);
      if (whole) seq_st(out + x, O * sum_sh[h]);
      else part[h * d.hds + c] = O;
    }
    // the new token's row: its position is the last of the last unit
    if (p.k_new && chunk == 0 && s.u1 == U) {
      const long long row = cache_row(p, p.table, s.b, s.kh, s.vis.len - 1);
      const long long at = (long long)s.b * p.ks + (long long)s.kh * p.hd;
      if (row >= 0)
        for (int c = threadIdx.x; c < p.hd; c += kDecThr) {
          ((E*)p.kc)[row * p.hd + c] = ((const E*)p.k_new)[at + c];
          ((E*)p.vc)[row * p.hd + c] = ((const E*)p.v_new)[at + c];
        }
    }
    cur += s.u1 - s.u0;
    __syncthreads();
  }
}

// Joins the pieces of the heads of (b, kh) that several blocks hold, writes
// empty sequences, and adds the step's weights: blockIdx.y = piece of
// kJoinSpan positions and of the outputs. Waits for decode_kernel, whose
// programmatic dependent it is. Per chunk of query heads the pieces' slots are
// listed once, a warp per head finds the common maximum and sum, and a thread
// per channel adds the pieces in order. Bound by the latency of these steps: 12 us
// for the 64 sequences above, 14 with weights for the two long ones (profiled, alone).
constexpr int kJoinSpan = 1024, kJoinThr = 512;
template <typename E>
__global__ void __launch_bounds__(kJoinThr)
    join_kernel(const __grid_constant__ CacheParams p, const __grid_constant__ DecodePlan d) {
  extern __shared__ float join_sh[];
  float* lse_sh = join_sh;                      // [G]
  float* inv_sh = lse_sh + p.G;                 // [heads]
  int* slots = (int*)(inv_sh + d.heads);        // [C]
  float* fac = (float*)(slots + d.C);           // [heads][C]: maxima, then factors
  float* sums = fac + d.heads * d.C;            // [heads][C]
  __shared__ long long sh[2 * kJoinThr / 32];
  const int b = blockIdx.x / p.K, kh = blockIdx.x - b * p.K;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  long long before, total;
  if (d.prefix) {
    before = d.prefix[b];
    total = d.prefix[p.B];
  } else {
    batch_units<kJoinThr>(p, d.unit, b, sh, before, total);
  }
  const int kcn = p.K * d.nchunk;
  total *= kcn;
  const Vis vis = vis_of(p, b);
  const int U = (vis.n + d.unit - 1) / d.unit;
  const long long bh0 = (long long)b * p.H + kh * p.G;
  ptx::grid_dep_wait();
  if (U == 0 && blockIdx.y == 0) {
    for (int x = threadIdx.x; x < p.G * p.hd; x += kJoinThr)
      seq_st((E*)p.out + bh0 * p.hd + x, 0.f);
    for (int h = threadIdx.x; h < p.G && p.lse; h += kJoinThr) p.lse[bh0 + h] = -INFINITY;
  }
  for (int chunk = 0; chunk < d.nchunk && U > 0; ++chunk) {
    const long long g0 = before * kcn + ((long long)kh * d.nchunk + chunk) * U, g1 = g0 + U;
    const int c0 = (int)quot((g0 + 1) * d.C - 1, total), c1 = (int)quot(g1 * d.C - 1, total);
    const int h0 = chunk * d.heads, hc = min(d.heads, p.G - h0);   // within the group
    if (c0 == c1) {
      if (p.w_out)
        for (int h = threadIdx.x; h < hc; h += kJoinThr) lse_sh[h0 + h] = d.lse2[bh0 + h0 + h];
      continue;
    }
    const int ns = c1 - c0 + 1;
    __syncthreads();
    for (int k = threadIdx.x; k < ns; k += kJoinThr) {
      const int c = c0 + k;
      const long long s0 = quot(c * total, d.C), s1 = quot((c + 1) * total, d.C);
      // a block without units has none of this; its first segment is in slot 0
      slots[k] = max(g0, s0) < min(g1, s1) ? 2 * c + (s0 >= g0 ? 0 : 1) : -1;
    }
    __syncthreads();
    auto piece = [&](int k, int h) {   // (no slot: some slot's, not used)
      return d.part + ((long long)max(slots[k], 0) * d.heads + h) * d.hds;
    };
    for (int h = warp; h < hc; h += kJoinThr / 32) {
      float M = -INFINITY, L = 0.f;
      for (int k = lane; k < ns; k += 32) {
        const float m = piece(k, h)[p.hd], l = piece(k, h)[p.hd + 1];
        fac[h * d.C + k] = slots[k] >= 0 ? m : -INFINITY;
        sums[h * d.C + k] = slots[k] >= 0 ? l : 0.f;
        M = fmaxf(M, fac[h * d.C + k]);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      const float mu = M == -INFINITY ? 0.f : M;
      for (int k = lane; k < ns; k += 32) {
        const float f = exp2f(fac[h * d.C + k] - mu);
        fac[h * d.C + k] = f;
        L = fmaf(sums[h * d.C + k], f, L);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
      if (lane == 0) {
        const float z = lse2_of(M, L);
        lse_sh[h0 + h] = z;
        inv_sh[h] = L == 0.f ? 0.f : 1.f / L;
        if (p.lse && blockIdx.y == 0) p.lse[bh0 + h0 + h] = z * kLn2;
      }
    }
    __syncthreads();
    // `lanes` neighbouring threads per output, each a part of the pieces (more where
    // there are more threads than outputs)
    const int all = hc * p.hd, threads = kJoinThr * gridDim.y;
    int lanes = 1;
    while (lanes < 32 && 2 * lanes * all <= threads) lanes *= 2;
    const int sub = threadIdx.x & (lanes - 1);
    for (int x0 = blockIdx.y * kJoinThr; x0 < all * lanes; x0 += threads) {
      const int x = (x0 + (int)threadIdx.x) / lanes;
      const int h = x < all ? x / p.hd : 0, c = x < all ? x - h * p.hd : 0;
      float O = 0.f;
#pragma unroll 8
      for (int k = sub; k < ns; k += lanes) {
        const float o = piece(k, h)[c];
        O = fmaf(slots[k] >= 0 ? o : 0.f, fac[h * d.C + k], O);
      }
      for (int o = lanes / 2; o > 0; o >>= 1) O += __shfl_xor_sync(0xffffffffu, O, o);
      if (x < all && sub == 0) seq_st((E*)p.out + (bh0 + h0) * p.hd + x, O * inv_sh[h]);
    }
  }
  if (!p.w_out) return;
  __syncthreads();
  const int p1 = (int)min((long long)vis.len, ((long long)blockIdx.y + 1) * kJoinSpan);
  const long long row = ((long long)b * p.K + kh) * p.max_len;
  for (int pos = blockIdx.y * kJoinSpan + threadIdx.x; pos < p1; pos += kJoinThr) {
    float w = p.w[row + pos];
    if (pos < vis.first || pos >= vis.first + vis.shift) {
      const int u = pos < vis.first ? pos : pos - vis.shift;
      const float* x = d.logits + bh0 * d.vis_max + u;
      float sum = 0.f;
#pragma unroll 8
      for (int h = 0; h < p.G; ++h) {
        const float a = x[h * d.vis_max];   // -inf: a bad page's position
        sum += a == -INFINITY ? 0.f : exp2f(a - lse_sh[h]);
      }
      w += sum;
    }
    p.w_out[row + pos] = w;
  }
}

// ---- evict -------------------------------------------------------------------------
// Order of weights as unsigned numbers, 1 .. 0xff800000: NaN lowest, then by value,
// -0 = +0. 0 stands for "no position", ~0 for one that always stays.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 1u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr int kSelThr = 1024, kSelRound = 4 * kSelThr;   // four positions a thread and round

// Weights of positions x .. x + 3 (zeros at and beyond n), in one load if rows start
// on 16 bytes.
__device__ __forceinline__ void load_weights(const float* w, int x, int n, bool wide,
                                             uint32_t (&v)[4]) {
  v[0] = v[1] = v[2] = v[3] = 0u;
  if (wide && x + 3 < n) {
    asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "l"(w + x));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (x + e < n) asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(v[e]) : "l"(w + x + e));
  }
}

struct SelectShared {
  alignas(16) uint32_t hist[2048 * 4];   // four counts of each bin; then of each round and warp
  uint32_t sums[3][1024];                // a cluster: this block's counts of two bins, by pass
  uint32_t bin, need, total, warp_sum[32];
};

// The blocks of a cluster: all have come here, and see what each wrote to its shared
// memory; a word of block `rank`.
__device__ __forceinline__ void team_sync() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t team_read(const uint32_t* at, int rank) {
  uint32_t a, v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(ptx::smem_u32(at)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// One digit of the threshold from the histograms (2048 bins, two a thread, from the
// top): the bin that holds the need-th largest key and how many of it are needed.
// The same in every block of a cluster.
template <int C>
__device__ __forceinline__ void pick_bin(SelectShared& sh, int pass, uint32_t need) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, top = 2047 - 2 * threadIdx.x;
  __syncthreads();
  const uint4 h = *reinterpret_cast<const uint4*>(&sh.hist[top * 4]);
  const uint4 g = *reinterpret_cast<const uint4*>(&sh.hist[top * 4 - 4]);
  uint32_t c0 = (h.x + h.y) + (h.z + h.w), c1 = (g.x + g.y) + (g.z + g.w);   // bins top, top - 1
  if constexpr (C > 1) {   // at most 32768 each
    sh.sums[pass][threadIdx.x] = c0 | c1 << 16;
    team_sync();
    uint32_t t[C];
#pragma unroll
    for (int v = 0; v < C; ++v) t[v] = team_read(&sh.sums[pass][threadIdx.x], v);
    c0 = c1 = 0;
#pragma unroll
    for (int v = 0; v < C; ++v) {
      c0 += t[v] & 0xffffu;
      c1 += t[v] >> 16;
    }
  }
  const uint32_t sum = c0 + c1;
  uint32_t inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t t = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += t;
  }
  if (lane == 31) sh.warp_sum[warp] = inc;
  __syncthreads();
  uint32_t t = lane < warp ? sh.warp_sum[lane] : 0u;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  const uint32_t before = t + inc - sum;
  if (before < need && need <= before + sum) {
    const bool first = need <= before + c0;
    sh.bin = first ? top : top - 1;
    sh.need = first ? need - before : need - before - c0;
  }
  __syncthreads();
}

// Which positions of (b, kv head) stay: a cluster of C blocks each. The always-kept
// positions have the largest key, so what stays is the `budget` largest keys of the
// sequence, ties at the threshold in order of position. The threshold is found
// digit by digit (11, 11 and 10 bits; wide digits, since weights share few
// exponents and shared-memory atomics on one bin queue up). A kept
// position's place in the output is the number of larger keys before it plus
// the ties before it that stay. With R > 0 a thread holds R groups of four
// positions (4096 apart) in registers and one scan over the counts of every warp
// and round gives all places (n <= 4096 R C); R = 0 (one block) reads the weights
// again in every pass and takes a contiguous run of positions per warp. Bound by
// the passes' instructions: 25 us for 64 x 32768 weights (29 with a position a
// thread at a time and the loads that takes).
template <int R, int C>
__global__ void __cluster_dims__(C, 1, 1) __launch_bounds__(kSelThr)
    evict_select_kernel(const __grid_constant__ CacheParams p, int* kept) {
  static_assert(C == 1 || R > 0, "a cluster holds its positions in registers");
  __shared__ SelectShared sh;
  ptx::grid_dep_launch();
  const int bk = blockIdx.x / C, rank = blockIdx.x - bk * C, b = bk / p.K, kh = bk - b * p.K;
  const int n = cache_len(p, b), keep = min(n, p.budget);
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const float* w = p.w + (long long)bk * p.max_len;
  float* w_out = p.w_out + (long long)bk * p.max_len;
  int* out = kept + (long long)bk * p.budget;
  if (kh == 0 && rank == 0 && threadIdx.x == 0) p.new_len[b] = keep;
  const int me = rank * kSelThr + threadIdx.x;
  if (n <= p.budget) {   // (every block of the cluster)
    for (int x = me; x < n; x += C * kSelThr) {
      out[x] = x;
      w_out[x] = w[x];
    }
    for (int x = n + me; x < p.budget; x += C * kSelThr) out[x] = -1;
    for (int x = n + me; x < p.max_len; x += C * kSelThr) w_out[x] = 0.f;
    return;
  }
  const int lo = p.sinks, hi = n - p.recent;       // positions outside stay
  const bool wide = (p.max_len & 3) == 0;
  auto key_of = [&](int x, uint32_t raw) {
    return x >= n ? 0u : (x < lo || x >= hi ? 0xffffffffu : weight_key(__uint_as_float(raw)));
  };
  // rounds of a block, and this thread's first position
  const int rounds = ((n + C - 1) / C + kSelRound - 1) / kSelRound;
  const int x0 = rank * rounds * kSelRound + 4 * threadIdx.x;
  uint32_t keys[R > 0 ? R : 1][4];   // weights as they come, then keys
  if constexpr (R > 0) {
#pragma unroll
    for (int r = 0; r < R; ++r) load_weights(w, x0 + r * kSelRound, r < rounds ? n : 0, wide, keys[r]);
    asm volatile("" ::: "memory");   // all loads before the first use of one
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        keys[r][e] = r < rounds ? key_of(x0 + r * kSelRound + e, keys[r][e]) : 0u;
  }
  for (int x = keep + me; x < p.max_len; x += C * kSelThr) w_out[x] = 0.f;
  uint32_t prefix = 0, need = (uint32_t)p.budget;
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    constexpr int kShift[3] = {21, 10, 0};
    uint4* z = reinterpret_cast<uint4*>(sh.hist);
    z[threadIdx.x] = z[kSelThr + threadIdx.x] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    uint32_t* mine = sh.hist + (lane & 3);   // lanes of a warp that share a bin queue up
    // keys that start with the digits so far: from `first`, this many of them
    const uint32_t first = pass == 0 ? 1u : prefix << (pass == 1 ? 21 : 10);
    const uint32_t many = pass == 0 ? 0xffffffffu : (pass == 1 ? 1u << 21 : 1u << 10);
    auto count = [&](uint32_t k) {
      if (k - first < many) atomicAdd(&mine[(k >> kShift[pass] & (pass == 2 ? 1023u : 2047u)) * 4], 1u);
    };
    if constexpr (R > 0) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (r >= rounds) break;
#pragma unroll
        for (int e = 0; e < 4; ++e) count(keys[r][e]);
      }
    } else {
      for (int x = 4 * threadIdx.x; x < n; x += kSelRound) {
        uint32_t v[4];
        load_weights(w, x, n, wide, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) count(key_of(x + e, v[e]));
      }
    }
    pick_bin<C>(sh, pass, need);
    prefix = pass == 0 ? sh.bin : (prefix << (pass == 1 ? 11 : 10)) | sh.bin;
    need = sh.need;
    __syncthreads();
  }
  const uint32_t thr = prefix, lt = (1u << lane) - 1u;
  // Four positions of a thread from x on, behind gt larger keys and eq ties.
  auto emit = [&](int x, const uint32_t (&k)[4], const uint32_t (&weight)[4], uint32_t gt,
                  uint32_t eq) {
    uint32_t g[4], q[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      g[e] = __ballot_sync(0xffffffffu, k[e] > thr);
      q[e] = __ballot_sync(0xffffffffu, k[e] == thr);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      gt += __popc(g[e] & lt);
      eq += __popc(q[e] & lt);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool larger = k[e] > thr, tie = k[e] == thr;
      if (larger || (tie && eq < need)) {
        const uint32_t at = gt + min(eq, need);
        out[at] = x + e;
        w_out[at] = __uint_as_float(weight[e]);
      }
      gt += larger;
      eq += tie;
    }
  };
  if constexpr (R > 0) {
    // larger keys and ties (high half) of every round and warp, in position order
#pragma unroll
    for (int r = 0; r < R; ++r) {
      uint32_t c = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        c += __popc(__ballot_sync(0xffffffffu, keys[r][e] > thr)) |
             __popc(__ballot_sync(0xffffffffu, keys[r][e] == thr)) << 16;
      if (lane == 0) sh.hist[r * 32 + warp] = c;
    }
    __syncthreads();
    const uint32_t c = (int)threadIdx.x < R * 32 ? sh.hist[threadIdx.x] : 0u;
    uint32_t inc = c;   // both halves at once: each total is at most 32768
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t t = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += t;
    }
    if (lane == 31) sh.warp_sum[warp] = inc;
    __syncthreads();
    uint32_t sum = 0;
#pragma unroll
    for (int v = 0; v < R; ++v) sum += v < warp ? sh.warp_sum[v] : 0u;
    if ((int)threadIdx.x < R * 32) sh.hist[threadIdx.x] = sum + inc - c;
    if ((int)threadIdx.x == R * 32 - 1) sh.total = sum + inc;
    uint32_t gt0 = 0, eq0 = 0;   // of the blocks before
    if constexpr (C > 1) {
      team_sync();
      uint32_t t[C];
#pragma unroll
      for (int v = 0; v < C; ++v) t[v] = team_read(&sh.total, v);
#pragma unroll
      for (int v = 0; v < C; ++v)
        if (v < rank) {
          gt0 += t[v] & 0xffffu;
          eq0 += t[v] >> 16;
        }
    } else {
      __syncthreads();
    }
    // (the weights once more, of threads that keep any: a key does not give back NaN
    // and -0)
#pragma unroll
    for (int r0 = 0; r0 < R; r0 += 2) {
      if (r0 >= rounds) break;
      uint32_t raw[2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (r0 + u >= R) break;
        const uint32_t* k = keys[r0 + u];
        const bool any = max(max(k[0], k[1]), max(k[2], k[3])) >= thr;
        load_weights(w, x0 + (r0 + u) * kSelRound, any ? n : 0, wide, raw[u]);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (r0 + u >= R) break;
        const uint32_t before = sh.hist[(r0 + u) * 32 + warp];
        emit(x0 + (r0 + u) * kSelRound, keys[r0 + u], raw[u], gt0 + (before & 0xffffu),
             eq0 + (before >> 16));
      }
    }
    if constexpr (C > 1) team_sync();   // no block leaves before its total is read
  } else {
    const int per = ((n + 31) / 32 + 127) / 128 * 128;   // positions of a warp
    const int w0 = (int)min((long long)n, (long long)warp * per), w1 = min(n, w0 + per);
    uint32_t gt = 0, eq = 0;
    for (int x = w0 + 4 * lane; x < w1; x += 128) {
      uint32_t v[4];
      load_weights(w, x, w1, wide, v);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t k = x + e < w1 ? key_of(x + e, v[e]) : 0u;
        gt += k > thr;
        eq += k == thr;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      gt += __shfl_xor_sync(0xffffffffu, gt, o);
      eq += __shfl_xor_sync(0xffffffffu, eq, o);
    }
    if (lane == 0) {
      sh.hist[warp] = gt;
      sh.hist[32 + warp] = eq;
    }
    __syncthreads();
    gt = eq = 0;
    for (int v = 0; v < warp; ++v) {
      gt += sh.hist[v];
      eq += sh.hist[32 + v];
    }
    for (int x = w0 + 4 * lane; x - 4 * lane < w1; x += 128) {
      uint32_t v[4], k[4];
      load_weights(w, x, w1, wide, v);
      uint32_t c = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) k[e] = x + e < w1 ? key_of(x + e, v[e]) : 0u;
      emit(x, k, v, gt, eq);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        c += __popc(__ballot_sync(0xffffffffu, k[e] > thr)) |
             __popc(__ballot_sync(0xffffffffu, k[e] == thr)) << 16;
      gt += c & 0xffffu;
      eq += c >> 16;
    }
  }
}

// The kept rows to their new pages, two chunks of 16 bytes of a K and a V row per
// thread. Bound by HBM: budget rows read once and written once, 268 MB in 44 us.
constexpr int kCopy = 2;
template <typename E>
__global__ void __launch_bounds__(256)
    evict_copy_kernel(const __grid_constant__ CacheParams p, const int* kept, int blocks) {
  constexpr int V = 16 / sizeof(E);
  const int cpr = p.hd / V;
  const int bk = blockIdx.x / blocks;   // `blocks` blocks per (b, kh)
  const int b = bk / p.K, kh = bk - b * p.K;
  const int x0 = (blockIdx.x - bk * blocks) * (256 * kCopy) + threadIdx.x;
  const int keep = min(cache_len(p, b), p.budget);
  uint4 k[kCopy], v[kCopy];
  long long dst[kCopy];
  ptx::grid_dep_wait();
#pragma unroll
  for (int u = 0; u < kCopy; ++u) {
    const int x = x0 + u * 256, r = x / cpr, c = (x - r * cpr) * V;
    dst[u] = -1;
    if (r >= keep) continue;
    const long long src = cache_row(p, p.table, b, kh, kept[(long long)bk * p.budget + r]);
    const long long to = cache_row(p, p.dst_table, b, kh, r);
    if (src < 0 || to < 0) continue;
    dst[u] = to * p.hd + c;
    k[u] = *reinterpret_cast<const uint4*>((const E*)p.kc + src * p.hd + c);
    v[u] = *reinterpret_cast<const uint4*>((const E*)p.vc + src * p.hd + c);
  }
#pragma unroll
  for (int u = 0; u < kCopy; ++u)
    if (dst[u] >= 0) {
      *reinterpret_cast<uint4*>((E*)p.kc + dst[u]) = k[u];
      *reinterpret_cast<uint4*>((E*)p.vc + dst[u]) = v[u];
    }
}

// ---- host --------------------------------------------------------------------------
struct DecodeShape {
  bool mma;
  int heads, nchunk, blocks, unit;
};
DecodeShape decode_shape(const CacheParams& p, int dtype) {
  DecodeShape s;
  s.mma = dtype == SWIN_DTYPE_BF16 && (p.hd == 32 || p.hd == 64 || p.hd == 128);
  s.heads = s.mma ? (p.G <= 8 ? 8 : 16) : 4;
  s.nchunk = (p.G + s.heads - 1) / s.heads;
  s.unit = s.mma ? (p.hd == 128 ? 64 : 128) : (p.hd <= 64 ? 32 : 16);   // each Core's kUnit
  // blocks that fit the card at once (shared memory of the ring; registers)
  const long long resident = (long long)kSeqSms * (s.mma ? 2 : 4);
  const long long cap = (long long)p.window + p.sinks;
  const long long vis = p.max_len < cap ? p.max_len : cap;
  const long long most = (long long)p.B * p.K * s.nchunk * ((vis + s.unit - 1) / s.unit);
  s.blocks = (int)(most < resident ? most : resident);
  return s;
}
long long vis_max(const CacheParams& p) {
  const long long cap = (long long)p.window + p.sinks;
  return p.max_len < cap ? p.max_len : cap;
}
size_t part_bytes(const CacheParams& p, const DecodeShape& s) {
  return align256((size_t)s.blocks * 2 * s.heads * (p.hd + 2) * 4);
}
size_t lse_bytes(const CacheParams& p) { return align256((size_t)p.B * p.H * 4); }
size_t prefix_bytes(const CacheParams& p) {
  return p.B > kScanBatch ? align256(((size_t)p.B + 1) * 8) : 0;
}

template <typename E, class Core>
cudaError_t decode_go(const CacheParams& p, const DecodePlan& d, cudaStream_t st) {
  cudaError_t e = allow_smem<decode_kernel<E, Core>>(Core::kSmem);
  if (e != cudaSuccess) return e;
  decode_kernel<E, Core><<<d.C, kDecThr, Core::kSmem, st>>>(p, d);
  note_launch();
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // a thread per output at least, eight where (b, kh) alone leave SMs idle
  const long long outs = ((long long)d.heads * p.hd + kJoinThr - 1) / kJoinThr;
  const long long spans = p.w_out ? (p.max_len + kJoinSpan - 1) / kJoinSpan : 1;
  const long long spare = 2LL * kSeqSms / ((long long)p.B * p.K);
  const long long wide = 8 * outs < spare ? 8 * outs : spare;
  const long long most = outs > spans ? outs : spans;
  const unsigned pieces = (unsigned)(most > wide ? most : wide);
  if (pieces > 65535) return cudaErrorInvalidConfiguration;
  const size_t smem = (size_t)(p.G + d.heads + d.C + 2 * d.heads * d.C) * 4;
  // the split of L1 that decode_kernel runs with, so that blocks of both fit an SM
  e = prefer_smem<join_kernel<E>>();
  if (e != cudaSuccess) return e;
  return launch_dependent(join_kernel<E>, dim3(p.B * p.K, pieces), kJoinThr, smem, st, p, d);
}

template <typename E>
cudaError_t decode_lanes(const CacheParams& p, const DecodePlan& d, cudaStream_t st) {
  if (p.hd <= 32) return decode_go<E, LaneCore<E, 1>>(p, d, st);
  if (p.hd <= 64) return decode_go<E, LaneCore<E, 2>>(p, d, st);
  if (p.hd <= 128) return decode_go<E, LaneCore<E, 4>>(p, d, st);
  return decode_go<E, LaneCore<E, 8>>(p, d, st);
}

template <int NT>
cudaError_t decode_mma(const CacheParams& p, const DecodePlan& d, cudaStream_t st) {
  using E = __nv_bfloat16;
  if (p.hd == 32) return decode_go<E, MmaCore<32, NT, 4, 32>>(p, d, st);
  if (p.hd == 64) return decode_go<E, MmaCore<64, NT, 3, 32>>(p, d, st);
  return decode_go<E, MmaCore<128, NT, 3, 16>>(p, d, st);
}

}  // namespace

// Partials and finished sums of decode, its logits for the weights, or the
// kept positions of evict: the calls share the space.
size_t cache_workspace(const CacheParams& p, int dtype) {
  const DecodeShape s = decode_shape(p, dtype);
  const size_t dec = part_bytes(p, s) + lse_bytes(p) + prefix_bytes(p) +
                     (p.with_weights ? align256((size_t)p.B * p.H * vis_max(p) * 4) : 0);
  const size_t evict = align256((size_t)p.B * p.K * p.budget * 4);
  return dec > evict ? dec : evict;
}

cudaError_t cache_append(const CacheParams& p, int dtype, cudaStream_t st) {
  const int cpr = p.hd / (dtype == SWIN_DTYPE_BF16 ? 8 : 4);
  const long long blocks = ((long long)p.T * p.K * cpr + 256 * kAppend - 1) / (256 * kAppend);
  if (blocks * 256 * kAppend > 0x7fffffffLL || blocks * p.B > 0x7fffffffLL)
    return cudaErrorInvalidConfiguration;
  const unsigned grid = (unsigned)(blocks * p.B);
  if (dtype == SWIN_DTYPE_BF16)
    append_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(p, (int)blocks);
  else
    append_kernel<float><<<grid, 256, 0, st>>>(p, (int)blocks);
  note_launch();
  return cudaGetLastError();
}

cudaError_t cache_decode(const CacheParams& p, int dtype, cudaStream_t st) {
  const DecodeShape s = decode_shape(p, dtype);
  DecodePlan d;
  d.C = s.blocks;
  d.heads = s.heads;
  d.nchunk = s.nchunk;
  d.unit = s.unit;
  d.hds = p.hd + 2;
  d.part = (float*)p.ws;
  d.lse2 = (float*)(p.ws + part_bytes(p, s));
  char* rest = p.ws + part_bytes(p, s) + lse_bytes(p);
  d.prefix = p.B > kScanBatch ? (long long*)rest : nullptr;
  d.logits = p.w_out ? (float*)(rest + prefix_bytes(p)) : nullptr;
  d.vis_max = vis_max(p);
  if (d.prefix) {
    units_scan_kernel<<<1, kScanThr, 0, st>>>(p, s.unit, d.prefix);
    note_launch();
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (s.mma) return s.heads == 8 ? decode_mma<1>(p, d, st) : decode_mma<2>(p, d, st);
  return dtype == SWIN_DTYPE_BF16 ? decode_lanes<__nv_bfloat16>(p, d, st)
                                  : decode_lanes<float>(p, d, st);
}

cudaError_t cache_evict(const CacheParams& p, int dtype, cudaStream_t st) {
  int* kept = p.kept ? p.kept : (int*)p.ws;
  const long long bk = (long long)p.B * p.K;
  if (bk > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  // Registers for the positions a sequence can have. Four blocks share a (b, kv head)
  // where one each would leave SMs idle (8 x 32768 weights: 19 us for the call, 29 with
  // one block each; 64 x 32768: 75 and 72), and where one could not hold the positions,
  // as long as that is two rounds of the card at most (2 x 131072: 32 us, 124 without
  // registers; 114 x 65504: 77 and 68).
  if (bk * 4 > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const unsigned grid = (unsigned)bk, grid4 = (unsigned)(4 * bk);
  if (p.max_len <= kSelRound)
    evict_select_kernel<1, 1><<<grid, kSelThr, 0, st>>>(p, kept);
  else if (p.max_len <= 8 * kSelRound && bk * 4 <= kSeqSms)
    evict_select_kernel<2, 4><<<grid4, kSelThr, 0, st>>>(p, kept);
  else if (p.max_len <= 8 * kSelRound)
    evict_select_kernel<8, 1><<<grid, kSelThr, 0, st>>>(p, kept);
  else if (p.max_len <= 32 * kSelRound && bk * 4 <= 2 * kSeqSms)
    evict_select_kernel<8, 4><<<grid4, kSelThr, 0, st>>>(p, kept);
  else
    evict_select_kernel<0, 1><<<grid, kSelThr, 0, st>>>(p, kept);
  note_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int cpr = p.hd / (dtype == SWIN_DTYPE_BF16 ? 8 : 4);
  const long long per = 256 * kCopy;
  const long long blocks = ((long long)p.budget * cpr + per - 1) / per;
  if ((long long)p.budget * cpr > 0x7fffff00LL || blocks * bk > 0x7fffffffLL)
    return cudaErrorInvalidConfiguration;
  const dim3 all((unsigned)(blocks * bk));
  return dtype == SWIN_DTYPE_BF16
             ? launch_dependent(evict_copy_kernel<__nv_bfloat16>, all, 256, 0, st, p,
                                (const int*)kept, (int)blocks)
             : launch_dependent(evict_copy_kernel<float>, all, 256, 0, st, p,
                                (const int*)kept, (int)blocks);
}

}  // namespace swin
