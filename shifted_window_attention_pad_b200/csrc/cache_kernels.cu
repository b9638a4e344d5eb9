// cache_kernels.cu -- the paged key-value cache: appending tokens, attention of
// one token per sequence, and eviction by accumulated attention weight
// (declared in include/swin_seqattn.h).
#include <math.h>

#include "seq_common.cuh"
#include "sm100_ptx.cuh"

namespace swin {
namespace {

constexpr int kDecThr = 128;    // decode block: 4 warps
constexpr int kUnit = 128;      // cache positions of a work unit, 32 per warp
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
// 16 bytes of one tensor's row per thread, channels fastest: reads and writes
// whole rows. Bound by HBM (every new row read once and written once).
template <typename E>
__global__ void __launch_bounds__(256) append_kernel(const __grid_constant__ CacheParams p) {
  constexpr int V = 16 / sizeof(E);
  const int cpr = p.hd / V;
  const long long per = (long long)p.T * p.K * cpr;
  const long long x = (long long)blockIdx.x * 256 + threadIdx.x;
  if (x >= per * p.B) return;
  const int b = (int)(x / per);
  long long y = x - (long long)b * per;
  const int t = (int)(y / (p.K * cpr));
  y -= (long long)t * (p.K * cpr);
  const int kh = (int)(y / cpr), c = (int)(y - (long long)kh * cpr);
  int cnt = p.T;
  if (p.counts) {
    cnt = p.counts[b];
    cnt = cnt < 0 ? 0 : (cnt > p.T ? p.T : cnt);
  }
  if (t >= cnt) return;
  const int pos = cache_len(p, b) - cnt + t;
  if (pos < 0) {
    atomicExch(p.status, SWIN_ERR_INVALID_ARG);
    return;
  }
  const long long row = cache_row(p, p.table, b, kh, pos);
  if (row < 0) return;
  const long long src = ((long long)b * p.T + t) * p.ks + (long long)kh * p.hd + c * V;
  const long long dst = row * p.hd + c * V;
  const uint4 k = *reinterpret_cast<const uint4*>((const E*)p.k_new + src);
  const uint4 v = *reinterpret_cast<const uint4*>((const E*)p.v_new + src);
  *reinterpret_cast<uint4*>((E*)p.kc + dst) = k;
  *reinterpret_cast<uint4*>((E*)p.vc + dst) = v;
}

// ---- decode ------------------------------------------------------------------------
// The visible positions of a sequence are numbered 0 .. n - 1: the sinks, then
// the window (vis_pos). They are cut into units of 128; the units of all
// sequences, kv heads and chunks of query heads form one list, and block c of
// C takes units c T / C .. (c + 1) T / C of the T there are, whatever the mix
// of lengths: every block gets the same number of bytes to read, which is what
// bounds the kernel. A block that has all units of a (sequence, kv head,
// chunk) writes its output; pieces go to the workspace and join_kernel adds
// them in order. All of this is computed on the device from the lengths, so a
// captured graph follows them.
struct DecodePlan {
  int C, heads, nchunk, hds;     // blocks, query heads of a chunk, chunks, row of partials
  float* part;                   // [C][2][heads][hds]: m, l (hds - 2, hds - 1) and O
  float* lse2;                   // [B][H] of finished heads, log2 units
  float* logits;                 // weights: [B][H][vis_max], log2 units
  long long vis_max;
};

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
__device__ __forceinline__ int units_of(const CacheParams& p, int b) {
  return (vis_of(p, b).n + kUnit - 1) / kUnit;
}

// Total units per (kv head, chunk) over the batch and, of them, those before
// sequence `b_stop` (block-wide; kDecThr threads; `sh` holds 10 values).
__device__ __forceinline__ void batch_units(const CacheParams& p, int b_stop, long long* sh,
                                            long long& before, long long& total) {
  long long bef = 0, tot = 0;
  for (int b = threadIdx.x; b < p.B; b += kDecThr) {
    const int u = units_of(p, b);
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
    sh[4 + threadIdx.x / 32] = tot;
  }
  __syncthreads();
  before = sh[0] + sh[1] + sh[2] + sh[3];
  total = sh[4] + sh[5] + sh[6] + sh[7];
  __syncthreads();
}

// Sequence that holds the target-th unit of the batch and the units before it.
__device__ __forceinline__ void find_seq(const CacheParams& p, long long target, long long* sh,
                                         int& b_out, long long& before_out) {
  // each thread a contiguous run of sequences, an exclusive scan over threads
  const int per = (p.B + kDecThr - 1) / kDecThr;
  const int b0 = threadIdx.x * per, b1 = min(p.B, b0 + per);
  long long sum = 0;
  for (int b = b0; b < b1; ++b) sum += units_of(p, b);
  long long inc = sum;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += t;
  }
  if (lane == 31) sh[threadIdx.x / 32] = inc;
  __syncthreads();
  for (int w = 0; w < (int)threadIdx.x / 32; ++w) inc += sh[w];
  long long before = inc - sum;
  if (target >= before && target < inc) {
    int b = b0;
    for (;;) {
      const int u = units_of(p, b);
      if (target < before + u) break;
      before += u;
      ++b;
    }
    sh[8] = b;
    sh[9] = before;
  }
  __syncthreads();
  b_out = (int)sh[8];
  before_out = sh[9];
  __syncthreads();
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
// warp runs alone over tiles of 32 positions through a ring of ST cp.async
// stages (16-byte chunks, swizzled against bank conflicts). Logits transposed,
// S^T = K Q^T, and O^T = V^T P^T, on mma.sync: the key and channel sides have
// 16 rows to give and the query heads are the 8-wide side, so the eight heads
// or fewer of a group fill a tile; P^T moves from the one product to the other
// through movmatrix. Arithmetic is a few per cent of the warp's time: the
// cache is read once, and its bytes bound the kernel.
template <int HD, int NT, int ST>
struct MmaCore {
  static constexpr int kHeads = 8 * NT;
  static constexpr int kCpr = HD / 8;                    // 16-byte chunks of a row
  static constexpr int kTileBytes = 32 * HD * 2;         // one of K, V
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

    // tiles warp, warp + 4, ... of the segment's 32-position tiles
    const int t_end = min(s.u1 * 4, (s.vis.n + 31) / 32);
    const int t0 = s.u0 * 4 + warp;
    const int cnt = t0 < t_end ? (t_end - t0 + 3) / 4 : 0;
    long long row_next = cnt > 0 ? lane_row(p, s, t0 * 32 + lane) : -1;
    auto issue = [&](int x) {   // tile x of this warp into stage x % ST
      if (x < cnt) {
        const int st = x % ST;
        const long long row = row_next;
        if (x + 1 < cnt) row_next = lane_row(p, s, (t0 + (x + 1) * 4) * 32 + lane);
        const uint32_t ok = __ballot_sync(0xffffffffu, row != -1);
        if (lane == 0) vmask[st] = ok;
        const uint32_t kb = base + st * 2 * kTileBytes, vb = kb + kTileBytes;
        constexpr int RPI = 32 / kCpr;   // rows per instruction
#pragma unroll
        for (int i = 0; i < 32 / RPI; ++i) {
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
      float sacc[2][NT][4];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
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
      uint32_t pf[2][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = mt * 16 + lane / 4 + (e >> 1) * 8;
            const float v = (ok >> key) & 1 ? sacc[mt][nt][e] * p.scale_log2 : -INFINITY;
            sacc[mt][nt][e] = v;
            mx[e & 1] = fmaxf(mx[e & 1], v);
          }
        if (d.logits) {
          const int u = (t0 + x * 4) * 32;
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
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
        for (int mt = 0; mt < 2; ++mt) {
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
      for (int mt = 0; mt < 2; ++mt)
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

// Any head size and type: lanes across the channels (HT per lane), four
// positions' rows in flight, up to four query heads. For fp32 its loads keep
// HBM busy; for narrow bf16 rows with many heads the dot products' shuffles
// bound it.
template <typename E, int HT>
struct LaneCore {
  static constexpr int kHeads = 4;
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
    const int t_end = min(s.u1 * 4, (s.vis.n + 31) / 32);
    for (int tile = s.u0 * 4 + warp; tile < t_end; tile += 4) {
      const long long row = lane_row(p, s, tile * 32 + lane);
      const int left = min(32, s.vis.n - tile * 32);
#pragma unroll 1
      for (int r0 = 0; r0 < left; r0 += 4) {
        float k[4][HT], v[4][HT];
        bool ok[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const long long rr = __shfl_sync(0xffffffffu, row, r0 + r);
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
#pragma unroll
        for (int h = 0; h < kHeads; ++h) {
          if (h >= s.hc) break;
          float a[4], mx = m[h];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            a[r] = 0.f;
#pragma unroll
            for (int t = 0; t < HT; ++t) a[r] = fmaf(q[h][t], k[r][t], a[r]);
          }
#pragma unroll
          for (int w = 16; w > 0; w >>= 1)
#pragma unroll
            for (int r = 0; r < 4; ++r) a[r] += __shfl_xor_sync(0xffffffffu, a[r], w);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            if (!ok[r]) a[r] = -INFINITY;
            mx = fmaxf(mx, a[r]);
          }
          if (d.logits && lane < 4 && r0 + lane < left) {
            const float x = lane == 0 ? a[0] : (lane == 1 ? a[1] : (lane == 2 ? a[2] : a[3]));
            d.logits[((long long)s.b * p.H + s.h0 + h) * d.vis_max + tile * 32 + r0 + lane] = x;
          }
          const float mu = mx == -INFINITY ? 0.f : mx;
          const float f = exp2f(m[h] - mu);
          m[h] = mx;
          l[h] *= f;
#pragma unroll
          for (int t = 0; t < HT; ++t) o[h][t] *= f;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float w = exp2f(a[r] - mu);
            l[h] += w;
#pragma unroll
            for (int t = 0; t < HT; ++t) o[h][t] = fmaf(w, v[r][t], o[h][t]);
          }
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
  __shared__ long long sh[10];
  float* res = (float*)smem;
  long long dummy, total;
  batch_units(p, 0, sh, dummy, total);
  const int kcn = p.K * d.nchunk;
  total *= kcn;
  long long cur = (long long)blockIdx.x * total / d.C;
  const long long start = cur, end = (long long)(blockIdx.x + 1) * total / d.C;
  if (cur >= end) return;
  int b;
  long long before;
  find_seq(p, cur / kcn, sh, b, before);
  const int hw = p.hd + 2;
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
    const int kc = (int)(rel / U);
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
    for (int x = threadIdx.x; x < s.hc * p.hd; x += kDecThr) {
      const int h = x / p.hd, c = x - h * p.hd;
      float m[4], M = -INFINITY, L = 0.f, O = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        m[w] = res[(w * Core::kHeads + h) * hw + p.hd];
        M = fmaxf(M, m[w]);
      }
      const float mu = M == -INFINITY ? 0.f : M;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float f = exp2f(m[w] - mu);
        L = fmaf(res[(w * Core::kHeads + h) * hw + p.hd + 1], f, L);
        O = fmaf(res[(w * Core::kHeads + h) * hw + c], f, O);
      }
      if (whole) {
        seq_st((E*)p.out + ((long long)s.b * p.H + s.h0 + h) * p.hd + c, L == 0.f ? 0.f : O / L);
        if (c == 0) {
          const float z = lse2_of(M, L);
          if (p.lse) p.lse[(long long)s.b * p.H + s.h0 + h] = z * kLn2;
          d.lse2[(long long)s.b * p.H + s.h0 + h] = z;
        }
      } else {
        part[h * d.hds + c] = O;
        if (c == 0) {
          part[h * d.hds + p.hd] = M;
          part[h * d.hds + p.hd + 1] = L;
        }
      }
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
// kJoinSpan positions (0 also joins). Waits for decode_kernel, whose
// programmatic dependent it is.
constexpr int kJoinSpan = 2048;
template <typename E>
__global__ void __launch_bounds__(kDecThr)
    join_kernel(const __grid_constant__ CacheParams p, const __grid_constant__ DecodePlan d) {
  extern __shared__ float lse_sh[];   // [G]
  __shared__ long long sh[10];
  const int b = blockIdx.x / p.K, kh = blockIdx.x - b * p.K;
  long long before, total;
  batch_units(p, b, sh, before, total);
  ptx::grid_dep_wait();
  const int kcn = p.K * d.nchunk;
  total *= kcn;
  const Vis vis = vis_of(p, b);
  const int U = (vis.n + kUnit - 1) / kUnit;
  for (int h = threadIdx.x; h < p.G && U == 0; h += kDecThr) lse_sh[h] = -INFINITY;
  if (U == 0 && blockIdx.y == 0) {
    for (int x = threadIdx.x; x < p.G * p.hd; x += kDecThr)
      seq_st((E*)p.out + ((long long)b * p.H + kh * p.G) * p.hd + x, 0.f);
    for (int h = threadIdx.x; h < p.G && p.lse; h += kDecThr)
      p.lse[(long long)b * p.H + kh * p.G + h] = -INFINITY;
  }
  if (U > 0)
    for (int chunk = 0; chunk < d.nchunk; ++chunk) {
      const long long g0 = (before * p.K * d.nchunk) + ((long long)kh * d.nchunk + chunk) * U;
      const long long g1 = g0 + U;
      const int c0 = (int)(((g0 + 1) * d.C - 1) / total), c1 = (int)((g1 * d.C - 1) / total);
      const int hc = min(d.heads, p.G - chunk * d.heads);
      const int h0 = chunk * d.heads;   // within the group
      if (c0 == c1) {
        for (int h = threadIdx.x; h < hc; h += kDecThr)
          lse_sh[h0 + h] = d.lse2[(long long)b * p.H + kh * p.G + h0 + h];
        continue;
      }
      auto slot = [&](int c) -> const float* {
        const long long s0 = c * total / d.C, s1 = (c + 1) * total / d.C;
        if (max(g0, s0) >= min(g1, s1)) return nullptr;   // a block without units
        return d.part + ((long long)c * 2 + (s0 >= g0 ? 0 : 1)) * d.heads * d.hds;
      };
      for (int x = threadIdx.x; x < hc * p.hd; x += kDecThr) {
        const int h = x / p.hd, c = x - h * p.hd;
        if (blockIdx.y > 0 && c > 0) continue;
        float M = -INFINITY, L = 0.f, O = 0.f;
        for (int k = c0; k <= c1; ++k) {
          const float* s = slot(k);
          if (s) M = fmaxf(M, s[h * d.hds + p.hd]);
        }
        const float mu = M == -INFINITY ? 0.f : M;
        for (int k = c0; k <= c1; ++k) {
          const float* s = slot(k);
          if (!s) continue;
          const float f = exp2f(s[h * d.hds + p.hd] - mu);
          L = fmaf(s[h * d.hds + p.hd + 1], f, L);
          O = fmaf(s[h * d.hds + c], f, O);
        }
        const long long at = (long long)b * p.H + kh * p.G + h0 + h;
        if (blockIdx.y == 0) seq_st((E*)p.out + at * p.hd + c, L == 0.f ? 0.f : O / L);
        if (c == 0) {
          const float z = lse2_of(M, L);
          lse_sh[h0 + h] = z;
          if (p.lse && blockIdx.y == 0) p.lse[at] = z * kLn2;
        }
      }
    }
  if (!p.w_out) return;
  __syncthreads();
  const int p1 = (int)min((long long)vis.len, ((long long)blockIdx.y + 1) * kJoinSpan);
  const long long row = ((long long)b * p.K + kh) * p.max_len;
  for (int pos = blockIdx.y * kJoinSpan + threadIdx.x; pos < p1; pos += kDecThr) {
    float w = p.w[row + pos];
    const bool see = pos < vis.first || pos >= vis.first + vis.shift;
    if (see) {
      const int u = pos < vis.first ? pos : pos - vis.shift;
      const float* x = d.logits + ((long long)b * p.H + kh * p.G) * d.vis_max + u;
      float sum = 0.f;
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
// Order of weights as unsigned numbers: NaN lowest, then by value, -0 = +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr int kSelThr = 1024;
constexpr int kSelCache = 40960;   // weights held in shared memory (160 KB)

// Which positions of (b, kv head) stay: one block each. The threshold is the
// m-th largest weight of the middle, found bit group by bit group (four
// passes over 8 bits with a histogram per warp); ties at the threshold are
// counted off in order of position. Then every warp takes a contiguous run of
// positions, and two scans over the warps give each its place in the output.
__global__ void __launch_bounds__(kSelThr)
    evict_select_kernel(const __grid_constant__ CacheParams p, int* kept, int cache_max) {
  extern __shared__ uint32_t sel[];
  uint32_t* hist = sel;                 // [32][256]
  uint32_t* keys = sel + 32 * 256;      // [cache_max]
  __shared__ uint32_t sh[2];
  __shared__ int wsum[32];
  const int b = blockIdx.x / p.K, kh = blockIdx.x - b * p.K;
  const int n = cache_len(p, b), keep = min(n, p.budget);
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const float* w = p.w + ((long long)b * p.K + kh) * p.max_len;
  float* w_out = p.w_out + ((long long)b * p.K + kh) * p.max_len;
  int* out = kept + ((long long)b * p.K + kh) * p.budget;
  if (kh == 0 && threadIdx.x == 0) p.new_len[b] = keep;
  for (int x = keep + threadIdx.x; x < p.budget; x += kSelThr) out[x] = -1;
  for (long long x = keep + threadIdx.x; x < p.max_len; x += kSelThr) w_out[x] = 0.f;
  if (n <= p.budget) {
    for (int x = threadIdx.x; x < n; x += kSelThr) {
      out[x] = x;
      w_out[x] = w[x];
    }
    return;
  }
  const int lo = p.sinks, hi = n - p.recent;       // the middle
  const int m = p.budget - p.sinks - p.recent;     // of which m stay, m < hi - lo
  const bool cached = hi - lo <= cache_max;
  if (cached)
    for (int x = lo + threadIdx.x; x < hi; x += kSelThr) keys[x - lo] = weight_key(w[x]);
  auto key_at = [&](int x) { return cached ? keys[x - lo] : weight_key(w[x]); };
  uint32_t prefix = 0, thr = 0xffffffffu;
  int need = m;       // ties at the threshold that stay
  if (m > 0) {
    for (int pass = 0; pass < 4; ++pass) {
      const int sh_bits = 24 - 8 * pass;
      for (int x = threadIdx.x; x < 32 * 256; x += kSelThr) hist[x] = 0;
      __syncthreads();
      for (int x = lo + threadIdx.x; x < hi; x += kSelThr) {
        const uint32_t k = key_at(x);
        if (pass == 0 || (k >> (sh_bits + 8)) == prefix)
          atomicAdd(&hist[warp * 256 + ((k >> sh_bits) & 255)], 1u);
      }
      __syncthreads();
      if (threadIdx.x < 256) {
        uint32_t s = 0;
#pragma unroll
        for (int v = 0; v < 32; ++v) s += hist[v * 256 + threadIdx.x];
        hist[threadIdx.x] = s;
      }
      __syncthreads();
      if (warp == 0) {
        // bins from the top, eight a lane
        uint32_t c[8], sum = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          c[e] = hist[255 - (lane * 8 + e)];
          sum += c[e];
        }
        uint32_t inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t t = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += t;
        }
        uint32_t before = inc - sum;
        if (before < (uint32_t)need && (uint32_t)need <= inc) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (before < (uint32_t)need && (uint32_t)need <= before + c[e]) {
              sh[0] = 255 - (lane * 8 + e);
              sh[1] = need - before;
              break;
            }
            before += c[e];
          }
        }
      }
      __syncthreads();
      prefix = (prefix << 8) | sh[0];
      need = (int)sh[1];
      __syncthreads();
    }
    thr = prefix;
  } else {
    need = 0;
    __syncthreads();
  }
  // positions of this warp
  const int per = ((n + 31) / 32 + 31) / 32 * 32;
  const int x0 = min(n, warp * per), x1 = min(n, x0 + per);
  int gt = 0, eq = 0;   // kept outright, ties
  for (int x = x0 + lane; x < x1; x += 32) {
    const bool mid = x >= lo && x < hi;
    const uint32_t k = mid ? key_at(x) : 0u;
    gt += !mid || (m > 0 && k > thr);
    eq += mid && m > 0 && k == thr;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    gt += __shfl_xor_sync(0xffffffffu, gt, o);
    eq += __shfl_xor_sync(0xffffffffu, eq, o);
  }
  auto before_warp = [&](int v) {   // sum of v over the warps before this one
    __syncthreads();
    if (lane == 0) wsum[warp] = v;
    __syncthreads();
    int s = lane < warp ? wsum[lane] : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
  };
  int ties = before_warp(eq);                      // ties before this warp's run
  const int mine = min(max(need - ties, 0), eq);
  int at = before_warp(gt + mine);
  for (int x = x0; x < x1; x += 32) {
    const int y = x + lane;
    const bool in = y < x1, mid = in && y >= lo && y < hi;
    const uint32_t k = mid ? key_at(y) : 0u;
    const bool tie = mid && m > 0 && k == thr;
    const uint32_t tb = __ballot_sync(0xffffffffu, tie);
    const int rank = ties + __popc(tb & ((1u << lane) - 1u));
    const bool stay = in && (!mid || (m > 0 && k > thr) || (tie && rank < need));
    const uint32_t kb = __ballot_sync(0xffffffffu, stay);
    if (stay) {
      const int r = at + __popc(kb & ((1u << lane) - 1u));
      out[r] = y;
      w_out[r] = w[y];
    }
    ties += __popc(tb);
    at += __popc(kb);
  }
}

// The kept rows to their new pages, 16 bytes of a K and a V row per thread.
// Bound by HBM: budget rows read once and written once.
template <typename E>
__global__ void __launch_bounds__(256)
    evict_copy_kernel(const __grid_constant__ CacheParams p, const int* kept, int blocks) {
  constexpr int V = 16 / sizeof(E);
  const int cpr = p.hd / V;
  const int bk = blockIdx.x / blocks;   // `blocks` blocks of 256 chunks per (b, kh)
  const int b = bk / p.K, kh = bk - b * p.K;
  const int x = (blockIdx.x - bk * blocks) * 256 + threadIdx.x;
  const int r = x / cpr, c = x - r * cpr;
  ptx::grid_dep_wait();
  if (r >= min(cache_len(p, b), p.budget)) return;
  const int pos = kept[(long long)bk * p.budget + r];
  const long long src = cache_row(p, p.table, b, kh, pos);
  const long long dst = cache_row(p, p.dst_table, b, kh, r);
  if (src < 0 || dst < 0) return;
  const uint4 k = *reinterpret_cast<const uint4*>((const E*)p.kc + src * p.hd + c * V);
  const uint4 v = *reinterpret_cast<const uint4*>((const E*)p.vc + src * p.hd + c * V);
  *reinterpret_cast<uint4*>((E*)p.kc + dst * p.hd + c * V) = k;
  *reinterpret_cast<uint4*>((E*)p.vc + dst * p.hd + c * V) = v;
}

// ---- host --------------------------------------------------------------------------
struct DecodeShape {
  bool mma;
  int heads, nchunk, blocks;
};
DecodeShape decode_shape(const CacheParams& p, int dtype) {
  DecodeShape s;
  s.mma = dtype == SWIN_DTYPE_BF16 && (p.hd == 32 || p.hd == 64 || p.hd == 128);
  s.heads = s.mma ? (p.G <= 8 ? 8 : 16) : 4;
  s.nchunk = (p.G + s.heads - 1) / s.heads;
  // blocks that fit the card at once (shared memory of the ring; registers)
  const long long resident = (long long)kSeqSms * (s.mma ? (p.hd == 128 ? 1 : 2) : 4);
  const long long cap = (long long)p.window + p.sinks;
  const long long vis = p.max_len < cap ? p.max_len : cap;
  const long long most = (long long)p.B * p.K * s.nchunk * ((vis + kUnit - 1) / kUnit);
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

template <typename K, typename... A>
cudaError_t launch_dependent(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t st,
                             A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e == cudaSuccess) note_launch();
  return e;
}

template <typename E, class Core>
cudaError_t decode_go(const CacheParams& p, const DecodePlan& d, cudaStream_t st) {
  auto kernel = decode_kernel<E, Core>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)Core::kSmem);
  if (e != cudaSuccess) return e;
  kernel<<<d.C, kDecThr, Core::kSmem, st>>>(p, d);
  note_launch();
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const unsigned pieces = p.w_out ? (unsigned)((p.max_len + kJoinSpan - 1) / kJoinSpan) : 1;
  if (pieces > 65535) return cudaErrorInvalidConfiguration;
  return launch_dependent(join_kernel<E>, dim3(p.B * p.K, pieces), kDecThr,
                          (size_t)p.G * sizeof(float), st, p, d);
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
  if (p.hd == 32) return decode_go<E, MmaCore<32, NT, 4>>(p, d, st);
  if (p.hd == 64) return decode_go<E, MmaCore<64, NT, 3>>(p, d, st);
  return decode_go<E, MmaCore<128, NT, 3>>(p, d, st);
}

}  // namespace

// Partials and finished sums of decode, its logits for the weights, or the
// kept positions of evict: the calls share the space.
size_t cache_workspace(const CacheParams& p, int dtype) {
  const DecodeShape s = decode_shape(p, dtype);
  const size_t dec = part_bytes(p, s) + lse_bytes(p) +
                     (p.with_weights ? align256((size_t)p.B * p.H * vis_max(p) * 4) : 0);
  const size_t evict = align256((size_t)p.B * p.K * p.budget * 4);
  return dec > evict ? dec : evict;
}

cudaError_t cache_append(const CacheParams& p, int dtype, cudaStream_t st) {
  const int cpr = p.hd / (dtype == SWIN_DTYPE_BF16 ? 8 : 4);
  const long long grid = ((long long)p.B * p.T * p.K * cpr + 255) / 256;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if (dtype == SWIN_DTYPE_BF16)
    append_kernel<__nv_bfloat16><<<(unsigned)grid, 256, 0, st>>>(p);
  else
    append_kernel<float><<<(unsigned)grid, 256, 0, st>>>(p);
  note_launch();
  return cudaGetLastError();
}

cudaError_t cache_decode(const CacheParams& p, int dtype, cudaStream_t st) {
  const DecodeShape s = decode_shape(p, dtype);
  DecodePlan d;
  d.C = s.blocks;
  d.heads = s.heads;
  d.nchunk = s.nchunk;
  d.hds = p.hd + 2;
  d.part = (float*)p.ws;
  d.lse2 = (float*)(p.ws + part_bytes(p, s));
  d.logits = p.w_out ? (float*)(p.ws + part_bytes(p, s) + lse_bytes(p)) : nullptr;
  d.vis_max = vis_max(p);
  if (s.mma) return s.heads == 8 ? decode_mma<1>(p, d, st) : decode_mma<2>(p, d, st);
  return dtype == SWIN_DTYPE_BF16 ? decode_lanes<__nv_bfloat16>(p, d, st)
                                  : decode_lanes<float>(p, d, st);
}

cudaError_t cache_evict(const CacheParams& p, int dtype, cudaStream_t st) {
  int* kept = p.kept ? p.kept : (int*)p.ws;
  const long long bk = (long long)p.B * p.K;
  if (bk > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const int cache_max = (int)(p.max_len < kSelCache ? p.max_len : kSelCache);
  const size_t smem = 32 * 256 * 4 + (size_t)cache_max * 4;
  cudaError_t e = cudaFuncSetAttribute(evict_select_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  evict_select_kernel<<<(unsigned)bk, kSelThr, smem, st>>>(p, kept, cache_max);
  note_launch();
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int cpr = p.hd / (dtype == SWIN_DTYPE_BF16 ? 8 : 4);
  const long long blocks = ((long long)p.budget * cpr + 255) / 256, grid = blocks * bk;
  if ((long long)p.budget * cpr > 0x7fffff00LL || grid > 0x7fffffffLL)
    return cudaErrorInvalidConfiguration;
  return dtype == SWIN_DTYPE_BF16
             ? launch_dependent(evict_copy_kernel<__nv_bfloat16>, dim3((unsigned)grid), 256, 0, st,
                                p, (const int*)kept, (int)blocks)
             : launch_dependent(evict_copy_kernel<float>, dim3((unsigned)grid), 256, 0, st, p,
                                (const int*)kept, (int)blocks);
}

}  // namespace swin
