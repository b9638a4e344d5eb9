// seq_tc.cuh -- what the tcgen05 kernels of sequence attention share: bounded
// waits, rings, the feed of work items, tiles of tokens in shared memory and
// their matrix descriptors.
#pragma once
#include "fast_common.cuh"
#include "seq_common.cuh"

namespace swin {
namespace {

// ---- waits -----------------------------------------------------------------------
// Bounded as mbar_wait is; the clock is read only after a number of tries (a read
// costs more than a product's wait usually lasts), and time in which softmax warps
// recompute rows (abort[1], see fix_out_row) does not count.
__device__ __noinline__ bool seq_wait_long(uint64_t* bar, uint32_t parity, volatile int* abort,
                                           int* status) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (ptx::mbar_try_wait(bar, parity)) return true;
  uint64_t t0 = ptx::globaltimer();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 16; ++i)
      if (ptx::mbar_try_wait(bar, parity)) return true;
    if (abort[0]) return false;
    const uint64_t now = ptx::globaltimer();
    if (abort[1]) t0 = now;
    if (now - t0 > kWaitLimitNs) {
      abort[0] = 1;
      atomicExch(status, SWIN_ERR_TIMEOUT);
      return false;
    }
  }
}
__device__ __forceinline__ bool seq_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                         int* status) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  return seq_wait_long(bar, parity, abort, status);
}
// A wait of a whole warp: every lane sees the phase, and all take the same way
// when the wait is given up.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                          int* status) {
  const bool ok = seq_wait(bar, parity, abort, status);
  return __all_sync(0xffffffffu, ok);
}

// True on one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(r));
  return r != 0;
}
// A value that is the same on all lanes, said so that it can live in a uniform
// register, where tcgen05.mma takes its operands.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

// Position in a ring of N buffers and the parity of its current round.
template <int N>
struct Ring {
  int s = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++s == N) {
      s = 0;
      parity ^= 1;
    }
  }
};

// ---- work items --------------------------------------------------------------------
// The grid has one block per item, in order of falling work; a running block
// takes the next block's place that has not started (cluster launch control)
// instead of leaving, so items go to whichever SM is free. The producer thread
// asks, works out what the item is (which takes a look at the lengths: some
// thousand cycles) and publishes it in a ring that every other role reads, so
// all of that runs while the roles are busy with the item before.
constexpr int kFeed = 3;
template <class Item>
struct Feed {
  uint4 answer;
  uint64_t answered, full[kFeed], empty[kFeed];
  Item item[kFeed];
  int more[kFeed];
};
template <class Item>
__device__ __forceinline__ void feed_init(Feed<Item>* f, int readers) {
  ptx::mbar_init(&f->answered, 1);
  for (int i = 0; i < kFeed; ++i) {
    ptx::mbar_init(&f->full[i], 1);
    ptx::mbar_init(&f->empty[i], readers);
  }
}
// The producer thread's side.
template <class Item>
struct FeedWrite {
  Feed<Item>* f;
  Ring<kFeed> r;
  uint32_t parity = 0;
  bool open = false;   // a question is out
  __device__ __forceinline__ bool put(const Item& it, bool more, volatile int* abort, int* status) {
    if (!seq_wait(&f->empty[r.s], r.parity ^ 1, abort, status)) return false;
    f->item[r.s] = it;
    f->more[r.s] = more;
    ptx::mbar_arrive(&f->full[r.s]);
    r.next();
    return true;
  }
  // The next block's place into *t; false: none is left (and none may be asked for
  // again), or the wait was given up.
  __device__ __forceinline__ bool next(long long* t, volatile int* abort, int* status) {
    ptx::mbar_arrive_expect_tx(&f->answered, 16);
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 "
        "[%0], [%1];" ::"r"(ptx::smem_u32(&f->answer)),
        "r"(ptx::smem_u32(&f->answered))
        : "memory");
    open = true;
    if (!seq_wait(&f->answered, parity, abort, status)) return false;
    open = false;
    parity ^= 1;
    const uint4 a = f->answer;
    uint32_t got, x;
    asm volatile(
        "{\n\t.reg .b128 h;\n\t.reg .b64 lo, hi;\n\t.reg .pred p;\n\t"
        "mov.b64 lo, {%2, %3};\n\tmov.b64 hi, {%4, %5};\n\t"
        "mov.b128 h, {lo, hi};\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
        "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
        : "=r"(got), "=r"(x)
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w));
    ptx::fence_proxy_async();   // the read comes before the next answer's write
    *t = x;
    return got != 0;
  }
  // An answer still in flight lands before the block leaves (after an abort).
  __device__ __forceinline__ void drain() {
    if (open) ptx::mbar_drain(&f->answered, parity, kTestLimitNs * 100);
  }
};
// A role's side (a whole warp calls together). The item stays in shared memory until
// the role asks for the next one.
template <class Item>
struct FeedRead {
  Feed<Item>* f;
  Ring<kFeed> r;
  bool held = false;
  // The next item, or nullptr at the end.
  __device__ __forceinline__ const Item* next(volatile int* abort, int* status) {
    if (held) {
      __syncwarp();
      if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(&f->empty[r.s]);
      r.next();
    }
    held = true;
    if (!warp_wait(&f->full[r.s], r.parity, abort, status)) return nullptr;
    return f->more[r.s] ? &f->item[r.s] : nullptr;
  }
};

// ---- tiles -------------------------------------------------------------------------
// [ROWS tokens][HD] of one head as channel halves of 64: [ROWS][64] regions with
// the 128-byte swizzle.
template <int ROWS, int HD>
__device__ __forceinline__ void load_tokens(const CUtensorMap* m, uint8_t* dst, int h, int row,
                                            int b, uint64_t* bar) {
#pragma unroll
  for (int hf = 0; hf < HD / 64; ++hf)
    ptx::tma_load_4d(dst + hf * ROWS * 128, m, bar, hf * 64, h, row, b);
}

// Zeroes rows from .. ROWS - 1 (a warp): what padding tokens hold must not meet a
// zero weight in a product (0 x NaN).
template <int ROWS, int HD>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int from) {
  const int lane = threadIdx.x & 31;
  for (int hf = 0; hf < HD / 64; ++hf)
    for (int x = from * 8 + lane; x < ROWS * 8; x += 32)
      ptx::st_shared_v4(ptx::smem_u32(tile + hf * ROWS * 128 + x * 16), 0u, 0u, 0u, 0u);
}

// Matrix descriptors are built once per buffer; a K step of 16 then adds a
// constant (the one issuing thread's instructions are on every step's path).
__device__ __forceinline__ uint64_t kmajor_base(uint32_t base) {
  return ptx::smem_desc(base, 16, 1024, ptx::kSwizzle128);
}
template <int ROWS>
__device__ __forceinline__ constexpr uint32_t kmajor_step(int k16) {
  return ((k16 >> 2) * (ROWS * 128) + (k16 & 3) * 32) >> 4;
}
// as MN-major B operand (the channels are N, 16 rows a K step)
template <int ROWS, int HD>
__device__ __forceinline__ uint64_t mnmajor_base(uint32_t base) {
  return ptx::smem_desc(base, HD > 64 ? ROWS * 128 : 1024, 1024, ptx::kSwizzle128);
}
__device__ __forceinline__ constexpr uint32_t mnmajor_step(int k16) {
  return (k16 * 16 * 128) >> 4;
}

// 32 values as 16 bf16 pairs, rounded; a pair of values as the pair of their top
// 16 bits and the rest rounded to bf16 (x = hi + lo to 2^-16).
__device__ __forceinline__ void round_pairs(const float* v, uint32_t* w) {
#pragma unroll
  for (int e = 0; e < 16; ++e) w[e] = ptx::pack_bf16(v[2 * e], v[2 * e + 1]);
}
__device__ __forceinline__ void split_pair(float2 v, uint32_t& hi, uint32_t& lo) {
  const uint32_t a = __float_as_uint(v.x), b = __float_as_uint(v.y);
  hi = __byte_perm(a, b, 0x7632);
  lo = ptx::pack_bf16(v.x - __uint_as_float(a & 0xFFFF0000u), v.y - __uint_as_float(b & 0xFFFF0000u));
}
// 8 consecutive 32-bit columns into this thread's TMEM lane (warp-collective).
__device__ __forceinline__ void tmem_st8u(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}
// 32 values split into two sets of 16 pairs, to TMEM columns `hi_at` and `lo_at`.
__device__ __forceinline__ void split_to_columns(uint32_t hi_at, uint32_t lo_at, const float* v) {
#pragma unroll
  for (int c = 0; c < 32; c += 16) {
    uint32_t hi[8], lo[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      split_pair(make_float2(v[c + 2 * e], v[c + 2 * e + 1]), hi[e], lo[e]);
    __syncwarp();
    tmem_st8u(hi_at + c / 2, hi);
    tmem_st8u(lo_at + c / 2, lo);
  }
}

// Query rows that see at most this many keys carry P and dS as hi + lo pairs and
// take D = sum_j P_ij dP_ij from a pass of its own: with few keys an entry's
// bf16 rounding (2^-8) does not average out, nor does the rounding of the stored
// o in D = dO.o. The first rows of a sequence are such rows; their errors were
// 0.04 (o) and 0.11 (gradients) of the tensor's RMS without, where other rows'
// are at the outputs' own rounding. Costs nothing that shows elsewhere.
constexpr int kFewKeys = 384;

// Warp-collective store of the warp's 32 rows as store_rows_coalesced does it, with
// only the first `valid` of the NCH 16-byte chunks written (a head_dim that does
// not fill the kernel's).
template <int NCH>
__device__ __forceinline__ void store_rows_clipped(uint4 (&a)[NCH], void* dst, int valid) {
  const int lane = threadIdx.x & 31, q = lane & (NCH - 1);
#pragma unroll
  for (int d = NCH / 2; d >= 1; d >>= 1) {
    const bool hi = (q & d) != 0;
#pragma unroll
    for (int x = 0; x < NCH; ++x) {
      if (x & d) continue;
      uint4 v = hi ? a[x] : a[x + d];   // the chunk that belongs to the other lane
      v.x = __shfl_xor_sync(0xffffffffu, v.x, d);
      v.y = __shfl_xor_sync(0xffffffffu, v.y, d);
      v.z = __shfl_xor_sync(0xffffffffu, v.z, d);
      v.w = __shfl_xor_sync(0xffffffffu, v.w, d);
      if (hi) a[x] = v; else a[x + d] = v;
    }
  }
#pragma unroll
  for (int t = 0; t < NCH; ++t) {
    const unsigned long long row =
        __shfl_sync(0xffffffffu, (unsigned long long)dst, (lane & ~(NCH - 1)) + t);
    if (row && q < valid)
      ptx::st_global_v4(reinterpret_cast<uint4*>(row) + q, a[t].x, a[t].y, a[t].z, a[t].w);
  }
}

// The map [hd, heads, S, B] of one operand, box [64, 1, rows, 1]; channels beyond hd
// read as zeros, so the kernels for 64 and 128 channels take every smaller head.
inline bool encode_tokens(CUtensorMap* m, const void* base, const SeqParams& p, int heads,
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

}  // namespace
}  // namespace swin
