// seq.h -- launchers and plans shared by the sequence-attention and key-value
// cache files (declared to users in include/swin_seqattn.h).
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "../../include/swin_seqattn.h"
#include "kernels.h"

namespace swin {

constexpr int kSeqSms = 148;          // B200; workspace sizes may not depend on a CUDA call
constexpr float kSeqLog2e = 1.4426950408889634f;

// How the key-side backward (dk, dv) is cut into work items. A key tile of T
// keys sees the queries j .. j + window - 1 of every query head of its group,
// a tile that holds sink tokens every later query. Three things keep the items
// even and the card full, all fixed by the description alone:
//  * gs > 1: the query heads of a group are split into gs parts, each with an
//    fp32 partial of dk and dv (few key heads);
//  * the first nst tiles hold the sinks: their queries are cut into qc chunks
//    of ch queries, each with a partial of the tile;
//  * partials are summed in order by dkv_reduce_kernel, so results do not
//    depend on timing.
struct DkvPlan {
  int T, ntiles, nst, qc, ch, gs;
  long long items;                 // B * K * gs * (nst * qc + ntiles - nst)
  size_t main_bytes, sink_bytes;   // partials of dk and dv together
};

// Launches a kernel as a programmatic dependent of the one before it on the stream:
// its blocks may start while that one ends, and wait (grid_dep_wait) before they
// touch what it wrote.
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

// Lets `Kernel` use `bytes` of dynamic shared memory, once per device.
template <auto Kernel>
cudaError_t allow_smem(size_t bytes) {
  static std::atomic<uint64_t> done{0};   // by device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (done.load(std::memory_order_relaxed) >> dev & 1)) return cudaSuccess;
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev, std::memory_order_relaxed);
  return e;
}

// Runs `Kernel` with the largest shared-memory share of L1, once per device: so its
// blocks can join those of a kernel that needs it on an SM.
template <auto Kernel>
cudaError_t prefer_smem() {
  static std::atomic<uint64_t> done{0};   // by device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (done.load(std::memory_order_relaxed) >> dev & 1)) return cudaSuccess;
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                           cudaSharedmemCarveoutMaxShared);
  if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev, std::memory_order_relaxed);
  return e;
}

struct SeqParams {
  int B, S, H, K, G, hd;
  int window, sinks;               // window in 1 .. S; sinks 0 when the window hides nothing
  long long qs, ks;                // elements from token to token
  const void *q, *k, *v, *o, *dout;
  const int* lengths;
  const float* lse_in;
  void *out, *dq, *dk, *dv;
  float* lse;
  float *nl, *nd;                  // backward: -lse log2 e and -D of every row, [B][H][ld_stride]
  long long ld_stride;             // S rounded up to whole tiles of 128 queries
  float *main_part, *sink_part;    // backward partials (see DkvPlan)
  DkvPlan plan;
  int* status;
  float scale, scale_log2;
  int test_timeout;
};

DkvPlan make_dkv_plan(int B, int S, int K, int G, int hd, int window, int sinks, int T);

// Portable kernels; T of their key tiles.
int seq_generic_tile(int B, int S, int H, int hd);
cudaError_t seq_generic_forward(const SeqParams& p, int dtype, cudaStream_t st);
cudaError_t seq_generic_backward(const SeqParams& p, int dtype, cudaStream_t st);
// (-lse log2 e, -D) of every row, and the sum of the partials: both families.
cudaError_t seq_prep(const SeqParams& p, int dtype, cudaStream_t st);
cudaError_t seq_reduce(const SeqParams& p, int dtype, cudaStream_t st);

// tcgen05 / TMA kernels (bf16, head_dim up to 128).
bool seq_fast_supported(int dtype, int hd);
cudaError_t seq_fast_forward(const SeqParams& p, cudaStream_t st);
cudaError_t seq_fast_backward(const SeqParams& p, cudaStream_t st);

// ---- paged cache ---------------------------------------------------------------
struct CacheParams {
  int B, H, K, G, hd, ps, pages, mp;
  int window, sinks, recent, budget;
  long long qs, ks;
  long long max_len;               // mp * ps
  const void *q, *k_new, *v_new;
  const int *lengths, *table, *dst_table, *counts;
  void *kc, *vc;
  const float* w;
  float* w_out;
  int* new_len;
  int* kept;
  void* out;
  float* lse;
  char* ws;                        // after the header
  int* status;
  float scale_log2;
  int T;                           // append: tokens per sequence
  bool with_weights;               // the workspace has room for decode's logits
};

size_t cache_workspace(const CacheParams& p, int dtype);
cudaError_t cache_append(const CacheParams& p, int dtype, cudaStream_t st);
cudaError_t cache_decode(const CacheParams& p, int dtype, cudaStream_t st);
cudaError_t cache_evict(const CacheParams& p, int dtype, cudaStream_t st);

}  // namespace swin
