// Keeps the accepted path of a drafted tree in the cache, sm_103a.
//
// Sequence b's last T_b keys are those of its drafted tokens; token i has slot
// first + i, first = L - T_b.  The accepted tokens p_0 < p_1 < ... < p_(n-1) move
// down: the key, value and state of slot first + p_i go to slot first + i, and the
// length becomes first + n.
//
// In place, without a second buffer: a thread owns one 16-byte column of a head's
// rows (or one state array of a head) for the whole path and walks it upwards,
// eight rows at a time, each batch read before it is written.  Row i is written
// after the rows p_0 .. p_i are read, and later sources lie at p_j >= j > i, so
// that nothing is written over before it is read; other threads own other columns.
// A path that does not rise, or leaves the tree, would break that: it is refused
// by the whole CTA before the first row moves.
//
// One CTA for each sequence: its barrier separates all reads of the length from the
// write of the new one (which may be the same word).  Bound by the chain of
// dependent loads (length and path, page ids, rows), not by bytes: a path's rows are
// a few KB per head.  One request 2.3 us, 64 in e4m3 with state 3.5, 256 over latent rows
// 3.0, of which a launch is most.
#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"

namespace splitkv {
namespace {

using namespace ptx;

constexpr int kAtOnce = 8;     // rows of a thread in flight
constexpr int kPathPart = 256; // tokens of the path looked up at a time

__global__ void __launch_bounds__(512) tree_commit_kernel(const __grid_constant__ CommitArgs a) {
  __shared__ int64_t from[kPathPart], to[kPathPart];  // lines of head 0's rows; from < 0: the row stays
  __shared__ int32_t from_slot[kPathPart];            // slot of the state, or -1
  launch_dependents();
  wait_prerequisites();
  const int b = blockIdx.x, tid = threadIdx.x, threads = blockDim.x;
  const int32_t* path = a.path + int64_t(b) * a.max_path;
  const int guess = tid < a.max_path ? path[tid] : 0;  // (in flight with the numbers that say how much of it counts)
  const int L = a.seq_lens[b], n = a.path_lens[b];
  const int64_t drafts = a.cu ? int64_t(a.cu[b + 1]) - a.cu[b] : a.T;
  const int64_t cap = int64_t(a.max_pages) * a.P;
  const int64_t first = L - drafts;
  int err = 0;
  if (L < 0 || L > cap || drafts < 0 || (first < 0 && L > 0))
    err = SPLITKV_DEVERR_SEQLEN;
  else if (L > 0 && (n < 0 || n > drafts || n > a.max_path))
    err = SPLITKV_DEVERR_PATH;
  const int count = err || L == 0 ? 0 : n;  // (a sequence without keys has nothing to keep)
  bool wrong = false;
  for (int i = tid; i < count; i += threads) {
    const int p = i == tid ? guess : path[i];
    wrong = wrong || p < 0 || p >= drafts || (i > 0 && path[i - 1] >= p);
  }
  if (__syncthreads_or(wrong)) err = SPLITKV_DEVERR_PATH;
  const int take = err ? 0 : count;
  if (tid == 0) {
    if (err && a.status) atomicOr(a.status, err);
    a.lens_out[b] = err || L == 0 ? L : int32_t(first) + n;
  }

  const int kc = a.k_row / 16, vc = a.v_row / 16;  // 16-byte columns of a row
  const int k_units = a.Hkv * kc, row_units = k_units + a.Hkv * vc;
  const int64_t head_step = a.nhd ? 1 : a.P;
  const int32_t* table = a.block_table + int64_t(b) * a.max_pages;
  for (int part = 0; part < take; part += kPathPart) {
    const int m = min(kPathPart, take - part);
    __syncthreads();  // (the part before is done)
    for (int i = tid; i < m; i += threads) {
      const int p = path[part + i];
      const int dst = int(first) + part + i, src = int(first) + p;
      int64_t f = -1, t = 0;
      if (src != dst) {
        const int ds = dst / a.P, ss = src / a.P;
        const int dp = table[ds], sp = table[ss];
        if (dp < 0 || dp >= a.num_pages || sp < 0 || sp >= a.num_pages) {
          if (a.status) atomicOr(a.status, SPLITKV_DEVERR_PAGE);
        } else {
          const int64_t page = int64_t(a.Hkv) * a.P, in = a.nhd ? a.Hkv : 1;
          f = sp * page + (src - ss * a.P) * in;
          t = dp * page + (dst - ds * a.P) * in;
        }
      }
      from[i] = f;
      to[i] = t;
      from_slot[i] = src != dst ? src : -1;
    }
    __syncthreads();
    for (int u = tid; u < row_units; u += threads) {
      const bool is_k = u < k_units;
      const int per = is_k ? kc : vc, w = is_k ? u : u - k_units;
      const int head = w / per;
      uint4* pool = static_cast<uint4*>(is_k ? a.k_pages : a.v_pages) + (w - head * per);
      const int64_t at = head * head_step;
      for (int i0 = 0; i0 < m; i0 += kAtOnce) {
        uint4 x[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
          if (i0 + i < m && from[i0 + i] >= 0) x[i] = pool[(from[i0 + i] + at) * per];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
          if (i0 + i < m && from[i0 + i] >= 0) pool[(to[i0 + i] + at) * per] = x[i];
      }
    }
    // the state, by the threads that have no rows first
    for (int u = threads - 1 - tid; u < 2 * a.Hkv; u += threads) {
      uint32_t* state = reinterpret_cast<uint32_t*>(u & 1 ? static_cast<void*>(a.key_positions) : a.key_weights);
      if (state == nullptr) continue;
      state += (int64_t(b) * a.Hkv + (u >> 1)) * cap;
      for (int i0 = 0; i0 < m; i0 += kAtOnce) {
        uint32_t x[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
          if (i0 + i < m && from_slot[i0 + i] >= 0) x[i] = state[from_slot[i0 + i]];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
          if (i0 + i < m && from_slot[i0 + i] >= 0) state[int(first) + part + i0 + i] = x[i];
      }
    }
  }
}

}  // namespace

cudaError_t launch_tree_commit(const CommitArgs& a, void* stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(a.batch), 1, 1);
  // a thread for each column of a token's rows and each state word, within [128, 512]
  const int64_t units = int64_t(a.Hkv) * ((a.k_row + a.v_row) / 16 + 2);
  cfg.blockDim = dim3(unsigned(units <= 128 ? 128 : units >= 512 ? 512 : (units + 31) / 32 * 32), 1, 1);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute la[1];
  la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  la[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = la;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_commit_kernel, a);
}

}  // namespace splitkv
