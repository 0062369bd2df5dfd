// Eviction from a paged cache by accumulated attention weight, sm_103a.
//
// Per sequence b and KV head h, with L = seq_lens[b] keys and n = min(L,
// budget): the keys are ranked by (protected, weight), ties to the lowest
// slot, and the n best stay.  Protected are the keys whose position is below
// `sink` or among the last `recent` positions (above the largest position
// minus `recent`).  Kept keys in slots >= n move, in order, into the slots
// < n of the keys that go: the i-th such key into the i-th such slot.
//
// Why moves and not a compaction that keeps the order: attention does not
// depend on the order of the keys, every source lies at or behind slot n and
// every destination before it, so all moves are independent of one another
// (no scratch copy, no order between CTAs), and no row is moved that could
// stay.  Keeping the order would move nearly every kept row.
//
// Two kernels.  select_kernel: one cluster per (sequence, head); the rank of
// a key is a 32-bit number (protected in the top bit, then the bits of the
// weight, whose order is that of non-negative floats), its n-th largest value
// is found by radix selection in three digits over histograms that the
// cluster's CTAs read from one another's shared memory; then ballots and
// prefix sums give every freed slot and every moving key its place in the
// list.  move_kernel copies the rows, persistent over the groups' lists.
// Bound: 8 bytes of state per key read once (the ranks stay in shared
// memory), 8 written per kept key, each moved row read and written once.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"

namespace splitkv {
namespace {

using namespace ptx;
namespace cg = cooperative_groups;

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;            // 11-bit digits: bits 31-21, 20-10, and 9-0
constexpr int kMaxCluster = 8;
constexpr int kRankCap = 40960;        // ranks a CTA keeps in shared memory (160 KB)
constexpr int kMoveThreads = 256;
constexpr int kMoveBatch = 32;         // moves a CTA takes at a time

struct SelShared {
  uint32_t hist[2][kBins];  // by turns, so that one cluster barrier per digit suffices
  int32_t warp_sum[kSelWarps];
  int32_t pub[4];   // read by the cluster: largest position, equals, holes, movers
  int32_t found[2]; // digit, keys above it
};

// Exclusive prefix sum of one int per warp; returns the block total.
__device__ __forceinline__ int warp_prefix(int mine, int warp, int lane, int32_t* sums, int* before) {
  __syncthreads();
  if (lane == 0) sums[warp] = mine;
  __syncthreads();
  const int v = sums[lane];
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  *before = __shfl_sync(kFull, x - v, warp);
  return __shfl_sync(kFull, x, 31);
}

__global__ void __launch_bounds__(kSelThreads, 1) select_kernel(const __grid_constant__ EvictArgs a,
                                                                int rank_cap) {
  extern __shared__ __align__(16) uint8_t smem[];
  SelShared& sh = *reinterpret_cast<SelShared*>(smem);
  uint32_t* ranks = reinterpret_cast<uint32_t*>(smem + sizeof(SelShared));
  cg::cluster_group cluster = cg::this_cluster();
  const int nc = cluster.num_blocks(), cr = cluster.block_rank();
  const int group = blockIdx.x / nc;
  const int b = group / a.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  launch_dependents();
  wait_prerequisites();
  const size_t cap = size_t(a.max_pages) * a.P;
  const int raw = a.seq_lens[b];
  const bool bad = raw < 0 || raw > int64_t(cap);
  if (bad && cr == 0 && threadIdx.x == 0 && a.status) atomicOr(a.status, SPLITKV_DEVERR_SEQLEN);
  const int L = bad ? 0 : raw;
  const int n = min(L, a.budget);
  const float* w = a.w_in + size_t(group) * cap;
  const int32_t* pos = a.pos_in ? a.pos_in + size_t(group) * cap : nullptr;
  float* wo = a.w_out + size_t(group) * cap;
  int32_t* po = a.pos_out ? a.pos_out + size_t(group) * cap : nullptr;
  const bool copy_w = wo != w, copy_p = po && po != pos;

  // this CTA's slots [lo, hi), this warp's [wlo, whi); multiples of 32
  const int per = int(((int64_t(L) + nc - 1) / nc + 31) & ~int64_t(31));
  const int lo = int(min(int64_t(L), int64_t(cr) * per)), hi = int(min(int64_t(L), int64_t(lo) + per));
  const int seg = ((per + kSelWarps - 1) / kSelWarps + 31) & ~31;
  const int wlo = int(min(int64_t(hi), int64_t(lo) + int64_t(warp) * seg));
  const int whi = int(min(int64_t(hi), int64_t(wlo) + seg));

  if (L <= n) {  // everything stays (the same for the whole cluster)
    for (int j = lo + threadIdx.x; j < hi; j += kSelThreads) {
      if (copy_w) wo[j] = w[j];
      if (copy_p) po[j] = pos[j];
    }
    if (cr == 0 && threadIdx.x == 0) {
      a.meta[2 * group] = 0;
      a.meta[2 * group + 1] = bad ? raw : n;
    }
    return;
  }

  // ---- the largest position
  int64_t newest = INT64_MIN;
  if (pos) {
    int m = INT32_MIN;
    for (int j = lo + threadIdx.x; j < hi; j += kSelThreads) m = max(m, pos[j]);
    m = __reduce_max_sync(kFull, m);
    if (lane == 0) sh.warp_sum[warp] = m;
    __syncthreads();
    if (warp == 0) {
      m = __reduce_max_sync(kFull, sh.warp_sum[lane]);
      if (lane == 0) sh.pub[0] = m;
    }
    cluster.sync();
    m = INT32_MIN;
    for (int c = 0; c < nc; ++c) m = max(m, cluster.map_shared_rank(sh.pub, c)[0]);
    newest = m;
  }
  auto rank_at = [&](int j) -> uint32_t {
    const float x = w[j];
    uint32_t r = x > 0.f ? __float_as_uint(x) : 0u;  // negative and NaN count as 0
    if (pos) {
      const int32_t p = pos[j];
      if (p < a.sink || int64_t(p) > newest - a.recent) r |= 0x80000000u;
    }
    return r;
  };
  const bool kept_in_smem = per <= rank_cap;
  auto rank_of = [&](int j) { return kept_in_smem ? ranks[j - lo] : rank_at(j); };

  // ---- radix selection: the n-th largest rank T, `above` keys beyond it
  uint32_t prefix = 0;  // digits found so far
  int above = 0;
  for (int d = 0; d < 3; ++d) {
    uint32_t* hist = sh.hist[d & 1];
    const int shift = d == 0 ? 21 : d == 1 ? 10 : 0;
    const int bits = d == 2 ? 10 : 11, nbins = 1 << bits;
    const uint32_t mask = d == 0 ? 0u : ~0u << (shift + bits);
    for (int i = threadIdx.x; i < kBins; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    for (int j0 = lo; j0 < hi; j0 += kSelThreads) {
      const int j = j0 + threadIdx.x;
      bool in = j < hi;
      uint32_t r = 0;
      if (in) {
        if (d == 0) {
          r = rank_at(j);
          if (kept_in_smem) ranks[j - lo] = r;
        } else {
          r = rank_of(j);
        }
        in = (r & mask) == prefix;
      }
      const int bin = in ? int((r >> shift) & (nbins - 1)) : -1;
      // one bin for the whole warp (equal weights): one addition
      const int lead = __shfl_sync(kFull, bin, 0);
      if (__all_sync(kFull, bin == lead)) {
        if (lane == 0 && lead >= 0) atomicAdd(hist + lead, 32u);
      } else if (bin >= 0) {
        atomicAdd(hist + bin, 1u);
      }
    }
    cluster.sync();
    // Every CTA sums the cluster's histograms from the top: thread i holds
    // bins nbins - 1 - 2 i and the one below it.
    const int top = nbins - 1 - 2 * int(threadIdx.x);
    int c0 = 0, c1 = 0;
    if (top >= 1) {
      for (int c = 0; c < nc; ++c) {
        const uint32_t* g = cluster.map_shared_rank(hist, c);
        c0 += int(g[top]);
        c1 += int(g[top - 1]);
      }
    }
    const int sum = c0 + c1;
    int x = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, x, o);
      if (lane >= o) x += y;
    }
    int before;
    warp_prefix(__shfl_sync(kFull, x, 31), warp, lane, sh.warp_sum, &before);
    const int start = above + before + x - sum;  // keys above this thread's bins
    if (top >= 1) {
      if (start < n && start + c0 >= n) {
        sh.found[0] = top;
        sh.found[1] = start;
      } else if (start + c0 < n && start + sum >= n) {
        sh.found[0] = top - 1;
        sh.found[1] = start + c0;
      }
    }
    __syncthreads();
    prefix |= uint32_t(sh.found[0]) << shift;
    above = sh.found[1];
    __syncthreads();
  }
  const uint32_t T = prefix;
  const int need = n - above;  // keys of rank T that stay: the lowest slots

  // ---- equals before this warp's slots
  int eq = 0;
  for (int j0 = wlo; j0 < whi; j0 += 32) {
    const int j = j0 + lane;
    eq += __popc(__ballot_sync(kFull, j < whi && rank_of(j) == T));
  }
  int eq_before;
  const int eq_cta = warp_prefix(eq, warp, lane, sh.warp_sum, &eq_before);
  if (threadIdx.x == 0) sh.pub[1] = eq_cta;
  cluster.sync();
  for (int c = 0; c < cr; ++c) eq_before += cluster.map_shared_rank(sh.pub, c)[1];

  // ---- what stays, 32 slots at a time
  auto walk = [&](auto&& visit) {
    int seen = eq_before;
    for (int j0 = wlo; j0 < whi; j0 += 32) {
      const int j = j0 + lane;
      const uint32_t r = j < whi ? rank_of(j) : 0u;
      const unsigned same = __ballot_sync(kFull, j < whi && r == T);
      const bool stays = j < whi && (r > T || (r == T && seen + __popc(same & ((1u << lane) - 1)) < need));
      seen += __popc(same);
      visit(j, stays);
    }
  };
  int holes = 0, movers = 0;
  walk([&](int j, bool stays) {
    holes += __popc(__ballot_sync(kFull, j < min(whi, n) && !stays));
    movers += __popc(__ballot_sync(kFull, j >= n && stays));
  });
  int hole_at, mover_at;
  const int holes_cta = warp_prefix(holes, warp, lane, sh.warp_sum, &hole_at);
  const int movers_cta = warp_prefix(movers, warp, lane, sh.warp_sum, &mover_at);
  if (threadIdx.x == 0) {
    sh.pub[2] = holes_cta;
    sh.pub[3] = movers_cta;
  }
  cluster.sync();
  int moves = 0;
  for (int c = 0; c < nc; ++c) {
    const int32_t* p = cluster.map_shared_rank(sh.pub, c);
    if (c < cr) {
      hole_at += p[2];
      mover_at += p[3];
    }
    moves += p[3];
  }
  int32_t* src = a.moves + size_t(group) * 2 * a.max_moves;
  int32_t* dst = src + a.max_moves;
  walk([&](int j, bool stays) {
    const bool hole = j < min(whi, n) && !stays, mover = j >= n && stays;
    const unsigned hb = __ballot_sync(kFull, hole), mb = __ballot_sync(kFull, mover);
    const unsigned under = (1u << lane) - 1;
    if (hole) dst[hole_at + __popc(hb & under)] = j;
    if (mover) src[mover_at + __popc(mb & under)] = j;
    hole_at += __popc(hb);
    mover_at += __popc(mb);
    if (stays && j < n) {
      if (copy_w) wo[j] = w[j];
      if (copy_p) po[j] = pos[j];
    }
  });
  if (cr == 0 && threadIdx.x == 0) {
    a.meta[2 * group] = moves;
    a.meta[2 * group + 1] = n;
  }
  cluster.sync();  // no CTA leaves while another reads its shared memory
}

__global__ void __launch_bounds__(kMoveThreads) move_kernel(const __grid_constant__ EvictArgs a) {
  __shared__ int64_t from[kMoveBatch], to[kMoveBatch];  // rows of the pools; from < 0: not moved
  __shared__ int32_t part[kMoveThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  launch_dependents();
  wait_prerequisites();
  const int groups = a.batch * a.Hkv;
  const size_t cap = size_t(a.max_pages) * a.P;
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < a.batch; b += kMoveThreads) a.lens_out[b] = a.meta[2 * (b * a.Hkv) + 1];

  // The batches of all groups form one line; this CTA takes every gridDim.x-th.
  int64_t want = blockIdx.x, passed = 0;
  for (int g0 = 0; g0 < groups; g0 += kMoveThreads) {
    const int g = g0 + threadIdx.x;
    const int mine = g < groups ? (a.meta[2 * g] + kMoveBatch - 1) / kMoveBatch : 0;
    int x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) part[warp] = x;
    __syncthreads();
    int64_t upto = passed + x, all = passed;
    for (int i = 0; i < kMoveThreads / 32; ++i) {
      if (i < warp) upto += part[i];
      all += part[i];
    }
    // the thread whose group holds batch `want` announces it
    __shared__ int32_t cur[2];
    while (want < all) {
      if (want < upto && want >= upto - mine) {
        cur[0] = g;
        cur[1] = int(want - (upto - mine));
      }
      __syncthreads();
      const int grp = cur[0], first = cur[1] * kMoveBatch;
      const int b = grp / a.Hkv, h = grp - b * a.Hkv;
      const int count = min(kMoveBatch, a.meta[2 * grp] - first);
      if (threadIdx.x < count) {
        const int32_t* src = a.moves + size_t(grp) * 2 * a.max_moves + first;
        const int s = src[threadIdx.x], d = src[a.max_moves + threadIdx.x];
        const int32_t* trow = a.block_table + size_t(b) * a.max_pages;
        auto line = [&](int j) -> int64_t {
          const int lp = j / a.P, ph = trow[lp], in = j - lp * a.P;
          if (ph < 0 || ph >= a.num_pages) return -1;
          return a.nhd ? (int64_t(ph) * a.P + in) * a.Hkv + h : (int64_t(ph) * a.Hkv + h) * a.P + in;
        };
        const int64_t ls = line(s), ld = line(d);
        if ((ls < 0 || ld < 0) && a.status) atomicOr(a.status, SPLITKV_DEVERR_PAGE);
        from[threadIdx.x] = ld < 0 ? -1 : ls;
        to[threadIdx.x] = ld;
        const size_t st = size_t(grp) * cap;
        a.w_out[st + d] = a.w_in[st + s];
        if (a.pos_out) a.pos_out[st + d] = a.pos_in[st + s];
      }
      __syncthreads();
      const int nk = a.k_row >> 4, np = nk + (a.v_row >> 4);  // 16-byte pieces of a key
      for (int p0 = threadIdx.x; p0 < count * np; p0 += 4 * kMoveThreads) {
        uint4 x4[4];
        uint4* out[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int p = p0 + r * kMoveThreads;
          out[r] = nullptr;
          if (p >= count * np) continue;
          const int m = p / np, c = p - m * np;
          if (from[m] < 0) continue;
          const bool is_k = c < nk;
          uint8_t* pool = static_cast<uint8_t*>(is_k ? a.k_pages : a.v_pages);
          const int row = is_k ? a.k_row : a.v_row, off = (is_k ? c : c - nk) << 4;
          x4[r] = *reinterpret_cast<const uint4*>(pool + from[m] * row + off);
          out[r] = reinterpret_cast<uint4*>(pool + to[m] * row + off);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (out[r]) *out[r] = x4[r];
      }
      __syncthreads();
      want += gridDim.x;
    }
    passed = all;
  }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t cap = int64_t(a.max_pages) * a.P;
  const int groups = a.batch * a.Hkv;
  // CTAs per (sequence, head): one for each 8192 slots of capacity, up to 8.
  int nc = 1;
  while (nc < kMaxCluster && cap > int64_t(nc) * 8192) nc *= 2;
  const int64_t per = ((cap + nc - 1) / nc + 31) & ~int64_t(31);
  const int rank_cap = per <= kRankCap ? int(per) : kRankCap;
  const int smem = int(sizeof(SelShared)) + rank_cap * 4;
  static cudaError_t attr = cudaFuncSetAttribute(
      select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(sizeof(SelShared)) + kRankCap * 4);
  if (attr != cudaSuccess) return attr;

  cudaLaunchAttribute la[2];
  la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  la[0].val.programmaticStreamSerializationAllowed = 1;
  la[1].id = cudaLaunchAttributeClusterDimension;
  la[1].val.clusterDim.x = nc;
  la[1].val.clusterDim.y = la[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(groups) * nc, 1, 1);
  cfg.blockDim = dim3(kSelThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = la;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, select_kernel, a, rank_cap);
  if (e != cudaSuccess) return e;

  int dev = 0, sms = 0;
  e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t most = int64_t(groups) * ((a.max_moves + kMoveBatch - 1) / kMoveBatch);
  const int64_t grid = most < int64_t(sms) * 8 ? (most > 0 ? most : 1) : int64_t(sms) * 8;
  cudaLaunchConfig_t mv = {};
  mv.gridDim = dim3(unsigned(grid), 1, 1);
  mv.blockDim = dim3(kMoveThreads, 1, 1);
  mv.stream = s;
  mv.attrs = la;
  mv.numAttrs = 1;
  return cudaLaunchKernelEx(&mv, move_kernel, a);
}

}  // namespace splitkv
