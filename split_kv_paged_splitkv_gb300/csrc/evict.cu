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
// weight, whose order is that of non-negative floats).  The n-th largest rank
// is found by radix selection in three digits over histograms that the
// cluster's CTAs add up in the shared memory of the first; then prefix sums
// give every freed slot and every moving key its place in the list.
// move_kernel copies the rows, persistent over the groups' lists.
//
// Bound: 8 bytes of state per key read once, 8 written per kept key, each moved
// row read and written once.  Many rows: the moves' bytes (32 sequences x 8
// heads of up to 131k keys cut to 16k: 220 us, of which the moves take 150 at
// 5.8 TB/s of scattered 256-byte rows; floor 136).  One sequence: the chain of
// barriers and passes of the selection: each of up to five passes over the ranks
// is a chain of shared-memory reads and shuffles, and a digit's exchange within
// the cluster takes 2 us whatever its size (64k latent rows: 24.1 us, floor 2.2;
// 5.9k keys of 2 heads: 12.1 us, of which two dependent launches take about 4).
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"

namespace splitkv {
namespace {

using namespace ptx;
namespace cg = cooperative_groups;

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBatch = 4;              // 16-byte vectors a lane loads at a time
constexpr int kBins = 2048;            // 11-bit digits: bits 31-21, 20-10, and 9-0
constexpr int kAlike = 2048;           // ranks set aside for the third digit
constexpr int kMaxCluster = 8;
// Ranks a CTA keeps in shared memory; a CTA with more slots makes them anew in
// each pass, from the L2: 64k latent rows, 8192 a CTA, 24.1 us (29.4 with none
// kept); 256 groups of up to 131k keys, whose CTAs have more, 219.7 us (218.5
// with all kept, in 176 KB and at one CTA per SM).
constexpr int kRankCap = 8192;
constexpr int kMoveThreads = 128, kMovePerSm = 8;
constexpr int kFewBatch = 16, kManyBatch = 32;  // moves a CTA takes at a time
constexpr int kMoveGroups = 1024;      // groups whose prefix a CTA holds at a time

// Rows of the pools that a batch of moves reads and writes.
template <int N>
struct Rows {
  int64_t from[N], to[N];  // from < 0: not moved
};

// Thread m < count looks up move `begin + m` of a group and moves its state.
template <int N>
__device__ __forceinline__ void look_up(const EvictArgs& a, int grp, int begin, int count, Rows<N>& rows) {
  if (int(threadIdx.x) >= count) return;
  const int b = grp / a.Hkv, h = grp - b * a.Hkv;
  const int32_t* src = a.moves + size_t(grp) * 2 * a.max_moves + begin;
  const int s = src[threadIdx.x], d = src[a.max_moves + threadIdx.x];
  const int32_t* trow = a.block_table + size_t(b) * a.max_pages;
  const int sp = s / a.P, dp = d / a.P;
  const int sph = trow[sp], dph = trow[dp];
  const size_t st = size_t(grp) * (size_t(a.max_pages) * a.P);
  a.w_out[st + d] = a.w_in[st + s];
  if (a.pos_out) a.pos_out[st + d] = a.pos_in[st + s];
  auto line = [&](int ph, int in) -> int64_t {
    return a.nhd ? (int64_t(ph) * a.P + in) * a.Hkv + h : (int64_t(ph) * a.Hkv + h) * a.P + in;
  };
  const bool ok = sph >= 0 && sph < a.num_pages && dph >= 0 && dph < a.num_pages;
  if (!ok && a.status) atomicOr(a.status, SPLITKV_DEVERR_PAGE);
  rows.from[threadIdx.x] = ok ? line(sph, s - sp * a.P) : -1;
  rows.to[threadIdx.x] = ok ? line(dph, d - dp * a.P) : 0;
}

// NT threads copy the rows of a batch; `meanwhile` runs once with the first
// rows in flight.
template <int NT, int UNROLL, int N, class F>
__device__ __forceinline__ void copy_rows(const EvictArgs& a, const Rows<N>& rows, int count, F&& meanwhile) {
  const int nk = a.k_row >> 4, np = nk + (a.v_row >> 4);  // 16-byte pieces of a key
  const int total = count * np;
  bool met = false;
#pragma unroll 1
  for (int p0 = threadIdx.x; p0 < total || !met; p0 += UNROLL * NT) {
    uint4 x[UNROLL];
    // piece u of this pass: its move, which pool, its byte offset in the row
    auto piece = [&](int u, int& m, bool& is_k) -> size_t {
      const int p = p0 + u * NT;
      m = p / np;
      const int c = p - m * np;
      is_k = c < nk;
      return size_t(is_k ? c : c - nk) << 4;
    };
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      if (p0 + u * NT >= total) break;
      bool is_k;
      int m;
      const size_t off = piece(u, m, is_k);
      const int64_t line = rows.from[m];
      if (line < 0) continue;
      x[u] = *reinterpret_cast<const uint4*>(static_cast<uint8_t*>(is_k ? a.k_pages : a.v_pages) +
                                             line * (is_k ? a.k_row : a.v_row) + off);
    }
    if (!met) {
      meanwhile();
      met = true;
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      if (p0 + u * NT >= total) break;
      bool is_k;
      int m;
      const size_t off = piece(u, m, is_k);
      if (rows.from[m] < 0) continue;
      *reinterpret_cast<uint4*>(static_cast<uint8_t*>(is_k ? a.k_pages : a.v_pages) +
                                rows.to[m] * (is_k ? a.k_row : a.v_row) + off) = x[u];
    }
  }
}

struct SelShared {
  uint32_t hist[kBins];      // this CTA's
  uint32_t total[3][kBins];  // the cluster's, a digit each, in its first CTA
  uint32_t alike[kAlike];    // ranks with the first digit found, for the third
  uint32_t n_alike;          // (more than kAlike: not all are there)
  int32_t warp_max[kSelWarps];
  int2 warp_sum[2][kSelWarps];  // of warps_prefix, in turn
  int32_t pub[4];    // read by the cluster: largest position, equals, holes, movers
  int32_t found[3];  // digit, keys above it, keys of it
};

// Exclusive prefixes over the CTA's warps of two values per warp; `total`
// receives the sums.  Calls use the two rows of `sums` in turn: a row is written
// again only behind the barrier of the call between, which its readers reach.
__device__ __forceinline__ int2 warps_prefix(int2 mine, int warp, int lane, int2* sums, int2* total) {
  if (lane == 0) sums[warp] = mine;
  __syncthreads();
  const int2 v = lane < kSelWarps ? sums[lane] : make_int2(0, 0);
  int2 x = v;
#pragma unroll
  for (int o = 1; o < kSelWarps; o <<= 1) {
    const int y0 = __shfl_up_sync(kFull, x.x, o), y1 = __shfl_up_sync(kFull, x.y, o);
    if (lane >= o) {
      x.x += y0;
      x.y += y1;
    }
  }
  *total = make_int2(__shfl_sync(kFull, x.x, kSelWarps - 1), __shfl_sync(kFull, x.y, kSelWarps - 1));
  return make_int2(__shfl_sync(kFull, x.x - v.x, warp), __shfl_sync(kFull, x.y - v.y, warp));
}

// Sum over the lanes before this one of popcounts of 4-bit masks, in slot
// order (lane, then bit); `total` receives the warp's.
__device__ __forceinline__ int lanes_before(uint32_t bits, int lane, int* total) {
  const unsigned under = (1u << lane) - 1;
  int before = 0, all = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const unsigned m = __ballot_sync(kFull, bits >> e & 1);
    before += __popc(m & under);
    all += __popc(m);
  }
  *total = all;
  return before;
}

__global__ void __launch_bounds__(kSelThreads, 2) select_kernel(const __grid_constant__ EvictArgs a,
                                                                int rank_cap) {
  extern __shared__ __align__(16) uint32_t ranks[];  // of this CTA's slots, if they fit
  __shared__ SelShared sh;
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
  const bool rank_pos = a.sink > 0 || a.recent > 0;
  auto of = [&](auto* mine, int c) {  // the same variable of the cluster's CTA c
    return nc > 1 ? cluster.map_shared_rank(mine, c) : mine;
  };

  // This CTA's slots [lo, hi) and this warp's [wlo, whi): multiples of 4, so
  // that a lane takes four at a time (a row of the state is padded to 16).
  const int per = int(((int64_t(L) + nc - 1) / nc + 3) & ~int64_t(3));
  const int lo = int(min(int64_t(L), int64_t(cr) * per)), hi = int(min(int64_t(L), int64_t(lo) + per));
  const int seg = ((per + kSelWarps - 1) / kSelWarps + 127) & ~127;
  const int wlo = int(min(int64_t(hi), int64_t(lo) + int64_t(warp) * seg));
  const int whi = int(min(int64_t(hi), int64_t(wlo) + seg));
  const bool in_smem = per <= rank_cap;
  const bool stay_all = L <= n;  // (the same for the whole cluster)

  // ---- the state: the largest position, and what stays in its slot handed
  // on (the move kernel fills the slots that are freed)
  int newest = INT32_MIN;
  if (!stay_all || wo != w || po != pos) {
    #pragma unroll 1
    for (int j0 = wlo; j0 < whi; j0 += 128 * kBatch) {
      uint4 x[kBatch];
      int4 y[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int j = j0 + u * 128 + lane * 4;
        if (j >= whi) continue;
        x[u] = *reinterpret_cast<const uint4*>(w + j);
        if (pos) y[u] = *reinterpret_cast<const int4*>(pos + j);
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int j = j0 + u * 128 + lane * 4;
        if (j >= whi) continue;
        if (in_smem && !stay_all) *reinterpret_cast<uint4*>(ranks + (j - lo)) = x[u];
        const int32_t ys[4] = {y[u].x, y[u].y, y[u].z, y[u].w};
        if (pos) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (j + e < whi) newest = max(newest, ys[e]);
        }
        if (j + 4 <= n) {
          if (wo != w) *reinterpret_cast<uint4*>(wo + j) = x[u];
          if (po != pos) *reinterpret_cast<int4*>(po + j) = y[u];
        } else if (j < n) {
          const uint32_t xs[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (j + e < n) {
              if (wo != w) wo[j + e] = __uint_as_float(xs[e]);
              if (po != pos) po[j + e] = ys[e];
            }
        }
      }
    }
  }
  if (stay_all) {
    if (cr == 0 && threadIdx.x == 0) {
      a.meta[2 * group] = 0;
      a.meta[2 * group + 1] = bad ? raw : n;
    }
    return;
  }
  for (int i = threadIdx.x; i < (cr == 0 ? 4 : 1) * (kBins / 4); i += kSelThreads)  // (hist, then total)
    reinterpret_cast<uint4*>(sh.hist)[i] = make_uint4(0, 0, 0, 0);
  if (threadIdx.x == 0) sh.n_alike = 0;
  newest = __reduce_max_sync(kFull, newest);
  if (lane == 0) sh.warp_max[warp] = newest;
  __syncthreads();
  newest = __reduce_max_sync(kFull, sh.warp_max[lane % kSelWarps]);
  if (nc > 1) {
    if (threadIdx.x == 0) sh.pub[0] = newest;
    cluster.sync();  // (the cleared totals, too)
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c)
      if (c < nc) newest = max(newest, of(sh.pub, c)[0]);
  }
  const int64_t after = int64_t(newest) - a.recent;  // protected: positions beyond it

  // The rank of a weight and its position; negative weights and NaN count as 0.
  auto rank = [&](uint32_t bits, int32_t p) -> uint32_t {
    uint32_t v = __uint_as_float(bits) > 0.f ? bits : 0u;
    if (rank_pos && (p < a.sink || int64_t(p) > after)) v |= 0x80000000u;
    return v;
  };
  auto ranks_at = [&](int j, uint4 x) -> uint4 {  // x: the weights of slots j .. j + 3
    int4 y = make_int4(0, 0, 0, 0);
    if (rank_pos) y = *reinterpret_cast<const int4*>(pos + j);
    return make_uint4(rank(x.x, y.x), rank(x.y, y.y), rank(x.z, y.z), rank(x.w, y.w));
  };
  // Visits this warp's slots in order, four to a lane: body(first slot of the
  // lane, ranks, mask of its slots that exist).
  auto visit = [&](auto&& body) {
#pragma unroll 1
    for (int j0 = wlo; j0 < whi; j0 += 128) {
      const int j = j0 + lane * 4;
      uint4 x = make_uint4(0, 0, 0, 0);
      uint32_t live = 0;
      if (j < whi) {
        x = in_smem ? *reinterpret_cast<const uint4*>(ranks + (j - lo))
                    : ranks_at(j, *reinterpret_cast<const uint4*>(w + j));
        live = whi - j >= 4 ? 15u : (1u << (whi - j)) - 1;
      }
      const uint32_t r[4] = {x.x, x.y, x.z, x.w};
      body(j, r, live);
    }
  };

  // ---- radix selection: the n-th largest rank T, `above` keys beyond it
  uint32_t T = 0;  // the digits found so far
  int above = 0, turn = 0;  // turn: of warps_prefix
#pragma unroll 1  // (code that runs once waits for its instructions)
  for (int d = 0; d < 3; ++d) {
    const int shift = d == 0 ? 21 : d == 1 ? 10 : 0;
    const int bits = d == 2 ? 10 : 11, nbins = 1 << bits;
    const uint32_t mask = d == 0 ? 0u : ~0u << (shift + bits);
    // Thread i has the kPer bins from nbins - kPer * (i + 1) on.
    constexpr int kPer = kBins / kSelThreads;
    static_assert(kPer == 4, "a vector of bins");
    const int low = nbins - kPer * (int(threadIdx.x) + 1);
    uint32_t* hist = sh.hist;
    // Counts four ranks of each lane; with the second digit, those that share
    // the first are put aside, so that the third need not look at all again.
    auto tally = [&](const uint32_t (&r)[4], uint32_t live) {
      // equal ranks throughout the warp's 128 slots: one addition
      const uint32_t r0 = __shfl_sync(kFull, r[0], 0);
      const bool same = live == 15u && r[0] == r0 && r[1] == r0 && r[2] == r0 && r[3] == r0;
      if (__all_sync(kFull, same)) {
        if (lane == 0 && (r0 & mask) == T) {
          atomicAdd(hist + ((r0 >> shift) & (nbins - 1)), 128u);
          if (d == 1) atomicAdd(&sh.n_alike, uint32_t(kAlike + 1));
        }
        return;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if ((live >> e & 1) && (r[e] & mask) == T) {
          atomicAdd(hist + ((r[e] >> shift) & (nbins - 1)), 1u);
          if (d == 1) {
            const uint32_t at = atomicAdd(&sh.n_alike, 1u);
            if (at < kAlike) sh.alike[at] = r[e];
          }
        }
    };
    if (d == 0 && in_smem) {
      // the weights in shared memory become ranks (a lane's own slots: no barrier)
#pragma unroll 1
      for (int j0 = wlo; j0 < whi; j0 += 128 * kBatch) {
        int4 y[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int j = j0 + u * 128 + lane * 4;
          y[u] = make_int4(0, 0, 0, 0);
          if (rank_pos && j < whi) y[u] = *reinterpret_cast<const int4*>(pos + j);
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          if (j0 + u * 128 >= whi) break;  // (the same for the warp)
          const int j = j0 + u * 128 + lane * 4;
          uint4 x = make_uint4(0, 0, 0, 0);
          if (j < whi) {
            x = *reinterpret_cast<const uint4*>(ranks + (j - lo));
            x = make_uint4(rank(x.x, y[u].x), rank(x.y, y[u].y), rank(x.z, y[u].z), rank(x.w, y[u].w));
            *reinterpret_cast<uint4*>(ranks + (j - lo)) = x;
          }
          const uint32_t r[4] = {x.x, x.y, x.z, x.w};
          tally(r, j >= whi ? 0u : whi - j >= 4 ? 15u : (1u << (whi - j)) - 1);
        }
      }
    } else if (d == 2 && sh.n_alike <= kAlike) {
      for (uint32_t i = threadIdx.x; i < sh.n_alike; i += kSelThreads)
        if ((sh.alike[i] & mask) == T) atomicAdd(hist + (sh.alike[i] & (nbins - 1)), 1u);
    } else {
      visit([&](int, const uint32_t (&r)[4], uint32_t live) { tally(r, live); });
    }
    __syncthreads();
    // This CTA's counts (of few bins) into the first CTA's sums, which all read.
    uint4 v = make_uint4(0, 0, 0, 0);
    if (low >= 0) {
      v = *reinterpret_cast<const uint4*>(hist + low);
      if (d < 2) *reinterpret_cast<uint4*>(hist + low) = make_uint4(0, 0, 0, 0);  // (for the next digit)
    }
    if (nc > 1) {
      uint32_t* total = cluster.map_shared_rank(sh.total[d], 0);
      if (v.x) atomicAdd(total + low, v.x);
      if (v.y) atomicAdd(total + low + 1, v.y);
      if (v.z) atomicAdd(total + low + 2, v.z);
      if (v.w) atomicAdd(total + low + 3, v.w);
      cluster.sync();
      if (low >= 0) v = *reinterpret_cast<const uint4*>(total + low);
    }
    const int c[kPer] = {int(v.w), int(v.z), int(v.y), int(v.x)};  // from the highest bin down
    const int sum = (c[0] + c[1]) + (c[2] + c[3]);
    int x = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, x, o);
      if (lane >= o) x += y;
    }
    int2 all;
    int start = above + x - sum +
                warps_prefix(make_int2(__shfl_sync(kFull, x, 31), 0), warp, lane, sh.warp_sum[turn++ & 1], &all).x;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {  // `start`: keys above this bin
      if (start < n && start + c[e] >= n) {
        sh.found[0] = low + kPer - 1 - e;
        sh.found[1] = start;
        sh.found[2] = c[e];
      }
      start += c[e];
    }
    __syncthreads();
    T |= uint32_t(sh.found[0]) << shift;
    above = sh.found[1];
    // all keys that share the digits so far stay: the other digits do not matter
    // (5.9k keys of 2 heads: 12.3 us, 13.6 without)
    if (above + sh.found[2] == n) break;
  }
  const int need = n - above;  // keys of rank T that stay: the lowest slots
  const bool ties = need < sh.found[2];

  // ---- keys of rank T before this warp's slots, if not all of them stay
  int eq_at = 0;
  if (ties) {
    int eq = 0;
    int2 eq_cta;
    visit([&](int, const uint32_t (&r)[4], uint32_t live) {
#pragma unroll
      for (int e = 0; e < 4; ++e) eq += (live >> e & 1) && r[e] == T;
    });
    eq_at = warps_prefix(make_int2(__reduce_add_sync(kFull, eq), 0), warp, lane, sh.warp_sum[turn++ & 1], &eq_cta).x;
    if (nc > 1) {
      if (threadIdx.x == 0) sh.pub[1] = eq_cta.x;
      cluster.sync();
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c)
        if (c < cr) eq_at += of(sh.pub, c)[1];
    }
  }

  // ---- what is freed below slot n and what moves from behind it
  auto changes = [&](auto&& body) {
    int seen = eq_at;
    visit([&](int j, const uint32_t (&r)[4], uint32_t live) {
      uint32_t stay = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) stay |= uint32_t(ties ? r[e] > T : r[e] >= T) << e;
      if (ties) {
        uint32_t same = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) same |= uint32_t(r[e] == T) << e;
        same &= live;
        int all, at = seen + lanes_before(same, lane, &all);
        seen += all;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (same >> e & 1) stay |= uint32_t(at++ < need) << e;
      }
      const uint32_t below = j >= n ? 0u : n - j >= 4 ? 15u : (1u << (n - j)) - 1;
      body(j, ~stay & below & live, stay & ~below & live);
    });
  };
  int holes = 0, movers = 0;
  changes([&](int, uint32_t hole, uint32_t mover) {
    holes += __popc(hole);
    movers += __popc(mover);
  });
  int2 cta;
  const int2 at = warps_prefix(make_int2(__reduce_add_sync(kFull, holes), __reduce_add_sync(kFull, movers)), warp, lane,
                               sh.warp_sum[turn & 1], &cta);
  int hole_at = at.x, mover_at = at.y, moves = cta.y;
  if (nc > 1) {
    if (threadIdx.x == 0) {
      sh.pub[2] = cta.x;
      sh.pub[3] = cta.y;
    }
    cluster.sync();
    moves = 0;
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c) {
      if (c >= nc) break;
      const int32_t* p = of(sh.pub, c);
      const int ho = p[2], mo = p[3];
      hole_at += c < cr ? ho : 0;
      mover_at += c < cr ? mo : 0;
      moves += mo;
    }
    cluster.barrier_arrive();  // (this CTA reads no more of the others')
  }
  int32_t* src = a.moves + size_t(group) * 2 * a.max_moves;
  int32_t* dst = src + a.max_moves;
  changes([&](int j, uint32_t hole, uint32_t mover) {
    if (__any_sync(kFull, hole)) {
      int all, at = hole_at + lanes_before(hole, lane, &all);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (hole >> e & 1) dst[at++] = j + e;
      hole_at += all;
    }
    if (__any_sync(kFull, mover)) {
      int all, at = mover_at + lanes_before(mover, lane, &all);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (mover >> e & 1) src[at++] = j + e;
      mover_at += all;
    }
  });
  if (cr == 0 && threadIdx.x == 0) {
    a.meta[2 * group] = moves;
    a.meta[2 * group + 1] = n;
  }
  if (nc > 1) cluster.barrier_wait();  // no CTA leaves while another reads its shared memory
}

// The moves of all groups, in batches of BATCH moves of one group; the
// batches form one line of which a CTA takes every gridDim.x-th.  While the
// rows of a batch are in flight, the first threads look up the next one's.
template <int BATCH, int UNROLL>
__global__ void __launch_bounds__(kMoveThreads, kMovePerSm) move_kernel(const __grid_constant__ EvictArgs a) {
  __shared__ int32_t upto[kMoveGroups];  // batches of the groups up to and with this one
  __shared__ int32_t part[kMoveThreads / 32];
  __shared__ Rows<BATCH> rows[2];
  __shared__ int32_t count[2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  launch_dependents();
  wait_prerequisites();
  const int groups = a.batch * a.Hkv;
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < a.batch; b += kMoveThreads) a.lens_out[b] = a.meta[2 * (b * a.Hkv) + 1];

  int64_t passed = 0;  // batches of the groups before g0
  for (int g0 = 0; g0 < groups; g0 += kMoveGroups) {
    const int ng = min(kMoveGroups, groups - g0);
    constexpr int PT = kMoveGroups / kMoveThreads;
    int mine[PT], sum = 0;
#pragma unroll
    for (int i = 0; i < PT; ++i) {
      const int g = int(threadIdx.x) * PT + i;
      mine[i] = g < ng ? (a.meta[2 * (g0 + g)] + BATCH - 1) / BATCH : 0;
      sum += mine[i];
    }
    int x = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) part[warp] = x;
    __syncthreads();
    int at = x - sum, all = 0;
#pragma unroll
    for (int i = 0; i < kMoveThreads / 32; ++i) {
      if (i < warp) at += part[i];
      all += part[i];
    }
#pragma unroll
    for (int i = 0; i < PT; ++i) {
      at += mine[i];
      upto[threadIdx.x * PT + i] = at;
    }
    __syncthreads();

    // looks up batch `i` of this stretch of groups
    auto find = [&](int i, int buf) {
      if (threadIdx.x >= BATCH || i >= all) return;
      int l = 0, r = ng - 1;  // the first group whose batches reach past i
      while (l < r) {
        const int m = (l + r) >> 1;
        if (upto[m] > i) r = m; else l = m + 1;
      }
      const int grp = g0 + l, begin = (i - (l ? upto[l - 1] : 0)) * BATCH;
      const int c = min(BATCH, a.meta[2 * grp] - begin);
      if (threadIdx.x == 0) count[buf] = c;
      look_up(a, grp, begin, c, rows[buf]);
    };

    int64_t skip = (int64_t(blockIdx.x) - passed) % int64_t(gridDim.x);
    int i = int(skip < 0 ? skip + gridDim.x : skip);
    int buf = 0;
    find(i, buf);
    __syncthreads();
    for (; i < all; i += gridDim.x, buf ^= 1) {
      copy_rows<kMoveThreads, UNROLL>(a, rows[buf], count[buf], [&]() { find(i + int(gridDim.x), buf ^ 1); });
      __syncthreads();
    }
    passed += all;
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t cap = int64_t(a.max_pages) * a.P;
  const int groups = a.batch * a.Hkv;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // CTAs per (sequence, head): one for each 2048 slots of capacity while the
  // groups do not fill the GPU, and one for each 32,768 slots in any case.
  // 5.9k slots of 2 heads: 12.2 us with four, 14.1 with eight, and 12.2 with one
  // too, whose longer passes cost what it saves in exchanges;
  // 64k slots of one: 24.1 with eight, 39 with four, 58 with two, and 2 more
  // with sixteen than with eight; 256 groups of 131k: 219.7 with four, 229 with
  // eight, 255 with two.
  int nc = 1;
  while (nc < kMaxCluster && ((cap > int64_t(nc) * 2048 && int64_t(groups) * nc * 2 <= int64_t(sms) * 4) ||
                              cap > int64_t(nc) * 32768))
    nc *= 2;
  const int64_t per = ((cap + nc - 1) / nc + 3) & ~int64_t(3);
  const int rank_cap = int(per <= kRankCap ? per : kRankCap);
  static std::atomic<uint64_t> allowed{0};
  e = allow_shared_memory(reinterpret_cast<const void*>(select_kernel), kRankCap * 4, allowed);
  if (e != cudaSuccess) return e;

  cudaLaunchAttribute la[2];
  la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  la[0].val.programmaticStreamSerializationAllowed = 1;
  la[1].id = cudaLaunchAttributeClusterDimension;
  la[1].val.clusterDim.x = nc;
  la[1].val.clusterDim.y = la[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(groups) * nc, 1, 1);
  cfg.blockDim = dim3(kSelThreads, 1, 1);
  cfg.dynamicSmemBytes = size_t(rank_cap) * 4;
  cfg.stream = s;
  cfg.attrs = la;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, select_kernel, a, rank_cap);
  if (e != cudaSuccess) return e;

  cudaLaunchConfig_t mv = {};
  mv.stream = s;
  mv.attrs = la;
  mv.numAttrs = 1;
  mv.blockDim = dim3(kMoveThreads, 1, 1);
  // Eight small CTAs per SM, so that some load while others wait at a barrier
  // (840k pairs of 256-byte rows: 219.4 us; four of 256 threads 223.7).  Few
  // moves go in small batches, so that more SMs take part (2.7k of those pairs:
  // 12.2 us in batches of 16, 13.3 of 32; 12k rows of 576 bytes: 24.1 and 25.6),
  // many in large ones, for bytes in flight.
  const bool few = int64_t(groups) * a.max_moves <= int64_t(sms) * 256;
  const int batch = few ? kFewBatch : kManyBatch;
  const int64_t most = int64_t(groups) * ((a.max_moves + batch - 1) / batch);
  const int64_t grid = most < int64_t(sms) * kMovePerSm ? (most > 0 ? most : 1) : int64_t(sms) * kMovePerSm;
  mv.gridDim = dim3(unsigned(grid), 1, 1);
  return few ? cudaLaunchKernelEx(&mv, move_kernel<kFewBatch, kFewBatch / 4>, a)
             : cudaLaunchKernelEx(&mv, move_kernel<kManyBatch, kManyBatch / 4>, a);
}

}  // namespace splitkv
