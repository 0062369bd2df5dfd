// Cross attention's kernel (cross_kernel.cuh) without a tree's masks, the merge of the
// partial results of both, and the rules by which their items are dealt.
#include "cross_kernel.cuh"

namespace splitkv {
namespace {

// Joins the partial results of the cut items (an item's pieces have consecutive
// slots).  A unit is 32 rows of an item, a lane each, and all 128 dims or, where there
// are few (a call of one or two trees), a quarter of them; the CTAs take the units of all cut
// items in turn (a CTA for every possible unit would be 1,216, of which most calls
// have no use).  A warp takes every eighth group of four dims, which lie side by side
// for the rows; the log-sum-exps and results of four pieces, of 16 with a quarter of the dims,
// are loaded at once, and the sums rescaled, after every four, when later ones are
// larger.
constexpr int kMergeWarps = 8, kMergeAtOnce = 4;
template <int PARTS>
__device__ __forceinline__ void merge_unit(const CrossArgs& a, const CrossSplit& sp, int r0, int part, uint2 (&rows_out)[32][33]) {
  constexpr int kGroups = 32 / kMergeWarps / PARTS, kDeep = kMergeAtOnce * PARTS;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = r0 + lane, g0 = part * (32 / PARTS) + warp;
  const bool live = row < sp.rows;
  float M = -INFINITY, sum = 0.f;
  float4 acc[kGroups];
#pragma unroll
  for (int i = 0; i < kGroups; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int k1 = 0; k1 < sp.cuts; k1 += kDeep) {
    float ls[kDeep];
    float4 v[kDeep][kGroups];
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      const size_t slot = k1 + k ? (sp.slot & -sp.step) + (k1 + k) * sp.step : sp.slot;
      const bool in = live && k1 + k < sp.cuts;
      ls[k] = in ? a.lse_part[slot * a.part_rows + row] : -INFINITY;
#pragma unroll
      for (int i = 0; i < kGroups; ++i)
        if (in) v[k][i] = reinterpret_cast<const float4*>(a.o_part)[(slot * 32 + g0 + i * kMergeWarps) * a.part_rows + row];
    }
#pragma unroll
    for (int k0 = 0; k0 < kDeep; k0 += kMergeAtOnce) {
      float m = M;
#pragma unroll
      for (int k = k0; k < k0 + kMergeAtOnce; ++k) m = max_nan(m, ls[k]);  // (a NaN piece makes the row NaN)
      if (m == -INFINITY) continue;
      const float old = ex2((M - m) * 1.4426950408889634f);
      M = m;
      sum *= old;
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        acc[i].x *= old;
        acc[i].y *= old;
        acc[i].z *= old;
        acc[i].w *= old;
      }
#pragma unroll
      for (int k = k0; k < k0 + kMergeAtOnce; ++k) {
        if (ls[k] == -INFINITY) continue;  // (a piece that is none, or without weight)
        const float w = ex2((ls[k] - m) * 1.4426950408889634f);
        sum += w;
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
          acc[i].x += w * v[k][i].x;
          acc[i].y += w * v[k][i].y;
          acc[i].z += w * v[k][i].z;
          acc[i].w += w * v[k][i].w;
        }
      }
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  __syncthreads();  // (the rows of the unit before are out)
#pragma unroll
  for (int i = 0; i < kGroups; ++i)
    rows_out[lane][warp + i * kMergeWarps] =
        make_uint2(pack_bf16(acc[i].x * inv, acc[i].y * inv), pack_bf16(acc[i].z * inv, acc[i].w * inv));
  __syncthreads();
  // whole rows (or quarters) out, a warp to PARTS rows
  constexpr int kLanes = 32 / PARTS;
  for (int i = warp * PARTS + lane / kLanes; i < 32 && r0 + i < sp.rows; i += kMergeWarps * PARTS) {
    const int tok = (sp.row0 + r0 + i) / a.G, g = (sp.row0 + r0 + i) - tok * a.G;
    const size_t out_row = (size_t(sp.first) + tok) * a.Hq + size_t(sp.head) * a.G + g;
    reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + out_row * 128)[part * kLanes + lane % kLanes] =
        rows_out[i][lane % kLanes];
  }
  if (warp == 0 && part == 0 && live && a.lse) {
    const int tok = (sp.row0 + row) / a.G, g = (sp.row0 + row) - tok * a.G;
    a.lse[(size_t(sp.first) + tok) * a.Hq + size_t(sp.head) * a.G + g] = sum == 0.f ? -INFINITY : M + lg2(sum) * kLn2;
  }
}

__global__ void __launch_bounds__(kMergeWarps * 32) cross_merge_kernel(const __grid_constant__ CrossArgs a, int units) {
  __shared__ uint2 rows_out[32][33];  // bf16 rows (of 32 pieces of 8 bytes, and one to spread the banks)
  launch_dependents();
  wait_prerequisites();
  const int last = *a.n_split * units;
  if (4 * last <= int(gridDim.x)) {
    const int u = blockIdx.x >> 2, q = u / units, r0 = (u - q * units) * 32;
    if (u >= last) return;
    const CrossSplit sp = a.split[q];
    if (sp.cuts != 0 && r0 < sp.rows) merge_unit<4>(a, sp, r0, blockIdx.x & 3, rows_out);
    return;
  }
  for (int u = blockIdx.x; u < last; u += gridDim.x) {
    const int q = u / units, r0 = (u - q * units) * 32;  // the q-th cut item, its rows from r0 on
    const CrossSplit sp = a.split[q];
    if (sp.cuts == 0 || r0 >= sp.rows) continue;
    merge_unit<1>(a, sp, r0, 0, rows_out);
  }
}

}  // namespace

// Row tiles of a call at most, however its tokens are dealt to the sequences.
int64_t cross_row_tiles(const splitkv_desc_t& d, int64_t n_tokens) {
  const int64_t G = d.num_q_heads / d.num_kv_heads;
  const int64_t full = n_tokens * G / Cross::ROWS, some = n_tokens < d.batch ? n_tokens : d.batch;
  return full + some;
}

// How the items are dealt.  Few: pieces of a cost.  Many of few rows (half a tile
// a sequence, on average): a line, so that a CTA's K and V keep coming while it goes
// from one item to the next (one token of 512 requests, 8 heads, 512 keys: 218 us,
// a CTA per item 309).  Many of more rows: a CTA per item, for its results pass
// through the shared memory that the next item's queries need (80 prompts of 40
// to 80 tokens, 32 heads on 8, 512 keys: 84 us, as a line 99; trees of 64 young
// requests 44 and 51; prompts of 4k tokens the same either way).
CrossDeal cross_deal(const splitkv_desc_t& d, int64_t n_tokens) {
  if (cross_row_tiles(d, n_tokens) * d.num_kv_heads <= kMaxPieces * kSmCount) return CrossDeal::kPieces;
  const int64_t rows = n_tokens * (d.num_q_heads / d.num_kv_heads);
  return 2 * rows <= Cross::ROWS * int64_t(d.batch) ? CrossDeal::kLine : CrossDeal::kItems;
}

int cross_part_rows(const splitkv_desc_t& d, int64_t n_tokens) {
  const int64_t rows = n_tokens * (d.num_q_heads / d.num_kv_heads);
  return int(rows < Cross::ROWS ? rows : Cross::ROWS);
}

int cross_box_rows(const splitkv_desc_t& d) {
  int br = 16;
  while (br < Cross::BK && d.page_size % (2 * br) == 0) br *= 2;
  return br;
}

cudaError_t launch_cross(const CrossArgs& a, int64_t row_tiles, const CrossMaps& maps, void* stream) {
  cudaError_t e = launch_cross_kernel<false, false>(a, maps, stream);
  return e == cudaSuccess ? launch_cross_merge(a, row_tiles, stream) : e;
}

cudaError_t launch_cross_merge(const CrossArgs& a, int64_t row_tiles, void* stream) {
  if (a.parts == 0) return cudaSuccess;
  // With an item per CTA at most, a cut costs 1 + kPieceCost + kCutCost at least:
  // items of so few key blocks that none costs more are never cut (a token over
  // 256 keys of 16 heads: 9.4 us, with the merge's launch 10.9).
  const int64_t blocks = (int64_t(a.max_pages) * a.P + Cross::BK - 1) / Cross::BK;
  if (row_tiles * a.Hkv <= a.parts && blocks <= 1 + kCutCost) return cudaSuccess;
  const int units = (a.part_rows + 31) / 32;  // of an item
  cudaLaunchAttribute la[1];
  la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  la[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(units > 1 ? 2 * a.parts : a.parts), 1, 1);
  cfg.blockDim = dim3(kMergeWarps * 32, 1, 1);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = la;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cross_merge_kernel, a, units);
}

}  // namespace splitkv
