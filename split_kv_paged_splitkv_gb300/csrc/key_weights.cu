// Attention weight of every cached key, sm_103a.
//
//   w_out[b][h][j] = decay * w_in[b][h][j]
//                    + sum over tokens t and query heads of KV head h, j <= L-T+t,
//                      of exp(scale * q . K_j - lse[b][t][head])
// with the log-sum-exps of the decode call over the same cache.
//
// Bound: K is read once (256 or 128 bytes per key and KV head, against 8 of
// state), so the kernel lives on bytes in flight.  A warp takes 16 keys of a
// KV head at a time as the M side of m16n8k16 products with 8 query rows on
// N.  The order of the 128 dims inside the products is free as long as both
// operands use the same one, so each lane owns 16-byte pieces of two key rows
// that are its A operand as they lie (four lanes read 64 consecutive bytes),
// and query pieces chosen the same way are its B operand.  A lane copies its
// pieces of the next tile into shared memory asynchronously and reads back
// only what it copied itself: no barrier at all, and the bytes in flight come
// from the number of warps (32 KB of a CTA's four; a third tile of a warp in
// flight costs more in CTAs per SM than it gives: 171 us against 165 below).
//
// Measured: 32 sequences of up to 131k keys, 8 heads, bf16: 165 us, 6.4 TB/s of
// the 6.8 a copy gets; 8 of 32k in e4m3: 27.2 us (floor 20.2, the rest the
// start and its chain of loads); one of 5.9k: 4.2 us, the chain alone.
//
// Work is split by the device lengths: the 16-key tiles of all (sequence, KV
// head) pairs form one line, cut into equal contiguous parts, one per warp.
// Each key belongs to one warp, so results do not depend on any order.
#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"

namespace splitkv {
namespace {

using namespace ptx;

constexpr int kWarps = 4;

// 16 bytes global -> shared, asynchronously, past L1.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
constexpr float kLog2e = 1.4426950408889634f;

// The length of sequence b, or 0 where the device value is not one the cache
// can hold.
__device__ __forceinline__ int seq_len(const WeightArgs& a, int b, bool report) {
  const int L = a.seq_lens[b];
  if (L >= 0 && L <= int64_t(a.max_pages) * a.P && (L == 0 || L >= a.T)) return L;
  if (report && a.status) atomicOr(a.status, SPLITKV_DEVERR_SEQLEN);
  return 0;
}

template <bool FP8, int NRG, int STAGES>
__global__ void __launch_bounds__(kWarps * 32) key_weights_kernel(const __grid_constant__ WeightArgs a) {
  const int lane = threadIdx.x & 31;
  const int gi = lane >> 2, ci = lane & 3;
  // this lane's pieces of a tile: piece i of stage s at ring + (s * 2 NC + i) * 512
  constexpr int NC = FP8 ? 2 : 4;  // 16-byte pieces of a row per lane
  extern __shared__ __align__(16) uint8_t smem[];
  const uint32_t ring = smem_u32(smem) + (threadIdx.x >> 5) * (STAGES * 2 * NC * 512) + lane * 16;
  launch_dependents();
  wait_prerequisites();

  // tiles of the whole batch, then this warp's part [i0, i1)
  static_assert(32 * ((kMaxSlots + 15) / 16) < int64_t(1) << 32, "32 sequences' tiles are added up in 32 bits, unsigned");
  int64_t total = 0;
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    const int bl = b0 + lane;
    uint32_t n = bl < a.batch ? (seq_len(a, bl, blockIdx.x == 0 && threadIdx.x < 32) + 15) >> 4 : 0;
#pragma unroll
    for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(kFull, n, o);
    total += int64_t(n) * a.Hkv;
  }
  const int64_t nw = int64_t(gridDim.x) * kWarps, w = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  int64_t i0 = total * w / nw;
  const int64_t i1 = total * (w + 1) / nw;
  if (i0 >= i1) return;

  // the sequence and head of tile i0 (32 sequences at a time)
  int b = -1, h = 0, tile = 0;
  int64_t before = 0;
  for (int b0 = 0; b < 0; b0 += 32) {
    const int bl = b0 + lane;
    const int n = bl < a.batch ? (seq_len(a, bl, false) + 15) >> 4 : 0;
    uint32_t sum = n;  // tiles of a head, up to and with sequence bl
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(kFull, sum, o);
      if (lane >= o) sum += v;
    }
    const unsigned past = __ballot_sync(kFull, before + int64_t(sum) * a.Hkv > i0);
    if (past) {
      const int first = __ffs(past) - 1;
      const int per = __shfl_sync(kFull, n, first);
      const int64_t at = i0 - before - (int64_t(__shfl_sync(kFull, sum, first)) - per) * a.Hkv;
      b = b0 + first;
      h = int(at / per);
      tile = int(at - int64_t(h) * per);
    } else {
      before += int64_t(__shfl_sync(kFull, sum, 31)) * a.Hkv;
    }
  }

  const int rph = a.T * a.G;
  const size_t cap = size_t(a.max_pages) * a.P;
  constexpr int RB = FP8 ? 128 : 256;      // bytes of a key row
  const size_t key_step = a.nhd ? size_t(a.Hkv) * RB : RB;

  while (i0 < i1) {
    // ---- one (sequence, head): its queries, row limits, log-sum-exps
    const int L = seq_len(a, b, false);
    const int per = (L + 15) >> 4;
    const int end = int(min(int64_t(per), tile + (i1 - i0)));
    uint32_t qf[NRG][8][2];
    int lim[NRG][2];
    float ls[NRG][2], sl[NRG][2];
    const float qk = a.k_scale ? a.qk_scale_log2 * a.k_scale[h] : a.qk_scale_log2;
#pragma unroll
    for (int rg = 0; rg < NRG; ++rg) {
      const int n = rg * 8 + gi;
      const bool live = n < rph;
      const int t = n / a.G, g = n - t * a.G;
      const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(a.q) +
                                ((size_t(b) * a.T + t) * a.Hq + size_t(h) * a.G + g) * 128;
      float down = 1.f;
      if (!FP8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 x = live ? reinterpret_cast<const uint4*>(qp)[ci + 4 * i] : make_uint4(0, 0, 0, 0);
          qf[rg][2 * i][0] = x.x;
          qf[rg][2 * i][1] = x.y;
          qf[rg][2 * i + 1][0] = x.z;
          qf[rg][2 * i + 1][1] = x.w;
        }
      } else {
        // f16 products: the row is scaled by a power of two so that its
        // largest component lies in [2^14, 2^15); exact, and a component
        // rounds only below 2^-29 of the largest
        uint4 x[2][2];
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            x[i][e] = live ? reinterpret_cast<const uint4*>(qp)[2 * (ci + 4 * i) + e] : make_uint4(0, 0, 0, 0);
            const uint32_t v[4] = {x[i][e].x, x[i][e].y, x[i][e].z, x[i][e].w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(v[k] << 16)), fabsf(__uint_as_float(v[k] & 0xffff0000u))));
          }
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
        int k2 = 0;
        if (amax > 0.f) k2 = min(126, max(-113, 14 - (int((__float_as_uint(amax) >> 23) & 0xff) - 127)));
        const float up = __uint_as_float(uint32_t(127 + k2) << 23);
        down = __uint_as_float(uint32_t(127 - k2) << 23);
        auto f16 = [&](uint32_t v) {
          return pack_f16(__uint_as_float(v << 16) * up, __uint_as_float(v & 0xffff0000u) * up);
        };
        // word j of a 16-code piece holds dims 4j .. 4j + 3
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            qf[rg][4 * i + 2 * e][0] = f16(x[i][e].x);
            qf[rg][4 * i + 2 * e][1] = f16(x[i][e].y);
            qf[rg][4 * i + 2 * e + 1][0] = f16(x[i][e].z);
            qf[rg][4 * i + 2 * e + 1][1] = f16(x[i][e].w);
          }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        // this lane's scores are of query rows 2 ci and 2 ci + 1
        const int r = rg * 8 + 2 * ci + e;
        sl[rg][e] = qk * __shfl_sync(kFull, down, (2 * ci + e) * 4);
        lim[rg][e] = -1;
        ls[rg][e] = INFINITY;  // (a row that is none, or has no keys, weighs nothing)
        if (r < rph) {
          const int rt = r / a.G, rgq = r - rt * a.G;
          const float v = a.lse[(size_t(b) * a.T + rt) * a.Hq + size_t(h) * a.G + rgq];
          if (v != -INFINITY) {
            ls[rg][e] = v * kLog2e;
            lim[rg][e] = L - a.T + rt;
          }
        }
      }
    }

    // ---- its tiles
    const int32_t* trow = a.block_table + size_t(b) * a.max_pages;
    const size_t state = (size_t(b) * a.Hkv + h) * cap;
    // The places of 32 tiles at a time, a lane each.  Copies run STAGES - 1 tiles
    // ahead, a group per tile (empty ones behind the last, so that the count of
    // groups says which have landed); the state one tile ahead.
    int tiles0 = -32;     // first tile of the lanes' rows
    int64_t rows_at = 0;  // where the rows of tile tiles0 + lane begin
    const uint8_t* mine = static_cast<const uint8_t*>(a.k_pages) + gi * key_step + ci * 16;
    auto fetch = [&](int tl) {
      if (tl < end) {
        if (tl >= tiles0 + 32) {
          tiles0 = tl;
          if (tl + lane < end) {
            const int lp = (tl + lane) * 16 / a.P, kp = (tl + lane) * 16 - lp * a.P;
            int ph = trow[lp];
            if (ph < 0 || ph >= a.num_pages) {
              if (a.status) atomicOr(a.status, SPLITKV_DEVERR_PAGE);
              ph = 0;
            }
            rows_at = (a.nhd ? (int64_t(ph) * a.P + kp) * a.Hkv + h : (int64_t(ph) * a.Hkv + h) * a.P + kp) * RB;
          }
        }
        const uint8_t* kr = mine + __shfl_sync(kFull, rows_at, tl - tiles0);
        const uint32_t dst = ring + (tl % STAGES) * (2 * NC * 512);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          copy16(dst + 2 * i * 512, kr + i * 64);
          copy16(dst + (2 * i + 1) * 512, kr + 8 * key_step + i * 64);
        }
      }
      copy_commit();
    };
    // lanes ci = 0 and 1 hold the state of keys gi and gi + 8
    auto state_of = [&](int tl) {
      const int key = tl * 16 + gi + 8 * ci;
      return tl < end && ci < 2 && key < L && a.w_in ? a.w_in[state + key] : 0.f;
    };
    for (int i = 0; i < STAGES - 1; ++i) fetch(tile + i);
    float old = state_of(tile);
    for (; tile < end; ++tile) {
      const int key0 = tile * 16;
      copy_wait<STAGES - 2>();  // this tile's copies
      uint4 x0[NC], x1[NC];
      {
        const uint32_t at = ring + (tile % STAGES) * (2 * NC * 512);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          x0[i] = lds16(at + 2 * i * 512);
          x1[i] = lds16(at + (2 * i + 1) * 512);
        }
      }
      // (into the stage read one tile ago)
      fetch(tile + STAGES - 1);
      const float next_old = state_of(tile + 1);

      const bool all_seen = key0 + 15 <= L - a.T;  // by every query token
      float wa = 0.f, wb = 0.f;
#pragma unroll
      for (int rg = 0; rg < NRG; ++rg) {
        float sc[4] = {0.f, 0.f, 0.f, 0.f}, sd[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          const uint32_t u[4] = {x0[i].x, x0[i].y, x0[i].z, x0[i].w};
          const uint32_t v[4] = {x1[i].x, x1[i].y, x1[i].z, x1[i].w};
          if (!FP8) {
            const uint32_t a0[4] = {u[0], v[0], u[1], v[1]}, a1[4] = {u[2], v[2], u[3], v[3]};
            mma_bf16(sc, a0, qf[rg][2 * i][0], qf[rg][2 * i][1]);
            mma_bf16(sd, a1, qf[rg][2 * i + 1][0], qf[rg][2 * i + 1][1]);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t ak[4] = {e4m3x2_lo(u[k]), e4m3x2_lo(v[k]), e4m3x2_hi(u[k]), e4m3x2_hi(v[k])};
              mma_f16(k & 1 ? sd : sc, ak, qf[rg][4 * i + k][0], qf[rg][4 * i + k][1]);
            }
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float ea = ex2(fmaf(sc[e] + sd[e], sl[rg][e], -ls[rg][e]));
          const float eb = ex2(fmaf(sc[2 + e] + sd[2 + e], sl[rg][e], -ls[rg][e]));
          // (NaN may lie behind the last key, and only there: a choice, no product)
          wa += all_seen || key0 + gi <= lim[rg][e] ? ea : 0.f;
          wb += all_seen || key0 + gi + 8 <= lim[rg][e] ? eb : 0.f;
        }
      }
      wa += __shfl_xor_sync(kFull, wa, 1);
      wb += __shfl_xor_sync(kFull, wb, 1);
      wa += __shfl_xor_sync(kFull, wa, 2);
      wb += __shfl_xor_sync(kFull, wb, 2);
      const int key = key0 + gi + 8 * ci;
      if (ci < 2 && key < L) a.w_out[state + key] = fmaf(a.decay, old, ci ? wb : wa);
      old = next_old;
      ++i0;
    }
    // ---- the next (sequence, head) with tiles
    if (tile == per) {
      tile = 0;
      if (++h == a.Hkv) {
        h = 0;
        if (i0 < i1) do ++b; while (seq_len(a, b, false) == 0);
      }
    }
  }
}

template <bool FP8, int NRG>
cudaError_t launch_weights_t(const WeightArgs& a, cudaStream_t s) {
  constexpr int STAGES = 2;
  constexpr int SMEM = kWarps * STAGES * (FP8 ? 2048 : 4096);
  static_assert(SMEM <= 48 * 1024, "no opt-in needed");
  // as many CTAs as the GPU holds at once
  int dev = 0, sms = 0, per_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess)
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, key_weights_kernel<FP8, NRG, STAGES>, kWarps * 32, SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  // (tiles at most, so that a short cache is not spread over idle CTAs)
  const int64_t most = (int64_t(a.batch) * a.Hkv * a.max_pages * (a.P / 16) + kWarps - 1) / kWarps;
  const int64_t grid = int64_t(sms) * (per_sm > 0 ? per_sm : 1);
  cfg.gridDim = dim3(unsigned(grid < most ? grid : most), 1, 1);
  cfg.blockDim = dim3(kWarps * 32, 1, 1);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = s;
  cudaLaunchAttribute la[1];
  la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  la[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = la;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, key_weights_kernel<FP8, NRG, STAGES>, a);
}

template <bool FP8>
cudaError_t launch_weights_f(const WeightArgs& a, cudaStream_t s) {
  const int rows = a.T * a.G;
  return rows <= 8 ? launch_weights_t<FP8, 1>(a, s)
                   : rows <= 16 ? launch_weights_t<FP8, 2>(a, s) : launch_weights_t<FP8, 4>(a, s);
}

}  // namespace

cudaError_t launch_key_weights(const WeightArgs& a, bool fp8, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return fp8 ? launch_weights_f<true>(a, s) : launch_weights_f<false>(a, s);
}

}  // namespace splitkv
