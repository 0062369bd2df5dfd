// Cross attention over a paged cache on the 5th-generation tensor cores
// (tcgen05, accumulators in TMEM), sm_103a:
//
//   out[n][head] = sum_j softmax_j(scale * q[n][head] . K_j) V_j
//
// for the query tokens n of every sequence over all L keys of its cache (an
// encoder's states, of another length than the queries; no causal mask), with
// the rows of 128 and the shared KV heads of the GQA decode.
//
// Work.  The T_b * G query rows that share a KV head form tiles of 256 rows,
// two MMA row blocks A and B of 128.  One CTA per (row tile, KV head, split of
// the keys); keys stream in blocks of 128.  Per key block and row block:
//   S = Q . K^T      (M=128 N=128 K=128, operands in shared memory)
//   softmax warps: one thread per query row; online softmax with a lazy
//     reference maximum (O is rescaled only when a row's maximum grows by more
//     than 2^8); P in bf16 over the first half of S
//   O += P . V       (M=128 N=128 K=128, P from TMEM)
// The two row blocks take turns: while the softmax warps of A work on block
// j, the tensor cores run PV_B(j - 1) and QK_B(j), and the other way round, so
// that a softmax may take as long as two products before the pipe idles.  The
// MMAs of a CTA are issued in the order ..., PV_A(j), QK_A(j+1), PV_B(j),
// QK_B(j+1), ...; they execute in that order, which makes the barrier of a
// finished S also say that the PV before it is done (P read, O at rest).
//
// K and V blocks pass in that order through one ring of five 32 KB slots that
// one producer warp fills by TMA, one box per page piece and 64-column half,
// 128-byte swizzled; K is read K-major, V with its dims on N.
// TMEM columns: S_A [0, 128), S_B [128, 256), O_A [256, 384), O_B [384, 512).
//
// Few rows (a decoder token over the encoder's states): the bound is the bytes
// of K and V, the keys are split so that every SM has a part, a row block
// without rows is left out, and merge_kernel joins the parts by their
// log-sum-exps.  Many rows: the bound is 4 * 128 * rows * L operations.
//
// P is rounded to bf16 for the second product (half a step, 2^-8 of a weight,
// as in the decode kernels); sums, maxima and O are fp32.
#include <cuda.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"

namespace splitkv {
namespace {

using namespace ptx;

struct Cross {
  static constexpr int ROWS = 256;               // query rows of a CTA
  static constexpr int BK = 128;                 // keys of a block
  static constexpr int TILE = BK * 256;          // a K or V block, or one row block of Q: 32 KB
  static constexpr int HALF = TILE / 2;          // its 64-column half: [128][128 B]
  static constexpr int NST = 5;
  static constexpr int OFF_RING = 2 * TILE;      // after Q's two row blocks
  static constexpr int OFF_BAR = OFF_RING + NST * TILE;
  static constexpr int SMEM = 1024 + OFF_BAR + 256;
  static constexpr int SOFTMAX_THREADS = 256;
  static constexpr int THREADS = SOFTMAX_THREADS + 64;
  static constexpr uint32_t TMEM_COLS = 512, S_COL = 0, O_COL = 256;  // + 128 per row block
  static constexpr float RESCALE_LOG2 = 8.f;
};
static_assert(Cross::SMEM <= 227 * 1024, "shared memory budget");

enum {
  B_Q = 0,                       // Q in shared memory (256 threads)
  B_FULL = 1,                    // [NST]
  B_EMPTY = B_FULL + Cross::NST, // [NST]
  B_S = B_EMPTY + Cross::NST,    // [2] S of a row block complete
  B_P = B_S + 2,                 // [2] P of a row block in TMEM (128 threads)
  B_O = B_P + 2,                 // [2] the last PV of a row block complete
  B_DONE = B_O + 2,
  B_COUNT
};

constexpr float kLn2 = 0.6931471805599453f;

// The length of sequence b, or 0 where the device value is not one the cache
// can hold.
__device__ __forceinline__ int keys_of(const CrossArgs& a, int b) {
  const int L = a.seq_lens[b];
  return L >= 0 && L <= int64_t(a.max_pages) * a.P ? L : 0;
}

// First token and number of tokens of sequence b, within [0, n_tokens].
__device__ __forceinline__ int tokens_of(const CrossArgs& a, int b, int* first) {
  if (!a.cu) {
    *first = b * a.T;
    return a.T;
  }
  const int t0 = min(max(a.cu[b], 0), a.n_tokens), t1 = min(a.cu[b + 1], a.n_tokens);
  *first = t0;
  return max(t1 - t0, 0);
}

// 64 consecutive fp32 columns of this warp's 32 TMEM lanes (one lane per thread).
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, float* v) {
  uint32_t r[64];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,"
      "%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,"
      "%62,%63}, [%64];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]),
        "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]),
        "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]),
        "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]),
        "=r"(r[63])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(r[i]);
}

// (a * s + b) for two numbers at once.
__device__ __forceinline__ void fma2(float& x, float& y, float s, float b) {
  asm("{\n\t.reg .b64 u, v, w;\n\tmov.b64 u, {%0, %1};\n\tmov.b64 v, {%2, %2};\n\tmov.b64 w, {%3, %3};\n\t"
      "fma.rn.f32x2 u, u, v, w;\n\tmov.b64 {%0, %1}, u;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(s), "f"(b));
}

__global__ void __launch_bounds__(Cross::THREADS, 1)
    cross_attend_kernel(const __grid_constant__ CrossArgs a, const __grid_constant__ CUtensorMap tk,
                        const __grid_constant__ CUtensorMap tv) {
  using C = Cross;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::OFF_BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + B_COUNT);
  int32_t* where = reinterpret_cast<int32_t*>(tmem_slot + 1);  // sequence, row tile
  auto bar = [&](int i) { return smem_u32(bars + i); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.y, split = blockIdx.z;

  if (threadIdx.x == 0) {
    mbar_init(bar(B_Q), C::SOFTMAX_THREADS);
    for (int s = 0; s < C::NST; ++s) {
      mbar_init(bar(B_FULL + s), 1);
      mbar_init(bar(B_EMPTY + s), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(B_S + t), 1);
      mbar_init(bar(B_P + t), 128);
      mbar_init(bar(B_O + t), 1);
    }
    mbar_init(bar(B_DONE), 1);
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
    if (lane == 0) {
      prefetch_tmap(&tk);
      prefetch_tmap(&tv);
    }
  }
  launch_dependents();
  wait_prerequisites();
  if (warp == 9) {
    // the sequence and row tile of this CTA: tiles of all sequences in a line
    int before = 0, b = -1, tile = 0;
    for (int b0 = 0; b0 < a.batch && b < 0; b0 += 32) {
      int first;
      const int bl = b0 + lane;
      const int rows = bl < a.batch ? tokens_of(a, bl, &first) * a.G : 0;
      const int n = (rows + C::ROWS - 1) / C::ROWS;
      int x = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += y;
      }
      const unsigned past = __ballot_sync(kFull, before + x > int(blockIdx.x));
      if (past) {
        const int f = __ffs(past) - 1;
        b = b0 + f;
        tile = int(blockIdx.x) - before - (__shfl_sync(kFull, x, f) - __shfl_sync(kFull, n, f));
      } else {
        before += __shfl_sync(kFull, x, 31);
      }
    }
    if (lane == 0) {
      where[0] = b;
      where[1] = tile;
    }
    // one CTA reports lengths that the cache cannot hold
    if (a.status && blockIdx.x == 0 && h == 0 && split == 0)
      for (int i = lane; i < a.batch; i += 32)
        if (a.seq_lens[i] != keys_of(a, i)) atomicOr(a.status, SPLITKV_DEVERR_SEQLEN);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int b = where[0];
  // (the grid counts tiles for any split of the tokens among the sequences)
  if (b >= 0) {
    int first;
    const int n_rows = tokens_of(a, b, &first) * a.G - where[1] * C::ROWS;  // from this tile on
    const int row0 = where[1] * C::ROWS;
    const int blocks = n_rows > 128 ? 2 : 1;  // row blocks with rows
    const int L = keys_of(a, b);
    // this split's key blocks
    const int all = (L + C::BK - 1) / C::BK;
    const int j0 = int(int64_t(all) * split / a.splits), j1 = int(int64_t(all) * (split + 1) / a.splits);
    const int nblk = j1 - j0, k_begin = j0 * C::BK, k_end = min(L, j1 * C::BK);

    if (warp == 8) {
      // ------------------------------------------------------------ producer
      // Item 2 j is K block j, item 2 j + 1 V block j; item i lies in slot
      // i % NST.  A block is BK / br pieces of br keys of one page each; lane
      // g holds the page of piece g.  Pieces behind the last key are not read.
      const int32_t* trow = a.block_table + size_t(b) * a.max_pages;
      const int br = a.box_rows;
      bool ok = true;
      int issued = 0;
      for (int j = 0; j < nblk && ok; ++j) {
        const int key0 = k_begin + j * C::BK;
        const int np = (min(C::BK, k_end - key0) + br - 1) / br;
        int ph = 0, in = 0;
        if (lane < np) {
          const int key = key0 + lane * br, lp = key / a.P;
          in = key - lp * a.P;
          ph = __ldg(trow + lp);
          if (ph < 0 || ph >= a.num_pages) {
            if (a.status) atomicOr(a.status, SPLITKV_DEVERR_PAGE);
            ph = 0;
          }
        }
        for (int v = 0; v < 2 && ok; ++v) {
          const int i = 2 * j + v, st = i % C::NST;
          if (i >= C::NST) ok = __all_sync(kFull, mbar_wait(bar(B_EMPTY + st), (i / C::NST - 1) & 1));
          if (!ok) break;
          mbar_arrive_expect_tx_warp(bar(B_FULL + st), uint32_t(np * br * 256));
          const uint32_t dst = smem_u32(sm + C::OFF_RING + st * C::TILE);
          const CUtensorMap* tm = v ? &tv : &tk;
          for (int g = 0; g < np; ++g) {
            const int pg = __shfl_sync(kFull, ph, g), kp = __shfl_sync(kFull, in, g);
            tma_load_5d_warp(dst + g * br * 128, tm, bar(B_FULL + st), 0, kp, 0, h, pg);
            tma_load_5d_warp(dst + C::HALF + g * br * 128, tm, bar(B_FULL + st), 0, kp, 1, h, pg);
          }
          issued = i + 1;
        }
      }
      if (!ok && lane == 0 && a.status) atomicOr(a.status, SPLITKV_DEVERR_TIMEOUT);
      // stay until every issued copy has landed
      if (lane == 0) {
        for (int st = 0; st < C::NST && st < issued; ++st) {
          const int last = st + C::NST * ((issued - 1 - st) / C::NST);
          if (!mbar_wait(bar(B_FULL + st), (last / C::NST) & 1)) break;
        }
      }
    } else if (warp == 9) {
      // ---------------------------------------------------------- MMA issuer
      constexpr uint32_t idesc_qk = umma_idesc_bf16(128, 128, 0, 0), idesc_pv = umma_idesc_bf16(128, 128, 0, 1);
      bool ok = true;
      auto wait = [&](int i, int phase) {
        ok = ok && __all_sync(kFull, mbar_wait(bar(i), phase & 1));
        return ok;
      };
      auto slot = [&](int i) { return smem_u32(sm + C::OFF_RING + (i % C::NST) * C::TILE); };
      auto qk = [&](int t, int j) {  // S_t = Q_t . K_j^T
        const uint32_t q = smem_u32(sm + t * C::TILE), k = slot(2 * j);
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int kin = 0; kin < 4; ++kin)
            umma_bf16_warp(tmem + C::S_COL + 128 * t, umma_desc(q + half * C::HALF + kin * 32, 16, 1024, 2),
                           umma_desc(k + half * C::HALF + kin * 32, 16, 1024, 2), idesc_qk, (half | kin) != 0);
        umma_commit_warp(bar(B_S + t));
        __syncwarp();
      };
      auto pv = [&](int t, int j) {  // O_t += P_t . V_j
        const uint32_t v = slot(2 * j + 1);
#pragma unroll
        for (int kin = 0; kin < 8; ++kin)
          umma_bf16_ta_warp(tmem + C::O_COL + 128 * t, tmem + C::S_COL + 128 * t + kin * 8,
                            umma_desc(v + kin * 16 * 128, C::HALF, 1024, 2), idesc_pv, (j | kin) != 0);
        if (j == nblk - 1) umma_commit_warp(bar(B_O + t));
        __syncwarp();
      };
      if (nblk > 0 && wait(B_Q, 0) && wait(B_FULL, 0)) {
        tc_fence_after();
        for (int t = 0; t < blocks; ++t) qk(t, 0);
        umma_commit_warp(bar(B_EMPTY));
        __syncwarp();
      }
      for (int j = 0; j < nblk && ok; ++j) {
        const int iv = 2 * j + 1, ik = 2 * j + 2;  // V block j, K block j + 1
        for (int t = 0; t < blocks && ok; ++t) {
          if (t == 0) {
            if (!wait(B_FULL + iv % C::NST, iv / C::NST)) break;
            const int valid = k_end - (k_begin + j * C::BK);
            if (valid < C::BK) {
              // key slots past the last key may hold anything (even NaN): zero
              // their V rows, so that 0 * V stays 0
              uint8_t* v = sm + C::OFF_RING + (iv % C::NST) * C::TILE;
              for (int x = lane; x < (C::BK - valid) * 16; x += 32)
                *reinterpret_cast<uint4*>(v + (x & 1) * C::HALF + (valid + (x >> 4)) * 128 + ((x >> 1) & 7) * 16) =
                    make_uint4(0, 0, 0, 0);
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
              __syncwarp();
            }
          }
          if (!wait(B_P + t, j)) break;
          tc_fence_after();
          pv(t, j);
          if (t == blocks - 1) {
            umma_commit_warp(bar(B_EMPTY + iv % C::NST));
            __syncwarp();
          }
          if (j + 1 < nblk) {
            if (t == 0 && !wait(B_FULL + ik % C::NST, ik / C::NST)) break;
            tc_fence_after();
            qk(t, j + 1);
            if (t == blocks - 1) {
              umma_commit_warp(bar(B_EMPTY + ik % C::NST));
              __syncwarp();
            }
          }
        }
      }
      if (!ok && lane == 0 && a.status) atomicOr(a.status, SPLITKV_DEVERR_TIMEOUT);
      // every MMA issued above completes before TMEM is released
      umma_commit_warp(bar(B_DONE));
      __syncwarp();
      mbar_wait(bar(B_DONE), 0);
    } else {
      // ------------------------------------------------------- softmax warps
      const int t = warp >> 2;                         // row block
      const int r = (warp & 3) * 32 + lane;            // TMEM lane
      const int row = t * 128 + r;                     // of the tile
      const bool live = row < n_rows;
      const uint32_t lanes = tmem + (uint32_t((warp & 3) * 32) << 16);
      const int tok = (row0 + row) / a.G, g = (row0 + row) - tok * a.G;
      const size_t out_row = (size_t(first) + tok) * a.Hq + size_t(h) * a.G + g;
      {
        // this row of Q, swizzled; rows behind the last are zero
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                          (int64_t(first) + tok) * a.q_stride + (h * a.G + g) * 128);
        uint8_t* dst = sm + t * C::TILE + r * 128;
        if (t < blocks) {
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const uint4 x = live ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(dst + (c >> 3) * C::HALF + (((c & 7) ^ (r & 7)) << 4)) = x;
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        mbar_arrive(bar(B_Q));
      }
      const bool any = __any_sync(kFull, live);  // a warp without rows only keeps step
      const uint32_t scol = C::S_COL + 128 * t, ocol = C::O_COL + 128 * t;
      const float sl2 = a.qk_scale_log2;
      float m_ref = -INFINITY, l = 0.f;
      bool ok = true;
      for (int j = 0; j < nblk && t < blocks; ++j) {
        ok = __all_sync(kFull, mbar_wait(bar(B_S + t), j & 1));
        if (!ok) break;
        tc_fence_after();
        if (any) {
          float s[128];
          tmem_ld64(lanes + scol, s);
          tmem_ld64(lanes + scol + 64, s + 64);
          const int valid = k_end - (k_begin + j * C::BK);
          if (valid < C::BK) {
#pragma unroll
            for (int k = 0; k < 128; ++k) s[k] = k < valid ? s[k] : -INFINITY;
          }
          // row maximum on the raw scores (the scale is positive)
          float m8[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) m8[i] = fmaxf(s[i], s[8 + i]);
#pragma unroll
          for (int k = 16; k < 128; k += 8)
#pragma unroll
            for (int i = 0; i < 8; ++i) m8[i] = fmaxf(m8[i], s[k + i]);
          const float mx = fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])),
                                 fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7]))) * sl2;
          float alpha = 1.f;
          bool rescale = false;
          if (mx > m_ref + C::RESCALE_LOG2 || (m_ref == -INFINITY && mx != -INFINITY)) {
            alpha = m_ref == -INFINITY ? 0.f : ex2(m_ref - mx);
            rescale = m_ref != -INFINITY;
            m_ref = mx;
            l *= alpha;
          }
          // (PV(j - 1) was issued before the product this S came from: O rests)
          if (__any_sync(kFull, rescale)) {
#pragma unroll 1
            for (int c0 = 0; c0 < 128; c0 += 32) {
              float o[32];
              tmem_ld32(lanes + ocol + c0, o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] *= alpha;
              tmem_st32(lanes + ocol + c0, o);
            }
          }
          const float nm = m_ref == -INFINITY ? 0.f : -m_ref;
          float l4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t pk[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              float& x = s[64 * c + 2 * i];
              float& y = s[64 * c + 2 * i + 1];
              fma2(x, y, sl2, nm);
              x = ex2(x);
              y = ex2(y);
              l4[(2 * i) & 3] += x;
              l4[(2 * i + 1) & 3] += y;
              pk[i] = pack_bf16(x, y);
            }
            tmem_st32u(lanes + scol + 32 * c, pk);
          }
          l += (l4[0] + l4[1]) + (l4[2] + l4[3]);
          tmem_wait_st();
        }
        tc_fence_before();
        mbar_arrive(bar(B_P + t));
      }
      if (!ok && lane == 0 && a.status) atomicOr(a.status, SPLITKV_DEVERR_TIMEOUT);

      // ---- epilogue
      if (t < blocks) {
        bool have = ok && nblk > 0;
        if (have && !__all_sync(kFull, mbar_wait(bar(B_O + t), 0))) {
          have = false;
          if (lane == 0 && a.status) atomicOr(a.status, SPLITKV_DEVERR_TIMEOUT);
        }
        if (have) tc_fence_after();
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const float lse = l > 0.f ? (m_ref + lg2(l)) * kLn2 : -INFINITY;
        const size_t part = size_t(split) * a.n_tokens * a.Hq + out_row;
        if (any) {
#pragma unroll 1
          for (int c0 = 0; c0 < 128; c0 += 32) {
            float o[32];
            if (have) {
              tmem_ld32(lanes + ocol + c0, o);
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = 0.f;
            }
            if (!live) continue;
            if (a.splits == 1) {
              uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + out_row * 128 + c0);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                dst[i] = make_uint4(pack_bf16(o[8 * i] * inv, o[8 * i + 1] * inv),
                                    pack_bf16(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                                    pack_bf16(o[8 * i + 4] * inv, o[8 * i + 5] * inv),
                                    pack_bf16(o[8 * i + 6] * inv, o[8 * i + 7] * inv));
            } else {
              float4* dst = reinterpret_cast<float4*>(a.o_part + part * 128 + c0);
#pragma unroll
              for (int i = 0; i < 8; ++i)
                dst[i] = make_float4(o[4 * i] * inv, o[4 * i + 1] * inv, o[4 * i + 2] * inv, o[4 * i + 3] * inv);
            }
          }
          if (live) {
            if (a.splits > 1) a.lse_part[part] = lse;
            else if (a.lse) a.lse[out_row] = lse;
          }
        }
      }
    }
  }

  // ---- teardown: TMEM is freed by the warp that allocated it
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// Joins the splits: a warp per (token, query head), four dims per lane.
// Tokens of no sequence are left as they are.
__global__ void __launch_bounds__(128) cross_merge_kernel(const __grid_constant__ CrossArgs a) {
  launch_dependents();
  wait_prerequisites();
  const int64_t rows = int64_t(a.n_tokens) * a.Hq, r = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (r >= rows) return;
  if (a.cu && (r < int64_t(a.cu[0]) * a.Hq || r >= int64_t(a.cu[a.batch]) * a.Hq)) return;
  const float ls = lane < a.splits ? a.lse_part[int64_t(lane) * rows + r] : -INFINITY;
  float M = ls;
#pragma unroll
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
  const float w = M == -INFINITY ? 0.f : ex2((ls - M) * 1.4426950408889634f);
  float sum = w;
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < a.splits; ++s) {
    const float ws = __shfl_sync(kFull, w, s);
    if (ws == 0.f) continue;  // (a part without keys may hold anything)
    const float4 x = *reinterpret_cast<const float4*>(a.o_part + (s * rows + r) * 128 + lane * 4);
    acc.x += ws * x.x;
    acc.y += ws * x.y;
    acc.z += ws * x.z;
    acc.w += ws * x.w;
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  uint2 v;
  v.x = pack_bf16(acc.x * inv, acc.y * inv);
  v.y = pack_bf16(acc.z * inv, acc.w * inv);
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + r * 128 + lane * 4) = v;
  if (lane == 0 && a.lse) a.lse[r] = sum > 0.f ? M + lg2(sum) * kLn2 : -INFINITY;
}

}  // namespace

// Row tiles of a call at most, however its tokens are dealt to the sequences.
int64_t cross_row_tiles(const splitkv_desc_t& d, int64_t n_tokens) {
  const int64_t G = d.num_q_heads / d.num_kv_heads;
  const int64_t full = n_tokens * G / Cross::ROWS, some = n_tokens < d.batch ? n_tokens : d.batch;
  return full + some;
}

// Key splits.  A CTA has an SM to itself; the call lasts as long as the SM
// with most work, in key blocks, plus about four blocks' time for a CTA's
// start and end and, with more than one split, two for the merge.
int cross_splits(const splitkv_desc_t& d, int64_t n_tokens) {
  const int64_t ctas = cross_row_tiles(d, n_tokens) * d.num_kv_heads;
  const int64_t blocks = (int64_t(d.max_pages_per_seq) * d.page_size + Cross::BK - 1) / Cross::BK;
  int best = 1;
  int64_t least = INT64_MAX;
  for (int s = 1; s <= kMaxCrossSplits && s <= blocks; ++s) {
    const int64_t waves = (ctas * s + kSmCount - 1) / kSmCount;
    const int64_t cost = waves * ((blocks + s - 1) / s + 4) + (s > 1 ? 2 : 0);
    if (cost < least) {
      least = cost;
      best = s;
    }
  }
  return best;
}

int cross_box_rows(const splitkv_desc_t& d) {
  int br = 16;
  while (br < Cross::BK && d.page_size % (2 * br) == 0) br *= 2;
  return br;
}

cudaError_t launch_cross(const CrossArgs& a, int64_t row_tiles, const TmaDesc& tk, const TmaDesc& tv, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  static cudaError_t attr =
      cudaFuncSetAttribute(cross_attend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cross::SMEM);
  if (attr != cudaSuccess) return attr;
  cudaLaunchAttribute la[1];
  la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  la[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(row_tiles), unsigned(a.Hkv), unsigned(a.splits));
  cfg.blockDim = dim3(Cross::THREADS, 1, 1);
  cfg.dynamicSmemBytes = Cross::SMEM;
  cfg.stream = s;
  cfg.attrs = la;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, cross_attend_kernel, a, *reinterpret_cast<const CUtensorMap*>(&tk),
                                     *reinterpret_cast<const CUtensorMap*>(&tv));
  if (e != cudaSuccess || a.splits == 1) return e;
  cfg.gridDim = dim3(unsigned((int64_t(a.n_tokens) * a.Hq + 3) / 4), 1, 1);
  cfg.blockDim = dim3(128, 1, 1);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, cross_merge_kernel, a);
}

}  // namespace splitkv
