// Rotary positions and the paged append, sm_103a.
//
// For every new token n of sequence b (the tokens [cu[b], cu[b + 1]) of the
// call, the last ones of the sequence's seq_lens[b] keys), with angle
//     a_i = positions[axis(i)][n] * freq_i,
// pair i = (u, v) of each query and key head row becomes
//     (u cos a_i - v sin a_i, u sin a_i + v cos a_i);
// the query goes to q_out, the key and the value into row j % P of page
// block_table[b][j / P], j = seq_lens[b] - (cu[b + 1] - n).
//
// Angles.  A position times a frequency needs more digits than 32-bit
// arithmetic has (2^20 * 1.0 rad leaves 2^-4 rad of it).  freq_i is held as a
// fraction of a full turn in 64-bit fixed point, so position * freq modulo a
// turn is one wrapping 64-bit product, off by at most |position| * 3 * 2^-65
// turns (the table's entries are added up from two rounded parts); its top 32
// bits, as a signed number of half turns in [-1, 1) rounded to 24 bits (off by
// 2^-25 half turns at most), go to sincospif.  Rotation is in fp32, rounded once: to bf16, or to e4m3 after
// the division by the cache's scale.
//
// Bound: the bytes of q (read and written), k and v (read, and written in the
// cache's type); a decode step of a few tokens is bound by one chain of
// loads, so nothing but the token's own loads precedes its stores.  Measured:
// 26k prompt tokens of 40 rows of 128: 95 us, 5.7 TB/s (floor 79 at the copy's
// 6.8: rows of 256 bytes go to as many places); one token 3.2 us, 32 in e4m3
// 3.7, of which a launch is most.
//
// One thread handles 32-byte units (two 16-byte chunks of a head row, the
// two halves of the same eight pairs where pairs are half a row apart), so
// every load and store is 16 bytes wide; a CTA computes the sines and cosines
// of its tokens once, for all heads.
#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"

namespace splitkv {
namespace {

using namespace ptx;

constexpr int kThreads = 256;
constexpr int kMaxTok = 32;  // tokens of a CTA, at most

struct Token {
  int32_t b, slot, page, in_page;  // b < 0: padding; page < 0: no key is stored
};

__device__ __forceinline__ uint32_t pack_e4m3x4(const float* x) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x[1]), "f"(x[0]));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x[3]), "f"(x[2]));
  return uint32_t(lo) | (uint32_t(hi) << 16);
}

__device__ __forceinline__ void unpack8(const uint4& r, float (&f)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                    pack_bf16(f[6], f[7]));
}

// The sequence whose tokens [cu[b], cu[b + 1]) hold n, or -1 (by a warp): 32 at a
// time are told apart at once, more by a search first (2,048 tokens of as many
// sequences, 48 rows each: 13.8 us, 20.9 by a pass over all sequences).
__device__ __forceinline__ int find_seq(const int32_t* cu, int batch, int n, int lane) {
  int lo = 0, len = batch;  // the sequence is among [lo, lo + len), or none
  while (len > 32) {
    const int step = (len + 31) / 32, b = lane * step;
    const unsigned m = __ballot_sync(kFull, b < len && cu[lo + b] <= n);
    const int at = m ? (31 - __clz(m)) * step : 0;
    lo += at;
    len = min(step, len - at);
  }
  const int ended = lo + __popc(__ballot_sync(kFull, lane < len && cu[lo + lane + 1] <= n));
  return ended < batch && cu[0] <= n ? ended : -1;
}

constexpr int kPasses = 5;  // over a CTA's units, at most

// U: units of a thread in flight.
template <int DK, int DV, bool FP8, int U>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendArgs a,
                                                          int tok_per_cta) {
  constexpr int UK = DK / 16, UV = DV / 16;  // units of a q or k row, of a v row
  __shared__ Token tok[kMaxTok];
  // Cosines and sines of two pairs of a chunk to a float4 (c, c, s, s), the
  // chunks of a row side by side: its lanes read consecutive 16 bytes.
  __shared__ float4 cs[kMaxTok * kMaxRotPairs / 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  launch_dependents();
  wait_prerequisites();

  const int n0 = blockIdx.x * tok_per_cta;
  const int ntok = min(tok_per_cta, a.n_tokens - n0);
  const int half = a.rope.rot_dim / 2;
  const int qu = a.q ? a.Hq * UK : 0, ku = a.Hkv * UK;
  const int per_tok = qu + ku + (a.v ? a.Hkv * UV : 0);
  const int total = ntok * per_tok;
  const int rot0 = a.rope.rot_offset / 8, rotc = a.rope.rot_dim / 8;  // rotated chunks
  const bool halves = a.rope.pairing == SPLITKV_ROPE_HALVES;
  const int chunk_pairs = halves ? 8 : 4, turned = half / chunk_pairs;  // pairs of a chunk, chunks with own pairs

  // Chunks of unit u of a row: the two halves of eight pairs while u counts
  // rotated pairs half a row apart, then the other chunks in order.
  auto chunks = [&](int u, int& c0, int& c1) {
    if (!halves || rotc == 0) {
      c0 = 2 * u;
      c1 = c0 + 1;
    } else if (u < rotc / 2) {
      c0 = rot0 + u;
      c1 = c0 + rotc / 2;
    } else {
      c0 = 2 * u - rotc;
      c1 = c0 + 1;
      c0 += c0 >= rot0 ? rotc : 0;
      c1 += c1 >= rot0 ? rotc : 0;
    }
  };
  // Unit i of the CTA: kind 0 q, 1 k, 2 v; token, head row, chunks.
  auto unit = [&](int i, int& kind, int& t, int& row, int& c0, int& c1) {
    t = int(__umulhi(unsigned(i), a.per_tok_magic));  // i / per_tok
    int u = i - t * per_tok;
    kind = u < qu ? 0 : u < qu + ku ? 1 : 2;
    if (kind < 2) {
      u -= kind ? qu : 0;
      row = u / UK;
      chunks(u - row * UK, c0, c1);
    } else {
      u -= qu + ku;
      row = u / UV;
      c0 = 2 * (u - row * UV);
      c1 = c0 + 1;
    }
  };
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + int64_t(n0) * a.q_stride;
  const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(a.k) + int64_t(n0) * a.k_stride;
  const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v) + int64_t(n0) * a.v_stride;
  __nv_bfloat16* q_out = static_cast<__nv_bfloat16*>(a.q_out) + int64_t(n0) * a.q_out_stride;

  bool ready = false;
  for (int base = blockIdx.y * (U * kThreads); base < total || !ready; base += gridDim.y * (U * kThreads)) {
    // The tokens' own rows first (those of padding are within the inputs
    // too): they are in flight while the tokens' places are looked up.
    uint4 x0[U], x1[U];
    uint32_t tag[U];  // token, kind, first chunk, second chunk (5, 2, 7, 7 bits)
    int rows[U];
#pragma unroll
    for (int r = 0; r < U; ++r) {
      const int i = base + r * kThreads + threadIdx.x;
      tag[r] = ~0u;
      if (i >= total) continue;
      int kind, t, c0, c1;
      unit(i, kind, t, rows[r], c0, c1);
      tag[r] = t | kind << 5 | c0 << 7 | c1 << 14;
      const __nv_bfloat16* from = kind == 0 ? q : kind == 1 ? k : v;
      const int stride = int(kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride);  // (below 2^31)
      const uint4* src = reinterpret_cast<const uint4*>(from + int64_t(t) * stride + rows[r] * (kind < 2 ? DK : DV));
      x0[r] = src[c0];
      x1[r] = src[c1];
    }
    if (!ready) {
      ready = true;
      // where the tokens' keys go, and their sines and cosines
      for (int i = warp; i < ntok; i += kThreads / 32) {
        const int n = n0 + i;
        Token t;
        t.b = a.cu ? find_seq(a.cu, a.batch, n, lane) : n / a.T;
        t.page = -1;
        t.slot = t.in_page = 0;
        if (t.b >= 0) {
          const int64_t cap = int64_t(a.max_pages) * a.P;
          const int64_t end = a.cu ? a.cu[t.b + 1] : int64_t(t.b + 1) * a.T;
          const int64_t slot = int64_t(a.seq_lens[t.b]) - (end - n);
          int err = 0;
          if (slot < 0 || slot >= cap) {
            err = SPLITKV_DEVERR_SEQLEN;
          } else {
            const int lp = int(slot) / a.P;
            const int ph = a.block_table[size_t(t.b) * a.max_pages + lp];
            if (ph < 0 || ph >= a.num_pages) {
              err = SPLITKV_DEVERR_PAGE;
            } else {
              t.page = ph;
              t.slot = int(slot);
              t.in_page = int(slot) - lp * a.P;
            }
          }
          if (err && lane == 0 && a.status && blockIdx.y == 0) atomicOr(a.status, err);
        }
        if (lane == 0) tok[i] = t;
      }
      for (int i = threadIdx.x; i < ntok * half; i += kThreads) {
        const int t = i / half, p = i - t * half;
        const int64_t pos = a.positions[size_t(a.rope.axis[p]) * a.n_tokens + n0 + t];
        const uint64_t phase = uint64_t(pos) * a.rope.turns[p];
        float s, c;
        sincospif(float(int32_t(phase >> 32)) * 0x1p-31f, &s, &c);
        const int ch = p / chunk_pairs, e = p - ch * chunk_pairs;
        float* z = reinterpret_cast<float*>(cs + t * (kMaxRotPairs / 2) + (e >> 1) * turned + ch) + (e & 1);
        z[0] = c;
        z[2] = s;
      }
      __syncthreads();
      // the state of the new keys
      if (blockIdx.y == 0 && (a.key_weights || a.key_positions)) {
        for (int i = threadIdx.x; i < ntok * a.Hkv; i += kThreads) {
          const int t = i / a.Hkv, h = i - t * a.Hkv;
          if (tok[t].page < 0) continue;
          const size_t at = (size_t(tok[t].b) * a.Hkv + h) * (size_t(a.max_pages) * a.P) + tok[t].slot;
          if (a.key_weights) a.key_weights[at] = 0.f;
          if (a.key_positions) a.key_positions[at] = a.positions[n0 + t];
        }
      }
    }
#pragma unroll
    for (int r = 0; r < U; ++r) {
      if (tag[r] == ~0u) continue;
      const int t = tag[r] & 31, kind = tag[r] >> 5 & 3, c0 = tag[r] >> 7 & 127, c1 = tag[r] >> 14 & 127, row = rows[r];
      const Token tk = tok[t];
      if (tk.b < 0 || (kind > 0 && tk.page < 0)) continue;
      float f0[8], f1[8];
      unpack8(x0[r], f0);
      unpack8(x1[r], f1);
      if (kind < 2 && rotc) {
        const float4* w = cs + t * (kMaxRotPairs / 2);
        auto turn = [](float& u, float& v, float c, float s) {
          const float x = u * c - v * s;
          v = u * s + v * c;
          u = x;
        };
        if (halves) {
          if (c0 >= rot0 && c0 < rot0 + rotc) {  // then c1 is the other half of the pairs
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float4 z = w[e * turned + c0 - rot0];
              turn(f0[2 * e], f1[2 * e], z.x, z.z);
              turn(f0[2 * e + 1], f1[2 * e + 1], z.y, z.w);
            }
          }
        } else {
          auto both = [&](float (&f)[8], int c) {
            if (c < rot0 || c >= rot0 + rotc) return;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float4 z = w[e * turned + c - rot0];
              turn(f[4 * e], f[4 * e + 1], z.x, z.z);
              turn(f[4 * e + 2], f[4 * e + 3], z.y, z.w);
            }
          };
          both(f0, c0);
          both(f1, c1);
        }
      }
      if (kind == 0) {
        uint4* dst = reinterpret_cast<uint4*>(q_out + int64_t(t) * int(a.q_out_stride) + row * DK);
        dst[c0] = pack8(f0);
        dst[c1] = pack8(f1);
        continue;
      }
      const size_t line = a.nhd ? (size_t(tk.page) * a.P + tk.in_page) * a.Hkv + row
                                : (size_t(tk.page) * a.Hkv + row) * a.P + tk.in_page;
      const bool is_k = kind == 1;
      const int D = is_k ? DK : DV;
      void* pool = is_k ? a.k_pages : a.v_pages;
      if (FP8) {
        const float* per_head = is_k ? a.k_scale : a.v_scale;
        const float sc = per_head ? per_head[row] : a.kv_scale;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          f0[e] = __fdiv_rn(f0[e], sc);
          f1[e] = __fdiv_rn(f1[e], sc);
        }
        uint2* dst = reinterpret_cast<uint2*>(static_cast<uint8_t*>(pool) + line * D);
        dst[c0] = make_uint2(pack_e4m3x4(f0), pack_e4m3x4(f0 + 4));
        dst[c1] = make_uint2(pack_e4m3x4(f1), pack_e4m3x4(f1 + 4));
      } else {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(pool) + line * D);
        dst[c0] = is_k ? pack8(f0) : x0[r];
        dst[c1] = is_k ? pack8(f1) : x1[r];
      }
    }
  }
}

template <int DK, int DV, bool FP8, int U>
cudaError_t launch_append_u(const AppendArgs& args, int per_tok, cudaStream_t s) {
  AppendArgs a = args;
  // i * magic >> 32 is i / per_tok for every unit i of a CTA, as i * per_tok is
  // below 2^32 or the CTA has one token (0: that token's, however many units)
  a.per_tok_magic = per_tok > 65536 ? 0 : unsigned(((uint64_t(1) << 32) + per_tok - 1) / per_tok);
  // A CTA's tokens.  In a long call the first number, of two passes or more over
  // its units (which share the lookup of the places and the sines: 26k tokens of
  // 40 rows, 99 us, with one pass 106), that leaves at most a twelfth of the
  // threads idle in the last, or else the best within kPasses (29k tokens of 17
  // latent rows, e4m3: four tokens 172 us, one 230).  A token of more units than
  // that goes to several CTAs.
  constexpr int pass = U * kThreads, most = (U == 1 ? 1 : kPasses) * pass;
  const int64_t slices = (int64_t(per_tok) + most - 1) / most;
  int most_tok = max(1, min(kMaxTok, most / per_tok)), tpc = most_tok;
  if (U > 1) {
    // (two CTAs per SM at least)
    tpc = most_tok = max(1, min(most_tok, a.n_tokens / (2 * kSmCount)));
    double least = 1e30;
    for (int t = 1; t <= most_tok && least > 1. / 12; ++t) {
      const int units = t * per_tok;
      const double idle = double((pass - units % pass) % pass) / units;
      if (units > pass && idle < least) {
        least = idle;
        tpc = t;
      }
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.n_tokens + tpc - 1) / tpc, unsigned(slices > 65535 ? 65535 : slices), 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute la[1];
  la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  la[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = la;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, append_kernel<DK, DV, FP8, U>, a, tpc);
}

// A call of few tokens takes one unit per thread, to use more of the GPU's
// SMs (32 tokens: 3.7 us, with four 8.8); a long one two, for bytes in flight
// (26k tokens: 97.8 us, with one 239, with four 99.2, with six 126; in e4m3
// 100, with four 137).
constexpr int64_t kFewUnits = 1 << 17;

template <int DK, int DV, bool FP8>
cudaError_t launch_append_t(const AppendArgs& a, cudaStream_t s) {
  const int per_tok = (a.q ? a.Hq * (DK / 16) : 0) + a.Hkv * (DK / 16 + (a.v ? DV / 16 : 0));
  return int64_t(per_tok) * a.n_tokens <= kFewUnits ? launch_append_u<DK, DV, FP8, 1>(a, per_tok, s)
                                                    : launch_append_u<DK, DV, FP8, 2>(a, per_tok, s);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, int qk_dim, int v_dim, bool fp8, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (qk_dim == 128 && v_dim == 128)
    return fp8 ? launch_append_t<128, 128, true>(a, s) : launch_append_t<128, 128, false>(a, s);
  return fp8 ? launch_append_t<576, 512, true>(a, s) : launch_append_t<576, 512, false>(a, s);
}

}  // namespace splitkv
