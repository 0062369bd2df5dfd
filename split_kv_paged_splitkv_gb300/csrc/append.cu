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
// With norms (splitkv_append_norm) the query and key rows are first divided by
// their root mean square and multiplied by a weight for each column:
//     x_i <- x_i * rsqrt(mean(x^2) + eps) * w_i,
// all in fp32, so that norm, rotation and store round once.  The mean of a row of
// 128 is a sum over the eight lanes that hold it (append_rows_kernel and, for long
// calls, append_stream_kernel); a latent row's 36 units
// lie across warps, so a warp adds up its 512 columns by itself while the token's
// place is looked up (1 KB read again, beside the 147 KB of the token's queries; 1.8k
// tokens of 129 rows into e4m3: 95 us, 5.6 TB/s, without norms 91, floor 79).
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

// Where the key of token n of sequence b (-1: padding) goes; what is wrong with it goes
// to the status, if this thread reports.
__device__ __forceinline__ Token place_in(const AppendArgs& a, int b, int n, bool report) {
  Token t;
  t.b = b;
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
    if (err && report && a.status) atomicOr(a.status, err);
  }
  return t;
}

// The same by a warp.
__device__ __forceinline__ Token place_of(const AppendArgs& a, int n, int lane, bool report) {
  return place_in(a, a.cu ? find_seq(a.cu, a.batch, n, lane) : n / a.T, n, report && lane == 0);
}

// The sines and cosines of a CTA's tokens (see `cs` of the kernels).
__device__ __forceinline__ void sines(const AppendArgs& a, int n0, int ntok, float4* cs) {
  const int half = a.rope.rot_dim / 2;
  const int chunk_pairs = a.rope.pairing == SPLITKV_ROPE_HALVES ? 8 : 4, turned = half / chunk_pairs;
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
}

// The state of a CTA's new keys.
template <int THREADS = kThreads>
__device__ __forceinline__ void new_state(const AppendArgs& a, int n0, int ntok, const Token* tok, int thread = threadIdx.x) {
  if (a.key_weights || a.key_positions) {
    for (int i = thread; i < ntok * a.Hkv; i += THREADS) {
      const int t = i / a.Hkv, h = i - t * a.Hkv;
      if (tok[t].page < 0) continue;
      const size_t at = (size_t(tok[t].b) * a.Hkv + h) * (size_t(a.max_pages) * a.P) + tok[t].slot;
      if (a.key_weights) a.key_weights[at] = 0.f;
      if (a.key_positions) a.key_positions[at] = a.positions[n0 + t];
    }
  }
}

// f * factor * weight, the weight of chunk c of its row (null: ones).
__device__ __forceinline__ void normed(float (&f)[8], float factor, const float* weight, int c) {
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] *= factor;
  if (weight == nullptr) return;
  const float4 lo = reinterpret_cast<const float4*>(weight)[2 * c], hi = reinterpret_cast<const float4*>(weight)[2 * c + 1];
  const float w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] *= w[e];
}

__device__ __forceinline__ float squares(const float (&f)[8]) {
  float x = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) x = fmaf(f[e], f[e], x);
  return x;
}

constexpr int kPasses = 5;  // over a CTA's units, at most

// U: units of a thread in flight.  NORM: the first DV columns of the (latent) keys are normalised.
template <int DK, int DV, bool FP8, int U, bool NORM>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendArgs a,
                                                          int tok_per_cta) {
  constexpr int UK = DK / 16, UV = DV / 16;  // units of a q or k row, of a v row
  __shared__ Token tok[kMaxTok];
  // Cosines and sines of two pairs of a chunk to a float4 (c, c, s, s), the
  // chunks of a row side by side: its lanes read consecutive 16 bytes.
  __shared__ float4 cs[kMaxTok * kMaxRotPairs / 2];
  static_assert(!NORM || DK != DV, "rows of 128 are normalised by append_rows_kernel");
  __shared__ float factor[NORM ? kMaxTok : 1];  // of the tokens' latent rows
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
  // A token's latent queries: the units that are not rotated first, rows one behind the
  // other (with 64 rotated columns a warp's units are a row's 512 others), which are copied as
  // they are, then those that are.  (29k tokens of 17 rows into e4m3: 180 us, with every row's
  // units together and unpacked 189.)
  const int turning = rotc / 2, plain = UK - turning;
  // Unit i of the CTA: kind 0 q, 1 k, 2 v; token, head row, chunks.
  auto unit = [&](int i, int& kind, int& t, int& row, int& c0, int& c1) {
    t = int(__umulhi(unsigned(i), a.per_tok_magic));  // i / per_tok
    int u = i - t * per_tok;
    kind = u < qu ? 0 : u < qu + ku ? 1 : 2;
    if (DK != DV && kind == 0) {
      if (u < a.Hq * plain) {
        row = plain == 32 ? u >> 5 : u / plain;
        c0 = 2 * (u - row * plain);
        c0 += c0 >= rot0 ? rotc : 0;
        c1 = c0 + 1;
      } else {
        u -= a.Hq * plain;
        row = u / turning;
        c0 = rot0 + (u - row * turning) * (halves ? 1 : 2);
        c1 = c0 + (halves ? turning : 1);
      }
    } else if (kind < 2) {
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
        const Token t = place_of(a, n, lane, blockIdx.y == 0);
        if (lane == 0) tok[i] = t;
        if (NORM) {
          const uint4* src = reinterpret_cast<const uint4*>(k + int64_t(i) * int(a.k_stride));
          float x = 0.f;
#pragma unroll
          for (int c = 0; c < DV / 8; c += 32) {
            float f[8];
            unpack8(src[c + lane], f);
            x += squares(f);
          }
#pragma unroll
          for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
          if (lane == 0) factor[i] = rsqrtf(fmaf(x, 1.f / DV, a.eps));
        }
      }
      sines(a, n0, ntok, cs);
      __syncthreads();
      if (blockIdx.y == 0) new_state(a, n0, ntok, tok);
    }
#pragma unroll
    for (int r = 0; r < U; ++r) {
      if (tag[r] == ~0u) continue;
      const int t = tag[r] & 31, kind = tag[r] >> 5 & 3, c0 = tag[r] >> 7 & 127, c1 = tag[r] >> 14 & 127, row = rows[r];
      const Token tk = tok[t];
      if (tk.b < 0 || (kind > 0 && tk.page < 0)) continue;
      if (DK != DV && kind == 0 && (c0 < rot0 || c0 >= rot0 + rotc)) {
        uint4* dst = reinterpret_cast<uint4*>(q_out + int64_t(t) * int(a.q_out_stride) + row * DK);
        dst[c0] = x0[r];
        dst[c1] = x1[r];
        continue;
      }
      float f0[8], f1[8];
      unpack8(x0[r], f0);
      unpack8(x1[r], f1);
      if (NORM && kind == 1) {
        if (c0 < DV / 8) normed(f0, factor[t], a.k_weight, c0);
        if (c1 < DV / 8) normed(f1, factor[t], a.k_weight, c1);
      }
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

// Two numbers at once.
using Two = unsigned long long;
__device__ __forceinline__ Two two(float x, float y) {
  Two z;
  asm("mov.b64 %0, {%1, %2};" : "=l"(z) : "f"(x), "f"(y));
  return z;
}
__device__ __forceinline__ void one(Two z, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(z)); }
__device__ __forceinline__ Two mul2(Two x, Two y) {
  Two z;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(z) : "l"(x), "l"(y));
  return z;
}
__device__ __forceinline__ Two fma2(Two x, Two y, Two w) {
  Two z;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(z) : "l"(x), "l"(y), "l"(w));
  return z;
}
__device__ __forceinline__ Two sub2(Two x, Two y) {
  Two z;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(z) : "l"(x), "l"(y));
  return z;
}

// Rows of 128 with norms: eight lanes to a row, whatever it is (query, key or value),
// each with the same two chunks of every row; components go two to an instruction.
struct RowShape {
  int nq, nk, per_tok;     // rows of a token: queries, and keys before nk, and values
  int rot0, rotc, turned;  // rotated chunks, those with pairs of their own
  bool halves;
  int w[4];                // float4s of a row of weights that are for this lane's chunks
  int c0, c1;              // this lane's chunks: the two halves of eight pairs while it
                           //   counts rotated pairs half a row apart, then the other chunks in order
  __device__ __forceinline__ RowShape(const AppendArgs& a, int l) {
    nq = a.q ? a.Hq : 0;
    nk = nq + a.Hkv;
    per_tok = nk + a.Hkv;
    rot0 = a.rope.rot_offset / 8;
    rotc = a.rope.rot_dim / 8;
    halves = a.rope.pairing == SPLITKV_ROPE_HALVES;
    turned = a.rope.rot_dim / 2 / (halves ? 8 : 4);
    c0 = 2 * l;
    c1 = c0 + 1;
    if (halves && rotc) {
      if (l < rotc / 2) {
        c0 = rot0 + l;
        c1 = c0 + rotc / 2;
      } else {
        c0 -= rotc;
        c1 -= rotc;
        c0 += c0 >= rot0 ? rotc : 0;
        c1 += c1 >= rot0 ? rotc : 0;
      }
    }
    w[0] = 2 * c0;
    w[1] = 2 * c0 + 1;
    w[2] = 2 * c1;
    w[3] = 2 * c1 + 1;
  }
};

// This lane's chunks x0, x1 of row `row` of N tokens, the first of them n (those that
// `live` says), normalised, turned by `z` (the tokens' sines, one behind the other) and stored.
// SHARED: the weights are in shared memory, the keys' from k_at on.
template <bool FP8, int N, bool SHARED>
__device__ __forceinline__ void append_row(const AppendArgs& a, const RowShape& sh, int64_t n, int row, const Token (&tk)[N],
                                           const bool (&live)[N], const uint4 (&x0)[N], const uint4 (&x1)[N],
                                           const float4* z, const ulonglong2* shared = nullptr, int k_at = 0) {
  const int nq = sh.nq, nk = sh.nk, rot0 = sh.rot0, rotc = sh.rotc, turned = sh.turned, c0 = sh.c0, c1 = sh.c1;
  const int lane = threadIdx.x & 31;
  const bool is_q = row < nq, is_k = !is_q && row < nk;
  const int head = is_q ? row : is_k ? row - nq : row - nk;
  uint4 y0[N], y1[N];
  Two f0[N][4], f1[N][4];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    y0[i] = x0[i];
    y1[i] = x1[i];
    const uint32_t w0[4] = {x0[i].x, x0[i].y, x0[i].z, x0[i].w}, w1[4] = {x1[i].x, x1[i].y, x1[i].z, x1[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f0[i][e] = two(__uint_as_float(w0[e] << 16), __uint_as_float(w0[e] & 0xffff0000u));
      f1[i][e] = two(__uint_as_float(w1[e] << 16), __uint_as_float(w1[e] & 0xffff0000u));
    }
  }
  if (is_q || is_k) {
    if (is_q ? a.norm_q : a.norm_k) {
      float x[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        Two sq = mul2(f0[i][0], f0[i][0]);
#pragma unroll
        for (int e = 1; e < 4; ++e) sq = fma2(f0[i][e], f0[i][e], sq);
#pragma unroll
        for (int e = 0; e < 4; ++e) sq = fma2(f1[i][e], f1[i][e], sq);
        float y;
        one(sq, x[i], y);
        x[i] += y;
      }
      // (a row's lanes are neighbours, none of which or all are here)
#pragma unroll
      for (int o = 4; o; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] += __shfl_xor_sync(0xffu << (lane & 24), x[i], o);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        x[i] = rsqrtf(fmaf(x[i], 1.f / 128, a.eps));
        const Two by = two(x[i], x[i]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          f0[i][e] = mul2(f0[i][e], by);
          f1[i][e] = mul2(f1[i][e], by);
        }
      }
      if (is_q ? a.q_weight : a.k_weight) {
        const int row_at = (is_q ? a.q_per_head : a.k_per_head) ? head * 32 : 0;
        ulonglong2 p0, p1, p2, p3;
        if (SHARED) {
          // (a lane's float4s lie 8 apart, so that the lanes' are side by side)
          const ulonglong2* w = shared + (is_q ? 0 : k_at) + row_at + (lane & 7);
          p0 = w[0];
          p1 = w[8];
          p2 = w[16];
          p3 = w[24];
        } else {
          const ulonglong2* w = reinterpret_cast<const ulonglong2*>(is_q ? a.q_weight : a.k_weight) + row_at;
          p0 = w[sh.w[0]];
          p1 = w[sh.w[1]];
          p2 = w[sh.w[2]];
          p3 = w[sh.w[3]];
        }
        const Two w0[4] = {p0.x, p0.y, p1.x, p1.y}, w1[4] = {p2.x, p2.y, p3.x, p3.y};
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            f0[i][e] = mul2(f0[i][e], w0[e]);
            f1[i][e] = mul2(f1[i][e], w1[e]);
          }
      }
    }
    if (sh.halves) {
      if (c0 >= rot0 && c0 < rot0 + rotc) {  // then c1 is the other half of the pairs
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const ulonglong2 w =  // cosines, sines
                *reinterpret_cast<const ulonglong2*>(z + i * (kMaxRotPairs / 2) + e * turned + c0 - rot0);
            const Two u = f0[i][e];
            f0[i][e] = sub2(mul2(u, w.x), mul2(f1[i][e], w.y));
            f1[i][e] = fma2(u, w.y, mul2(f1[i][e], w.x));
          }
      }
    } else {
      auto both = [&](Two (&f)[4], const float4* zi, int c) {
        if (c < rot0 || c >= rot0 + rotc) return;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4 w = zi[(e >> 1) * turned + c - rot0];
          const float co = e & 1 ? w.y : w.x, si = e & 1 ? w.w : w.z;
          float u, v;
          one(f[e], u, v);
          f[e] = two(u * co - v * si, u * si + v * co);
        }
      };
#pragma unroll
      for (int i = 0; i < N; ++i) {
        both(f0[i], z + i * (kMaxRotPairs / 2), c0);
        both(f1[i], z + i * (kMaxRotPairs / 2), c1);
      }
    }
    if (!FP8 || is_q) {
      auto pack = [](const Two (&f)[4]) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float lo, hi;
          one(f[e], lo, hi);
          w[e] = pack_bf16(lo, hi);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
      };
#pragma unroll
      for (int i = 0; i < N; ++i) {
        y0[i] = pack(f0[i]);
        y1[i] = pack(f1[i]);
      }
    }
  }
  if (is_q) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (!live[i]) continue;
      uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.q_out) + (n + i) * a.q_out_stride + row * 128);
      dst[c0] = y0[i];
      dst[c1] = y1[i];
    }
    return;
  }
  void* pool = is_k ? a.k_pages : a.v_pages;
  const float* per_head = is_k ? a.k_scale : a.v_scale;
  const float sc = FP8 ? per_head ? per_head[head] : a.kv_scale : 1.f;
  // (the reciprocal of a power of two is exact, and then so is the product)
  const uint32_t bits = __float_as_uint(sc);
  const bool exact = (bits & 0x7fffffu) == 0 && bits >= 0x01000000u && bits < 0x7e000000u;
  const float inv = __uint_as_float(0x7f000000u - bits);
  auto codes = [&](const Two (&f)[4]) {
    float x[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) one(f[e], x[2 * e], x[2 * e + 1]);
    if (exact) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= inv;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = __fdiv_rn(x[e], sc);
    }
    return make_uint2(pack_e4m3x4(x), pack_e4m3x4(x + 4));
  };
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (!live[i] || tk[i].page < 0) continue;
    const size_t line = a.nhd ? (size_t(tk[i].page) * a.P + tk[i].in_page) * a.Hkv + head
                              : (size_t(tk[i].page) * a.Hkv + head) * a.P + tk[i].in_page;
    if (FP8) {
      uint2* dst = reinterpret_cast<uint2*>(static_cast<uint8_t*>(pool) + line * 128);
      dst[c0] = codes(f0[i]);
      dst[c1] = codes(f1[i]);
    } else {
      uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(pool) + line * 128);
      dst[c0] = y0[i];
      dst[c1] = y1[i];
    }
  }
}

// A short call: a row per lane group in flight, as many CTAs as that makes.
template <bool FP8>
__global__ void __launch_bounds__(kThreads) append_rows_kernel(const __grid_constant__ AppendArgs a, int tok_per_cta) {
  constexpr int kGroups = kThreads / 8;
  __shared__ Token tok[kMaxTok];
  __shared__ float4 cs[kMaxTok * kMaxRotPairs / 2];  // (as in append_kernel)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  launch_dependents();
  wait_prerequisites();

  const int n0 = blockIdx.x * tok_per_cta;
  const int ntok = min(tok_per_cta, a.n_tokens - n0);
  const RowShape sh(a, threadIdx.x & 7);
  const int total = ntok * sh.per_tok;

  bool ready = false;
  for (int base = blockIdx.y * kGroups; base < total || !ready; base += gridDim.y * kGroups) {
    // The token's own row first (that of padding is within the inputs too): it is in
    // flight while the tokens' places are looked up.
    const int j = base + (threadIdx.x >> 3);
    const int t = int(__umulhi(unsigned(j), a.per_tok_magic)), row = j - t * sh.per_tok;
    uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0;
    if (j < total) {
      const int kind = row < sh.nq ? 0 : row < sh.nk ? 1 : 2, head = kind == 0 ? row : kind == 1 ? row - sh.nq : row - sh.nk;
      const __nv_bfloat16* from = static_cast<const __nv_bfloat16*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v);
      const int64_t stride = kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride;
      const uint4* src = reinterpret_cast<const uint4*>(from + (n0 + t) * stride + head * 128);
      x0 = src[sh.c0];
      x1 = src[sh.c1];
    }
    if (!ready) {
      ready = true;
      for (int i = warp; i < ntok; i += kThreads / 32) {
        const Token p = place_of(a, n0 + i, lane, blockIdx.y == 0);
        if (lane == 0) tok[i] = p;
      }
      sines(a, n0, ntok, cs);
      __syncthreads();
      if (blockIdx.y == 0) new_state(a, n0, ntok, tok);
    }
    if (j >= total) continue;
    const Token tk = tok[t];
    if (tk.b >= 0)
      append_row<FP8, 1, false>(a, sh, n0 + t, row, {tk}, {true}, {x0}, {x1}, cs + t * (kMaxRotPairs / 2));
  }
}

// A long call.  Norm, weights and rotation take a row so long that loads which wait for
// them leave the memory idle (threads that load their own rows, four CTAs to an SM: 143 us
// for 32k tokens of 40 rows).  Here two CTAs stay on each SM, and a token's rows come by
// bulk copies (its heads are adjacent) into a ring of stages of a few tokens, asked for as
// soon as a stage is free; two warps look up the places and compute the sines of the
// stages ahead (one warp: 122 us, four, which leave the others fewer registers, 119).
// Measured: 106 us, 6.2 TB/s (floor 97 at the copy's 6.8); into e4m3 110 (floor 92).
struct Stream {
  int tps;       // tokens of a stage
  int stages;
  int w_floats;  // of the weights that are copied to shared memory first: q's, then k's; 0: none
};
constexpr int kStreamTok = 4, kStreamStages = 4;  // (tokens: even)
constexpr int kStreamInfo = 64;  // threads for places and sines
constexpr int kStreamThreads = kThreads + 32 + kStreamInfo;  // warp 8: copies
struct StreamInfo {
  float4 cs[kStreamTok * kMaxRotPairs / 2];
  Token tok[kStreamTok];
};

template <bool FP8, bool SHARED>
__global__ void __launch_bounds__(kStreamThreads, 2) append_stream_kernel(const __grid_constant__ AppendArgs a, const Stream st) {
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ uint64_t bars[2 * kStreamStages];
  __shared__ StreamInfo info[kStreamStages];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const RowShape sh(a, threadIdx.x & 7);
  const int q_bytes = sh.nq * 256, k_bytes = a.Hkv * 256, tok_bytes = q_bytes + 2 * k_bytes;
  float* weights = reinterpret_cast<float*>(sm);
  uint8_t* ring = sm + st.w_floats * 4;
  auto full = [&](int s) { return smem_u32(bars + s); };
  auto empty = [&](int s) { return smem_u32(bars + kStreamStages + s); };
  if (threadIdx.x == 0) {
    for (int s = 0; s < st.stages; ++s) {
      mbar_init(full(s), 1 + kStreamInfo / 32);  // copies; places and sines
      mbar_init(empty(s), kThreads / 32);
    }
    fence_mbar_init();
  }
  launch_dependents();
  wait_prerequisites();
  const int k_at = !a.q_weight ? 0 : a.q_per_head ? a.Hq * 32 : 32;  // (float4s)
  if (SHARED) {
    for (int i = threadIdx.x; i < st.w_floats / 4; i += kStreamThreads) {
      const float4* from = reinterpret_cast<const float4*>(i < k_at ? a.q_weight : a.k_weight) + ((i < k_at ? i : i - k_at) & ~31);
      reinterpret_cast<float4*>(weights)[i] = from[RowShape(a, i & 7).w[i >> 3 & 3]];
    }
  }
  __syncthreads();

  const int groups = (a.n_tokens + st.tps - 1) / st.tps;
  bool ok = true;
  int it = 0;
  auto each = [&](auto&& body) {
    for (int g = blockIdx.x; g < groups && ok; g += gridDim.x, ++it) {
      const int n0 = g * st.tps;
      body(it % st.stages, it / st.stages, n0, min(st.tps, a.n_tokens - n0));
    }
  };
  if (warp == kThreads / 32) {
    // ---- copies
    each([&](int s, int use, int n0, int ntok) {
      if (use > 0) ok = __all_sync(kFull, mbar_wait(empty(s), (use - 1) & 1));
      if (!ok) return;
      if (lane == 0) mbar_arrive_expect_tx(full(s), uint32_t(ntok * tok_bytes));
      __syncwarp();
      if (lane < ntok) {
        const uint32_t dst = smem_u32(ring) + uint32_t(s * st.tps + lane) * tok_bytes;
        const int64_t n = n0 + lane;
        if (q_bytes) bulk_load(dst, static_cast<const __nv_bfloat16*>(a.q) + n * a.q_stride, q_bytes, full(s));
        bulk_load(dst + q_bytes, static_cast<const __nv_bfloat16*>(a.k) + n * a.k_stride, k_bytes, full(s));
        bulk_load(dst + q_bytes + k_bytes, static_cast<const __nv_bfloat16*>(a.v) + n * a.v_stride, k_bytes, full(s));
      }
    });
    if (!ok) --it;  // (not asked for)
    // stay until every copy has landed: the last use of each stage
    for (int i = it - 1; i >= 0 && i >= it - st.stages; --i) mbar_wait(full(i % st.stages), (i / st.stages) & 1);
  } else if (warp > kThreads / 32) {
    // ---- places (the first of the warps) and sines
    const int part = threadIdx.x - kThreads - 32;
    const int half = a.rope.rot_dim / 2, chunk_pairs = sh.halves ? 8 : 4;
    each([&](int s, int use, int n0, int ntok) {
      if (use > 0) ok = __all_sync(kFull, mbar_wait(empty(s), (use - 1) & 1));
      if (!ok) return;
      StreamInfo& to = info[s];
      if (part < ntok) {
        const int n = n0 + part;
        int b = n / a.T;
        if (a.cu) {
          int lo = 0, hi = a.batch;  // how many sequences have ended
          while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (a.cu[mid + 1] <= n) lo = mid + 1;
            else hi = mid;
          }
          b = lo < a.batch && a.cu[0] <= n ? lo : -1;
        }
        to.tok[part] = place_in(a, b, n, true);
      }
      for (int p = part; p < half; p += kStreamInfo) {  // (a pair's place once, for all tokens)
        const int ch = p / chunk_pairs, e = p - ch * chunk_pairs;
        float* z = reinterpret_cast<float*>(to.cs + (e >> 1) * sh.turned + ch) + (e & 1);
        const int32_t* at = a.positions + size_t(a.rope.axis[p]) * a.n_tokens + n0;
        const uint64_t turns = a.rope.turns[p];
        int32_t pos[kStreamTok];
#pragma unroll
        for (int t = 0; t < kStreamTok; ++t) pos[t] = at[min(t, ntok - 1)];
#pragma unroll
        for (int t = 0; t < kStreamTok; ++t) {
          float s, c;
          sincospif(float(int32_t((uint64_t(int64_t(pos[t])) * turns) >> 32)) * 0x1p-31f, &s, &c);
          if (t >= ntok) break;
          z[t * (2 * kMaxRotPairs)] = c;
          z[t * (2 * kMaxRotPairs) + 2] = s;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(full(s));
      if (part < 32) new_state<32>(a, n0, ntok, to.tok, part);
      __syncwarp();
    });
  } else {
    // ---- rows
    each([&](int s, int use, int n0, int ntok) {
      ok = __all_sync(kFull, mbar_wait(full(s), use & 1));
      if (!ok) return;
      const uint8_t* rows = ring + size_t(s) * st.tps * tok_bytes;
      const StreamInfo& from = info[s];
      // (the same row of two tokens at a time: their latencies overlap, and the weights serve both)
      for (int j = threadIdx.x >> 3; j < (ntok + 1) / 2 * sh.per_tok; j += kThreads / 8) {
        const int pair = int(__umulhi(unsigned(j), a.per_tok_magic)), row = j - pair * sh.per_tok, t = 2 * pair;
        const int t2 = min(t + 1, ntok - 1);
        const Token tk[2] = {from.tok[t], from.tok[t2]};
        const bool live[2] = {tk[0].b >= 0, t2 > t && tk[1].b >= 0};
        if (!live[0] && !live[1]) continue;
        const uint4* s0 = reinterpret_cast<const uint4*>(rows + t * tok_bytes + row * 256);
        const uint4* s1 = reinterpret_cast<const uint4*>(rows + t2 * tok_bytes + row * 256);
        append_row<FP8, 2, SHARED>(a, sh, n0 + t, row, tk, live, {s0[sh.c0], s1[sh.c0]}, {s0[sh.c1], s1[sh.c1]},
                                   from.cs + t * (kMaxRotPairs / 2), reinterpret_cast<const ulonglong2*>(weights), k_at);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(s));
    });
  }
  if (!ok && lane == 0 && a.status) atomicOr(a.status, SPLITKV_DEVERR_TIMEOUT);
}

// The grid of a call, tokens of a CTA first.  A pass is the units (or rows) that a CTA
// has in flight; `longer`: a long call.
dim3 append_grid(AppendArgs& a, int per_tok, int pass, bool longer, int* tok_per_cta) {
  // i * magic >> 32 is i / per_tok for every unit i of a CTA, as i * per_tok is
  // below 2^32 or the CTA has one token (0: that token's, however many units)
  a.per_tok_magic = per_tok > 65536 ? 0 : unsigned(((uint64_t(1) << 32) + per_tok - 1) / per_tok);
  // A CTA's tokens.  In a long call the first number, of two passes or more over
  // its units (which share the lookup of the places and the sines: 26k tokens of
  // 40 rows, 99 us, with one pass 106), that leaves at most a twelfth of the
  // threads idle in the last, or else the best within kPasses (29k tokens of 17
  // latent rows, e4m3: four tokens 172 us, one 230, before plain units went by themselves).  A token of more units than
  // that goes to several CTAs.
  const int most = (longer ? kPasses : 1) * pass;
  const int64_t slices = (int64_t(per_tok) + most - 1) / most;
  int most_tok = max(1, min(kMaxTok, most / per_tok)), tpc = most_tok;
  if (longer) {
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
  *tok_per_cta = tpc;
  return dim3((a.n_tokens + tpc - 1) / tpc, unsigned(slices > 65535 ? 65535 : slices), 1);
}

cudaError_t launch_append_kernel(void (*kernel)(AppendArgs, int), const AppendArgs& args, int per_tok, int pass, bool longer,
                                 cudaStream_t s) {
  AppendArgs a = args;
  int tpc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = append_grid(a, per_tok, pass, longer, &tpc);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute la[1];
  la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  la[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = la;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, tpc);
}

// A call of few tokens takes one unit per thread, to use more of the GPU's
// SMs (32 tokens: 3.7 us, with four 8.8); a long one two, for bytes in flight
// (26k tokens: 97.8 us, with one 239, with four 99.2, with six 126; in e4m3
// 100, with four 137).
constexpr int64_t kFewUnits = 1 << 17;

// Rows with norms: what the stages of a CTA of a long call hold, how many they are at
// least, and the weights beside them (two CTAs to an SM); and the rows of a short call.
constexpr int kStreamBytes = 80 * 1024, kStreamMin = 2, kStreamWeights = 20 * 1024;
constexpr int64_t kShortRows = 1 << 16;  // (62k rows: 14.4 us either way, 34k 8.6 and 9.7, 240k 42.9 and 31.6)

template <int DK, int DV, bool FP8, bool NORM = false>
cudaError_t launch_append_t(const AppendArgs& a, cudaStream_t s) {
  const int per_tok = (a.q ? a.Hq * (DK / 16) : 0) + a.Hkv * (DK / 16 + (a.v ? DV / 16 : 0));
  return int64_t(per_tok) * a.n_tokens <= kFewUnits
             ? launch_append_kernel(append_kernel<DK, DV, FP8, 1, NORM>, a, per_tok, kThreads, false, s)
             : launch_append_kernel(append_kernel<DK, DV, FP8, 2, NORM>, a, per_tok, 2 * kThreads, true, s);
}

template <bool FP8>
cudaError_t launch_append_rows(const AppendArgs& args, cudaStream_t s) {
  AppendArgs a = args;
  const int per_tok = (a.q ? a.Hq : 0) + 2 * a.Hkv, tok_bytes = per_tok * 256;
  Stream st;
  st.tps = min(kStreamTok, kStreamBytes / kStreamMin / tok_bytes);
  if (st.tps > 1) st.tps &= ~1;
  if (st.tps < 1 || int64_t(per_tok) * a.n_tokens <= kShortRows)
    return launch_append_kernel(append_rows_kernel<FP8>, a, per_tok, kThreads / 8, false, s);
  st.stages = min(kStreamStages, kStreamBytes / (st.tps * tok_bytes));
  st.w_floats = (a.q_weight ? a.q_per_head ? a.Hq * 128 : 128 : 0) + (a.k_weight ? a.k_per_head ? a.Hkv * 128 : 128 : 0);
  if (st.w_floats * 4 > kStreamWeights) st.w_floats = 0;
  a.per_tok_magic = unsigned(((uint64_t(1) << 32) + per_tok - 1) / per_tok);
  static std::atomic<uint64_t> allowed[2];
  auto* kernel = st.w_floats ? append_stream_kernel<FP8, true> : append_stream_kernel<FP8, false>;
  cudaError_t e = allow_shared_memory(reinterpret_cast<const void*>(kernel), kStreamBytes + kStreamWeights, allowed[st.w_floats != 0]);
  if (e != cudaSuccess) return e;
  const int groups = (a.n_tokens + st.tps - 1) / st.tps;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(min(2 * kSmCount, groups)), 1, 1);
  cfg.blockDim = dim3(kStreamThreads, 1, 1);
  cfg.dynamicSmemBytes = size_t(st.w_floats) * 4 + size_t(st.stages) * st.tps * tok_bytes;
  cfg.stream = s;
  cudaLaunchAttribute la[1];
  la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  la[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = la;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, st);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, int qk_dim, int v_dim, bool fp8, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (qk_dim == 128 && v_dim == 128) {
    if (a.norm_q || a.norm_k) return fp8 ? launch_append_rows<true>(a, s) : launch_append_rows<false>(a, s);
    return fp8 ? launch_append_t<128, 128, true>(a, s) : launch_append_t<128, 128, false>(a, s);
  }
  if (a.norm_k) return fp8 ? launch_append_t<576, 512, true, true>(a, s) : launch_append_t<576, 512, false, true>(a, s);
  return fp8 ? launch_append_t<576, 512, true>(a, s) : launch_append_t<576, 512, false>(a, s);
}

}  // namespace splitkv
