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
// two MMA row blocks A and B of 128; an item is one (sequence, KV head, row
// tile) over all key blocks of 128.  Per key block and row block:
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
// Where a power of two of at most 32 query heads share a KV head, 32 rows of it are a
// box of the queries' and the results' tensors: a warp's Q comes, and its whole results
// go, by TMA.  (Others go by 16 bytes a lane, row by row.  Trees of 64 young requests: 50
// us, by lanes 71; the prompts below 715 and 735; in larger code.)
//
// K and V blocks pass in that order through one ring of five 32 KB slots that
// two producer warps fill by TMA, each a 64-column half of every slot, one box
// per page piece, 128-byte swizzled; K is read K-major, V with its dims on N.
// TMEM columns: S_A [0, 128), S_B [128, 256), O_A [256, 384), O_B [384, 512).
//
// Many items: a CTA per item (prompts), or a line of all items' key blocks that the
// CTAs share (batches of few rows a sequence; cross_deal has the rule).  The bound
// of prompts is 4 * 128 * rows * L operations.  Two sequences of 4k tokens, 32 heads on 4, over 8k keys: 675 to
// 715 us, 1,490 to 1,585 TFLOP/s (floor 561 at 1,906), near the GPU's limit of
// 1,400 W and with the tensor pipe waiting for the softmax's turn of the row
// blocks.
//
// Few items (a decoder token over the encoder's states, short prompts): one CTA
// per SM, which finds by the device lengths how finely to cut the items' keys
// and walks its pieces (the ring and the barriers run on across them); cut
// items leave partial results that cross_merge_kernel joins by their
// log-sum-exps.  An item of up to 128 rows uses the second row block for every
// other key block of the same rows.  Bound: the bytes of K and V, some 43 bytes
// a nanosecond into each SM once the copies flow, behind a start of 5 us (2.3
// the plan, 2.6 the first blocks), an end of 3 (the last softmax, P . V, the
// result) and the merge's 1.5 (one token of 8 requests over 1.2k keys of 16
// heads: 25 us, floor 11.6), or the longest piece's chain of products and the
// 32-bit partial results (prompts of 37 to 900 tokens over 1 to 4.1k keys:
// 21.4 us, floor 2.9).
//
// The code is kept small: what runs once in a piece waits for its own instructions, and
// the loops of all warps together have to stay in the SM's instruction cache.  So waits
// and what is rare are rolled or functions of their own, the next piece is taken in two
// places, and the MMAs stand in a branch that one elected lane takes, not under its
// predicate, where each is some 30 instructions.  With all that (200 KB of code before,
// 146 after) the prompts above 707 -> 690 us, one token of 8 requests 27.2 -> 25, of 512
// requests over 512 keys 236 -> 218, trees of 8 tokens over 5.9k keys 16.7 -> 15.  (Too small: the
// producers' boxes in a rolled loop, trees of 32 requests over up to 131k keys 587 us
// for 567; the rescaling of O and the loop over the row blocks stay as they are.)
//
// P is rounded to bf16 for the second product (half a step, 2^-8 of a weight,
// as in the decode kernels); sums, maxima and O are fp32.
//
// TREE (splitkv_tree_attend): the query tokens are the last T_b of the sequence's
// own keys, drafted as a tree, and see the keys before them and those of the tree
// that their mask names.  Only the key blocks that reach past L - T_b are masked: a
// thread shifts its row's mask words to the block's keys, and takes -inf for the
// scores whose bit is off.  The V rows that no token of the tile sees are zeroed,
// as those behind the length are (0 * NaN would be NaN).  The trees' line (plan_line)
// takes any lengths, as an item counts there for what it costs beside its blocks.
// Measured, bf16: 8 tokens over 5.9k keys 14 us (floor 0.9: the chain of plan, first
// blocks, one softmax, result and merge), 400 tokens of 32 requests over 256 to 131k keys
// 563 us (floor 529), trees of 64 requests over 1 to 300 keys 43 us (floor 9: an item's
// chain is 9 us, a CTA to an SM).
//
// Trees' softmax holds 64 columns of S at a time and reads half of S twice, in loops of
// half the length, for the instruction cache again, in which a neighbour at another kind
// of piece takes its share.  (Before the code was made smaller: trees of 33 tokens of 8
// requests over 31k keys in e4m3, pieces of 256 and of 8 rows: 222 us, all of S in
// registers 286, with three times the misses there; 64 tokens of 19 requests over 8k keys
// 131 both.  Parts of 32: 205 and 138.  Cross attention's long prompts, all at the same
// code, take 750 us in halves and 707 so.)
//
// FP8 (e4m3 caches, with TREE): K is multiplied as it is stored.  A query row, times the
// power of two that brings its largest component into [2^7, 2^8), is a sum of two e4m3
// codes a column, four of its eight bits each (exact, but for components below 2^-9 of the
// largest: codes below 2^-6 go in steps of 2^-9, so that their two roundings are off by 2^-9
// together, 2^-16 of the largest, at most), and S is the sum of two products of twice the
// rate.  V's codes land in the second half of their slot, [128 keys][128], just
// where the rows of the second 64 columns will lie, and four converter warps turn each row
// in place into the two swizzled halves, as f16 (exact, one instruction for a pair of codes;
// bf16 would take four).  P is f16 too, times 2^P_UP: a weight is at most 2^8 of the reference
// maximum's, so that at most 2^15 is stored, and the steps of 2^-24 that f16 has below 2^-14 are
// 2^-31 of that maximum's weight (2^-24 without, of which long tails of small weights beside
// one large one lost all that was below a half).  Sums are of the weights times 2^P_UP as well,
// which cancels but in the log-sum-exp.  The caches' scales join the scores' and the results'.  K's ring has four slots of 16 KB, V's three of 32 KB, a producer each.
// Measured: 16 tokens of 19 requests over 8k keys 78 us (floor 47; in bf16 105 of 94), 64
// tokens 130 (in bf16 115), trees of 16 to 61 tokens of 8 requests over 32k keys 133 (floor
// 54).  In larger code 85, 141 and 148; with K converted as well, both in one ring of five slots, and the softmax's
// registers taken from the other warps' (S in one part) the three took 109, 155 and 182.
#pragma once

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
  static constexpr int SOFTMAX_WARPS = 8;
  // warps: two producers (a half of every K and V block each), the issuer of the MMAs
  static constexpr int PRODUCER = SOFTMAX_WARPS, ISSUER = SOFTMAX_WARPS + 2;
  static constexpr uint32_t TMEM_COLS = 512, S_COL = 0, O_COL = 256;  // + 128 per row block
  static constexpr float RESCALE_LOG2 = 8.f;
};
template <bool TREE, bool FP8>
struct CrossCta : Cross {
  static constexpr int PART = TREE ? 64 : 128;  // columns of S that a softmax thread holds
  static constexpr float P_UP = FP8 ? 7.f : 0.f;  // log2 of what P is multiplied with
  static constexpr float P_DOWN = FP8 ? 0x1p-7f : 1.f;
  // e4m3: four converters, none on the issuer's scheduler (every fourth warp; trees of 8
  // requests over 32k keys 147 us, with one there 149)
  static constexpr int CONVERTER = SOFTMAX_WARPS + 3, IDLE = SOFTMAX_WARPS + 6;
  static_assert((IDLE - ISSUER) % 4 == 0, "beside the issuer: no converter");
  static constexpr int WARPS = SOFTMAX_WARPS + (FP8 ? 8 : 3);
  static constexpr int THREADS = WARPS * 32;
  static constexpr int TAIL = FP8 ? 2048 : 1536; // barriers, plan
  static constexpr int SMEM = 1024 + OFF_BAR + TAIL;
  // e4m3: a ring for K's codes, one for V's and what becomes of them
  static constexpr int K_SLOTS = 4, V_SLOTS = 3, SLOTS = K_SLOTS + V_SLOTS;
  static_assert(K_SLOTS * HALF + V_SLOTS * TILE == NST * TILE, "in the place of the one ring");
  static_assert(SMEM <= 227 * 1024, "shared memory budget");
};

enum {
  B_Q = 0,                       // [2] Q of a row block in shared memory (128 threads, or 4 warps' copies)
  B_FULL = 2,                    // [NST]
  B_EMPTY = B_FULL + Cross::NST, // [NST]
  B_S = B_EMPTY + Cross::NST,    // [2] S of a row block complete
  B_P = B_S + 2,                 // [2] P of a row block in TMEM (128 threads)
  B_O = B_P + 2,                 // [2] the last PV of a row block complete
  B_ML = B_O + 2,                // narrow pieces: B's maxima and sums written (128 threads)
  B_JOINED,                      //   A has read them and B's O (128 threads)
  B_DONE,
  B_COUNT,
  // e4m3: instead of B_FULL and B_EMPTY those of K's ring and, K_SLOTS further, of V's;
  // B_CONV [V_SLOTS]: the slot holds f16 (a lane of each converter warp); B_DOWN: the rows' exponents
  // of a narrow piece of two blocks or more (128 threads of A).  (B_Q is for the issuer alone: A fills
  // Q for pieces that B has no part in, without waiting for it, and a turn that B does not
  // see in time it would wait for in vain.  B has a part in all pieces that B_DOWN tells of.)
  B_FULL_FP8 = B_COUNT,
  B_EMPTY_FP8 = B_FULL_FP8 + CrossCta<true, true>::SLOTS,
  B_CONV = B_EMPTY_FP8 + CrossCta<true, true>::SLOTS,
  B_DOWN = B_CONV + CrossCta<true, true>::V_SLOTS,
  B_COUNT_FP8
};

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kRowBox = kRowBoxRows;  // query rows, or rows of the result, of a warp's box

// The length of sequence b, or 0 where the device value is not one the cache
// can hold.
__device__ __forceinline__ int keys_of(const CrossArgs& a, int b) {
  const int L = a.seq_lens[b];
  return L >= 0 && L <= int64_t(a.max_pages) * a.P ? L : 0;
}
// The same for the keys of a tree's sequence, which end with those of its tokens.
template <bool TREE>
__device__ __forceinline__ int keys_of(const CrossArgs& a, int b, int tokens) {
  const int L = keys_of(a, b);
  return TREE && L < tokens ? 0 : L;
}

// First token and number of tokens of sequence b, within [0, n_tokens] whatever the
// offsets are.
__device__ __forceinline__ int tokens_of(const CrossArgs& a, int b, int* first) {
  if (!a.cu) {
    *first = b * a.T;
    return a.T;
  }
  const int t0 = min(max(a.cu[b], 0), a.n_tokens), t1 = min(max(a.cu[b + 1], t0), a.n_tokens);
  *first = t0;
  return t1 - t0;
}

// Key blocks of an item over n_keys keys; an item without keys counts as one
// (it writes its zeros).
__device__ __forceinline__ int blocks_of(int n_keys) { return max(1, (n_keys + Cross::BK - 1) / Cross::BK); }

// One piece of an item: `nblk` key blocks from j0 on (0: an item without keys).
struct Piece {
  int b, h, first, row0, n_rows, L, j0, nblk;  // n_rows: rows from row0 on (may exceed a tile)
  int slot;                                    // of its partial result; -1: the whole item
};
constexpr int kMaxPieces = 4;  // of a CTA
// Where the plan stops counting a KV head's pieces.  A call's items are at most
// kMaxPieces * kSmCount, cut into 32 each; offsets out of order may give every
// sequence all tokens, and a wrapped count would pass for one that fits.
constexpr int kManyPieces = 32767;
static_assert(kMaxPieces * kSmCount * 32 <= kManyPieces && int64_t(kManyPieces) * 65535 < (int64_t(1) << 31), "no call's count");
constexpr int kPieceCost = 2, kCutCost = 2;  // in key blocks: of each piece, and of cutting anything
constexpr int kLineCost = 8;  // and of a line of all key blocks
// What counts in a line: a key block of an item of up to 128 rows and of one of more, and
// an item beside them (trees'; with that the parts of a line cost the same whatever the
// items' lengths are: 400 tokens of 32 requests over 256 to 131k keys took 629 us, with 3
// blocks instead of 10 709, with 14 634; as equal pieces 1,304.  Wide and narrow blocks
// counted alike: 8 to 130 tokens of those 1,006 us, so 968; 400 in e4m3 520 and 483.)
template <bool TREE, bool FP8>
struct Line {
  static constexpr int WIDE = TREE ? 6 : 1, NARROW = TREE ? (FP8 ? 4 : 5) : 1, ITEM = TREE ? 50 : 0;
  static __device__ __forceinline__ int block(int rows) { return rows <= 128 ? NARROW : WIDE; }
};

// Where a warp is in a line: the next key block, and the item that holds it (of sequence b,
// from block `off` on) with its sequence's numbers.
struct Walk {
  int64_t x;
  int b, item, off, first, rows, L, tiles, nb;
};

// Behind the barriers.
template <int WARPS>
struct Tail {
  uint32_t tmem;   // written by the allocation
  int32_t pieces;  // in `piece`; -1: the line's blocks [lo, hi), `share` to a CTA
  int64_t lo, hi, share;  // (those that begin in it)
  Piece piece[kMaxPieces];
  Walk walk[WARPS];
  Piece now[WARPS];
  uint8_t down[128];  // e4m3: of a narrow piece's rows, the exponent of what undoes their power of two
};
static_assert(B_COUNT * 8 + sizeof(Tail<CrossCta<false, false>::WARPS>) <= CrossCta<false, false>::TAIL, "barriers, then the tail");
static_assert(B_COUNT_FP8 * 8 + sizeof(Tail<CrossCta<true, true>::WARPS>) <= CrossCta<true, true>::TAIL, "barriers, then the tail");

// Pieces of about t key blocks that an item of nb is cut into.  (In floating
// point, for speed: any count in 1 .. nb is right, as long as all agree on it.)
__device__ __forceinline__ int cuts_of(int nb, float t) {
  return max(1, min(nb, int(ceilf(__fdividef(float(nb), t) - 1e-3f))));
}

// Lane's sequence of a plan: its first token, query rows, keys, row tiles, and
// the key blocks of each of its items.
struct Lane {
  int first, rows, L, tiles, nb;
};
template <bool TREE>
__device__ __forceinline__ Lane lane_of(const CrossArgs& a, int b) {
  Lane x = {0, 0, 0, 0, 1};
  if (b < a.batch) {
    const int tokens = tokens_of(a, b, &x.first);
    x.L = keys_of<TREE>(a, b, tokens);
    x.rows = tokens * a.G;
    x.tiles = (x.rows + Cross::ROWS - 1) / Cross::ROWS;
    x.nb = blocks_of(x.L);
  }
  return x;
}

// What a sequence's items take of a line.
template <class U>
__device__ __forceinline__ int64_t units_of(const CrossArgs& a, const Lane& s) {
  if (s.tiles == 0) return 0;
  const int last = U::block(s.rows - (s.tiles - 1) * Cross::ROWS);
  return a.Hkv * (int64_t(s.tiles - 1) * (s.nb * U::WIDE + U::ITEM) + s.nb * last + U::ITEM);
}

// Sum over the lanes before this one.
template <class T>
__device__ __forceinline__ T lanes_before(T n, int lane, T* total) {
  T x = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  *total = __shfl_sync(kFull, x, 31);
  return x - n;
}

// The line of plan_pieces: all items' key blocks, one after the other (sequence,
// KV head, row tile), of which CTA c takes `share` from c * share on, whole items
// but for the first and the last (the last CTAs may have less; equal parts cut
// more items and were up to 9 % slower).  Here: where this CTA begins.
//
// Few items, of like lengths and few rows, that do not fill the last round of
// CTAs: one token of 10 requests, 160 items over 152 CTAs, 1.5k keys, takes 42.7
// us, in whole items 49.7; over 4k keys 79 and 111.  kLineCost is what leaves 8
// requests, 27.7 us and as a line 30.2, and 16, 51.8 and 55.3, as they are.
template <bool TREE, int WARPS>
__device__ __noinline__ void plan_line(const CrossArgs& a, int lane, int64_t all, Tail<WARPS>& tail) {
  using U = Line<TREE, WARPS == CrossCta<true, true>::WARPS>;
  // (no CTA between an item's first and its last is without a block of it)
  const int64_t share = max(int64_t(U::WIDE), (all + a.parts - 1) / a.parts);
  const int64_t lo = min(all, int64_t(blockIdx.x) * share), hi = min(all, lo + share);
  Walk w = {lo, 0, 0, 0, 0, 0, 0, 0, 1};
  int64_t passed = 0, total;
  for (int b0 = 0; lo < hi && b0 < a.batch; b0 += 32) {
    const Lane s = lane_of<TREE>(a, b0 + lane);
    const int64_t n = units_of<U>(a, s);
    const int64_t at = passed + lanes_before(n, lane, &total);
    const unsigned m = __ballot_sync(kFull, lo >= at && lo < at + n);
    passed += total;
    if (m) {
      const int f = __ffs(m) - 1;
      w.b = b0 + f;
      w.first = __shfl_sync(kFull, s.first, f);
      w.rows = __shfl_sync(kFull, s.rows, f);
      w.L = __shfl_sync(kFull, s.L, f);
      w.tiles = __shfl_sync(kFull, s.tiles, f);
      w.nb = __shfl_sync(kFull, s.nb, f);
      int64_t in = lo - __shfl_sync(kFull, at, f);
      const int whole = w.nb * U::WIDE + U::ITEM, last = U::block(w.rows - (w.tiles - 1) * Cross::ROWS);
      const int64_t head = int64_t(w.tiles - 1) * whole + w.nb * last + U::ITEM;
      const int h = int(in / head);
      in -= h * head;
      const int tile = min(w.tiles - 1, int(in / whole)), each = tile < w.tiles - 1 ? U::WIDE : last;
      in -= int64_t(tile) * whole;
      w.item = h * w.tiles + tile;
      w.off = min(w.nb, (int(in) + each - 1) / each);
      w.x = lo - in + int64_t(w.off) * each;
      break;
    }
  }
  if (lane < WARPS) tail.walk[lane] = w;
  if (lane == 0) {
    tail.pieces = -1;
    tail.lo = lo;
    tail.hi = hi;
    tail.share = share;
    a.split[blockIdx.x].cuts = 0;
    if (blockIdx.x == 0) *a.n_split = a.parts;
  }
}

// A CTA per item: head blockIdx.y, and a row tile that is found by a search, 32
// sequences at a time.  With x(b) rows before sequence b, its tiles are those from
// number x(b) / ROWS + b on (rounded down): the next sequence's begin late enough,
// and a number past the last tile has nothing to do.  (Adding up the tiles of the
// sequences before would take 0.25 us for every 32 of them, in each CTA.)
template <bool TREE, int WARPS>
__device__ __forceinline__ void plan_one(const CrossArgs& a, int lane, Tail<WARPS>& tail) {
  const int p = blockIdx.x;
  int first0 = 0;
  if (a.cu) first0 = min(max(a.cu[0], 0), a.n_tokens);
  auto number = [&](int b) {
    const int first = a.cu ? min(max(a.cu[b], 0), a.n_tokens) : b * a.T;
    return int64_t(first - first0) * a.G / Cross::ROWS + b;
  };
  int lo = 0, hi = a.batch;  // the last sequence in [lo, hi) whose first number is p or before
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, b = lo + lane * step;
    const unsigned m = __ballot_sync(kFull, b < hi && number(b) <= p);
    lo += m ? (31 - __clz(m)) * step : 0;
    hi = min(hi, lo + step);
  }
  Piece q;
  q.b = lo;
  q.h = blockIdx.y;
  const int tokens = tokens_of(a, lo, &q.first), rows = tokens * a.G;
  const int64_t tile = p - number(lo);
  const bool some = tile >= 0 && tile * Cross::ROWS < rows;
  q.row0 = some ? int(tile) * Cross::ROWS : 0;
  q.n_rows = rows - q.row0;
  q.L = keys_of<TREE>(a, lo, tokens);
  q.j0 = 0;
  q.nblk = q.L > 0 ? blocks_of(q.L) : 0;
  q.slot = -1;
  if (lane == 0) {
    tail.piece[0] = q;
    tail.pieces = some;
  }
}

// By warp `me`, in a line: its next piece, into tail.now[me]; false behind the last.
template <bool TREE, int WARPS>
__device__ __noinline__ bool next_piece(const CrossArgs& a, Tail<WARPS>& tail, int me, int lane) {
  Walk& walk = tail.walk[me];
  __syncwarp();  // (the piece before has been read)
  Walk w = walk;
  using U = Line<TREE, WARPS == CrossCta<true, true>::WARPS>;
  int tile, each;
  auto weigh = [&]() {
    tile = w.tiles > 1 ? w.item % w.tiles : 0;
    each = U::block(w.rows - tile * Cross::ROWS);
  };
  weigh();
  auto item_done = [&]() {
    w.x += (w.nb - w.off) * each + U::ITEM;
    if (w.x >= tail.hi) return;
    w.off = 0;
    if (++w.item == w.tiles * a.Hkv) {  // the next sequence with tokens
      w.item = 0;
      Lane s;
      do s = lane_of<TREE>(a, ++w.b); while (s.tiles == 0 && w.b < a.batch);
      w.first = s.first;
      w.rows = s.rows;
      w.L = s.L;
      w.tiles = s.tiles;
      w.nb = s.nb;
    }
    weigh();
  };
  if (TREE && w.x < tail.hi && w.off >= w.nb) item_done();  // (the line's part begins behind an item's blocks)
  if (w.x >= tail.hi) return false;
  const int len = int(min(int64_t(w.nb - w.off), (tail.hi - w.x + each - 1) / each));  // blocks
  Piece q;
  q.b = w.b;
  q.h = w.tiles > 1 ? w.item / w.tiles : w.item;
  q.first = w.first;
  q.row0 = tile * Cross::ROWS;
  q.n_rows = w.rows - q.row0;
  q.L = w.L;
  q.j0 = w.off;
  q.nblk = w.L > 0 ? len : 0;
  q.slot = len < w.nb ? 2 * int(blockIdx.x) + (w.off == 0) : -1;
  if (me == Cross::ISSUER && lane == 0 && len < w.nb && w.off == 0) {  // (the CTA's last piece: an item's first)
    const int last = int((w.x + (w.nb - 1) * each) / tail.share);  // CTA of the item's last block
    const CrossSplit r = {last - int(blockIdx.x) + 1, q.slot, 2, q.first, q.h, q.row0, min(q.n_rows, Cross::ROWS)};
    a.split[blockIdx.x] = r;
  }
  w.x += len * each;
  w.off += len;
  if (w.off == w.nb && w.x < tail.hi) item_done();
  __syncwarp();
  if (lane == 0) {
    tail.now[me] = q;
    walk = w;
  }
  __syncwarp();
  return true;
}

// By a warp: which pieces this CTA computes.
//
// A CTA per item (a.parts = 0): plan_one.  A line whatever the lengths (a.line):
// plan_line.
//
// Few items: every item of nb key blocks is cut into ceil(nb / t) equal pieces,
// and CTA c takes pieces c, c + parts, ... of the line of all items' pieces.
// Lane i weighs t = ceil(longest nb / (i + 1)): the blocks of the CTA with most,
// kPieceCost for each of its pieces, and kCutCost if anything is cut.  Where few
// rows keep the partial results small and the items, of like lengths, do not fill
// the last round of CTAs, a line may cost less still; that of trees does for any rows
// and lengths, as it counts what an item costs.  (What that
// chooses for 16 heads: two key blocks stay whole, 12.5 us with one token and
// 12.7 cut; four are cut, 13.1 and 14.8 whole, and with 256 tokens 17.3 and 20.2.)
template <bool TREE, int WARPS>
__device__ __forceinline__ void plan_pieces(const CrossArgs& a, int lane, Tail<WARPS>& tail) {
  if (a.parts == 0) {
    plan_one<TREE>(a, lane, tail);
    return;
  }
  Lane mine;
  auto read = [&](int b0) { mine = lane_of<TREE>(a, b0 + lane); };
  int items = 0, longest = 1, shortest = INT32_MAX, widest = 0;
  using U = Line<TREE, WARPS == CrossCta<true, true>::WARPS>;
  int64_t all = 0;  // units of a line
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    read(b0);
    const int64_t units = units_of<U>(a, mine);
    if (a.line) {
      int64_t sum;
      lanes_before(units, lane, &sum);
      all += sum;
      continue;
    }
    all += __reduce_add_sync(kFull, int(min(int64_t(1) << 25, units)));  // (items are few: more need not be exact)
    items += __reduce_add_sync(kFull, mine.tiles);
    longest = max(longest, __reduce_max_sync(kFull, mine.tiles > 0 ? mine.nb : 1));
    shortest = min(shortest, __reduce_min_sync(kFull, mine.tiles > 0 ? mine.nb : INT32_MAX));
    widest = max(widest, __reduce_max_sync(kFull, mine.rows));
  }
  if (a.line) {
    plan_line<TREE>(a, lane, all, tail);
    return;
  }
  items *= a.Hkv;
  const float t = ceilf(__fdividef(longest, lane + 1));
  int n = 0;
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    if (a.batch > 32) read(b0);
    for (int i = 0; i < min(32, a.batch - b0); ++i)
      n = min(n + __shfl_sync(kFull, mine.tiles, i) * cuts_of(__shfl_sync(kFull, mine.nb, i), t), kManyPieces);
  }
  n *= a.Hkv;
  // (cut pieces have a slot each; uncut items need none)
  const bool fits = lane == 0 || n <= 2 * a.parts;
  const uint32_t cost = (n + a.parts - 1) / a.parts * (uint32_t(t) + kPieceCost) + (n > items ? kCutCost : 0);
  const int best = __reduce_min_sync(kFull, fits ? cost * 32 + lane : ~0u) & 31;
  const float T = __shfl_sync(kFull, t, best);
  const int P = __shfl_sync(kFull, n, best);
  const int64_t share = (all + a.parts - 1) / a.parts / U::block(widest);  // key blocks
  if ((TREE || widest <= 128) && all >= a.parts * U::WIDE && all < (1 << 25) && (TREE || share <= 2 * int64_t(shortest)) &&
      share + kLineCost < __shfl_sync(kFull, cost, best)) {
    plan_line<TREE>(a, lane, all, tail);
    return;
  }
  int k = 0;
  for (int p = blockIdx.x; p < P && k < kMaxPieces; p += a.parts, ++k) {
    Piece q;
    int passed = 0, cut_items = 0, total;  // pieces and cut items of the sequences before
    bool found = false;
    for (int b0 = 0; b0 < a.batch && !found; b0 += 32) {
      if (a.batch > 32) read(b0);
      const int s = cuts_of(mine.nb, T);
      const int n = mine.tiles * a.Hkv * s;
      const int at = passed + lanes_before(n, lane, &total);
      const unsigned m = __ballot_sync(kFull, p >= at && p < at + n);
      passed += total;
      const int cut_here = s > 1 ? mine.tiles * a.Hkv : 0;
      if (m) {
        const int f = __ffs(m) - 1;
        found = true;
        const int cuts = __shfl_sync(kFull, s, f);
        const int in = p - __shfl_sync(kFull, at, f);
        const int item = cuts > 1 ? in / cuts : in, cut = in - item * cuts;
        const int ts = __shfl_sync(kFull, mine.tiles, f), blocks = __shfl_sync(kFull, mine.nb, f);
        const int h = ts > 1 ? item / ts : item;
        const int tile = item - h * ts;
        q.b = b0 + f;
        q.h = h;
        q.first = __shfl_sync(kFull, mine.first, f);
        q.row0 = tile * Cross::ROWS;
        q.n_rows = __shfl_sync(kFull, mine.rows, f) - q.row0;
        q.L = __shfl_sync(kFull, mine.L, f);
        const int base = cuts > 1 ? blocks / cuts : blocks, over = blocks - base * cuts;  // `over` pieces have one more
        q.j0 = cut * base + min(cut, over);
        q.nblk = q.L > 0 ? base + (cut < over) : 0;
        q.slot = cuts > 1 ? p : -1;
        if (cuts > 1 && cut == 0) {  // the merge's record, with the first piece of a cut item
          cut_items += __reduce_add_sync(kFull, lane < f ? cut_here : 0);
          const CrossSplit r = {cuts, p, 1, q.first, q.h, q.row0, min(q.n_rows, Cross::ROWS)};
          if (lane == 0) a.split[cut_items + item] = r;
        }
      } else {
        cut_items += __reduce_add_sync(kFull, cut_here);
      }
    }
    if (!found) break;
    if (lane == 0) tail.piece[k] = q;
  }
  if (lane == 0) tail.pieces = k;
  // the number of those records
  if (blockIdx.x == 0) {
    int cut_items = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 32) {
      if (a.batch > 32) read(b0);
      cut_items += __reduce_add_sync(kFull, cuts_of(mine.nb, T) > 1 ? mine.tiles * a.Hkv : 0);
    }
    if (lane == 0) *a.n_split = cut_items;
  }
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

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, "
      "[%16];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16};\n\ttcgen05.wait::st.sync.aligned;" ::"r"(taddr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]),
      "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
      : "memory");
}

__device__ __forceinline__ void tmem_st2(uint32_t taddr, float x, float y) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};\n\ttcgen05.wait::st.sync.aligned;" ::"r"(taddr),
               "f"(x), "f"(y)
               : "memory");
}
__device__ __forceinline__ void tmem_ld2(uint32_t taddr, float& x, float& y) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];\n\ttcgen05.wait::ld.sync.aligned;"
               : "=f"(x), "=f"(y)
               : "r"(taddr)
               : "memory");
}

// 8 columns, without a wait.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
               "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

__device__ __forceinline__ float max3(float x, float y, float z) {
  float m;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(x), "f"(y), "f"(z));
  return m;
}

// Two sums at once.
__device__ __forceinline__ void add2(float& x, float& y, float u, float v) {
  asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\tadd.rn.f32x2 p, p, q;\n\t"
      "mov.b64 {%0, %1}, p;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(u), "f"(v));
}

// (a * s + b) for two numbers at once.
__device__ __forceinline__ void fma2(float& x, float& y, float s, float b) {
  asm("{\n\t.reg .b64 u, v, w;\n\tmov.b64 u, {%0, %1};\n\tmov.b64 v, {%2, %2};\n\tmov.b64 w, {%3, %3};\n\t"
      "fma.rn.f32x2 u, u, v, w;\n\tmov.b64 {%0, %1}, u;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(s), "f"(b));
}

// Eight MMAs of one K = 128 product, issued by a converged warp: one lane,
// elected once, takes the branch that issues all of them (between two MMAs nothing but the next
// descriptors' additions, in units of 16 bytes).
// S = Q . K^T: both operands are two 64-column halves, 32 bytes per step; or (e4m3) Q is
// a sum of two tiles of 128 columns, each multiplied by the one of K.
template <bool FP8>
__device__ __forceinline__ void mma_qk(uint32_t d, uint64_t a_desc, uint64_t b_desc, uint32_t idesc) {
  if constexpr (FP8) {
    asm volatile(
        "{\n\t"
        ".reg .pred e, q, y;\n\t"
        ".reg .b64 a, b;\n\t"
        "setp.ne.b32 q, %4, 0;\n\t"
        "setp.eq.b32 y, 0, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
      "@!e bra DONE%=;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, q;\n\t"
        "add.s64 a, %1, 2;\n\t"
        "add.s64 b, %2, 2;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, y;\n\t"
        "add.s64 a, %1, 4;\n\t"
        "add.s64 b, %2, 4;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, y;\n\t"
        "add.s64 a, %1, 6;\n\t"
        "add.s64 b, %2, 6;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, y;\n\t"
        "add.s64 a, %1, 1024;\n\t"
        "add.s64 b, %2, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, y;\n\t"
        "add.s64 a, %1, 1026;\n\t"
        "add.s64 b, %2, 2;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, y;\n\t"
        "add.s64 a, %1, 1028;\n\t"
        "add.s64 b, %2, 4;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, y;\n\t"
        "add.s64 a, %1, 1030;\n\t"
        "add.s64 b, %2, 6;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, y;\n\t"
        "DONE%=:\n\t"
      "}" ::"r"(d),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(0)
        : "memory");
  } else {
    asm volatile(
        "{\n\t"
        ".reg .pred e, q, y;\n\t"
        ".reg .b64 a, b;\n\t"
        "setp.ne.b32 q, %4, 0;\n\t"
        "setp.eq.b32 y, 0, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
      "@!e bra DONE%=;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, q;\n\t"
        "add.s64 a, %1, 2;\n\t"
        "add.s64 b, %2, 2;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, y;\n\t"
        "add.s64 a, %1, 4;\n\t"
        "add.s64 b, %2, 4;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, y;\n\t"
        "add.s64 a, %1, 6;\n\t"
        "add.s64 b, %2, 6;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, y;\n\t"
        "add.s64 a, %1, 1024;\n\t"
        "add.s64 b, %2, 1024;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, y;\n\t"
        "add.s64 a, %1, 1026;\n\t"
        "add.s64 b, %2, 1026;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, y;\n\t"
        "add.s64 a, %1, 1028;\n\t"
        "add.s64 b, %2, 1028;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, y;\n\t"
        "add.s64 a, %1, 1030;\n\t"
        "add.s64 b, %2, 1030;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, y;\n\t"
        "DONE%=:\n\t"
      "}" ::"r"(d),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(0)
        : "memory");
  }
}
// O (+)= P . V: P in TMEM, 8 columns per step; V 16 keys of 128 bytes per step.
__device__ __forceinline__ void mma_pv(uint32_t d, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t more) {
  asm volatile(
      "{\n\t"
      ".reg .pred e, q, y;\n\t"
      ".reg .b64 b;\n\t"
      ".reg .b32 a;\n\t"
      "setp.ne.b32 q, %4, 0;\n\t"
      "setp.eq.b32 y, 0, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@!e bra DONE%=;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, q;\n\t"
      "add.s32 a, %1, 8;\n\t"
      "add.s64 b, %2, 128;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, y;\n\t"
      "add.s32 a, %1, 16;\n\t"
      "add.s64 b, %2, 256;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, y;\n\t"
      "add.s32 a, %1, 24;\n\t"
      "add.s64 b, %2, 384;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, y;\n\t"
      "add.s32 a, %1, 32;\n\t"
      "add.s64 b, %2, 512;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, y;\n\t"
      "add.s32 a, %1, 40;\n\t"
      "add.s64 b, %2, 640;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, y;\n\t"
      "add.s32 a, %1, 48;\n\t"
      "add.s64 b, %2, 768;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, y;\n\t"
      "add.s32 a, %1, 56;\n\t"
      "add.s64 b, %2, 896;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, y;\n\t"
      "DONE%=:\n\t"
      "}" ::"r"(d),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(more)
      : "memory");
}

// A token's mask beside the keys of a block whose first key lies `d` before the
// drafted ones (or -d behind their first): words m[0 .. 4] of which bit -d + i is for
// key i, ones before the drafted keys and zeros behind the mask.
__device__ __forceinline__ void mask_words(const uint32_t* row, int words, int d, uint32_t (&m)[5]) {
  const int k0 = (-d) >> 5;
#pragma unroll
  for (int i = 0; i < 5; ++i) m[i] = k0 + i < 0 ? ~0u : k0 + i < words ? row[k0 + i] : 0u;
}
// The same as 4 words of the block's keys, of which `valid` exist.
__device__ __forceinline__ void visible(const uint32_t (&m)[5], int d, int valid, uint32_t (&vis)[4]) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const int left = valid - 32 * w;
    vis[w] = __funnelshift_r(m[w], m[w + 1], (-d) & 31) & (left >= 32 ? ~0u : left <= 0 ? 0u : (1u << left) - 1);
  }
}

// mbar_wait in less code.
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
#pragma unroll 1
  for (int i = 1; !mbar_try_wait(bar, parity); ++i)
    if (i % 16 == 0 && clock64() - t0 > kWaitTimeoutCycles) return false;
  return true;
}

// Which of a block's keys some token of tokens t0 .. t1 sees (see mask_words), by a warp.
__device__ __noinline__ uint4 seen_by(const uint32_t* mask, int words, int t0, int t1, int d, int valid, int lane) {
  uint32_t seen[5] = {0u, 0u, 0u, 0u, 0u}, vis[4];
#pragma unroll 1
  for (int tok = t0 + lane; tok <= t1; tok += 32) {
    uint32_t m[5];
    mask_words(mask + int64_t(tok) * words, words, d, m);
#pragma unroll
    for (int i = 0; i < 5; ++i) seen[i] |= m[i];
  }
#pragma unroll
  for (int i = 0; i < 5; ++i) seen[i] = __reduce_or_sync(kFull, seen[i]);
  visible(seen, d, valid, vis);
  return make_uint4(vis[0], vis[1], vis[2], vis[3]);
}
// Zeros over the 16-bit rows of a V block's other keys, by a warp.
__device__ __noinline__ void zero_unseen(uint8_t* rows, uint4 vis, int lane) {
#pragma unroll 1
  for (int w = 0; w < 4; ++w) {
    const uint32_t x = w < 2 ? (w ? vis.y : vis.x) : (w == 2 ? vis.z : vis.w);
    if (~x >> lane & 1)
#pragma unroll 4
      for (int i = 0; i < 16; ++i)  // (in eight orders, so that the lanes write to all banks)
        *reinterpret_cast<uint4*>(rows + (i & 1) * Cross::HALF + (32 * w + lane) * 128 + (((i >> 1) + lane) & 7) * 16) =
            make_uint4(0, 0, 0, 0);
  }
  if ((vis.x & vis.y & vis.z & vis.w) != ~0u) {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
  }
}

// In place, by a converter warp: `rows` rows of 128 e4m3 codes from `raw` on (128 bytes
// each, in the slot's second half) become the f16 rows of both halves, swizzled.
// Eight lanes to a row, all of which have read before any writes.
__device__ __forceinline__ void convert_rows(uint8_t* raw, int rows, int lane) {
  const int seg = lane & 7, col = 2 * (seg & 3), second = seg >> 2;
  constexpr int kBatch = 2;  // (4: no faster, and more code)
#pragma unroll 1
  for (int r0 = 0; r0 < rows; r0 += 4 * kBatch) {
    uint4 x[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      x[i] = *reinterpret_cast<const uint4*>(raw + (r0 + 4 * i + (lane >> 3)) * 128 + seg * 16);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = r0 + 4 * i + (lane >> 3);
      const uint4 lo = make_uint4(e4m3x2_lo(x[i].x), e4m3x2_hi(x[i].x), e4m3x2_lo(x[i].y), e4m3x2_hi(x[i].y));
      const uint4 hi = make_uint4(e4m3x2_lo(x[i].z), e4m3x2_hi(x[i].z), e4m3x2_lo(x[i].w), e4m3x2_hi(x[i].w));
      uint8_t* row = raw + r * 128 - (second ? 0 : Cross::HALF);
      // (the two halves' rows share banks: their lanes write odd and even pieces in turn)
      *reinterpret_cast<uint4*>(row + (((col + second) ^ (r & 7)) << 4)) = second ? hi : lo;
      *reinterpret_cast<uint4*>(row + (((col + 1 - second) ^ (r & 7)) << 4)) = second ? lo : hi;
    }
  }
}

template <bool TREE, bool FP8>
__global__ void __launch_bounds__(CrossCta<TREE, FP8>::THREADS, 1)
    cross_attend_kernel(const __grid_constant__ CrossArgs a, const __grid_constant__ CUtensorMap tk,
                        const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tq,
                        const __grid_constant__ CUtensorMap to) {
  static_assert(TREE || !FP8, "e4m3 caches are served with TREE");
  using C = CrossCta<TREE, FP8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::OFF_BAR);
  auto& tail = *reinterpret_cast<Tail<C::WARPS>*>(bars + (FP8 ? B_COUNT_FP8 : B_COUNT));
  auto bar = [&](int i) { return smem_u32(bars + i); };
  // The slot of the n-th key block's K (v = 0) or V (v = 1), counted over all pieces: its
  // barriers, its turn's phase and its place.
  auto slot_of = [&](int v, int n) {
    return !FP8 ? (2 * n + v) % C::NST : v ? C::K_SLOTS + n % C::V_SLOTS : n % C::K_SLOTS;
  };
  auto turn_of = [&](int v, int n) { return !FP8 ? (2 * n + v) / C::NST : n / (v ? C::V_SLOTS : C::K_SLOTS); };
  auto full = [&](int v, int n) { return bar((FP8 ? B_FULL_FP8 : B_FULL) + slot_of(v, n)); };
  auto empty = [&](int v, int n) { return bar((FP8 ? B_EMPTY_FP8 : B_EMPTY) + slot_of(v, n)); };
  auto slot_at = [&](int v, int n) {
    return C::OFF_RING + (!FP8 ? slot_of(v, n) * C::TILE : v ? C::K_SLOTS * C::HALF + n % C::V_SLOTS * C::TILE
                                                             : slot_of(0, n) * C::HALF);
  };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < (FP8 ? C::SLOTS : C::NST); ++s) {
      mbar_init(bar((FP8 ? B_FULL_FP8 : B_FULL) + s), FP8 ? 1 : 2);  // (e4m3: one producer's; else a half by each)
      mbar_init(bar((FP8 ? B_EMPTY_FP8 : B_EMPTY) + s), 1);
    }
    for (int s = 0; FP8 && s < C::V_SLOTS; ++s) mbar_init(bar(B_CONV + s), 4);
    if (FP8) mbar_init(bar(B_DOWN), 128);
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(B_Q + t), !FP8 && a.row_boxes ? 4 : 128);
      mbar_init(bar(B_S + t), 1);
      mbar_init(bar(B_P + t), 128);
      mbar_init(bar(B_O + t), 1);
    }
    mbar_init(bar(B_ML), 128);
    mbar_init(bar(B_JOINED), 128);
    mbar_init(bar(B_DONE), 1);
    fence_mbar_init();
  }
  if (warp == C::PRODUCER) {
    tmem_alloc(smem_u32(&tail.tmem), C::TMEM_COLS);
    if (lane == 0) {
      prefetch_tmap(&tk);
      prefetch_tmap(&tv);
      if (a.row_boxes) {
        prefetch_tmap(&tq);
        prefetch_tmap(&to);
      }
    }
  }
  launch_dependents();
  wait_prerequisites();
  if (warp == C::ISSUER) {
    plan_pieces<TREE>(a, lane, tail);
  } else {  // (meanwhile: where the pages' ids begin)
    for (int b = threadIdx.x; b < a.batch; b += C::SOFTMAX_WARPS * 32)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(a.block_table + size_t(b) * a.max_pages));
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&tail.tmem);
  const int pieces = *reinterpret_cast<volatile int32_t*>(&tail.pieces);
  int n_taken = 0;  // by this warp
  auto take = [&]() -> const Piece* {
    if (pieces >= 0) return n_taken < pieces ? &tail.piece[n_taken++] : nullptr;
    return next_piece<TREE>(a, tail, warp, lane) ? &tail.now[warp] : nullptr;
  };

  if (warp == C::PRODUCER || warp == C::PRODUCER + 1) {
    // ------------------------------------------------------------- producers
    // Of all pieces, key block j's K is ring item 2 j, its V item 2 j + 1; item
    // i lies in slot i % NST.  Each of the two warps copies a 64-column half of
    // every item (a warp issues a box in some 100 cycles: one alone would take
    // 1,600 for a block in pages of 16 keys).  A block is BK / br groups of br
    // keys of one page each; lane g holds the page of group g.  Groups behind the
    // last key are not read.
    const int half = warp - C::PRODUCER;
    const int br = a.box_rows;
    // (e4m3: one warp copies the whole rows of K, the other those of V, into the second
    // half of the slot.)
    bool ok = true;
    int n = 0;       // key blocks so far
    int issued = 0;  // what this warp asked for: K, V, K, ..., or (e4m3) the blocks of one of them
    const Piece* taken;
    while (ok && (taken = take()) != nullptr) {
      const Piece pc = *taken;
      const int32_t* trow = a.block_table + size_t(pc.b) * a.max_pages;
      int next_ph = 0, next_in = 0;  // of the block after this one, asked for a block ahead
      auto look_up = [&](int j) {
        const int key = (pc.j0 + j) * C::BK + lane * br, lp = key / a.P;
        next_in = key - lp * a.P;
        next_ph = lane < C::BK / br && key < pc.L ? trow[lp] : 0;
      };
      if (pc.nblk > 0) look_up(0);
      for (int j = 0; j < pc.nblk && ok; ++j, ++n) {
        const int np = (min(C::BK, pc.L - (pc.j0 + j) * C::BK) + br - 1) / br;
        int ph = next_ph;
        const int in = next_in;
        if (ph < 0 || ph >= a.num_pages) {
          if (a.status) atomicOr(a.status, SPLITKV_DEVERR_PAGE);
          ph = 0;
        }
        if (j + 1 < pc.nblk) look_up(j + 1);
#pragma unroll 1
        for (int v = FP8 ? half : 0; v < (FP8 ? half + 1 : 2); ++v) {
          if (turn_of(v, n) > 0) ok = __all_sync(kFull, wait_for(empty(v, n), (turn_of(v, n) - 1) & 1));
          if (!ok) break;
          mbar_arrive_expect_tx_warp(full(v, n), uint32_t(np * br * 128));
          const uint32_t dst = smem_u32(sm + slot_at(v, n)) + (FP8 ? v : half) * C::HALF;
          const CUtensorMap* tm = v ? &tv : &tk;
          for (int g = 0; g < np; ++g) {
            const int pg = __shfl_sync(kFull, ph, g), kp = __shfl_sync(kFull, in, g);
            tma_load_5d_warp(dst + g * br * 128, tm, full(v, n), 0, kp, FP8 ? 0 : half, pc.h, pg);
          }
          ++issued;
        }
      }
    }
    if (!ok && lane == 0 && a.status) atomicOr(a.status, SPLITKV_DEVERR_TIMEOUT);
    // Stay until every copy has landed: the last of each slot.
    if (lane == 0)
      for (int i = issued - 1; i >= 0 && i >= issued - (!FP8 ? C::NST : half ? C::V_SLOTS : C::K_SLOTS); --i) {
        const int v = FP8 ? half : i & 1;
        wait_for(full(v, FP8 ? i : i >> 1), turn_of(v, FP8 ? i : i >> 1) & 1);
      }
  } else if (warp == C::ISSUER) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t idesc_qk = FP8 ? umma_idesc_e4m3(128, 128) : umma_idesc_bf16(128, 128, 0, 0),
                       idesc_pv = FP8 ? umma_idesc_f16(128, 128, 0, 1) : umma_idesc_bf16(128, 128, 0, 1);
    // one CTA reports lengths that the cache cannot hold
    if (a.status && blockIdx.x == 0 && blockIdx.y == 0)
      for (int i = lane; i < a.batch; i += 32) {
        int first;
        if (a.seq_lens[i] != keys_of<TREE>(a, i, TREE ? tokens_of(a, i, &first) : 0)) atomicOr(a.status, SPLITKV_DEVERR_SEQLEN);
      }
    bool ok = true;
    int n = 0;                  // key blocks of the pieces before
    uint32_t n_q = 0, n_p = 0;  // phases of B_Q and B_P so far, a bit per row block
    auto wait = [&](int i, int phase) {
      ok = ok && __all_sync(kFull, wait_for(bar(i), phase & 1));
      return ok;
    };
    auto landed = [&](int v, int n) {
      ok = ok && __all_sync(kFull, wait_for(full(v, n), turn_of(v, n) & 1));
      return ok;
    };
    auto v_in_smem = [&](int n) { return FP8 ? wait(B_CONV + n % C::V_SLOTS, turn_of(1, n)) : landed(1, n); };
    static_assert(C::HALF >> 4 == 1024, "descriptor steps of mma_qk");
    auto qk = [&](int t, int q, int n) {  // S_t = Q_q . K^T
      mma_qk<FP8>(tmem + C::S_COL + 128 * t, umma_desc(smem_u32(sm + q * C::TILE), 16, 1024, 2),
                  umma_desc(smem_u32(sm + slot_at(0, n)), 16, 1024, 2), idesc_qk);
      umma_commit_warp(bar(B_S + t));
    };
    auto pv = [&](int t, int n, bool more) {  // O_t (+)= P_t . V
      mma_pv(tmem + C::O_COL + 128 * t, tmem + C::S_COL + 128 * t, umma_desc(smem_u32(sm + slot_at(1, n)), C::HALF, 1024, 2),
             idesc_pv, more);
    };
    auto release = [&](int v, int n) { umma_commit_warp(empty(v, n)); };
    // V of key block j of a piece has landed; key slots past the last key may
    // hold anything (even NaN): their V rows are zeroed, so that 0 * V stays 0.
    // So are those of drafted keys that no token of the tile sees.
    int drafts = 0;   // tokens of the piece's sequence
    int seen_j = -1;  // the block that `vis` is of: those of its keys that some token of the tile sees
    uint4 vis;
    auto look = [&](const Piece& pc, int j) {
      const int valid = pc.L - (pc.j0 + j) * C::BK;
      vis = seen_by(a.mask + int64_t(pc.first) * a.words, a.words, pc.row0 / a.G,
                    (pc.row0 + min(pc.n_rows, C::ROWS) - 1) / a.G, valid - drafts, valid, lane);
      seen_j = j;
    };
    auto v_ready = [&](const Piece& pc, int j, int n) {
      const int valid = pc.L - (pc.j0 + j) * C::BK;
      if constexpr (TREE) {
        const bool masked = valid - drafts < C::BK;
        if (masked && seen_j != j) look(pc, j);
        if (!v_in_smem(n)) return false;
        if (masked) zero_unseen(sm + slot_at(1, n), vis, lane);
        return true;
      }
      if (!v_in_smem(n)) return false;
      if (valid < C::BK) {
        uint8_t* v = sm + slot_at(1, n);
        for (int x = lane; x < (C::BK - valid) * 16; x += 32)
          *reinterpret_cast<uint4*>(v + (x & 1) * C::HALF + (valid + (x >> 4)) * 128 + ((x >> 1) & 7) * 16) =
              make_uint4(0, 0, 0, 0);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
      }
      return true;
    };
    const Piece* taken;
    while (ok && (taken = take()) != nullptr) {
      const Piece pc = *taken;
      if (pc.nblk == 0) continue;
      if (TREE) {
        drafts = (pc.row0 + pc.n_rows) / a.G;
        // (the first block with drafted keys, while queries and keys are on their way)
        const int before = pc.L - drafts - pc.j0 * C::BK, j = before > 0 ? before / C::BK : 0;
        seen_j = -1;
        if (j < pc.nblk) look(pc, j);
      }
      if (pc.n_rows <= 128) {
        // narrow: A takes the even key blocks, B the odd ones, of the same rows
        const bool q_in = wait(B_Q, n_q);
        n_q ^= 1u;
#pragma unroll 1
        for (int j = 0; j < min(2, pc.nblk) && q_in; ++j) {
          if (!landed(0, n + j)) break;
          tc_fence_after();
          qk(j, 0, n + j);
          release(0, n + j);
        }
        for (int j = 0; j < pc.nblk && ok; ++j) {
          const int t = j & 1;
          if (!v_ready(pc, j, n + j) || !wait(B_P + t, n_p >> t)) break;
          n_p ^= 1u << t;
          tc_fence_after();
          pv(t, n + j, j > 1);
          if (j + 2 < pc.nblk) {
            release(1, n + j);  // (K of the next block but one is waited for in the slot that V before this one left)
            if (!landed(0, n + j + 2)) break;
            tc_fence_after();
            qk(t, 0, n + j + 2);
            release(0, n + j + 2);
          } else {
            umma_commit_warp(bar(B_O + t));
            release(1, n + j);
          }
        }
        n += pc.nblk;
        continue;
      }
#pragma unroll 1
      for (int t = 0; t < 2 && ok; ++t) {
        const bool q_in = wait(B_Q + t, n_q >> t);
        n_q ^= 1u << t;
        if (!q_in || (t == 0 && !landed(0, n))) break;
        tc_fence_after();
        qk(t, t, n);
        if (t == 1) release(0, n);
      }
      for (int j = 0; j < pc.nblk && ok; ++j) {
        const int next = n + j + 1;
        bool k_in = true;
        for (int t = 0; t < 2 && ok; ++t) {
          if (t == 0) {
            // (off the way from P to the next product, if K has landed by now)
            if (j + 1 < pc.nblk)
              k_in = __all_sync(kFull, mbar_test(full(0, next), turn_of(0, next) & 1));
            if (!v_ready(pc, j, n + j)) break;
          }
          if (!wait(B_P + t, n_p >> t)) break;
          n_p ^= 1u << t;
          tc_fence_after();
          pv(t, n + j, j > 0);
          if (j + 1 < pc.nblk) {
            if (!k_in) {
              if (!landed(0, next)) break;
              tc_fence_after();
              k_in = true;
            }
            qk(t, t, next);
          } else {
            umma_commit_warp(bar(B_O + t));
          }
          // (behind the products, which are not to wait for it)
          if (t == 1) {
            release(1, n + j);
            if (j + 1 < pc.nblk) release(0, next);
          }
        }
      }
      n += pc.nblk;
    }
    if (!ok && lane == 0 && a.status) atomicOr(a.status, SPLITKV_DEVERR_TIMEOUT);
    // every MMA issued above completes before TMEM is released
    umma_commit_warp(bar(B_DONE));
    __syncwarp();
    wait_for(bar(B_DONE), 0);
  } else if (FP8 && warp >= C::SOFTMAX_WARPS) {
    // ------------------------------------------------------------ converters
    // A warp turns 32 rows of every V (those that hold keys).
    bool ok = true;
    int n = 0;
    const int row0 = 32 * (warp - C::CONVERTER - (warp > C::IDLE));
    const Piece* taken;
    while (warp != C::IDLE && ok && (taken = take()) != nullptr) {
      const int nblk = taken->nblk;
      int left = taken->L - taken->j0 * C::BK - row0;
      for (int j = 0; j < nblk; ++j, ++n, left -= C::BK) {
        ok = __all_sync(kFull, wait_for(full(1, n), turn_of(1, n) & 1));
        if (!ok) break;
        convert_rows(sm + slot_at(1, n) + C::HALF + row0 * 128, min(32, left), lane);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_CONV + n % C::V_SLOTS));
      }
    }
    if (!ok && lane == 0 && a.status) atomicOr(a.status, SPLITKV_DEVERR_TIMEOUT);
  } else {
    // --------------------------------------------------------- softmax warps
    const int t = warp >> 2;                       // row block
    const int r = (warp & 3) * 32 + lane;          // TMEM lane
    // this warp's lanes and the columns of S and, + 256 - 128 t, of O
    const uint32_t scol = tmem + (uint32_t((warp & 3) * 32) << 16) + C::S_COL + 128 * t;
    const uint32_t ocol = scol + (C::O_COL - C::S_COL);
    float sl2 = a.qk_scale_log2;  // scores to log2 units, of this piece's row
    uint32_t n_down = 0;          // e4m3, B: phases of B_DOWN so far
    uint32_t n_s = 0, n_o = 0;  // phases of B_S and B_O so far
    bool ok = true;
    // 16-byte chunk `ch` of row `rr` of the row block's Q in shared memory.
    auto chunk_at = [&](int rr, int ch) -> uint8_t* {
      return sm + t * C::TILE + (ch >> 3) * C::HALF + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4);
    };
    // Visits this warp's 32 rows of a piece, 16 lanes to a row: body(row of the
    // row block, whether it exists, its token and head).  Rolled, but for four rows at
    // once, as is all that runs once for a piece: such code waits for its own instructions.
    auto each_row = [&](const Piece& q, auto&& body) {
      int rr = (warp & 3) * 32 + (lane >> 4);
      const int first = q.row0 + t * 128 + rr;  // (not called for B's share of a narrow piece)
      int tok = first / a.G, g = first - tok * a.G;
#pragma unroll 2
      for (int i = 0; i < 16; ++i, rr += 2) {
        body(rr, t * 128 + rr < q.n_rows, int64_t(q.first) + tok, q.h * a.G + g);
        for (g += 2; g >= a.G; g -= a.G) ++tok;
      }
    };
    // e4m3: 16-byte chunk `ch` of a row before it is a code.  A row's chunks 2 i and 2 i + 1
    // lie where its codes' chunk i of both tiles will.
    auto raw_at = [&](int rr, int ch) -> uint8_t* {
      return sm + t * C::TILE + (ch & 1) * C::HALF + rr * 128 + (((ch >> 1) ^ (rr & 7)) << 4);
    };
    // The row of this lane, in place, as the sum of two codes a column, times the power of
    // two that brings its largest into [2^7, 2^8).  Returns that power's inverse.  (Rolled: as
    // straight code for eight rows at once, 16 lanes to a row, it waited 11 us for itself.)
    auto encode_row = [&]() {
      uint32_t top = 0;
#pragma unroll 1
      for (int i = 0; i < 16; ++i) {
        const uint4 x = *reinterpret_cast<const uint4*>(raw_at(r, i));
        top = max_u16x2(max_u16x2(top, max_u16x2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu)),
                        max_u16x2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
      }
      top = max(top & 0xffffu, top >> 16);
      int k = 0;
      if (top > 0) k = min(126, max(-120, 7 - (int(top >> 7) - 127)));
      // (an infinity is no code: its row is NaN, as its softmax would be)
      const float up = top >= 0x7f80u ? NAN : __uint_as_float(uint32_t(127 + k) << 23);
#pragma unroll 1
      for (int i = 0; i < 8; ++i) {
        uint4* at[2] = {reinterpret_cast<uint4*>(raw_at(r, 2 * i)), reinterpret_cast<uint4*>(raw_at(r, 2 * i + 1))};
        uint32_t code[2][4];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint4 x = *at[c];
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float z[4] = {__uint_as_float(w[2 * e] << 16) * up, __uint_as_float(w[2 * e] & 0xffff0000u) * up,
                          __uint_as_float(w[2 * e + 1] << 16) * up, __uint_as_float(w[2 * e + 1] & 0xffff0000u) * up};
            float y[4];
#pragma unroll
            for (int f = 0; f < 4; ++f) {
              y[f] = __uint_as_float(__float_as_uint(z[f]) & 0xfff00000u);  // (four of its eight bits)
              z[f] -= y[f];
            }
            code[0][2 * c + e] = pack_e4m3x4(y);
            code[1][2 * c + e] = pack_e4m3x4(z);
          }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) *at[c] = make_uint4(code[c][0], code[c][1], code[c][2], code[c][3]);
      }
      return uint32_t(127 - k);
    };
    // The next piece with rows of this row block: its query rows, swizzled, on
    // their way into shared memory (rows behind the last are zero).  Not before
    // the products that read the Q before are done.
    const Piece* next = nullptr;
    int n_q_boxes = 0;  // pieces whose Q came by boxes
    auto take_piece = [&]() {
      bool skip;
      do {
        next = take();
        if (next == nullptr) return false;
        skip = t == 1 && next->n_rows <= 128 && next->nblk < 2;
      } while (skip);
      if (t == 1 && next->n_rows <= 128) return true;
      if (!FP8 && a.row_boxes && lane == 0)  // (queries, or zeros of an item without keys, go where whole results came from)
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
      if (next->nblk == 0) {
        __syncwarp();
        return true;
      }
      if (!FP8 && a.row_boxes) {
        // (rows of other sequences' tokens behind the last come along, and are not used)
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        const int token = next->first + (next->row0 + t * 128 + (warp & 3) * kRowBox) / a.G;
        const uint32_t dst = smem_u32(sm + t * C::TILE + (warp & 3) * kRowBox * 128);
        mbar_arrive_expect_tx_warp(bar(B_Q + t), 2 * kRowBox * 128);
        tma_load_4d_warp(dst, &tq, bar(B_Q + t), 0, 0, next->h * a.G, token);
        tma_load_4d_warp(dst + C::HALF, &tq, bar(B_Q + t), 0, 1, next->h * a.G, token);
        ++n_q_boxes;
      } else {
        each_row(*next, [&](int rr, bool in, int64_t token, int head) {
          const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) + (in ? token * a.q_stride + head * 128 : 0);
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(FP8 ? raw_at(rr, lane & 15) : chunk_at(rr, lane & 15))),
                       "l"(src + 8 * (lane & 15)), "r"(in ? 16 : 0)
                       : "memory");
        });
      }
      return true;
    };
    uint32_t n_ml = 0, n_ob = 0;  // phases of B_ML and, seen by A, of B's B_O
    bool joining = false;         // B: A has still to read its last narrow piece's O
    bool taken = false;  // (the next piece is)
    while (ok) {
      if (!taken && !take_piece()) break;
      taken = false;
      if (!ok) break;
      const Piece pc = *next;
      // A narrow piece (up to 128 rows) has its key blocks dealt to A and B in
      // turn, as if they were two row blocks, and A joins the two results: a
      // single row block's chain of products and softmaxes would be longer
      // than K and V take to arrive.
      const bool narrow = pc.n_rows <= 128, two = narrow && pc.nblk > 1;
      const int row = narrow ? r : t * 128 + r;  // of the tile
      const bool live = row < pc.n_rows;
      const bool any = __any_sync(kFull, live);  // a warp without rows only keeps step
      const bool whole = pc.slot < 0;
      // A whole result goes through this warp's rows of Q's shared memory, so
      // that whole rows are written; a partial one (whose layout puts a
      // column's rows side by side), and one of a few rows, straight from
      // registers, with the next piece's Q already on its way.
      const bool staged = whole && !narrow;
      if (pc.nblk > 0 && (t == 0 || !narrow) && (FP8 || !a.row_boxes)) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        if constexpr (FP8) {
          __syncwarp();
          const uint32_t down = any ? encode_row() : 127;
          if (two) tail.down[r] = uint8_t(down);  // (B has read those before: A has had its maxima since)
          sl2 = a.qk_scale_log2 * (a.k_scale ? a.k_scale[pc.h] : 1.f) * __uint_as_float(down << 23);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        mbar_arrive(bar(B_Q + t));
        if (FP8 && two) mbar_arrive(bar(B_DOWN));
      }
      if (FP8 && t == 1 && two) {
        ok = __all_sync(kFull, wait_for(bar(B_DOWN), n_down++ & 1));
        if (!ok) break;
        sl2 = a.qk_scale_log2 * (a.k_scale ? a.k_scale[pc.h] : 1.f) * __uint_as_float(uint32_t(tail.down[r]) << 23);
      }
      float m_ref = -INFINITY, l = 0.f;
      const int step = narrow ? 2 : 1;
      int valid = pc.L - (pc.j0 + (narrow ? t : 0)) * C::BK;  // keys from the block's first on
      const int drafts = TREE ? (pc.row0 + pc.n_rows) / a.G : 0;
      const uint32_t* mask =
          TREE ? a.mask + (int64_t(pc.first) + (pc.row0 + (live ? row : 0)) / a.G) * a.words : nullptr;
      for (int j = narrow ? t : 0; j < pc.nblk; j += step, valid -= step * C::BK) {
        const int d = valid - drafts;  // keys of the block before the drafted ones
        uint32_t vis[4];
        const bool masked = TREE ? d < C::BK : valid < C::BK;
        if (TREE && masked) {  // (while S is waited for)
          uint32_t m[5];
          mask_words(mask, a.words, d, m);
          visible(m, d, valid, vis);
        }
        // Part i of S, C::PART columns of it.
        auto read_part = [&](float (&s)[C::PART], int i) {
          if constexpr (C::PART == 128) {
            tmem_ld64(scol, s);
            tmem_ld64(scol + 64, s + 64);
          } else if constexpr (C::PART == 64) {
            tmem_ld64(scol + 64 * i, s);
          } else {
            tmem_ld32(scol + 32 * i, s);
          }
          if (!masked) return;
          if constexpr (TREE) {
            uint32_t w[C::PART / 32];
#pragma unroll
            for (int k = 0; k < C::PART / 32; ++k)
              w[k] = C::PART == 128 ? vis[k] : C::PART == 64 ? (i ? vis[2 + k % 2] : vis[k % 2]) : i < 2 ? (i ? vis[1] : vis[0]) : (i == 2 ? vis[2] : vis[3]);
#pragma unroll
            for (int k = 0; k < C::PART; ++k) s[k] = w[k >> 5] & (1u << (k & 31)) ? s[k] : -INFINITY;
          } else {
#pragma unroll
            for (int k = 0; k < C::PART; ++k) s[k] = C::PART * i + k < valid ? s[k] : -INFINITY;
          }
        };
        ok = __all_sync(kFull, wait_for(bar(B_S + t), n_s++ & 1));
        if (!ok) break;
        tc_fence_after();
        if (joining) {  // (B's O is written over by what its next P starts)
          joining = false;
          ok = __all_sync(kFull, wait_for(bar(B_JOINED), (n_ml - 1) & 1));
          if (!ok) break;
        }
        if (any) {
          // S in parts, the first last, which stays: the others are read once more below, when
          // P is written over those before
          float s[C::PART];
          float mx = -INFINITY;
#pragma unroll 1
          for (int h = 128 / C::PART - 1; h >= 0; --h) {
            read_part(s, h);
            float m4[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) m4[i] = fmaxf(s[i], s[4 + i]);
#pragma unroll
            for (int k = 8; k < C::PART; k += 8)
#pragma unroll
              for (int i = 0; i < 4; ++i) m4[i] = max3(m4[i], s[k + i], s[k + 4 + i]);
            mx = max3(mx, fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
          }
          mx *= sl2;  // (the scale is positive)
          float alpha = 1.f;
          bool rescale = false;
          if (mx > m_ref + C::RESCALE_LOG2 || (m_ref == -INFINITY && mx != -INFINITY)) {
            alpha = m_ref == -INFINITY ? 0.f : ex2(m_ref - mx);
            rescale = m_ref != -INFINITY;
            m_ref = mx;
            l *= alpha;
          }
          // (the PV before was issued before the product this S came from: O rests)
          if (__any_sync(kFull, rescale)) {
#pragma unroll 1
            for (int c0 = 0; c0 < 128; c0 += 16) {
              float o[16];
              tmem_ld16(ocol + c0, o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] *= alpha;
              tmem_st16(ocol + c0, o);
            }
          }
          const float nm = m_ref == -INFINITY ? 0.f : FP8 ? C::P_UP - m_ref : -m_ref;
          float l4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
          for (int h = 0; h < 128 / C::PART; ++h) {
            if (h > 0) read_part(s, h);
#pragma unroll
            for (int q = 0; q < C::PART / 16; ++q) {
              uint32_t pk[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                float x = s[16 * q + 2 * i], y = s[16 * q + 2 * i + 1];
                fma2(x, y, sl2, nm);
                x = ex2(x);
                y = ex2(y);
                add2(l4[(2 * i) & 3], l4[(2 * i + 1) & 3], x, y);
                pk[i] = FP8 ? pack_f16(x, y) : pack_bf16(x, y);
              }
              tmem_st8(scol + C::PART / 2 * h + 8 * q, pk);
            }
          }
          l += (l4[0] + l4[1]) + (l4[2] + l4[3]);
          tmem_wait_st();
        }
        tc_fence_before();
        mbar_arrive(bar(B_P + t));
      }

      // ---- the piece's result (S of its last block has come: Q is read; in a
      // narrow piece B may still be at its own last block, which A waits for)
      if (!ok) break;
      if (two && t == 1) {
        // (m, l) into the last two columns of S_B, behind P_B: they are S's again
        // only when the next product is issued, after A's next Q
        tmem_st2(scol + 126, m_ref, l);
        tc_fence_before();
        mbar_arrive(bar(B_ML));
        ++n_ml;
        ++n_o;
        joining = true;
        continue;
      }
      float2 other = make_float2(0.f, 0.f);
      if (two) {
        ok = __all_sync(kFull, wait_for(bar(B_ML), n_ml++ & 1));
        tc_fence_after();
        if (ok) tmem_ld2(scol + 128 + 126, other.x, other.y);  // (before the next queries, with which S_B is written)
        tc_fence_before();
        if (ok) ok = __all_sync(kFull, wait_for(bar(B_O + 1), n_ob & 1));
      }
      n_ob += two || (!narrow && pc.nblk > 0);
      bool more = true;
      if (ok && !staged) taken = more = take_piece();
      if (ok && pc.nblk > 0) ok = __all_sync(kFull, wait_for(bar(B_O + t), n_o++ & 1));
      if (!ok) break;
      tc_fence_after();
      // weights of A's own result and of B's
      float wa = 1.f, wb = 0.f;
      if (two) {
        const float m = fmaxf(m_ref, other.x);
        wa = m_ref == -INFINITY ? 0.f : ex2(m_ref - m);
        wb = other.x == -INFINITY ? 0.f : ex2(other.x - m);
        l = l * wa + other.y * wb;
        m_ref = m;
      }
      if (any) {
        // (a row without keys has l = 0; a NaN or a score of +inf makes l NaN, and the row)
        const float inv = l == 0.f ? 0.f : (FP8 ? a.v_scale ? a.v_scale[pc.h] : a.o_scale : 1.f) / l;
        const float lse = l == 0.f ? -INFINITY : (m_ref + lg2(l * C::P_DOWN)) * kLn2;
        wa *= inv;
        wb *= inv;
        const size_t slot = pc.slot;
        const int tok = (pc.row0 + row) / a.G, g = (pc.row0 + row) - tok * a.G;
        const size_t out_row = (size_t(pc.first) + tok) * a.Hq + size_t(pc.h) * a.G + g;
#pragma unroll 1
        for (int c0 = 0; c0 < 128; c0 += 32) {
          float o[32];
          if (pc.nblk > 0) {
            tmem_ld32(ocol + c0, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= wa;
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0.f;
          }
          if (two) {
            float ob[32];
            tmem_ld32(ocol + 128 + c0, ob);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = fmaf(ob[i], wb, o[i]);
          }
          if (whole) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint4 x = make_uint4(pack_bf16(o[8 * i], o[8 * i + 1]), pack_bf16(o[8 * i + 2], o[8 * i + 3]),
                                         pack_bf16(o[8 * i + 4], o[8 * i + 5]), pack_bf16(o[8 * i + 6], o[8 * i + 7]));
              if (staged)
                *reinterpret_cast<uint4*>(chunk_at(r, c0 / 8 + i)) = x;
              else if (live)
                reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + out_row * 128 + c0)[i] = x;
            }
          } else if (live) {
            float4* dst = reinterpret_cast<float4*>(a.o_part) + (slot * 32 + c0 / 4) * a.part_rows + row;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              dst[size_t(i) * a.part_rows] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          }
        }
        if (staged && !FP8 && a.row_boxes && t * 128 + (warp & 3) * kRowBox + kRowBox <= pc.n_rows) {
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            const int token = pc.first + (pc.row0 + t * 128 + (warp & 3) * kRowBox) / a.G;
            for (int half = 0; half < 2; ++half)
              tma_store_4d(&to, smem_u32(sm + t * C::TILE + half * C::HALF + (warp & 3) * kRowBox * 128), 0, half, pc.h * a.G, token);
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
        } else if (staged) {
          __syncwarp();
          each_row(pc, [&](int rr, bool in, int64_t token, int head) {
            if (in)
              reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + (token * a.Hq + head) * 128)[lane & 15] =
                  *reinterpret_cast<const uint4*>(chunk_at(rr, lane & 15));
          });
          __syncwarp();
        }
        if (live) {
          if (!whole) a.lse_part[slot * a.part_rows + row] = lse;
          else if (a.lse) a.lse[out_row] = lse;
        }
      }
      if (two) {  // B's O and (m, l) are read
        tc_fence_before();
        mbar_arrive(bar(B_JOINED));
      }
      if (!more) break;
    }
    if (!FP8) {
      asm volatile("cp.async.wait_all;" ::: "memory");  // (after a wait that ran out)
      if (!ok && n_q_boxes > 0) wait_for(bar(B_Q + t), (n_q_boxes - 1) & 1);
      if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    if (!ok && lane == 0 && a.status) atomicOr(a.status, SPLITKV_DEVERR_TIMEOUT);
  }

  // ---- teardown: TMEM is freed by the warp that allocated it
  tc_fence_before();
  __syncthreads();
  if (warp == C::PRODUCER) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <bool TREE, bool FP8>
cudaError_t launch_cross_kernel(const CrossArgs& a, const CrossMaps& maps, void* stream) {
  using C = CrossCta<TREE, FP8>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_shared_memory(reinterpret_cast<const void*>(cross_attend_kernel<TREE, FP8>), C::SMEM, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute la[1];
  la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  la[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = a.parts ? dim3(unsigned(a.parts), 1, 1)
                        : dim3(unsigned(int64_t(a.n_tokens) * a.G / C::ROWS + a.batch), unsigned(a.Hkv), 1);
  cfg.blockDim = dim3(C::THREADS, 1, 1);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = la;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cross_attend_kernel<TREE, FP8>, a, *reinterpret_cast<const CUtensorMap*>(&maps.k),
                            *reinterpret_cast<const CUtensorMap*>(&maps.v), *reinterpret_cast<const CUtensorMap*>(&maps.q),
                            *reinterpret_cast<const CUtensorMap*>(&maps.out));
}

}  // namespace
}  // namespace splitkv
