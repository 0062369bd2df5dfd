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
// K and V blocks pass in that order through one ring of five 32 KB slots that
// two producer warps fill by TMA, each a 64-column half of every slot, one box
// per page piece, 128-byte swizzled; K is read K-major, V with its dims on N.
// TMEM columns: S_A [0, 128), S_B [128, 256), O_A [256, 384), O_B [384, 512).
//
// Many items: a CTA per item (prompts), or a line of all items' key blocks that the
// CTAs share (batches of few rows a sequence; cross_deal has the rule).  The bound
// of prompts is 4 * 128 * rows * L operations.  Two sequences of 4k tokens, 32 heads on 4, over 8k keys: 740 to
// 775 us, 1,380 to 1,445 TFLOP/s (floor 552 at 1,938), near the GPU's limit of
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
// heads: 27.7 us, floor 11.6), or the longest piece's chain of products and the
// 32-bit partial results (prompts of 37 to 900 tokens over 1 to 4.1k keys:
// 21.6 us, floor 2.9).
//
// The code that runs once in a piece is kept small: it waits for its own
// instructions, and the softmax's loop runs slower beside more of them (the
// epilogue's columns unrolled by two: 754 us for the prompts above, rolled
// 800; the rescaling of O unrolled as well: 810).
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
  static constexpr int TAIL = 1536;              // barriers, plan
  static constexpr int SMEM = 1024 + OFF_BAR + TAIL;
  static constexpr int SOFTMAX_WARPS = 8;
  // warps: two producers (a half of every K and V block each), the issuer of the MMAs
  static constexpr int PRODUCER = SOFTMAX_WARPS, ISSUER = SOFTMAX_WARPS + 2;
  static constexpr int THREADS = (SOFTMAX_WARPS + 3) * 32;
  static constexpr uint32_t TMEM_COLS = 512, S_COL = 0, O_COL = 256;  // + 128 per row block
  static constexpr float RESCALE_LOG2 = 8.f;
};
static_assert(Cross::SMEM <= 227 * 1024, "shared memory budget");

enum {
  B_Q = 0,                       // [2] Q of a row block in shared memory (128 threads)
  B_FULL = 2,                    // [NST]
  B_EMPTY = B_FULL + Cross::NST, // [NST]
  B_S = B_EMPTY + Cross::NST,    // [2] S of a row block complete
  B_P = B_S + 2,                 // [2] P of a row block in TMEM (128 threads)
  B_O = B_P + 2,                 // [2] the last PV of a row block complete
  B_ML = B_O + 2,                // narrow pieces: B's maxima and sums written (128 threads)
  B_JOINED,                      //   A has read them and B's O (128 threads)
  B_DONE,
  B_COUNT
};

constexpr float kLn2 = 0.6931471805599453f;

// The length of sequence b, or 0 where the device value is not one the cache
// can hold.
__device__ __forceinline__ int keys_of(const CrossArgs& a, int b) {
  const int L = a.seq_lens[b];
  return L >= 0 && L <= int64_t(a.max_pages) * a.P ? L : 0;
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

// Where a warp is in a line: the next key block, and the item that holds it (of
// sequence b, from block `off` on) with its sequence's numbers.
struct Walk {
  int64_t x;
  int b, item, off, first, rows, L, tiles, nb;
};

// Behind the barriers.
struct Tail {
  uint32_t tmem;   // written by the allocation
  int32_t pieces;  // in `piece`; -1: the line's blocks [lo, hi), `share` to a CTA
  int64_t lo, hi, share;
  Piece piece[kMaxPieces];
  Walk walk[Cross::THREADS / 32];
  Piece now[Cross::THREADS / 32];
};
static_assert(B_COUNT * 8 + sizeof(Tail) <= Cross::TAIL, "barriers, then the tail");

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
__device__ __forceinline__ Lane lane_of(const CrossArgs& a, int b) {
  Lane x = {0, 0, 0, 0, 1};
  if (b < a.batch) {
    x.L = keys_of(a, b);
    x.rows = tokens_of(a, b, &x.first) * a.G;
    x.tiles = (x.rows + Cross::ROWS - 1) / Cross::ROWS;
    x.nb = blocks_of(x.L);
  }
  return x;
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
__device__ __noinline__ void plan_line(const CrossArgs& a, int lane, int64_t all, Tail& tail) {
  const int64_t share = (all + a.parts - 1) / a.parts;
  const int64_t lo = min(all, int64_t(blockIdx.x) * share), hi = min(all, lo + share);
  Walk w = {lo, 0, 0, 0, 0, 0, 0, 0, 1};
  int64_t passed = 0, total;
  for (int b0 = 0; lo < hi && b0 < a.batch; b0 += 32) {
    const Lane s = lane_of(a, b0 + lane);
    const int64_t n = int64_t(s.tiles) * a.Hkv * s.nb;
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
      const int64_t in = lo - __shfl_sync(kFull, at, f);
      w.item = int(in / w.nb);
      w.off = int(in - int64_t(w.item) * w.nb);
      break;
    }
  }
  if (lane < Cross::THREADS / 32) tail.walk[lane] = w;
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
__device__ __forceinline__ void plan_one(const CrossArgs& a, int lane, Tail& tail) {
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
  const int rows = tokens_of(a, lo, &q.first) * a.G;
  const int64_t tile = p - number(lo);
  const bool some = tile >= 0 && tile * Cross::ROWS < rows;
  q.row0 = some ? int(tile) * Cross::ROWS : 0;
  q.n_rows = rows - q.row0;
  q.L = keys_of(a, lo);
  q.j0 = 0;
  q.nblk = q.L > 0 ? blocks_of(q.L) : 0;
  q.slot = -1;
  if (lane == 0) {
    tail.piece[0] = q;
    tail.pieces = some;
  }
}

// By warp `me`, in a line: its next piece, into tail.now[me]; false behind the last.
__device__ __noinline__ bool next_piece(const CrossArgs& a, Tail& tail, int me, int lane) {
  Walk& walk = tail.walk[me];
  __syncwarp();  // (the piece before has been read)
  Walk w = walk;
  if (w.x >= tail.hi) return false;
  const int len = int(min(int64_t(w.nb - w.off), tail.hi - w.x));
  Piece q;
  q.b = w.b;
  q.h = w.tiles > 1 ? w.item / w.tiles : w.item;
  q.first = w.first;
  q.row0 = (w.item - q.h * w.tiles) * Cross::ROWS;
  q.n_rows = w.rows - q.row0;
  q.L = w.L;
  q.j0 = w.off;
  q.nblk = w.L > 0 ? len : 0;
  q.slot = len < w.nb ? 2 * int(blockIdx.x) + (w.x > tail.lo) : -1;
  if (me == Cross::ISSUER && lane == 0 && len < w.nb && w.off == 0) {  // (the CTA's last piece: an item's first)
    const int last = int((w.x + w.nb - 1) / tail.share);               // CTA of the item's last block
    const CrossSplit r = {last - int(blockIdx.x) + 1, q.slot, 2, q.first, q.h, q.row0, min(q.n_rows, Cross::ROWS)};
    a.split[blockIdx.x] = r;
  }
  w.x += len;
  w.off += len;
  if (w.off == w.nb && w.x < tail.hi) {
    w.off = 0;
    if (++w.item == w.tiles * a.Hkv) {  // the next sequence with tokens
      w.item = 0;
      Lane s;
      do s = lane_of(a, ++w.b); while (s.tiles == 0 && w.b < a.batch);
      w.first = s.first;
      w.rows = s.rows;
      w.L = s.L;
      w.tiles = s.tiles;
      w.nb = s.nb;
    }
  }
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
// the last round of CTAs, a line may cost less still.  (What that
// chooses for 16 heads: two key blocks stay whole, 12.5 us with one token and
// 12.7 cut; four are cut, 13.1 and 14.8 whole, and with 256 tokens 17.3 and 20.2.)
__device__ __forceinline__ void plan_pieces(const CrossArgs& a, int lane, Tail& tail) {
  if (a.parts == 0) {
    plan_one(a, lane, tail);
    return;
  }
  Lane mine;
  auto read = [&](int b0) { mine = lane_of(a, b0 + lane); };
  int items = 0, longest = 1, shortest = INT32_MAX, widest = 0;
  int64_t all = 0;  // key blocks
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    read(b0);
    const int64_t blocks = int64_t(mine.tiles) * a.Hkv * mine.nb;
    if (a.line) {
      int64_t sum;
      lanes_before(blocks, lane, &sum);
      all += sum;
      continue;
    }
    all += __reduce_add_sync(kFull, int(min(int64_t(1) << 25, blocks)));  // (items are few: more need not be exact)
    items += __reduce_add_sync(kFull, mine.tiles);
    longest = max(longest, __reduce_max_sync(kFull, mine.tiles > 0 ? mine.nb : 1));
    shortest = min(shortest, __reduce_min_sync(kFull, mine.tiles > 0 ? mine.nb : INT32_MAX));
    widest = max(widest, __reduce_max_sync(kFull, mine.rows));
  }
  if (a.line) {
    plan_line(a, lane, all, tail);
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
  const int64_t share = (all + a.parts - 1) / a.parts;
  if (widest <= 128 && all >= a.parts && all < (1 << 25) && share <= 2 * int64_t(shortest) &&
      share + kLineCost < __shfl_sync(kFull, cost, best)) {
    plan_line(a, lane, all, tail);
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

// NaN if either is.
__device__ __forceinline__ float max_nan(float x, float y) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(x), "f"(y));
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
// elected once, issues all of them (between two MMAs nothing but the next
// descriptors' additions, in units of 16 bytes).
// S = Q . K^T: both operands are two 64-column halves, 32 bytes per step.
__device__ __forceinline__ void mma_qk(uint32_t d, uint64_t a_desc, uint64_t b_desc, uint32_t idesc) {
  asm volatile(
      "{\n\t"
      ".reg .pred e, q, y;\n\t"
      ".reg .b64 a, b;\n\t"
      "setp.ne.b32 q, %4, 0;\n\t"
      "setp.eq.b32 y, 0, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, q;\n\t"
      "add.s64 a, %1, 2;\n\t"
      "add.s64 b, %2, 2;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, y;\n\t"
      "add.s64 a, %1, 4;\n\t"
      "add.s64 b, %2, 4;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, y;\n\t"
      "add.s64 a, %1, 6;\n\t"
      "add.s64 b, %2, 6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, y;\n\t"
      "add.s64 a, %1, 1024;\n\t"
      "add.s64 b, %2, 1024;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, y;\n\t"
      "add.s64 a, %1, 1026;\n\t"
      "add.s64 b, %2, 1026;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, y;\n\t"
      "add.s64 a, %1, 1028;\n\t"
      "add.s64 b, %2, 1028;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, y;\n\t"
      "add.s64 a, %1, 1030;\n\t"
      "add.s64 b, %2, 1030;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, y;\n\t"
      "}" ::"r"(d),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(0)
      : "memory");
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
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, q;\n\t"
      "add.s32 a, %1, 8;\n\t"
      "add.s64 b, %2, 128;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, y;\n\t"
      "add.s32 a, %1, 16;\n\t"
      "add.s64 b, %2, 256;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, y;\n\t"
      "add.s32 a, %1, 24;\n\t"
      "add.s64 b, %2, 384;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, y;\n\t"
      "add.s32 a, %1, 32;\n\t"
      "add.s64 b, %2, 512;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, y;\n\t"
      "add.s32 a, %1, 40;\n\t"
      "add.s64 b, %2, 640;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, y;\n\t"
      "add.s32 a, %1, 48;\n\t"
      "add.s64 b, %2, 768;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, y;\n\t"
      "add.s32 a, %1, 56;\n\t"
      "add.s64 b, %2, 896;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, y;\n\t"
      "}" ::"r"(d),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(more)
      : "memory");
}

__global__ void __launch_bounds__(Cross::THREADS, 1)
    cross_attend_kernel(const __grid_constant__ CrossArgs a, const __grid_constant__ CUtensorMap tk,
                        const __grid_constant__ CUtensorMap tv) {
  using C = Cross;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::OFF_BAR);
  Tail& tail = *reinterpret_cast<Tail*>(bars + B_COUNT);
  auto bar = [&](int i) { return smem_u32(bars + i); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NST; ++s) {
      mbar_init(bar(B_FULL + s), 2);  // (a half by each producer)
      mbar_init(bar(B_EMPTY + s), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(B_Q + t), 128);
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
    }
  }
  launch_dependents();
  wait_prerequisites();
  if (warp == C::ISSUER) {
    plan_pieces(a, lane, tail);
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
    return next_piece(a, tail, warp, lane) ? &tail.now[warp] : nullptr;
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
    bool ok = true;
    int item = 0;
    const Piece* taken;
    while (ok && (taken = take()) != nullptr) {
      const Piece pc = *taken;
      const int32_t* trow = a.block_table + size_t(pc.b) * a.max_pages;
      for (int j = 0; j < pc.nblk && ok; ++j) {
        const int key0 = (pc.j0 + j) * C::BK;
        const int np = (min(C::BK, pc.L - key0) + br - 1) / br;
        int ph = 0, in = 0;
        if (lane < np) {
          const int key = key0 + lane * br, lp = key / a.P;
          in = key - lp * a.P;
          ph = trow[lp];
          if (ph < 0 || ph >= a.num_pages) {
            if (a.status) atomicOr(a.status, SPLITKV_DEVERR_PAGE);
            ph = 0;
          }
        }
#pragma unroll 1
        for (int v = 0; v < 2; ++v, ++item) {
          const int st = item % C::NST;
          if (item >= C::NST) ok = __all_sync(kFull, mbar_wait(bar(B_EMPTY + st), (item / C::NST - 1) & 1));
          if (!ok) break;
          mbar_arrive_expect_tx_warp(bar(B_FULL + st), uint32_t(np * br * 128));
          const uint32_t dst = smem_u32(sm + C::OFF_RING + st * C::TILE) + half * C::HALF;
          const CUtensorMap* tm = v ? &tv : &tk;
          for (int g = 0; g < np; ++g) {
            const int pg = __shfl_sync(kFull, ph, g), kp = __shfl_sync(kFull, in, g);
            tma_load_5d_warp(dst + g * br * 128, tm, bar(B_FULL + st), 0, kp, half, pc.h, pg);
          }
        }
      }
    }
    if (!ok && lane == 0 && a.status) atomicOr(a.status, SPLITKV_DEVERR_TIMEOUT);
    // Stay until every copy has landed: the last item of each slot.
    if (lane == 0)
      for (int i = item - 1; i >= 0 && i >= item - C::NST; --i)  // (item: the first that was not issued)
        mbar_wait(bar(B_FULL + i % C::NST), (i / C::NST) & 1);
  } else if (warp == C::ISSUER) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t idesc_qk = umma_idesc_bf16(128, 128, 0, 0), idesc_pv = umma_idesc_bf16(128, 128, 0, 1);
    // one CTA reports lengths that the cache cannot hold
    if (a.status && blockIdx.x == 0 && blockIdx.y == 0)
      for (int i = lane; i < a.batch; i += 32)
        if (a.seq_lens[i] != keys_of(a, i)) atomicOr(a.status, SPLITKV_DEVERR_SEQLEN);
    bool ok = true;
    int item = 0;                      // ring items consumed
    uint32_t n_q = 0, n_p = 0;  // phases of B_Q and B_P so far, a bit per row block
    auto wait = [&](int i, int phase) {
      ok = ok && __all_sync(kFull, mbar_wait(bar(i), phase & 1));
      return ok;
    };
    auto slot = [&](int i) { return smem_u32(sm + C::OFF_RING + (i % C::NST) * C::TILE); };
    static_assert(C::HALF >> 4 == 1024, "descriptor steps of mma_qk");
    auto qk = [&](int t, int q, int i) {  // S_t = Q_q . K^T, K in ring item i
      mma_qk(tmem + C::S_COL + 128 * t, umma_desc(smem_u32(sm + q * C::TILE), 16, 1024, 2), umma_desc(slot(i), 16, 1024, 2),
             idesc_qk);
      umma_commit_warp(bar(B_S + t));
    };
    auto pv = [&](int t, int i, bool more) {  // O_t (+)= P_t . V, V in ring item i
      mma_pv(tmem + C::O_COL + 128 * t, tmem + C::S_COL + 128 * t, umma_desc(slot(i), C::HALF, 1024, 2), idesc_pv, more);
    };
    auto release = [&](int i) {
      umma_commit_warp(bar(B_EMPTY + i % C::NST));
    };
    // V of key block j of a piece has landed; key slots past the last key may
    // hold anything (even NaN): their V rows are zeroed, so that 0 * V stays 0.
    auto v_ready = [&](const Piece& pc, int j, int iv) {
      if (!wait(B_FULL + iv % C::NST, iv / C::NST)) return false;
      const int valid = pc.L - (pc.j0 + j) * C::BK;
      if (valid < C::BK) {
        uint8_t* v = sm + C::OFF_RING + (iv % C::NST) * C::TILE;
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
      if (pc.n_rows <= 128) {
        // narrow: A takes the even key blocks, B the odd ones, of the same rows
        const bool q_in = wait(B_Q, n_q);
        n_q ^= 1u;
        for (int j = 0; j < min(2, pc.nblk) && q_in; ++j) {
          if (!wait(B_FULL + (item + 2 * j) % C::NST, (item + 2 * j) / C::NST)) break;
          tc_fence_after();
          qk(j, 0, item + 2 * j);
          release(item + 2 * j);
        }
        for (int j = 0; j < pc.nblk && ok; ++j) {
          const int t = j & 1, iv = item + 2 * j + 1, ik = item + 2 * j + 4;  // V of this block, K of the next but one
          if (!v_ready(pc, j, iv) || !wait(B_P + t, n_p >> t)) break;
          n_p ^= 1u << t;
          tc_fence_after();
          pv(t, iv, j > 1);
          if (j + 2 < pc.nblk) {
            if (!wait(B_FULL + ik % C::NST, ik / C::NST)) break;
            tc_fence_after();
            qk(t, 0, ik);
            release(iv);
            release(ik);
          } else {
            umma_commit_warp(bar(B_O + t));
            release(iv);
          }
        }
        item += 2 * pc.nblk;
        continue;
      }
      for (int t = 0; t < 2 && ok; ++t) {
        const bool q_in = wait(B_Q + t, n_q >> t);
        n_q ^= 1u << t;
        if (!q_in || (t == 0 && !wait(B_FULL + item % C::NST, item / C::NST))) break;
        tc_fence_after();
        qk(t, t, item);
        if (t == 1) release(item);
      }
      for (int j = 0; j < pc.nblk && ok; ++j) {
        const int iv = item + 2 * j + 1, ik = iv + 1;  // V of this block, K of the next
        bool k_in = true;
        for (int t = 0; t < 2 && ok; ++t) {
          if (t == 0) {
            // (off the way from P to the next product, if K has landed by now)
            if (j + 1 < pc.nblk)
              k_in = __all_sync(kFull, mbar_test(bar(B_FULL + ik % C::NST), (ik / C::NST) & 1));
            if (!v_ready(pc, j, iv)) break;
          }
          if (!wait(B_P + t, n_p >> t)) break;
          n_p ^= 1u << t;
          tc_fence_after();
          pv(t, iv, j > 0);
          if (j + 1 < pc.nblk) {
            if (!k_in) {
              if (!wait(B_FULL + ik % C::NST, ik / C::NST)) break;
              tc_fence_after();
              k_in = true;
            }
            qk(t, t, ik);
          } else {
            umma_commit_warp(bar(B_O + t));
          }
          // (behind the products, which are not to wait for it)
          if (t == 1) {
            release(iv);
            if (j + 1 < pc.nblk) release(ik);
          }
        }
      }
      item += 2 * pc.nblk;
    }
    if (!ok && lane == 0 && a.status) atomicOr(a.status, SPLITKV_DEVERR_TIMEOUT);
    // every MMA issued above completes before TMEM is released
    umma_commit_warp(bar(B_DONE));
    __syncwarp();
    mbar_wait(bar(B_DONE), 0);
  } else {
    // --------------------------------------------------------- softmax warps
    const int t = warp >> 2;                       // row block
    const int r = (warp & 3) * 32 + lane;          // TMEM lane
    // this warp's lanes and the columns of S and, + 256 - 128 t, of O
    const uint32_t scol = tmem + (uint32_t((warp & 3) * 32) << 16) + C::S_COL + 128 * t;
    const uint32_t ocol = scol + (C::O_COL - C::S_COL);
    const float sl2 = a.qk_scale_log2;
    uint32_t n_s = 0, n_o = 0;  // phases of B_S and B_O so far
    bool ok = true;
    // 16-byte chunk `ch` of row `rr` of the row block's Q in shared memory.
    auto chunk_at = [&](int rr, int ch) -> uint8_t* {
      return sm + t * C::TILE + (ch >> 3) * C::HALF + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4);
    };
    // Visits this warp's 32 rows of a piece, 16 lanes to a row: body(row of the
    // row block, whether it exists, its token and head).  Rolled, as is all
    // that runs once for a piece: such code waits for its own instructions.
    auto each_row = [&](const Piece& q, auto&& body) {
      int rr = (warp & 3) * 32 + (lane >> 4);
      const int first = q.row0 + t * 128 + rr;  // (not called for B's share of a narrow piece)
      int tok = first / a.G, g = first - tok * a.G;
#pragma unroll 1
      for (int i = 0; i < 16; ++i, rr += 2) {
        body(rr, t * 128 + rr < q.n_rows, int64_t(q.first) + tok, q.h * a.G + g);
        for (g += 2; g >= a.G; g -= a.G) ++tok;
      }
    };
    // The next piece with rows of this row block: its query rows, swizzled, on
    // their way into shared memory (rows behind the last are zero).  Not before
    // the products that read the Q before are done.
    const Piece* next = nullptr;
    auto take_piece = [&]() {
      do {
        next = take();
        if (next == nullptr) return false;
      } while (t == 1 && next->n_rows <= 128 && next->nblk < 2);
      if (next->nblk > 0 && (t == 0 || next->n_rows > 128))
        each_row(*next, [&](int rr, bool in, int64_t token, int head) {
          const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) + (in ? token * a.q_stride + head * 128 : 0);
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(chunk_at(rr, lane & 15))),
                       "l"(src + 8 * (lane & 15)), "r"(in ? 16 : 0)
                       : "memory");
        });
      return true;
    };
    uint32_t n_ml = 0, n_ob = 0;  // phases of B_ML and, seen by A, of B's B_O
    bool joining = false;         // B: A has still to read its last narrow piece's O
    bool more = take_piece();
    while (ok && more) {
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
      if (pc.nblk > 0 && (t == 0 || !narrow)) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        mbar_arrive(bar(B_Q + t));
      }
      float m_ref = -INFINITY, l = 0.f;
      const int step = narrow ? 2 : 1;
      int valid = pc.L - (pc.j0 + (narrow ? t : 0)) * C::BK;  // keys from the block's first on
      for (int j = narrow ? t : 0; j < pc.nblk; j += step, valid -= step * C::BK) {
        ok = __all_sync(kFull, mbar_wait(bar(B_S + t), n_s++ & 1));
        if (!ok) break;
        tc_fence_after();
        if (joining) {  // (B's O is written over by what its next P starts)
          joining = false;
          ok = __all_sync(kFull, mbar_wait(bar(B_JOINED), (n_ml - 1) & 1));
          if (!ok) break;
        }
        if (any) {
          float s[128];
          tmem_ld64(scol, s);
          tmem_ld64(scol + 64, s + 64);
          if (valid < C::BK) {
#pragma unroll
            for (int k = 0; k < 128; ++k) s[k] = k < valid ? s[k] : -INFINITY;
          }
          // row maximum on the raw scores (the scale is positive)
          float m4[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) m4[i] = fmaxf(s[i], s[4 + i]);
#pragma unroll
          for (int k = 8; k < 128; k += 8)
#pragma unroll
            for (int i = 0; i < 4; ++i) m4[i] = max3(m4[i], s[k + i], s[k + 4 + i]);
          const float mx = fmaxf(max3(m4[0], m4[1], m4[2]), m4[3]) * sl2;
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
          const float nm = m_ref == -INFINITY ? 0.f : -m_ref;
          float l4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            uint32_t pk[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float x = s[16 * q + 2 * i], y = s[16 * q + 2 * i + 1];
              fma2(x, y, sl2, nm);
              x = ex2(x);
              y = ex2(y);
              add2(l4[(2 * i) & 3], l4[(2 * i + 1) & 3], x, y);
              pk[i] = pack_bf16(x, y);
            }
            tmem_st8(scol + 8 * q, pk);
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
        more = take_piece();
        continue;
      }
      if (two) {
        ok = __all_sync(kFull, mbar_wait(bar(B_ML), n_ml++ & 1));
        if (ok) ok = __all_sync(kFull, mbar_wait(bar(B_O + 1), n_ob & 1));
      }
      n_ob += two || (!narrow && pc.nblk > 0);
      if (ok && !staged) more = take_piece();
      if (ok && pc.nblk > 0) ok = __all_sync(kFull, mbar_wait(bar(B_O + t), n_o++ & 1));
      if (!ok) break;
      tc_fence_after();
      // weights of A's own result and of B's
      float wa = 1.f, wb = 0.f;
      if (two) {
        float2 other;
        tmem_ld2(scol + 128 + 126, other.x, other.y);
        const float m = fmaxf(m_ref, other.x);
        wa = m_ref == -INFINITY ? 0.f : ex2(m_ref - m);
        wb = other.x == -INFINITY ? 0.f : ex2(other.x - m);
        l = l * wa + other.y * wb;
        m_ref = m;
      }
      if (any) {
        // (a row without keys has l = 0; a NaN or a score of +inf makes l NaN, and the row)
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const float lse = l == 0.f ? -INFINITY : (m_ref + lg2(l)) * kLn2;
        wa *= inv;
        wb *= inv;
        const size_t slot = pc.slot;
        const int tok = (pc.row0 + row) / a.G, g = (pc.row0 + row) - tok * a.G;
        const size_t out_row = (size_t(pc.first) + tok) * a.Hq + size_t(pc.h) * a.G + g;
#pragma unroll 2
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
        if (staged) {
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
      if (staged) more = take_piece();
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // (after a wait that ran out)
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

// Joins the partial results of the cut items (an item's pieces have consecutive
// slots).  A unit is 32 rows of an item, a lane each; the CTAs take the units
// of all cut items in turn (a CTA for every possible unit would be 1,216, of which
// most calls have no use).  A warp takes every eighth group of four dims, which
// lie side by side for the rows; the log-sum-exps and results of four pieces
// are loaded at once, and the sums rescaled when later ones are larger.
constexpr int kMergeWarps = 8, kMergeAtOnce = 4, kMergeGroups = 32 / kMergeWarps;
__global__ void __launch_bounds__(kMergeWarps * 32) cross_merge_kernel(const __grid_constant__ CrossArgs a, int units) {
  __shared__ uint2 rows_out[32][33];  // bf16 rows (of 32 pieces of 8 bytes, and one to spread the banks)
  launch_dependents();
  wait_prerequisites();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int last = *a.n_split * units;
  for (int u = blockIdx.x; u < last; u += gridDim.x) {
    const int q = u / units, r0 = (u - q * units) * 32;  // the q-th cut item, its rows from r0 on
    const CrossSplit sp = a.split[q];
    if (sp.cuts == 0 || r0 >= sp.rows) continue;
    const int row = r0 + lane;
    const bool live = row < sp.rows;
    float M = -INFINITY, sum = 0.f;
    float4 acc[kMergeGroups];
#pragma unroll
    for (int i = 0; i < kMergeGroups; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int k0 = 0; k0 < sp.cuts; k0 += kMergeAtOnce) {
      float ls[kMergeAtOnce];
      float4 v[kMergeAtOnce][kMergeGroups];
#pragma unroll
      for (int k = 0; k < kMergeAtOnce; ++k) {
        const size_t slot = k0 + k ? (sp.slot & -sp.step) + (k0 + k) * sp.step : sp.slot;
        const bool in = live && k0 + k < sp.cuts;
        ls[k] = in ? a.lse_part[slot * a.part_rows + row] : -INFINITY;
#pragma unroll
        for (int i = 0; i < kMergeGroups; ++i)
          if (in) v[k][i] = reinterpret_cast<const float4*>(a.o_part)[(slot * 32 + warp + i * kMergeWarps) * a.part_rows + row];
      }
      float m = M;
#pragma unroll
      for (int k = 0; k < kMergeAtOnce; ++k) m = max_nan(m, ls[k]);  // (a NaN piece makes the row NaN)
      if (m == -INFINITY) continue;
      const float old = ex2((M - m) * 1.4426950408889634f);
      M = m;
      sum *= old;
#pragma unroll
      for (int i = 0; i < kMergeGroups; ++i) {
        acc[i].x *= old;
        acc[i].y *= old;
        acc[i].z *= old;
        acc[i].w *= old;
      }
#pragma unroll
      for (int k = 0; k < kMergeAtOnce; ++k) {
        if (ls[k] == -INFINITY) continue;  // (a piece that is none, or without weight)
        const float w = ex2((ls[k] - m) * 1.4426950408889634f);
        sum += w;
#pragma unroll
        for (int i = 0; i < kMergeGroups; ++i) {
          acc[i].x += w * v[k][i].x;
          acc[i].y += w * v[k][i].y;
          acc[i].z += w * v[k][i].z;
          acc[i].w += w * v[k][i].w;
        }
      }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    __syncthreads();  // (the rows of the unit before are out)
#pragma unroll
    for (int i = 0; i < kMergeGroups; ++i)
      rows_out[lane][warp + i * kMergeWarps] =
          make_uint2(pack_bf16(acc[i].x * inv, acc[i].y * inv), pack_bf16(acc[i].z * inv, acc[i].w * inv));
    __syncthreads();
    // whole rows out, a warp to a row
    for (int i = warp; i < 32 && r0 + i < sp.rows; i += kMergeWarps) {
      const int tok = (sp.row0 + r0 + i) / a.G, g = (sp.row0 + r0 + i) - tok * a.G;
      const size_t out_row = (size_t(sp.first) + tok) * a.Hq + size_t(sp.head) * a.G + g;
      reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + out_row * 128)[lane] = rows_out[i][lane];
    }
    if (warp == 0 && live && a.lse) {
      const int tok = (sp.row0 + row) / a.G, g = (sp.row0 + row) - tok * a.G;
      a.lse[(size_t(sp.first) + tok) * a.Hq + size_t(sp.head) * a.G + g] = sum == 0.f ? -INFINITY : M + lg2(sum) * kLn2;
    }
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
// from one item to the next (one token of 512 requests, 8 heads, 512 keys: 280 us,
// a CTA per item 405).  Many of more rows: a CTA per item, for its results pass
// through the shared memory that the next item's queries need (80 prompts of 40
// to 80 tokens, 32 heads on 8, 512 keys: 99 us, as a line 116; prompts of 4k
// tokens the same either way).
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

cudaError_t launch_cross(const CrossArgs& a, int64_t row_tiles, const TmaDesc& tk, const TmaDesc& tv, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_shared_memory(reinterpret_cast<const void*>(cross_attend_kernel), Cross::SMEM, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute la[1];
  la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  la[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = a.parts ? dim3(unsigned(a.parts), 1, 1)
                        : dim3(unsigned(int64_t(a.n_tokens) * a.G / Cross::ROWS + a.batch), unsigned(a.Hkv), 1);
  cfg.blockDim = dim3(Cross::THREADS, 1, 1);
  cfg.dynamicSmemBytes = Cross::SMEM;
  cfg.stream = s;
  cfg.attrs = la;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, cross_attend_kernel, a, *reinterpret_cast<const CUtensorMap*>(&tk),
                                     *reinterpret_cast<const CUtensorMap*>(&tv));
  if (e != cudaSuccess || a.parts == 0) return e;
  // With an item per CTA at most, a cut costs 1 + kPieceCost + kCutCost at least:
  // items of so few key blocks that none costs more are never cut (a token over
  // 256 keys of 16 heads: 9.4 us, with the merge's launch 10.9).
  const int64_t blocks = (int64_t(a.max_pages) * a.P + Cross::BK - 1) / Cross::BK;
  if (row_tiles * a.Hkv <= a.parts && blocks <= 1 + kCutCost) return e;
  const int units = (a.part_rows + 31) / 32;  // of an item
  cfg.gridDim = dim3(unsigned(units > 1 ? 2 * a.parts : a.parts), 1, 1);
  cfg.blockDim = dim3(kMergeWarps * 32, 1, 1);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, cross_merge_kernel, a, units);
}

}  // namespace splitkv
