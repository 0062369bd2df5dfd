// C-ABI layer of the cache operators: append with norms and rotary positions, key
// weights, eviction, cross attention, attention and commit of drafted trees.  Argument validation, workspace layout, launches.
#include <cuda_runtime.h>

#include <cmath>
#include <new>

#include "internal.h"

namespace splitkv {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

bool misaligned(const void* p, uintptr_t bytes) {
  return p && (reinterpret_cast<uintptr_t>(p) & (bytes - 1));
}

// Whether [a, a + an) and [b, b + bn) share bytes.
bool overlap(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && an && bn && x < y + bn && y < x + an;
}

// `out` may be `in` itself or a buffer of its own.
bool half_shared(const void* in, const void* out, size_t bytes) {
  return in != out && overlap(in, bytes, out, bytes);
}

size_t state_bytes(const splitkv_desc_t& d) {
  return size_t(d.batch) * d.num_kv_heads * d.max_pages_per_seq * d.page_size * 4;
}

// A cache these operators serve: rows of 128 (keys and values apart) or the
// MLA family's rows of 576 (with the values in them, or apart in rows of 512).
splitkv_status validate_cache(const splitkv_desc_t* d) {
  splitkv_status st = validate_shape(d);
  if (st != SPLITKV_OK) return st;
  if (int64_t(d->max_pages_per_seq) * d->page_size > kMaxSlots)
    return fail(SPLITKV_EINVAL, "max_pages_per_seq * page_size must be at most 2^31 - 4096");
  const bool rows128 = d->qk_dim == 128 && d->v_dim == 128 && !d->v_shares_k;
  const bool latent = d->qk_dim == 576 && d->v_dim == 512 && d->num_kv_heads == 1;
  if (!rows128 && !latent)
    return fail(SPLITKV_EUNSUPPORTED,
                "no kernel for qk_dim=%d v_dim=%d v_shares_k=%d num_kv_heads=%d (qk_dim = v_dim = 128, "
                "or one KV head with qk_dim=576, v_dim=512)",
                d->qk_dim, d->v_dim, d->v_shares_k, d->num_kv_heads);
  return SPLITKV_OK;
}

splitkv_status check_scales(bool fp8, float kv_scale, const float* k_scale, const float* v_scale,
                            bool both) {
  if (!fp8) {
    if (k_scale || v_scale) return fail(SPLITKV_EINVAL, "k_scale and v_scale apply to e4m3 caches only");
    return SPLITKV_OK;
  }
  if (both && !k_scale != !v_scale) return fail(SPLITKV_EINVAL, "k_scale and v_scale must both be given");
  if (misaligned(k_scale, 4) || misaligned(v_scale, 4))
    return fail(SPLITKV_EINVAL, "k_scale and v_scale must be 4-byte aligned");
  if (!k_scale && (!(kv_scale > 0.f) || !(kv_scale < 1e30f)))
    return fail(SPLITKV_EINVAL, "kv_scale must be positive and finite");
  return SPLITKV_OK;
}

size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

// The records of cross attention's cut items (each has two of 2 * parts pieces at
// least), and their number.
size_t split_bytes(size_t parts) { return align256(parts * sizeof(CrossSplit) + sizeof(int32_t)); }

// The workspace of a call that is not dealt as whole items.
size_t cross_bytes(const splitkv_desc_t& d, int32_t n_tokens) {
  const size_t parts = kSmCount;
  return align256(2 * parts * cross_part_rows(d, n_tokens) * 129 * sizeof(float)) + split_bytes(parts);
}

// The shape of a call of cross attention's kernel, how its items are dealt, and where
// in the workspace what lies.
void fill_cross(CrossArgs& a, const splitkv_desc_t& d, int32_t n_tokens, void* workspace) {
  const CrossDeal deal = cross_deal(d, n_tokens);
  a.parts = deal == CrossDeal::kItems ? 0 : kSmCount;
  a.line = deal == CrossDeal::kLine;
  a.part_rows = cross_part_rows(d, n_tokens);
  if (a.parts > 0) {
    a.o_part = static_cast<float*>(workspace);
    a.lse_part = a.o_part + size_t(2) * a.parts * a.part_rows * 128;
    a.split = reinterpret_cast<CrossSplit*>(static_cast<unsigned char*>(workspace) + cross_bytes(d, n_tokens) -
                                            split_bytes(a.parts));
    a.n_split = reinterpret_cast<int32_t*>(a.split + a.parts);
  }
  a.n_tokens = n_tokens;
  a.batch = d.batch;
  a.T = d.q_tokens;
  a.Hq = d.num_q_heads;
  a.Hkv = d.num_kv_heads;
  a.G = d.num_q_heads / d.num_kv_heads;
  a.P = d.page_size;
  a.max_pages = d.max_pages_per_seq;
  a.num_pages = d.num_pages_total;
  a.box_rows = cross_box_rows(d);
  a.row_boxes = d.kv_dtype == SPLITKV_BF16 && kRowBoxRows % a.G == 0;
}

// Moves of one (sequence, head), at most: the kept keys behind the budget.
int64_t max_moves(const splitkv_desc_t& d, int32_t budget) {
  const int64_t cap = int64_t(d.max_pages_per_seq) * d.page_size;
  return budget >= cap ? 0 : (budget < cap - budget ? budget : cap - budget);
}

// Eviction starts up to eight CTAs for each (sequence, KV head).
splitkv_status validate_groups(const splitkv_desc_t* d) {
  splitkv_status st = validate_cache(d);
  if (st != SPLITKV_OK) return st;
  if (int64_t(d->batch) * d->num_kv_heads >= (int64_t(1) << 28))
    return fail(SPLITKV_EINVAL, "batch * num_kv_heads must be below 2^28");
  return SPLITKV_OK;
}

splitkv_status validate_cross(const splitkv_desc_t* d, int32_t n_tokens) {
  splitkv_status st = validate_cache(d);
  if (st != SPLITKV_OK) return st;
  if (d->qk_dim != 128 || d->kv_dtype != SPLITKV_BF16)
    return fail(SPLITKV_EUNSUPPORTED, "cross attention needs qk_dim = v_dim = 128 and a bf16 cache");
  if (n_tokens < 0 || int64_t(n_tokens) * d->num_q_heads >= (int64_t(1) << 31) || d->num_kv_heads > 65535)
    return fail(SPLITKV_EINVAL, "n_tokens must be >= 0 with n_tokens * num_q_heads < 2^31, and num_kv_heads at most 65535");
  return SPLITKV_OK;
}

splitkv_status validate_tree(const splitkv_desc_t* d, int32_t n_tokens) {
  splitkv_status st = validate_cache(d);
  if (st != SPLITKV_OK) return st;
  if (n_tokens < 0 || int64_t(n_tokens) * d->num_q_heads >= (int64_t(1) << 31) || d->num_kv_heads > 65535)
    return fail(SPLITKV_EINVAL, "n_tokens must be >= 0 with n_tokens * num_q_heads < 2^31, and num_kv_heads at most 65535");
  if (d->qk_dim == 128) return SPLITKV_OK;
  if (family_of(*d) != Family::kMla)
    return fail(SPLITKV_EUNSUPPORTED, "trees over latent rows need 128 query heads, q_tokens <= 16, pages of 16, 32 or a "
                "multiple of 64, and in e4m3 the values in the rows");
  if (n_tokens != 0 && int64_t(d->batch) * d->q_tokens != n_tokens)
    return fail(SPLITKV_EINVAL, "over latent rows n_tokens (%d) must be batch * q_tokens", n_tokens);
  return SPLITKV_OK;
}

// The workspace of a tree over latent rows: the splits of every sequence, where what
// lies (bytes from its start), and its size.
struct LatentTree {
  int32_t splits, items;
  size_t groups, log, status, lse, o, total;
};
LatentTree latent_tree(const splitkv_desc_t& d) {
  LatentTree w;
  // As many splits as cost least over a full cache, in its blocks of 64 keys: the longest
  // in each round of CTAs (two for every token, sequence and split, one to an SM), and
  // some 12 blocks' time to begin and to end it.  (12 tokens over 64k rows: 6 splits in
  // one round; 16 tokens 9 splits in two rather than 4 in one.)
  const int64_t blocks = (int64_t(d.max_pages_per_seq) * d.page_size + 63) / 64;
  int64_t least = INT64_MAX;
  w.splits = 1;
  for (int s = 1; s <= kMaxSplits && s <= d.max_pages_per_seq; ++s) {
    const int64_t rounds = (int64_t(d.batch) * s * 2 * d.q_tokens + kSmCount - 1) / kSmCount;
    const int64_t cost = rounds * ((blocks + s - 1) / s + 12);
    if (cost < least) {
      least = cost;
      w.splits = s;
    }
  }
  const int64_t items = int64_t(d.batch) * w.splits, rows = items * d.q_tokens * d.num_q_heads;
  w.items = int32_t(items);
  w.groups = 0;
  w.log = w.groups + align256(size_t(d.batch) * kGroupFields * 4);
  w.status = w.log + align256(size_t(items) * 2 * d.q_tokens * kLogFields * 4);
  w.lse = w.status + 256;
  w.o = w.lse + (w.splits > 1 ? align256(size_t(rows) * 4) : 0);
  w.total = w.o + (w.splits > 1 ? size_t(rows) * d.v_dim * 4 : 0);
  return w;
}

}  // namespace

cudaError_t set_attribute(const void* kernel, cudaFuncAttribute attribute, int value, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  return once_per_device(done, dev, cudaSuccess, [&] { return cudaFuncSetAttribute(kernel, attribute, value); });
}

}  // namespace splitkv

using namespace splitkv;

extern "C" {

splitkv_status splitkv_rope_create(int32_t rot_offset, int32_t rot_dim, int32_t n_axes,
                                   const int32_t* sections_host, int32_t pairing, double base,
                                   const double* freqs_host, splitkv_rope_t** rope_out) {
  if (!rope_out) return fail(SPLITKV_EINVAL, "rope_out is NULL");
  *rope_out = nullptr;
  if (rot_dim < 16 || rot_dim % 16 || rot_dim > 2 * kMaxRotPairs)
    return fail(SPLITKV_EINVAL, "rot_dim (%d) must be a multiple of 16 in [16, %d]", rot_dim,
                2 * kMaxRotPairs);
  if (rot_offset < 0 || rot_offset % 16)
    return fail(SPLITKV_EINVAL, "rot_offset (%d) must be a non-negative multiple of 16", rot_offset);
  if (n_axes < 1 || n_axes > kMaxAxes)
    return fail(SPLITKV_EINVAL, "n_axes (%d) must be in [1, %d]", n_axes, kMaxAxes);
  if (pairing != SPLITKV_ROPE_HALVES && pairing != SPLITKV_ROPE_NEIGHBOURS)
    return fail(SPLITKV_EINVAL, "unknown pairing %d", pairing);
  const int half = rot_dim / 2;
  if (n_axes > 1 && !sections_host) return fail(SPLITKV_EINVAL, "sections_host is NULL");
  if (sections_host) {
    int64_t sum = 0;
    for (int i = 0; i < n_axes; ++i) {
      if (sections_host[i] < 0) return fail(SPLITKV_EINVAL, "sections must be >= 0");
      sum += sections_host[i];
    }
    if (sum != half)
      return fail(SPLITKV_EINVAL, "sections sum to %lld, not to rot_dim / 2 = %d", (long long)sum, half);
  }
  if (!freqs_host && (!(base > 0.0) || !std::isfinite(base)))
    return fail(SPLITKV_EINVAL, "base must be positive and finite");
  for (int i = 0; freqs_host && i < half; ++i)
    if (!(std::fabs(freqs_host[i]) < 1e6))
      return fail(SPLITKV_EINVAL, "freqs[%d] must be finite and below 1e6 in magnitude", i);
  splitkv_rope_s* r = new (std::nothrow) splitkv_rope_s();
  if (!r) return fail(SPLITKV_EINVAL, "out of host memory");
  r->rot_offset = rot_offset;
  r->rot_dim = rot_dim;
  r->n_axes = n_axes;
  r->pairing = pairing;
  int axis = 0, left = sections_host ? sections_host[0] : half;
  for (int i = 0; i < half; ++i) {
    while (left == 0) left = sections_host[++axis];
    r->axis[i] = static_cast<unsigned char>(axis);
    --left;
    const double f = freqs_host ? freqs_host[i] : std::pow(base, -double(i) / half);
    // |f| / (2 pi) modulo 1 in 64-bit fixed point, from the product with
    // 1 / (2 pi) in two doubles (so that no digit of f is lost)
    const double inv_hi = 0.15915494309189535, inv_lo = -9.839338337591243e-18;
    const double m = std::fabs(f), hi = m * inv_hi, lo = std::fma(m, inv_hi, -hi) + m * inv_lo;
    const uint64_t turns = static_cast<uint64_t>(std::ldexp(hi - std::floor(hi), 64)) +
                           static_cast<uint64_t>(static_cast<int64_t>(std::llround(std::ldexp(lo, 64))));
    r->turns[i] = f < 0 ? 0 - turns : turns;
  }
  *rope_out = r;
  return SPLITKV_OK;
}

void splitkv_rope_destroy(splitkv_rope_t* rope) { delete rope; }

static splitkv_status append(const splitkv_desc_t* desc, const splitkv_norm_t* norm, const splitkv_rope_t* rope,
                             int32_t n_tokens, const int32_t* cu_tokens, const int32_t* positions,
                             const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                             const void* v, int64_t v_stride, const int32_t* block_table,
                             const int32_t* seq_lens, float kv_scale, const float* k_scale,
                             const float* v_scale, void* q_out, int64_t q_out_stride,
                             void* k_pages, void* v_pages, float* key_weights,
                             int32_t* key_positions, int32_t* status, void* stream) {
  splitkv_status st = validate_cache(desc);
  if (st != SPLITKV_OK) return st;
  const splitkv_desc_t& d = *desc;
  const bool fp8 = d.kv_dtype == SPLITKV_FP8_E4M3;
  if (n_tokens < 0) return fail(SPLITKV_EINVAL, "n_tokens must be >= 0");
  if (!cu_tokens && int64_t(d.batch) * d.q_tokens != n_tokens)
    return fail(SPLITKV_EINVAL, "without cu_tokens, n_tokens (%d) must be batch * q_tokens", n_tokens);
  if (norm) {
    if ((norm->norm_q || norm->norm_k) && !(norm->eps > 0.f && norm->eps < 1e30f))
      return fail(SPLITKV_EINVAL, "eps must be positive and finite");
    if ((norm->q_weight && !norm->norm_q) || (norm->k_weight && !norm->norm_k))
      return fail(SPLITKV_EINVAL, "a weight is given for rows that are not normalised");
    if (norm->norm_q && d.qk_dim != 128)
      return fail(SPLITKV_EUNSUPPORTED, "queries of latent caches are not normalised (norm_q must be 0)");
    if (misaligned(norm->q_weight, 16) || misaligned(norm->k_weight, 16))
      return fail(SPLITKV_EINVAL, "the weights of the norms must be 16-byte aligned");
  }
  if (n_tokens == 0) return SPLITKV_OK;
  if (!k || !block_table || !seq_lens || !k_pages)
    return fail(SPLITKV_EINVAL, "k, block_table, seq_lens and k_pages must not be NULL");
  if (!q != !q_out) return fail(SPLITKV_EINVAL, "q and q_out must both be given or both be NULL");
  if (d.v_shares_k && (v || v_pages))
    return fail(SPLITKV_EINVAL, "v and v_pages must be NULL when v_shares_k");
  if (!d.v_shares_k && (!v || !v_pages)) return fail(SPLITKV_EINVAL, "v or v_pages is NULL");
  if ((rope || key_positions) && !positions) return fail(SPLITKV_EINVAL, "positions is NULL");
  if (rope && rope->rot_offset + rope->rot_dim > d.qk_dim)
    return fail(SPLITKV_EINVAL, "the rotated columns [%d, %d) exceed qk_dim = %d", rope->rot_offset,
                rope->rot_offset + rope->rot_dim, d.qk_dim);
  const void* wide[] = {q, k, v, q_out, k_pages, v_pages};
  for (const void* p : wide)
    if (misaligned(p, 16)) return fail(SPLITKV_EINVAL, "q, k, v and the pages must be 16-byte aligned");
  const void* words[] = {cu_tokens, positions, block_table, seq_lens, key_weights, key_positions, status};
  for (const void* p : words)
    if (misaligned(p, 4)) return fail(SPLITKV_EINVAL, "index and state arrays must be 4-byte aligned");
  const int64_t q_row = int64_t(d.num_q_heads) * d.qk_dim, k_row = int64_t(d.num_kv_heads) * d.qk_dim,
                v_row = int64_t(d.num_kv_heads) * d.v_dim;
  const int64_t big = (int64_t(1) << 31) - 8;
  if ((q && (q_stride < q_row || q_stride % 8 || q_stride > big || q_out_stride < q_row || q_out_stride % 8 ||
             q_out_stride > big)) ||
      k_stride < k_row || k_stride % 8 || k_stride > big || (v && (v_stride < v_row || v_stride % 8 || v_stride > big)))
    return fail(SPLITKV_EINVAL,
                "token strides must be multiples of 8 elements, hold a token's heads and be below 2^31");
  if (q && !(q == q_out && q_stride == q_out_stride) &&
      overlap(q, size_t((n_tokens - 1) * q_stride + q_row) * 2, q_out,
              size_t((n_tokens - 1) * q_out_stride + q_row) * 2))
    return fail(SPLITKV_EINVAL, "q_out overlaps q without being q");
  st = check_scales(fp8, kv_scale, k_scale, v_scale, !d.v_shares_k);
  if (st != SPLITKV_OK) return st;
  AppendArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_out = q_out;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_out_stride = q_out_stride;
  a.cu = cu_tokens;
  a.positions = positions;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.key_weights = key_weights;
  a.key_positions = key_positions;
  a.status = status;
  a.kv_scale = kv_scale;
  a.n_tokens = n_tokens;
  a.batch = d.batch;
  a.T = d.q_tokens;
  a.Hq = d.num_q_heads;
  a.Hkv = d.num_kv_heads;
  a.P = d.page_size;
  a.max_pages = d.max_pages_per_seq;
  a.num_pages = d.num_pages_total;
  a.nhd = d.kv_layout == SPLITKV_LAYOUT_NHD;
  if (rope) a.rope = *rope;
  if (norm) {
    a.norm_q = q && norm->norm_q;
    a.norm_k = norm->norm_k;
    a.q_weight = norm->q_weight;
    a.k_weight = norm->k_weight;
    a.q_per_head = norm->q_per_head;
    a.k_per_head = norm->k_per_head;
    a.eps = norm->eps;
  }
  cudaError_t e = launch_append(a, d.qk_dim, d.v_dim, fp8, stream);
  if (e != cudaSuccess) return cuda_fail(e, "launching the append kernel");
  return SPLITKV_OK;
}

splitkv_status splitkv_append(const splitkv_desc_t* desc, const splitkv_rope_t* rope,
                              int32_t n_tokens, const int32_t* cu_tokens, const int32_t* positions,
                              const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                              const void* v, int64_t v_stride, const int32_t* block_table,
                              const int32_t* seq_lens, float kv_scale, const float* k_scale,
                              const float* v_scale, void* q_out, int64_t q_out_stride,
                              void* k_pages, void* v_pages, float* key_weights,
                              int32_t* key_positions, int32_t* status, void* stream) {
  return append(desc, nullptr, rope, n_tokens, cu_tokens, positions, q, q_stride, k, k_stride, v, v_stride, block_table,
                seq_lens, kv_scale, k_scale, v_scale, q_out, q_out_stride, k_pages, v_pages, key_weights, key_positions,
                status, stream);
}

splitkv_status splitkv_append_norm(const splitkv_desc_t* desc, const splitkv_norm_t* norm,
                                   const splitkv_rope_t* rope,
                                   int32_t n_tokens, const int32_t* cu_tokens, const int32_t* positions,
                                   const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                   const void* v, int64_t v_stride, const int32_t* block_table,
                                   const int32_t* seq_lens, float kv_scale, const float* k_scale,
                                   const float* v_scale, void* q_out, int64_t q_out_stride,
                                   void* k_pages, void* v_pages, float* key_weights,
                                   int32_t* key_positions, int32_t* status, void* stream) {
  if (!norm) return fail(SPLITKV_EINVAL, "norm is NULL");
  return append(desc, norm, rope, n_tokens, cu_tokens, positions, q, q_stride, k, k_stride, v, v_stride, block_table,
                seq_lens, kv_scale, k_scale, v_scale, q_out, q_out_stride, k_pages, v_pages, key_weights, key_positions,
                status, stream);
}

splitkv_status splitkv_key_weights(const splitkv_desc_t* desc, const void* q, const void* k_pages,
                                   const int32_t* block_table, const int32_t* seq_lens,
                                   const float* lse, float scale, float kv_scale,
                                   const float* k_scale, float decay, const float* weights_in,
                                   float* weights_out, int32_t* status, void* stream) {
  splitkv_status st = validate_cache(desc);
  if (st != SPLITKV_OK) return st;
  const splitkv_desc_t& d = *desc;
  if (family_of(d) != Family::kGqa)
    return fail(SPLITKV_EUNSUPPORTED, "key weights need qk_dim = v_dim = 128 and at most 32 query rows "
                "(q_tokens * num_q_heads / num_kv_heads) per KV head");
  const bool fp8 = d.kv_dtype == SPLITKV_FP8_E4M3;
  if (!q || !k_pages || !block_table || !seq_lens || !lse || !weights_out)
    return fail(SPLITKV_EINVAL, "q, k_pages, block_table, seq_lens, lse and weights_out must not be NULL");
  if (!(scale > 0.f) || !(scale < 1e30f)) return fail(SPLITKV_EINVAL, "scale must be positive and finite");
  if (!std::isfinite(decay)) return fail(SPLITKV_EINVAL, "decay must be finite");
  if (decay != 0.f && !weights_in) return fail(SPLITKV_EINVAL, "weights_in is NULL and decay is not 0");
  if (misaligned(q, 16) || misaligned(k_pages, 16))
    return fail(SPLITKV_EINVAL, "q and k_pages must be 16-byte aligned");
  const void* words[] = {block_table, seq_lens, lse, weights_in, weights_out, status};
  for (const void* p : words)
    if (misaligned(p, 4)) return fail(SPLITKV_EINVAL, "index, lse and weight arrays must be 4-byte aligned");
  if (decay != 0.f && half_shared(weights_in, weights_out, state_bytes(d)))
    return fail(SPLITKV_EINVAL, "weights_out overlaps weights_in without being it");
  st = check_scales(fp8, kv_scale, k_scale, nullptr, false);
  if (st != SPLITKV_OK) return st;
  WeightArgs a{};
  a.q = q;
  a.k_pages = k_pages;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.lse = lse;
  a.k_scale = k_scale;
  a.w_in = decay != 0.f ? weights_in : nullptr;
  a.w_out = weights_out;
  a.status = status;
  a.qk_scale_log2 = scale * kLog2e * (fp8 && !k_scale ? kv_scale : 1.f);
  a.decay = decay;
  a.batch = d.batch;
  a.T = d.q_tokens;
  a.Hq = d.num_q_heads;
  a.Hkv = d.num_kv_heads;
  a.G = d.num_q_heads / d.num_kv_heads;
  a.P = d.page_size;
  a.max_pages = d.max_pages_per_seq;
  a.num_pages = d.num_pages_total;
  a.nhd = d.kv_layout == SPLITKV_LAYOUT_NHD;
  cudaError_t e = launch_key_weights(a, fp8, stream);
  if (e != cudaSuccess) return cuda_fail(e, "launching the key weight kernel");
  return SPLITKV_OK;
}

size_t splitkv_evict_workspace_size(const splitkv_desc_t* desc, int32_t budget) {
  if (validate_groups(desc) != SPLITKV_OK || budget < 1) return 0;
  const size_t groups = size_t(desc->batch) * desc->num_kv_heads;
  return align256(groups * 8) + align256(groups * 2 * size_t(max_moves(*desc, budget)) * 4) + 256;
}

splitkv_status splitkv_evict(const splitkv_desc_t* desc, int32_t budget, int32_t sink,
                             int32_t recent, void* k_pages, void* v_pages,
                             const int32_t* block_table, const int32_t* seq_lens,
                             const float* weights_in, const int32_t* positions_in,
                             float* weights_out, int32_t* positions_out, int32_t* seq_lens_out,
                             void* workspace, size_t workspace_bytes, int32_t* status,
                             void* stream) {
  splitkv_status st = validate_groups(desc);
  if (st != SPLITKV_OK) return st;
  const splitkv_desc_t& d = *desc;
  if (budget < 1) return fail(SPLITKV_EINVAL, "budget must be >= 1");
  if (sink < 0 || recent < 0) return fail(SPLITKV_EINVAL, "sink and recent must be >= 0");
  if (!k_pages || !block_table || !seq_lens || !weights_in || !weights_out || !seq_lens_out)
    return fail(SPLITKV_EINVAL,
                "k_pages, block_table, seq_lens, weights_in, weights_out and seq_lens_out must not be NULL");
  if (d.v_shares_k ? v_pages != nullptr : v_pages == nullptr)
    return fail(SPLITKV_EINVAL, d.v_shares_k ? "v_pages must be NULL when v_shares_k" : "v_pages is NULL");
  if (!positions_in != !positions_out)
    return fail(SPLITKV_EINVAL, "positions_in and positions_out must both be given or both be NULL");
  if ((sink > 0 || recent > 0) && !positions_in)
    return fail(SPLITKV_EINVAL, "sink and recent need positions");
  const void* wide[] = {k_pages, v_pages, weights_in, positions_in, weights_out, positions_out};
  for (const void* p : wide)
    if (misaligned(p, 16)) return fail(SPLITKV_EINVAL, "the pages and state arrays must be 16-byte aligned");
  const void* words[] = {block_table, seq_lens, seq_lens_out, status};
  for (const void* p : words)
    if (misaligned(p, 4)) return fail(SPLITKV_EINVAL, "index arrays must be 4-byte aligned");
  const size_t sb = state_bytes(d), lb = size_t(d.batch) * 4;
  if (half_shared(weights_in, weights_out, sb) || half_shared(positions_in, positions_out, sb) ||
      half_shared(seq_lens, seq_lens_out, lb))
    return fail(SPLITKV_EINVAL, "an output overlaps its input without being it");
  if (!workspace) return fail(SPLITKV_EWORKSPACE, "workspace is NULL");
  if (misaligned(workspace, 16)) return fail(SPLITKV_EINVAL, "workspace must be 16-byte aligned");
  const size_t need = splitkv_evict_workspace_size(desc, budget);
  if (workspace_bytes < need)
    return fail(SPLITKV_EWORKSPACE, "workspace has %zu bytes, the call needs %zu", workspace_bytes, need);
  EvictArgs a{};
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.w_in = weights_in;
  a.pos_in = positions_in;
  a.w_out = weights_out;
  a.pos_out = positions_out;
  a.lens_out = seq_lens_out;
  a.meta = static_cast<int32_t*>(workspace);
  a.moves = reinterpret_cast<int32_t*>(static_cast<unsigned char*>(workspace) +
                                       align256(size_t(d.batch) * d.num_kv_heads * 8));
  a.status = status;
  a.batch = d.batch;
  a.Hkv = d.num_kv_heads;
  a.P = d.page_size;
  a.max_pages = d.max_pages_per_seq;
  a.num_pages = d.num_pages_total;
  a.nhd = d.kv_layout == SPLITKV_LAYOUT_NHD;
  a.budget = budget;
  a.sink = sink;
  a.recent = recent;
  a.max_moves = int32_t(max_moves(d, budget));
  const int elem = d.kv_dtype == SPLITKV_FP8_E4M3 ? 1 : 2;
  a.k_row = d.qk_dim * elem;
  a.v_row = d.v_shares_k ? 0 : d.v_dim * elem;
  cudaError_t e = launch_evict(a, stream);
  if (e != cudaSuccess) return cuda_fail(e, "launching the eviction kernels");
  return SPLITKV_OK;
}

size_t splitkv_cross_workspace_size(const splitkv_desc_t* desc, int32_t n_tokens) {
  if (validate_cross(desc, n_tokens) != SPLITKV_OK || n_tokens == 0) return 0;
  if (cross_deal(*desc, n_tokens) == CrossDeal::kItems) return 0;
  return cross_bytes(*desc, n_tokens);
}

splitkv_status splitkv_cross_attend(const splitkv_desc_t* desc, int32_t n_tokens,
                                    const int32_t* cu_tokens, const void* q, int64_t q_stride,
                                    const void* k_pages, const void* v_pages,
                                    const int32_t* block_table, const int32_t* seq_lens,
                                    float scale, void* out, float* lse, void* workspace,
                                    size_t workspace_bytes, int32_t* status, void* stream) {
  splitkv_status st = validate_cross(desc, n_tokens);
  if (st != SPLITKV_OK) return st;
  const splitkv_desc_t& d = *desc;
  if (!cu_tokens && int64_t(d.batch) * d.q_tokens != n_tokens)
    return fail(SPLITKV_EINVAL, "without cu_tokens, n_tokens (%d) must be batch * q_tokens", n_tokens);
  if (n_tokens == 0) return SPLITKV_OK;
  if (!q || !k_pages || !v_pages || !block_table || !seq_lens || !out)
    return fail(SPLITKV_EINVAL, "q, k_pages, v_pages, block_table, seq_lens and out must not be NULL");
  const void* wide[] = {q, k_pages, v_pages, out};
  for (const void* p : wide)
    if (misaligned(p, 16)) return fail(SPLITKV_EINVAL, "q, out and the pages must be 16-byte aligned");
  const void* words[] = {cu_tokens, block_table, seq_lens, lse, status};
  for (const void* p : words)
    if (misaligned(p, 4)) return fail(SPLITKV_EINVAL, "index arrays and lse must be 4-byte aligned");
  const int64_t row = int64_t(d.num_q_heads) * 128;
  if (q_stride < row || q_stride % 8 || q_stride > (int64_t(1) << 31) - 8)
    return fail(SPLITKV_EINVAL, "q_stride must be a multiple of 8 elements, hold a token's heads and be below 2^31");
  if (overlap(q, size_t((n_tokens - 1) * q_stride + row) * 2, out, size_t(n_tokens) * row * 2))
    return fail(SPLITKV_EINVAL, "out overlaps q");
  if (!(scale > 0.f) || !(scale < 1e30f)) return fail(SPLITKV_EINVAL, "scale must be positive and finite");
  const size_t need = splitkv_cross_workspace_size(desc, n_tokens);
  if (need > 0) {
    if (!workspace) return fail(SPLITKV_EWORKSPACE, "workspace is NULL");
    if (misaligned(workspace, 16)) return fail(SPLITKV_EINVAL, "workspace must be 16-byte aligned");
    if (workspace_bytes < need)
      return fail(SPLITKV_EWORKSPACE, "workspace has %zu bytes, the call needs %zu", workspace_bytes, need);
  }
  CrossArgs a{};
  fill_cross(a, d, n_tokens, workspace);
  a.q = q;
  a.cu = cu_tokens;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.out = out;
  a.lse = lse;
  a.status = status;
  a.q_stride = q_stride;
  a.qk_scale_log2 = scale * kLog2e;
  CrossMaps maps{};
  st = make_cross_maps(&maps, a, k_pages, v_pages, d);
  if (st != SPLITKV_OK) return st;
  cudaError_t e = launch_cross(a, cross_row_tiles(d, n_tokens), maps, stream);
  if (e != cudaSuccess) return cuda_fail(e, "launching the cross attention kernels");
  return SPLITKV_OK;
}

size_t splitkv_tree_workspace_size(const splitkv_desc_t* desc, int32_t n_tokens) {
  if (validate_tree(desc, n_tokens) != SPLITKV_OK || n_tokens == 0) return 0;
  if (desc->qk_dim != 128) return latent_tree(*desc).total;
  if (cross_deal(*desc, n_tokens) == CrossDeal::kItems) return 0;
  return cross_bytes(*desc, n_tokens);
}

splitkv_status splitkv_tree_attend(const splitkv_desc_t* desc, int32_t n_tokens,
                                   const int32_t* cu_tokens, const uint32_t* tree_mask,
                                   int32_t mask_words, const void* q, int64_t q_stride,
                                   const void* k_pages, const void* v_pages,
                                   const int32_t* block_table, const int32_t* seq_lens, float scale,
                                   float kv_scale, const float* k_scale, const float* v_scale,
                                   void* out, float* lse, void* workspace, size_t workspace_bytes,
                                   int32_t* status, void* stream) {
  splitkv_status st = validate_tree(desc, n_tokens);
  if (st != SPLITKV_OK) return st;
  const splitkv_desc_t& d = *desc;
  const bool fp8 = d.kv_dtype == SPLITKV_FP8_E4M3, latent = d.qk_dim != 128;
  if (latent && cu_tokens) return fail(SPLITKV_EINVAL, "over latent rows every sequence has q_tokens tokens: cu_tokens must be NULL");
  if (!cu_tokens && int64_t(d.batch) * d.q_tokens != n_tokens)
    return fail(SPLITKV_EINVAL, "without cu_tokens, n_tokens (%d) must be batch * q_tokens", n_tokens);
  if (n_tokens == 0) return SPLITKV_OK;
  if (!tree_mask || !q || !k_pages || !block_table || !seq_lens || !out)
    return fail(SPLITKV_EINVAL, "tree_mask, q, k_pages, block_table, seq_lens and out must not be NULL");
  if (d.v_shares_k ? v_pages != nullptr : v_pages == nullptr)
    return fail(SPLITKV_EINVAL, d.v_shares_k ? "v_pages must be NULL when v_shares_k" : "v_pages is NULL");
  if (mask_words < 1 || mask_words > kMaxMaskWords)
    return fail(SPLITKV_EINVAL, "mask_words (%d) must be in [1, %d]", mask_words, kMaxMaskWords);
  const void* wide[] = {q, k_pages, v_pages, out};
  for (const void* p : wide)
    if (misaligned(p, 16)) return fail(SPLITKV_EINVAL, "q, out and the pages must be 16-byte aligned");
  const void* words[] = {cu_tokens, tree_mask, block_table, seq_lens, lse, status};
  for (const void* p : words)
    if (misaligned(p, 4)) return fail(SPLITKV_EINVAL, "the mask, index arrays and lse must be 4-byte aligned");
  const int64_t row = int64_t(d.num_q_heads) * d.qk_dim, out_row = int64_t(d.num_q_heads) * d.v_dim;
  if (q_stride < row || q_stride % 8 || q_stride > (int64_t(1) << 31) - 8)
    return fail(SPLITKV_EINVAL, "q_stride must be a multiple of 8 elements, hold a token's heads and be below 2^31");
  if (latent && n_tokens > 1 && q_stride != row)
    return fail(SPLITKV_EINVAL, "over latent rows the tokens of q must be adjacent");
  if (overlap(q, size_t((n_tokens - 1) * q_stride + row) * 2, out, size_t(n_tokens) * out_row * 2))
    return fail(SPLITKV_EINVAL, "out overlaps q");
  if (!(scale > 0.f) || !(scale < 1e30f)) return fail(SPLITKV_EINVAL, "scale must be positive and finite");
  st = check_scales(fp8, kv_scale, k_scale, v_scale, true);
  if (st != SPLITKV_OK) return st;
  if (latent && k_scale) return fail(SPLITKV_EUNSUPPORTED, "k_scale and v_scale apply to rows of 128 only");
  const size_t need = splitkv_tree_workspace_size(desc, n_tokens);
  if (need > 0) {
    if (!workspace) return fail(SPLITKV_EWORKSPACE, "workspace is NULL");
    if (misaligned(workspace, 16)) return fail(SPLITKV_EINVAL, "workspace must be 16-byte aligned");
    if (workspace_bytes < need)
      return fail(SPLITKV_EWORKSPACE, "workspace has %zu bytes, the call needs %zu", workspace_bytes, need);
  }
  const float qk_scale = scale * kLog2e * (fp8 && !k_scale ? kv_scale : 1.f), o_scale = fp8 ? kv_scale : 1.f;
  if (latent) {
    const LatentTree w = latent_tree(d);
    if (int64_t(w.items) * 2 * d.q_tokens >= (int64_t(1) << 31))
      return fail(SPLITKV_EINVAL, "batch * q_tokens must be below 2^30");
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    DecodeArgs a{};
    a.groups = reinterpret_cast<const int32_t*>(ws + w.groups);
    a.cta_log = reinterpret_cast<int32_t*>(ws + w.log);
    a.status = status ? status : reinterpret_cast<int32_t*>(ws + w.status);
    a.lse_part = reinterpret_cast<float*>(ws + w.lse);
    a.o_part = reinterpret_cast<float*>(ws + w.o);
    a.block_table = block_table;
    a.seq_lens = seq_lens;
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.n_items = w.items;
    a.n_groups = w.splits > 1 ? d.batch : 0;
    a.batch = d.batch;
    a.T = d.q_tokens;
    a.Hq = d.num_q_heads;
    a.Hkv = 1;
    a.G = d.num_q_heads;
    a.P = d.page_size;
    a.max_pages = d.max_pages_per_seq;
    a.num_pages = d.num_pages_total;
    a.rows = d.q_tokens * d.num_q_heads;
    a.dv = d.v_dim;
    a.qk_scale_log2 = qk_scale;
    a.o_scale = o_scale;
    a.fixed = 1;
    a.max_splits = w.splits;
    a.hpi = 1;
    a.fx = {seq_lens, w.splits, 1, 1, d.page_size, d.q_tokens, int64_t(d.max_pages_per_seq) * d.page_size};
    a.mask = tree_mask;
    a.words = mask_words;
    TmaDesc tk, tv;
    st = make_mla_maps(&tk, &tv, k_pages, v_pages, d);
    if (st != SPLITKV_OK) return st;
    cudaError_t e = launch_mla(a, tk, d.v_shares_k ? nullptr : &tv, fp8, stream);
    if (e == cudaSuccess) e = launch_combine(a, true, stream);
    if (e != cudaSuccess) return cuda_fail(e, "launching the tree attention kernels");
    return SPLITKV_OK;
  }
  CrossArgs a{};
  fill_cross(a, d, n_tokens, workspace);
  a.q = q;
  a.cu = cu_tokens;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.out = out;
  a.lse = lse;
  a.status = status;
  a.q_stride = q_stride;
  a.qk_scale_log2 = qk_scale;
  a.mask = tree_mask;
  a.words = mask_words;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.o_scale = o_scale;
  CrossMaps maps{};
  st = make_cross_maps(&maps, a, k_pages, v_pages, d);
  if (st != SPLITKV_OK) return st;
  cudaError_t e = launch_tree(a, cross_row_tiles(d, n_tokens), maps, fp8, stream);
  if (e != cudaSuccess) return cuda_fail(e, "launching the tree attention kernels");
  return SPLITKV_OK;
}

splitkv_status splitkv_tree_commit(const splitkv_desc_t* desc, int32_t max_path, const int32_t* path,
                                   const int32_t* path_lens, const int32_t* cu_tokens, void* k_pages,
                                   void* v_pages, const int32_t* block_table, const int32_t* seq_lens,
                                   float* key_weights, int32_t* key_positions, int32_t* seq_lens_out,
                                   int32_t* status, void* stream) {
  splitkv_status st = validate_cache(desc);
  if (st != SPLITKV_OK) return st;
  const splitkv_desc_t& d = *desc;
  if (max_path < 1) return fail(SPLITKV_EINVAL, "max_path must be >= 1");
  if (!path || !path_lens || !k_pages || !block_table || !seq_lens || !seq_lens_out)
    return fail(SPLITKV_EINVAL, "path, path_lens, k_pages, block_table, seq_lens and seq_lens_out must not be NULL");
  if (d.v_shares_k ? v_pages != nullptr : v_pages == nullptr)
    return fail(SPLITKV_EINVAL, d.v_shares_k ? "v_pages must be NULL when v_shares_k" : "v_pages is NULL");
  if (misaligned(k_pages, 16) || misaligned(v_pages, 16))
    return fail(SPLITKV_EINVAL, "the pages must be 16-byte aligned");
  const void* words[] = {path, path_lens, cu_tokens, block_table, seq_lens, key_weights, key_positions, seq_lens_out, status};
  for (const void* p : words)
    if (misaligned(p, 4)) return fail(SPLITKV_EINVAL, "index and state arrays must be 4-byte aligned");
  if (half_shared(seq_lens, seq_lens_out, size_t(d.batch) * 4))
    return fail(SPLITKV_EINVAL, "seq_lens_out overlaps seq_lens without being it");
  CommitArgs a{};
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.path = path;
  a.path_lens = path_lens;
  a.cu = cu_tokens;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.key_weights = key_weights;
  a.key_positions = key_positions;
  a.lens_out = seq_lens_out;
  a.status = status;
  a.batch = d.batch;
  a.T = d.q_tokens;
  a.Hkv = d.num_kv_heads;
  a.P = d.page_size;
  a.max_pages = d.max_pages_per_seq;
  a.num_pages = d.num_pages_total;
  a.nhd = d.kv_layout == SPLITKV_LAYOUT_NHD;
  a.max_path = max_path;
  const int elem = d.kv_dtype == SPLITKV_FP8_E4M3 ? 1 : 2;
  a.k_row = d.qk_dim * elem;
  a.v_row = d.v_shares_k ? 0 : d.v_dim * elem;
  cudaError_t e = launch_tree_commit(a, stream);
  if (e != cudaSuccess) return cuda_fail(e, "launching the commit kernel");
  return SPLITKV_OK;
}

}  // extern "C"
