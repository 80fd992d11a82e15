// Host side of the paged cache and of the rotary positions: descriptor,
// frequency and axis tables and the argument checks of the device calls
// (bgg_assign.hip, bgg_rotary.hip, bgg_attention.hip).  No GPU work happens
// here.
#include "bgg_cache.h"

#include <cmath>
#include <cstring>
#include <initializer_list>

namespace bgg {

bgg_status check_cache(const bgg_cache_desc* c) {
  if (!c) return fail(BGG_ERR_NULL, "cache descriptor is NULL");
  bgg_cache_desc ref;
  if (c->magic != BGG_CACHE_MAGIC || c->version != BGG_CACHE_VERSION)
    return fail(BGG_ERR_DESC, "cache descriptor magic/version mismatch");
  if (bgg_cache_describe(c->type, c->pages, c->page_size, c->kv_heads, c->head_dim, &ref) != BGG_OK)
    return fail(BGG_ERR_DESC, "cache descriptor fields describe no valid cache");
  if (std::memcmp(&ref, c, sizeof ref) != 0)
    return fail(BGG_ERR_DESC, "cache descriptor fields were modified after bgg_cache_describe");
  return BGG_OK;
}

static bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

static bgg_status check_type(const char* who, int32_t type) {
  if (type != BGG_TYPE_F16 && type != BGG_TYPE_BF16)
    return fail(BGG_ERR_FORMAT, "%s: activations of type %d", who, (int)type);
  return BGG_OK;
}

// A cache read or written by activations of `type`: scales come with an
// E4M3 cache and with no other.
static bgg_status check_cache_type(const char* who, const bgg_cache_desc* c, int32_t type,
                                   const float* k_scale, const float* v_scale) {
  if (c->type != BGG_TYPE_E4M3) {
    if (c->type != type)
      return fail(BGG_ERR_FORMAT, "%s: a 16-bit cache of type %d with activations of type %d", who,
                  (int)c->type, (int)type);
    if (k_scale || v_scale)
      return fail(BGG_ERR_FORMAT, "%s: scales for a 16-bit cache", who);
    return BGG_OK;
  }
  if (!k_scale || !v_scale) return fail(BGG_ERR_NULL, "%s: NULL scales of an E4M3 cache", who);
  if (!aligned(k_scale, 4) || !aligned(v_scale, 4))
    return fail(BGG_ERR_BUFFER, "%s: misaligned scales", who);
  return BGG_OK;
}

// A row operand: 16-byte aligned rows of `row` values, `stride` apart.
static bgg_status check_rows(const char* who, const char* what, const void* p, int64_t stride,
                             int64_t row) {
  if (!aligned(p, 16)) return fail(BGG_ERR_BUFFER, "%s: misaligned %s", who, what);
  if (stride < row || stride % 8 || stride > (int64_t(1) << 40))
    return fail(BGG_ERR_SHAPE, "%s: stride %lld of %s (rows hold %lld values)", who,
                (long long)stride, what, (long long)row);
  return BGG_OK;
}

static bgg_status check_rotary(const char* who, const bgg_cache_desc* c, const bgg_rotary_args* a) {
  bgg_status st = check_cache(c);
  if (st) return st;
  if (!a) return fail(BGG_ERR_NULL, "%s: NULL arguments", who);
  if (!a->k_dev != !a->v_dev) return fail(BGG_ERR_NULL, "%s: keys and values come together", who);
  if (!a->k_dev && !a->q_dev) return fail(BGG_ERR_NULL, "%s: neither queries nor keys", who);
  if (a->layout != BGG_ROTARY_HALF && a->layout != BGG_ROTARY_INTERLEAVED)
    return fail(BGG_ERR_FORMAT, "%s: unknown layout %d", who, (int)a->layout);
  if (a->reserved != 0) return fail(BGG_ERR_SHAPE, "%s: reserved must be 0", who);
  if (a->rotary_dim < 2 || a->rotary_dim > c->head_dim || a->rotary_dim % 2)
    return fail(BGG_ERR_SHAPE, "%s: rotary_dim %lld of a head of %lld", who,
                (long long)a->rotary_dim, (long long)c->head_dim);
  if (a->tokens < 0 || a->tokens > kMaxTokens)
    return fail(BGG_ERR_SHAPE, "%s: %lld tokens", who, (long long)a->tokens);
  if ((st = check_type(who, a->type))) return st;
  if (!a->positions_dev || !a->freqs_dev) return fail(BGG_ERR_NULL, "%s: NULL buffer", who);
  if (!aligned(a->positions_dev, 4) || !aligned(a->freqs_dev, 4))
    return fail(BGG_ERR_BUFFER, "%s: misaligned buffer", who);
  if (a->q_dev) {
    if (!a->q_out_dev) return fail(BGG_ERR_NULL, "%s: NULL buffer", who);
    if (a->q_heads < 1 || a->q_heads > kMaxQHeads)
      return fail(BGG_ERR_SHAPE, "%s: %lld query heads", who, (long long)a->q_heads);
    if ((st = check_rows(who, "q", a->q_dev, a->q_stride, a->q_heads * c->head_dim))) return st;
    if ((st = check_rows(who, "q_out", a->q_out_dev, a->q_out_stride, a->q_heads * c->head_dim))) return st;
    if (a->q_out_dev == a->q_dev && a->q_out_stride != a->q_stride)
      return fail(BGG_ERR_SHAPE, "%s: q rotated in place with two strides", who);
  } else if (a->q_heads != 0) {
    return fail(BGG_ERR_NULL, "%s: query heads without q", who);
  }
  if (a->k_dev) {
    if ((st = check_cache_type(who, c, a->type, a->k_scale_dev, a->v_scale_dev))) return st;
    if (!a->slots_dev || !a->k_cache_dev || !a->v_cache_dev)
      return fail(BGG_ERR_NULL, "%s: NULL buffer", who);
    if (!aligned(a->slots_dev, 8) || !aligned(a->k_cache_dev, 16) || !aligned(a->v_cache_dev, 16))
      return fail(BGG_ERR_BUFFER, "%s: misaligned buffer", who);
    if ((st = check_rows(who, "k", a->k_dev, a->k_stride, c->kv_heads * c->head_dim))) return st;
    if ((st = check_rows(who, "v", a->v_dev, a->v_stride, c->kv_heads * c->head_dim))) return st;
  }
  return BGG_OK;
}

bgg_status check_rotary(const bgg_cache_desc* c, const bgg_rotary_args* a) {
  return check_rotary("bgg_rotary_append", c, a);
}

bgg_status check_rotary_axes(const bgg_cache_desc* c, const bgg_rotary_args* a,
                             const bgg_rotary_axes_args* x) {
  const char* who = "bgg_rotary_append_axes";
  bgg_status st = check_rotary(who, c, a);
  if (st) return st;
  if (!x || !x->axis_of_pair_dev) return fail(BGG_ERR_NULL, "%s: NULL axes", who);
  if (x->axes < 1 || x->axes > BGG_MAX_AXES)
    return fail(BGG_ERR_SHAPE, "%s: %lld axes", who, (long long)x->axes);
  if (x->stride != 0 && (x->stride < a->tokens || x->stride > (int64_t(1) << 40)))
    return fail(BGG_ERR_SHAPE, "%s: rows of %lld positions %lld apart", who, (long long)a->tokens,
                (long long)x->stride);
  return BGG_OK;
}

bgg_status check_assign(const bgg_cache_desc* c, const bgg_assign_args* a) {
  const char* who = "bgg_cache_assign";
  bgg_status st = check_cache(c);
  if (st) return st;
  if (!a) return fail(BGG_ERR_NULL, "%s: NULL arguments", who);
  if (a->batch < 0 || a->batch > kMaxBatch)
    return fail(BGG_ERR_SHAPE, "%s: batch of %lld", who, (long long)a->batch);
  if (a->rows < 0 || a->rows > kMaxTokens)
    return fail(BGG_ERR_SHAPE, "%s: %lld rows", who, (long long)a->rows);
  if (a->table_width < 1 || a->table_width > 0x7FFFFFFF / c->page_size ||
      a->batch * a->table_width > (int64_t(1) << 31))
    return fail(BGG_ERR_SHAPE, "%s: %lld pages of %lld tokens for each of %lld sequences", who,
                (long long)a->table_width, (long long)c->page_size, (long long)a->batch);
  if (a->table_stride < a->table_width || a->table_stride > (int64_t(1) << 40))
    return fail(BGG_ERR_SHAPE, "%s: table stride %lld below its width %lld", who,
                (long long)a->table_stride, (long long)a->table_width);
  if (a->free_capacity < 1 || a->free_capacity > 0x7FFFFFFF)
    return fail(BGG_ERR_SHAPE, "%s: room for %lld free pages", who, (long long)a->free_capacity);
  if (!a->free_pages_dev || !a->free_count_dev || !a->free_count_out_dev || !a->starts_dev)
    return fail(BGG_ERR_NULL, "%s: NULL buffer", who);
  if (a->batch && (!a->lengths_dev || !a->counts_dev || !a->page_table_dev || !a->lengths_out_dev || !a->past_dev))
    return fail(BGG_ERR_NULL, "%s: NULL buffer", who);
  if (a->rows && (!a->positions_dev || !a->slots_dev)) return fail(BGG_ERR_NULL, "%s: NULL buffer", who);
  for (const void* p : {(const void*)a->lengths_dev, (const void*)a->counts_dev, (const void*)a->shared_pages_dev,
                        (const void*)a->page_table_dev, (const void*)a->free_pages_dev, (const void*)a->free_count_dev,
                        (const void*)a->lengths_out_dev, (const void*)a->free_count_out_dev, (const void*)a->past_dev,
                        (const void*)a->starts_dev, (const void*)a->positions_dev})
    if (!aligned(p, 4)) return fail(BGG_ERR_BUFFER, "%s: misaligned buffer", who);
  if (!aligned(a->slots_dev, 8)) return fail(BGG_ERR_BUFFER, "%s: misaligned slots", who);
  return BGG_OK;
}

static bool heads_ok(const bgg_cache_desc* c, int64_t q_heads) {
  return q_heads >= 1 && q_heads <= kMaxQHeads && q_heads % c->kv_heads == 0;
}

static bgg_status check_attention(const char* who, const bgg_cache_desc* c, const bgg_attention_args* a) {
  bgg_status st = check_cache(c);
  if (st) return st;
  if (!a) return fail(BGG_ERR_NULL, "%s: NULL arguments", who);
  if ((st = check_type(who, a->type))) return st;
  if ((st = check_cache_type(who, c, a->type, a->k_scale_dev, a->v_scale_dev))) return st;
  if (!heads_ok(c, a->q_heads))
    return fail(BGG_ERR_SHAPE, "%s: %lld query heads on %lld key heads", who, (long long)a->q_heads,
                (long long)c->kv_heads);
  if (a->batch < 0 || a->batch > kMaxBatch)
    return fail(BGG_ERR_SHAPE, "%s: batch of %lld", who, (long long)a->batch);
  if (a->window < 0) return fail(BGG_ERR_SHAPE, "%s: window %lld", who, (long long)a->window);
  if (!std::isfinite(a->scale)) return fail(BGG_ERR_SHAPE, "%s: scale is not finite", who);
  if (a->table_width < 1 || a->table_width > 0x7FFFFFFF / c->page_size)
    return fail(BGG_ERR_SHAPE, "%s: %lld pages of %lld tokens per sequence", who,
                (long long)a->table_width, (long long)c->page_size);
  if (a->table_stride < a->table_width || a->table_stride > (int64_t(1) << 40))
    return fail(BGG_ERR_SHAPE, "%s: table stride %lld below its width %lld", who,
                (long long)a->table_stride, (long long)a->table_width);
  if (!a->q_dev || !a->out_dev || !a->k_cache_dev || !a->v_cache_dev || !a->page_table_dev ||
      !a->lengths_dev || !a->workspace)
    return fail(BGG_ERR_NULL, "%s: NULL buffer", who);
  if (!aligned(a->k_cache_dev, 16) || !aligned(a->v_cache_dev, 16) || !aligned(a->workspace, 16) ||
      !aligned(a->page_table_dev, 4) || !aligned(a->lengths_dev, 4) || !aligned(a->lse_dev, 4))
    return fail(BGG_ERR_BUFFER, "%s: misaligned buffer", who);
  if ((st = check_rows(who, "q", a->q_dev, a->q_stride, a->q_heads * c->head_dim))) return st;
  if ((st = check_rows(who, "out", a->out_dev, a->out_stride, a->q_heads * c->head_dim))) return st;
  if (a->out_dev == a->q_dev && a->out_stride != a->q_stride && a->batch > 1)
    return fail(BGG_ERR_SHAPE, "%s: out in the place of q with two strides", who);
  return BGG_OK;
}

bgg_status check_attention(const bgg_cache_desc* c, const bgg_attention_args* a) {
  return check_attention("bgg_paged_attention", c, a);
}

bgg_status check_shared(const bgg_cache_desc* c, const bgg_attention_args* a, const bgg_shared_args* s) {
  const char* who = "bgg_shared_attention";
  bgg_status st = check_attention(who, c, a);
  if (st) return st;
  if (!s) return fail(BGG_ERR_NULL, "%s: NULL groups", who);
  if (s->groups < 0 || s->groups > a->batch)
    return fail(BGG_ERR_SHAPE, "%s: %lld groups of %lld sequences", who, (long long)s->groups, (long long)a->batch);
  if (s->groups == 0) return BGG_OK;
  if (!s->group_starts_dev || !s->shared_pages_dev) return fail(BGG_ERR_NULL, "%s: NULL buffer", who);
  if (!aligned(s->group_starts_dev, 4) || !aligned(s->shared_pages_dev, 4))
    return fail(BGG_ERR_BUFFER, "%s: misaligned buffer", who);
  return BGG_OK;
}

}  // namespace bgg

using namespace bgg;

extern "C" {

bgg_status bgg_cache_describe(int32_t type, int64_t pages, int64_t page_size, int64_t kv_heads,
                              int64_t head_dim, bgg_cache_desc* out) {
  if (!out) return fail(BGG_ERR_NULL, "bgg_cache_describe: out is NULL");
  if (type != BGG_TYPE_F16 && type != BGG_TYPE_BF16 && type != BGG_TYPE_E4M3)
    return fail(BGG_ERR_FORMAT, "bgg_cache_describe: unknown type %d", (int)type);
  if (pages < 1 || pages > 0x7FFFFFFF)
    return fail(BGG_ERR_SHAPE, "bgg_cache_describe: %lld pages", (long long)pages);
  if (page_size < 16 || page_size > BGG_MAX_PAGE_SIZE || (page_size & (page_size - 1)))
    return fail(BGG_ERR_SHAPE, "bgg_cache_describe: page size %lld is not a power of two in 16..%d",
                (long long)page_size, BGG_MAX_PAGE_SIZE);
  if (kv_heads < 1 || kv_heads > 1024)
    return fail(BGG_ERR_SHAPE, "bgg_cache_describe: %lld key heads", (long long)kv_heads);
  if (head_dim != 64 && head_dim != 96 && head_dim != 128 && head_dim != 192 && head_dim != 256)
    return fail(BGG_ERR_SHAPE, "bgg_cache_describe: head dimension %lld is not 64, 96, 128, 192 or 256",
                (long long)head_dim);
  bgg_cache_desc d;
  std::memset(&d, 0, sizeof d);
  d.magic = BGG_CACHE_MAGIC;
  d.version = BGG_CACHE_VERSION;
  d.type = type;
  d.pages = pages;
  d.page_size = page_size;
  d.kv_heads = kv_heads;
  d.head_dim = head_dim;
  d.page_bytes = (uint64_t)(kv_heads * page_size * head_dim) * (type == BGG_TYPE_E4M3 ? 1 : 2);
  if ((uint64_t)pages > (uint64_t(1) << 46) / d.page_bytes)
    return fail(BGG_ERR_SHAPE, "bgg_cache_describe: %lld pages of %llu bytes are too many",
                (long long)pages, (unsigned long long)d.page_bytes);
  d.total_bytes = (uint64_t)pages * d.page_bytes;
  *out = d;
  clear_error();
  return BGG_OK;
}

bgg_status bgg_rotary_frequencies(int64_t rotary_dim, double base, int32_t scaling, double factor,
                                  double trained_length, double low, double high, float* freqs,
                                  float* magnitude) {
  const char* who = "bgg_rotary_frequencies";
  if (!freqs || !magnitude) return fail(BGG_ERR_NULL, "%s: NULL output", who);
  if (scaling < BGG_ROTARY_NONE || scaling > BGG_ROTARY_PARTS)
    return fail(BGG_ERR_FORMAT, "%s: unknown scaling %d", who, (int)scaling);
  if (rotary_dim < 2 || rotary_dim > 256 || rotary_dim % 2 ||
      (scaling == BGG_ROTARY_BASE && rotary_dim < 4))
    return fail(BGG_ERR_SHAPE, "%s: rotary_dim %lld", who, (long long)rotary_dim);
  if (!(base > 1.0) || !std::isfinite(base)) return fail(BGG_ERR_SHAPE, "%s: base %g", who, base);
  if (scaling != BGG_ROTARY_NONE && (!(factor >= 1.0) || !std::isfinite(factor)))
    return fail(BGG_ERR_SHAPE, "%s: factor %g", who, factor);
  if (scaling == BGG_ROTARY_PARTS && (!(trained_length > 0.0) || !std::isfinite(trained_length) ||
                                      !std::isfinite(low) || !std::isfinite(high) || !(high > low)))
    return fail(BGG_ERR_SHAPE, "%s: trained length %g, bounds %g and %g", who, trained_length, low, high);
  const double d = (double)rotary_dim, two_pi = 6.283185307179586476925;
  const double b = scaling == BGG_ROTARY_BASE ? base * std::pow(factor, d / (d - 2.0)) : base;
  for (int64_t i = 0; i < rotary_dim / 2; ++i) {
    double f = std::pow(b, -2.0 * (double)i / d);
    if (scaling == BGG_ROTARY_LINEAR) f /= factor;
    if (scaling == BGG_ROTARY_PARTS) {
      const double r = trained_length * f / two_pi;
      const double g = std::fmin(std::fmax((r - low) / (high - low), 0.0), 1.0);
      f = (1.0 - g) * f / factor + g * f;
    }
    freqs[i] = (float)f;
  }
  *magnitude = scaling == BGG_ROTARY_PARTS ? (float)(1.0 + 0.1 * std::log(factor)) : 1.0f;
  clear_error();
  return BGG_OK;
}

bgg_status bgg_rotary_axes(const int64_t* sections, int64_t axes, int32_t arrangement,
                           uint8_t* axis_of_pair) {
  const char* who = "bgg_rotary_axes";
  if (!sections || !axis_of_pair) return fail(BGG_ERR_NULL, "%s: NULL argument", who);
  if (arrangement != BGG_AXES_BLOCKS && arrangement != BGG_AXES_CYCLIC)
    return fail(BGG_ERR_FORMAT, "%s: unknown arrangement %d", who, (int)arrangement);
  if (axes < 1 || axes > BGG_MAX_AXES) return fail(BGG_ERR_SHAPE, "%s: %lld axes", who, (long long)axes);
  int64_t pairs = 0;
  for (int64_t a = 0; a < axes; ++a) {
    if (sections[a] < 0 || sections[a] > 128)
      return fail(BGG_ERR_SHAPE, "%s: %lld pairs of axis %lld", who, (long long)sections[a], (long long)a);
    pairs += sections[a];
  }
  if (pairs < 1 || pairs > 128) return fail(BGG_ERR_SHAPE, "%s: %lld pairs", who, (long long)pairs);
  if (arrangement == BGG_AXES_BLOCKS) {
    int64_t i = 0;
    for (int64_t a = 0; a < axes; ++a)
      for (int64_t k = 0; k < sections[a]; ++k) axis_of_pair[i++] = (uint8_t)a;
  } else {
    for (int64_t a = 1; a < axes; ++a)  // its last pair is a + axes * (sections[a] - 1)
      if (sections[a] > 0 && a + axes * (sections[a] - 1) >= pairs)
        return fail(BGG_ERR_SHAPE, "%s: %lld pairs of axis %lld do not lie among %lld in turn", who,
                    (long long)sections[a], (long long)a, (long long)pairs);
    for (int64_t i = 0; i < pairs; ++i)
      axis_of_pair[i] = (uint8_t)(i < axes * sections[i % axes] ? i % axes : 0);
  }
  clear_error();
  return BGG_OK;
}

}  // extern "C"
