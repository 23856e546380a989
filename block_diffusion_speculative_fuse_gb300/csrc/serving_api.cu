// C ABI of the serving operators: argument checks, workspace layout, launches.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "dflash.h"
#include "kernels.h"
#include "prefix_attention.cuh"

using namespace dflash;

namespace {

constexpr size_t kHeaderBytes = 64 * 1024;  // of every workspace (status word first)
constexpr double kTwoPi = 6.283185307179586476925;

size_t al256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int terms_of(const dflash_heads* h) { return h->kv_terms == 2 ? 2 : 1; }

int check_heads(const dflash_heads* h) {
  if (h == nullptr || h->n_layers < 1) return DFLASH_ERR_INVALID_ARG;
  if ((h->head_dim != 64 && h->head_dim != 128) || h->page_size != 16 || h->n_kv_heads < 1 ||
      h->n_q_heads < 1 || h->n_q_heads % h->n_kv_heads || h->n_q_heads / h->n_kv_heads > 16 ||
      h->n_q_heads > 65536 || h->kv_terms < 0 || h->kv_terms > 2)
    return DFLASH_ERR_UNSUPPORTED;
  return DFLASH_OK;
}

int check_cache(const dflash_heads* h, int32_t layer, const dflash_kv* kv) {
  if (kv == nullptr || kv->pool == nullptr || kv->page_table == nullptr || kv->n_pages <= 0 ||
      kv->max_pages <= 0 || kv->n_rows <= 0 || (kv->dtype != 0 && kv->dtype != 1) ||
      !aligned(kv->pool, 16) || !aligned(kv->page_table, 4) || layer < 0 || layer >= h->n_layers)
    return DFLASH_ERR_INVALID_ARG;
  // positions and page-table entries are counted in 32 bits
  if (kv->max_pages > (1 << 26)) return DFLASH_ERR_UNSUPPORTED;
  if (kv->dtype == 1) {
    if (kv->scales == nullptr || !aligned(kv->scales, 16)) return DFLASH_ERR_INVALID_ARG;
    if (terms_of(h) != 1) return DFLASH_ERR_UNSUPPORTED;
  }
  return DFLASH_OK;
}

int check_ws(const void* ws, size_t ws_bytes, size_t need) {
  if (ws == nullptr || !aligned(ws, 256)) return DFLASH_ERR_INVALID_ARG;
  return ws_bytes < need ? DFLASH_ERR_CAPACITY : DFLASH_OK;
}

// elements of one layer of the pool
size_t layer_elems(const dflash_heads* h, const dflash_kv* kv) {
  return static_cast<size_t>(kv->n_pages) * 2 * terms_of(h) * h->n_kv_heads * 16 * h->head_dim;
}

// The fraction of a turn that the angle f is, in units of 2^-64, off by one at most
// for f up to 1e9: the quotient by 2 pi as two doubles (the first alone is off by
// 286 units at f = 1, and loses what its whole turns take).
unsigned long long turn_fraction(double f) {
  constexpr double kTwoPiLow = 2.449293598294706414e-16;  // 2 pi - kTwoPi
  const double q = f / kTwoPi;
  const double low = (std::fma(-q, kTwoPi, f) - q * kTwoPiLow) / kTwoPi;
  auto units = [](double t) { return static_cast<unsigned long long>(std::ldexp(t - std::floor(t), 64)); };
  return low < 0.0 ? units(q) - units(-low) : units(q) + units(low);
}

// Workspace of the prefix attention: header, the lists' chunk offsets, then
// the partial results.  Returns the bytes; fills the pointers when base is set.
size_t layout_prefix(PrefixParams* p, int d, uint8_t* base) {
  size_t off = kHeaderBytes;
  auto take = [&](size_t bytes) {
    uint8_t* q = base == nullptr ? nullptr : base + off;
    off = al256(off + bytes);
    return q;
  };
  for (PrefixList& L : p->list) {
    const size_t rows = static_cast<size_t>(p->hkv) * (static_cast<size_t>(p->ng) * L.prefix_tiles * L.prefix_rows +
                                                       static_cast<size_t>(p->batch) * L.suffix_tiles * L.suffix_rows) +
                        static_cast<size_t>(L.workers) * L.worker_rows;
    L.off = reinterpret_cast<int*>(take((p->ng + p->batch + 1) * sizeof(int)));
    L.unit = reinterpret_cast<int*>(take((p->ng + p->batch + 1) * sizeof(int)));
    L.part_o = reinterpret_cast<float*>(take(rows * d * sizeof(float)));
    L.part_ml = reinterpret_cast<float*>(take(rows * 2 * sizeof(float)));
  }
  return off;
}

bool prefix_sizes(const dflash_heads* h, int32_t batch, int32_t n, int32_t group, PrefixParams* p) {
  if (batch < 1 || batch > kMaxPrefixBatch || n < 1 || n > 32 || group < 1 || batch % group) return false;
  std::memset(p, 0, sizeof(*p));
  p->batch = batch;
  p->n = n;
  p->group = group;
  p->hq = h->n_q_heads;
  p->hkv = h->n_kv_heads;
  prefix_attention_shape(p);
  return true;
}

}  // namespace

extern "C" {

int dflash_rope_init(dflash_rope* rope, int32_t rot_dim, int32_t interleaved, double base,
                     int32_t scaling, double factor, int32_t orig_ctx, double beta_fast,
                     double beta_slow) {
  if (rope == nullptr || (interleaved != 0 && interleaved != 1) || !(base > 1.0) ||
      !std::isfinite(base))
    return DFLASH_ERR_INVALID_ARG;
  if (rot_dim < 0 || rot_dim > 128 || rot_dim % 16) return DFLASH_ERR_UNSUPPORTED;
  if (scaling < DFLASH_ROPE_NONE || scaling > DFLASH_ROPE_YARN) return DFLASH_ERR_INVALID_ARG;
  if (scaling != DFLASH_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor)))
    return DFLASH_ERR_INVALID_ARG;
  if (scaling == DFLASH_ROPE_YARN &&
      (orig_ctx < 1 || !(beta_slow > 0.0) || !(beta_fast > beta_slow) || !std::isfinite(beta_fast)))
    return DFLASH_ERR_INVALID_ARG;
  std::memset(rope, 0, sizeof(*rope));
  rope->rot_dim = rot_dim;
  rope->interleaved = interleaved;
  rope->mscale = 1.0;
  const int half = rot_dim / 2;
  double b = base;
  if (scaling == DFLASH_ROPE_NTK && rot_dim > 0) b *= std::pow(factor, rot_dim / (rot_dim - 2.0));
  // YaRN: the (fractional) pair that turns beta times in orig_ctx positions
  double low = 0.0, high = 0.0;
  if (scaling == DFLASH_ROPE_YARN) {
    auto pair_of = [&](double beta) {
      return rot_dim * std::log(orig_ctx / (beta * kTwoPi)) / (2.0 * std::log(base));
    };
    low = std::max(std::floor(pair_of(beta_fast)), 0.0);
    high = std::min(std::ceil(pair_of(beta_slow)), rot_dim - 1.0);
    rope->mscale = 0.1 * std::log(factor) + 1.0;
  }
  for (int p = 0; p < half; ++p) {
    double f = std::pow(b, -2.0 * p / rot_dim);
    if (scaling == DFLASH_ROPE_LINEAR) f /= factor;
    if (scaling == DFLASH_ROPE_YARN) {
      const double slow = std::min(std::max((p - low) / std::max(high - low, 1e-3), 0.0), 1.0);
      f = f / factor * slow + f * (1.0 - slow);
    }
    rope->inv_freq[p] = f;
  }
  return DFLASH_OK;
}

int dflash_kv_rope_append(const dflash_heads* heads, const dflash_rope* rope, int32_t layer,
                          const void* q, int64_t ld_q, const void* k, int64_t ld_k, const void* v,
                          int64_t ld_v, int32_t in_dtype, const void* q_norm, const void* k_norm,
                          float eps, const int32_t* row_req, const int32_t* row_pos, int32_t T,
                          void* q_out, int64_t ld_qo, const dflash_kv* kv, void* ws,
                          size_t ws_bytes, void* stream) {
  int rc = check_heads(heads);
  if (rc) return rc;
  if (rope == nullptr || k == nullptr || v == nullptr || row_req == nullptr || row_pos == nullptr ||
      T < 1 || (in_dtype != 0 && in_dtype != 1) || (q == nullptr) != (q_out == nullptr) ||
      !(eps >= 0.f))
    return DFLASH_ERR_INVALID_ARG;
  const int d = heads->head_dim;
  const int64_t per16 = in_dtype == 1 ? 4 : 8;  // elements of 16 bytes
  const int64_t kv_row = static_cast<int64_t>(heads->n_kv_heads) * d;
  const int64_t q_row = static_cast<int64_t>(heads->n_q_heads) * d;
  if (!aligned(k, 16) || !aligned(v, 16) || ld_k < kv_row || ld_v < kv_row || ld_k % per16 ||
      ld_v % per16 || !aligned(row_req, 4) || !aligned(row_pos, 4))
    return DFLASH_ERR_INVALID_ARG;
  if (q != nullptr && (!aligned(q, 16) || !aligned(q_out, 16) || ld_q < q_row || ld_qo < q_row ||
                       ld_q % per16 || ld_qo % 8 || (q == q_out && (in_dtype != 0 || ld_q != ld_qo))))
    return DFLASH_ERR_INVALID_ARG;
  if ((q_norm != nullptr && !aligned(q_norm, 16)) || (k_norm != nullptr && !aligned(k_norm, 16)))
    return DFLASH_ERR_INVALID_ARG;
  if (rope->rot_dim < 0 || rope->rot_dim % 16 || rope->rot_dim > d) return DFLASH_ERR_UNSUPPORTED;
  if ((rope->interleaved != 0 && rope->interleaved != 1) || !std::isfinite(static_cast<float>(rope->mscale)))
    return DFLASH_ERR_INVALID_ARG;
  rc = check_cache(heads, layer, kv);
  if (!rc) rc = check_ws(ws, ws_bytes, kHeaderBytes);
  if (rc) return rc;
  RopeAppendParams p;
  std::memset(&p, 0, sizeof(p));
  for (int j = 0; j < rope->rot_dim / 2; ++j) {
    const double f = rope->inv_freq[j];
    if (!(f >= 0.0) || !std::isfinite(f)) return DFLASH_ERR_INVALID_ARG;
    p.turns[j] = turn_fraction(f);
  }
  p.q = q;
  p.k = k;
  p.v = v;
  p.ld_q = ld_q;
  p.ld_k = ld_k;
  p.ld_v = ld_v;
  p.q_norm = static_cast<const uint16_t*>(q_norm);
  p.k_norm = static_cast<const uint16_t*>(k_norm);
  p.row_req = row_req;
  p.row_pos = row_pos;
  p.q_out = static_cast<uint16_t*>(q_out);
  p.ld_qo = ld_qo;
  const size_t le = layer_elems(heads, kv) * layer;
  if (kv->dtype == 1) {
    p.pool8 = static_cast<uint8_t*>(kv->pool) + le;
    p.scales8 = kv->scales + le / d;
  } else {
    p.pool = static_cast<uint16_t*>(kv->pool) + le;
  }
  p.page_table = kv->page_table;
  p.status = static_cast<int32_t*>(ws);
  p.T = T;
  p.hq = heads->n_q_heads;
  p.hkv = heads->n_kv_heads;
  p.rot_dim = rope->rot_dim;
  p.interleaved = rope->interleaved;
  p.kv_terms = terms_of(heads);
  p.max_pages = kv->max_pages;
  p.n_pages = kv->n_pages;
  p.n_req = kv->n_rows;
  p.eps = eps;
  p.mscale = static_cast<float>(rope->mscale);
  const cudaError_t e = rope_append_launch(p, d, in_dtype == 1, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DFLASH_OK : record_cuda_error(e);
}

size_t dflash_attention_prefix_bytes(const dflash_heads* heads, int32_t batch, int32_t n,
                                     int32_t group) {
  PrefixParams p;
  if (check_heads(heads) || !prefix_sizes(heads, batch, n, group, &p)) return 0;
  return layout_prefix(&p, heads->head_dim, nullptr);
}

int dflash_attention_prefix(const dflash_heads* heads, int32_t layer, const void* q, int32_t batch,
                            int32_t n, int32_t group, int32_t causal, float scale,
                            const dflash_kv* kv, const int32_t* ctx_len,
                            const int32_t* prefix_len, void* out, float* lse, void* ws,
                            size_t ws_bytes, void* stream) {
  int rc = check_heads(heads);
  if (rc) return rc;
  if (q == nullptr || out == nullptr || ctx_len == nullptr || prefix_len == nullptr ||
      !aligned(q, 16) || !aligned(out, 16) || !aligned(ctx_len, 4) || !aligned(prefix_len, 4) ||
      !aligned(lse, 4) || (causal != 0 && causal != 1) || !(scale >= 0.f) || !std::isfinite(scale))
    return DFLASH_ERR_INVALID_ARG;
  PrefixParams p;
  if (!prefix_sizes(heads, batch, n, group, &p)) return DFLASH_ERR_INVALID_ARG;
  rc = check_cache(heads, layer, kv);
  if (rc) return rc;
  if (kv->dtype != 0 || terms_of(heads) != 1) return DFLASH_ERR_UNSUPPORTED;
  if (batch > kv->n_rows) return DFLASH_ERR_CAPACITY;
  const int d = heads->head_dim;
  // costs are counted in 32 bits, the units of an entity in 20
  for (const PrefixList& L : p.list) {
    const double units = static_cast<double>(p.hkv) *
                         (static_cast<double>(p.ng) * L.prefix_tiles + static_cast<double>(batch) * L.suffix_tiles);
    const double cost = (1 << std::max(L.prefix_cost, L.suffix_cost)) *
                        (static_cast<double>(kv->max_pages) * 16 / (1 << L.chunk_shift) + 1) + L.unit_cost;
    if (units * cost >= 1073741824.0 ||
        static_cast<double>(p.hkv) * std::max(L.prefix_tiles, L.suffix_tiles) >= 1048576.0)
      return DFLASH_ERR_UNSUPPORTED;
  }
  rc = check_ws(ws, ws_bytes, layout_prefix(&p, d, static_cast<uint8_t*>(ws)));
  if (rc) return rc;
  p.q = static_cast<const uint16_t*>(q);
  p.causal = causal;
  p.scale_log2 = static_cast<float>((scale == 0.f ? 1.0 / std::sqrt(static_cast<double>(d)) : scale) *
                                    1.44269504088896340736);
  if (!std::isfinite(p.scale_log2)) return DFLASH_ERR_INVALID_ARG;
  p.pool = static_cast<const uint16_t*>(kv->pool) + layer_elems(heads, kv) * layer;
  p.page_table = kv->page_table;
  p.max_pages = kv->max_pages;
  p.n_pages = kv->n_pages;
  p.ctx_len = ctx_len;
  p.prefix_len = prefix_len;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.status = static_cast<int32_t*>(ws);
  CUtensorMap map;
  const uint64_t layer_groups = static_cast<uint64_t>(kv->n_pages) * 2 * heads->n_kv_heads * 2;
  const uint64_t groups = layer_groups * heads->n_layers;
  if (p.list[1].workers > 0) {
    // TMA coordinates are 32 bits
    if (groups >= (1ull << 31) - 2) return DFLASH_ERR_UNSUPPORTED;
    rc = encode_kv_pages(&map, kv->pool, groups, d);
    if (rc) return rc;
  }
  const cudaError_t e = prefix_attention_launch(p, d, &map, static_cast<int>(layer_groups * layer),
                                                static_cast<int>(groups), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DFLASH_OK : record_cuda_error(e);
}

size_t dflash_sample_filtered_bytes(int32_t rows, int32_t vocab) {
  if (rows < 1 || vocab < 1 || vocab > kMaxSampleVocab) return 0;
  return kHeaderBytes;  // the status word; a row's work stays in shared memory
}

int dflash_sample_filtered(const float* logits, int64_t ld, int32_t rows, int32_t vocab,
                           const float* temperature, const int32_t* top_k, const float* top_p,
                           const float* min_p, const double* a, int32_t* token, int32_t* n_kept,
                           float* logprob, void* ws, size_t ws_bytes, void* stream) {
  if (logits == nullptr || temperature == nullptr || a == nullptr || token == nullptr || rows < 1 ||
      vocab < 1 || ld < vocab || !aligned(logits, 4) || !aligned(temperature, 4) ||
      !aligned(top_k, 4) || !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(a, 8) ||
      !aligned(token, 4) || !aligned(n_kept, 4) || !aligned(logprob, 4))
    return DFLASH_ERR_INVALID_ARG;
  if (vocab > kMaxSampleVocab || rows > (1 << 24)) return DFLASH_ERR_UNSUPPORTED;
  const int rc = check_ws(ws, ws_bytes, dflash_sample_filtered_bytes(rows, vocab));
  if (rc) return rc;
  SampleFilteredParams p;
  p.logits = logits;
  p.ld = ld;
  p.rows = rows;
  p.vocab = vocab;
  p.temperature = temperature;
  p.top_k = top_k;
  p.top_p = top_p;
  p.min_p = min_p;
  p.a = a;
  p.token = token;
  p.n_kept = n_kept;
  p.logprob = logprob;
  p.status = static_cast<int32_t*>(ws);
  const cudaError_t e = sample_filtered_launch(p, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DFLASH_OK : record_cuda_error(e);
}

}  // extern "C"
