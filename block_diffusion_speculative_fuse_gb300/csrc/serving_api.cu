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

// Workspace of the chunk attention: header, the workers' records, the pieces'
// partial results.  Returns the bytes; fills the pointers when base is set.
size_t layout_chunk(ChunkParams* p, int d, uint8_t* base) {
  size_t off = kHeaderBytes;
  auto take = [&](size_t bytes) {
    uint8_t* q = base == nullptr ? nullptr : base + off;
    off = al256(off + bytes);
    return q;
  };
  const size_t ranges = kChunkWorkers * static_cast<size_t>(p->phases);
  const size_t rows = 2 * ranges * p->slot_rows;
  p->records = take(ranges * 32);
  p->part_ml = reinterpret_cast<float*>(take(rows * 2 * sizeof(float)));
  p->part_o = reinterpret_cast<float*>(take(rows * d * sizeof(float)));
  return off;
}

bool chunk_sizes(const dflash_heads* h, int32_t batch, int32_t T, ChunkParams* p) {
  if (batch < 1 || T < 1) return false;
  std::memset(p, 0, sizeof(*p));
  p->batch = batch;
  p->T = T;
  p->hq = h->n_q_heads;
  p->hkv = h->n_kv_heads;
  p->G = p->hq / p->hkv;
  p->tokens = 128 / p->G;
  p->slot_rows = T <= p->tokens ? T * p->G : 256;
  // few rows read the keys few times again, and need no workspace for many phases
  p->phases = 1;
  while (p->phases < kChunkPhases && p->phases * 8 * p->tokens <= T) p->phases *= 2;
  p->halves = h->head_dim / 64;
  return true;
}

// The softmax's scale in base 2: 0 stands for 1 / sqrt(d).
bool scale_of(float scale, int d, float* scale_log2) {
  if (!(scale >= 0.f) || !std::isfinite(scale)) return false;
  *scale_log2 = static_cast<float>((scale == 0.f ? 1.0 / std::sqrt(static_cast<double>(d)) : scale) *
                                   1.44269504088896340736);
  return std::isfinite(*scale_log2);
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

size_t dflash_attention_chunk_bytes(const dflash_heads* heads, int32_t batch, int32_t T) {
  ChunkParams p;
  if (check_heads(heads) || !chunk_sizes(heads, batch, T, &p)) return 0;
  return layout_chunk(&p, heads->head_dim, nullptr);
}

int dflash_attention_chunk(const dflash_heads* heads, int32_t layer, const void* q, int64_t ld_q,
                           const int32_t* row_start, int32_t batch, int32_t T, int32_t causal,
                           float scale, const dflash_kv* kv, const int32_t* ctx_len, void* out,
                           int64_t ld_out, float* lse, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_heads(heads);
  if (rc) return rc;
  ChunkParams p;
  if (q == nullptr || out == nullptr || row_start == nullptr || ctx_len == nullptr || !aligned(q, 16) ||
      !aligned(out, 16) || !aligned(row_start, 4) || !aligned(ctx_len, 4) || !aligned(lse, 4) ||
      (causal != 0 && causal != 1) || !chunk_sizes(heads, batch, T, &p))
    return DFLASH_ERR_INVALID_ARG;
  const int d = heads->head_dim;
  const int64_t row = static_cast<int64_t>(p.hq) * d;
  if (q == out || ld_q < row || ld_out < row || ld_q % 8 || ld_out % 8 || !scale_of(scale, d, &p.scale_log2))
    return DFLASH_ERR_INVALID_ARG;
  rc = check_cache(heads, layer, kv);
  if (rc) return rc;
  if (kv->dtype != 0 || terms_of(heads) != 1) return DFLASH_ERR_UNSUPPORTED;
  if (batch > kv->n_rows) return DFLASH_ERR_CAPACITY;
  // TMA coordinates are 32 bits, a map's strides 40
  const uint64_t layer_groups = static_cast<uint64_t>(kv->n_pages) * 2 * heads->n_kv_heads * 2;
  const uint64_t groups = layer_groups * heads->n_layers;
  if (groups >= (1ull << 31) - 2 || T > (1 << 30) || ld_q >= (1ll << 38)) return DFLASH_ERR_UNSUPPORTED;
  p.max_pages = kv->max_pages;
  if (!attention_chunk_fits(p)) return DFLASH_ERR_UNSUPPORTED;
  rc = check_ws(ws, ws_bytes, layout_chunk(&p, d, static_cast<uint8_t*>(ws)));
  if (rc) return rc;
  p.row_start = row_start;
  p.ctx_len = ctx_len;
  p.page_table = kv->page_table;
  p.causal = causal;
  p.n_pages = kv->n_pages;
  // A unit's last piece can join them all where units have one tile and, on average, few
  // rows; that saves a kernel, but one CTA reads all of a unit's partials.  With and
  // without: a row of 4096 keys 18.6 and 23.3 us, of 30000 35.0 and 41.9, 8 rows 23.3 and
  // 23.8, 16 rows 31.7 and 24.5, 32 rows of 16000 keys 50.9 and 33.2.
  p.fused = T <= p.tokens && T <= 8 * static_cast<int64_t>(batch) &&
            static_cast<int64_t>(batch) * p.hkv <= (32 * 1024 - 256) / 4;
  p.out = static_cast<uint16_t*>(out);
  p.ld_out = ld_out;
  p.wide = aligned(out, 32) && ld_out % 16 == 0;
  p.lse = lse;
  p.status = static_cast<int32_t*>(ws);
  CUtensorMap kv_map, q_map;
  rc = encode_kv_pages(&kv_map, kv->pool, groups, d);
  if (!rc) rc = encode_q_rows(&q_map, q, ld_q, T, p.hq, p.G, p.tokens, d);
  if (rc) return rc;
  const cudaError_t e = attention_chunk_launch(p, d, kv_map, q_map, static_cast<int>(layer_groups * layer),
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

size_t dflash_attention_mass_bytes(const dflash_heads* heads, int32_t batch, int32_t T) {
  if (check_heads(heads) || batch < 1 || batch > kMaxMassBatch || T < 1) return 0;
  return kHeaderBytes;  // the status word
}

int dflash_attention_mass(const dflash_heads* heads, int32_t layer, const void* q, int64_t ld_q,
                          const int32_t* row_start, int32_t batch, int32_t T, int32_t last, int32_t causal,
                          float scale, const dflash_kv* kv, const int32_t* ctx_len, const float* lse,
                          float* mass, int64_t ld_mass, int32_t accumulate, void* ws, size_t ws_bytes,
                          void* stream) {
  int rc = check_heads(heads);
  if (rc) return rc;
  MassParams p;
  std::memset(&p, 0, sizeof(p));
  const int d = heads->head_dim;
  if (q == nullptr || row_start == nullptr || ctx_len == nullptr || lse == nullptr || mass == nullptr ||
      !aligned(q, 16) || !aligned(row_start, 4) || !aligned(ctx_len, 4) || !aligned(lse, 4) || !aligned(mass, 4) ||
      batch < 1 || T < 1 || last < 0 || (causal != 0 && causal != 1) || (accumulate != 0 && accumulate != 1) ||
      ld_mass < 1 || ld_q < static_cast<int64_t>(heads->n_q_heads) * d || ld_q % 8 || !scale_of(scale, d, &p.scale_log2))
    return DFLASH_ERR_INVALID_ARG;
  rc = check_cache(heads, layer, kv);
  if (rc) return rc;
  if (kv->dtype != 0 || terms_of(heads) != 1 || batch > kMaxMassBatch) return DFLASH_ERR_UNSUPPORTED;
  if (batch > kv->n_rows) return DFLASH_ERR_CAPACITY;
  const uint64_t layer_groups = static_cast<uint64_t>(kv->n_pages) * 2 * heads->n_kv_heads * 2;
  const uint64_t groups = layer_groups * heads->n_layers;
  // TMA coordinates are 32 bits, a map's strides 40; units are counted in 31 bits
  if (groups >= (1ull << 31) - 2 || T > (1 << 30) || ld_q >= (1ll << 38) ||
      static_cast<double>(batch) * heads->n_kv_heads * (kv->max_pages / 16 + 1) >= 1073741824.0)
    return DFLASH_ERR_UNSUPPORTED;
  rc = check_ws(ws, ws_bytes, kHeaderBytes);
  if (rc) return rc;
  p.row_start = row_start;
  p.ctx_len = ctx_len;
  p.page_table = kv->page_table;
  p.batch = batch;
  p.T = T;
  p.hq = heads->n_q_heads;
  p.hkv = heads->n_kv_heads;
  p.G = p.hq / p.hkv;
  p.tokens = 128 / p.G;
  p.last = last;
  p.few = (last > 0 && last <= 2 * p.tokens) || T <= 2 * p.tokens;
  p.causal = causal;
  p.max_pages = kv->max_pages;
  p.n_pages = kv->n_pages;
  p.accumulate = accumulate;
  p.lse = lse;
  p.mass = mass;
  p.ld_mass = ld_mass;
  p.status = static_cast<int32_t*>(ws);
  CUtensorMap kv_map, q_map;
  rc = encode_kv_pages(&kv_map, kv->pool, groups, d);
  if (!rc) rc = encode_q_rows(&q_map, q, ld_q, T, p.hq, p.G, p.tokens, d);
  if (rc) return rc;
  const cudaError_t e = attention_mass_launch(p, d, kv_map, q_map, static_cast<int>(layer_groups * layer),
                                              static_cast<int>(groups), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DFLASH_OK : record_cuda_error(e);
}

size_t dflash_kv_evict_bytes(const dflash_heads* heads, int32_t batch, int32_t dst_pages) {
  if (check_heads(heads) || heads->n_kv_heads > 65535 || batch < 1 || batch > 65535 || dst_pages < 1) return 0;
  return kHeaderBytes + 256 + al256(static_cast<size_t>(dst_pages) * 4);
}

int dflash_kv_evict(const dflash_heads* heads, int32_t layer, const dflash_kv* src, const dflash_kv* dst,
                    int32_t batch, const int32_t* ctx_len, const int32_t* keep, int32_t sink, int32_t recent,
                    const float* mass, int64_t ld_mass, int32_t* kept, int64_t ld_kept, int32_t* new_len,
                    float* mass_out, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_heads(heads);
  if (!rc) rc = check_cache(heads, layer, src);
  if (!rc) rc = check_cache(heads, layer, dst);
  if (rc) return rc;
  if (ctx_len == nullptr || keep == nullptr || mass == nullptr || kept == nullptr || batch < 1 || sink < 0 ||
      recent < 0 || ld_mass < 1 || ld_kept < 1 || mass_out == mass || new_len == ctx_len || new_len == keep ||
      !aligned(ctx_len, 4) || !aligned(keep, 4) || !aligned(mass, 4) || !aligned(kept, 4) || !aligned(new_len, 4) || !aligned(mass_out, 4) ||
      src->dtype != dst->dtype)
    return DFLASH_ERR_INVALID_ARG;
  // (heads and requests are rows and layers of the copy's grid)
  if (batch > 65535 || heads->n_kv_heads > 65535 ||
      static_cast<int64_t>(batch) * heads->n_kv_heads > (1 << 26) || ld_mass > (1 << 30) || ld_kept > (1 << 30))
    return DFLASH_ERR_UNSUPPORTED;
  if (batch > src->n_rows || batch > dst->n_rows) return DFLASH_ERR_CAPACITY;
  const int elem = src->dtype == 1 ? 1 : 2, d = heads->head_dim;
  const size_t src_layer = layer_elems(heads, src) * elem, dst_layer = layer_elems(heads, dst) * elem;
  // two caches are the same pool or apart
  const bool same = src->pool == dst->pool;
  auto meet = [&](const void* x, size_t x_layer, const void* y, size_t y_layer) {
    const auto a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
    return a < b + y_layer * heads->n_layers && b < a + x_layer * heads->n_layers;
  };
  if (same ? src->n_pages != dst->n_pages || src->scales != dst->scales
           : meet(src->pool, src_layer, dst->pool, dst_layer) ||
                 (elem == 1 && meet(src->scales, src_layer / d * 4, dst->scales, dst_layer / d * 4)))
    return DFLASH_ERR_INVALID_ARG;
  rc = check_ws(ws, ws_bytes, dflash_kv_evict_bytes(heads, batch, dst->n_pages));
  if (rc) return rc;
  EvictParams p;
  std::memset(&p, 0, sizeof(p));
  p.src_pool = static_cast<const uint8_t*>(src->pool) + src_layer * layer;
  p.dst_pool = static_cast<uint8_t*>(dst->pool) + dst_layer * layer;
  if (src->dtype == 1) {
    p.src_scales = src->scales + layer_elems(heads, src) / d * layer;
    p.dst_scales = dst->scales + layer_elems(heads, dst) / d * layer;
  }
  p.src_table = src->page_table;
  p.dst_table = dst->page_table;
  p.src_pages = src->n_pages;
  p.src_max_pages = src->max_pages;
  p.dst_pages = dst->n_pages;
  p.dst_max_pages = dst->max_pages;
  p.same_pool = same;
  p.batch = batch;
  p.hkv = heads->n_kv_heads;
  p.planes = 2 * terms_of(heads);
  p.ctx_len = ctx_len;
  p.keep = keep;
  p.sink = sink;
  p.recent = recent;
  p.mass = mass;
  p.mass_out = mass_out;
  p.ld_mass = ld_mass;
  p.ld_kept = ld_kept;
  p.kept = kept;
  p.new_len = new_len;
  uint8_t* w = static_cast<uint8_t*>(ws) + kHeaderBytes;
  p.conflict = reinterpret_cast<int*>(w);
  p.owner = reinterpret_cast<unsigned*>(w + 256);
  p.status = static_cast<int32_t*>(ws);
  const cudaError_t e = kv_evict_launch(p, d * elem, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DFLASH_OK : record_cuda_error(e);
}

size_t dflash_score_tokens_bytes(int32_t rows, int32_t vocab, int32_t n_top) {
  if (rows < 1 || vocab < 1 || vocab > kMaxSampleVocab || n_top < 0 || n_top > kMaxScoreTop) return 0;
  return kHeaderBytes;  // the status word; a row's work stays on chip
}

int dflash_score_tokens(const void* logits, int64_t ld, int32_t rows, int32_t vocab, int32_t in_dtype,
                        const float* temperature, const int32_t* ids, float* logprob, int32_t* rank,
                        float* entropy, int32_t n_top, int32_t* top_id, float* top_logprob, void* ws,
                        size_t ws_bytes, void* stream) {
  if (logits == nullptr || rows < 1 || vocab < 1 || ld < vocab || (in_dtype != 0 && in_dtype != 1) ||
      n_top < 0 || (n_top > 0 && (top_id == nullptr || top_logprob == nullptr)) ||
      (ids == nullptr && (logprob != nullptr || rank != nullptr)) ||
      !aligned(logits, in_dtype == 1 ? 4 : 2) || !aligned(temperature, 4) || !aligned(ids, 4) ||
      !aligned(logprob, 4) || !aligned(rank, 4) || !aligned(entropy, 4) || !aligned(top_id, 4) ||
      !aligned(top_logprob, 4))
    return DFLASH_ERR_INVALID_ARG;
  if (vocab > kMaxSampleVocab || rows > (1 << 24) || n_top > kMaxScoreTop) return DFLASH_ERR_UNSUPPORTED;
  const int rc = check_ws(ws, ws_bytes, kHeaderBytes);
  if (rc) return rc;
  ScoreParams p;
  p.logits = logits;
  p.ld = ld;
  p.rows = rows;
  p.vocab = vocab;
  p.n_top = n_top;
  p.temperature = temperature;
  p.ids = ids;
  p.logprob = logprob;
  p.rank = rank;
  p.entropy = entropy;
  p.top_id = top_id;
  p.top_logprob = top_logprob;
  p.status = static_cast<int32_t*>(ws);
  const cudaError_t e = score_tokens_launch(p, in_dtype == 0, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DFLASH_OK : record_cuda_error(e);
}

}  // extern "C"
