// The C ABI of the low-bit key/value cache (include/gptq_cache.h): argument checks and dispatch.
#include <climits>

#include "gptq_cache.h"
#include "kernels.h"

using namespace gptq;

static bool valid_dtype(int dt) { return dt == GPTQ_F32 || dt == GPTQ_F16 || dt == GPTQ_BF16; }
static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

static bool valid_cfg(const gptq_cache_config* cfg) {
  if (!cfg || (cfg->sym != 0 && cfg->sym != 1) || cfg->group_size < 0) return false;
  if (cfg->kind == GPTQ_CACHE_MX) return cfg->bits == 4;
  return cfg->kind == GPTQ_CACHE_GRID && (cfg->bits == 4 || cfg->bits == 8);
}

static gptq_status run(bool write, const void* K, const void* V, int dtype, int64_t tokens,
                       int64_t k_ld_token, int64_t k_ld_head, int64_t v_ld_token,
                       int64_t v_ld_head, const gptq_cache_config* cfg, const gptq_cache* c,
                       const gptq_cache_rows* r, int32_t* dev_status, void* stream) {
  if (!valid_cfg(cfg) || !c || !r || !valid_dtype(dtype)) return GPTQ_ERR_INVALID_ARG;
  if (tokens < 0 || tokens > INT_MAX || r->seqs < 0 || r->seqs >= INT_MAX) return GPTQ_ERR_INVALID_ARG;
  if (c->pages < 0 || c->pages > INT_MAX || c->page_size < 1 || c->page_size > INT_MAX ||
      c->heads < 1 || c->heads > INT_MAX || c->dim < 1 || c->dim > INT_MAX)
    return GPTQ_ERR_INVALID_ARG;
  if (r->width < 0 || r->width > INT_MAX || r->table_ld < r->width) return GPTQ_ERR_INVALID_ARG;
  int words, groups;
  if (!cache_shape(*cfg, c->dim, words, groups)) return GPTQ_ERR_UNSUPPORTED;
  if (tokens == 0 || r->seqs == 0) return GPTQ_OK;
  if (!K || !V || !r->cu || !r->start || (r->width > 0 && !r->table)) return GPTQ_ERR_INVALID_ARG;
  if (c->pages > 0 && (!c->k_codes || !c->v_codes || !c->k_grids || !c->v_grids))
    return GPTQ_ERR_INVALID_ARG;
  if (!aligned16(c->k_codes) || !aligned16(c->v_codes) || !aligned16(c->k_grids) ||
      !aligned16(c->v_grids))
    return GPTQ_ERR_INVALID_ARG;
  return cache_run(as_stream(stream), write, K, V, dtype, tokens, k_ld_token, k_ld_head,
                   v_ld_token, v_ld_head, *cfg, *c, *r, dev_status);
}

extern "C" {

size_t gptq_cache_words(const gptq_cache_config* cfg, int64_t dim) {
  int words, groups;
  return valid_cfg(cfg) && cache_shape(*cfg, dim, words, groups) ? size_t(words) : 0;
}

size_t gptq_cache_grid_bytes(const gptq_cache_config* cfg, int64_t dim) {
  int words, groups;
  if (!valid_cfg(cfg) || !cache_shape(*cfg, dim, words, groups)) return 0;
  return size_t(groups) * (cfg->kind == GPTQ_CACHE_MX ? 1 : 8);
}

gptq_status gptq_cache_write(const void* K, const void* V, int dtype, int64_t tokens,
                             int64_t k_ld_token, int64_t k_ld_head, int64_t v_ld_token,
                             int64_t v_ld_head, const gptq_cache_config* cfg,
                             const gptq_cache* cache, const gptq_cache_rows* rows,
                             int32_t* dev_status, void* stream) {
  CallRange range_("gptq_cache_write");
  return run(true, K, V, dtype, tokens, k_ld_token, k_ld_head, v_ld_token, v_ld_head, cfg, cache,
             rows, dev_status, stream);
}

gptq_status gptq_cache_read(const gptq_cache_config* cfg, const gptq_cache* cache,
                            const gptq_cache_rows* rows, void* K, void* V, int dtype,
                            int64_t tokens, int64_t k_ld_token, int64_t k_ld_head,
                            int64_t v_ld_token, int64_t v_ld_head, int32_t* dev_status,
                            void* stream) {
  CallRange range_("gptq_cache_read");
  return run(false, K, V, dtype, tokens, k_ld_token, k_ld_head, v_ld_token, v_ld_head, cfg, cache,
             rows, dev_status, stream);
}

}  // extern "C"
