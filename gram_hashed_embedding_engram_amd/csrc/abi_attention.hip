// The C ABI of the attention sub-layer (include/engram.h): host-side checks
// and dispatch.  Every check runs before any launch.
#include <cmath>

#include "attention.h"

using namespace engram;

#define CHECK(cond, code, ...)                                                               \
    do {                                                                                     \
        if (!(cond))                                                                         \
            return fail(code, __VA_ARGS__);                                                  \
    } while (0)

namespace {

// tokens a call: the grids lay a workgroup's threads over tokens in 32 bits
constexpr int64_t kMaxTokens = (int64_t)1 << 22;
constexpr int32_t kMaxSequences = 1 << 16;
constexpr int32_t kMaxHeads = 1024;

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

// Whether an input and an output share memory: several workgroups read what
// one of them would already have written.
bool overlap(const void *in, uint64_t in_bytes, const void *out, uint64_t out_bytes)
{
    const uintptr_t a = (uintptr_t)in, b = (uintptr_t)out;
    return a < b ? b - a < in_bytes : a - b < out_bytes;
}

Launch on(void *stream)
{
    Launch l;
    l.stream = as_stream(stream);
    return l;
}

int32_t check_cache(const engram_cache *c, const char *who)
{
    CHECK(c, ENGRAM_E_ARG, "engram %s: NULL cache", who);
    CHECK(c->head_dim == 64 || c->head_dim == 128 || c->head_dim == 256, ENGRAM_E_UNSUPPORTED,
          "engram %s: head_dim %d (64, 128 or 256)", who, c->head_dim);
    CHECK(c->kv_heads >= 1 && c->kv_heads <= kMaxHeads, ENGRAM_E_UNSUPPORTED,
          "engram %s: %d key heads, 1 to %d supported", who, c->kv_heads, kMaxHeads);
    CHECK(c->n_pages >= 1 && c->n_pages < ((int64_t)1 << 31), ENGRAM_E_ARG,
          "engram %s: a cache of %lld pages", who, (long long)c->n_pages);
    CHECK(c->d_k && c->d_v && c->d_k_scales && c->d_v_scales, ENGRAM_E_ARG,
          "engram %s: NULL pointer in the cache", who);
    CHECK(aligned(c->d_k, 16) && aligned(c->d_v, 16) && aligned(c->d_k_scales, 4) &&
              aligned(c->d_v_scales, 4),
          ENGRAM_E_ARG, "engram %s: the cache's codes must be 16-byte, its scales 4-byte aligned",
          who);
    return ENGRAM_OK;
}

int32_t check_seqs(const engram_seqs *s, int64_t T, const char *who, Seqs *out)
{
    CHECK(s, ENGRAM_E_ARG, "engram %s: NULL sequences", who);
    CHECK(T >= 0, ENGRAM_E_ARG, "engram %s: T = %lld", who, (long long)T);
    CHECK(T <= kMaxTokens, ENGRAM_E_RANGE, "engram %s: %lld tokens exceed %lld", who, (long long)T,
          (long long)kMaxTokens);
    CHECK(s->batch >= 1 && s->batch <= kMaxSequences, ENGRAM_E_ARG,
          "engram %s: %d sequences, 1 to %d supported", who, s->batch, kMaxSequences);
    CHECK(s->max_pages >= 1 && s->max_pages < (1 << 25), ENGRAM_E_ARG,
          "engram %s: %d pages a sequence", who, s->max_pages);
    CHECK(s->d_pages && s->d_start, ENGRAM_E_ARG, "engram %s: NULL pages or starts", who);
    CHECK(aligned(s->d_pages, 4) && aligned(s->d_start, 4) && aligned(s->d_cu, 4) &&
              aligned(s->d_err, 4),
          ENGRAM_E_ARG, "engram %s: pages, starts, token bounds and err must be 4-byte aligned",
          who);
    CHECK(s->d_cu || T % s->batch == 0, ENGRAM_E_ARG,
          "engram %s: %lld tokens do not divide among %d sequences (pass their bounds)", who,
          (long long)T, s->batch);
    *out = Seqs{s->d_pages, s->d_start, s->d_cu,   s->d_err,
                s->batch,   s->max_pages, (int32_t)T, s->d_cu ? 0 : (int32_t)(T / s->batch)};
    return ENGRAM_OK;
}

int32_t check_heads(const uint16_t *p, int64_t token, int64_t head, int32_t heads, int64_t T,
                    int32_t d, const char *who, const char *what)
{
    CHECK(p, ENGRAM_E_ARG, "engram %s: NULL %s", who, what);
    CHECK(aligned(p, 16), ENGRAM_E_ARG, "engram %s: %s must be 16-byte aligned", who, what);
    CHECK(token % 8 == 0 && head % 8 == 0 && token >= 0 && head >= 0 && token < ((int64_t)1 << 40) &&
              head < ((int64_t)1 << 40),
          ENGRAM_E_UNSUPPORTED,
          "engram %s: strides %lld and %lld of %s must be multiples of 8 values", who,
          (long long)token, (long long)head, what);
    CHECK((heads == 1 || head >= d) && (T == 1 || token >= d), ENGRAM_E_ARG,
          "engram %s: strides %lld and %lld of %s are below head_dim %d", who, (long long)token,
          (long long)head, what, d);
    return ENGRAM_OK;
}

}  // namespace

extern "C" {

int32_t engram_add_norm(const uint16_t *d_x, const void *d_res, int32_t res_bf16,
                        const uint16_t *d_w, float eps, void *d_sum, uint8_t *d_codes,
                        uint8_t *d_scales, int64_t rows, int64_t dim, void *stream)
{
    CHECK(rows >= 0, ENGRAM_E_ARG, "engram add_norm: %lld rows", (long long)rows);
    CHECK(rows < ((int64_t)1 << 31), ENGRAM_E_RANGE, "engram add_norm: %lld rows exceed 2^31-1",
          (long long)rows);
    CHECK(dim >= ENGRAM_NORM_GROUP && dim % ENGRAM_NORM_GROUP == 0 && dim <= 65536,
          ENGRAM_E_UNSUPPORTED, "engram add_norm: dim = %lld must be a multiple of 32 up to 65536",
          (long long)dim);
    CHECK(std::isfinite(eps) && eps >= 0.0f, ENGRAM_E_ARG, "engram add_norm: eps = %g",
          (double)eps);
    if (rows == 0)
        return ENGRAM_OK;
    CHECK(d_res && d_w && d_sum && d_codes && d_scales, ENGRAM_E_ARG,
          "engram add_norm: NULL pointer");
    CHECK(aligned(d_x, 16) && aligned(d_res, 16) && aligned(d_w, 16) && aligned(d_sum, 16) &&
              aligned(d_codes, 8),
          ENGRAM_E_ARG,
          "engram add_norm: x, res, w and sum must be 16-byte, codes 8-byte aligned");
    return launch_add_norm(d_x, d_res, res_bf16 != 0, d_w, eps, d_sum, d_codes, d_scales, rows,
                           dim, on(stream));
}

int32_t engram_project_w4(const void *d_x, const uint8_t *d_x_scales, const uint8_t *d_w,
                          const uint8_t *d_w_scales, uint16_t *d_y, int64_t T, int64_t K,
                          int64_t N, void *stream)
{
    CHECK(T >= 0, ENGRAM_E_ARG, "engram project_w4: T = %lld", (long long)T);
    CHECK(T <= kMaxTokens, ENGRAM_E_RANGE, "engram project_w4: %lld tokens exceed %lld",
          (long long)T, (long long)kMaxTokens);
    CHECK(K >= 128 && K % 128 == 0 && K <= (1 << 20), ENGRAM_E_UNSUPPORTED,
          "engram project_w4: K = %lld must be a positive multiple of 128 up to 2^20",
          (long long)K);
    CHECK(N >= 16 && N % 16 == 0 && N <= (1 << 24), ENGRAM_E_UNSUPPORTED,
          "engram project_w4: N = %lld must be a positive multiple of 16 up to 2^24",
          (long long)N);
    if (T == 0)
        return ENGRAM_OK;
    CHECK(d_x && d_w && d_w_scales && d_y, ENGRAM_E_ARG, "engram project_w4: NULL pointer");
    CHECK(aligned(d_x, 16) && aligned(d_w, 16) && aligned(d_x_scales, 4) &&
              aligned(d_w_scales, 4) && aligned(d_y, 8),
          ENGRAM_E_ARG,
          "engram project_w4: x and w must be 16-byte, y 8-byte, scales 4-byte aligned");
    CHECK(!overlap(d_x, (uint64_t)(T * K) * (d_x_scales ? 1 : 2), d_y, (uint64_t)(T * N) * 2),
          ENGRAM_E_ARG, "engram project_w4: y overlaps x");
    return launch_w4(d_x, d_x_scales, d_w, d_w_scales, d_y, T, K, N, on(stream));
}

int32_t engram_cache_append(const engram_cache *cache, const engram_seqs *seqs,
                            const uint16_t *d_k, int64_t k_token_stride, int64_t k_head_stride,
                            const uint16_t *d_v, int64_t v_token_stride, int64_t v_head_stride,
                            const uint16_t *d_q, int64_t q_token_stride, int64_t q_head_stride,
                            uint16_t *d_q_out, int32_t q_heads, const float *d_freq, int32_t rot,
                            int32_t halves, int64_t T, void *stream)
{
    int32_t rc = check_cache(cache, "cache_append");
    Seqs s;
    if (rc == ENGRAM_OK)
        rc = check_seqs(seqs, T, "cache_append", &s);
    if (rc != ENGRAM_OK)
        return rc;
    CHECK(q_heads >= 0 && q_heads <= kMaxHeads, ENGRAM_E_ARG,
          "engram cache_append: %d query heads, 0 to %d supported", q_heads, kMaxHeads);
    CHECK(rot >= 0 && rot % 16 == 0 && rot <= cache->head_dim, ENGRAM_E_UNSUPPORTED,
          "engram cache_append: %d rotated values must be a multiple of 16 up to head_dim %d", rot,
          cache->head_dim);
    if (T == 0)
        return ENGRAM_OK;
    CHECK(rot == 0 || (d_freq && aligned(d_freq, 4)), ENGRAM_E_ARG,
          "engram cache_append: NULL or unaligned freq");
    rc = check_heads(d_k, k_token_stride, k_head_stride, cache->kv_heads, T, cache->head_dim,
                     "cache_append", "k");
    if (rc == ENGRAM_OK)
        rc = check_heads(d_v, v_token_stride, v_head_stride, cache->kv_heads, T, cache->head_dim,
                         "cache_append", "v");
    if (rc == ENGRAM_OK && q_heads > 0)
        rc = check_heads(d_q, q_token_stride, q_head_stride, q_heads, T, cache->head_dim,
                         "cache_append", "q");
    if (rc != ENGRAM_OK)
        return rc;
    CHECK(q_heads == 0 || (d_q_out && aligned(d_q_out, 16)), ENGRAM_E_ARG,
          "engram cache_append: NULL or unaligned q_out (16 bytes)");
    return launch_append(*cache, s, Heads{d_k, k_token_stride, k_head_stride},
                         Heads{d_v, v_token_stride, v_head_stride},
                         Heads{d_q, q_token_stride, q_head_stride}, d_q_out, q_heads,
                         Rotation{d_freq, rot, halves != 0}, on(stream));
}

size_t engram_cache_attend_bytes(const engram_cache *cache, const engram_seqs *seqs,
                                 int32_t q_heads, int64_t T)
{
    Seqs s;
    if (check_cache(cache, "cache_attend") != ENGRAM_OK ||
        check_seqs(seqs, T, "cache_attend", &s) != ENGRAM_OK || q_heads < cache->kv_heads ||
        q_heads % cache->kv_heads != 0 || q_heads > kMaxHeads || T == 0)
        return 0;
    return attend_bytes(*cache, s, q_heads);
}

int32_t engram_cache_attend(const engram_cache *cache, const engram_seqs *seqs,
                            const uint16_t *d_q, int64_t q_token_stride, int64_t q_head_stride,
                            uint16_t *d_out, int32_t q_heads, int64_t T, float scale,
                            int64_t window, void *d_ws, size_t ws_bytes, void *stream)
{
    int32_t rc = check_cache(cache, "cache_attend");
    Seqs s;
    if (rc == ENGRAM_OK)
        rc = check_seqs(seqs, T, "cache_attend", &s);
    if (rc != ENGRAM_OK)
        return rc;
    CHECK(q_heads >= cache->kv_heads && q_heads % cache->kv_heads == 0 && q_heads <= kMaxHeads,
          ENGRAM_E_UNSUPPORTED,
          "engram cache_attend: %d query heads must be a multiple of the %d key heads, up to %d",
          q_heads, cache->kv_heads, kMaxHeads);
    CHECK(std::isfinite(scale), ENGRAM_E_ARG, "engram cache_attend: scale = %g", (double)scale);
    CHECK(window >= 0, ENGRAM_E_ARG, "engram cache_attend: window = %lld", (long long)window);
    if (T == 0)
        return ENGRAM_OK;
    rc = check_heads(d_q, q_token_stride, q_head_stride, q_heads, T, cache->head_dim,
                     "cache_attend", "q");
    if (rc != ENGRAM_OK)
        return rc;
    CHECK(d_out && aligned(d_out, 8), ENGRAM_E_ARG,
          "engram cache_attend: NULL or unaligned out (8 bytes)");
    const size_t need = attend_bytes(*cache, s, q_heads);
    CHECK(ws_bytes >= need, ENGRAM_E_RANGE,
          "engram cache_attend: a workspace of %zu bytes, %zu needed", ws_bytes, need);
    CHECK(need == 0 || (d_ws && aligned(d_ws, 256)), ENGRAM_E_ARG,
          "engram cache_attend: NULL or unaligned workspace (256 bytes)");
    const uint64_t q_values = (uint64_t)(T - 1) * (uint64_t)q_token_stride +
                              (uint64_t)(q_heads - 1) * (uint64_t)q_head_stride + cache->head_dim;
    CHECK(!overlap(d_q, 2 * q_values, d_out, (uint64_t)T * q_heads * cache->head_dim * 2),
          ENGRAM_E_ARG, "engram cache_attend: out overlaps q");
    return launch_attend(*cache, s, Heads{d_q, q_token_stride, q_head_stride}, d_out, q_heads,
                         scale, window, d_ws, on(stream));
}

}  // extern "C"
