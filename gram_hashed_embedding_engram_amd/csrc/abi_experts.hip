// The C ABI of the experts' sub-layer (include/engram.h): host-side checks and
// dispatch.  Every check runs before any launch.
#include <cmath>

#include "experts.h"

using namespace engram;

#define CHECK(cond, code, ...)                                                               \
    do {                                                                                     \
        if (!(cond))                                                                         \
            return fail(code, __VA_ARGS__);                                                  \
    } while (0)

namespace {

constexpr int64_t kMaxTokens = (int64_t)1 << 22;
constexpr int64_t kMaxSlots = (int64_t)1 << 24;

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

// What a call reads or writes; none where p is NULL.
struct Bytes {
    const char *name;
    const void *p;
    uint64_t n;
};

bool overlap(const Bytes &a, const Bytes &b)
{
    const uintptr_t i = (uintptr_t)a.p, j = (uintptr_t)b.p;
    return a.p && b.p && a.n && b.n && (i < j ? j - i < a.n : i - j < b.n);
}

// What a call writes overlaps nothing else of it.
template <size_t W, size_t R>
int32_t check_apart(const char *who, const Bytes (&writes)[W], const Bytes (&reads)[R])
{
    for (size_t i = 0; i < W; i++) {
        for (const Bytes &r : reads)
            CHECK(!overlap(writes[i], r), ENGRAM_E_ARG, "engram %s: the %s overlaps the %s", who,
                  writes[i].name, r.name);
        for (size_t j = i + 1; j < W; j++)
            CHECK(!overlap(writes[i], writes[j]), ENGRAM_E_ARG, "engram %s: the %s overlaps the %s",
                  who, writes[i].name, writes[j].name);
    }
    return ENGRAM_OK;
}

Launch on(void *stream)
{
    Launch l;
    l.stream = as_stream(stream);
    return l;
}

uint64_t scale_bytes(int64_t rows, int64_t K, bool f32)
{
    return (uint64_t)rows * (uint64_t)(f32 ? K / kF8Block * 4 : K / ENGRAM_NORM_GROUP);
}

uint64_t block_bytes(int64_t matrices, int64_t N, int64_t K)
{
    return (uint64_t)matrices * (uint64_t)((N + kF8Block - 1) / kF8Block) * (uint64_t)(K / kF8Block) * 4;
}

uint64_t slot_bytes(const engram_routes *r) { return (uint64_t)r->tokens * (uint64_t)r->chosen * 4; }
uint64_t offset_bytes(const engram_routes *r) { return 4 * ((uint64_t)r->experts + 1); }

int32_t check_routes(const engram_routes *r, const char *who)
{
    CHECK(r, ENGRAM_E_ARG, "engram %s: NULL routes", who);
    CHECK(r->tokens >= 0, ENGRAM_E_ARG, "engram %s: %lld tokens", who, (long long)r->tokens);
    CHECK(r->tokens <= kMaxTokens, ENGRAM_E_RANGE, "engram %s: %lld tokens exceed %lld", who,
          (long long)r->tokens, (long long)kMaxTokens);
    CHECK(r->experts >= 1 && r->experts <= kMaxExperts, ENGRAM_E_UNSUPPORTED,
          "engram %s: %d experts, 1 to %d supported", who, r->experts, kMaxExperts);
    CHECK(r->chosen >= 1 && r->chosen <= r->experts && r->chosen <= kMaxChosen,
          ENGRAM_E_UNSUPPORTED, "engram %s: %d experts a token, 1 to %d of the %d supported", who,
          r->chosen, kMaxChosen, r->experts);
    CHECK(r->tokens * r->chosen <= kMaxSlots, ENGRAM_E_RANGE,
          "engram %s: %lld tokens of %d experts exceed %lld slots", who, (long long)r->tokens,
          r->chosen, (long long)kMaxSlots);
    return ENGRAM_OK;
}

// the arrays of a call with tokens
int32_t check_route_arrays(const engram_routes *r, const char *who)
{
    CHECK(r->d_ids && r->d_weights && r->d_offsets && r->d_order, ENGRAM_E_ARG,
          "engram %s: NULL pointer in the routes", who);
    CHECK(aligned(r->d_ids, 4) && aligned(r->d_weights, 4) && aligned(r->d_offsets, 4) &&
              aligned(r->d_order, 4) && aligned(r->d_err, 4),
          ENGRAM_E_ARG, "engram %s: the routes' arrays must be 4-byte aligned", who);
    return ENGRAM_OK;
}

Plan plan_of(const engram_routes *r)
{
    return Plan{r->d_ids, r->d_offsets, r->d_order, r->d_weights, r->d_err, r->experts, r->chosen,
                (int32_t)r->tokens, (int32_t)(r->tokens * r->chosen)};
}

int32_t check_k(int64_t K, const char *who, const char *name)
{
    CHECK(K >= kF8Block && K % kF8Block == 0 && K <= (1 << 20), ENGRAM_E_UNSUPPORTED,
          "engram %s: %s = %lld must be a positive multiple of 128 up to 2^20", who, name,
          (long long)K);
    return ENGRAM_OK;
}

int32_t check_n(int64_t N, const char *who)
{
    CHECK(N >= 16 && N % 16 == 0 && N <= (1 << 24), ENGRAM_E_UNSUPPORTED,
          "engram %s: N = %lld must be a positive multiple of 16 up to 2^24", who, (long long)N);
    return ENGRAM_OK;
}

int32_t check_operands(const uint8_t *x, const void *xs, const uint8_t *w, const float *ws,
                       const char *who)
{
    CHECK(x && xs && w && ws, ENGRAM_E_ARG, "engram %s: NULL pointer", who);
    CHECK(aligned(x, 16) && aligned(w, 16) && aligned(xs, 4) && aligned(ws, 4), ENGRAM_E_ARG,
          "engram %s: rows and weights must be 16-byte, scales 4-byte aligned", who);
    return ENGRAM_OK;
}

}  // namespace

extern "C" {

size_t engram_route_bytes(const engram_routes *routes)
{
    if (check_routes(routes, "route") != ENGRAM_OK || routes->tokens == 0)
        return 0;
    return route_bytes(routes->tokens, routes->experts);
}

int32_t engram_route(const engram_routes *routes, const void *d_logits, int32_t logits_bf16,
                     int64_t logits_stride, const float *d_bias, int32_t softmax, int32_t groups,
                     int32_t top_groups, int32_t group_best, int32_t renorm, float factor,
                     void *d_ws, size_t ws_bytes, void *stream)
{
    int32_t rc = check_routes(routes, "route");
    if (rc != ENGRAM_OK)
        return rc;
    const int64_t T = routes->tokens, E = routes->experts;
    CHECK(groups >= 1 && groups <= 64 && E % groups == 0, ENGRAM_E_UNSUPPORTED,
          "engram route: %d groups must divide the %lld experts, up to 64", groups, (long long)E);
    CHECK(top_groups >= 1 && top_groups <= groups, ENGRAM_E_ARG,
          "engram route: %d of %d groups kept", top_groups, groups);
    CHECK(group_best == 1 || group_best == 2, ENGRAM_E_UNSUPPORTED,
          "engram route: a group's %d best scores (1 or 2)", group_best);
    CHECK(std::isfinite(factor), ENGRAM_E_ARG, "engram route: factor = %g", (double)factor);
    CHECK(logits_stride >= E && logits_stride < ((int64_t)1 << 40), ENGRAM_E_ARG,
          "engram route: rows of %lld experts %lld apart", (long long)E, (long long)logits_stride);
    if (T == 0)
        return ENGRAM_OK;
    rc = check_route_arrays(routes, "route");
    if (rc != ENGRAM_OK)
        return rc;
    CHECK(d_logits, ENGRAM_E_ARG, "engram route: NULL logits");
    CHECK(aligned(d_logits, logits_bf16 ? 2 : 4) && aligned(d_bias, 4), ENGRAM_E_ARG,
          "engram route: logits must be aligned to their size, the bias to 4 bytes");
    const size_t need = route_bytes(T, routes->experts);
    CHECK(ws_bytes >= need, ENGRAM_E_RANGE, "engram route: a workspace of %zu bytes, %zu needed",
          ws_bytes, need);
    CHECK(need == 0 || (d_ws && aligned(d_ws, 256)), ENGRAM_E_ARG,
          "engram route: NULL or unaligned workspace (256 bytes)");
    const Bytes writes[] = {{"workspace", need ? d_ws : nullptr, need},
                            {"routes' ids", routes->d_ids, slot_bytes(routes)},
                            {"routes' weights", routes->d_weights, slot_bytes(routes)},
                            {"routes' offsets", routes->d_offsets, offset_bytes(routes)},
                            {"routes' order", routes->d_order, slot_bytes(routes)},
                            {"error word", routes->d_err, 4}};
    const Bytes reads[] = {
        {"logits", d_logits, ((uint64_t)(T - 1) * logits_stride + E) * (logits_bf16 ? 2 : 4)},
        {"bias", d_bias, 4 * (uint64_t)E}};
    rc = check_apart("route", writes, reads);
    if (rc != ENGRAM_OK)
        return rc;
    const Routing r{d_logits, d_bias, logits_stride, factor, (int32_t)T, (int32_t)E,
                    routes->chosen, groups, top_groups, group_best, logits_bf16 != 0, softmax != 0,
                    renorm != 0, routes->d_ids, routes->d_offsets, routes->d_order, routes->d_err,
                    routes->d_weights};
    return launch_route(r, d_ws, on(stream));
}

int32_t engram_project_f8(const uint8_t *d_x, const void *d_x_scales, int32_t x_f32,
                          const uint8_t *d_w, const float *d_w_scales, uint16_t *d_y, int64_t T,
                          int64_t K, int64_t N, void *stream)
{
    CHECK(T >= 0, ENGRAM_E_ARG, "engram project_f8: T = %lld", (long long)T);
    CHECK(T <= kMaxTokens, ENGRAM_E_RANGE, "engram project_f8: %lld tokens exceed %lld",
          (long long)T, (long long)kMaxTokens);
    int32_t rc = check_k(K, "project_f8", "K");
    if (rc == ENGRAM_OK)
        rc = check_n(N, "project_f8");
    if (rc != ENGRAM_OK || T == 0)
        return rc;
    rc = check_operands(d_x, d_x_scales, d_w, d_w_scales, "project_f8");
    if (rc != ENGRAM_OK)
        return rc;
    CHECK(d_y && aligned(d_y, 16), ENGRAM_E_ARG,
          "engram project_f8: NULL or unaligned y (16 bytes)");
    const Bytes writes[] = {{"output", d_y, (uint64_t)T * (uint64_t)N * 2}};
    const Bytes reads[] = {{"rows", d_x, (uint64_t)T * (uint64_t)K},
                           {"rows' scales", d_x_scales, scale_bytes(T, K, x_f32 != 0)},
                           {"weights", d_w, (uint64_t)N * (uint64_t)K},
                           {"weights' scales", d_w_scales, block_bytes(1, N, K)}};
    rc = check_apart("project_f8", writes, reads);
    if (rc != ENGRAM_OK)
        return rc;
    return launch_project_f8(Rows8{d_x, d_x_scales, x_f32 != 0}, Blocks8{d_w, d_w_scales}, d_y, T,
                             K, N, on(stream));
}

int32_t engram_experts_up(const engram_routes *routes, const uint8_t *d_x, const void *d_x_scales,
                          int32_t x_f32, const uint8_t *d_w, const float *d_w_scales, uint8_t *d_h,
                          uint8_t *d_h_scales, int64_t K, int64_t I, void *stream)
{
    int32_t rc = check_routes(routes, "experts_up");
    if (rc == ENGRAM_OK)
        rc = check_k(K, "experts_up", "K");
    if (rc == ENGRAM_OK)
        rc = check_k(I, "experts_up", "I");
    if (rc != ENGRAM_OK)
        return rc;
    const int64_t T = routes->tokens;
    CHECK(T * K < ((int64_t)1 << 31), ENGRAM_E_RANGE,
          "engram experts_up: %lld tokens of %lld values exceed 2^31-1", (long long)T, (long long)K);
    if (T == 0)
        return ENGRAM_OK;
    rc = check_route_arrays(routes, "experts_up");
    if (rc == ENGRAM_OK)
        rc = check_operands(d_x, d_x_scales, d_w, d_w_scales, "experts_up");
    if (rc != ENGRAM_OK)
        return rc;
    CHECK(d_h && d_h_scales && aligned(d_h, 16) && aligned(d_h_scales, 4), ENGRAM_E_ARG,
          "engram experts_up: NULL or unaligned h (16 bytes) or scales of h (4)");
    const int64_t slots = T * routes->chosen, E = routes->experts;
    const Bytes writes[] = {{"output", d_h, (uint64_t)slots * (uint64_t)I},
                            {"output's scales", d_h_scales, scale_bytes(slots, I, false)},
                            {"error word", routes->d_err, 4}};
    const Bytes reads[] = {{"rows", d_x, (uint64_t)T * (uint64_t)K},
                           {"rows' scales", d_x_scales, scale_bytes(T, K, x_f32 != 0)},
                           {"weights", d_w, 2 * (uint64_t)E * (uint64_t)I * (uint64_t)K},
                           {"weights' scales", d_w_scales, block_bytes(2 * E, I, K)},
                           {"routes' ids", routes->d_ids, slot_bytes(routes)},
                           {"routes' weights", routes->d_weights, slot_bytes(routes)},
                           {"routes' offsets", routes->d_offsets, offset_bytes(routes)},
                           {"routes' order", routes->d_order, slot_bytes(routes)}};
    rc = check_apart("experts_up", writes, reads);
    if (rc != ENGRAM_OK)
        return rc;
    return launch_experts_up(plan_of(routes), Rows8{d_x, d_x_scales, x_f32 != 0},
                             Blocks8{d_w, d_w_scales}, d_h, d_h_scales, K, I, on(stream));
}

size_t engram_experts_down_bytes(const engram_routes *routes, int64_t N)
{
    if (check_routes(routes, "experts_down") != ENGRAM_OK ||
        check_n(N, "experts_down") != ENGRAM_OK || routes->tokens == 0)
        return 0;
    return experts_down_bytes(plan_of(routes), N);
}

int32_t engram_experts_down(const engram_routes *routes, const uint8_t *d_h,
                            const void *d_h_scales, int32_t h_f32, const uint8_t *d_w,
                            const float *d_w_scales, uint16_t *d_y, int64_t K, int64_t N,
                            void *d_ws, size_t ws_bytes, void *stream)
{
    int32_t rc = check_routes(routes, "experts_down");
    if (rc == ENGRAM_OK)
        rc = check_k(K, "experts_down", "K");
    if (rc == ENGRAM_OK)
        rc = check_n(N, "experts_down");
    if (rc != ENGRAM_OK || routes->tokens == 0)
        return rc;
    rc = check_route_arrays(routes, "experts_down");
    if (rc == ENGRAM_OK)
        rc = check_operands(d_h, d_h_scales, d_w, d_w_scales, "experts_down");
    if (rc != ENGRAM_OK)
        return rc;
    CHECK(d_y && aligned(d_y, 16), ENGRAM_E_ARG,
          "engram experts_down: NULL or unaligned y (16 bytes)");
    const Plan p = plan_of(routes);
    const size_t need = experts_down_bytes(p, N);
    CHECK(ws_bytes >= need, ENGRAM_E_RANGE,
          "engram experts_down: a workspace of %zu bytes, %zu needed", ws_bytes, need);
    CHECK(need == 0 || (d_ws && aligned(d_ws, 256)), ENGRAM_E_ARG,
          "engram experts_down: NULL or unaligned workspace (256 bytes)");
    const int64_t E = routes->experts;
    const Bytes writes[] = {{"workspace", need ? d_ws : nullptr, need},
                            {"output", d_y, (uint64_t)routes->tokens * (uint64_t)N * 2},
                            {"error word", routes->d_err, 4}};
    const Bytes reads[] = {{"rows", d_h, (uint64_t)p.slots * (uint64_t)K},
                           {"rows' scales", d_h_scales, scale_bytes(p.slots, K, h_f32 != 0)},
                           {"weights", d_w, (uint64_t)E * (uint64_t)N * (uint64_t)K},
                           {"weights' scales", d_w_scales, block_bytes(E, N, K)},
                           {"routes' ids", routes->d_ids, slot_bytes(routes)},
                           {"routes' weights", routes->d_weights, slot_bytes(routes)},
                           {"routes' offsets", routes->d_offsets, offset_bytes(routes)},
                           {"routes' order", routes->d_order, slot_bytes(routes)}};
    rc = check_apart("experts_down", writes, reads);
    if (rc != ENGRAM_OK)
        return rc;
    return launch_experts_down(p, Rows8{d_h, d_h_scales, h_f32 != 0}, Blocks8{d_w, d_w_scales}, d_y,
                               K, N, d_ws, on(stream));
}

}  // extern "C"
