// Shared pieces of the experts' kernels (route.hip, f8_rows.hip, f8_tiles.hip):
// the plan that a routing makes and how work items find their expert in it, the
// launchers.  Internal to the library.
#pragma once

#include "attention.h"

namespace engram {

constexpr int kF8Block = ENGRAM_F8_BLOCK;
constexpr int32_t kMaxExperts = 1024;
constexpr int32_t kMaxChosen = 32;

// A plan as the kernels see it: slots (token * k + j) sorted by expert.
struct Plan {
    const int32_t *ids, *offsets, *order;
    const float *weights;
    int32_t *err;
    int32_t E, k, T, slots;         // slots = T * k
};

// The plan's rows of expert e, within what the call's arrays hold.
struct Span {
    int32_t from, n;
};

__device__ __forceinline__ Span span_of(const Plan &p, int e)
{
    const int32_t a = p.offsets[e], b = p.offsets[e + 1];
    const bool ok = a >= 0 && b >= a && b <= p.slots;
    return Span{ok ? a : 0, ok ? b - a : 0};
}

// Work item i where expert e has pieces(rows) of them, in the experts' order:
// the expert, the piece of it and its rows.  Whole wavefronts, uniform i;
// false past the last item.
template <class F>
__device__ __forceinline__ bool find_expert(int i, const Plan &p, F pieces, int &expert, int &piece,
                                            Span &span)
{
    const int lane = threadIdx.x & 63;
    for (int base = 0; base < p.E; base += 64) {
        const Span s = base + lane < p.E ? span_of(p, base + lane) : Span{0, 0};
        const int own = pieces(s.n);
        const int sum = wave_scan(own);
        const uint64_t over = __ballot(sum > i);
        if (over) {
            const int at = __builtin_ctzll(over);
            expert = base + at;
            piece = i - __builtin_amdgcn_readlane(sum - own, at);
            span = Span{__builtin_amdgcn_readlane(s.from, at), __builtin_amdgcn_readlane(s.n, at)};
            return true;
        }
        i -= __builtin_amdgcn_readlane(sum, 63);
    }
    return false;
}

// How many items find_expert finds.
template <class F>
__device__ __forceinline__ int all_pieces(const Plan &p, F pieces)
{
    const int lane = threadIdx.x & 63;
    int sum = 0;
    for (int base = 0; base < p.E; base += 64)
        sum += base + lane < p.E ? pieces(span_of(p, base + lane).n) : 0;
    return __builtin_amdgcn_readlane(wave_scan(sum), 63);
}

// Spans that do not hold set the error bit (one workgroup of a call).
__device__ __forceinline__ void raise_bad_plan(const Plan &p)
{
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
        const int32_t a = p.offsets[e], b = p.offsets[e + 1];
        if (!(a >= 0 && b >= a && b <= p.slots))
            raise(p.err, ENGRAM_DEVERR_ROUTE);
    }
}

// silu(g) * u
__device__ __forceinline__ float gated(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// ------------------------------------------------------------------ host

// 8-bit rows and their scales: E8M0 per 32 values, or f32 per 128.
struct Rows8 {
    const uint8_t *x;
    const void *s;
    bool f32;
};

// 8-bit weights with an f32 scale per 128 x 128 block.
struct Blocks8 {
    const uint8_t *w;
    const float *s;
};

struct Routing {
    const void *logits;
    const float *bias;
    int64_t stride;
    float factor;
    int32_t T, E, k, groups, top_groups, group_best;
    bool bf16, softmax, renorm;
    int32_t *ids, *offsets, *order, *err;
    float *weights;
};

size_t route_bytes(int64_t T, int32_t E);
int32_t launch_route(const Routing &r, void *ws, const Launch &l);

int32_t launch_project_f8(const Rows8 &x, const Blocks8 &w, uint16_t *y, int64_t T, int64_t K,
                          int64_t N, const Launch &l);
int32_t launch_experts_up(const Plan &p, const Rows8 &x, const Blocks8 &w, uint8_t *h, uint8_t *hs,
                          int64_t K, int64_t I, const Launch &l);
size_t experts_down_bytes(const Plan &p, int64_t N);
int32_t launch_experts_down(const Plan &p, const Rows8 &h, const Blocks8 &w, uint16_t *y, int64_t K,
                            int64_t N, void *ws, const Launch &l);

}  // namespace engram
