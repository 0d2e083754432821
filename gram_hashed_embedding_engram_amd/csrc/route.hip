// Routing to experts: scores, choice, weights, and the plan that the experts'
// products follow.
//
//   score = 1 / (1 + e^-x)  or  e^(x - max) / sum e^(x - max) over open experts
//   key   = score + bias, or the logit itself where there is no bias (it orders
//           experts as the score does, to the last bit)
//   a token's experts: of the top_groups groups with the largest sum of their
//   group_best best scores + bias, the k with the largest keys
//
// A wavefront takes a token: expert e is value e / 64 of lane e % 64, and each
// of the k choices is one maximum over the wavefront's keys as ordered integers.
// Choices are whole numbers, so they must not hang on how a score is rounded:
// keys are formed in f32, whose error is bounded here, and a token where two
// keys that are to be told apart lie nearer than that is taken again in 64 bits.
//
// The plan needs no atomics whose order could show: a workgroup's 64 tokens
// set one bit each in an expert's 64-bit word, so a token's place among them is
// the number of bits below its own.  Calls of more tokens count per 64 tokens
// and place in a second launch, which sums the counts before its own.
#include <float.h>

#include "experts.h"

namespace engram {
namespace {

constexpr int kBlockTokens = 64;
constexpr int kWaves = 16;
// counts of this many blocks are summed once more before the blocks are placed
constexpr int kSegment = 64;
constexpr int kMostBlocks = 256;        // placed from the counts alone

typedef unsigned long long u64;

// Where in f32 two keys may stand in the other order than in exact arithmetic.
// A sigmoid is off by 2^-22 of itself at most (e^-x by an ulp, two roundings),
// a softmax score by 2^-20 (the rounding of x - max, the sum), a key's own
// rounding is 2^-24 of it; a group's sum holds two.
__device__ __forceinline__ bool near_keys(float a, float b, bool softmax, float terms)
{
    return a - b <= terms * ((softmax ? 0x1p-19f : 0x1p-21f) + 0x1p-22f * fmaxf(fabsf(a), fabsf(b)));
}

// f32 in the order of its value as an unsigned number above 0; 0 = shut.  (-0,
// which equals 0, becomes 0.)
__device__ __forceinline__ uint32_t ordered(float v)
{
    const uint32_t u = __float_as_uint(v + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u)
{
    return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v)
{
    v = max(v, (uint32_t)dpp_from<0x111, 0xF>((int)v));
    v = max(v, (uint32_t)dpp_from<0x112, 0xF>((int)v));
    v = max(v, (uint32_t)dpp_from<0x114, 0xF>((int)v));
    v = max(v, (uint32_t)dpp_from<0x118, 0xF>((int)v));
    v = max(v, (uint32_t)dpp_from<0x142, 0xA>((int)v));
    v = max(v, (uint32_t)dpp_from<0x143, 0xC>((int)v));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

__device__ __forceinline__ double wave_sum_f64(double v)
{
#pragma unroll
    for (int m = 1; m < 64; m *= 2)
        v += __shfl_xor(v, m);
    return v;
}

// The largest of the wavefront's (key, expert) pairs, the lowest expert among equals.
__device__ __forceinline__ void wave_best_f64(double &v, int &e)
{
#pragma unroll
    for (int m = 1; m < 64; m *= 2) {
        const double ov = __shfl_xor(v, m);
        const int oe = __shfl_xor(e, m);
        if (ov > v || (ov == v && oe < e)) {
            v = ov;
            e = oe;
        }
    }
}

struct Choice {
    int32_t id;         // lane j: the token's j-th expert, -1 = none left
    double score;       // its score
};

// The token in 64 bits.
template <int NR>
__device__ __forceinline__ Choice choose_f64(const Routing &a, const float (&x)[NR], const float *bias,
                                          uint32_t open)
{
    const int lane = threadIdx.x & 63;
    const double low = -INFINITY;
    double score[NR], key[NR];
    if (a.softmax) {
        double top = low;
#pragma unroll
        for (int r = 0; r < NR; r++)
            if (open >> r & 1)
                top = fmax(top, (double)x[r]);
#pragma unroll
        for (int m = 1; m < 64; m *= 2)
            top = fmax(top, __shfl_xor(top, m));
        double sum = 0.0;
#pragma unroll
        for (int r = 0; r < NR; r++) {
            score[r] = open >> r & 1 ? exp((double)x[r] - top) : 0.0;
            sum += score[r];
        }
        sum = wave_sum_f64(sum);
#pragma unroll
        for (int r = 0; r < NR; r++)
            score[r] = sum > 0.0 ? score[r] / sum : 0.0;
    } else {
#pragma unroll
        for (int r = 0; r < NR; r++)
            score[r] = open >> r & 1 ? 1.0 / (1.0 + exp(-(double)x[r])) : 0.0;
    }
#pragma unroll
    for (int r = 0; r < NR; r++)
        key[r] = open >> r & 1 ? score[r] + (bias ? (double)bias[64 * r + lane] : 0.0) : low;
    if (a.groups > 1) {
        const int size = a.E / a.groups;
        double mine = low;              // lane g: group g's sum
        for (int g = 0; g < a.groups; g++) {
            double sum = low;
            int out = -1;
            for (int z = 0; z < a.group_best; z++) {
                double v = low;
                int e = 1 << 30;
#pragma unroll
                for (int r = 0; r < NR; r++) {
                    const int i = 64 * r + lane;
                    if (i / size == g && i != out && key[r] > v) {
                        v = key[r];
                        e = i;
                    }
                }
                wave_best_f64(v, e);
                if (v == low)
                    break;
                sum = z ? sum + v : v;
                out = e;
            }
            if (lane == g)
                mine = sum;
        }
        int ahead = 0;
        for (int h = 0; h < a.groups; h++) {
            const double v = __shfl(mine, h);
            ahead += v > mine || (v == mine && h < lane);
        }
        const u64 kept = __ballot(lane < a.groups && mine > low && ahead < a.top_groups);
#pragma unroll
        for (int r = 0; r < NR; r++) {
            const int i = 64 * r + lane;
            if (i < a.E && !(kept >> (i / size) & 1))
                key[r] = low;
        }
    }
    if (!bias)
#pragma unroll
        for (int r = 0; r < NR; r++)
            if (key[r] > low)
                key[r] = x[r];
    Choice c{-1, 0.0};
    for (int j = 0; j < a.k; j++) {
        double v = low;
        int e = 1 << 30;
#pragma unroll
        for (int r = 0; r < NR; r++)
            if (key[r] > v) {
                v = key[r];
                e = 64 * r + lane;
            }
        wave_best_f64(v, e);
        if (v == low)
            break;
        double s = 0.0;
#pragma unroll
        for (int r = 0; r < NR; r++)
            if (64 * r + lane == e) {
                s = score[r];
                key[r] = low;
            }
        s = wave_sum_f64(s);
        if (lane == j)
            c = Choice{e, s};
    }
    return c;
}

// One token; lane j < k returns its j-th expert and weight.  keys: the
// wavefront's own LDS, E floats (groups only).
template <int NR>
__device__ __forceinline__ void choose(const Routing &a, const float (&x)[NR],
                                       const float (&b)[NR], uint32_t open, const int (&gbit)[NR],
                                       int spread, float *keys, int &id, float &weight)
{
    const int lane = threadIdx.x & 63;
    float score[NR];
    uint32_t key[NR];
    if (a.softmax) {
        float top = -FLT_MAX;
#pragma unroll
        for (int r = 0; r < NR; r++)
            if (open >> r & 1)
                top = fmaxf(top, x[r]);
        top = unordered(wave_max_u32(ordered(top)));
        float sum = 0.0f;
#pragma unroll
        for (int r = 0; r < NR; r++) {
            score[r] = open >> r & 1 ? expf(x[r] - top) : 0.0f;
            sum += score[r];
        }
        sum = wave_sum(sum);
        const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
        for (int r = 0; r < NR; r++)
            score[r] *= inv;
    } else {
#pragma unroll
        for (int r = 0; r < NR; r++)
            score[r] = open >> r & 1 ? 1.0f / (1.0f + expf(-x[r])) : 0.0f;
    }
    bool close = false;
#pragma unroll
    for (int r = 0; r < NR; r++)
        key[r] = !(open >> r & 1) ? 0u : ordered(a.bias ? score[r] + b[r] : x[r]);
    if (a.groups > 1) {
        const int size = a.E / a.groups, g = lane / spread, sub = lane & (spread - 1);
#pragma unroll
        for (int r = 0; r < NR; r++)
            if (64 * r + lane < a.E)
                keys[64 * r + lane] = open >> r & 1 ? score[r] + b[r] : -INFINITY;
        float first = -INFINITY, second = -INFINITY;
        if (g < a.groups)
            for (int i = sub; i < size; i += spread) {
                const float v = keys[g * size + i];
                second = fmaxf(second, fminf(first, v));
                first = fmaxf(first, v);
            }
        for (int m = 1; m < spread; m *= 2) {
            const float f = __shfl_xor(first, m), s = __shfl_xor(second, m);
            second = fmaxf(fmaxf(second, s), fminf(first, f));
            first = fmaxf(first, f);
        }
        float sum = first;
        if (a.group_best > 1 && second > -INFINITY)
            sum += second;
        int ahead = 0;
        for (int h = 0; h < a.groups; h++) {
            const float v = __uint_as_float(
                (uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(sum), h * spread));
            ahead += v > sum || (v == sum && h < g);
        }
        const bool in = g < a.groups && sum > -INFINITY, keep = in && ahead < a.top_groups;
        const u64 kept = __ballot(keep);
        if (__ballot(in && !keep)) {
            const float worst = -unordered(wave_max_u32(keep ? ordered(-sum) : 0u));
            const float next = unordered(wave_max_u32(in && !keep ? ordered(sum) : 0u));
            close = near_keys(worst, next, a.softmax, 2.0f);
        }
#pragma unroll
        for (int r = 0; r < NR; r++)
            if (!(kept >> gbit[r] & 1))
                key[r] = 0u;
    }
    // lane j: the j-th key, its expert and score; one more than k are taken
    uint32_t mine = 0u;
    float s = 0.0f;
    id = -1;
    for (int j = 0; j <= a.k; j++) {
        uint32_t v = key[0];
#pragma unroll
        for (int r = 1; r < NR; r++)
            v = max(v, key[r]);
        v = wave_max_u32(v);
        if (v == 0u)
            break;
        bool found = false;
#pragma unroll
        for (int r = 0; r < NR; r++) {
            const u64 at = __ballot(key[r] == v);
            if (!found && at) {
                found = true;
                const int l = __builtin_ctzll(at);
                const float sc = __uint_as_float(
                    (uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(score[r]), l));
                if (lane == j) {
                    mine = v;
                    id = 64 * r + l;
                    s = sc;
                }
                if (lane == l)
                    key[r] = 0u;
            }
        }
    }
    if (a.bias) {
        const uint32_t next = (uint32_t)__shfl_down((int)mine, 1);
        close = close || __ballot(lane < a.k && next != 0u && mine != 0u &&
                                  near_keys(unordered(mine), unordered(next), a.softmax, 1.0f));
    }
    if (lane >= a.k) {
        id = -1;
        s = 0.0f;
    }
    float sum = wave_sum(s);
    if (__ballot(close) || (sum < 0x1p-90f && __ballot(id >= 0))) {
        const Choice c = choose_f64<NR>(a, x, a.bias, open);
        id = lane < a.k ? c.id : -1;
        const double sc = id >= 0 ? c.score : 0.0;
        const double total = wave_sum_f64(sc);
        weight = (float)((a.renorm ? (total > 0.0 ? sc / total : 0.0) : sc) * (double)a.factor);
        return;
    }
    weight = (a.renorm ? (sum > 0.0f ? s / sum : 0.0f) : s) * a.factor;
}

// Exclusive sums over the experts' counts (E <= blockDim.x: thread e has
// expert e's); returns the one before e, `all` = the sum of all.
__device__ __forceinline__ int before_expert(int count, int *part, int &all)
{
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int sum = wave_scan(count);
    if (lane == 63)
        part[wv] = sum;
    __syncthreads();
    int before = 0;
    all = 0;
    for (int i = 0; i < kWaves; i++) {
        before += i < wv ? part[i] : 0;
        all += part[i];
    }
    __syncthreads();
    return before + sum - count;
}

template <bool BF16, int NR>
__global__ __launch_bounds__(64 * kWaves) void route_kernel(Routing a, uint8_t *counts, int pitch)
{
    __shared__ u64 mask[64 * NR];
    __shared__ int32_t ids_s[kBlockTokens * kMaxChosen];
    __shared__ int start[64 * NR];
    __shared__ int part[kWaves];
    __shared__ float keys_s[kWaves][64 * NR];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int t0 = blockIdx.x * kBlockTokens;
    for (int i = tid; i < 64 * NR; i += 64 * kWaves)
        mask[i] = 0;
    // lanes a group's experts are looked through by: a power of two
    int spread = 64;
    while (spread * a.groups > 64)
        spread /= 2;
    float b[NR];
    int gbit[NR];
    uint32_t known = 0;
    bool odd = false;
#pragma unroll
    for (int r = 0; r < NR; r++) {
        const int e = 64 * r + lane;
        b[r] = a.bias && e < a.E ? a.bias[e] : 0.0f;
        odd |= b[r] > FLT_MAX || b[r] != b[r];
        known |= (uint32_t)(e < a.E && fabsf(b[r]) <= FLT_MAX) << r;
        gbit[r] = e < a.E ? e / (a.E / a.groups) * spread : 0;
    }
    __syncthreads();
    for (int t = t0 + wv; t < min(t0 + kBlockTokens, a.T); t += kWaves) {
        float x[NR];
        uint32_t open = 0;
#pragma unroll
        for (int r = 0; r < NR; r++) {
            const int e = 64 * r + lane;
            const int64_t at = (int64_t)t * a.stride + e;
            x[r] = -INFINITY;
            if (e < a.E)
                x[r] = BF16 ? bf16_lo(((const uint16_t *)a.logits)[at]) : ((const float *)a.logits)[at];
            odd |= x[r] > FLT_MAX || x[r] != x[r];
            open |= (uint32_t)((known >> r & 1) && fabsf(x[r]) <= FLT_MAX) << r;
        }
        int id;
        float weight;
        choose<NR>(a, x, b, open, gbit, spread, keys_s[wv], id, weight);
        if (lane < a.k) {
            const int64_t slot = (int64_t)t * a.k + lane;
            a.ids[slot] = id;
            a.weights[slot] = weight;
            ids_s[(t - t0) * a.k + lane] = id;
            if (id >= 0)
                atomicOr(&mask[id], 1ull << (t - t0));
        }
    }
    if (odd)
        raise(a.err, ENGRAM_DEVERR_ROUTE);
    __syncthreads();
    if (counts) {                       // placed by the next launch
        for (int e = tid; e < pitch; e += 64 * kWaves)
            counts[(int64_t)blockIdx.x * pitch + e] = e < 64 * NR ? (uint8_t)__popcll(mask[e]) : 0;
        return;
    }
    int all;
    const int before = before_expert(tid < 64 * NR ? __popcll(mask[tid]) : 0, part, all);
    if (tid < a.E) {
        start[tid] = before;
        a.offsets[tid] = before;
    }
    if (tid == 0)
        a.offsets[a.E] = all;
    __syncthreads();
    for (int i = tid; i < (min(t0 + kBlockTokens, a.T) - t0) * a.k; i += 64 * kWaves) {
        const int e = ids_s[i], t = i / a.k;
        if (e >= 0)
            a.order[start[e] + __popcll(mask[e] & ((1ull << t) - 1))] = i;
    }
}

// Sums of kSegment blocks' counts.
__global__ __launch_bounds__(256) void segment_kernel(const uint8_t *__restrict__ counts,
                                                      int32_t *__restrict__ sums, int blocks, int pitch)
{
    const int first = blockIdx.x * kSegment, last = min(first + kSegment, blocks);
    for (int e = threadIdx.x; e < pitch; e += 256) {
        int sum = 0;
        for (int i = first; i < last; i++)
            sum += counts[(int64_t)i * pitch + e];
        sums[(int64_t)blockIdx.x * pitch + e] = sum;
    }
}

// A block's slots to their places, after the counts of the blocks before it.
// segments: sums of kSegment blocks each, or null (the counts alone).
__global__ __launch_bounds__(64 * kWaves) void place_kernel(Routing a, const uint8_t *counts,
                                                            const int32_t *segments, int blocks,
                                                            int pitch)
{
    __shared__ u64 mask[kMaxExperts];
    __shared__ int before_s[kMaxExperts], all_s[kMaxExperts], part[kWaves];
    const int tid = threadIdx.x, block = blockIdx.x, t0 = block * kBlockTokens;
    mask[tid] = 0;
    before_s[tid] = all_s[tid] = 0;
    __syncthreads();
    const int words = pitch / 4, w = tid % words;     // pitch <= 1024: four experts a word
    const int rows = 64 * kWaves / words, row = tid / words;
    int sum[4] = {}, all[4] = {};
    if (row < rows) {
        int first = 0, last = blocks;
        if (segments) {
            const int mine = block / kSegment, n = (blocks + kSegment - 1) / kSegment;
            for (int i = row; i < n; i += rows)
#pragma unroll
                for (int z = 0; z < 4; z++) {
                    const int v = segments[(int64_t)i * pitch + 4 * w + z];
                    all[z] += v;
                    sum[z] += i < mine ? v : 0;
                }
            first = mine * kSegment;
            last = block;
        }
#pragma unroll 4
        for (int i = first + row; i < last; i += rows) {
            const uint32_t v = *(const uint32_t *)(counts + (int64_t)i * pitch + 4 * w);
#pragma unroll
            for (int z = 0; z < 4; z++) {
                const int c = (v >> (8 * z)) & 0xFF;
                all[z] += segments ? 0 : c;
                sum[z] += i < block ? c : 0;
            }
        }
#pragma unroll
        for (int z = 0; z < 4; z++) {
            atomicAdd(&before_s[4 * w + z], sum[z]);
            atomicAdd(&all_s[4 * w + z], all[z]);
        }
    }
    const int n = (min(t0 + kBlockTokens, a.T) - t0) * a.k;
    const int32_t *ids = a.ids + (int64_t)t0 * a.k;
    for (int i = tid; i < n; i += 64 * kWaves)
        if (ids[i] >= 0)
            atomicOr(&mask[ids[i]], 1ull << (i / a.k));
    __syncthreads();
    int total;
    const int start = before_expert(tid < pitch ? all_s[tid] : 0, part, total);
    if (tid < a.E) {
        if (block == 0)
            a.offsets[tid] = start;
        before_s[tid] += start;
    }
    if (block == 0 && tid == 0)
        a.offsets[a.E] = total;
    __syncthreads();
    for (int i = tid; i < n; i += 64 * kWaves) {
        const int e = ids[i];
        if (e >= 0)
            a.order[before_s[e] + __popcll(mask[e] & ((1ull << (i / a.k)) - 1))] = t0 * a.k + i;
    }
}

int pitch_of(int32_t E) { return (E + 15) / 16 * 16; }
int64_t blocks_of(int64_t T) { return (T + kBlockTokens - 1) / kBlockTokens; }
size_t counts_bytes(int64_t T, int32_t E) { return ((size_t)(blocks_of(T) * pitch_of(E)) + 255) & ~(size_t)255; }

template <bool BF16, int NR>
void launch_scores(const Routing &r, uint8_t *counts, const Launch &l)
{
    dispatch(route_kernel<BF16, NR>, dim3((unsigned)blocks_of(r.T)), dim3(64 * kWaves), l, true,
             !counts, r, counts, pitch_of(r.E));
}

template <bool BF16>
void launch_type(const Routing &r, uint8_t *counts, const Launch &l)
{
    r.E <= 64    ? launch_scores<BF16, 1>(r, counts, l)
    : r.E <= 128 ? launch_scores<BF16, 2>(r, counts, l)
    : r.E <= 256 ? launch_scores<BF16, 4>(r, counts, l)
    : r.E <= 512 ? launch_scores<BF16, 8>(r, counts, l)
                 : launch_scores<BF16, 16>(r, counts, l);
}

}  // namespace

size_t route_bytes(int64_t T, int32_t E)
{
    const int64_t blocks = blocks_of(T);
    if (blocks <= 1)
        return 0;
    size_t n = counts_bytes(T, E);
    if (blocks > kMostBlocks)
        n += (size_t)((blocks + kSegment - 1) / kSegment) * pitch_of(E) * sizeof(int32_t);
    return n;
}

int32_t launch_route(const Routing &r, void *ws, const Launch &l)
{
    const int64_t blocks = blocks_of(r.T);
    uint8_t *counts = blocks > 1 ? (uint8_t *)ws : nullptr;
    r.bf16 ? launch_type<true>(r, counts, l) : launch_type<false>(r, counts, l);
    if (counts) {
        int32_t *sums = blocks > kMostBlocks ? (int32_t *)(counts + counts_bytes(r.T, r.E)) : nullptr;
        if (sums)
            dispatch(segment_kernel, dim3((unsigned)((blocks + kSegment - 1) / kSegment)), dim3(256),
                     l, false, false, (const uint8_t *)counts, sums, (int)blocks, pitch_of(r.E));
        dispatch(place_kernel, dim3((unsigned)blocks), dim3(64 * kWaves), l, false, true, r,
                 (const uint8_t *)counts, (const int32_t *)sums, (int)blocks, pitch_of(r.E));
    }
    return launch_status("engram route kernels");
}

}  // namespace engram
