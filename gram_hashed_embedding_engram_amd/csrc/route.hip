// Routing to experts: scores, choice, weights, and the plan that the experts'
// products follow.
//
//   score = 1 / (1 + e^-x)  or  e^(x - max) / sum e^(x - max) over open experts
//   key   = score + bias, or the logit itself where there is no bias (it orders
//           experts as the score does, to the last bit)
//   a token's experts: of the top_groups groups with the largest sum of their
//   group_best best scores + bias, the k with the largest keys
//
// A wavefront takes a token: of NR experts a lane, expert e is value e % NR of lane
// e / NR.  A bound below the largest key, found by trial, leaves a few more
// candidates than k, one a lane, and each lane counts those ahead of its own.
// Choices are whole numbers, so they must not hang on how a score is rounded:
// keys are formed in f32, whose error is bounded here, and a token where two
// keys that are to be told apart lie nearer than that is taken again in 64 bits.
//
// The plan needs no atomics whose order could show: a workgroup's 64 tokens
// set one bit each in an expert's 64-bit word, so a token's place among them is
// the number of bits below its own.  Calls of more tokens count per 64 tokens
// and place in a second launch, which sums the counts before its own.
//
// 16384 tokens of 256 experts in 8 groups (17 MB): 27 to 28 us, of which the second
// launch is 6.  It waits on itself: the vector units are busy 44% of the time and LDS
// 10%, with one workgroup of 16 wavefronts a CU (128 registers), each wavefront a chain
// of some 450 instructions a token, many of them across lanes.  The 64-bit paths stand
// in the same function, and what does not fit into 128 registers goes to scratch: none
// of a lane's for up to 256 experts, 34 for 512, 178 for 1024 (16384 tokens of 384
// experts 42 us, of 1024 141 to 161).  One token: 6.2 us, a launch and a chain of some
// thousand cycles; 64, in one workgroup, 20.6.  Rows with more than k + 16 equal best keys, such
// as logits of nothing but zeros, find no bound and choose one expert after the other
// in 64 bits: three times as long (16384 such rows 87 us, 64 of them 80; of 1024
// experts 320).  Each choice as a maximum of its own took 54 us, 22 of them the few
// tokens taken again in 64 bits one choice after the other; now the candidates alone
// are ranked again.
#include <float.h>

#include "experts.h"

namespace engram {
namespace {

constexpr int kBlockTokens = 64;        // at most: a bit each
constexpr int kWaves = 16;
// counts of this many blocks are summed once more before the blocks are placed
constexpr int kSegment = 64;
constexpr int kMostBlocks = 256;        // placed from the counts alone
// candidates for a token's choice beyond those needed: 7, 15 and 30 take 28.3, 28.3 and
// 29.4 us for 16384 tokens of 256 experts (more trials, more to rank)
constexpr int kSpare = 15;

typedef unsigned long long u64;

// Where in f32 two keys may stand in the other order than in exact arithmetic:
// unit covers what their scores are off by together.  e^-x is off by (1.5 |x| + 2)
// 2^-24 of itself (the product with log2 e, the instruction), which a sigmoid, whose
// slope times |x| is below 0.23, passes on as less than 2^-22, and its sum and
// reciprocal add another: 2^-20 for two.  A softmax score is off by (1.5 |d| + 2) 2^-24
// of itself at a distance d from the largest logit, so by less than 2.6 * 2^-24 of the
// largest score, and by NR + 9 roundings of the sum, the reciprocal and the product:
// 2^-18 of the largest score for two, at NR = 16.  A key's own rounding is 2^-24 of it.
__device__ __forceinline__ bool near_keys(float a, float b, float unit)
{
    return a - b <= unit + 0x1p-22f * fmaxf(fabsf(a), fabsf(b));
}

// How far a group's sum (half the sum of two keys, or one key) is off: by half of
// unit, by its keys' roundings and by its own, which are 2^-24 of the larger key
// each, and by as much where it is compared.  The sum may be far smaller than its
// keys, so their size counts.
__device__ __forceinline__ float sum_error(float first, float second, float unit)
{
    return 0.5f * unit + 0x1.8p-23f * fmaxf(fabsf(first), second > -INFINITY ? fabsf(second) : 0.0f);
}

// Where the scores of logits a >= b may be one and the same number of 64 bits, or
// f32's and theirs differ: next to each other, where a sigmoid is almost 1, or where
// either vanishes.  (Equal logits have equal scores.)
__device__ __forceinline__ bool near_logits(float a, float b, float top, bool softmax)
{
    return a != b && (a - b < 0x1p-40f || (!softmax && a > 16.0f) || b - top < -600.0f);
}

// f32 in the order of its value as an unsigned number.  (-0, which equals 0,
// becomes 0.)
__device__ __forceinline__ uint32_t ordered(float v)
{
    const uint32_t u = __float_as_uint(v + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
// The largest of the wavefront's values.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_max(float v)
{
    const int u = __float_as_int(v);
    return fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(u, u, CTRL, ROWS, 0xF, false)));
}
__device__ __forceinline__ float wave_max(float v)
{
    v = dpp_max<0x111, 0xF>(v);
    v = dpp_max<0x112, 0xF>(v);
    v = dpp_max<0x114, 0xF>(v);
    v = dpp_max<0x118, 0xF>(v);
    v = dpp_max<0x142, 0xA>(v);
    v = dpp_max<0x143, 0xC>(v);
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
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

// e^x to (1.5 |x| + 2) 2^-24 of itself
__device__ __forceinline__ float fast_exp(float x)
{
    return __builtin_amdgcn_exp2f(x * 1.44269504088896340736f);
}

// The two largest of what lanes hold, over the 2, 4, .. `lanes` lanes around each.
template <int CTRL>
__device__ __forceinline__ void merge_dpp(float &first, float &second)
{
    const float f = __int_as_float(dpp_from<CTRL, 0xF>(__float_as_int(first)));
    const float s = __int_as_float(dpp_from<CTRL, 0xF>(__float_as_int(second)));
    second = fmaxf(fmaxf(second, s), fminf(first, f));
    first = fmaxf(first, f);
}
__device__ __forceinline__ void merge_best(float &first, float &second, int lanes)
{
    if (lanes > 1)
        merge_dpp<0xB1>(first, second);              // quad_perm [1,0,3,2]
    if (lanes > 2)
        merge_dpp<0x4E>(first, second);              // quad_perm [2,3,0,1]
    if (lanes > 4)
        merge_dpp<0x141>(first, second);             // row_half_mirror
    if (lanes > 8)
        merge_dpp<0x140>(first, second);             // row_mirror
    for (int m = 16; m < lanes; m *= 2) {
        const float f = __shfl_xor(first, m), s = __shfl_xor(second, m);
        second = fmaxf(fmaxf(second, s), fminf(first, f));
        first = fmaxf(first, f);
    }
}

// How a wavefront looks through groups of experts.  lanes: a group is
// `spread` whole lanes; otherwise `spread` lanes look through a group's experts
// in LDS.  spread is a power of two.
struct Groups {
    int spread;
    bool lanes;
};

// What a token's scores in 64 bits are made of.
struct Exact {
    double top, sum;                    // of a softmax
    bool softmax;
    __device__ __forceinline__ double score(double x) const
    {
        return softmax ? exp(x - top) / sum : 1.0 / (1.0 + exp(-x));
    }
};
template <int NR>
__device__ __forceinline__ Exact exact_of(const Routing &a, const float (&x)[NR])
{
    Exact e{0.0, 1.0, a.softmax};
    if (a.softmax) {
        float top = -FLT_MAX;
#pragma unroll
        for (int r = 0; r < NR; r++)
            top = fmaxf(top, x[r]);
        e.top = wave_max(top);
        e.sum = 0.0;
#pragma unroll
        for (int r = 0; r < NR; r++)
            if (x[r] > -INFINITY)
                e.sum += exp((double)x[r] - e.top);
        e.sum = wave_sum_f64(e.sum);
    }
    return e;
}

// The groups kept by sums in 64 bits, a bit each: `spread` lanes look through a
// group's experts.
template <int NR>
__device__ __forceinline__ u64 groups_f64(const Routing &a, const Groups &gr, const float (&x)[NR],
                                          float *values)
{
    const int lane = threadIdx.x & 63, g = lane / gr.spread, size = a.E / a.groups;
    const double low = -INFINITY;
    const Exact exact = exact_of<NR>(a, x);
#pragma unroll
    for (int r = 0; r < NR; r++)
        values[NR * lane + r] = x[r];
    double first = low, second = low;
    if (g < a.groups)
        for (int i = g * size + (lane & (gr.spread - 1)); i < (g + 1) * size; i += gr.spread) {
            const float v = values[i];
            if (v == -INFINITY)
                continue;
            const double key = exact.score(v) + (a.bias ? (double)a.bias[i] : 0.0);
            second = fmax(second, fmin(first, key));
            first = fmax(first, key);
        }
    for (int m = 1; m < gr.spread; m *= 2) {
        const double f = __shfl_xor(first, m), s = __shfl_xor(second, m);
        second = fmax(fmax(second, s), fmin(first, f));
        first = fmax(first, f);
    }
    if (a.group_best > 1 && second > low)
        first += second;
    const double mine = __shfl(first, lane < a.groups ? lane * gr.spread : 0);   // lane g: group g's sum
    int ahead = 0;
    for (int h = 0; h < a.groups; h++) {
        const double v = __shfl(mine, h);
        ahead += v > mine || (v == mine && h < lane);
    }
    return __ballot(lane < a.groups && mine > low && ahead < a.top_groups);
}

// Choices one by one from scores and keys in 64 bits: lane j < k gets its
// expert and score.
template <int NR>
__device__ __forceinline__ Choice choose_f64(const Routing &a, double (&score)[NR], double (&key)[NR])
{
    const int lane = threadIdx.x & 63;
    const double low = -INFINITY;
    Choice c{-1, 0.0};
    for (int j = 0; j < a.k; j++) {
        double v = low;
        int e = 1 << 30;
#pragma unroll
        for (int r = 0; r < NR; r++)
            if (key[r] > v) {
                v = key[r];
                e = NR * lane + r;
            }
        wave_best_f64(v, e);
        if (v == low)
            break;
        double s = 0.0;
#pragma unroll
        for (int r = 0; r < NR; r++)
            if (NR * lane + r == e) {
                s = score[r];
                key[r] = low;
            }
        s = wave_sum_f64(s);
        if (lane == j)
            c = Choice{e, s};
    }
    return c;
}

__device__ __forceinline__ float lane_value(float v, int lane)
{
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}
__device__ __forceinline__ int lanes_below(u64 mask)
{
    return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}

// How many of lanes 0, step, 2 step, .. (n of them, and one more where n is odd,
// which holds the least) hold more than this lane's v, or as much
// and are before it: `own` is its number among them.
__device__ __forceinline__ int rank_of(uint32_t v, int own, int n, int step)
{
    const u64 key = (u64)v << 32 | (uint32_t)(63 - own);
    int rank = 0;
    for (int i = 0; i < n; i += 2)
#pragma unroll
        for (int z = 0; z < 2; z++) {
            const u64 o = (u64)(uint32_t)__builtin_amdgcn_readlane((int)v, (i + z) * step) << 32 |
                          (uint32_t)(63 - i - z);
            rank += o > key;
        }
    return rank;
}

// a / b to an ulp or two, for b and its reciprocal normal numbers
__device__ __forceinline__ float quotient(float a, float b)
{
    const float r = __builtin_amdgcn_rcpf(b), q = a * r;
    return __builtin_fmaf(__builtin_fmaf(-b, q, a), r, q);
}

// n candidates, lane i's expert e: in the order of their keys in 64 bits.
template <int NR>
__device__ __forceinline__ int rank_f64(const Routing &a, const float (&x)[NR], float *values,
                                        int n, int e)
{
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int r = 0; r < NR; r++)
        values[NR * lane + r] = x[r];
    const Exact exact = exact_of<NR>(a, x);
    const double key = e >= 0 ? exact.score(values[e]) + (double)a.bias[e] : 0.0;
    int rank = 0;
    for (int i = 0; i < n; i++) {
        const double o = __shfl(key, i);
        const int oe = __builtin_amdgcn_readlane(e, i);
        rank += o > key || (o == key && oe < e);
    }
    if (lane < n)
        values[rank] = __int_as_float(e);
    return lane < n ? __float_as_int(values[lane]) : -1;
}

// One token; lane j < k returns its j-th expert and weight.  x is -inf where an
// expert is shut.  values: the wavefront's own LDS, 64 * NR floats (128 at least).
// slack: how far below the largest key the last token's bound was.  gbit: the lane
// that speaks for each expert's group (where groups are not whole lanes).
template <int NR>
__device__ __forceinline__ void choose(const Routing &a, const Groups &gr, const float (&x)[NR],
                                       const float (&b)[NR], const int (&gbit)[NR], float *values,
                                       float &slack, int &id, float &weight)
{
    const int lane = threadIdx.x & 63;
    float score[NR], key[NR];
    float top = 0.0f, all = 0.0f, unit = 0x1p-20f;
    if (a.softmax) {
        top = -FLT_MAX;
#pragma unroll
        for (int r = 0; r < NR; r++)
            top = fmaxf(top, x[r]);
        top = wave_max(top);
#pragma unroll
        for (int r = 0; r < NR; r++) {
            score[r] = fast_exp(x[r] - top);
            all += score[r];
        }
        all = wave_sum(all);
        const float inv = all > 0.0f ? 1.0f / all : 0.0f;
#pragma unroll
        for (int r = 0; r < NR; r++)
            score[r] *= inv;
        unit = 0x1p-18f * inv;
    } else {
#pragma unroll
        for (int r = 0; r < NR; r++)
            score[r] = __builtin_amdgcn_rcpf(1.0f + fast_exp(-x[r]));
    }
#pragma unroll
    for (int r = 0; r < NR; r++)
        key[r] = !a.bias || x[r] == -INFINITY ? x[r] : score[r] + b[r];
    if (a.groups > 1) {
        float first = -INFINITY, second = -INFINITY;
        const int g = lane / gr.spread;
        // one best score without a bias: the largest logits say which is more
        const bool logits = !a.bias && a.group_best == 1;
        if (gr.lanes) {
#pragma unroll
            for (int r = 0; r < NR; r++) {
                const float v = logits || x[r] == -INFINITY ? x[r] : score[r] + b[r];
                second = fmaxf(second, fminf(first, v));
                first = fmaxf(first, v);
            }
        } else {
#pragma unroll
            for (int r = 0; r < NR; r++)
                values[NR * lane + r] = logits || x[r] == -INFINITY ? x[r] : score[r] + b[r];
            const int size = a.E / a.groups;
            if (g < a.groups)
                for (int i = lane & (gr.spread - 1); i < size; i += gr.spread) {
                    const float v = values[g * size + i];
                    second = fmaxf(second, fminf(first, v));
                    first = fmaxf(first, v);
                }
        }
        merge_best(first, second, gr.spread);
        // (of two, half their sum: two of f32's lowest or largest values, which masks
        // are, have a sum past its range)
        float sum = first;
        if (a.group_best > 1)
            sum = 0.5f * first + (second > -INFINITY ? 0.5f * second : 0.0f);
        // (lanes past the groups hold -inf)
        const int ahead = rank_of(ordered(sum), g, a.groups, gr.spread);
        const bool in = g < a.groups && sum > -INFINITY;
        bool keep = in && ahead < a.top_groups;
        u64 kept = __ballot(keep);
        bool near = false;
        if (const u64 next = __ballot(in && ahead == a.top_groups)) {
            if (logits) {
                // (where the last kept and the next are equal, others may be near both)
                const u64 last = __ballot(in && ahead == a.top_groups - 1);
                const float u = lane_value(sum, __builtin_ctzll(last)), v = lane_value(sum, __builtin_ctzll(next));
                near = __ballot(in && near_logits(keep ? sum : u, keep ? v : sum, top, a.softmax));
            } else {
                // the least that a kept sum may be, the most that another may
                const float e = sum_error(first, a.group_best > 1 ? second : first, unit);
                near = wave_max(keep ? e - sum : -INFINITY) + wave_max(in && !keep ? sum + e : -INFINITY) >= 0.0f;
            }
        }
        if (near) {
            const u64 by_group = groups_f64<NR>(a, gr, x, values);
            keep = g < a.groups && (by_group >> g & 1);
            kept = __ballot(keep);
        }
#pragma unroll
        for (int r = 0; r < NR; r++)
            if (gr.lanes ? !keep : !(kept >> gbit[r] & 1))
                key[r] = -INFINITY;
    }
    // The candidates: keys not below a bound that leaves more than k of them (or
    // all that there are) and at most kSpare besides, found by trial from where the
    // last token's was.
    float high = key[0];
#pragma unroll
    for (int r = 1; r < NR; r++)
        high = fmaxf(high, key[r]);
    high = wave_max(high);
    int total = 0;
#pragma unroll
    for (int r = 0; r < NR; r++)
        total += __popcll(__ballot(key[r] > -INFINITY));
    const int want = min(a.k + 1, total), most = want + kSpare;
    int n = total;
    float bound = -FLT_MAX;
    for (int turn = 0; n > most && turn < 16; turn++) {
        bound = high - slack;
        n = 0;
#pragma unroll
        for (int r = 0; r < NR; r++)
            n += __popcll(__ballot(key[r] >= bound));
        if (n >= want && n <= most)
            break;
        slack = fminf(fmaxf(slack * (n < want ? 1.5f : n > 2 * most ? 0.5f : 0.75f), 0x1p-20f), 0x1p20f);
        n = 64 * NR + 1;
    }
    float mine = -INFINITY;
    int at = -1;
    bool exact = false;
    if (n <= 64) {
        // (key, id) pairs, the id's bits as a float: the same LDS holds logits before
        // and after, so every access to it is of one type
        const auto put = [&](int i, float key, int id) {
            values[2 * i] = key;
            values[2 * i + 1] = __int_as_float(id);
        };
        // to the lanes, in the experts' order
        int before = 0;
#pragma unroll
        for (int r = 0; r < NR; r++)
            before += lanes_below(__ballot(key[r] >= bound));
#pragma unroll
        for (int r = 0; r < NR; r++)
            if (key[r] >= bound)
                put(before++, key[r], NR * lane + r);
        if (lane < n) {
            mine = values[2 * lane];
            at = __float_as_int(values[2 * lane + 1]);
        }
        const int rank = rank_of(ordered(mine), lane, n, 1);
        // in the order of their keys
        if (lane < n) {
            put(rank, mine, at);
            mine = values[2 * lane];
            at = __float_as_int(values[2 * lane + 1]);
        }
        if (a.bias) {
            const int low = __float_as_int(-INFINITY);
            const float next = __int_as_float(                       // of lane j + 1
                __builtin_amdgcn_update_dpp(low, __float_as_int(mine), 0x130, 0xF, 0xF, false));
            if (__ballot(lane < a.k && next > -INFINITY && near_keys(mine, next, unit))) {
                // told apart in 64 bits, if nobody outside can stand among the first k
                const float least = lane_value(mine, n - 1), kth = lane_value(mine, min(a.k, n) - 1);
                exact = n < total && near_keys(kth, least, unit);
                if (!exact)
                    at = rank_f64<NR>(a, x, values, n, at);
            }
        }
    } else {
        exact = true;
    }
    id = -1;
    float s = 0.0f;
    if (!exact) {
#pragma unroll
        for (int r = 0; r < NR; r++)
            values[NR * lane + r] = x[r];
        id = lane < a.k ? at : -1;
        if (id >= 0) {
            const float v = values[id];
            s = a.softmax ? quotient(expf(v - top), all) : 1.0f / (1.0f + expf(-v));
        }
    }
    const float sum = wave_sum(s);
    // (a score below 2^-90, whose e^-x or own value f32 holds with few bits or not at
    // all, is taken in 64 bits as well)
    if (exact || __ballot(id >= 0 && s < 0x1p-90f)) {
        double s64[NR], k64[NR];
        const Exact e64 = exact_of<NR>(a, x);
#pragma unroll
        for (int r = 0; r < NR; r++) {
            s64[r] = x[r] > -INFINITY ? e64.score(x[r]) : 0.0;
            k64[r] = key[r] == -INFINITY ? -INFINITY : a.bias ? s64[r] + (double)b[r] : (double)x[r];
        }
        const Choice c = choose_f64<NR>(a, s64, k64);
        id = lane < a.k ? c.id : -1;
        const double sc = id >= 0 ? c.score : 0.0;
        const double total64 = wave_sum_f64(sc);
        weight = (float)((a.renorm ? (total64 > 0.0 ? sc / total64 : 0.0) : sc) * (double)a.factor);
        return;
    }
    weight = (a.renorm ? quotient(s, sum > 0.0f ? sum : 1.0f) : s) * a.factor;
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
__global__ __launch_bounds__(64 * kWaves) void route_kernel(Routing a, Groups gr, int block,
                                                            uint8_t *counts, int pitch)
{
    __shared__ u64 mask[64 * NR];
    __shared__ int32_t ids_s[kBlockTokens * kMaxChosen];
    __shared__ int start[64 * NR];
    __shared__ int part[kWaves];
    __shared__ __attribute__((aligned(8))) float values[kWaves][NR > 1 ? 64 * NR : 128];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int t0 = blockIdx.x * block;
    for (int i = tid; i < 64 * NR; i += 64 * kWaves)
        mask[i] = 0;
    float b[NR];
    int gbit[NR];
    // a class of f32: NaN and +inf, or the finite ones
    constexpr int kOdd = 0x203, kFinite = 0x1F8;
    bool known[NR];
    bool odd = false;
    const auto logits = [&](int t, float (&x)[NR]) {
        const int64_t row = (int64_t)t * a.stride;
#pragma unroll
        for (int r = 0; r < NR; r++) {
            const int e = NR * lane + r;
            x[r] = -INFINITY;
            if (e < a.E)
                x[r] = BF16 ? bf16_lo(((const uint16_t *)a.logits + row)[e])
                            : ((const float *)a.logits + row)[e];
        }
    };
    const int t1 = min(t0 + block, a.T);
    float slack = a.bias ? 0.3f : 1.4f, ahead[NR];   // (of scores, of normal logits)
    if (t0 + wv < t1)
        logits(t0 + wv, ahead);
#pragma unroll
    for (int r = 0; r < NR; r++) {
        const int e = NR * lane + r;
        b[r] = a.bias && e < a.E ? a.bias[e] : 0.0f;
        odd |= __builtin_amdgcn_classf(b[r], kOdd);
        known[r] = e < a.E && __builtin_amdgcn_classf(b[r], kFinite);
        gbit[r] = gr.lanes || e >= a.E ? 0 : e / (a.E / a.groups) * gr.spread;
    }
    __syncthreads();
    for (int t = t0 + wv; t < t1; t += kWaves) {
        float x[NR];
#pragma unroll
        for (int r = 0; r < NR; r++) {
            odd |= __builtin_amdgcn_classf(ahead[r], kOdd);
            x[r] = known[r] && __builtin_amdgcn_classf(ahead[r], kFinite) ? ahead[r] : -INFINITY;
        }
        if (t + kWaves < t1)
            logits(t + kWaves, ahead);
        int id;
        float weight;
        choose<NR>(a, gr, x, b, gbit, values[wv], slack, id, weight);
        if (lane < a.k) {
            const int64_t first = (int64_t)t * a.k;
            (a.ids + first)[lane] = id;
            (a.weights + first)[lane] = weight;
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
    for (int i = tid; i < (t1 - t0) * a.k; i += 64 * kWaves) {
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
                                                            const int32_t *segments, int tokens,
                                                            int blocks, int pitch)
{
    __shared__ u64 mask[kMaxExperts];
    __shared__ int before_s[kMaxExperts], all_s[kMaxExperts], part[kWaves];
    const int tid = threadIdx.x, block = blockIdx.x, t0 = block * tokens;
    const int n = (min(t0 + tokens, a.T) - t0) * a.k;
    const int32_t *ids = a.ids + (int64_t)t0 * a.k;
    const int id0 = tid < n ? ids[tid] : -1;        // on its way beside the counts
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
#pragma unroll 16
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
    const auto id_of = [&](int i) { return i == tid ? id0 : ids[i]; };
    for (int i = tid; i < n; i += 64 * kWaves) {
        const int e = id_of(i);
        if (e >= 0)
            atomicOr(&mask[e], 1ull << (i / a.k));
    }
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
        const int e = id_of(i);
        if (e >= 0)
            a.order[before_s[e] + __popcll(mask[e] & ((1ull << (i / a.k)) - 1))] = t0 * a.k + i;
    }
}

int pitch_of(int32_t E) { return (E + 15) / 16 * 16; }
// A block's tokens: a multiple of one a wavefront that makes kMostBlocks blocks at
// most, and all of a call's that one block holds, which needs one launch and no
// workspace.  777 tokens of 60 experts in blocks of 16 and of 64: 9.7 and 14 us, of 256
// experts 13 and 24; 16384 in blocks of 32 and of 64: 38 and 28 us, whose blocks each
// add up the counts of all.  17, 33 and 64 tokens of 256 experts in one block 9.7, 13.0
// and 20.6 us, in blocks of 16 and two launches 11.6, 11.7 and 12.0.
int64_t block_of(int64_t T)
{
    const int64_t n = (T + kMostBlocks * kWaves - 1) / (kMostBlocks * kWaves) * kWaves;
    return T <= kBlockTokens || n > kBlockTokens ? kBlockTokens : n;
}
int64_t blocks_of(int64_t T) { return (T + block_of(T) - 1) / block_of(T); }
size_t counts_bytes(int64_t blocks, int32_t E) { return ((size_t)(blocks * pitch_of(E)) + 255) & ~(size_t)255; }

template <bool BF16, int NR>
void launch_scores(const Routing &r, uint8_t *counts, const Launch &l)
{
    // groups of whole lanes, a power of two of them, or looked through in LDS
    const int size = r.E / r.groups;
    Groups gr{size / NR, size % NR == 0 && (size / NR & (size / NR - 1)) == 0};
    if (!gr.lanes)
        for (gr.spread = 64; gr.spread * r.groups > 64;)
            gr.spread /= 2;
    dispatch(route_kernel<BF16, NR>, dim3((unsigned)blocks_of(r.T)), dim3(64 * kWaves), l, true,
             !counts, r, gr, (int)block_of(r.T), counts, pitch_of(r.E));
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
    // (calls of fewer tokens may have smaller and so more blocks, up to kMostBlocks: a
    // workspace serves them too)
    const int64_t small = (T + kWaves - 1) / kWaves, most = small < kMostBlocks ? small : kMostBlocks;
    size_t n = counts_bytes(most > blocks ? most : blocks, E);
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
        int32_t *sums = blocks > kMostBlocks ? (int32_t *)(counts + counts_bytes(blocks, r.E)) : nullptr;
        if (sums)
            dispatch(segment_kernel, dim3((unsigned)((blocks + kSegment - 1) / kSegment)), dim3(256),
                     l, false, false, (const uint8_t *)counts, sums, (int)blocks, pitch_of(r.E));
        dispatch(place_kernel, dim3((unsigned)blocks), dim3(64 * kWaves), l, false, true, r,
                 (const uint8_t *)counts, (const int32_t *)sums, (int)block_of(r.T), (int)blocks,
                 pitch_of(r.E));
    }
    return launch_status("engram route kernels");
}

}  // namespace engram
