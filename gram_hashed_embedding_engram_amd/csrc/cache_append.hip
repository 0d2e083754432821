// The position rotation of a step's queries and keys, and the append of its
// keys and values to the paged 8-bit cache.
//
// One launch with two kinds of workgroup: the keys or the values of one page,
// of one or several heads in turn, or a run of tokens' queries.  Bound by memory:
// a key or value is read once as bf16 and written once as a code, and stays in
// registers between the page's maximum and the codes.  Angles, whose 64-bit
// reduction and series are most of the arithmetic, are formed once a workgroup
// and token and wait in LDS.
//
// Ragged prompts of 4096 tokens at most (338 MB for 48 heads of 128): 71 us, 4.7
// TB/s, where a plain copy reaches 5.0.  A step of 64 single tokens: 7 us.
#include "attention.h"

namespace engram {
namespace {

// Threads a workgroup: twice as many where a page's angles take 64 KiB of LDS.
template <int D>
constexpr int threads_of = D == 256 ? 512 : 256;

// cos and sin of a 64-bit angle, rounded to f32.  The angle less the nearest
// multiple n of pi/2 (pi/2 as the sum of two doubles, so the remainder keeps
// an absolute error below 2^-60 n), then the Taylor series to x^11 and x^10
// on [-pi/4, pi/4] (next terms below 2^-33, far under f32's half step),
// swapped and signed by n mod 4.
struct Turn {
    float c, s;
};
__device__ __forceinline__ Turn turn_of(int pos, float freq)
{
    const double a = (double)pos * (double)freq;
    const double n = rint(a * 0.63661977236758134308);
    const double x = fma(-n, 6.123233995736766036e-17, fma(-n, 1.57079632679489661923, a));
    const double z = x * x;
    double s = -1.0 / 39916800.0, c = -1.0 / 3628800.0;
    s = fma(s, z, 1.0 / 362880.0);
    s = fma(s, z, -1.0 / 5040.0);
    c = fma(c, z, 1.0 / 40320.0);
    s = fma(s, z, 1.0 / 120.0);
    c = fma(c, z, -1.0 / 720.0);
    s = fma(s, z, -1.0 / 6.0);
    c = fma(c, z, 1.0 / 24.0);
    s = fma(s * z, x, x);
    c = fma(c, z, -0.5);
    c = fma(c, z, 1.0);
    const int q = (int)((int64_t)n & 3);
    const float fs = (float)(q & 1 ? c : s), fc = (float)(q & 1 ? s : c);
    return Turn{q == 1 || q == 2 ? -fc : fc, q & 2 ? -fs : fs};
}

// A thread's eight values of a head: values i0 .. i0+3 and i1 .. i1+3.
//   pairs (i, i + rot/2), inside the turned part: i1 = i0 + rot/2, so the
//   thread holds both ends of four pairs;
//   otherwise i1 = i0 + 4 and pairs are neighbours.
struct Place {
    int i0, i1, pair;           // pair < 0: not turned
};
template <int D>
__device__ __forceinline__ Place place_of(int e, const Rotation &r)
{
    Place p;
    if (r.halves && 8 * e < r.rot) {
        p.i0 = 4 * e;
        p.i1 = 4 * e + r.rot / 2;
        p.pair = 4 * e;
    } else {
        p.i0 = 8 * e;
        p.i1 = 8 * e + 4;
        p.pair = 8 * e < r.rot ? 4 * e : -1;
    }
    return p;
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// A thread's values, as one access where they lie side by side for all; that
// one streams past the caches (12 000 tokens of 48 heads: 77 -> 72 us), while
// two halves of a line would each fetch it that way (20 -> 25 us).
template <bool HALVES>
__device__ __forceinline__ void load8(const uint16_t *p, const Place &at, float (&v)[8])
{
    u32x4 x;
    if (HALVES) {
        const u32x2 a = *(const u32x2 *)(p + at.i0), b = *(const u32x2 *)(p + at.i1);
        x = u32x4{a.x, a.y, b.x, b.y};
    } else {
        x = __builtin_nontemporal_load((const u32x4 *)(p + at.i0));
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
        v[2 * i] = bf16_lo(x[i]);
        v[2 * i + 1] = bf16_hi(x[i]);
    }
}

template <bool HALVES>
__device__ __forceinline__ void store8(uint16_t *p, const Place &at, const float (&v)[8])
{
    const u32x2 a = {cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3])};
    const u32x2 b = {cvt_bf16x2(v[4], v[5]), cvt_bf16x2(v[6], v[7])};
    if (HALVES) {
        *(u32x2 *)(p + at.i0) = a;
        *(u32x2 *)(p + at.i1) = b;
    } else {
        __builtin_nontemporal_store(u32x4{a.x, a.y, b.x, b.y}, (u32x4 *)(p + at.i0));
    }
}

template <bool HALVES>
__device__ __forceinline__ void store8_codes(uint8_t *p, const Place &at, const float (&v)[8], float f)
{
    const uint32_t a = e4m3x4(v[0] * f, v[1] * f, v[2] * f, v[3] * f);
    const uint32_t b = e4m3x4(v[4] * f, v[5] * f, v[6] * f, v[7] * f);
    if (HALVES) {
        *(uint32_t *)(p + at.i0) = a;
        *(uint32_t *)(p + at.i1) = b;
    } else {
        *(u32x2 *)(p + at.i0) = u32x2{a, b};
    }
}

// The values' four pairs by t[0..3].
__device__ __forceinline__ void turn8(float (&v)[8], bool halves, const Turn *t)
{
#pragma unroll
    for (int i = 0; i < 4; i++) {
        float &a = v[halves ? i : 2 * i], &b = v[halves ? 4 + i : 2 * i + 1];
        const float x = a, y = b, c = t[i].c, s = t[i].s;
        a = x * c - y * s;
        b = x * s + y * c;
    }
}

// f(t, p) for tokens t < n and pairs p < half, shared out over the threads (one
// division a thread).
template <int THREADS, class F>
__device__ __forceinline__ void each_turn(int half, int n, F f)
{
    if (half == 0)
        return;
    const int dt = THREADS / half, dp = THREADS - dt * half;
    int t = threadIdx.x / half, p = threadIdx.x - t * half;
    while (t < n) {
        f(t, p);
        t += dt;
        p += dp;
        if (p >= half) {
            p -= half;
            t++;
        }
    }
}

// Tokens that a queries' workgroup and heads that a page's workgroup take at
// most: more share the angles, fewer leave more workgroups to overlap (the
// prompts above with runs of 4, 8 and 16 tokens: 73, 72 and 88 us; with 4 and 8
// heads: 77 and 72).
constexpr int kRunTokens = 8;
constexpr int kRunHeads = 8;

struct AppendArgs {
    engram_cache c;
    Seqs s;
    Heads k, v, q;
    uint16_t *q_out;
    Rotation r;
    int32_t q_heads, pieces;    // grid: keys and values of `pieces` pages, `heads` heads a
    int32_t run, heads;         // workgroup, then queries, `run` tokens a workgroup
};

// The keys (z 0) or values (z 1) of heads h0 .. h1-1 of one page.
template <int D, bool HALVES>
__device__ __forceinline__ void append_page(const AppendArgs &a, const Seq &q, int blk,
                                            int32_t page, int h0, int h1, bool z,
                                            Turn (*turns)[D / 2])
{
    constexpr int kThreads = threads_of<D>;
    constexpr int E = D / 8;                    // threads a token
    constexpr int TOK = kThreads / E;           // tokens at a time
    constexpr int N = kPage / TOK;
    __shared__ float part[2][kThreads / 64];
    const int tid = threadIdx.x, e = tid % E, g = tid / E;
    const int page0 = blk * kPage;
    const int older = max(q.start - page0, 0);
    const int last = min(q.start + q.n - page0, kPage);
    const Heads &src = z ? a.v : a.k;
    Rotation r = a.r;
    r.halves = HALVES;
    if (z)
        r.rot = 0;
    const Place pl = place_of<D>(e, r);
    const uint16_t *row[N];
#pragma unroll
    for (int i = 0; i < N; i++)
        row[i] = src.p + (q.t0 + (int64_t)(page0 + g + TOK * i - q.start)) * src.token;
    const int half = r.rot / 2;
    if (half) {
        each_turn<kThreads>(half, last - older, [&](int t, int p) {
            turns[older + t][p] = turn_of(page0 + older + t, r.freq[p]);
        });
        __syncthreads();
    }
    for (int h = h0; h < h1; h++) {
        const int64_t at = (int64_t)page * a.c.kv_heads + h;
        uint8_t *codes = (z ? a.c.d_v : a.c.d_k) + at * kPage * D;
        float *scale = (z ? a.c.d_v_scales : a.c.d_k_scales) + at;
        const float had = older > 0 ? *scale : 0.0f;
        float v[N][8];
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < N; i++) {
            const int slot = g + TOK * i;
            if (slot >= older && slot < last)
                load8<HALVES>(row[i] + h * src.head, pl, v[i]);
        }
#pragma unroll
        for (int i = 0; i < N; i++) {
            const int slot = g + TOK * i;
            if (slot >= older && slot < last) {
                if (pl.pair >= 0)
                    turn8(v[i], HALVES, &turns[slot][pl.pair]);
#pragma unroll
                for (int j = 0; j < 8; j++)
                    amax = fmaxf(amax, finite_abs(v[i][j]));
            }
        }
        amax = max_x16(amax);
#pragma unroll
        for (int m = 1; m < 16; m <<= 1)
            amax = fmaxf(amax, __shfl_xor(amax, m));
        if ((tid & 63) == 0)
            part[h & 1][tid >> 6] = amax;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kThreads / 64; i++)
            amax = fmaxf(amax, part[h & 1][i]);
        const float now = fmaxf(had, exp2_int(e4m3_scale_exp(amax)));
        if (now != had) {                       // (never where the page is new)
            const float ratio = had / now;
            for (int i = tid; i < older * (D / 4); i += kThreads) {
                uint32_t *p = (uint32_t *)codes + i;
                const uint32_t x = *p;
                *p = e4m3x4(e4m3_at<0>(x) * ratio, e4m3_at<1>(x) * ratio, e4m3_at<2>(x) * ratio,
                            e4m3_at<3>(x) * ratio);
            }
        }
        const float inv = 1.0f / now;
#pragma unroll
        for (int i = 0; i < N; i++) {
            const int slot = g + TOK * i;
            if (slot >= older && slot < last)
                store8_codes<HALVES>(codes + slot * D, pl, v[i], inv);
        }
        if (tid == 0)                           // all have read it before the barrier
            *scale = now;
    }
}

template <int D, bool HALVES>
__global__ __launch_bounds__(threads_of<D>) void append_kernel(AppendArgs a)
{
    constexpr int kThreads = threads_of<D>;
    __shared__ int tok_s[kRunTokens], pos_s[kRunTokens];
    __shared__ Turn turn_s[kPage][D / 2];
    const int tid = threadIdx.x;
    const int groups = (a.c.kv_heads + a.heads - 1) / a.heads;
    const int pages = 2 * a.pieces * groups;
    if (blockIdx.x == 0)
        raise_bad(a.s);
    if ((int)blockIdx.x < pages) {
        const bool z = blockIdx.x & 1;
        const int h = blockIdx.x / 2 % groups * a.heads;
        int i = blockIdx.x / 2 / groups, b, piece;
        Seq q;
        const auto touched = [](const Seq &x) {
            return x.bad || x.n == 0 ? 0 : (x.start + x.n - 1) / kPage - x.start / kPage + 1;
        };
        if (!a.s.cu) {                          // every sequence has room for as many pages
            const int each = a.pieces / a.s.B;
            b = i / each;
            piece = i % each;
            q = even_seq(a.s, b);
            if (piece >= touched(q))
                return;
        } else if (!find_piece(i, a.s, touched, b, piece, q)) {
            return;
        }
        const int blk = q.start / kPage + piece;
        const int32_t page = a.s.pages[(int64_t)b * a.s.max_pages + blk];
        if (page < 0 || page >= a.c.n_pages) {
            if (h == 0 && tid == 0)
                raise(a.s.err, ENGRAM_DEVERR_PAGE);
            return;
        }
        append_page<D, HALVES>(a, q, blk, page, h, min(h + a.heads, a.c.kv_heads), z, turn_s);
        return;
    }
    // queries: where the run's tokens lie, their angles, then eight values a thread
    const int t0 = (blockIdx.x - pages) * a.run;
    for (int i = tid >> 6; i < a.run; i += kThreads / 64) {
        int b = 0, piece = 0;
        Seq q{0, 0, 0, true};
        if (!a.s.cu) {
            piece = (t0 + i) % a.s.each;
            if (t0 + i < a.s.T)
                q = even_seq(a.s, (t0 + i) / a.s.each);
        } else {
            find_piece(t0 + i, a.s, [](const Seq &x) { return x.bad ? 0 : x.n; }, b, piece, q);
        }
        if ((tid & 63) == 0) {
            tok_s[i] = q.bad ? -1 : q.t0 + piece;
            pos_s[i] = q.start + piece;
        }
    }
    __syncthreads();
    const int half = a.r.rot / 2;
    each_turn<kThreads>(half, a.run, [&](int t, int p) {
        if (tok_s[t] >= 0)
            turn_s[t][p] = turn_of(pos_s[t], a.r.freq[p]);
    });
    __syncthreads();
    const float per_head = 1.0f / (float)a.q_heads;
    constexpr int E = D / 8, ROWS = kThreads / E, AT_ONCE = 2;
    const int e = tid % E;
    Rotation r = a.r;
    r.halves = HALVES;
    const Place pl = place_of<D>(e, r);
    for (int row0 = tid / E; row0 < a.run * a.q_heads; row0 += ROWS * AT_ONCE) {
        float v[AT_ONCE][8];
        int tok[AT_ONCE], head[AT_ONCE], run[AT_ONCE];
#pragma unroll
        for (int i = 0; i < AT_ONCE; i++) {
            const int row = row0 + ROWS * i;
            run[i] = (int)(((float)row + 0.5f) * per_head);      // row / q_heads, both below 2^14
            head[i] = row - run[i] * a.q_heads;
            tok[i] = row < a.run * a.q_heads ? tok_s[run[i]] : -1;
            if (tok[i] >= 0)
                load8<HALVES>(a.q.p + (int64_t)tok[i] * a.q.token + head[i] * a.q.head, pl, v[i]);
        }
#pragma unroll
        for (int i = 0; i < AT_ONCE; i++) {
            if (tok[i] < 0)
                continue;
            if (pl.pair >= 0)
                turn8(v[i], HALVES, &turn_s[run[i]][pl.pair]);
            uint16_t *o = a.q_out + ((int64_t)tok[i] * a.q_heads + head[i]) * D;
            store8<HALVES>(o, pl, v[i]);
        }
    }
}

int64_t blocks_of(const AppendArgs &a)
{
    const int64_t runs = a.q_heads ? (a.s.T + a.run - 1) / a.run : 0;
    const int64_t groups = (a.c.kv_heads + a.heads - 1) / a.heads;
    return 2 * (int64_t)a.pieces * groups + runs;
}

template <int D>
void launch_dim(const AppendArgs &a, const Launch &l)
{
    const dim3 grid((unsigned)blocks_of(a)), block(threads_of<D>);
    if (a.r.halves)
        dispatch(append_kernel<D, true>, grid, block, l, true, true, a);
    else
        dispatch(append_kernel<D, false>, grid, block, l, true, true, a);
}

}  // namespace

int32_t launch_append(const engram_cache &c, const Seqs &s, const Heads &k, const Heads &v,
                      const Heads &q, uint16_t *q_out, int32_t q_heads, const Rotation &r,
                      const Launch &l)
{
    // pages a call can touch: n tokens meet (n + 62) / 64 + 1 at most
    const int64_t pieces = s.cu ? s.T / kPage + 2 * (int64_t)s.B
                                : (int64_t)s.B * ((s.each + kPage - 2) / kPage + 1);
    if (2 * pieces * c.kv_heads + s.T >= ((int64_t)1 << 24))
        return fail(ENGRAM_E_RANGE, "engram cache_append: %lld pages of %d heads in one call",
                    (long long)pieces, c.kv_heads);
    // several tokens a workgroup once there are enough of them
    const int64_t run = s.T / (4 * device_cus());
    const AppendArgs a{c, s, k, v, q, q_out, r, q_heads, (int32_t)pieces,
                       (int32_t)(run < 1 ? 1 : run > kRunTokens ? kRunTokens : run),
                       run < 2 ? 1 : kRunHeads};
    // (a grid's threads are counted in 32 bits)
    const int64_t threads = c.head_dim == 256 ? threads_of<256> : threads_of<64>;
    if (blocks_of(a) * threads >= ((int64_t)1 << 32))
        return fail(ENGRAM_E_RANGE, "engram cache_append: %lld workgroups of %lld threads in one call",
                    (long long)blocks_of(a), (long long)threads);
    if (c.head_dim == 64)
        launch_dim<64>(a, l);
    else if (c.head_dim == 128)
        launch_dim<128>(a, l);
    else
        launch_dim<256>(a, l);
    return launch_status("engram cache_append kernel");
}

}  // namespace engram
