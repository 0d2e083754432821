// The position rotation of a step's queries and keys, and the append of its
// keys and values to the paged 8-bit cache.
//
// One launch with two kinds of workgroup: the keys or the values of one page
// and head, or a run of tokens' queries.  Bound by memory: a key or value is
// read once as bf16 and written once as a code, and stays in registers between
// the page's maximum and the codes; a query's angles are formed once a token.
#include "attention.h"

namespace engram {
namespace {

constexpr int kThreads = 256;

// cos and sin of a 64-bit angle, rounded to f32.  The angle less the nearest
// multiple n of pi/2 (pi/2 as the sum of two doubles, so the remainder keeps
// an absolute error below 2^-60 n), then the Taylor series to x^13 and x^14
// on [-pi/4, pi/4] (next term below 2^-44), swapped and signed by n mod 4.
struct Turn {
    float c, s;
};
__device__ __forceinline__ Turn turn_of(int pos, float freq)
{
    const double a = (double)pos * (double)freq;
    const double n = rint(a * 0.63661977236758134308);
    const double x = fma(-n, 6.123233995736766036e-17, fma(-n, 1.57079632679489661923, a));
    const double z = x * x;
    double s = 1.0 / 6227020800.0, c = -1.0 / 87178291200.0;
    s = fma(s, z, -1.0 / 39916800.0);
    c = fma(c, z, 1.0 / 479001600.0);
    s = fma(s, z, 1.0 / 362880.0);
    c = fma(c, z, -1.0 / 3628800.0);
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

__device__ __forceinline__ void load8(const uint16_t *p, const Place &at, float (&v)[8])
{
    const u32x2 a = *(const u32x2 *)(p + at.i0), b = *(const u32x2 *)(p + at.i1);
    v[0] = bf16_lo(a.x);
    v[1] = bf16_hi(a.x);
    v[2] = bf16_lo(a.y);
    v[3] = bf16_hi(a.y);
    v[4] = bf16_lo(b.x);
    v[5] = bf16_hi(b.x);
    v[6] = bf16_lo(b.y);
    v[7] = bf16_hi(b.y);
}

__device__ __forceinline__ void turn8(float (&v)[8], const Place &at, bool halves, const Turn (&t)[4])
{
    if (at.pair < 0)
        return;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        float &a = v[halves ? i : 2 * i], &b = v[halves ? 4 + i : 2 * i + 1];
        const float x = a, y = b;
        a = x * t[i].c - y * t[i].s;
        b = x * t[i].s + y * t[i].c;
    }
}

constexpr int kRunTokens = 8;       // tokens a queries' workgroup takes at most

struct AppendArgs {
    engram_cache c;
    Seqs s;
    Heads k, v, q;
    uint16_t *q_out;
    Rotation r;
    int32_t q_heads, pieces;    // grid: keys and values of `pieces` x kv_heads pages,
    int32_t run;                // then queries, `run` tokens a workgroup
};

// The keys (z 0) or values (z 1) of one page and key head.
template <int D, bool HALVES>
__device__ __forceinline__ void append_page(const AppendArgs &a, const Seq &q, int blk,
                                            int32_t page, int h, bool z)
{
    constexpr int E = D / 8;                    // threads a token
    constexpr int TOK = kThreads / E;           // tokens at a time
    constexpr int N = kPage / TOK;
    __shared__ float part[kThreads / 64];
    const int tid = threadIdx.x, e = tid % E, g = tid / E;
    const int page0 = blk * kPage;
    const int older = max(q.start - page0, 0);
    const int last = min(q.start + q.n - page0, kPage);
    const int64_t at = (int64_t)page * a.c.kv_heads + h;
    const Heads &src = z ? a.v : a.k;
    uint8_t *codes = (z ? a.c.d_v : a.c.d_k) + at * kPage * D;
    float *scale = (z ? a.c.d_v_scales : a.c.d_k_scales) + at;
    Rotation r = a.r;
    r.halves = HALVES;
    if (z)
        r.rot = 0;
    const Place pl = place_of<D>(e, r);
    float v[N][8];
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < N; i++) {
        const int slot = g + TOK * i;
        if (slot >= older && slot < last) {
            const int pos = page0 + slot;
            load8(src.p + (q.t0 + (int64_t)(pos - q.start)) * src.token + h * src.head, pl, v[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < N; i++) {
        const int slot = g + TOK * i;
        if (slot >= older && slot < last) {
            if (!z && pl.pair >= 0) {
                Turn t[4];
#pragma unroll
                for (int j = 0; j < 4; j++)
                    t[j] = turn_of(page0 + slot, r.freq[pl.pair + j]);
                turn8(v[i], pl, HALVES, t);
            }
#pragma unroll
            for (int j = 0; j < 8; j++)
                amax = fmaxf(amax, finite_abs(v[i][j]));
        }
    }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1)
        amax = fmaxf(amax, __shfl_xor(amax, m));
    if ((tid & 63) == 0)
        part[tid >> 6] = amax;
    const float had = older > 0 ? *scale : 0.0f;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 64; i++)
        amax = fmaxf(amax, part[i]);
    const float need = exp2_int(e4m3_scale_exp(amax));
    const float now = fmaxf(had, need);
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
        if (slot >= older && slot < last) {
            uint8_t *p = codes + slot * D;
            *(uint32_t *)(p + pl.i0) = e4m3x4(v[i][0] * inv, v[i][1] * inv, v[i][2] * inv, v[i][3] * inv);
            *(uint32_t *)(p + pl.i1) = e4m3x4(v[i][4] * inv, v[i][5] * inv, v[i][6] * inv, v[i][7] * inv);
        }
    }
    if (tid == 0)                           // all have read it before the barrier
        *scale = now;
}

template <int D, bool HALVES>
__global__ __launch_bounds__(kThreads) void append_kernel(AppendArgs a)
{
    __shared__ int tok_s[kRunTokens], pos_s[kRunTokens];
    __shared__ Turn turn_s[kRunTokens][D / 2];
    const int tid = threadIdx.x;
    const int pages = 2 * a.pieces * a.c.kv_heads;
    if (blockIdx.x == 0)
        for (int i = tid; i < a.s.B; i += kThreads)
            if (seq_at(a.s, i).bad)
                raise(a.s.err, ENGRAM_DEVERR_SEQUENCE);
    if ((int)blockIdx.x < pages) {
        const bool z = blockIdx.x & 1;
        const int h = blockIdx.x / 2 % a.c.kv_heads;
        int i = blockIdx.x / 2 / a.c.kv_heads, b, piece;
        const auto touched = [&](int x) {
            const Seq q = seq_at(a.s, x);
            return q.bad || q.n == 0 ? 0 : (q.start + q.n - 1) / kPage - q.start / kPage + 1;
        };
        if (!a.s.cu) {                          // every sequence has room for as many pages
            const int each = a.pieces / a.s.B;
            b = i / each;
            piece = i % each;
            if (piece >= touched(b))
                return;
        } else if (!find_piece(i, a.s.B, touched, b, piece)) {
            return;
        }
        const Seq q = seq_at(a.s, b);
        const int blk = q.start / kPage + piece;
        const int32_t page = a.s.pages[(int64_t)b * a.s.max_pages + blk];
        if (page < 0 || page >= a.c.n_pages) {
            if (h == 0 && tid == 0)
                raise(a.s.err, ENGRAM_DEVERR_PAGE);
            return;
        }
        append_page<D, HALVES>(a, q, blk, page, h, z);
        return;
    }
    // queries: where the run's tokens lie, their angles, then eight values a thread
    const int t0 = (blockIdx.x - pages) * a.run;
    for (int i = tid >> 6; i < a.run; i += kThreads / 64) {
        int b = 0, piece = 0;
        bool found;
        if (!a.s.cu) {
            b = (t0 + i) / a.s.each;
            piece = (t0 + i) % a.s.each;
            found = t0 + i < a.s.T;
        } else {
            found = find_piece(t0 + i, a.s.B,
                               [&](int x) {
                                   const Seq q = seq_at(a.s, x);
                                   return q.bad ? 0 : q.n;
                               },
                               b, piece);
        }
        if ((tid & 63) == 0) {
            const Seq q = found ? seq_at(a.s, b) : Seq{0, 0, 0, true};
            tok_s[i] = q.bad ? -1 : q.t0 + piece;
            pos_s[i] = q.start + piece;
        }
    }
    __syncthreads();
    for (int i = tid; i < a.run * (a.r.rot / 2); i += kThreads) {
        const int t = i / (a.r.rot / 2), p = i % (a.r.rot / 2);
        if (tok_s[t] >= 0)
            turn_s[t][p] = turn_of(pos_s[t], a.r.freq[p]);
    }
    __syncthreads();
    constexpr int E = D / 8, ROWS = kThreads / E, AT_ONCE = 4;
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
            run[i] = row / a.q_heads;
            head[i] = row - run[i] * a.q_heads;
            tok[i] = row < a.run * a.q_heads ? tok_s[run[i]] : -1;
            if (tok[i] >= 0)
                load8(a.q.p + (int64_t)tok[i] * a.q.token + head[i] * a.q.head, pl, v[i]);
        }
#pragma unroll
        for (int i = 0; i < AT_ONCE; i++) {
            if (tok[i] < 0)
                continue;
            if (pl.pair >= 0) {
                Turn t[4];
#pragma unroll
                for (int j = 0; j < 4; j++)
                    t[j] = turn_s[run[i]][pl.pair + j];
                turn8(v[i], pl, HALVES, t);
            }
            uint16_t *o = a.q_out + ((int64_t)tok[i] * a.q_heads + head[i]) * D;
            u32x2 lo, hi;
            lo.x = pack_bf16x2(v[i][0], v[i][1]);
            lo.y = pack_bf16x2(v[i][2], v[i][3]);
            hi.x = pack_bf16x2(v[i][4], v[i][5]);
            hi.y = pack_bf16x2(v[i][6], v[i][7]);
            *(u32x2 *)(o + pl.i0) = lo;
            *(u32x2 *)(o + pl.i1) = hi;
        }
    }
}

template <int D>
void launch_dim(const AppendArgs &a, const Launch &l)
{
    const unsigned runs = a.q_heads ? (a.s.T + a.run - 1) / a.run : 0;
    const dim3 grid(2u * a.pieces * a.c.kv_heads + runs), block(kThreads);
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
                       (int32_t)(run < 1 ? 1 : run > kRunTokens ? kRunTokens : run)};
    if (c.head_dim == 64)
        launch_dim<64>(a, l);
    else if (c.head_dim == 128)
        launch_dim<128>(a, l);
    else
        launch_dim<256>(a, l);
    return launch_status("engram cache_append kernel");
}

}  // namespace engram
