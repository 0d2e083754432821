// Shared pieces of the attention sub-layer's kernels (norm.hip, w4.hip,
// cache_append.hip, cache_attend.hip): 8-bit codes and their scales, the
// sequences of a step, the launchers.  Internal to the library.
#pragma once

#include <float.h>

#include "common.h"

namespace engram {

constexpr int kPage = ENGRAM_PAGE_TOKENS;

// ---------------------------------------------------------------- device

// Exponent k of the least 2^k, k >= -126, with amax <= 448 * 2^k.  From the
// bits: amax = 1.m * 2^e, and 448 = 1.75 * 2^8, so k = e - 8, one more where
// 1.m > 1.75.  Subnormal amax (e = -127 here) falls under the floor.
__device__ __forceinline__ int e4m3_scale_exp(float amax)
{
    const uint32_t u = __float_as_uint(fminf(amax, FLT_MAX));
    const int k = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return k < -126 ? -126 : k;
}

// 2^k for k in -126..127.
__device__ __forceinline__ float exp2_int(int k) { return __uint_as_float((uint32_t)(k + 127) << 23); }

// |x|, or 0 where x is not finite (a scale covers finite values only).
__device__ __forceinline__ float finite_abs(float x)
{
    const float a = fabsf(x);
    return a <= FLT_MAX ? a : 0.0f;
}

// Four f32 -> four e4m3 codes, first in the low byte (round to nearest even;
// the callers' values lie within +-448 or are not finite, which gives NaN).
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d)
{
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
}

// Two f32 -> two bf16, first in the low half (the hardware's rounding, to
// nearest even; NaN stays NaN).
typedef float f32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t cvt_bf16x2(float a, float b)
{
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, b2));
}

// Byte I of a dword of e4m3 codes as f32.
template <int I>
__device__ __forceinline__ float e4m3_at(uint32_t w)
{
    return __builtin_amdgcn_cvt_f32_fp8((int)w, I);
}

// max / sum over lanes l and l ^ 32 (both get it)
__device__ __forceinline__ float max_x32(float v)
{
    const uint32_t u = __float_as_uint(v);
    auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float add_x32(float v)
{
    const uint32_t u = __float_as_uint(v);
    auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// max / sum over lanes l, l ^ 16, l ^ 32, l ^ 48
__device__ __forceinline__ float max_x16(float v)
{
    const uint32_t u = __float_as_uint(v);
    auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    return max_x32(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float add_x16(float v)
{
    const uint32_t u = __float_as_uint(v);
    auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    return add_x32(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

// The sequences of a step, as the kernels see them: T tokens, `each` tokens a
// sequence where cu is null.
struct Seqs {
    const int32_t *pages, *start, *cu;
    int32_t *err;
    int32_t B, max_pages;
    int32_t T, each;
};

// A sequence: its first token, how many it brings and the position of the
// first; n = 0 with `bad` set where its token bounds do not hold.
struct Seq {
    int32_t t0, n, start;
    bool bad;
};

__device__ __forceinline__ Seq make_seq(const Seqs &s, int32_t t0, int32_t n, int32_t start,
                                        bool tokens)
{
    Seq q{t0, tokens ? n : 0, start, false};
    q.bad = !tokens || start < 0 || (int64_t)start + q.n > (int64_t)s.max_pages * kPage;
    return q;
}

// Sequence b of a call without token bounds.
__device__ __forceinline__ Seq even_seq(const Seqs &s, int b)
{
    return make_seq(s, b * s.each, s.each, s.start[b], true);
}

__device__ __forceinline__ void raise(int32_t *err, int32_t bits)
{
    if (err)
        atomicOr(err, bits);
}

// Inclusive sum (or, of values >= 0, maximum) over the wavefront's lanes, in
// data-parallel moves: within rows of 16 lanes by shifts of 1, 2, 4, 8, then
// rows 0 and 2 into 1 and 3 and row 1 into 2 and 3.
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_from(int v)
{
    return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ int wave_scan(int v)
{
    v += dpp_from<0x111, 0xF>(v);
    v += dpp_from<0x112, 0xF>(v);
    v += dpp_from<0x114, 0xF>(v);
    v += dpp_from<0x118, 0xF>(v);
    v += dpp_from<0x142, 0xA>(v);
    v += dpp_from<0x143, 0xC>(v);
    return v;
}
__device__ __forceinline__ int wave_max_scan(int v)
{
    v = max(v, dpp_from<0x111, 0xF>(v));
    v = max(v, dpp_from<0x112, 0xF>(v));
    v = max(v, dpp_from<0x114, 0xF>(v));
    v = max(v, dpp_from<0x118, 0xF>(v));
    v = max(v, dpp_from<0x142, 0xA>(v));
    v = max(v, dpp_from<0x143, 0xC>(v));
    return v;
}

// Sequences base .. base+63, one a lane (no tokens past the last).  With token
// bounds a sequence may not begin before the end of an earlier one: no token
// counts twice, so that a call's sequences never bring more than its T tokens,
// which its grid, its workspace and 32-bit counts are laid out for.  reach: the
// furthest end of the sequences before base, moved on past these.
__device__ __forceinline__ Seq seqs_at(const Seqs &s, int base, int32_t &reach)
{
    const int b = base + (threadIdx.x & 63);
    const Seq none{0, 0, 0, false};
    if (!s.cu)
        return b < s.B ? even_seq(s, b) : none;
    const bool in = b < s.B;
    const int32_t t0 = in ? s.cu[b] : 0, t1 = in ? s.cu[b + 1] : 0, start = in ? s.start[b] : 0;
    const bool own = t0 >= 0 && t1 >= t0 && t1 <= s.T;
    const int ends = wave_max_scan(own ? t1 : 0);
    const int before = max((int)reach, dpp_from<0x138, 0xF>(ends));     // up to lane l - 1
    reach = max((int)reach, __builtin_amdgcn_readlane(ends, 63));
    return in ? make_seq(s, t0, t1 - t0, start, own && t0 >= before) : none;
}

__device__ __forceinline__ Seq lane_seq(const Seq &q, int l)
{
    return Seq{__builtin_amdgcn_readlane(q.t0, l), __builtin_amdgcn_readlane(q.n, l),
               __builtin_amdgcn_readlane(q.start, l), (bool)__builtin_amdgcn_readlane(q.bad, l)};
}

// Sequences whose bounds do not hold set their error bit (one workgroup of a
// call; whole wavefronts).
__device__ __forceinline__ void raise_bad(const Seqs &s)
{
    if (!s.cu) {
        for (int b = threadIdx.x; b < s.B; b += blockDim.x)
            if (even_seq(s, b).bad)
                raise(s.err, ENGRAM_DEVERR_SEQUENCE);
    } else if (threadIdx.x < 64) {
        int32_t reach = 0;
        for (int base = 0; base < s.B; base += 64)
            if (seqs_at(s, base, reach).bad)
                raise(s.err, ENGRAM_DEVERR_SEQUENCE);
    }
}

// Work item i of a grid laid over sequences with token bounds: finds the
// sequence b, which is q, and the piece of it, where a sequence has pieces(q) of
// them (none if it brings no token), in order.  Called by whole wavefronts with
// a uniform i; false past the last item.
template <class F>
__device__ __forceinline__ bool find_piece(int i, const Seqs &s, F pieces, int &b, int &piece, Seq &q)
{
    int32_t reach = 0;
    for (int base = 0; base < s.B; base += 64) {
        const Seq lane = seqs_at(s, base, reach);
        const int own = pieces(lane);
        const int sum = wave_scan(own);
        const uint64_t over = __ballot(sum > i);
        if (over) {
            const int at = __builtin_ctzll(over);
            b = base + at;
            piece = i - __builtin_amdgcn_readlane(sum - own, at);
            q = lane_seq(lane, at);
            return true;
        }
        i -= __builtin_amdgcn_readlane(sum, 63);
    }
    return false;
}

// ------------------------------------------------------------------ host

// bf16 heads in memory: head h of token t at p + t*token + h*head.
struct Heads {
    const uint16_t *p;
    int64_t token, head;
};

struct Rotation {
    const float *freq;
    int32_t rot, halves;
};

int32_t launch_add_norm(const uint16_t *x, const void *res, bool res_bf16, const uint16_t *w,
                        float eps, void *sum, uint8_t *codes, uint8_t *scales, int64_t rows,
                        int64_t dim, const Launch &l);
int32_t launch_w4(const void *x, const uint8_t *xs, const uint8_t *w, const uint8_t *ws,
                  uint16_t *y, int64_t T, int64_t K, int64_t N, const Launch &l);
int32_t launch_append(const engram_cache &c, const Seqs &s, const Heads &k, const Heads &v,
                      const Heads &q, uint16_t *q_out, int32_t q_heads, const Rotation &r,
                      const Launch &l);
size_t attend_bytes(const engram_cache &c, const Seqs &s, int32_t q_heads);
int32_t launch_attend(const engram_cache &c, const Seqs &s, const Heads &q, uint16_t *out,
                      int32_t q_heads, float scale, int64_t window, void *ws, const Launch &l);

}  // namespace engram
