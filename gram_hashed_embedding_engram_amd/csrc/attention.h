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

// Sequence b: its first token, how many it brings and the position of the
// first; n = 0 with `bad` set where its bounds do not hold.
struct Seq {
    int32_t t0, n, start;
    bool bad;
};

__device__ __forceinline__ Seq seq_at(const Seqs &s, int b)
{
    Seq q;
    int32_t t1;
    if (s.cu) {
        q.t0 = s.cu[b];
        t1 = s.cu[b + 1];
    } else {
        q.t0 = b * s.each;
        t1 = q.t0 + s.each;
    }
    q.start = s.start[b];
    const bool tokens = q.t0 >= 0 && t1 >= q.t0 && t1 <= s.T;
    q.n = tokens ? t1 - q.t0 : 0;
    q.bad = !tokens || q.start < 0 ||
            (int64_t)q.start + q.n > (int64_t)s.max_pages * kPage;
    return q;
}

__device__ __forceinline__ void raise(int32_t *err, int32_t bits)
{
    if (err)
        atomicOr(err, bits);
}

// Inclusive sum over the wavefront's lanes, in data-parallel moves: within
// rows of 16 lanes by shifts of 1, 2, 4, 8, then rows 0 and 2 into 1 and 3 and
// row 1 into 2 and 3.
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_iadd(int v)
{
    return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ int wave_scan(int v)
{
    v = dpp_iadd<0x111, 0xF>(v);
    v = dpp_iadd<0x112, 0xF>(v);
    v = dpp_iadd<0x114, 0xF>(v);
    v = dpp_iadd<0x118, 0xF>(v);
    v = dpp_iadd<0x142, 0xA>(v);
    v = dpp_iadd<0x143, 0xC>(v);
    return v;
}

// Work item i of a grid laid over the sequences: finds the sequence b and the
// piece of it, where sequence b has pieces(b) of them, in order.  Called by
// whole wavefronts with a uniform i; false past the last item.
template <class F>
__device__ __forceinline__ bool find_piece(int i, int B, F pieces, int &b, int &piece)
{
    const int lane = threadIdx.x & 63;
    for (int base = 0; base < B; base += 64) {
        const int own = base + lane < B ? pieces(base + lane) : 0;
        const int sum = wave_scan(own);
        const uint64_t over = __ballot(sum > i);
        if (over) {
            const int at = __builtin_ctzll(over);
            b = base + at;
            piece = i - __builtin_amdgcn_readlane(sum - own, at);
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
