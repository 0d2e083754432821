// Pieces that the attention kernels share: matrix-core types, the split of a
// query into two 8-bit parts, the masks' bounds, partial results.
#pragma once

#include "attention.h"

namespace engram {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr float kLog2e = 1.44269504088896340736f;
// E8M0 scale of a query's second part, which is held 2^4 times larger: the
// residual of e4m3's four bits is at most 2^-4 of the value.
constexpr int kOne = 127, kLoScale = 127 - 4;

// Thirty-two bf16 query values as two e4m3 parts, q = 2^k (hi + lo / 16):
// bf16 has eight significant bits and each part four.  The row's largest value
// lies in (224, 448] and lo's finest step is 2^-9 / 16 = 2^-13, so eight bits
// fit down to values of 2^-6, which is 2^-13.8 of the largest or less; below, a
// value is off by at most 2^-14, 2^-21.8 of the largest.  The matrix
// instructions then take keys as the codes they are.  They cut the products of
// eight neighbours towards zero below 2^-13 of the largest one's power of two
// and add in f32: some 2^-16 of a logit's size for normal values, little beside
// the keys' four bits, where bf16 products would need every key widened and
// staged at twice its bytes.
__device__ __forceinline__ void split_query(const u32x4 (&x)[4], float inv, i32x8 &hi, i32x8 &lo)
{
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const uint32_t a = i & 1 ? x[i / 2].z : x[i / 2].x, b = i & 1 ? x[i / 2].w : x[i / 2].y;
        const float v0 = bf16_lo(a) * inv, v1 = bf16_hi(a) * inv, v2 = bf16_lo(b) * inv,
                    v3 = bf16_hi(b) * inv;
        const uint32_t h = e4m3x4(v0, v1, v2, v3);
        hi[i] = (int)h;
        lo[i] = (int)e4m3x4((v0 - e4m3_at<0>(h)) * 16.0f, (v1 - e4m3_at<1>(h)) * 16.0f,
                            (v2 - e4m3_at<2>(h)) * 16.0f, (v3 - e4m3_at<3>(h)) * 16.0f);
    }
}

__device__ __forceinline__ float amax_bf16(const u32x4 (&x)[4])
{
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
        for (int j = 0; j < 4; j++)
            a = fmaxf(a, fmaxf(fabsf(bf16_lo(x[i][j])), fabsf(bf16_hi(x[i][j]))));
    return a;
}

template <bool HALF>
__device__ __forceinline__ uint32_t widen2(uint32_t x)
{
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, 1.0f, HALF));
}

// Each byte of x that is a NaN code -> 0xFF in the result.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t x)
{
    const uint32_t top = ((x & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
    return (top >> 7) * 0xFFu;
}

// What the attention kernels get beside the cache and the sequences.
struct AttendArgs {
    engram_cache c;
    Seqs s;
    Heads q;
    uint16_t *out;
    int32_t heads, g;         // query heads, query heads a key head
    float scale;              // of the logits, times log2(e)
    int32_t window;           // 0 = none (a window past every position counts as none)
    int32_t window_pages;     // pages a tile's windows meet at most, 0 = no bound
    int32_t parts, least;     // workgroups that share the pages; pages each takes at least
    int32_t join_rows;        // rows of a unit that the join provides for
    int32_t splits;           // workgroups that share a 128-row tile's pages
    float *part;              // partial results: two places a workgroup (128-row tiles: one)
};

// A partial result: kRows rows of m, of l, then of D output sums.
constexpr int kRows = 16;
constexpr int64_t part_floats(int d) { return kRows * (int64_t)(d + 2); }

// A row tile: 16 rows of one sequence and key head.  Row r is query head
// h*g + r % g of the sequence's token r / g.
struct RowTile {
    int32_t b, h, row0, rows;     // rows of the sequence: n * g
    Seq q;
};

// A row's parts first, first + by, ... < n, joined for four output values: the
// running maximum and sum again, U parts' loads under way at a time.  place(i)
// is part i: ROWS rows of m, of l, then of D sums.
struct Joined {
    float m, l;
    f32x4 acc;
    __device__ __forceinline__ void add(float pm, float pl, const f32x4 &po)
    {
        const float top = fmaxf(m, pm), zero = top == -INFINITY ? 0.0f : top;
        const float k = __builtin_amdgcn_exp2f(m - zero), pk = __builtin_amdgcn_exp2f(pm - zero);
        m = top;
        l = k * l + pk * pl;
        acc = k * acc + pk * po;
    }
};
template <int D, int ROWS, int U, class P>
__device__ __forceinline__ Joined join_row(int first, int by, int n, int r, int d, P place)
{
    Joined j{-INFINITY, 0.0f, {0.0f, 0.0f, 0.0f, 0.0f}};
    for (int i = first; i < n; i += U * by) {
        float m[U], l[U];
        f32x4 o[U];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const float *x = place(min(i + u * by, n - 1));
            m[u] = x[r];
            l[u] = x[ROWS + r];
            o[u] = *(const f32x4 *)(x + 2 * ROWS + r * D + d);
        }
#pragma unroll
        for (int u = 0; u < U; u++)
            if (i + u * by < n)
                j.add(m[u], l[u], o[u]);
    }
    return j;
}

// Row tiles of the many-row kernel (attend_prompt.hip) in a call, times heads,
// and the workspace that it needs.
int64_t prompt_tiles(const engram_cache &c, const Seqs &s, int32_t g);
size_t prompt_bytes(const engram_cache &c, const Seqs &s, int32_t g);
int32_t launch_attend_prompt(const AttendArgs &a, const Launch &l);

}  // namespace engram
