// Attention over the paged 8-bit cache for many rows a sequence (prompt
// chunks): tiles of 128 rows against 64-token pages staged through LDS.
#include "attend.h"

namespace engram {
namespace {

constexpr int kTileWaves = 4;
constexpr float kSlack = 8.0f;
constexpr int kTileRows = 32 * kTileWaves;

// 16-byte chunk of a staged row, moved so that eight lanes reading (or
// writing) eight rows meet different banks.
template <int D>
__device__ __forceinline__ int k_chunk(int row, int c)
{
    return D == 64 ? c ^ ((row >> 1) & 3) : c ^ (row & 7);
}
__device__ __forceinline__ int v_chunk(int d, int c) { return c ^ ((d ^ (d >> 2)) & 7); }

// A workgroup's four wavefronts take 32 rows each against the same pages.
//
// S^T = K Q^T: lane l holds query l % 32 and, of each 32 tokens, tokens
// 8j + 4(l / 32) + e.  Maximum, sum and rescaling are per lane (and lane ^ 32),
// and the probabilities, taken in the order 16s + 4h + {0..3}, 16s + 8 + 4h +
// {0..3}, are the second operand of O^T = V^T P^T as they stand.  Keys are
// staged as codes, values transposed and widened to bf16 with their tokens in
// that order.
template <int D>
__global__ __launch_bounds__(64 * kTileWaves, D == 256 ? 1 : 2) void attend_tile_kernel(AttendArgs a)
{
    constexpr int KS = D / 64, DT = D / 32, CH = D / 16;
    constexpr int KB = kPage * D, VB = 2 * kPage * D;
    constexpr int KL = KB / 16 / 256;             // 16-byte chunks of keys a thread stages
    constexpr int VL = D / 128 > 0 ? D / 128 : 1; // 8-token x 4-value blocks of values
    __shared__ __attribute__((aligned(16))) uint8_t lds_k[2][KB];
    __shared__ __attribute__((aligned(16))) uint8_t lds_v[2][VB];
    __shared__ int poison_s;          // some page held a NaN that only some rows see
    const int tid = threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r32 = lane & 31, h = lane >> 5;

    // ---- which rows
    const int kv = a.c.kv_heads;
    const int head = blockIdx.x % kv;
    const int64_t item = blockIdx.x / kv;
    int b, piece, tiles;
    if (blockIdx.x == 0)
        for (int i = tid; i < a.s.B; i += 64 * kTileWaves)
            if (seq_at(a.s, i).bad)
                raise(a.s.err, ENGRAM_DEVERR_SEQUENCE);
    if (!a.s.cu) {
        tiles = (int)(((int64_t)a.s.each * a.g + kTileRows - 1) / kTileRows);
        b = (int)(item / tiles);
        piece = (int)(item - (int64_t)b * tiles);
    } else if (!find_piece(item, a.s.B,
                           [&](int i) { return (int)(((int64_t)seq_at(a.s, i).n * a.g + kTileRows - 1) / kTileRows); },
                           b, piece)) {
        return;
    }
    const Seq q = seq_at(a.s, b);
    const int rows = q.n * a.g;
    tiles = (rows + kTileRows - 1) / kTileRows;
    const int row0 = (tiles - 1 - piece) * kTileRows;      // those that see most keys first
    const int row = row0 + 32 * w + r32;
    const bool valid = row < rows;
    const int tok = min(row, rows - 1) / a.g;
    const int pos = q.start + tok;
    const int lo = a.window > 0 ? max(pos - a.window + 1, 0) : 0;
    const int row_last = min(row0 + kTileRows - 1, rows - 1);
    const int pos_lo = q.start + row0 / a.g, pos_hi = q.start + row_last / a.g;
    const int see_lo = a.window > 0 ? max(pos_lo - a.window + 1, 0) : 0;
    // of the wavefront's own rows
    const int my_lo = q.start + min(row0 + 32 * w, rows - 1) / a.g;
    const int my_hi = q.start + min(row0 + 32 * w + 31, rows - 1) / a.g;
    const int my_see = a.window > 0 ? max(my_lo - a.window + 1, 0) : 0;
    const int my_all = a.window > 0 ? max(my_hi - a.window + 1, 0) : 0;
    const int first = see_lo / kPage, last = q.bad ? first : pos_hi / kPage + 1;

    // ---- queries
    i32x8 qh[KS], ql[KS];
    float qs;
    {
        const uint16_t *qp = a.q.p + (int64_t)(q.t0 + tok) * a.q.token +
                             (int64_t)(head * a.g + min(row, rows - 1) % a.g) * a.q.head;
        u32x4 x[KS][4];
        float amax = 0.0f;
#pragma unroll
        for (int s = 0; s < KS; s++) {
#pragma unroll
            for (int i = 0; i < 4; i++)
                x[s][i] = *(const u32x4 *)(qp + 64 * s + 32 * h + 8 * i);
            amax = fmaxf(amax, amax_bf16(x[s]));
        }
        const int k = e4m3_scale_exp(max_x32(amax));
        qs = exp2_int(k) * fabsf(a.scale);
        const float inv = a.scale < 0.0f ? -exp2_int(-k) : exp2_int(-k);
#pragma unroll
        for (int s = 0; s < KS; s++)
            split_query(x[s], inv, qh[s], ql[s]);
    }

    float m = -INFINITY, l = 0.0f;
    f32x16 o[DT];
#pragma unroll
    for (int i = 0; i < DT; i++)
#pragma unroll
        for (int e = 0; e < 16; e++)
            o[i][e] = 0.0f;

    // ---- staging: a thread's chunks of keys and blocks of values
    const int32_t *table = a.s.pages + (int64_t)b * a.s.max_pages;
    u32x4 kr[KL];
    uint32_t vr[VL][8];
    const bool v_on = D >= 128 || tid < 128;
    // block: tokens 16s + 4hh + {0..3, 8..11} and values 4*quad .. +3
    const int quad = tid % (D / 4);
    const auto v_group = [&](int i) { return tid / (D / 4) + i * (1024 / D); };
    const auto v_token = [&](int i, int e) { return 16 * (v_group(i) >> 1) + 4 * (v_group(i) & 1) + (e & 3) + 8 * (e >> 2); };
    const auto fetch = [&](int page) {
        const int64_t at = (int64_t)page * kv + head;
        const uint8_t *kp = a.c.d_k + at * KB, *vp = a.c.d_v + at * KB;
#pragma unroll
        for (int i = 0; i < KL; i++)
            kr[i] = *(const u32x4 *)(kp + (uint32_t)(16 * (tid + 256 * i)));
        if (v_on)
#pragma unroll
            for (int i = 0; i < VL; i++)
#pragma unroll
                for (int e = 0; e < 8; e++)
                    vr[i][e] = *(const uint32_t *)(vp + (uint32_t)(v_token(i, e) * D + 4 * quad));
    };
    // whether some row of the workgroup does not see page blk whole
    const auto cut = [&](int blk) {
        return blk * kPage + kPage - 1 > pos_lo ||
               (a.window > 0 && blk * kPage < pos_hi - a.window + 1);
    };
    // Stages page blk of the sequence.  Of a cut page, values that no row sees
    // are zeroed (0 * NaN is NaN), and a NaN that only some rows see is zeroed
    // and noted: those rows get it at the end.
    const auto stage = [&](int buf, int blk) {
#pragma unroll
        for (int i = 0; i < KL; i++) {
            const int c = tid + 256 * i, r = c / CH;
            *(u32x4 *)(lds_k[buf] + 16 * (r * CH + k_chunk<D>(r, c % CH))) = kr[i];
        }
        if (!v_on)
            return;
        if (cut(blk)) {
            uint32_t any = 0;
#pragma unroll
            for (int i = 0; i < VL; i++)
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const int p = blk * kPage + v_token(i, e);
                    uint32_t x = p <= pos_hi && p >= see_lo ? vr[i][e] : 0u;
                    const uint32_t nan = nan_bytes(x);
                    any |= nan;
                    vr[i][e] = x & ~nan;
                }
            if (any)
                poison_s = 1;
        }
#pragma unroll
        for (int i = 0; i < VL; i++) {
            uint32_t ab[2][2], cd[2][2];
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const uint32_t x0 = vr[i][4 * j], x1 = vr[i][4 * j + 1], x2 = vr[i][4 * j + 2],
                               x3 = vr[i][4 * j + 3];
                ab[j][0] = __builtin_amdgcn_perm(x1, x0, 0x05010400u);
                ab[j][1] = __builtin_amdgcn_perm(x1, x0, 0x07030602u);
                cd[j][0] = __builtin_amdgcn_perm(x3, x2, 0x05010400u);
                cd[j][1] = __builtin_amdgcn_perm(x3, x2, 0x07030602u);
            }
            const int g = v_group(i);
#pragma unroll
            for (int d = 0; d < 4; d++) {
                const int n = d / 2;
                const u32x4 y = d & 1 ? u32x4{widen2<true>(ab[0][n]), widen2<true>(cd[0][n]),
                                              widen2<true>(ab[1][n]), widen2<true>(cd[1][n])}
                                      : u32x4{widen2<false>(ab[0][n]), widen2<false>(cd[0][n]),
                                              widen2<false>(ab[1][n]), widen2<false>(cd[1][n])};
                const int r = 4 * quad + d;
                *(u32x4 *)(lds_v[buf] + 128 * r + 16 * v_chunk(r, g)) = y;
            }
        }
    };
    // the next page from blk on that lies in the cache (last if none)
    const auto seek = [&](int blk, int &page) {
        for (; blk < last; blk++) {
            page = __builtin_amdgcn_readfirstlane(table[blk]);
            if (page >= 0 && page < a.c.n_pages)
                return blk;
            if (tid == 0)
                raise(a.s.err, ENGRAM_DEVERR_PAGE);
        }
        return last;
    };

    int page = 0, blk = seek(first, page), buf = 0;
    if (tid == 0)
        poison_s = 0;
    __syncthreads();
    if (blk < last) {
        fetch(page);
        stage(0, blk);
    }
    __syncthreads();
    while (blk < last) {
        const int64_t at = (int64_t)page * kv + head;
        const float ks = a.c.d_k_scales[at], vs = a.c.d_v_scales[at];
        const bool plain = vs >= 0x1p-100f && vs <= 0x1p100f;
        const int v_bits = (int)(__float_as_uint(vs) >> 23) - 127;
        const float v_exp = plain ? (float)v_bits : 0.0f;
        const float v_inv = plain ? exp2_int(-v_bits) : 1.0f;
        const float v_rest = plain ? vs * v_inv : vs;
        int next_page = 0;
        const int next = seek(blk + 1, next_page);
        if (next < last)
            fetch(next_page);
        const int base = blk * kPage;
        // a wavefront whose rows see none of the page passes it by
        if (row0 + 32 * w < rows && base <= my_hi && base + kPage > my_see) {
            // ---- logits
            f32x16 s[2];
#pragma unroll
            for (int t = 0; t < 2; t++) {
#pragma unroll
                for (int e = 0; e < 16; e++)
                    s[t][e] = 0.0f;
#pragma unroll
                for (int u = 0; u < KS; u++) {
                    const int r = 32 * t + r32;
                    const u32x4 x = *(const u32x4 *)(lds_k[buf] + 16 * (r * CH + k_chunk<D>(r, 4 * u + 2 * h)));
                    const u32x4 y = *(const u32x4 *)(lds_k[buf] + 16 * (r * CH + k_chunk<D>(r, 4 * u + 2 * h + 1)));
                    const i32x8 kf = {(int)x.x, (int)x.y, (int)x.z, (int)x.w,
                                      (int)y.x, (int)y.y, (int)y.z, (int)y.w};
                    s[t] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(kf, qh[u], s[t], 0, 0, 0, kOne, 0, kOne);
                    s[t] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(kf, ql[u], s[t], 0, 0, 0, kOne, 0, kLoScale);
                }
            }
            // logits are s * f, f >= 0 (the scale's sign went into the queries)
            const float f = qs * ks;
            const bool edge = base + kPage - 1 > my_lo || base < my_all;
            if (edge) {
#pragma unroll
                for (int t = 0; t < 2; t++)
#pragma unroll
                    for (int e = 0; e < 16; e++) {
                        const int p = base + 32 * t + 8 * (e / 4) + 4 * h + e % 4;
                        s[t][e] = p <= pos && p >= lo ? s[t][e] : -INFINITY;
                    }
            }
            float top = -INFINITY;
#pragma unroll
            for (int t = 0; t < 2; t++)
#pragma unroll
                for (int e = 0; e < 16; e++)
                    top = fmaxf(top, s[t][e]);
            top = max_x32(top);
            top = top == -INFINITY ? top : top * f;
            // the base m follows the maximum once that is 2^8 past it: sums and
            // probabilities stay far inside f32's and bf16's range
            if (__any(top > m + kSlack)) {
                const float now = fmaxf(m, top);
                const float keep = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - now);
                m = now;
                l *= keep;
#pragma unroll
                for (int i = 0; i < DT; i++)
                    o[i] *= keep;
            }
            // probabilities times the page's value scale: its power of two
            // joins the exponent, what is left (1 but for scales that
            // cache_append does not write) multiplies
            const float zero = (m == -INFINITY ? 0.0f : m) - v_exp;
            float sum = 0.0f;
            u32x4 pb[4];
            if (!edge && v_rest == 1.0f) {
#pragma unroll
                for (int t = 0; t < 2; t++)
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][e], f, -zero));
                        const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][e + 1], f, -zero));
                        sum += p0 + p1;
                        pb[2 * t + e / 8][(e % 8) / 2] = cvt_bf16x2(p0, p1);
                    }
            } else {
#pragma unroll
                for (int t = 0; t < 2; t++)
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][e], f, -zero));
                        float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][e + 1], f, -zero));
                        p0 = s[t][e] == -INFINITY ? 0.0f : p0;
                        p1 = s[t][e + 1] == -INFINITY ? 0.0f : p1;
                        sum += p0 + p1;
                        p0 = s[t][e] == -INFINITY ? 0.0f : p0 * v_rest;
                        p1 = s[t][e + 1] == -INFINITY ? 0.0f : p1 * v_rest;
                        pb[2 * t + e / 8][(e % 8) / 2] = cvt_bf16x2(p0, p1);
                    }
            }
            l += sum * v_inv;
            // ---- values
#pragma unroll
            for (int i = 0; i < DT; i++)
#pragma unroll
                for (int c = 0; c < 4; c++) {
                    const int r = 32 * i + r32;
                    const u32x4 x = *(const u32x4 *)(lds_v[buf] + 128 * r + 16 * v_chunk(r, 2 * c + h));
                    o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, x),
                                                                   __builtin_bit_cast(bf16x8, pb[c]), o[i], 0, 0, 0);
                }
        }
        if (next < last) {
            stage(buf ^ 1, next);       // its last readers passed the previous barrier
            __syncthreads();
        }
        buf ^= 1;
        blk = next;
        page = next_page;
    }

    if (poison_s) {
        // how many NaN codes of the cut pages each row sees, by the values'
        // product with ones for both
        for (int i = first; i < last; i++) {
            const int32_t id = __builtin_amdgcn_readfirstlane(table[i]);
            if (!cut(i) || id < 0 || id >= a.c.n_pages)
                continue;
            const uint8_t *vp = a.c.d_v + ((int64_t)id * kv + head) * KB;
            for (int c = 0; c < 4; c++) {
                const int t0 = i * kPage + 16 * c + 4 * h;
                u32x4 see;
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int p = t0 + (2 * e & 3) + 8 * (e >> 1);
                    see[e] = cvt_bf16x2(p <= pos && p >= lo ? 1.0f : 0.0f,
                                        p + 1 <= pos && p + 1 >= lo ? 1.0f : 0.0f);
                }
#pragma unroll
                for (int d = 0; d < DT; d++) {
                    u32x4 nan = {0u, 0u, 0u, 0u};
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        const int p = t0 + (e & 3) + 8 * (e >> 2);
                        if (p <= pos_hi && p >= see_lo &&
                            (vp[(p - i * kPage) * D + 32 * d + r32] & 0x7F) == 0x7F)
                            nan[e / 2] |= 0x3F80u << (16 * (e & 1));
                    }
                    f32x16 n;
#pragma unroll
                    for (int e = 0; e < 16; e++)
                        n[e] = 0.0f;
                    n = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                        __builtin_bit_cast(bf16x8, nan), __builtin_bit_cast(bf16x8, see), n, 0, 0, 0);
#pragma unroll
                    for (int e = 0; e < 16; e++)
                        o[d][e] = n[e] > 0.0f ? __uint_as_float(0x7FC00000u) : o[d][e];
                }
            }
        }
    }
    l = add_x32(l);
    const float inv = l != 0.0f ? 1.0f / l : 0.0f;
    if (!valid)
        return;
    uint16_t *out = a.out + ((int64_t)(q.t0 + tok) * a.heads + head * a.g + row % a.g) * D;
#pragma unroll
    for (int i = 0; i < DT; i++)
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
            u32x2 y;
            y.x = cvt_bf16x2(o[i][e] * inv, o[i][e + 1] * inv);
            y.y = cvt_bf16x2(o[i][e + 2] * inv, o[i][e + 3] * inv);
            *(u32x2 *)(out + 32 * i + 2 * e + 4 * h) = y;
        }
}

}  // namespace

int64_t prompt_tiles(const engram_cache &c, const Seqs &s, int32_t g)
{
    return (s.cu ? (int64_t)s.T * g / kTileRows + s.B
                 : (((int64_t)s.each * g + kTileRows - 1) / kTileRows) * s.B) * c.kv_heads;
}

int32_t launch_attend_prompt(const AttendArgs &a, const Launch &l)
{
    const dim3 grid((unsigned)prompt_tiles(a.c, a.s, a.g)), block(64 * kTileWaves);
    if (a.c.head_dim == 64)
        dispatch(attend_tile_kernel<64>, grid, block, l, true, true, a);
    else if (a.c.head_dim == 128)
        dispatch(attend_tile_kernel<128>, grid, block, l, true, true, a);
    else
        dispatch(attend_tile_kernel<256>, grid, block, l, true, true, a);
    return launch_status("engram cache_attend prompt kernel");
}

}  // namespace engram
