// Products of few 8-bit rows with 8-bit weights that carry an f32 scale per
// 128 x 128 block: y[t][n] = sum_b ws[n/128][b] * (sum of block b's 128 products of
// codes and row scales).
//
// One pass over the weights.  A wavefront loads 16 x 128 tiles of them straight
// into a matrix instruction's registers (four lanes a row of 64 bytes, two such
// loads a tile), multiplies all its rows of x with each, and joins the block's
// scale as it adds the block's sum in f32.  K is split over the wavefronts of a
// workgroup, which keeps enough loads in flight where there are few outputs; the
// parts meet in LDS.  An expert's rows are found by a scan over the plan's spans.
//
// Bound by the weights' bytes.  One token of 4096 x 6144: 6.8 to 7.1 us, of which a
// launch and two trips to memory are 4; sixteen of 6144 x 20480 (126 MB) 27 us; one
// token's eight experts of 4096 x (2 x 2048) (134 MB) 28 us; 64 tokens over 256 of
// them, 164 met (2.75 GB), 440 to 515 us as the clocks go, 6.2 to 5.3 TB/s; their down
// projection (1.4 GB) 247 to 277 us with its sum, 5.6 to 5 TB/s.  Rows with f32 scales
// take the same (up 461 to 509, down 250 to 283).
//
// Measured on the way: loads marked non-temporal are slower (444 -> 500 us and
// more: an expert's second tile and the next call find nothing in the caches); more
// than two steps of loads ahead, or a fence between loads and products, takes
// wavefronts away (64 tokens over 256 experts, a wavefront a tile: 575 us with four
// steps and a fence, 497 without); one wavefront a tile instead of four 486 us.
#include "f8.h"

namespace engram {
namespace {

// Rows from which the tiles take over (f8_tiles.hip).  Both ways in us, these
// kernels first: T = 17, 4096 x 4096 8.5 and 12.4; 32 9.7 and 12.5; 24, 6144 x 20480
// 28.6 and 30.3; 48 50 and 33; 32, 4096 x 20480 18.5 and 17.5; 40, 4096 x 14336 27 and 13.
constexpr int64_t kMostRows = 32;
// The same for an expert's rows on average.  Up, 64 experts of 4096 x 2048: 4 rows
// 162 and 165, 8 rows 185 and 173; 256 of 2048 x 1024, 8 rows 194 and 183; 16
// experts, 2 rows 38 and 49, 8 rows 57 and 65.  Down, 64 of 2048 x 4096: 4 rows 95
// and 96, 6 rows 106 and 98, 8 rows 118 and 100; 256 experts, 8 rows 437 and 355; 16
// experts, 2 rows 23 and 23, 8 rows 34 and 29.5.
constexpr int64_t kTileRows = 8;
constexpr int kFewSlots = 16, kFewWaves = 16;
// Wavefronts that share an expert's K.  Up, 1, 2, 4 and 8 of them: one token 50, 31,
// 28 and 28 us, 64 tokens 486, 452, 444 and 458.  Down, 1, 2 and 4: 64 tokens 244, 245
// and 250, three 40, 38 and 36, 8 tokens 84, 81 and 80 (with products as f16: as f32
// 64 tokens take 3 more).
constexpr int kUpWaves = 4, kDownWaves = 2;

__device__ __forceinline__ i32x8 operand(const u32x4 &a, const u32x4 &b)
{
    return i32x8{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}

// Row p's 32 outputs from n0 on, of which this lane has 16i + 4q .. + 3, of an
// expert's products (kUp: v[0..1] of the gate, v[2..3] of the up matrix).
template <F8Mode MODE>
__device__ __forceinline__ void give(const F8Args &a, const f32x4 (&v)[4], int64_t p, bool in, int n0,
                                     int q)
{
    int slot = 0;
    if (in) {
        slot = a.p.order[p];
        if ((uint32_t)slot >= (uint32_t)a.p.slots) {
            raise(a.p.err, ENGRAM_DEVERR_ROUTE);
            in = false;
        }
    }
    if (MODE == kUp) {
        float h[2][4], amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 2; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                h[i][e] = gated(v[i][e], v[2 + i][e]);
                amax = fmaxf(amax, finite_abs(h[i][e]));
            }
        const int k = e4m3_scale_exp(max_x16(amax));
        const float inv = exp2_int(-k);
        if (!in)
            return;
#pragma unroll
        for (int i = 0; i < 2; i++)
            *(uint32_t *)((uint8_t *)a.y + p * a.N + n0 + 16 * i + 4 * q) =
                e4m3x4(h[i][0] * inv, h[i][1] * inv, h[i][2] * inv, h[i][3] * inv);
        if (q == 0)
            a.hs[p * (a.N / 32) + n0 / 32] = (uint8_t)(k + 127);
        return;
    }
    // (as f32: f16 under shared exponents would gain 244 against 248 us for 64 tokens
    // over 256 experts, and nothing for 8)
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const int n = n0 + 16 * i + 4 * q;
        if (in && n < a.N)
            *(f32x4 *)((float *)a.y + (int64_t)slot * a.N + n) = v[i];
    }
}

// Steps of 128 values whose loads go out together: two, where the registers that
// two wavefronts a SIMD leave each hold them.
constexpr int steps_ahead(int rt, int mt)
{
    return (190 - 4 * rt * mt) / (8 * rt + 9 * mt) >= 2 ? 2 : 1;
}

// A workgroup takes 16 * OT outputs (kUp: of each half) of 16 * MT rows; its W
// wavefronts split K and their sums meet in LDS.
template <F8Mode MODE, bool XF32, int OT, int MT, int W>
__global__ __launch_bounds__(64 * W) void rows_kernel(F8Args a)
{
    constexpr int H = MODE == kUp ? 2 : 1, RT = OT * H, U = steps_ahead(RT, MT);
    __shared__ f32x4 red[W / 2][MT][RT][64];
    const int lane = threadIdx.x & 63, r16 = lane & 15, q = lane >> 4;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = blockIdx.x * 16 * OT, KB = a.K / 128, NB = (a.N + 127) / 128;
    for (int item = blockIdx.y;; item += gridDim.y) {
        int expert = 0, tile = item;
        Span span{0, a.T};
        if (MODE != kDense) {
            if (blockIdx.x == 0 && item == 0)
                raise_bad_plan(a.p);
            if (!find_expert(item, a.p, [](int n) { return (n + 16 * MT - 1) / (16 * MT); }, expert,
                             tile, span))
                return;
        } else if (16 * MT * item >= a.T) {
            return;
        }
        const int rows = min(16 * MT, span.n - 16 * MT * tile);
        const int64_t first = span.from + 16 * MT * tile;
        // the row of x behind row 16j + l % 16 (past the last: the last one)
        const uint8_t *x[MT];
        const uint8_t *xs[MT];
#pragma unroll
        for (int j = 0; j < MT; j++) {
            int64_t row = first + min(16 * j + r16, rows - 1);
            if (MODE == kUp) {
                const int slot = a.p.order[row];
                row = (uint32_t)slot < (uint32_t)a.p.slots ? slot / a.p.k : 0;
            }
            x[j] = a.x + row * a.K + 16 * q;
            xs[j] = (const uint8_t *)a.xs + row * (a.K / 32) + (XF32 ? 0 : q);
        }
        // the weights through a descriptor of the workgroup's own rows: what lies
        // past them, or past the wavefront's steps, comes back as zeros
        const int64_t m0 = (int64_t)expert * H * a.N + n0;
        const int bytes = min(16 * OT, a.N - n0) * a.K;
        const __amdgpu_buffer_rsrc_t w0 =
            __builtin_amdgcn_make_buffer_rsrc((void *)(a.w + m0 * a.K), 0, bytes, 0x00020000);
        const __amdgpu_buffer_rsrc_t w1 = __builtin_amdgcn_make_buffer_rsrc(
            (void *)(a.w + (m0 + (H - 1) * (int64_t)a.N) * a.K), 0, bytes, 0x00020000);
        constexpr uint32_t kPast = 0xFFFFFF00u;
        const uint32_t at = r16 * (uint32_t)a.K + 16 * q;
        const int begin = KB * wv / W, end = KB * (wv + 1) / W;
        f32x4 acc[RT][MT];
#pragma unroll
        for (int i = 0; i < RT; i++)
#pragma unroll
            for (int j = 0; j < MT; j++)
                acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        // the scales of row block i (16 * OT rows may meet two blocks of 128)
        const float *ws[RT];
#pragma unroll
        for (int i = 0; i < RT; i++)
            ws[i] = a.ws + (((int64_t)expert * H + i / OT) * NB +
                            min(n0 + 16 * (i % OT), a.N - 1) / 128) * KB;
        for (int k0 = begin; k0 < end; k0 += U) {
            u32x4 wr[U][RT][2], xr[U][MT][2];
            uint32_t xsc[U][MT];
#pragma unroll
            for (int u = 0; u < U; u++)
#pragma unroll
                for (int i = 0; i < RT; i++)
#pragma unroll
                    for (int z = 0; z < 2; z++) {
                        const uint32_t off = k0 + u < end
                            ? at + 16 * (i % OT) * a.K + 128 * (k0 + u) + 64 * z : kPast;
                        wr[u][i][z] = i < OT ? __builtin_amdgcn_raw_buffer_load_b128(w0, off, 0, 0)
                                            : __builtin_amdgcn_raw_buffer_load_b128(w1, off, 0, 0);
                    }
#pragma unroll
            for (int u = 0; u < U; u++) {
                const int k = min(k0 + u, end - 1);
#pragma unroll
                for (int j = 0; j < MT; j++) {
                    xr[u][j][0] = *(const u32x4 *)(x[j] + 128 * k);
                    xr[u][j][1] = *(const u32x4 *)(x[j] + 128 * k + 64);
                    xsc[u][j] = XF32 ? *(const uint32_t *)(xs[j] + 4 * k) : xs[j][4 * k];
                }
            }
#pragma unroll
            for (int u = 0; u < U; u++) {
                // (not multiplied past the end, where a NaN would meet zeros)
                if (k0 + u >= end)
                    break;
                BlockScale f[RT];
#pragma unroll
                for (int i = 0; i < RT; i++)
                    f[i] = block_scale<XF32>(ws[i][k0 + u]);
#pragma unroll
                for (int j = 0; j < MT; j++) {
                    const i32x8 xf = operand(xr[u][j][0], xr[u][j][1]);
                    const float t = XF32 ? __uint_as_float(xsc[u][j]) : 1.0f;
#pragma unroll
                    for (int i = 0; i < RT; i++) {
                        const f32x4 v = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            operand(wr[u][i][0], wr[u][i][1]), xf, f32x4{0.0f, 0.0f, 0.0f, 0.0f},
                            kFp8, kFp8, 0, f[i].e, 0, XF32 ? kOne : (int)xsc[u][j]);
                        const float g = XF32 ? f[i].m * t : f[i].m;
#pragma unroll
                        for (int e = 0; e < 4; e++)
                            acc[i][j][e] = __builtin_fmaf(v[e], g, acc[i][j][e]);
                    }
                }
            }
        }
        // the wavefronts' sums: the upper half's to the lower's, which leave theirs
        if (wv >= W / 2)
#pragma unroll
            for (int i = 0; i < RT; i++)
#pragma unroll
                for (int j = 0; j < MT; j++)
                    red[wv - W / 2][j][i][lane] = acc[i][j];
        __syncthreads();
        if (wv < W / 2)
#pragma unroll
            for (int i = 0; i < RT; i++)
#pragma unroll
                for (int j = 0; j < MT; j++) {
                    acc[i][j] += red[wv][j][i][lane];
                    red[wv][j][i][lane] = acc[i][j];
                }
        __syncthreads();
        const auto sum = [&](int i, int j) {
            f32x4 v = red[0][j][i][lane];
#pragma unroll
            for (int z = 1; z < W / 2; z++)
                v += red[z][j][i][lane];
            return v;
        };
        // accumulator e of block (i, j) is output 16i + 4q + e, row 16j + l % 16; a
        // wavefront finishes every W-th block (of rows, for the experts)
#pragma unroll
        for (int j = 0; j < MT; j++) {
            const int r = 16 * j + r16;
            if constexpr (MODE == kDense) {
#pragma unroll
                for (int i = 0; i < OT; i++) {
                    const int n = n0 + 16 * i + 4 * q;
                    if ((j * OT + i) % W != wv)
                        continue;
                    const f32x4 v = sum(i, j);
                    if (r < rows && n < a.N)
                        *(u32x2 *)((uint16_t *)a.y + (first + r) * a.N + n) =
                            u32x2{cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3])};
                }
            } else {
                static_assert(OT == 2, "an expert's outputs leave 32 at a time");
                if (j % W != wv)
                    continue;
                const f32x4 v[4] = {sum(0, j), sum(1, j), sum(RT - 2, j), sum(RT - 1, j)};
                give<MODE>(a, v, first + r, r < rows, n0, q);
            }
        }
        __syncthreads();                            // the next item's sums take their place
    }
}

// y[t] = sum_j weight[t][j] * product[t * k + j], in j's order, in f32.  Products
// are f32, or f16 where exps has an exponent for each 64 outputs of one.  Bound by
// their bytes: 4096 tokens of eight experts, 4096 outputs (268 MB of f16), 58 us, 4.6
// TB/s.
template <bool F16>
__global__ __launch_bounds__(256) void sum_kernel(const void *__restrict__ v,
                                                  const int8_t *__restrict__ exps,
                                                  const int32_t *__restrict__ ids,
                                                  const float *__restrict__ weights,
                                                  uint16_t *__restrict__ y, int T, int N, int k, int E)
{
    typedef _Float16 h8 __attribute__((ext_vector_type(8)));
    const int64_t pieces = N / 8, all = T * pieces;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < all; i += gridDim.x * 256ll) {
        const int t = (int)(i / pieces), n = 8 * (int)(i - t * pieces);
        float s[8] = {};
#pragma unroll 4
        for (int j = 0; j < k; j++) {
            const int64_t slot = (int64_t)t * k + j;
            if ((uint32_t)ids[slot] >= (uint32_t)E)
                continue;
            if (F16) {
                const h8 x = __builtin_bit_cast(h8, *(const u32x4 *)((const uint16_t *)v + slot * N + n));
                const float f = exp2_int(exps[slot * ((N + 63) / 64) + n / 64]);
#pragma unroll
                for (int e = 0; e < 8; e++)
                    s[e] += (float)x[e] * f * weights[slot];
            } else {
                const f32x4 *const x = (const f32x4 *)((const float *)v + slot * N + n);
                const f32x4 lo = x[0], hi = x[1];
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    s[e] += lo[e] * weights[slot];
                    s[4 + e] += hi[e] * weights[slot];
                }
            }
        }
        *(u32x4 *)(y + (int64_t)t * N + n) = u32x4{cvt_bf16x2(s[0], s[1]), cvt_bf16x2(s[2], s[3]),
                                                   cvt_bf16x2(s[4], s[5]), cvt_bf16x2(s[6], s[7])};
    }
}

// Down projection and weighted sum of up to kFewSlots slots in one launch: a
// workgroup has 16 outputs, its wavefronts take pieces of K, `split` of each expert
// that the plan meets, and the slots' sums stay in LDS until all are there.
template <bool XF32>
__global__ __launch_bounds__(64 * kFewWaves) void down_few_kernel(F8Args a, int split)
{
    constexpr int U = 4;
    __shared__ float part[kFewSlots][17];           // [split][slots], split * slots <= kFewSlots
    const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, q = lane >> 4;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n0 = blockIdx.x * 16, KB = a.K / 128, NB = (a.N + 127) / 128;
    if (blockIdx.x == 0)
        raise_bad_plan(a.p);
    for (int i = tid; i < kFewSlots * 17; i += 64 * kFewWaves)
        (&part[0][0])[i] = 0.0f;
    __syncthreads();
    int met = 0;
    for (int base = 0; base < a.p.E; base += 64) {
        const Span s = base + lane < a.p.E ? span_of(a.p, base + lane) : Span{0, 0};
        for (uint64_t mask = __ballot(s.n > 0); mask; mask &= mask - 1, met += split) {
            const int piece = (wv + kFewWaves - met % kFewWaves) % kFewWaves;
            if (piece >= split)
                continue;
            const int begin = KB * piece / split, end = KB * (piece + 1) / split;
            const int at = __builtin_ctzll(mask);
            const int from = __builtin_amdgcn_readlane(s.from, at), n = __builtin_amdgcn_readlane(s.n, at);
            const int64_t m0 = (int64_t)(base + at) * a.N + n0;
            const uint8_t *w = a.w + (m0 + r16) * a.K + 16 * q;
            const float *ws = a.ws + ((int64_t)(base + at) * NB + n0 / 128) * KB;
            for (int r0 = 0; r0 < n; r0 += 16) {
                const int64_t row = from + r0 + min(r16, n - r0 - 1);
                const uint8_t *x = a.x + row * a.K + 16 * q;
                const uint8_t *xs = (const uint8_t *)a.xs + row * (a.K / 32) + (XF32 ? 0 : q);
                f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
                for (int k0 = begin; k0 < end; k0 += U) {
                    u32x4 wr[U][2], xr[U][2];
                    uint32_t xsc[U];
                    float f[U];
#pragma unroll
                    for (int u = 0; u < U; u++) {
                        const int k = min(k0 + u, end - 1);
#pragma unroll
                        for (int z = 0; z < 2; z++) {
                            wr[u][z] = *(const u32x4 *)(w + 128 * k + 64 * z);
                            xr[u][z] = *(const u32x4 *)(x + 128 * k + 64 * z);
                        }
                        xsc[u] = XF32 ? *(const uint32_t *)(xs + 4 * k) : xs[4 * k];
                        f[u] = ws[k];
                    }
                    // all loads are under way before the first is waited for
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int u = 0; u < U; u++) {
                        if (k0 + u >= end)
                            break;
                        const BlockScale b = block_scale<XF32>(f[u]);
                        const f32x4 v = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            operand(wr[u][0], wr[u][1]), operand(xr[u][0], xr[u][1]),
                            f32x4{0.0f, 0.0f, 0.0f, 0.0f}, kFp8, kFp8, 0, b.e, 0,
                            XF32 ? kOne : (int)xsc[u]);
                        const float g = XF32 ? b.m * __uint_as_float(xsc[u]) : b.m;
#pragma unroll
                        for (int e = 0; e < 4; e++)
                            acc[e] = __builtin_fmaf(v[e], g, acc[e]);
                    }
                }
                if (r16 < n - r0) {
                    const int slot = a.p.order[row];
                    if ((uint32_t)slot < (uint32_t)a.p.slots) {
#pragma unroll
                        for (int e = 0; e < 4; e++)
                            part[piece * a.p.slots + slot][4 * q + e] = acc[e];
                    } else {
                        raise(a.p.err, ENGRAM_DEVERR_ROUTE);
                    }
                }
            }
        }
    }
    __syncthreads();
    for (int i = tid; i < a.T * 8; i += 64 * kFewWaves) {
        const int t = i / 8, n = 2 * (i & 7);
        float s0 = 0.0f, s1 = 0.0f;
        for (int j = 0; j < a.p.k; j++) {
            const int slot = t * a.p.k + j;
            if ((uint32_t)a.p.ids[slot] >= (uint32_t)a.p.E)
                continue;
            float v0 = part[slot][n], v1 = part[slot][n + 1];
            for (int i = 1; i < split; i++) {
                v0 += part[i * a.p.slots + slot][n];
                v1 += part[i * a.p.slots + slot][n + 1];
            }
            s0 += v0 * a.p.weights[slot];
            s1 += v1 * a.p.weights[slot];
        }
        *(uint32_t *)((uint16_t *)a.y + (int64_t)t * a.N + n0 + n) = cvt_bf16x2(s0, s1);
    }
}

template <F8Mode MODE, int OT, int MT, int W>
void launch_split(const F8Args &a, bool f32, int64_t tiles, bool last, const Launch &l)
{
    const dim3 grid((unsigned)((a.N + 16 * OT - 1) / (16 * OT)), (unsigned)(tiles < 65535 ? tiles : 65535));
    if (f32)
        dispatch(rows_kernel<MODE, true, OT, MT, W>, grid, dim3(64 * W), l, true, last, a);
    else
        dispatch(rows_kernel<MODE, false, OT, MT, W>, grid, dim3(64 * W), l, true, last, a);
}

// Outputs a workgroup: at most 80 (whose sums and loads fill the registers), as
// many as give every CU the same number of workgroups.  Every workgroup reads all
// its rows' values, so fewer, wider ones are better.
template <int MT>
void launch_dense(const F8Args &a, bool f32, const Launch &l)
{
    const int64_t tiles = (a.T + 16 * MT - 1) / (16 * MT), cus = device_cus();
    const int64_t n = a.N / 16 * tiles, rounds = (n + 5 * cus - 1) / (5 * cus);
    const int64_t ot = (n + rounds * cus - 1) / (rounds * cus);
    ot <= 1   ? launch_split<kDense, 1, MT, 8>(a, f32, tiles, true, l)
    : ot == 2 ? launch_split<kDense, 2, MT, 8>(a, f32, tiles, true, l)
    : ot == 3 ? launch_split<kDense, 3, MT, 8>(a, f32, tiles, true, l)
    : ot == 4 ? launch_split<kDense, 4, MT, 8>(a, f32, tiles, true, l)
              : launch_split<kDense, 5, MT, 8>(a, f32, tiles, true, l);
}

}  // namespace

int32_t launch_project_f8(const Rows8 &x, const Blocks8 &w, uint16_t *y, int64_t T, int64_t K,
                          int64_t N, const Launch &l)
{
    const F8Args a{Plan{}, x.x, x.s, w.w, w.s, y, nullptr, (int)T, (int)K, (int)N};
    if (T > kMostRows)
        return launch_f8_tiles<kDense>(a, x.f32, true, l);
    T <= 16 ? launch_dense<1>(a, x.f32, l) : launch_dense<2>(a, x.f32, l);
    return launch_status("engram project_f8 kernel");
}

int32_t launch_experts_up(const Plan &p, const Rows8 &x, const Blocks8 &w, uint8_t *h, uint8_t *hs,
                          int64_t K, int64_t I, const Launch &l)
{
    const F8Args a{p, x.x, x.s, w.w, w.s, h, hs, p.T, (int)K, (int)I};
    if (p.slots / p.E >= kTileRows)
        return launch_f8_tiles<kUp>(a, x.f32, true, l);
    launch_split<kUp, 2, 1, kUpWaves>(a, x.f32, f8_most_tiles(p, 16), true, l);
    return launch_status("engram experts_up kernel");
}

// Whether a call's products stay in LDS.  Both ways in us, 2048 x 4096: 2 slots 8.9
// and 10.9, 8 slots 14.9 and 18.8, 16 slots 23 and 29, 32 slots 39 and 45, but LDS for
// as many takes 2 slots from 8.9 to 14; 1024 x 1024, whose workgroups are few: 4 slots
// 8.4 and 8.9, 16 slots 13 and 10.7.
static bool down_few(const Plan &p, int64_t N)
{
    return p.slots <= kFewSlots && (p.slots <= 4 || N >= 2048) && p.slots / p.E < kTileRows;
}

size_t experts_down_bytes(const Plan &p, int64_t N)
{
    if (down_few(p, N))
        return 0;
    // f32 products of few rows; f16 ones and their exponents of tiles, and no less than
    // f32 ones of the most rows that no tiles take, so that a workspace serves every
    // call of fewer tokens
    const int64_t few = kTileRows * p.E - 1;
    const size_t f32 = (size_t)(p.slots < few ? p.slots : few) * N * sizeof(float);
    const size_t f16 = (size_t)p.slots * (2 * N + (N + 63) / 64);
    return p.slots / p.E >= kTileRows && f16 > f32 ? f16 : f32;
}

int32_t launch_experts_down(const Plan &p, const Rows8 &h, const Blocks8 &w, uint16_t *y, int64_t K,
                            int64_t N, void *ws, const Launch &l)
{
    if (down_few(p, N)) {
        const F8Args a{p, h.x, h.s, w.w, w.s, y, nullptr, p.T, (int)K, (int)N};
        const dim3 grid((unsigned)(N / 16));
        int split = 1;
        while (2 * split * p.slots <= kFewSlots && 2 * split <= K / kF8Block)
            split *= 2;
        if (h.f32)
            dispatch(down_few_kernel<true>, grid, dim3(64 * kFewWaves), l, true, true, a, split);
        else
            dispatch(down_few_kernel<false>, grid, dim3(64 * kFewWaves), l, true, true, a, split);
        return launch_status("engram experts_down kernel");
    }
    const int64_t blocks = (p.T * (N / 8) + 255) / 256;
    const dim3 grid((unsigned)(blocks < 65536 ? blocks : 65536));
    if (p.slots / p.E >= kTileRows) {
        uint8_t *exps = (uint8_t *)ws + 2 * (int64_t)p.slots * N;
        const F8Args a{p, h.x, h.s, w.w, w.s, ws, exps, p.T, (int)K, (int)N};
        const int32_t rc = launch_f8_tiles<kDown>(a, h.f32, false, l);
        if (rc != ENGRAM_OK)
            return rc;
        dispatch(sum_kernel<true>, grid, dim3(256), l, false, true, (const void *)ws,
                 (const int8_t *)exps, p.ids, p.weights, y, p.T, (int)N, p.k, p.E);
    } else {
        const F8Args a{p, h.x, h.s, w.w, w.s, ws, nullptr, p.T, (int)K, (int)N};
        launch_split<kDown, 2, 1, kDownWaves>(a, h.f32, f8_most_tiles(p, 16), false, l);
        dispatch(sum_kernel<false>, grid, dim3(256), l, false, true, (const void *)ws,
                 (const int8_t *)nullptr, p.ids, p.weights, y, p.T, (int)N, p.k, p.E);
    }
    return launch_status("engram experts_down kernels");
}

}  // namespace engram
