// Products of 8-bit rows with 8-bit weights that carry an f32 scale per
// 128 x 128 block.
#include "f8.h"

namespace engram {
namespace {

// lane l's operand of a 16 x 128 tile: row l % 16, bytes 16(l / 16) and 64 on
__device__ __forceinline__ i32x8 operand(const uint8_t *p)
{
    const u32x4 a = *(const u32x4 *)p, b = *(const u32x4 *)(p + 64);
    return i32x8{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}

// A wavefront a tile of 16 rows and 32 outputs.
template <F8Mode MODE, bool XF32>
__global__ __launch_bounds__(64) void tile_kernel(F8Args a)
{
    const int lane = threadIdx.x, r16 = lane & 15, q = lane >> 4;
    const int n0 = blockIdx.x * 32, KB = a.K / 128, NB = (a.N + 127) / 128;
    int expert = 0, tile = blockIdx.y;
    Span span{0, a.T};
    if (MODE != kDense) {
        if (blockIdx.x == 0 && blockIdx.y == 0)
            raise_bad_plan(a.p);
        if (!find_expert(blockIdx.y, a.p, [](int n) { return (n + 15) / 16; }, expert, tile, span))
            return;
    }
    const int rows = min(16, span.n - 16 * tile);
    const int first = span.from + 16 * tile, p = first + min(r16, rows - 1);
    int slot = p;
    bool fine = true;
    if (MODE != kDense) {
        slot = a.p.order[p];
        fine = slot >= 0 && slot < a.p.slots;
        if (!fine) {
            raise(a.p.err, ENGRAM_DEVERR_ROUTE);
            slot = 0;
        }
    }
    const int64_t row = MODE == kUp ? slot / a.p.k : p;
    const uint8_t *x = a.x + row * a.K + 16 * q;
    const uint8_t *xs8 = (const uint8_t *)a.xs + row * (a.K / 32) + q;
    const float *xs32 = (const float *)a.xs + row * KB;
    constexpr int H = MODE == kUp ? 2 : 1;
    const uint8_t *w[H][2];
    const float *ws[H];
    for (int h = 0; h < H; h++) {
        const int64_t m = (int64_t)expert * H + h;
        for (int i = 0; i < 2; i++)
            w[h][i] = a.w + (m * a.N + min(n0 + 16 * i + r16, a.N - 1)) * a.K + 16 * q;
        ws[h] = a.ws + (m * NB + n0 / 128) * KB;
    }
    f32x4 acc[H][2] = {};
    for (int kb = 0; kb < KB; kb++) {
        const i32x8 xf = operand(x + 128 * kb);
        const int sx = XF32 ? kOne : xs8[4 * kb];
        const float f = XF32 ? xs32[kb] : 1.0f;
        for (int h = 0; h < H; h++)
            for (int i = 0; i < 2; i++) {
                const f32x4 v = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    operand(w[h][i] + 128 * kb), xf, f32x4{}, kFp8, kFp8, 0, kOne, 0, sx);
                for (int e = 0; e < 4; e++)
                    acc[h][i][e] += v[e] * (ws[h][kb] * f);
            }
    }
    if (MODE == kUp) {
        float v[2][4], amax = 0.0f;
        for (int i = 0; i < 2; i++)
            for (int e = 0; e < 4; e++) {
                v[i][e] = gated(acc[0][i][e], acc[H - 1][i][e]);
                amax = fmaxf(amax, finite_abs(v[i][e]));
            }
        const int k = e4m3_scale_exp(max_x16(amax));
        const float inv = exp2_int(-k);
        if (r16 < rows && fine) {
            for (int i = 0; i < 2; i++)
                *(uint32_t *)((uint8_t *)a.y + (int64_t)p * a.N + n0 + 16 * i + 4 * q) =
                    e4m3x4(v[i][0] * inv, v[i][1] * inv, v[i][2] * inv, v[i][3] * inv);
            if (q == 0)
                a.hs[(int64_t)p * (a.N / 32) + n0 / 32] = (uint8_t)(k + 127);
        }
        return;
    }
    int k16 = 0;
    if (MODE == kDown) {
        float amax = 0.0f;
        for (int i = 0; i < 2; i++)
            for (int e = 0; e < 4; e++)
                amax = fmaxf(amax, finite_abs(acc[0][i][e]));
        k16 = f16_scale_exp(max_x16(amax));
    }
    const float to_f16 = exp2_int(-k16);
    for (int i = 0; i < 2; i++) {
        const int n = n0 + 16 * i + 4 * q;
        if (r16 >= rows || n >= a.N || !fine)
            continue;
        const f32x4 v = acc[0][i];
        if (MODE == kDense)
            *(u32x2 *)((uint16_t *)a.y + (int64_t)p * a.N + n) =
                u32x2{cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3])};
        else
            *(u32x2 *)((uint16_t *)a.y + (int64_t)slot * a.N + n) =
                u32x2{cvt_f16x2(v[0] * to_f16, v[1] * to_f16), cvt_f16x2(v[2] * to_f16, v[3] * to_f16)};
        if (MODE == kDown && q == 0 && i == 0)
            a.hs[(int64_t)slot * ((a.N + 31) / 32) + n0 / 32] = (uint8_t)k16;
    }
}

// y[t] = sum_j weight[t][j] * product[t * k + j], in j's order; GROUP outputs
// of a product share an exponent
template <int GROUP>
__global__ __launch_bounds__(256) void sum_kernel(const uint16_t *__restrict__ v,
                                                  const int8_t *__restrict__ exps,
                                                  const int32_t *__restrict__ ids,
                                                  const float *__restrict__ weights,
                                                  uint16_t *__restrict__ y, int T, int N, int k, int E)
{
    typedef _Float16 h8 __attribute__((ext_vector_type(8)));
    const int groups = (N + GROUP - 1) / GROUP;
    const int64_t pieces = N / 8, all = T * pieces;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < all; i += gridDim.x * 256ll) {
        const int t = (int)(i / pieces), n = 8 * (int)(i - t * pieces);
        float s[8] = {};
#pragma unroll 4
        for (int j = 0; j < k; j++) {
            const int64_t slot = (int64_t)t * k + j;
            if ((uint32_t)ids[slot] >= (uint32_t)E)
                continue;
            const h8 x = __builtin_bit_cast(h8, *(const u32x4 *)(v + slot * N + n));
            const float f = exp2_int(exps[slot * groups + n / GROUP]) ;
#pragma unroll
            for (int e = 0; e < 8; e++)
                s[e] += (float)x[e] * f * weights[slot];
        }
        *(u32x4 *)(y + (int64_t)t * N + n) = u32x4{cvt_bf16x2(s[0], s[1]), cvt_bf16x2(s[2], s[3]),
                                                   cvt_bf16x2(s[4], s[5]), cvt_bf16x2(s[6], s[7])};
    }
}

template <F8Mode MODE>
void launch_tiles(const F8Args &a, bool f32, int64_t tiles, bool last, const Launch &l)
{
    const dim3 grid((unsigned)((a.N + 31) / 32), (unsigned)tiles);
    if (f32)
        dispatch(tile_kernel<MODE, true>, grid, dim3(64), l, true, last, a);
    else
        dispatch(tile_kernel<MODE, false>, grid, dim3(64), l, true, last, a);
}

}  // namespace

int32_t launch_project_f8(const Rows8 &x, const Blocks8 &w, uint16_t *y, int64_t T, int64_t K,
                          int64_t N, const Launch &l)
{
    const F8Args a{Plan{}, x.x, x.s, w.w, w.s, y, nullptr, (int)T, (int)K, (int)N};
    if (T > 128)
        launch_f8_tiles<kDense>(a, x.f32, true, l);
    else
        launch_tiles<kDense>(a, x.f32, (T + 15) / 16, true, l);
    return launch_status("engram project_f8 kernel");
}

int32_t launch_experts_up(const Plan &p, const Rows8 &x, const Blocks8 &w, uint8_t *h, uint8_t *hs,
                          int64_t K, int64_t I, const Launch &l)
{
    const F8Args a{p, x.x, x.s, w.w, w.s, h, hs, p.T, (int)K, (int)I};
    if (p.slots / p.E >= 48)
        launch_f8_tiles<kUp>(a, x.f32, true, l);
    else
        launch_tiles<kUp>(a, x.f32, f8_most_tiles(p, 16), true, l);
    return launch_status("engram experts_up kernel");
}

size_t experts_down_bytes(const Plan &p, int64_t N)
{
    return (size_t)p.slots * (2 * N + (N + 31) / 32);
}

int32_t launch_experts_down(const Plan &p, const Rows8 &h, const Blocks8 &w, uint16_t *y, int64_t K,
                            int64_t N, void *ws, const Launch &l)
{
    uint16_t *products = (uint16_t *)ws;
    uint8_t *exps = (uint8_t *)(products + (int64_t)p.slots * N);
    const F8Args a{p, h.x, h.s, w.w, w.s, products, exps, p.T, (int)K, (int)N};
    const int64_t blocks = (p.T * (N / 8) + 255) / 256;
    const dim3 grid((unsigned)(blocks < 65536 ? blocks : 65536));
    if (p.slots / p.E >= 48) {
        launch_f8_tiles<kDown>(a, h.f32, false, l);
        dispatch(sum_kernel<64>, grid, dim3(256), l, false, true, (const uint16_t *)products,
                 (const int8_t *)exps, p.ids, p.weights, y, p.T, (int)N, p.k, p.E);
    } else {
        launch_tiles<kDown>(a, h.f32, f8_most_tiles(p, 16), false, l);
        dispatch(sum_kernel<32>, grid, dim3(256), l, false, true, (const uint16_t *)products,
                 (const int8_t *)exps, p.ids, p.weights, y, p.T, (int)N, p.k, p.E);
    }
    return launch_status("engram experts_down kernels");
}

}  // namespace engram
