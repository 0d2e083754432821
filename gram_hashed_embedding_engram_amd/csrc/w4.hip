// The projection of few tokens through 4-bit weights with a power-of-two
// scale per 32 values: y[t][n] = bf16(sum_k x[t][k] * w[n][k]).
//
// One pass over the weights, as a stream: a workgroup owns 16*RT output rows
// for up to 64 tokens, its four wavefronts take chunks of 512 k in turn and
// their sums meet in LDS.  The weights are the matrix instructions' first
// operand as they lie in memory (lane l: row l % 16, the 16 bytes of 32 values
// from 32(l / 16) on, four rows' worth of 64 contiguous bytes an instruction).
// e4m3 activations go in as codes beside their scales (the instruction applies
// both scales per 32 values); for bf16 activations the weights are widened to
// bf16 in registers, which holds a code times its power of two exactly.
#include "attention.h"

namespace engram {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));

constexpr int kW4Waves = 4;
constexpr int kW4Tokens = 64;       // tokens a workgroup takes
constexpr int kFp4 = 4;             // the instruction's format numbers
constexpr int kFp8 = 0;

// A dword of scale bytes -> the float 2^(s - 127) of byte q.
__device__ __forceinline__ float scale_f32(uint32_t bytes, int q)
{
    return __uint_as_float(((bytes >> (8 * q)) & 0xFFu) << 23);
}

// Eight e2m1 codes (a dword) times `scale` as eight bf16.
__device__ __forceinline__ u32x4 widen8(uint32_t c, float scale)
{
    return u32x4{
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 0)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 1)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 2)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 3))};
}

template <bool FP8, int RT, int MT>
__global__ __launch_bounds__(64 * kW4Waves, RT *MT > 8 ? 2 : 3) void w4_kernel(
    const uint8_t *__restrict__ x, const uint8_t *__restrict__ xs, const uint8_t *__restrict__ w,
    const uint8_t *__restrict__ ws, uint16_t *__restrict__ y, int T, int K, int N)
{
    __shared__ f32x4 red[kW4Waves][RT][MT][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, q = lane >> 4;
    const int n0 = blockIdx.x * 16 * RT, t0 = blockIdx.y * kW4Tokens;
    const int kg = K / 32;

    // rows past N read the last tile's (never stored), tokens past T the last token
    const uint8_t *wrow[RT], *wsrow[RT];
#pragma unroll
    for (int i = 0; i < RT; i++) {
        const int64_t n = min(n0 + 16 * i, N - 16) + r16;
        wrow[i] = w + n * (K / 2) + 16 * q;
        wsrow[i] = ws + n * kg;
    }
    const uint8_t *xrow[MT], *xsrow[MT];
#pragma unroll
    for (int i = 0; i < MT; i++) {
        const int64_t t = min(t0 + 16 * i + r16, T - 1);
        // e4m3: the operand's lane l holds values 16(l / 16) and 64 + 16(l / 16)
        // on of a 128-value step; bf16: 32(l / 16) on, eight an instruction
        xrow[i] = x + (FP8 ? t * K + 16 * q : 2 * (t * K + 32 * q));
        xsrow[i] = FP8 ? xs + t * kg : nullptr;
    }
    f32x4 acc[RT][MT];
#pragma unroll
    for (int i = 0; i < RT; i++)
#pragma unroll
        for (int j = 0; j < MT; j++)
            acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    // one 128-value step from value k on
    const auto step = [&](const u32x4 (&wr)[RT], const uint32_t (&wsc)[RT],
                          const uint32_t (&xsc)[MT], int64_t k) {
        if (FP8) {
#pragma unroll
            for (int j = 0; j < MT; j++) {
                const u32x4 a = *(const u32x4 *)(xrow[j] + k);
                const u32x4 b = *(const u32x4 *)(xrow[j] + k + 64);
                const i32x8 xf = {(int)a.x, (int)a.y, (int)a.z, (int)a.w,
                                  (int)b.x, (int)b.y, (int)b.z, (int)b.w};
#pragma unroll
                for (int i = 0; i < RT; i++) {
                    const i32x8 wf = {(int)wr[i].x, (int)wr[i].y, (int)wr[i].z, (int)wr[i].w,
                                      0, 0, 0, 0};
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        wf, xf, acc[i][j], kFp4, kFp8, 0, (int)(wsc[i] >> (8 * q)), 0,
                        (int)(xsc[j] >> (8 * q)));
                }
            }
        } else {
#pragma unroll
            for (int u = 0; u < 4; u++) {
                u32x4 xf[MT];
#pragma unroll
                for (int j = 0; j < MT; j++)
                    xf[j] = *(const u32x4 *)(xrow[j] + 2 * k + 16 * u);
#pragma unroll
                for (int i = 0; i < RT; i++) {
                    const u32x4 wf = widen8(wr[i][u], scale_f32(wsc[i], q));
#pragma unroll
                    for (int j = 0; j < MT; j++)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8, wf), __builtin_bit_cast(bf16x8, xf[j]),
                            acc[i][j], 0, 0, 0);
                }
            }
        }
    };

    const int chunks = K / 512;
    for (int c = wv; c < chunks; c += kW4Waves) {
        u32x4 wr[4][RT], wsc[RT], xsc[MT];
#pragma unroll
        for (int i = 0; i < RT; i++) {
#pragma unroll
            for (int s = 0; s < 4; s++)
                wr[s][i] = __builtin_nontemporal_load((const u32x4 *)(wrow[i] + 256 * c + 64 * s));
            wsc[i] = *(const u32x4_a4 *)(wsrow[i] + 16 * c);
        }
#pragma unroll
        for (int j = 0; j < MT; j++)
            if (FP8)
                xsc[j] = *(const u32x4_a4 *)(xsrow[j] + 16 * c);
#pragma unroll
        for (int s = 0; s < 4; s++) {
            uint32_t a[RT], b[MT];
#pragma unroll
            for (int i = 0; i < RT; i++)
                a[i] = wsc[i][s];
#pragma unroll
            for (int j = 0; j < MT; j++)
                b[j] = FP8 ? xsc[j][s] : 0;
            step(wr[s], a, b, 512 * (int64_t)c + 128 * s);
        }
    }
    // the last K % 512: up to three steps, one a wavefront
    for (int u = 4 * chunks + wv; u < K / 128; u += kW4Waves) {
        u32x4 wr[RT];
        uint32_t a[RT], b[MT];
#pragma unroll
        for (int i = 0; i < RT; i++) {
            wr[i] = __builtin_nontemporal_load((const u32x4 *)(wrow[i] + 64 * u));
            a[i] = *(const uint32_t *)(wsrow[i] + 4 * u);
        }
#pragma unroll
        for (int j = 0; j < MT; j++)
            b[j] = FP8 ? *(const uint32_t *)(xsrow[j] + 4 * u) : 0;
        step(wr, a, b, 128 * (int64_t)u);
    }

#pragma unroll
    for (int i = 0; i < RT; i++)
#pragma unroll
        for (int j = 0; j < MT; j++)
            red[wv][i][j][lane] = acc[i][j];
    __syncthreads();
    // accumulator e of lane l: output 16i + 4(l / 16) + e, token 16j + l % 16
    for (int u = wv; u < RT * MT; u += kW4Waves) {
        const int i = u / MT, j = u - i * MT;
        f32x4 v = red[0][i][j][lane];
#pragma unroll
        for (int z = 1; z < kW4Waves; z++)
            v += red[z][i][j][lane];
        const int t = t0 + 16 * j + r16, n = n0 + 16 * i + 4 * q;
        if (t < T && n < N) {
            u32x2 o;
            o.x = pack_bf16x2(v.x, v.y);
            o.y = pack_bf16x2(v.z, v.w);
            *(u32x2 *)(y + (int64_t)t * N + n) = o;
        }
    }
}

template <bool FP8, int RT, int MT>
void launch_one(const void *x, const uint8_t *xs, const uint8_t *w, const uint8_t *ws, uint16_t *y,
                int64_t T, int64_t K, int64_t N, const Launch &l)
{
    const dim3 grid((unsigned)((N / 16 + RT - 1) / RT),
                    (unsigned)((T + kW4Tokens - 1) / kW4Tokens));
    dispatch(w4_kernel<FP8, RT, MT>, grid, dim3(64 * kW4Waves), l, true, true, (const uint8_t *)x,
             xs, w, ws, y, (int)T, (int)K, (int)N);
}

template <bool FP8>
void launch_tokens(const void *x, const uint8_t *xs, const uint8_t *w, const uint8_t *ws,
                   uint16_t *y, int64_t T, int64_t K, int64_t N, const Launch &l)
{
    // every workgroup reads all its tokens' values, so more rows a workgroup
    // as the tokens grow, while there are enough row tiles to fill the chip
    const bool wide = N / 16 >= 2 * (int64_t)device_cus();
    if (T <= 16)
        wide ? launch_one<FP8, 2, 1>(x, xs, w, ws, y, T, K, N, l)
             : launch_one<FP8, 1, 1>(x, xs, w, ws, y, T, K, N, l);
    else if (T <= 32)
        wide ? launch_one<FP8, 2, 2>(x, xs, w, ws, y, T, K, N, l)
             : launch_one<FP8, 1, 2>(x, xs, w, ws, y, T, K, N, l);
    else if (T <= 48)
        wide ? launch_one<FP8, 4, 3>(x, xs, w, ws, y, T, K, N, l)
             : launch_one<FP8, 1, 3>(x, xs, w, ws, y, T, K, N, l);
    else
        wide ? launch_one<FP8, 4, 4>(x, xs, w, ws, y, T, K, N, l)
             : launch_one<FP8, 1, 4>(x, xs, w, ws, y, T, K, N, l);
}

}  // namespace

int32_t launch_w4(const void *x, const uint8_t *xs, const uint8_t *w, const uint8_t *ws,
                  uint16_t *y, int64_t T, int64_t K, int64_t N, const Launch &l)
{
    if (xs)
        launch_tokens<true>(x, xs, w, ws, y, T, K, N, l);
    else
        launch_tokens<false>(x, xs, w, ws, y, T, K, N, l);
    return launch_status("engram w4 kernel");
}

}  // namespace engram
