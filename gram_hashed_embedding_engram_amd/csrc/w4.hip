// The projection of few tokens through 4-bit weights with a power-of-two
// scale per 32 values: y[t][n] = bf16(sum_k x[t][k] * w[n][k]).
#include "attention.h"

namespace engram {
namespace {

// 2^(s - 127) of a scale byte; 255 is NaN.
__device__ __forceinline__ float e8m0(uint32_t s)
{
    return s == 0 ? 0x1p-127f : s == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float(s << 23);
}

// e2m1 code -> f32: sign, two exponent bits (bias 1), one of mantissa.
__device__ __forceinline__ float e2m1(uint32_t c)
{
    const uint32_t e = (c >> 1) & 3, m = c & 1;
    const float v = e == 0 ? 0.5f * m : (1.0f + 0.5f * m) * (float)(1 << (e - 1));
    return c & 8 ? -v : v;
}

// One wavefront per (output row, token); lanes take whole groups of 32 values.
template <bool FP8>
__global__ __launch_bounds__(256) void w4_kernel(const void *__restrict__ x,
                                                 const uint8_t *__restrict__ xs,
                                                 const uint8_t *__restrict__ w,
                                                 const uint8_t *__restrict__ ws,
                                                 uint16_t *__restrict__ y, int64_t T, int64_t K,
                                                 int64_t N)
{
    const int lane = threadIdx.x & 63;
    const int64_t n = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (n >= N)
        return;
    for (int64_t t = blockIdx.y; t < T; t += gridDim.y) {
        float acc = 0.0f;
        for (int64_t g = lane; g < K / 32; g += 64) {
            float a = 0.0f;
            for (int i = 0; i < 32; i++) {
                const uint32_t c = (w[(n * K + 32 * g + i) / 2] >> (4 * (i & 1))) & 15u;
                const float v = FP8 ? e4m3_to_f32(((const uint8_t *)x)[t * K + 32 * g + i])
                                    : bf16_lo(((const uint16_t *)x)[t * K + 32 * g + i]);
                a += v * e2m1(c);
            }
            a *= e8m0(ws[n * (K / 32) + g]);
            acc += FP8 ? a * e8m0(xs[t * (K / 32) + g]) : a;
        }
        acc = wave_sum(acc);
        if (lane == 0)
            y[t * N + n] = f32_to_bf16(acc);
    }
}

}  // namespace

int32_t launch_w4(const void *x, const uint8_t *xs, const uint8_t *w, const uint8_t *ws,
                  uint16_t *y, int64_t T, int64_t K, int64_t N, const Launch &l)
{
    const dim3 grid((unsigned)((N + 3) / 4), (unsigned)(T < 32768 ? T : 32768)), block(256);
    if (xs)
        dispatch(w4_kernel<true>, grid, block, l, true, true, x, xs, w, ws, y, T, K, N);
    else
        dispatch(w4_kernel<false>, grid, block, l, true, true, x, xs, w, ws, y, T, K, N);
    return launch_status("engram w4 kernel");
}

}  // namespace engram
