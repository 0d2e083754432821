// The residual's addition with the root-mean-square norm and an 8-bit output:
//   s = res + x,  y = s * w / sqrt(mean(s^2) + eps),
//   codes = e4m3(y / 2^k), one k per 32 values.
#include "attention.h"

namespace engram {
namespace {

constexpr int kNormThreads = 256;

template <bool BF16>
__device__ __forceinline__ float load_res(const void *p, int64_t i)
{
    return BF16 ? bf16_lo(((const uint16_t *)p)[i]) : ((const float *)p)[i];
}

template <bool BF16>
__global__ __launch_bounds__(kNormThreads) void add_norm_kernel(
    const uint16_t *__restrict__ x, const void *res, const uint16_t *__restrict__ w, float eps,
    void *sum, uint8_t *__restrict__ codes, uint8_t *__restrict__ scales, int dim)
{
    __shared__ float part[kNormThreads / 64];
    const int tid = threadIdx.x;
    const int64_t row = (int64_t)blockIdx.x * dim;
    float ss = 0.0f;
    for (int i = tid; i < dim; i += kNormThreads) {
        float v = load_res<BF16>(res, row + i) + (x ? bf16_lo(x[row + i]) : 0.0f);
        if (BF16) {
            const uint16_t b = f32_to_bf16(v);
            ((uint16_t *)sum)[row + i] = b;
            v = bf16_lo(b);
        } else {
            ((float *)sum)[row + i] = v;
        }
        ss += v * v;
    }
    ss = wave_sum(ss);
    if ((tid & 63) == 0)
        part[tid >> 6] = ss;
    __syncthreads();
    ss = 0.0f;
    for (int i = 0; i < kNormThreads / 64; i++)
        ss += part[i];
    const float r = 1.0f / sqrtf(ss / (float)dim + eps);
    for (int g = tid; g < dim / 32; g += kNormThreads) {
        float y[32], amax = 0.0f;
        for (int i = 0; i < 32; i++) {
            y[i] = load_res<BF16>(sum, row + 32 * g + i) * r * bf16_lo(w[32 * g + i]);
            amax = fmaxf(amax, finite_abs(y[i]));
        }
        const int k = e4m3_scale_exp(amax);
        const float inv = exp2_int(-k);
        uint32_t *o = (uint32_t *)(codes + row + 32 * g);
        for (int i = 0; i < 8; i++)
            o[i] = e4m3x4(y[4 * i] * inv, y[4 * i + 1] * inv, y[4 * i + 2] * inv,
                          y[4 * i + 3] * inv);
        scales[row / 32 + g] = (uint8_t)(k + 127);
    }
}

}  // namespace

int32_t launch_add_norm(const uint16_t *x, const void *res, bool res_bf16, const uint16_t *w,
                        float eps, void *sum, uint8_t *codes, uint8_t *scales, int64_t rows,
                        int64_t dim, const Launch &l)
{
    const dim3 grid((unsigned)rows), block(kNormThreads);
    if (res_bf16)
        dispatch(add_norm_kernel<true>, grid, block, l, true, true, x, res, w, eps, sum, codes,
                 scales, (int)dim);
    else
        dispatch(add_norm_kernel<false>, grid, block, l, true, true, x, res, w, eps, sum, codes,
                 scales, (int)dim);
    return launch_status("engram add_norm kernel");
}

}  // namespace engram
