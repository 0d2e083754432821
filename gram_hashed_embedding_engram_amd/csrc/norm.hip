// The residual's addition with the root-mean-square norm and an 8-bit output:
//   s = res + x,  y = s * w / sqrt(mean(s^2) + eps),
//   codes = e4m3(y / 2^k), one k per 32 values.
//
// One pass over the row: a thread keeps its values in registers between the
// sum of squares and the codes.  Bound by memory (11 bytes a value with an f32
// residual, 7 with bf16): 16384 rows of 4096 f32 in 132 us (5.6 TB/s, where a
// plain copy reaches 5.0), 777 rows of 7200 bf16 in 10.3 us; one row in 3 us,
// which is a launch and one round trip to memory.
//
// Codes and bf16 sums stream past the caches (8160 x 4160 bf16: 52.8 -> 50.2
// us); f32 sums do not, whose 16-byte halves of 32 bytes a lane would each be
// written out (132 -> 137 us), nor do loads, whose data the kernel before has
// just left there (1674 x 4640 f32: 18 -> 20 us).
#include "attention.h"

namespace engram {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// THREADS threads a row, each with C chunks of eight values THREADS * 8 apart;
// a group of 32 values is four neighbouring lanes.  LOOP: rows longer than
// THREADS * C * 8 values, whose sums are read back for the second part.
template <bool BF16, int THREADS, int C, bool LOOP>
__global__ __launch_bounds__(THREADS) void add_norm_kernel(
    const uint16_t *__restrict__ x, const void *res, const uint16_t *__restrict__ w, float eps,
    void *sum, uint8_t *__restrict__ codes, uint8_t *__restrict__ scales, int dim, int rows)
{
    __shared__ float part[2][THREADS / 64];
    const int tid = threadIdx.x;
    int turn = 0;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x, turn ^= 1) {
        const int64_t row = r * dim;
        float v[C][8];
        float ss = 0.0f;
        // adds the chunk at value i, stores the sum, returns it in s
        const auto take = [&](int i, float (&s)[8]) {
            if (BF16) {
                const u32x4 a = *(const u32x4 *)((const uint16_t *)res + row + i);
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    s[2 * j] = bf16_lo(a[j]);
                    s[2 * j + 1] = bf16_hi(a[j]);
                }
            } else {
                const f32x4 a = *(const f32x4 *)((const float *)res + row + i);
                const f32x4 b = *(const f32x4 *)((const float *)res + row + i + 4);
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    s[j] = a[j];
                    s[4 + j] = b[j];
                }
            }
            if (x) {
                const u32x4 a = *(const u32x4 *)(x + row + i);
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    s[2 * j] += bf16_lo(a[j]);
                    s[2 * j + 1] += bf16_hi(a[j]);
                }
            }
            const bool store = x || sum != res;
            if (BF16) {
                u32x4 o;
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    o[j] = cvt_bf16x2(s[2 * j], s[2 * j + 1]);
                    s[2 * j] = bf16_lo(o[j]);          // the norm is that of the sum as kept
                    s[2 * j + 1] = bf16_hi(o[j]);
                }
                if (store)
                    __builtin_nontemporal_store(o, (u32x4 *)((uint16_t *)sum + row + i));
            } else if (store) {
                *(f32x4 *)((float *)sum + row + i) = f32x4{s[0], s[1], s[2], s[3]};
                *(f32x4 *)((float *)sum + row + i + 4) = f32x4{s[4], s[5], s[6], s[7]};
            }
        };
        // the chunk's codes and its group's scale; whole groups of four lanes
        const auto give = [&](int i, const float (&s)[8], float inv_rms) {
            const u32x4 a = *(const u32x4 *)(w + i);
            float y[8], amax = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; j++) {
                y[2 * j] = s[2 * j] * inv_rms * bf16_lo(a[j]);
                y[2 * j + 1] = s[2 * j + 1] * inv_rms * bf16_hi(a[j]);
            }
#pragma unroll
            for (int j = 0; j < 8; j++)
                amax = fmaxf(amax, finite_abs(y[j]));
            amax = fmaxf(amax, __shfl_xor(amax, 1));
            amax = fmaxf(amax, __shfl_xor(amax, 2));
            const int k = e4m3_scale_exp(amax);
            const float inv = exp2_int(-k);
            u32x2 o;
            o.x = e4m3x4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
            o.y = e4m3x4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv);
            __builtin_nontemporal_store(o, (u32x2 *)(codes + row + i));
            if ((tid & 3) == 0)
                scales[(row + i) / 32] = (uint8_t)(k + 127);
        };
#pragma unroll
        for (int c = 0; c < C; c++) {
            const int i = 8 * (c * THREADS + tid);
            if (i < dim) {
                take(i, v[c]);
#pragma unroll
                for (int j = 0; j < 8; j++)
                    ss += v[c][j] * v[c][j];
            }
        }
        if (LOOP)
            for (int i = 8 * (C * THREADS + tid); i < dim; i += 8 * THREADS) {
                float s[8];
                take(i, s);
#pragma unroll
                for (int j = 0; j < 8; j++)
                    ss += s[j] * s[j];
            }
        ss = wave_sum(ss);
        if (THREADS > 64) {
            if ((tid & 63) == 0)
                part[turn][tid >> 6] = ss;
            __syncthreads();
        }
        // the root in 64 bits: its rounding would meet every value of the row
        double total = ss;
        if (THREADS > 64) {
            total = 0.0;
#pragma unroll
            for (int i = 0; i < THREADS / 64; i++)
                total += part[turn][i];
        }
        const float inv_rms = (float)(1.0 / sqrt(total / dim + (double)eps));
#pragma unroll
        for (int c = 0; c < C; c++) {
            const int i = 8 * (c * THREADS + tid);
            if (i < dim)
                give(i, v[c], inv_rms);
        }
        if (LOOP)
            for (int i = 8 * (C * THREADS + tid); i < dim; i += 8 * THREADS) {
                float s[8];                          // this thread's own stores
#pragma unroll
                for (int j = 0; j < 8; j++)
                    s[j] = BF16 ? bf16_lo(((const uint16_t *)sum)[row + i + j])
                                : ((const float *)sum)[row + i + j];
                give(i, s, inv_rms);
            }
    }
}

template <bool BF16>
void launch_type(const uint16_t *x, const void *res, const uint16_t *w, float eps, void *sum,
                 uint8_t *codes, uint8_t *scales, int64_t rows, int64_t dim, const Launch &l)
{
    const int64_t most = 1 << 20;                  // workgroups; longer calls take rows in turn
    const dim3 grid((unsigned)(rows < most ? rows : most));
#define ENGRAM_NORM_CASE(THREADS_, C_, LOOP_)                                                    \
    {                                                                                            \
        dispatch(add_norm_kernel<BF16, THREADS_, C_, LOOP_>, grid, dim3(THREADS_), l, true,      \
                 true, x, res, w, eps, sum, codes, scales, (int)dim, (int)rows);                 \
        return;                                                                                  \
    }
    if (dim <= 512)
        ENGRAM_NORM_CASE(64, 1, false)
    if (dim <= 2048)
        ENGRAM_NORM_CASE(256, 1, false)
    if (dim <= 4096)
        ENGRAM_NORM_CASE(256, 2, false)
    if (dim <= 8192)
        ENGRAM_NORM_CASE(512, 2, false)
    if (dim <= 16384)
        ENGRAM_NORM_CASE(1024, 2, false)
    ENGRAM_NORM_CASE(1024, 2, true)
#undef ENGRAM_NORM_CASE
}

}  // namespace

int32_t launch_add_norm(const uint16_t *x, const void *res, bool res_bf16, const uint16_t *w,
                        float eps, void *sum, uint8_t *codes, uint8_t *scales, int64_t rows,
                        int64_t dim, const Launch &l)
{
    if (res_bf16)
        launch_type<true>(x, res, w, eps, sum, codes, scales, rows, dim, l);
    else
        launch_type<false>(x, res, w, eps, sum, codes, scales, rows, dim, l);
    return launch_status("engram add_norm kernel");
}

}  // namespace engram
