// The projection of few tokens through 4-bit weights with a power-of-two
// scale per 32 values: y[t][n] = bf16(sum_k x[t][k] * w[n][k]).
//
// One pass over the weights, laid out so that a whole CU's share is in flight
// at once: a workgroup a CU owns 16*RT output rows for up to 64 tokens, its
// eight wavefronts split K into equal runs of 256 values, load ahead of the
// matrix instructions, and their sums meet in LDS.
//
// A matrix instruction wants neighbouring lanes in different rows, memory wants
// them side by side (each row's 16 bytes is a lookup of its own: loaded that
// way, 63 MB of weights took 25 us however many loads were in flight).  So
// weights and activations are loaded as whole 128-byte lines, eight lanes a
// row, and turned in the wavefront's own 4 KiB of LDS.  e4m3 activations go in
// as codes beside their scales: the instruction applies both scales per 32
// values, and cuts the products of eight neighbours towards zero below 2^-13 of
// the largest one's power of two before it adds them in f32 (some 2^-16 of a
// sum of normal values, where the result's rounding is 2^-9).  For bf16
// activations the weights are widened to bf16 in registers, which holds a code
// times its power of two exactly; nothing is cut.
//
// 6144 x 20480, sixteen e4m3 tokens (67 MB): 15 us, 4.4 TB/s; of that 10 are the
// bytes at a read-only stream's rate, the rest a launch, the first loads' way
// and the last sums.  4096 x 6144, one token: 5.7 us, a launch and two trips to
// memory.  4096 x 14336, 37 bf16 tokens: 13.8 us, bound by the activations that
// every workgroup reads from L2 and turns in LDS (2.6 times the weights' bytes).
// Weights a run ahead of the instructions, with registers loaded again as they
// were used, took longer (64 bf16 tokens of 6144 x 20480: 28 -> 37 us).
#include "attention.h"

namespace engram {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kW4Tokens = 64;       // tokens a workgroup takes
constexpr int kFp4 = 4;             // the instruction's format numbers
constexpr int kFp8 = 0;

// Eight e2m1 codes (a dword) times `scale` as eight bf16.
__device__ __forceinline__ u32x4 widen8(uint32_t c, float scale)
{
    return u32x4{
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 0)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 1)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 2)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 3))};
}

constexpr int kW4Waves = 8;

// Registers for loads ahead, beside the sums: runs of 256 values whose weights
// are loaded at once, and steps of 128 whose activations are.
constexpr int regs_left(int rt, int mt) { return (mt == 1 ? 212 : rt * mt < 20 ? 196 : 166) - 4 * rt * mt; }
constexpr int runs_ahead(bool fp8, int rt, int mt)
{
    const int u = regs_left(rt, mt) / (9 * rt + (fp8 ? 17 : 32) * mt);
    return u < 1 ? 1 : u > 3 ? 3 : u;
}
constexpr int steps_ahead(bool fp8, int rt, int mt)
{
    return runs_ahead(fp8, rt, mt) > 1 || regs_left(rt, mt) >= 9 * rt + (fp8 ? 17 : 32) * mt
               ? 2 * runs_ahead(fp8, rt, mt) : 1;
}

// Sixteen rows of 128 bytes, loaded eight lanes a row (a: rows 0-7, b: rows
// 8-15), into pieces q and 4 + q of row l % 16 in lane l.  The 16-byte pieces
// of a row are swapped by its number, so that eight lanes that write a row or
// read eight rows meet all banks.  Only this wavefront touches `stage`, and its
// LDS accesses execute in order.
__device__ __forceinline__ void turn_rows(uint8_t *stage, int lane, u32x4 &a, u32x4 &b)
{
    const int r = lane >> 3, p = lane & 7, r16 = lane & 15, q = lane >> 4;
    *(u32x4 *)(stage + 128 * r + 16 * (p ^ r)) = a;
    *(u32x4 *)(stage + 128 * (8 + r) + 16 * (p ^ r)) = b;
    a = *(const u32x4 *)(stage + 128 * r16 + 16 * (q ^ (r16 & 7)));
    b = *(const u32x4 *)(stage + 128 * r16 + 16 * ((4 + q) ^ (r16 & 7)));
}

// Sixteen rows of 256 bytes, sixteen lanes a row (x[i]: rows 4i + l / 16), into
// pieces 4q + i of row l % 16.
__device__ __forceinline__ void turn_long_rows(uint8_t *stage, int lane, u32x4 (&x)[4])
{
    const int r16 = lane & 15, q = lane >> 4;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int r = 4 * i + q;
        *(u32x4 *)(stage + 256 * r + 16 * (r16 ^ (r & 7))) = x[i];
    }
#pragma unroll
    for (int i = 0; i < 4; i++)
        x[i] = *(const u32x4 *)(stage + 256 * r16 + 16 * ((4 * q + i) ^ (r16 & 7)));
}

template <bool FP8, int RT, int MT>
__global__ __launch_bounds__(64 * kW4Waves, 1) void w4_kernel(
    const uint8_t *__restrict__ x, const uint8_t *__restrict__ xs, const uint8_t *__restrict__ w,
    const uint8_t *__restrict__ ws, uint16_t *__restrict__ y, int T, int K, int N)
{
    constexpr int W = kW4Waves, U = runs_ahead(FP8, RT, MT), XS = steps_ahead(FP8, RT, MT);
    constexpr int XL = FP8 ? 2 : 4;                 // loads of a token tile's step
    __shared__ __attribute__((aligned(16))) uint8_t stage_s[W][4096];
    __shared__ f32x4 red[W / 2][RT][MT][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, q = lane >> 4;
    const int n0 = blockIdx.x * 16 * RT, t0 = blockIdx.y * kW4Tokens;
    const int kg = K / 32, kb = K / 2;
    uint8_t *stage = stage_s[wv];

    // The weights are read through a buffer descriptor of the workgroup's own
    // rows: what lies past its end (rows past N, values past K or the run's
    // end) comes back as zeros, so no load hangs on a branch.
    const int rows = min(16 * RT, N - n0);
    const __amdgpu_buffer_rsrc_t wb = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(w + (int64_t)n0 * kb), 0, rows * kb, 0x00027000);
    const __amdgpu_buffer_rsrc_t wsb = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(ws + (int64_t)n0 * kg), 0, rows * kg, 0x00027000);
    constexpr uint32_t kPast = 0xFFFFFF00u;
    constexpr int kStream = 2;                      // non-temporal
    const int p = lane & 7;
    const uint32_t w_off = (lane >> 3) * kb + 16 * p;
    // scales: lane l loads four steps' bytes of row l / 4
    const uint32_t ws_off = (lane >> 2) * kg;
    // tokens past T read the last one (never stored)
    const uint8_t *xt = x + (FP8 ? (int64_t)t0 * K : 2 * (int64_t)t0 * K);
    const uint8_t *xst = FP8 ? xs + (int64_t)t0 * kg : nullptr;
    uint32_t x_off[MT][XL], xs_off[MT];
#pragma unroll
    for (int j = 0; j < MT; j++) {
#pragma unroll
        for (int z = 0; z < XL; z++) {
            const int r = FP8 ? 8 * z + (lane >> 3) : 4 * z + q;
            const uint32_t t = min(t0 + 16 * j + r, T - 1) - t0;
            x_off[j][z] = FP8 ? t * K + 16 * p : 2 * t * K + 16 * r16;
        }
        xs_off[j] = (min(t0 + 16 * j + r16, T - 1) - t0) * kg;
    }
    f32x4 acc[RT][MT];
#pragma unroll
    for (int i = 0; i < RT; i++)
#pragma unroll
        for (int j = 0; j < MT; j++)
            acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    const int steps = K / 128, runs = (steps + 1) / 2;
    const int begin = (int)((int64_t)runs * wv / W), end = (int)((int64_t)runs * (wv + 1) / W);
    u32x4 xr[XS][MT][XL];
    uint32_t xsc[XS][MT];
    const auto load_x = [&](int k0) {               // XS steps from step k0 on
#pragma unroll
        for (int u = 0; u < XS; u++) {
            const int k = min(k0 + u, steps - 1);
#pragma unroll
            for (int j = 0; j < MT; j++) {
#pragma unroll
                for (int z = 0; z < XL; z++)
                    xr[u][j][z] = *(const u32x4 *)(xt + (FP8 ? 128 : 256) * (int64_t)k + x_off[j][z]);
                xsc[u][j] = FP8 ? *(const uint32_t *)(xst + 4 * k + xs_off[j]) : 0;
            }
        }
    };
    for (int k0 = begin; k0 < end; k0 += U) {
        u32x4 wr[U][RT][2];
        uint32_t wsc[(U + 1) / 2][RT];
#pragma unroll
        for (int u = 0; u < U; u++)
#pragma unroll
            for (int i = 0; i < RT; i++)
#pragma unroll
                for (int z = 0; z < 2; z++)
                    wr[u][i][z] = __builtin_amdgcn_raw_buffer_load_b128(
                        wb, k0 + u < end && 128 * (k0 + u) + 16 * p < kb
                                ? w_off + (16 * i + 8 * z) * kb + 128 * (k0 + u) : kPast,
                        0, kStream);
#pragma unroll
        for (int u = 0; u < (U + 1) / 2; u++)
#pragma unroll
            for (int i = 0; i < RT; i++) {
                const int at = 8 * k0 + 16 * u + 4 * (lane & 3);
                wsc[u][i] = __builtin_amdgcn_raw_buffer_load_b32(
                    wsb, at < kg ? ws_off + 16 * i * kg + at : kPast, 0, 0);
            }
        if (XS > 1)
            load_x(2 * k0);
        // all loads are under way before the first is waited for
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < U; u++) {
            if (k0 + u >= end)
                break;
#pragma unroll
            for (int i = 0; i < RT; i++)
                turn_rows(stage, lane, wr[u][i][0], wr[u][i][1]);
#pragma unroll
            for (int h = 0; h < 2; h++) {           // step 2(k0 + u) + h
                // (not multiplied past the end, where an infinite x would meet zeros)
                if (2 * (k0 + u) + h >= steps)
                    break;
                if (XS == 1)
                    load_x(2 * (k0 + u) + h);
                const int xu = XS == 1 ? 0 : 2 * u + h;
                uint32_t sc[RT];                    // of row l % 16, group l / 16
#pragma unroll
                for (int i = 0; i < RT; i++)
                    sc[i] = (uint32_t)__builtin_amdgcn_ds_bpermute(
                                4 * (4 * r16 + 2 * (u & 1) + h), (int)wsc[u / 2][i]) >> (8 * q);
#pragma unroll
                for (int j = 0; j < MT; j++) {
                    if constexpr (FP8) {
                        turn_rows(stage, lane, xr[xu][j][0], xr[xu][j][1]);
                        const u32x4 a = xr[xu][j][0], b = xr[xu][j][1];
                        const i32x8 xf = {(int)a.x, (int)a.y, (int)a.z, (int)a.w,
                                          (int)b.x, (int)b.y, (int)b.z, (int)b.w};
#pragma unroll
                        for (int i = 0; i < RT; i++) {
                            const u32x4 c = wr[u][i][h];
                            const i32x8 wf = {(int)c.x, (int)c.y, (int)c.z, (int)c.w, 0, 0, 0, 0};
                            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                                wf, xf, acc[i][j], kFp4, kFp8, 0, (int)sc[i], 0,
                                (int)(xsc[xu][j] >> (8 * q)));
                        }
                    } else {
                        turn_long_rows(stage, lane, xr[xu][j]);
                    }
                }
                if constexpr (!FP8) {
#pragma unroll
                    for (int i = 0; i < RT; i++)
#pragma unroll
                        for (int z = 0; z < 4; z++) {
                            const u32x4 wf = widen8(wr[u][i][h][z],
                                                    __uint_as_float((sc[i] & 0xFFu) << 23));
#pragma unroll
                            for (int j = 0; j < MT; j++)
                                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                    __builtin_bit_cast(bf16x8, wf),
                                    __builtin_bit_cast(bf16x8, xr[xu][j][z]), acc[i][j], 0, 0, 0);
                        }
                }
            }
        }
    }

    // the wavefronts' sums, halved until four are left
#pragma unroll
    for (int i = 0; i < RT; i++)
#pragma unroll
        for (int j = 0; j < MT; j++)
            if (wv >= W / 2)
                red[wv - W / 2][i][j][lane] = acc[i][j];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < RT; i++)
#pragma unroll
        for (int j = 0; j < MT; j++)
            if (wv < W / 2) {
                acc[i][j] += red[wv][i][j][lane];
                red[wv][i][j][lane] = acc[i][j];
            }
    __syncthreads();
    // accumulator e of lane l: output 16i + 4(l / 16) + e, token 16j + l % 16
    for (int u = wv; u < RT * MT; u += W) {
        const int i = u / MT, j = u - i * MT;
        f32x4 v = red[0][i][j][lane];
#pragma unroll
        for (int z = 1; z < W / 2; z++)
            v += red[z][i][j][lane];
        const int t = t0 + 16 * j + r16, n = n0 + 16 * i + 4 * q;
        if (t < T && n < N) {
            u32x2 o;
            o.x = cvt_bf16x2(v.x, v.y);
            o.y = cvt_bf16x2(v.z, v.w);
            *(u32x2 *)(y + (int64_t)t * N + n) = o;
        }
    }
}

struct Args {
    const void *x;
    const uint8_t *xs, *w, *ws;
    uint16_t *y;
    int64_t T, K, N;
};

template <bool FP8, int RT, int MT>
void launch_one(const Args &a, const Launch &l)
{
    const dim3 grid((unsigned)((a.N / 16 + RT - 1) / RT),
                    (unsigned)((a.T + kW4Tokens - 1) / kW4Tokens));
    dispatch(w4_kernel<FP8, RT, MT>, grid, dim3(64 * kW4Waves), l, true, true, (const uint8_t *)a.x,
             a.xs, a.w, a.ws, a.y, (int)a.T, (int)a.K, (int)a.N);
}

// Row tiles a workgroup: at most five (whose sums and loads fill the
// registers), as many as give every CU the same number of workgroups.  Every
// workgroup reads all its tokens' values, so fewer, wider ones are better.
template <bool FP8, int MT>
void launch_rows(const Args &a, const Launch &l)
{
    const int64_t tiles = a.N / 16, cus = device_cus();
    const int64_t rounds = (tiles + 5 * cus - 1) / (5 * cus);
    const int64_t rt = (tiles + rounds * cus - 1) / (rounds * cus);
    rt <= 1   ? launch_one<FP8, 1, MT>(a, l)
    : rt == 2 ? launch_one<FP8, 2, MT>(a, l)
    : rt == 3 ? launch_one<FP8, 3, MT>(a, l)
    : rt == 4 ? launch_one<FP8, 4, MT>(a, l)
              : launch_one<FP8, 5, MT>(a, l);
}

template <bool FP8>
void launch_tokens(const Args &a, const Launch &l)
{
    a.T <= 16   ? launch_rows<FP8, 1>(a, l)
    : a.T <= 32 ? launch_rows<FP8, 2>(a, l)
    : a.T <= 48 ? launch_rows<FP8, 3>(a, l)
                : launch_rows<FP8, 4>(a, l);
}

}  // namespace

int32_t launch_w4(const void *x, const uint8_t *xs, const uint8_t *w, const uint8_t *ws,
                  uint16_t *y, int64_t T, int64_t K, int64_t N, const Launch &l)
{
    const Args a{x, xs, w, ws, y, T, K, N};
    if (xs)
        launch_tokens<true>(a, l);
    else
        launch_tokens<false>(a, l);
    return launch_status("engram w4 kernel");
}

}  // namespace engram
