// Attention of a step's queries over the paged 8-bit cache:
//   out = softmax_j(scale * q . k_j) v_j over j <= p (and j > p - window).
#include "attention.h"

namespace engram {
namespace {

// One wavefront per (token, query head).  Keys are taken 64 at a time, a lane
// each; the running maximum m and sum l of the softmax are per wavefront, and
// lane i holds the output's values i, i + 64, ...
template <int D>
__global__ __launch_bounds__(64) void attend_kernel(engram_cache c, Seqs s, Heads q,
                                                    uint16_t *out, int heads, float scale,
                                                    int64_t window)
{
    __shared__ float qs[D], ps[64];
    int b, piece;
    const auto pieces = [&](int i) {
        const Seq e = seq_at(s, i);
        if (e.bad)
            raise(s.err, ENGRAM_DEVERR_SEQUENCE);
        return e.n;
    };
    if (!find_piece(blockIdx.x, s.B, pieces, b, piece))
        return;
    const Seq e = seq_at(s, b);
    const int lane = threadIdx.x, h = blockIdx.y, kh = h / (heads / c.kv_heads);
    const int64_t t = e.t0 + piece;
    for (int i = lane; i < D; i += 64)
        qs[i] = bf16_lo(q.p[t * q.token + h * q.head + i]) * scale;
    __syncthreads();
    float m = -INFINITY, sum = 0.0f, o[D / 64] = {};
    const int pos = e.start + piece;
    const int64_t lo = window > 0 ? (pos - window + 1 > 0 ? pos - window + 1 : 0) : 0;
    if (!e.bad) {
        for (int blk = (int)(lo / kPage); blk <= pos / kPage; blk++) {
            const int32_t page = s.pages[(int64_t)b * s.max_pages + blk];
            if (page < 0 || page >= c.n_pages) {
                raise(s.err, ENGRAM_DEVERR_PAGE);
                continue;
            }
            const int64_t at = (int64_t)page * c.kv_heads + kh;
            const uint8_t *kc = c.d_k + at * kPage * D, *vc = c.d_v + at * kPage * D;
            const float ks = c.d_k_scales[at], vs = c.d_v_scales[at];
            const int j = blk * kPage + lane;
            float a = -INFINITY;
            if (j <= pos && j >= lo) {
                a = 0.0f;
                for (int i = 0; i < D; i++)
                    a += qs[i] * e4m3_to_f32(kc[lane * D + i]);
                a *= ks;
            }
            float top = a;
            for (int x = 1; x < 64; x <<= 1)
                top = fmaxf(top, __shfl_xor(top, x));
            top = fmaxf(top, m);
            const float base = top == -INFINITY ? 0.0f : top;
            const float p = expf(a - base), keep = expf(m - base);
            m = top;
            sum = sum * keep + wave_sum(p);
            __syncthreads();
            ps[lane] = p;
            __syncthreads();
            for (int u = 0; u < D / 64; u++) {
                float acc = 0.0f;
                for (int i = 0; i < kPage; i++)
                    if (blk * kPage + i <= pos && blk * kPage + i >= lo)
                        acc += ps[i] * e4m3_to_f32(vc[i * D + 64 * u + lane]);
                o[u] = o[u] * keep + acc * vs;
            }
        }
    }
    for (int u = 0; u < D / 64; u++)
        out[(t * heads + h) * D + 64 * u + lane] = f32_to_bf16(sum != 0.0f ? o[u] / sum : 0.0f);
}

}  // namespace

size_t attend_bytes(const engram_cache &c, const Seqs &s, int32_t q_heads) { return 0; }

int32_t launch_attend(const engram_cache &c, const Seqs &s, const Heads &q, uint16_t *out,
                      int32_t q_heads, float scale, int64_t window, void *ws, const Launch &l)
{
    const dim3 grid((unsigned)s.T, q_heads), block(64);
    if (c.head_dim == 64)
        dispatch(attend_kernel<64>, grid, block, l, true, true, c, s, q, out, (int)q_heads, scale,
                 window);
    else if (c.head_dim == 128)
        dispatch(attend_kernel<128>, grid, block, l, true, true, c, s, q, out, (int)q_heads,
                 scale, window);
    else
        dispatch(attend_kernel<256>, grid, block, l, true, true, c, s, q, out, (int)q_heads,
                 scale, window);
    return launch_status("engram cache_attend kernel");
}

}  // namespace engram
