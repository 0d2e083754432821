// The position rotation of a step's queries and keys, and the append of its
// keys and values to the paged 8-bit cache.
#include "attention.h"

namespace engram {
namespace {

// x[i] of a head after the rotation by position pos.
__device__ __forceinline__ float turned(const uint16_t *x, int i, const Rotation &r, int pos)
{
    const float v = bf16_lo(x[i]);
    if (i >= r.rot)
        return v;
    const int half = r.rot / 2;
    const int pair = r.halves ? (i < half ? i : i - half) : i / 2;
    const bool first = r.halves ? i < half : !(i & 1);
    const double a = (double)pos * (double)r.freq[pair];
    const float c = (float)cos(a), s = (float)sin(a);
    const float u = bf16_lo(x[r.halves ? (first ? i + half : i - half) : i ^ 1]);
    return first ? v * c - u * s : u * s + v * c;
}

// One workgroup per (page of a sequence, head, keys or values).
__global__ __launch_bounds__(256) void append_pages_kernel(engram_cache c, Seqs s, Heads k,
                                                           Heads v, Rotation r)
{
    int b, piece;
    const auto pieces = [&](int i) {
        const Seq q = seq_at(s, i);
        if (q.bad)
            raise(s.err, ENGRAM_DEVERR_SEQUENCE);
        return q.bad || q.n == 0 ? 0 : (q.start + q.n - 1) / kPage - q.start / kPage + 1;
    };
    if (!find_piece(blockIdx.x, s.B, pieces, b, piece))
        return;
    const Seq q = seq_at(s, b);
    const int blk = q.start / kPage + piece;
    const int32_t page = s.pages[(int64_t)b * s.max_pages + blk];
    if (page < 0 || page >= c.n_pages) {
        raise(s.err, ENGRAM_DEVERR_PAGE);
        return;
    }
    const int h = blockIdx.y, d = c.head_dim;
    const bool is_v = blockIdx.z;
    const Heads &src = is_v ? v : k;
    Rotation rot = r;
    if (is_v)
        rot.rot = 0;
    const int64_t at = (int64_t)page * c.kv_heads + h;
    uint8_t *codes = (is_v ? c.d_v : c.d_k) + at * kPage * d;
    float *scale = (is_v ? c.d_v_scales : c.d_k_scales) + at;
    const int older = max(q.start - blk * kPage, 0);
    const int last = min(q.start + q.n - blk * kPage, kPage);
    __shared__ float part[4];
    const auto value = [&](int i) {
        const int pos = blk * kPage + older + i / d;
        return turned(src.p + (q.t0 + (pos - q.start)) * src.token + h * src.head, i % d, rot, pos);
    };
    float amax = 0.0f;
    for (int i = threadIdx.x; i < (last - older) * d; i += 256)
        amax = fmaxf(amax, finite_abs(value(i)));
    for (int m = 1; m < 64; m <<= 1)
        amax = fmaxf(amax, __shfl_xor(amax, m));
    if ((threadIdx.x & 63) == 0)
        part[threadIdx.x >> 6] = amax;
    const float had = older > 0 ? *scale : 0.0f;
    __syncthreads();
    amax = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
    const float now = fmaxf(had, exp2_int(e4m3_scale_exp(amax)));
    if (now != had) {
        const float ratio = had / now;
        for (int i = threadIdx.x; i < older * d; i += 256)
            codes[i] = (uint8_t)e4m3x4(e4m3_to_f32(codes[i]) * ratio, 0.0f, 0.0f, 0.0f);
    }
    for (int i = threadIdx.x; i < (last - older) * d; i += 256)
        codes[older * d + i] = (uint8_t)e4m3x4(value(i) / now, 0.0f, 0.0f, 0.0f);
    __syncthreads();
    if (threadIdx.x == 0)
        *scale = now;
}

// One workgroup per token's queries.
__global__ __launch_bounds__(256) void turn_queries_kernel(Seqs s, Heads q, Rotation r,
                                                           uint16_t *out, int heads, int d)
{
    int b, piece;
    const auto pieces = [&](int i) {
        const Seq e = seq_at(s, i);
        return e.bad ? 0 : e.n;
    };
    if (!find_piece(blockIdx.x, s.B, pieces, b, piece))
        return;
    const Seq e = seq_at(s, b);
    const int64_t t = e.t0 + piece;
    for (int i = threadIdx.x; i < heads * d; i += 256)
        out[t * heads * d + i] =
            f32_to_bf16(turned(q.p + t * q.token + i / d * q.head, i % d, r, e.start + piece));
}

}  // namespace

int32_t launch_append(const engram_cache &c, const Seqs &s, const Heads &k, const Heads &v,
                      const Heads &q, uint16_t *q_out, int32_t q_heads, const Rotation &r,
                      const Launch &l)
{
    // pages: at most one partly filled at each end of a sequence
    const int64_t pieces = s.T / kPage + 2 * (int64_t)s.B;
    dispatch(append_pages_kernel, dim3((unsigned)pieces, c.kv_heads, 2), dim3(256), l, true,
             q_heads == 0, c, s, k, v, r);
    if (q_heads)
        dispatch(turn_queries_kernel, dim3((unsigned)s.T), dim3(256), l, false, true, s, q, r,
                 q_out, (int)q_heads, (int)c.head_dim);
    return launch_status("engram cache_append kernel");
}

}  // namespace engram
