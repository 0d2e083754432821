// Attention over the paged 8-bit cache for many rows a sequence (prompt
// chunks): tiles of 128 rows against 64-token pages staged through LDS.
#include <type_traits>

#include "attend.h"

namespace engram {
namespace {

constexpr int kTileWaves = 4;
constexpr int kTileRows = 32 * kTileWaves;

// 16-byte chunk of a staged row, moved so that eight lanes reading (or
// writing) eight rows meet different banks.
template <int D>
__device__ __forceinline__ int k_chunk(int row, int c)
{
    return D == 64 ? c ^ ((row >> 1) & 3) : c ^ (row & 7);
}
__device__ __forceinline__ int v_chunk(int d, int c) { return c ^ ((d ^ (d >> 2)) & 7); }

constexpr int64_t tile_floats(int d) { return kTileRows * (int64_t)(d + 2); }

// Tile `item` of a call: rows row0 .. of sequence b's.
struct Tile {
    Seq q;
    int b, row0, rows;
    bool on;
};
__device__ __forceinline__ Tile prompt_tile(const AttendArgs &a, int item)
{
    Tile t{{0, 0, 0, false}, 0, 0, 0, true};
    int piece;
    if (!a.s.cu) {
        const int each = (int)(((int64_t)a.s.each * a.g + kTileRows - 1) / kTileRows);
        t.b = (uint32_t)item / (uint32_t)each;
        piece = item - t.b * each;
        t.q = even_seq(a.s, t.b);
    } else {
        t.on = find_piece(item, a.s,
                          [&](const Seq &q) { return (int)(((int64_t)q.n * a.g + kTileRows - 1) / kTileRows); },
                          t.b, piece, t.q);
        if (!t.on)
            return t;
    }
    t.rows = t.q.n * a.g;
    // those that see most keys first
    t.row0 = ((t.rows + kTileRows - 1) / kTileRows - 1 - piece) * kTileRows;
    return t;
}

// A workgroup's four wavefronts take 32 rows each against the same pages, all
// that the rows see or, with SPLIT, one of a.splits equal runs of them, whose
// maxima, sums and outputs go to the workspace.
//
// S^T = K Q^T: lane l holds query l % 32 and, of each 32 tokens, tokens
// 8j + 4(l / 32) + e.  Maximum, sum and rescaling are per lane (and lane ^ 32),
// and the probabilities, taken in the order 16s + 4h + {0..3}, 16s + 8 + 4h +
// {0..3}, are the second operand of O^T = V^T P^T as they stand.  Keys are
// staged as codes, values transposed and widened to bf16 with their tokens in
// that order.
//
// Bound by the matrix and the vector units together, which only overlap where
// their instructions alternate (a wavefront issues in order), and by the
// latency of LDS where little is in flight.  So the pages that every row sees
// whole go through a pipeline of half pages: while a half's probabilities are
// formed, the logits of the next half are multiplied and the values that the
// half needs are read.  One barrier a page; pages are loaded two ahead.  The
// pages with masks come after, one by one.
//
// Two ragged chunks of 4096 tokens at most, 32 heads of 128 over 1500 cached
// positions: 268-280 us, 0.98-1.02 PFLOP/s (a library's bf16 product of 8192^3
// runs at 1.22; pages one by one, without the pipeline, took 351 us), matrix
// units busy 43% of the time and vector units 48%.  4096 tokens after 4096:
// 64-wide heads 243 us, 0.85 PFLOP/s (the vector work of a logit is the same
// beside half the matrix work: 59% and 35%), 256-wide ones 918 us, 0.90 (their
// sums and queries leave one wavefront a SIMD).
template <int D, bool SPLIT>
__global__ __launch_bounds__(64 * kTileWaves, D == 256 ? 1 : 2) void attend_tile_kernel(AttendArgs a)
{
    constexpr int KS = D / 64, DT = D / 32, CH = D / 16;
    constexpr int KB = kPage * D, VB = 2 * kPage * D;
    constexpr int KL = KB / 16 / 256;             // 16-byte chunks of keys a thread stages
    constexpr int VL = D / 128 > 0 ? D / 128 : 1; // 8-token x 4-value blocks of values
    __shared__ __attribute__((aligned(16))) uint8_t lds_k[2][KB];
    __shared__ __attribute__((aligned(16))) uint8_t lds_v[3][VB];
    __shared__ int poison_s;          // some page held a NaN that only some rows see
    const int tid = threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r32 = lane & 31, h = lane >> 5;

    // ---- which rows
    const int kv = a.c.kv_heads;
    const int split = SPLIT ? blockIdx.x % a.splits : 0, at = SPLIT ? blockIdx.x / a.splits : blockIdx.x;
    const int item = (uint32_t)at / (uint32_t)kv, head = at - item * kv;
    const Tile tile = prompt_tile(a, item);
    if (!tile.on) {
        if (blockIdx.x == 0)
            raise_bad(a.s);
        return;
    }
    const Seq q = tile.q;
    const int b = tile.b, rows = tile.rows, row0 = tile.row0;
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
    int first = see_lo / kPage, last = q.bad ? first : pos_hi / kPage + 1;
    if (SPLIT) {
        const int each = (uint32_t)(last - first + a.splits - 1) / (uint32_t)a.splits;
        first += split * each;
        last = min(first + each, last);
    }

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
    const uint32_t k_off = 16 * tid;
    const uint32_t v_off = (16 * (v_group(0) >> 1) + 4 * (v_group(0) & 1)) * D + 4 * quad;
    const auto fetch = [&](int page) {
        const int64_t at = ((int64_t)page * kv + head) * KB;
        const __amdgpu_buffer_rsrc_t kp = __builtin_amdgcn_make_buffer_rsrc(a.c.d_k + at, 0, KB, 0x00027000);
        const __amdgpu_buffer_rsrc_t vp = __builtin_amdgcn_make_buffer_rsrc(a.c.d_v + at, 0, KB, 0x00027000);
#pragma unroll
        for (int i = 0; i < KL; i++)
            kr[i] = __builtin_amdgcn_raw_buffer_load_b128(kp, k_off + 4096 * i, 0, 0);
#pragma unroll
        for (int i = 0; i < VL; i++)
#pragma unroll
            for (int e = 0; e < 8; e++)      // (groups are 1024 / D apart: whole 16-token steps)
                vr[i][e] = __builtin_amdgcn_raw_buffer_load_b32(
                    vp, v_off + (16 * (i * (1024 / D) / 2) + (e & 3) + 8 * (e >> 2)) * D, 0, 0);
    };
    const auto stage_k = [&](int slot) {
#pragma unroll
        for (int i = 0; i < KL; i++) {
            const int c = tid + 256 * i, r = c / CH;
            *(u32x4 *)(lds_k[slot] + 16 * (r * CH + k_chunk<D>(r, c % CH))) = kr[i];
        }
    };
    const auto stage_v = [&](int slot) {
        if (!v_on)
            return;
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
                *(u32x4 *)(lds_v[slot] + 128 * r + 16 * v_chunk(r, g)) = y;
            }
        }
    };
    // whether some row of the workgroup does not see page blk whole
    const auto cut = [&](int blk) {
        return blk * kPage + kPage - 1 > pos_lo ||
               (a.window > 0 && blk * kPage < pos_hi - a.window + 1);
    };

    // ---- the sequence's pages, 64 at a time and one a lane: id and scales
    int from = first, id = -1;
    float ks_lane = 0.0f, vs_lane = 0.0f;
    uint64_t todo = 0;
    // FAST: pages seen whole whose value scale is a power of two (what
    // cache_append writes) of so few bits that, with weights up to 2^40, values
    // up to 2^9 and 2^17 tokens, sums stay in f32's range; else the cache's
    // other pages
    const auto look = [&](auto fast_c) {
        constexpr bool fast = decltype(fast_c)::value;
        const int blk = from + lane;
        id = blk < last ? table[blk] : -1;
        if (id < 0 || id >= a.c.n_pages) {
            if (fast && blk < last)
                raise(a.s.err, ENGRAM_DEVERR_PAGE);
            id = -1;
        } else {
            ks_lane = a.c.d_k_scales[(int64_t)id * kv + head];
            vs_lane = a.c.d_v_scales[(int64_t)id * kv + head];
        }
        const bool plain = vs_lane >= 0x1p-60f && vs_lane <= 0x1p60f &&
                           (__float_as_uint(vs_lane) & 0x7FFFFFu) == 0;
        todo = __ballot(id >= 0 && fast == (plain && !cut(blk)));
    };
    struct Page {
        int id, blk;
        float f, vs;
    };
    const auto next_page = [&](auto fast_c) {
        while (!todo && from + 64 < last) {
            from += 64;
            look(fast_c);
        }
        if (!todo)
            return Page{-1, 0, 0.0f, 0.0f};
        const int i = __builtin_ctzll(todo);
        todo &= todo - 1;
        return Page{__builtin_amdgcn_readlane(id, i), from + i,
                    __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(ks_lane), i)),
                    __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(vs_lane), i))};
    };

    // ---- the steps of half a page (32 tokens)
    uint32_t k_at[KS][2], v_at[4];             // a lane's pieces of row l % 32
#pragma unroll
    for (int u = 0; u < KS; u++)
#pragma unroll
        for (int i = 0; i < 2; i++)
            k_at[u][i] = 16 * (r32 * CH + k_chunk<D>(r32, 4 * u + 2 * h + i));
#pragma unroll
    for (int c = 0; c < 4; c++)
        v_at[c] = 128 * r32 + 16 * v_chunk(r32, 2 * c + h);
    const auto read_keys = [&](const uint8_t *kp, int t, i32x8 (&kf)[KS]) {
#pragma unroll
        for (int u = 0; u < KS; u++) {
            const u32x4 x = *(const u32x4 *)(kp + k_at[u][0] + 32 * D * t);
            const u32x4 y = *(const u32x4 *)(kp + k_at[u][1] + 32 * D * t);
            kf[u] = i32x8{(int)x.x, (int)x.y, (int)x.z, (int)x.w,
                          (int)y.x, (int)y.y, (int)y.z, (int)y.w};
        }
    };
    const auto logits = [&](const uint8_t *kp, int t, f32x16 &s) {
        i32x8 kf[KS];
        read_keys(kp, t, kf);
#pragma unroll
        for (int e = 0; e < 16; e++)
            s[e] = 0.0f;
#pragma unroll
        for (int u = 0; u < KS; u++) {
            s = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(kf[u], qh[u], s, 0, 0, 0, kOne, 0, kOne);
            s = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(kf[u], ql[u], s, 0, 0, 0, kOne, 0, kLoScale);
        }
    };
    // Logits are s * f, f >= 0 (the scale's sign went into the queries).  Moves
    // the base m to their maximum.
    const auto rebase = [&](const f32x16 &s, float f) {
        float top[4];
#pragma unroll
        for (int i = 0; i < 4; i++)
            top[i] = s[i];
#pragma unroll
        for (int e = 4; e < 16; e += 4)
#pragma unroll
            for (int i = 0; i < 4; i++)
                top[i] = __builtin_elementwise_maximum(top[i], s[e + i]);
        // (a NaN passes through, and makes its row NaN whatever the base)
        float t = max_x32(__builtin_elementwise_maximum(__builtin_elementwise_maximum(top[0], top[1]),
                                                        __builtin_elementwise_maximum(top[2], top[3])));
        t = t == -INFINITY ? t : t * f;
        if (__any(t > m)) {
            const float now = fmaxf(m, t);
            const float keep = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - now);
            m = now;
            l *= keep;
#pragma unroll
            for (int i = 0; i < DT; i++)
                o[i] *= keep;
        }
    };
    // 256-wide heads have registers for one of a half's two 16-token steps: the
    // second takes the first's place as that is multiplied
    constexpr int VC = D == 256 ? 1 : 2;
    const auto read_values = [&](const uint8_t *vp, int t, u32x4 (&vf)[VC][DT]) {
#pragma unroll
        for (int c = 0; c < VC; c++)
#pragma unroll
            for (int i = 0; i < DT; i++)
                vf[c][i] = *(const u32x4 *)(vp + v_at[2 * t + c] + 4096 * i);
    };
    const auto values = [&](const uint8_t *vp, int t, u32x4 (&vf)[VC][DT], const u32x4 (&pb)[2]) {
#pragma unroll
        for (int c = 0; c < 2; c++)
#pragma unroll
            for (int i = 0; i < DT; i++) {
                o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, vf[c % VC][i]),
                                                               __builtin_bit_cast(bf16x8, pb[c]), o[i], 0, 0, 0);
                if (c + 1 == VC && VC == 1)
                    vf[0][i] = *(const u32x4 *)(vp + v_at[2 * t + 1] + 4096 * i);
            }
    };
    // 2^(s f - m) times 2^v, a power of two that joins the exponent
    const auto weights = [&](const f32x16 &s, float f, float v, u32x4 (&pb)[2]) {
        const float zero = m - v;
        float sum[4] = {};
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
            const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e], f, -zero));
            const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e + 1], f, -zero));
            sum[e % 4] += p0;
            sum[e % 4 + 1] += p1;
            pb[e / 8][(e % 8) / 2] = cvt_bf16x2(p0, p1);
        }
        return sum[0] + sum[1] + (sum[2] + sum[3]);
    };
    // A step of the pipeline: half t of the page with values at vp, whose logits
    // are s, while those of the next half, half 1-t of the keys at kp, go to
    // s_next.  The base stays where it is until a sum passes 2^40: sums and
    // probabilities are floating point and lose nothing below that.
    const auto half_turn = [&](const Page &cur, const uint8_t *vp, int t, f32x16 &s, const uint8_t *kp,
                               f32x16 &s_next) {
        const float f = qs * cur.f;
        const int v_bits = (int)(__float_as_uint(cur.vs) >> 23) - 127;
        const float zero = m - (float)v_bits;
        u32x4 pb[2], vf[VC][DT];
        i32x8 kf[KS];
        read_keys(kp, 1 - t, kf);
        read_values(vp, t, vf);
        // the instructions in turn: what the vector unit does of these weights, then
        // a matrix instruction of the next logits, which each wait for the last
        constexpr int TURNS = 2 * KS, EACH = 16 / TURNS;
        float part[4] = {};
#pragma unroll
        for (int e = 0; e < 16; e++)
            s_next[e] = 0.0f;
#pragma unroll
        for (int i = 0; i < TURNS; i++) {
#pragma unroll
            for (int e = EACH * i; e < EACH * (i + 1); e += 2) {
                const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e], f, -zero));
                const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e + 1], f, -zero));
                part[e % 4] += p0;
                part[e % 4 + 1] += p1;
                pb[e / 8][(e % 8) / 2] = cvt_bf16x2(p0, p1);
            }
            if (D != 256)
                __builtin_amdgcn_sched_barrier(0);
            s_next = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                kf[i / 2], i & 1 ? ql[i / 2] : qh[i / 2], s_next, 0, 0, 0, kOne, 0, i & 1 ? kLoScale : kOne);
            if (D != 256)
                __builtin_amdgcn_sched_barrier(0);
        }
        // (256-wide heads have no registers for all their keys at once: their reads
        // take turns too)
        if (D == 256) {
            __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
#pragma unroll
            for (int i = 0; i < TURNS; i++) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
                __builtin_amdgcn_sched_group_barrier(0x002, 40 / TURNS, 0);
                __builtin_amdgcn_sched_group_barrier(0x400, 16 / TURNS, 0);
            }
        }
        float sum = part[0] + part[1] + (part[2] + part[3]);
        // (a use of the logits here, or they would be multiplied past the branch,
        // after the vector unit's work instead of beside it)
        asm volatile("" : : "v"(s_next));
        __builtin_amdgcn_sched_barrier(0);
        const float one = exp2_int(-v_bits);
        if (__any(sum * one > 0x1p40f)) {
            rebase(s, f);
            sum = weights(s, f, (float)v_bits, pb);
        }
        l += sum * one;
        values(vp, t, vf, pb);
        __builtin_amdgcn_sched_barrier(0);
    };

    if (tid == 0)
        poison_s = 0;
    look(std::true_type{});
    {
        // p[0]: at work, its values in slot v_slot of three and its keys in slot
        // k_slot of two; p[1]: staged; p[2]: in the registers
        Page p[3];
        p[0] = next_page(std::true_type{});
        if (p[0].id >= 0) {
            for (int i = 1; i < 3; i++)
                p[i] = p[i - 1].id >= 0 ? next_page(std::true_type{}) : p[i - 1];
            // (past the last page p[0] is loaded again, and not used)
            const auto load = [&](const Page &x) { fetch(x.id >= 0 ? x.id : p[0].id); };
            load(p[0]);
            stage_k(0);
            stage_v(0);
            load(p[1]);
            stage_k(1);
            stage_v(1);
            load(p[2]);
            __syncthreads();
            int k_slot = 0, v_slot = 0;
            f32x16 sa, sb;
            logits(lds_k[0], 0, sa);
            rebase(sa, qs * p[0].f);
            while (true) {
                const uint8_t *vp = lds_v[v_slot];
                half_turn(p[0], vp, 0, sa, lds_k[k_slot], sb);
                __syncthreads();                // p[0]'s keys are used, p[1] is staged
                half_turn(p[0], vp, 1, sb, lds_k[k_slot ^ 1], sa);
                if (p[1].id < 0)
                    break;
                stage_k(k_slot);
                v_slot = v_slot == 2 ? 0 : v_slot + 1;
                stage_v(v_slot == 2 ? 0 : v_slot + 1);
                k_slot ^= 1;
                p[0] = p[1];
                p[1] = p[2];
                p[2] = p[1].id >= 0 ? next_page(std::true_type{}) : p[1];
                load(p[2]);
            }
        }
    }

    // ---- the pages that some row does not see whole
    from = first;
    look(std::false_type{});
    while (true) {
        const Page cur = next_page(std::false_type{});
        if (cur.id < 0)
            break;
        const int base = cur.blk * kPage;
        fetch(cur.id);
        __syncthreads();                        // the slots' last readers are done
        // values that no row sees are zeroed (0 * NaN is NaN); a NaN that only
        // some rows see is zeroed and noted: those rows get it at the end
        if (v_on && cut(cur.blk)) {
            uint32_t any = 0;
#pragma unroll
            for (int i = 0; i < VL; i++)
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const int p = base + v_token(i, e);
                    const uint32_t x = p <= pos_hi && p >= see_lo ? vr[i][e] : 0u;
                    const uint32_t nan = nan_bytes(x);
                    any |= nan;
                    vr[i][e] = x & ~nan;
                }
            if (any)
                poison_s = 1;
        }
        stage_k(0);
        stage_v(0);
        __syncthreads();
        // a wavefront whose rows see none of the page passes it by
        if (row0 + 32 * w < rows && base <= my_hi && base + kPage > my_see) {
            const float f = qs * cur.f;
#pragma unroll
            for (int t = 0; t < 2; t++) {
                f32x16 s;
                logits(lds_k[0], t, s);
#pragma unroll
                for (int e = 0; e < 16; e++) {
                    const int p = base + 32 * t + 8 * (e / 4) + 4 * h + e % 4;
                    s[e] = p <= pos && p >= lo ? s[e] : -INFINITY;
                }
                rebase(s, f);
                const float zero = m == -INFINITY ? 0.0f : m;
                u32x4 pb[2], vf[VC][DT];
                read_values(lds_v[0], t, vf);
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    float p[2];
#pragma unroll
                    for (int i = 0; i < 2; i++) {     // (f may be 0, and 0 * -inf NaN)
                        const bool masked = s[e + i] == -INFINITY;
                        p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e + i], f, -zero));
                        l += masked ? 0.0f : p[i];
                        p[i] = masked ? 0.0f : p[i] * cur.vs;
                    }
                    pb[e / 8][(e % 8) / 2] = cvt_bf16x2(p[0], p[1]);
                }
                values(lds_v[0], t, vf, pb);
            }
        }
    }
    __syncthreads();                            // poison_s
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
    if (blockIdx.x == 0)            // last: nothing waits for it
        raise_bad(a.s);
    l = add_x32(l);
    if (!valid)
        return;
    if (SPLIT) {
        float *part = a.part + (int64_t)blockIdx.x * tile_floats(D);
        const int r = 32 * w + r32;
        if (h == 0) {
            part[r] = m;
            part[kTileRows + r] = l;
        }
        part += 2 * kTileRows + r * D;
#pragma unroll
        for (int i = 0; i < DT; i++)
#pragma unroll
            for (int e = 0; e < 16; e += 4)
                *(f32x4 *)(part + 32 * i + 2 * e + 4 * h) = f32x4{o[i][e], o[i][e + 1], o[i][e + 2], o[i][e + 3]};
        return;
    }
    const float inv = l != 0.0f ? 1.0f / l : 0.0f;
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

// Joins the runs of a tile's rows, 16 rows a workgroup.
constexpr int kJoinRows = 16, kJoins = kTileRows / kJoinRows;

template <int D>
__global__ __launch_bounds__(256) void attend_tile_join_kernel(AttendArgs a)
{
    constexpr int QUADS = D / 4;
    const int at = blockIdx.x / kJoins, group = blockIdx.x % kJoins;
    const int item = (uint32_t)at / (uint32_t)a.c.kv_heads, head = at - item * a.c.kv_heads;
    const Tile t = prompt_tile(a, item);
    if (!t.on)
        return;
    const float *parts = a.part + (int64_t)at * a.splits * tile_floats(D);
    const auto place = [&](int i) { return parts + i * tile_floats(D); };
    for (int i = threadIdx.x; i < kJoinRows * QUADS; i += 256) {
        const int r = kJoinRows * group + i / QUADS, d = 4 * (i % QUADS), row = t.row0 + r;
        if (row >= t.rows)
            continue;
        const Joined j = join_row<D, kTileRows, 4>(0, 1, a.splits, r, d, place);
        const float inv = j.l != 0.0f ? 1.0f / j.l : 0.0f;
        const int tok = (uint32_t)row / (uint32_t)a.g;
        u32x2 y;
        y.x = cvt_bf16x2(j.acc.x * inv, j.acc.y * inv);
        y.y = cvt_bf16x2(j.acc.z * inv, j.acc.w * inv);
        *(u32x2 *)(a.out + ((int64_t)(t.q.t0 + tok) * a.heads + head * a.g + row - tok * a.g) * D + d) = y;
    }
}

// Workgroups that share a tile's pages: as many as the chip holds beside each
// other, while each has so many pages of the table's width to read that the time
// it saves (1.2, 1.7 and 3-4 us a page of 64-, 128- and 256-wide heads) exceeds
// the join's 5 us.  512 tokens after 30000, 32 heads of 128 over 8: 565 -> 245
// us; 818 tokens of 6 heads of 64 after 227: 22 -> 18; 2 x 805 of 6 heads of 256
// over 2 after 786: 71 -> 45.  With pieces of 4 pages 64-wide heads lost (750
// tokens in three ragged chunks: 18 -> 21), with 6 256-wide ones (9 pages: 31 -> 36).
// A table much wider than its sequences is cut for its width (256 tokens of 32
// heads without a cache: 13 us, 24 with a table of 2048 columns).
int32_t splits_of(const engram_cache &c, const Seqs &s, int32_t g)
{
    constexpr int64_t kMost = 16;
    const int64_t least = c.head_dim == 64 ? 8 : c.head_dim == 128 ? 6 : 4;
    const int64_t resident = device_cus() * (c.head_dim == 256 ? 1 : 2);
    int64_t n = resident / prompt_tiles(c, s, g);
    n = n < s.max_pages / least ? n : s.max_pages / least;
    return (int32_t)(n < 1 ? 1 : n > kMost ? kMost : n);
}

template <int D>
void launch_dim(const AttendArgs &a, const Launch &l)
{
    const int64_t tiles = prompt_tiles(a.c, a.s, a.g);
    const dim3 block(64 * kTileWaves);
    if (a.splits == 1) {
        dispatch(attend_tile_kernel<D, false>, dim3((unsigned)tiles), block, l, true, true, a);
        return;
    }
    dispatch(attend_tile_kernel<D, true>, dim3((unsigned)(tiles * a.splits)), block, l, true, false, a);
    dispatch(attend_tile_join_kernel<D>, dim3((unsigned)(tiles * kJoins)), dim3(256), l, false, true, a);
}

}  // namespace

int64_t prompt_tiles(const engram_cache &c, const Seqs &s, int32_t g)
{
    return (s.cu ? (int64_t)s.T * g / kTileRows + s.B
                 : (((int64_t)s.each * g + kTileRows - 1) / kTileRows) * s.B) * c.kv_heads;
}

size_t prompt_bytes(const engram_cache &c, const Seqs &s, int32_t g)
{
    const int32_t n = splits_of(c, s, g);
    return n == 1 ? 0 : sizeof(float) * (size_t)(prompt_tiles(c, s, g) * n * tile_floats(c.head_dim));
}

int32_t launch_attend_prompt(const AttendArgs &args, const Launch &l)
{
    AttendArgs a = args;
    a.splits = splits_of(a.c, a.s, a.g);
    if (a.c.head_dim == 64)
        launch_dim<64>(a, l);
    else if (a.c.head_dim == 128)
        launch_dim<128>(a, l);
    else
        launch_dim<256>(a, l);
    return launch_status("engram cache_attend prompt kernel");
}

}  // namespace engram
