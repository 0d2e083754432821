// Attention of a step's queries over the paged 8-bit cache:
//   out = softmax_j(scale * q . k_j) v_j over j <= p (and j > p - window).
//
// One pass over the keys with a running maximum m and sum l of the softmax
// (in base 2): a page's logits s give p = 2^(s - m), and what was summed under
// an older m is multiplied by 2^(m_old - m).  m, l and the sums are f32.
// Roundings to fewer bits: those of p (to bf16, the matrix instructions' type
// for values: at most 2^-8 of a term, in either direction; l sums p as it was,
// which leaves the term's rounding alone in the result), of the result, and in
// the logits those of split_query.
//
// Single tokens are bound by memory, the cache's bytes: 64 sequences of up to
// 8192 positions (581 MB) in 103 us, 99 of them in the kernel that reads
// (5.9 TB/s, where a stream that only reads reaches 6.6); one of 131072
// positions with 256-wide heads (268 MB) in 52 us, 47 and 5 for the join.
// Short calls are bound by latency: 4.4 us with no page to read, 5.9 with one,
// and a CU takes in some 51 bytes a ns (8 pages of 128-wide heads by a CU a unit:
// 8.4 us; by two, each with half the values: 7.4).
#include <type_traits>

#include "attend.h"

namespace engram {
namespace {

// ---- how the keys are divided
//
// A unit is a row tile and a key head.  Every unit of a sequence counts the
// same number of pages, and all units' pages lie in one row, sequence by
// sequence, that the workgroups share out whatever the sequences' lengths are,
// so that all end together.  Where units are fewer than workgroups, a unit's
// pages are cut into equal pieces, one a workgroup; else workgroup i takes
// pages i*share .. (i+1)*share-1 of the row.  A unit that lies in one workgroup
// is written out there; parts of a unit go to the workgroup's two places in the
// workspace (0 for its first part, 1 for a last one that is not its first) and
// are joined by a second kernel.

// Pages that each unit of sequence b counts: 0 where it brings no token.
__device__ __forceinline__ int unit_pages(const AttendArgs &a, const Seq &q)
{
    if (q.n == 0)
        return 0;
    if (q.bad)
        return 1;
    const int all = (q.start + q.n - 1) / kPage + 1;
    const int reach = a.window_pages;
    return reach > 0 && reach < all ? reach : all;
}
__device__ __forceinline__ int unit_tiles(const AttendArgs &a, const Seq &q)
{
    return (int)(((int64_t)q.n * a.g + kRows - 1) / kRows);
}

// Sequences base .. base+63, one a lane, with their units and pieces and the
// sums of both up to and with them (a call's units x pages stay below 2^30).
// A piece is a page, or, with most > 0, a run of `most` pages of a unit (the
// last one what is left).
struct Lanes {
    Seq q;
    int each, units, pieces, sum_u, sum_p;          // each: pieces a unit
    int32_t reach;                                  // the furthest token up to and with them
    __device__ __forceinline__ int all_units() const { return __builtin_amdgcn_readlane(sum_u, 63); }
    __device__ __forceinline__ int all_pieces() const { return __builtin_amdgcn_readlane(sum_p, 63); }
    __device__ __forceinline__ void cut(int most)
    {
        each = (int)((uint32_t)(each + most - 1) / (uint32_t)most);
        pieces = units * each;
        sum_p = wave_scan(pieces);
    }
};
// (reach: that of the sequences before base.)
__device__ __forceinline__ Lanes lanes_at(const AttendArgs &a, int base, int32_t reach, int most = 0)
{
    Lanes c;
    c.reach = reach;
    c.q = seqs_at(a.s, base, c.reach);
    c.each = unit_pages(a, c.q);
    c.units = unit_tiles(a, c.q) * a.c.kv_heads;
    c.pieces = c.units * c.each;
    c.sum_u = wave_scan(c.units);
    if (most > 0)
        c.cut(most);
    else
        c.sum_p = wave_scan(c.pieces);
    return c;
}

// How a call's pages are shared out: pieces a workgroup, pieces in all, and the
// pages a piece holds (0: pieces are pages).
struct Plan {
    int share, total, most;
};

// A workgroup whose share ends inside a unit and goes on in the next one begins
// anew there, which takes as long as 16 pages of its four wavefronts (4 us; 16
// sequences of 1180 positions with 256-wide heads took 18 us that way).  So
// units are cut evenly unless the longest piece then passes a share by more.
constexpr int kBeginPages = 16;

// (c: the first sequences' lanes, cut as the plan says.)
__device__ __forceinline__ Plan plan_of(const AttendArgs &a, Lanes &c)
{
    int total = c.all_pieces(), units = c.all_units();
    int32_t reach = c.reach;
    for (int base = 64; base < a.s.B; base += 64) {
        const Lanes next = lanes_at(a, base, reach);
        total += next.all_pieces();
        units += next.all_units();
        reach = next.reach;
    }
    const int share = max((int)(((uint32_t)total + a.parts - 1) / (uint32_t)a.parts), a.least);
    if (units < a.parts) {
        // pieces of a share's pages, if no more than workgroups come of it; else of
        // so many that they are at most total / most + units <= parts
        const int pages = c.each;
        int most = share;
#pragma unroll 1
        do {
            c.each = pages;
            c.cut(most);
            int pieces = c.all_pieces();
            reach = c.reach;
            for (int base = 64; base < a.s.B; base += 64) {
                const Lanes next = lanes_at(a, base, reach, most);
                pieces += next.all_pieces();
                reach = next.reach;
            }
            if (pieces <= a.parts)
                return Plan{1, pieces, most};
            const uint32_t left = a.parts - units;
            most = (int)(((uint32_t)total + left - 1) / left);      // > share: pieces were too many
        } while (most <= share + kBeginPages);
        c.each = pages;
        c.cut(1);
    }
    return Plan{share, total, 0};
}

__device__ __forceinline__ RowTile tile_at(const AttendArgs &a, int b, int unit, const Seq &q)
{
    RowTile t;
    t.b = b;
    const int tile = (uint32_t)unit / (uint32_t)a.c.kv_heads;
    t.h = unit - tile * a.c.kv_heads;
    t.row0 = tile * kRows;
    t.q = q;
    t.rows = q.n * a.g;
    return t;
}

__device__ __forceinline__ uint16_t *out_row(const AttendArgs &a, const RowTile &t, int row, int D)
{
    const int tok = (uint32_t)row / (uint32_t)a.g;
    return a.out + ((int64_t)(t.q.t0 + tok) * a.heads + t.h * a.g + row - tok * a.g) * D;
}

template <int D>
__device__ __forceinline__ void store_row(const AttendArgs &a, const RowTile &t, int row, int d,
                                          f32x4 acc, float l)
{
    const float inv = l != 0.0f ? 1.0f / l : 0.0f;
    u32x2 y;
    y.x = cvt_bf16x2(acc.x * inv, acc.y * inv);
    y.y = cvt_bf16x2(acc.z * inv, acc.w * inv);
    *(u32x2 *)(out_row(a, t, row, D) + d) = y;
}

// O^T += V^T P^T over a page's 64 tokens: vf[j][e] holds, of token
// 16j + 4(l / 16) + e, the D/16 codes from value (l % 16) * D/16 on, pb[j] the
// probabilities of those four tokens as bf16.  Output tile u takes value
// (l % 16) * D/16 + u of every lane: get(u) is what it starts from, put(u, sum)
// receives it.  Codes of four tokens are paired by byte permutes and widened
// to bf16, whose eight bits hold a code exactly.
template <int D, class G, class P>
__device__ __forceinline__ void values_product(const uint32_t (&vf)[4][4][D / 64],
                                               const uint32_t (&pb)[4][2], G get, P put)
{
    u32x4 pv[2];
#pragma unroll
    for (int h = 0; h < 2; h++)
        pv[h] = u32x4{pb[2 * h][0], pb[2 * h][1], pb[2 * h + 1][0], pb[2 * h + 1][1]};
#pragma unroll
    for (int u = 0; u < D / 64; u++) {
        f32x4 acc[4];
#pragma unroll
        for (int i = 0; i < 4; i++)
            acc[i] = get(4 * u + i);
#pragma unroll
        for (int h = 0; h < 2; h++) {
            uint32_t ab[2][2], cd[2][2];          // byte pairs of tokens 0,1 and 2,3
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const uint32_t(&x)[4][D / 64] = vf[2 * h + j];
                ab[j][0] = __builtin_amdgcn_perm(x[1][u], x[0][u], 0x05010400u);
                ab[j][1] = __builtin_amdgcn_perm(x[1][u], x[0][u], 0x07030602u);
                cd[j][0] = __builtin_amdgcn_perm(x[3][u], x[2][u], 0x05010400u);
                cd[j][1] = __builtin_amdgcn_perm(x[3][u], x[2][u], 0x07030602u);
            }
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int b = i / 2;
                const u32x4 vv = i & 1 ? u32x4{widen2<true>(ab[0][b]), widen2<true>(cd[0][b]),
                                               widen2<true>(ab[1][b]), widen2<true>(cd[1][b])}
                                       : u32x4{widen2<false>(ab[0][b]), widen2<false>(cd[0][b]),
                                               widen2<false>(ab[1][b]), widen2<false>(cd[1][b])};
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    __builtin_bit_cast(bf16x8, vv), __builtin_bit_cast(bf16x8, pv[h]), acc[i], 0, 0,
                    0);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; i++)
            put(4 * u + i, acc[i]);
    }
}

// Pages p0 .. p0+np-1 of a unit, by W wavefronts.
//
// The wavefronts take pages in turn and keep m, l and the output sums of
// their own; the sums meet in LDS at the end.  S^T = K Q^T puts a query in each
// lane column (lane l holds query l % 16 and tokens 16t + 4(l / 16) + e of a
// page), so m, l and the rescaling are per lane, and the probabilities are
// already laid out as the second operand of O^T = V^T P^T, whose contraction
// takes the tokens in that same order.  Keys go from memory into matrix
// instructions as the codes they are (the query is split into two e4m3 parts);
// values are paired by token with byte permutes and widened to bf16.  Nothing
// of the cache passes through LDS.  Output values v0 .. v0+DV-1 of the head.
template <int DV, int W>
struct Reduce {
    float o[W][kRows][DV + 4];
    float m[W][kRows], l[W][kRows];
};

template <int D, int W, int DV>
__device__ __forceinline__ void attend_unit(const AttendArgs &a, const RowTile &t, int p0, int np,
                                            int v0, float *part, Reduce<DV, W> &red)
{
    constexpr int KS = D == 64 ? 1 : D / 128;     // 128-value steps of the logits
    constexpr int VW = DV / 64;                   // dwords of a token's values a lane holds
    int tid = threadIdx.x;
    // opaque, so that what is derived from it is not kept in registers over
    // the caller's loop
    asm volatile("" : "+v"(tid));
    const int lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, q4 = lane >> 4;

    // ---- what the rows see
    const int row = t.row0 + r16;
    const bool valid = row < t.rows;
    const int tok = valid ? (uint32_t)row / (uint32_t)a.g : 0;
    const int pos = t.q.start + tok;
    const int lo = a.window > 0 ? max(pos - a.window + 1, 0) : 0;
    const int pos_lo = t.q.start + (uint32_t)t.row0 / (uint32_t)a.g;          // the tile's first and last position
    const int pos_hi = t.q.start + (uint32_t)min(t.row0 + kRows - 1, t.rows - 1) / (uint32_t)a.g;
    const int see_lo = a.window > 0 ? max(pos_lo - a.window + 1, 0) : 0;     // seen by any row
    const int all_lo = a.window > 0 ? max(pos_hi - a.window + 1, 0) : 0;     // seen by every row
    const int first = see_lo / kPage + p0;
    const int last = t.q.bad ? first : min(first + np, pos_hi / kPage + 1);

    float m = -INFINITY, l = 0.0f;
    f32x4 o[DV / 16];
#pragma unroll
    for (int i = 0; i < DV / 16; i++)
        o[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    i32x8 kf[4][KS];
    uint32_t vf[4][4][VW];
    float ks = 0.0f, vs = 0.0f, vs_next = 0.0f;
    // a lane's place in a page: 32 bits on top of the page's uniform address
    const uint32_t k_off = r16 * D + (D == 64 ? 16 : 32) * q4;
    const uint32_t v_off = 4 * q4 * D + v0 + r16 * (4 * VW);
    const auto load_k = [&](int64_t at) {
        const uint8_t *kp = a.c.d_k + at * (kPage * D);
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int s = 0; s < KS; s++) {
                const uint8_t *p = kp + 16 * i * D + 128 * s;
                const u32x4 u = __builtin_nontemporal_load((const u32x4 *)(p + k_off));
                const u32x4 v = D == 64 ? u : __builtin_nontemporal_load((const u32x4 *)(p + 16 + k_off));
                kf[i][s] = i32x8{(int)u.x, (int)u.y, (int)u.z, (int)u.w,
                                 (int)v.x, (int)v.y, (int)v.z, (int)v.w};
            }
        ks = a.c.d_k_scales[at];
        vs_next = a.c.d_v_scales[at];
    };
    const auto load_v = [&](int64_t at) {
        const uint8_t *vp = a.c.d_v + at * (kPage * D);
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const uint8_t *p = vp + (16 * i + e) * D + v_off;
                if (VW == 1) {
                    vf[i][e][0] = __builtin_nontemporal_load((const uint32_t *)p);
                } else if (VW == 2) {
                    const u32x2 u = __builtin_nontemporal_load((const u32x2 *)p);
                    vf[i][e][0] = u.x;
                    vf[i][e][1] = u.y;
                } else {
                    const u32x4 u = __builtin_nontemporal_load((const u32x4 *)p);
                    vf[i][e][0] = u.x;
                    vf[i][e][1] = u.y;
                    vf[i][e][2 % VW] = u.z;
                    vf[i][e][3 % VW] = u.w;
                }
            }
    };

    // The wavefront's pages, 64 at a time and one a lane: first those that
    // every row sees whole, then the others.  The first is on its way before
    // the queries are looked at.
    const int32_t *table = a.s.pages + (int64_t)t.b * a.s.max_pages;
    uint64_t whole = 0, rest = 0;
    int id = -1;
    const auto entry = [&](int p) { return p + W * lane < last ? table[p + W * lane] : -1; };
    const auto sort = [&](int p, int entry_id) {
        const int mine = p + W * lane;
        id = entry_id;
        if (id < 0 || id >= a.c.n_pages) {
            if (mine < last)
                raise(a.s.err, ENGRAM_DEVERR_PAGE);
            id = -1;
        }
        const bool full = mine * kPage + kPage - 1 <= pos_lo && mine * kPage >= all_lo;
        whole = __ballot(id >= 0 && full);
        rest = __ballot(id >= 0 && !full);
    };
    // the place of the page to come next, -1 past the last
    const auto ahead = [&] { return whole ? __builtin_ctzll(whole) : rest ? __builtin_ctzll(rest) : -1; };
    const auto load = [&](int i) {
        const int64_t at = (int64_t)__builtin_amdgcn_readlane(id, i) * a.c.kv_heads + t.h;
        load_k(at);
        load_v(at);
    };

    // ---- the queries
    const int entry_0 = entry(first + w);
    u32x4 x[KS][4];
    const uint16_t *qp = a.q.p + (int64_t)(t.q.t0 + tok) * a.q.token +
                         (int64_t)(t.h * a.g + (valid ? row - tok * a.g : 0)) * a.q.head;
#pragma unroll
    for (int s = 0; s < KS; s++)
#pragma unroll
        for (int i = 0; i < 4; i++)
            x[s][i] = *(const u32x4 *)(qp + (D == 64 ? 16 * q4 : 128 * s + 32 * q4) +
                                       8 * (D == 64 ? i & 1 : i));
    sort(first + w, entry_0);
    int i = ahead();
    if (i >= 0)
        load(i);
    __builtin_amdgcn_sched_barrier(0);

    i32x8 qh[KS], ql[KS];
    float qs = 0.0f;
    {
        float amax = 0.0f;
#pragma unroll
        for (int s = 0; s < KS; s++) {
#pragma unroll
            for (int i = 0; i < 4; i++)
                if (!valid)
                    x[s][i] = u32x4{0u, 0u, 0u, 0u};
            amax = fmaxf(amax, amax_bf16(x[s]));
        }
        const int k = e4m3_scale_exp(max_x16(amax));
        qs = exp2_int(k) * a.scale;
#pragma unroll
        for (int s = 0; s < KS; s++)
            split_query(x[s], exp2_int(-k), qh[s], ql[s]);
    }
    // head_dim 64: one instruction takes both parts.  A lane's first 16 codes
    // are the contraction's indices 16(l / 16) on, under the scales of lanes
    // 0-31, its last 16 those from 64 on, under the scales of lanes 32-63.
    const int sel_scale = D == 64 && q4 >= 2 ? kLoScale : kOne;
    if (D == 64)
#pragma unroll
        for (int i = 0; i < 4; i++)
            qh[0][4 + i] = ql[0][i];

    // One page.  FULL: every row sees all of it, and the next such page is
    // loaded meanwhile: its keys once this one's are used, its values likewise
    // (the barriers keep the compiler from loading into other registers and
    // waiting for them in order to copy).
    const auto step = [&](auto full_c, int page, int base, int next) {
        constexpr bool edge = !decltype(full_c)::value;
        const int64_t at_next = (int64_t)next * a.c.kv_heads + t.h;
        // ---- logits
        f32x4 s[4];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            s[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int u = 0; u < KS; u++) {
                s[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(kf[j][u], qh[u], s[j], 0, 0, 0,
                                                                        kOne, 0, sel_scale);
                if (D != 64)
                    s[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        kf[j][u], ql[u], s[j], 0, 0, 0, kOne, 0, kLoScale);
            }
        }
        const float f = qs * ks;
        vs = vs_next;
        if (!edge) {
            __builtin_amdgcn_sched_barrier(0);
            if (next >= 0)
                load_k(at_next);
            __builtin_amdgcn_sched_barrier(0);
        }
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; j++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                s[j][e] *= f;
                if (edge) {
                    const int p = base + 16 * j + 4 * q4 + e;
                    s[j][e] = p <= pos && p >= lo ? s[j][e] : -INFINITY;
                }
                top = fmaxf(top, s[j][e]);
            }
        top = fmaxf(max_x16(top), m);
        const float zero = top == -INFINITY ? 0.0f : top;
        if (__any(top != m)) {
            const float keep = __builtin_amdgcn_exp2f(m - zero);
            m = top;
            l *= keep;
#pragma unroll
            for (int j = 0; j < DV / 16; j++)
                o[j] *= keep;
        }
        uint32_t pb[4][2];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            float p[4];
#pragma unroll
            for (int e = 0; e < 4; e++) {
                p[e] = __builtin_amdgcn_exp2f(s[j][e] - zero);
                l += p[e];
                const bool masked = edge && s[j][e] == -INFINITY;
                p[e] = masked ? 0.0f : p[e] * vs;
            }
            pb[j][0] = cvt_bf16x2(p[0], p[1]);
            pb[j][1] = cvt_bf16x2(p[2], p[3]);
        }
        // ---- values: what no row sees is zeroed (0 * NaN is NaN); a NaN that
        // only some rows see is zeroed here and given to them below
        bool poison = false;
        if (edge) {
#pragma unroll
            for (int j = 0; j < 4; j++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int p = base + 16 * j + 4 * q4 + e;
                    const bool seen = p <= pos_hi && p >= see_lo;
#pragma unroll
                    for (int u = 0; u < VW; u++)
                        vf[j][e][u] = seen ? vf[j][e][u] : 0u;
                }
            if (pos_lo != pos_hi) {
                uint32_t any = 0;
#pragma unroll
                for (int j = 0; j < 4; j++)
#pragma unroll
                    for (int e = 0; e < 4; e++)
#pragma unroll
                        for (int u = 0; u < VW; u++) {
                            const uint32_t nan = nan_bytes(vf[j][e][u]);
                            any |= nan;
                            vf[j][e][u] &= ~nan;
                        }
                poison = __any(any != 0);
            }
        }
        values_product<DV>(vf, pb, [&](int u) { return o[u]; },
                           [&](int u, const f32x4 &sum) { o[u] = sum; });
        if (poison) {
            // how many NaN codes each row sees, by the same product
            load_v((int64_t)page * a.c.kv_heads + t.h);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                float p[4];
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int at = base + 16 * j + 4 * q4 + e;
                    p[e] = at <= pos && at >= lo ? 1.0f : 0.0f;
#pragma unroll
                    for (int u = 0; u < VW; u++)      // 0x38 is 1.0
                        vf[j][e][u] = nan_bytes(vf[j][e][u]) & 0x38383838u;
                }
                pb[j][0] = cvt_bf16x2(p[0], p[1]);
                pb[j][1] = cvt_bf16x2(p[2], p[3]);
            }
            values_product<DV>(vf, pb, [&](int) { return f32x4{0.0f, 0.0f, 0.0f, 0.0f}; },
                               [&](int u, const f32x4 &n) {
#pragma unroll
                for (int e = 0; e < 4; e++)
                    o[u][e] = n[e] > 0.0f ? __uint_as_float(0x7FC00000u) : o[u][e];
            });
        }
        if (!edge) {
            __builtin_amdgcn_sched_barrier(0);
            if (next >= 0)
                load_v(at_next);
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    for (int p = first + w; p < last; p += 64 * W) {
        if (p != first + w) {
            sort(p, entry(p));
            i = ahead();
            if (i >= 0)
                load(i);
        }
        while (whole) {
            whole &= whole - 1;
            const int page = __builtin_amdgcn_readlane(id, i), base = (p + W * i) * kPage;
            i = ahead();
            step(std::true_type{}, page, base, i >= 0 ? __builtin_amdgcn_readlane(id, i) : -1);
        }
        while (rest) {
            rest &= rest - 1;
            step(std::false_type{}, __builtin_amdgcn_readlane(id, i), (p + W * i) * kPage, -1);
            i = ahead();
            if (i >= 0)
                load(i);
        }
    }

    // ---- the wavefronts' sums
    l = add_x16(l);
    if (q4 == 0) {
        red.m[w][r16] = m;
        red.l[w][r16] = l;
    }
#pragma unroll
    for (int e = 0; e < 4; e++)
#pragma unroll
        for (int u = 0; u < DV / 16; u += 4)
            *(f32x4 *)&red.o[w][r16][(4 * q4 + e) * (DV / 16) + u] =
                f32x4{o[u][e], o[u + 1][e], o[u + 2][e], o[u + 3][e]};
    __syncthreads();
    constexpr int QUADS = DV / 4;
    const int rows = min(kRows, t.rows - t.row0);
    for (int i = tid; i < rows * QUADS; i += 64 * W) {
        const int r = i / QUADS, d = 4 * (i % QUADS);
        float mm = -INFINITY;
#pragma unroll
        for (int u = 0; u < W; u++)
            mm = fmaxf(mm, red.m[u][r]);
        const float zero = mm == -INFINITY ? 0.0f : mm;
        float ll = 0.0f;
        f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int u = 0; u < W; u++) {
            const float k = __builtin_amdgcn_exp2f(red.m[u][r] - zero);
            ll += k * red.l[u][r];
            acc += k * *(const f32x4 *)&red.o[u][r][d];
        }
        if (!part) {
            store_row<D>(a, t, t.row0 + r, v0 + d, acc, ll);
        } else {
            *(f32x4 *)(part + 2 * kRows + r * D + d) = acc;
            if (d == 0) {
                part[r] = mm;
                part[kRows + r] = ll;
            }
        }
    }
}

__device__ __forceinline__ void raise_bad(const AttendArgs &a)
{
    if (blockIdx.x == 0)
        raise_bad(a.s);
}

// Short tables: a workgroup a unit and DV of its output values, nothing to join.
template <int D, int W, int DV>
__global__ __launch_bounds__(64 * W, W == 8 ? 2 : 1) void attend_unit_kernel(AttendArgs a)
{
    __shared__ Reduce<DV, W> red;
    const int v0 = DV * (blockIdx.x % (D / DV)), at = blockIdx.x / (D / DV);
    int b, unit;
    Seq q;
    if (!a.s.cu) {
        const int units = (int)(((int64_t)a.s.each * a.g + kRows - 1) / kRows) * a.c.kv_heads;
        b = at / units;
        unit = at % units;
        q = even_seq(a.s, b);
    } else {
        unit = at;
        Lanes c = lanes_at(a, 0, 0);
        int base = 0;
        while (unit >= c.all_units()) {
            unit -= c.all_units();
            base += 64;
            if (base >= a.s.B) {
                raise_bad(a);
                return;
            }
            c = lanes_at(a, base, c.reach);
        }
        const int l = __builtin_ctzll(__ballot(c.sum_u > unit));
        b = base + l;
        unit -= __builtin_amdgcn_readlane(c.sum_u - c.units, l);
        q = lane_seq(c.q, l);
    }
    const RowTile t = tile_at(a, b, unit, q);
    attend_unit<D, W, DV>(a, t, 0, 1 << 26, v0, nullptr, red);
    raise_bad(a);                               // last: nothing waits for it
}

// Long tables: a workgroup a share of the row of pages.
template <int D, int W>
__global__ __launch_bounds__(64 * W, D == 256 ? 1 : 2) void attend_share_kernel(AttendArgs a)
{
    __shared__ Reduce<D, W> red;
    __shared__ Seq seqs[64];
    __shared__ int each_s[64], units_s[64];
    Lanes c = lanes_at(a, 0, 0);
    const Plan plan = plan_of(a, c);
    if ((int64_t)blockIdx.x * plan.share >= plan.total) {
        raise_bad(a);
        return;
    }
    int at = blockIdx.x * plan.share;
    const int end = min((int64_t)at + plan.share, (int64_t)plan.total);
    // the sequence, unit and piece that the share begins with; the sequences
    // wait in LDS while a unit is at work (its registers are all taken)
    int base = 0, before = 0;
    while (before + c.all_pieces() <= at) {
        before += c.all_pieces();
        base += 64;
        c = lanes_at(a, base, c.reach, plan.most);
    }
    int l = __builtin_ctzll(__ballot(before + c.sum_p > at));
    int p0 = at - before - __builtin_amdgcn_readlane(c.sum_p - c.pieces, l);
    int unit = (uint32_t)p0 / (uint32_t)__builtin_amdgcn_readlane(c.each, l);
    p0 -= unit * __builtin_amdgcn_readlane(c.each, l);
    const auto keep = [&] {
        __syncthreads();                        // the sequences before these have been read
        if (threadIdx.x < 64) {
            seqs[threadIdx.x] = c.q;
            each_s[threadIdx.x] = c.each;
            units_s[threadIdx.x] = c.pieces ? c.units : 0;
        }
        __syncthreads();
    };
    keep();
    const int step = plan.most > 0 ? plan.most : 1;
    float *part = a.part + 2 * (int64_t)blockIdx.x * part_floats(D);
    int place = 0;
    while (true) {
        const int each = __builtin_amdgcn_readfirstlane(each_s[l]);
        const int np = min(each - p0, end - at);
        const Seq q{__builtin_amdgcn_readfirstlane(seqs[l].t0), __builtin_amdgcn_readfirstlane(seqs[l].n),
                    __builtin_amdgcn_readfirstlane(seqs[l].start),
                    (bool)__builtin_amdgcn_readfirstlane(seqs[l].bad)};
        attend_unit<D, W, D>(a, tile_at(a, base + l, unit, q), p0 * step, np * step, 0,
                             np == each ? nullptr : part + place * part_floats(D), red);
        at += np;
        if (at >= end)
            break;
        place = 1;
        p0 = 0;
        __syncthreads();                        // the sums in LDS have been read
        if (++unit == __builtin_amdgcn_readfirstlane(units_s[l])) {
            unit = 0;
            do {                                // (at < end: there is one)
                if (++l == 64) {
                    l = 0;
                    base += 64;
                    const Lanes next = lanes_at(a, base, c.reach, plan.most);
                    c = next;
                    keep();
                }
            } while (__builtin_amdgcn_readfirstlane(units_s[l]) == 0);
        }
    }
    raise_bad(a);
}

// Joins the parts of a unit's rows.  A workgroup takes a unit, or, with
// SPLIT, where units are few and their parts many, a unit's row; G thread
// groups of D/4 then take parts in turn.
template <int D, bool SPLIT>
__global__ __launch_bounds__(512) void attend_join_kernel(AttendArgs a)
{
    constexpr int QUADS = D / 4, GROUPS = 512 / QUADS;
    __shared__ f32x4 acc_s[GROUPS][QUADS];
    __shared__ float l_s[GROUPS], m_s[GROUPS];
    const int tid = threadIdx.x;
    const int r0 = SPLIT ? blockIdx.x % a.join_rows : 0;
    int unit = SPLIT ? blockIdx.x / a.join_rows : blockIdx.x;
    Lanes c = lanes_at(a, 0, 0);
    const Plan plan = plan_of(a, c);
    int base = 0, before = 0;
    while (unit >= c.all_units()) {
        unit -= c.all_units();
        before += c.all_pieces();
        base += 64;
        if (base >= a.s.B)
            return;
        c = lanes_at(a, base, c.reach, plan.most);
    }
    const int l = __builtin_ctzll(__ballot(c.sum_u > unit));
    unit -= __builtin_amdgcn_readlane(c.sum_u - c.units, l);
    const RowTile t = tile_at(a, base + l, unit, lane_seq(c.q, l));
    const int each = __builtin_amdgcn_readlane(c.each, l);
    const int begin = before + __builtin_amdgcn_readlane(c.sum_p - c.pieces, l) + unit * each;
    int i0 = begin, n = each;
    if (plan.share > 1) {
        i0 = (uint32_t)begin / (uint32_t)plan.share;
        n = (uint32_t)(begin + each - 1) / (uint32_t)plan.share - i0 + 1;
    }
    const int rows = min(kRows, t.rows - t.row0);
    if (n == 1 || r0 >= rows)
        return;
    // part i of the unit
    const auto place = [&](int i) {
        return a.part + (2 * (int64_t)(i0 + i) + ((i0 + i) * plan.share >= begin ? 0 : 1)) * part_floats(D);
    };
    const int g = tid / QUADS, d = tid % QUADS;
    if (!SPLIT) {
        for (int r = g; r < rows; r += GROUPS) {
            const Joined j = join_row<D, kRows, 2>(0, 1, n, r, 4 * d, place);
            store_row<D>(a, t, t.row0 + r, 4 * d, j.acc, j.l);
        }
        return;
    }
    Joined j = n <= GROUPS ? join_row<D, kRows, 1>(g, GROUPS, n, r0, 4 * d, place)
                           : join_row<D, kRows, 8>(g, GROUPS, n, r0, 4 * d, place);
    acc_s[g][d] = j.acc;
    if (d == 0) {
        m_s[g] = j.m;
        l_s[g] = j.l;
    }
    __syncthreads();
    if (g == 0) {
        const int groups = min(n, GROUPS);
        for (int u = 1; u < groups; u++)
            j.add(m_s[u], l_s[u], acc_s[u][d]);
        store_row<D>(a, t, t.row0 + r0, 4 * d, j.acc, j.l);
    }
}

// Which kernel a call takes: tiles of 128 rows where the call has a workgroup
// of them for every eighth CU, else tiles of 16 whose keys are shared out.  (In
// us, 16-row tiles against 128-row ones with their pages shared out: 534 tokens
// of 48 heads over 8 key heads 53 and 20; 816 tokens of 16 heads over 2 35 and
// 23; 818 tokens of 6 64-wide heads over 1 after 227, 39 tiles, 15 and 18; 2 x
// 4096 ragged tokens of 32 heads 1662 and 279; 64 tokens of 32 heads over 8, 16
// tiles, 9 and 20 after 500, 29 and 25 after 4000; 3 x 16 tokens of 64 64-wide
// heads over 8 after 834 8 and 19.)  It holds for the whole call: single tokens
// beside a prompt go through its tiles, one workgroup a key head each where the
// prompt's tiles fill the chip (4096 tokens and one over 131000: 2527 us, 168 and
// 56 in two calls).
bool many_rows(const engram_cache &c, const Seqs &s, int32_t g)
{
    return (int64_t)s.T * g >= 64 * (int64_t)s.B && prompt_tiles(c, s, g) >= device_cus() / 8;
}

// Units of 16 rows that a call has at most.
int64_t row_units(const engram_cache &c, const Seqs &s, int32_t g)
{
    return (s.cu ? (int64_t)s.T * g / kRows + s.B
                 : (((int64_t)s.each * g + kRows - 1) / kRows) * s.B) * c.kv_heads;
}

// Tables of so few pages are read without a join, whose launch costs 4.7 us.
// In us, without and with it, for 8 units of 128-wide heads: 8 pages 8.4 and 10.4,
// 16 11.4 and 10.7, 24 14.7 and 11.0; 64-wide heads: 16 pages 8.1 and 9.0, 24
// 10.4 and 9.3; 256-wide: 8 pages 12.1 and 14.0, 12 15.4 and 14.6, 16 18.4 and
// 14.9.  With 512 units it is faster up to 32 pages at least (128-wide: 39.6 and
// 45.0).  The table's width counts, not the sequences': the host does not see
// their lengths.
constexpr int kShortPages = 16;
constexpr int kLeastShare = 4;

// Workgroups that share the pages out: two a CU, one with 256-wide heads
// (whose wavefronts need a SIMD's registers alone).
int32_t parts_of(const engram_cache &c)
{
    return device_cus() * (c.head_dim == 256 ? 1 : 2);
}

}  // namespace

size_t attend_bytes(const engram_cache &c, const Seqs &s, int32_t q_heads)
{
    if (many_rows(c, s, q_heads / c.kv_heads))
        return prompt_bytes(c, s, q_heads / c.kv_heads);
    if (s.max_pages <= kShortPages)
        return 0;
    return sizeof(float) * 2 * (size_t)parts_of(c) * (size_t)part_floats(c.head_dim);
}

template <int D>
static void launch_rows(const AttendArgs &a, int64_t units, const Launch &l)
{
    if (a.s.max_pages <= kShortPages) {
        // Where units leave CUs idle, one takes a unit's keys and 64 of its values
        // a workgroup: a CU takes in only so much (see above).
        constexpr int W = D == 256 ? 4 : 8;
        if (D > 64 && units * (D / 64) <= device_cus())
            dispatch(attend_unit_kernel<D, 8, 64>, dim3((unsigned)(units * (D / 64))), dim3(512), l,
                     true, true, a);
        else
            dispatch(attend_unit_kernel<D, W, D>, dim3((unsigned)units), dim3(64 * W), l, true, true,
                     a);
        return;
    }
    dispatch(attend_share_kernel<D, 4>, dim3((unsigned)a.parts), dim3(256), l, true, false, a);
    if (units < a.parts / 2)
        dispatch(attend_join_kernel<D, true>, dim3((unsigned)(units * a.join_rows)), dim3(512), l,
                 false, true, a);
    else
        dispatch(attend_join_kernel<D, false>, dim3((unsigned)units), dim3(512), l, false, true,
                 a);
}

int32_t launch_attend(const engram_cache &c, const Seqs &s, const Heads &q, uint16_t *out,
                      int32_t q_heads, float scale, int64_t window, void *ws, const Launch &l)
{
    const int32_t g = q_heads / c.kv_heads;
    const int32_t w = window < ((int64_t)1 << 31) ? (int32_t)window : 0;
    AttendArgs a{c, s, q, out, q_heads, g, scale * kLog2e, w, 0, 0, 0, 0, 1, (float *)ws};
    const bool many = many_rows(c, s, g);
    const int64_t units = many ? prompt_tiles(c, s, g) : row_units(c, s, g);
    a.join_rows = !s.cu && (int64_t)s.each * g < kRows ? s.each * g : kRows;
    if (units * (many ? 1 : a.join_rows) >= ((int64_t)1 << 23))
        return fail(ENGRAM_E_RANGE, "engram cache_attend: %lld row tiles in one call",
                    (long long)units);
    if (!many && units * s.max_pages >= ((int64_t)1 << 30))
        return fail(ENGRAM_E_RANGE,
                    "engram cache_attend: %lld row tiles of up to %d pages exceed 2^30 in one call",
                    (long long)units, s.max_pages);
    if (many)
        return launch_attend_prompt(a, l);
    a.parts = parts_of(c);
    a.least = kLeastShare;
    // pages that 16 rows' windows can meet
    a.window_pages = w > 0 && w < (1 << 30) ? (w + kRows + kPage - 2) / kPage + 1 : 0;
    if (c.head_dim == 64)
        launch_rows<64>(a, units, l);
    else if (c.head_dim == 128)
        launch_rows<128>(a, units, l);
    else
        launch_rows<256>(a, units, l);
    return launch_status("engram cache_attend kernel");
}

}  // namespace engram
