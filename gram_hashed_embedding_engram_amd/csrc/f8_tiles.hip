// Products of many 8-bit rows with 8-bit weights that carry an f32 scale per
// 128 x 128 block: a plain projection, the experts' gated up projection, and
// their down projection, as tiles of one matrix kernel.
//
// A workgroup's eight wavefronts take a tile of rows by a tile of weight rows, K in
// blocks of 128.  One matrix instruction makes a 16 x 16 piece's sum over a block
// from zero, and four multiply-adds join it to the piece's f32 sum under the block's
// scale: half as many vector cycles as matrix cycles, beside which they run.  The
// weights are the instruction's rows, so that a lane's sums are neighbouring outputs
// of one token, and an expert's gate and up rows share a wavefront, so that
// silu(gate) * up, the 32 values' largest and the codes need no other lane's sums.
//
// Data goes from memory to LDS without registers (buffer loads of 1 KiB that fill
// eight rows of 128 bytes, pieces of 16 bytes swapped so that reads meet all banks),
// a token's row by its slot in the plan.  Loads are counted, never waited for as a
// whole: with 256 x 256 tiles a block and a half ahead; with smaller ones one or two
// blocks ahead, which leaves LDS for a second workgroup on the CU (1000 tokens of
// 6144 x 20480 in tiles of 128 x 128: 176 us with four stages, 151 with two; 500 of
// 4096 x 4096 in tiles of 64 x 64: 25 us with five or more, 18 with three), and what
// they read from LDS is less for four wavefronts than for eight (15 us).  Rows'
// scales are loaded eight blocks at a time: a dword a row and block asks L2 for as many
// lines as the codes do (507 -> 476 us below).
//
// Consecutive workgroups go to the XCDs in turn, so each XCD gets a contiguous run
// of tiles: neighbours share weights and rows in its L2.
//
// 4096 tokens of 6144 x 20480 (1.03 TFLOP): 472 to 515 us, 2.18 to 2.0 PFLOP/s, where
// the same without its loads takes 395 (without its barriers 375): matrix and vector
// instructions at the clock that the power limit leaves; the library's product
// without block scales takes 402.  A round of 256 tiles of 256 x 256 costs 1.8 us a
// block and 8.6 once (the first loads, the stores of all CUs at once).  500 tokens of
// 2048 x 5200: 12 to 12.7 us, bound by the trips of its 16 blocks; 37 of 4096 x 14336:
// 12.5 to 13 us.  4096 tokens of eight of 64 experts: up (4096 -> 2 x 2048) 714 to 777
// us, 1.54 to 1.42 PFLOP/s, unevenly filled tiles, their borders and silu; down 445 to
// 474 us, 58 to 61 of them the sum's.  Rows with f32 scales take the same.
//
// Tried and set aside: a workgroup a CU that loads on into its next tile under the
// stores (a tile's fixed cost 8.6 -> 5.9 us, a block 1.82 -> 1.90, and static shares
// of uneven tiles: up 724 -> 766); whole tiles before the experts' last ones, an XCD
// its share of each (740 -> 766: weights are read twice); two workgroups a CU for the
// experts' tiles, of 128 x 128 (up 721 -> 769); lines touched ahead for L2 (507 ->
// 655); explicit turns of matrix, vector and LDS instructions (476 -> 500); raised
// wavefront priority around the matrix instructions (489 -> 513).
#include <type_traits>

#include "f8.h"

namespace engram {
namespace {

constexpr int XCDS = 8;
// Rows of an expert, on average, from which tiles of 256 and of 128 rows are taken.
// In us, tiles of 256, 128 and 64 rows, 64 experts.  Up, 4096 x 2048: 32 rows 223, 206,
// 200; 64 rows 244, 223, 230; 128 rows 329, 282, 323; 192 rows 390, 367, 411; 256 rows
// 445, 445, 518; 375 rows 570, 592, 713; 512 rows 719, 760, 925.  Down, 2048 x 4096: 64
// rows 147, 140, 146; 128 rows 190, 175, 195; 192 rows 236, 227, 254; 256 rows 266, 271,
// 318.  Eight experts of 250 rows: up 71, 83, 87, down 45, 52, 54, for which the border
// lies at 192 and not at 256.  Products of few tiles lose by it: eight experts of 250
// rows take 41, 25 and 32 us for 2048 x 1024, 27, 17 and 12 for 1024 x 512.
constexpr int64_t kRows8 = 192, kRows4 = 64;
// What a tile on every CU costs, and what each of several does, in 0.1 us at K = 4096,
// of tiles of 256 x 256, 128 x 256, 128 x 128, 64 x 128 and 64 x 64 (two workgroups a CU
// from 128 x 128 down): the size with the least is taken.  4096 x 10240, 1000 tokens:
// 62, 69, 57, 62, 69 us; 4096 x 4096, 2000 tokens: 59, 41, 40, 49, 56, 500 tokens: 57,
// 34, 24, 18, 16; 4096 x 6144, 100 tokens: 54, 33, 23, 17, 13; 4096 x 14336, 200 tokens:
// 56, 35, 25, 24, 30; 6144 x 20480, 1000 tokens: 183, 173, 150, 196, 238.  The costs are
// compared with each other, so the same serve every K: of 66 products of 40 to 4096
// tokens, 4096 to 20480 outputs and K = 128 to 6144, 52 take the best size or one
// within 5% of it, the others within 14%, but one (1000 tokens of 512 x 20480: 26 us
// and 22).
constexpr int64_t kAlone[5] = {610, 380, 245, 165, 127}, kEach[5] = {610, 380, 200, 120, 72};
// The same for few rows of large weights, where rows' reads from L2 slow the stream of
// weights.  In us, tiles of 128 x 128, 64 x 128 and 64 x 64, for three matrices in turn
// (which the last-level cache of 256 MB does not hold) and for one again and again: 64
// tokens, 59 MB 23, 17, 13 both ways; 101 MB 31, 25, 27 and 24, 18, 18; 126 MB 42, 35, 40
// and 33, 24, 25; 168 MB 56, 46, 49 and 42, 31, 30; 128 tokens, 88 MB 38, 28, 31 and 33,
// 24, 23; 101 MB 32, 35, 34 and 26, 24, 24; 126 MB 45, 54, 51 and 34, 35, 35; 168 MB 57,
// 64, 63 and 44, 42, 42.
constexpr int64_t kEachStreamed[5] = {610, 380, 200, 130, 100};
constexpr int64_t kStreamedRows = 128, kStreamedBytes = (int64_t)96 << 20;

typedef __attribute__((address_space(3))) void *lptr_t;

// chunk c of an LDS row of 128 bytes sits at c ^ swizzle(r): any 8 or 16
// neighbouring rows read at one chunk meet all banks
__device__ __forceinline__ int swizzle(int r) { return (r >> 1) & 7; }

// a pointer that all lanes share, in scalar registers
__device__ __forceinline__ const uint8_t *uniform(const uint8_t *p)
{
    const uint64_t v = (uint64_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return (const uint8_t *)((uint64_t)hi << 32 | lo);
}

// scales of the rows for this many blocks of K are loaded at once: a dword a row
// and block, loaded block by block, would ask for as many lines as the codes
constexpr int SB = 8;
// dwords from eight rows' scales to the next eight's: the halves of sixteen rows are
// read from different banks (500 tokens of 2048 x 5200 14.3 -> 13.5 us)
constexpr int SG = 8 * SB + 4;

// the same for weight rows, which are read 4 * RUN * (l / 4) + l % 4
template <int RUN>
__device__ __forceinline__ int w_swizzle(int r)
{
    return (r >> 1 & 1) | (r >> (RUN == 4 ? 4 : 3) & 3) << 1;
}

template <int BM, int BN>
struct Stage {
    u32x4 tok[BM * 8];
    u32x4 w[BN * 8];
};

// (one object: of several, the compiler would wait for all loads in flight to
// one before each read of another)
template <int BM, int BN, int S>
struct Shared {
    Stage<BM, BN> stage[S];
    uint32_t xs[2][BM / 8 * SG];
};

// A tile of BM rows and BN weight rows (kUp: half of them the gate's, half the up
// matrix's), S stages of K.  Wavefronts: two halves of the rows by OQ parts of the
// outputs, TB by WB blocks of 16 each.
template <F8Mode MODE, bool XF32, int BM, int BN, int S, int OQ>
__global__ __launch_bounds__(128 * OQ, 2) void tiles_kernel(F8Args a)
{
    constexpr int NW = 2 * OQ, TB = BM / 32, WB = BN / (16 * OQ);
    // rows that a wavefront loads, eight at a time
    constexpr int RT = BM / NW, RW = BN / NW, LT = RT / 8, LW = RW / 8;
    // blocks whose outputs a lane has side by side: row m of block i is weight row
    // 4 * RUN * (m / 4) + 4 * i + m % 4 of the wavefront's, so that a lane's sums,
    // rows 4q .. 4q + 3 of every block, are 4 * RUN neighbours
    constexpr int RUN = MODE == kUp ? 2 : WB;
    static_assert(RUN == 2 || RUN == 4, "outputs leave 16 bytes at a time");
    typedef Stage<BM, BN> Stage;
    __shared__ Shared<BM, BN, S> sh;
    Stage *const stage = sh.stage;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int th = wave / OQ, oq = wave % OQ;        // half of the tokens, part of the outputs
    const int r16 = lane & 15, q = lane >> 4;
    const int KB = a.K / 128;
    constexpr int NT = MODE == kUp ? BN / 2 : BN;    // outputs a tile
    const int tiles_n = (a.N + NT - 1) / NT;

    // ---- this workgroup's tile: each XCD takes a contiguous run of them
    int expert = 0, tm, tn;
    Span span{0, a.T};
    const auto mine = [&](int total) {
        const int b = blockIdx.x, xcd = b % XCDS, per = total / XCDS, rem = total % XCDS;
        return xcd * per + min(xcd, rem) + b / XCDS;
    };
    if (MODE == kDense) {
        constexpr int GROUP_M = 8;
        const int tiles_m = (a.T + BM - 1) / BM, L = mine(tiles_m * tiles_n);
        const int in_group = GROUP_M * tiles_n, first = L / in_group * GROUP_M;
        const int size = min(tiles_m - first, GROUP_M);
        tm = first + L % in_group % size;
        tn = L % in_group / size;
    } else {
        if (blockIdx.x == 0)
            raise_bad_plan(a.p);
        const auto pieces = [&](int n) { return (n + BM - 1) / BM * tiles_n; };
        const int total = all_pieces(a.p, pieces);
        int piece;
        if ((int)blockIdx.x >= total || !find_expert(mine(total), a.p, pieces, expert, piece, span))
            return;
        const int tiles_m = (span.n + BM - 1) / BM;
        tn = piece / tiles_m;
        tm = piece - tn * tiles_m;
    }
    tm = __builtin_amdgcn_readfirstlane(tm);
    tn = __builtin_amdgcn_readfirstlane(tn);
    const int n0 = tn * NT, m0 = tm * BM, rows = min(BM, span.n - m0);
    const int64_t p0 = span.from + m0;               // first row of the plan (or token)

    // ---- loader.  A load of 1 KiB fills eight LDS rows; lane l brings to slot
    // l % 8 of row l / 8 the chunk that belongs there.
    constexpr int H = MODE == kUp ? 2 : 1;
    const int half = MODE == kUp ? wave & 1 : 0;
    const int64_t mat = (int64_t)expert * H + half;
    // (kUp: LDS rows 64u .. 64u+31 are gate rows 32u .., 64u+32 .. their up rows)
    static_assert(MODE != kUp || (WB == 4 && RW == 32), "32 values of h share a scale");
    const int w_first = n0 + RW * (MODE == kUp ? wave >> 1 : wave);
    // (a descriptor bounds a lane's own offset, not the scalar one, which stays
    // within a row: rows past N read as zeros)
    const uint8_t *const w_from = uniform(a.w + (mat * a.N + w_first) * a.K);
    const int w_bytes0 = __builtin_amdgcn_readfirstlane(max(0, min(16, a.N - w_first)) * a.K);
    const int w_bytes1 = __builtin_amdgcn_readfirstlane(max(0, min(16, a.N - w_first - 16)) * a.K);
    const __amdgpu_buffer_rsrc_t rw0 = __builtin_amdgcn_make_buffer_rsrc(
        (void *)w_from, 0, w_bytes0, 0x00020000);
    const __amdgpu_buffer_rsrc_t rw1 = __builtin_amdgcn_make_buffer_rsrc(
        (void *)uniform(w_from + 16 * (int64_t)a.K), 0, w_bytes1, 0x00020000);
    const int64_t x_first = MODE == kUp ? 0 : p0;
    const uint32_t x_rows = MODE == kUp ? a.T : rows;
    const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(a.x + x_first * a.K), 0, (int)(x_rows * (uint32_t)a.K), 0x00020000);
    const int xs_pitch = XF32 ? 4 * KB : a.K / 32;   // the same: a dword a row and block
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        (void *)((const uint8_t *)a.xs + x_first * xs_pitch), 0, (int)(x_rows * (uint32_t)xs_pitch),
        0x00020000);
    const int lr = lane >> 3, ls = lane & 7;
    // the row of x behind tile row r (past the tile's end: its last one's scales, and
    // zeros from past the descriptor, which ask L2 for nothing: 721 -> 715 us below)
    const auto x_row = [&](int r) {
        r = min(r, rows - 1);
        if (MODE != kUp)
            return (uint32_t)r;
        const int slot = a.p.order[p0 + r];
        return (uint32_t)slot < (uint32_t)a.p.slots ? (uint32_t)slot / (uint32_t)a.p.k : 0u;
    };
    uint32_t w_at[4], x_at[4];           // (LW and LT are used)
#pragma unroll
    for (int j = 0; j < LW; j++)
        w_at[j] = (uint32_t)(8 * (j & 1) + lr) * a.K +
                  16 * (ls ^ w_swizzle<RUN>(RW * wave + 8 * j + lr));
    // this wavefront's rows of the first half of the tokens, then of the second
    constexpr int LH = LT > 1 ? LT / 2 : 1;
    const auto t_row = [&](int j) { return j / LH * (BM / 2) + wave * (8 * LH) + 8 * (j % LH); };
#pragma unroll
    for (int j = 0; j < LT; j++) {
        const int r = t_row(j) + lr;
        x_at[j] = r < rows ? x_row(r) * (uint32_t)a.K + 16 * (ls ^ swizzle(r)) : 0xFFFFFF00u;
    }
    uint32_t s_at[4];                    // (LT are used) rows 8j .. of this wavefront's
#pragma unroll
    for (int j = 0; j < LT; j++)
        s_at[j] = x_row(RT * wave + 8 * j + lr) * (uint32_t)xs_pitch + 4 * ls;
    const auto issue_w = [&](int kt, Stage &s) {
        const int k = min(kt, KB - 1);
#pragma unroll
        for (int j = 0; j < LW; j++)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(j < 2 ? rw0 : rw1,
                                                     (lptr_t)&s.w[(RW * wave + 8 * j) * 8], 16,
                                                     w_at[j], 128 * k, 0, 0);
    };
    const auto issue_s = [&](int part) {
#pragma unroll
        for (int j = 0; j < LT; j++)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rs, (lptr_t)&sh.xs[part & 1][(wave * LT + j) * SG], 4,
                s_at[j] + 4 * SB * part, 0, 0, 0);
    };
    const auto issue_x = [&](int kt, Stage &s) {
        const int k = min(kt, KB - 1);
#pragma unroll
        for (int j = 0; j < LT; j++)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lptr_t)&s.tok[t_row(j) * 8], 16, x_at[j], 128 * k, 0, 0);
    };

    // ---- block scales: kept a block a lane, 64 at a time
    const float *ws[H];
#pragma unroll
    for (int h = 0; h < H; h++)
        ws[h] = a.ws + (((int64_t)expert * H + h) * ((a.N + 127) / 128) +
                        min(MODE == kUp ? n0 : n0 + 16 * WB * oq, a.N - 1) / 128) * KB;
    float wsv[H];

    f32x4 acc[WB][TB];
#pragma unroll
    for (int i = 0; i < WB; i++)
#pragma unroll
        for (int j = 0; j < TB; j++)
            acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // a fragment's two pieces of row r16: at these offsets from its first row
    const int at0 = 128 * r16 + 16 * (q ^ swizzle(r16)), at1 = at0 ^ 64;
    const int w_row = 4 * RUN * (r16 >> 2) + (r16 & 3);
    const int w_at0 = 128 * w_row + 16 * (q ^ w_swizzle<RUN>(w_row));
    const auto fragment = [&](const char *p0_, const char *p1_, int r) {
        const u32x4 x = *(const u32x4 *)(p0_ + 128 * r), y = *(const u32x4 *)(p1_ + 128 * r);
        return i32x8{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, (int)y.w};
    };
    i32x8 wf[WB];
    BlockScale f[H];
    const auto read_w = [&](const Stage &s) {
        const char *w0 = (const char *)s.w + oq * 16 * WB * 128 + w_at0, *w1 = w0 - w_at0 + (w_at0 ^ 64);
#pragma unroll
        for (int i = 0; i < WB; i++)
            wf[i] = fragment(w0, w1, i / RUN * 32 + i % RUN * 4);
    };
    const int xs_at = (2 * th + (r16 >> 3)) * SG + (r16 & 7) * SB;
    // blocks J0 .. J0 + NJ - 1 of the wavefront's tokens
    const auto some = [&](int kt, const Stage &s, auto j0, auto nj) {
        const char *t0 = (const char *)s.tok + th * 16 * 128 + at0, *t1 = t0 - at0 + at1;
        const char *xs0 = (const char *)&sh.xs[kt / SB & 1][xs_at + kt % SB] + (XF32 ? 0 : q);
        constexpr int J0 = decltype(j0)::value, NJ = decltype(nj)::value;
#pragma unroll
        for (int j = J0; j < J0 + NJ; j++) {
            const i32x8 xf = fragment(t0, t1, 32 * j);
            const uint32_t xs = XF32 ? *(const uint32_t *)(xs0 + 16 * SG * j)
                                     : *(const uint8_t *)(xs0 + 16 * SG * j);
            float g[H];
#pragma unroll
            for (int h = 0; h < H; h++)
                g[h] = XF32 ? f[h].m * __uint_as_float(xs) : f[h].m;
#pragma unroll
            for (int i = 0; i < WB; i++) {
                const f32x4 v = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    wf[i], xf, f32x4{0.0f, 0.0f, 0.0f, 0.0f}, kFp8, kFp8, 0,
                    f[MODE == kUp ? i >> 1 : 0].e, 0, XF32 ? kOne : (int)xs);
#pragma unroll
                for (int e = 0; e < 4; e++)
                    acc[i][j][e] = __builtin_fmaf(v[e], g[MODE == kUp ? i >> 1 : 0], acc[i][j][e]);
            }
        }
    };
    // the rows from block J0 to J0 + NJ; of an expert's last rows only what there
    // is, to half of them
    const auto part = [&](int kt, const Stage &s, auto j0, auto nj) {
        constexpr int J0 = decltype(j0)::value, NJ = decltype(nj)::value;
        if (MODE == kDense || rows > 32 * (J0 + NJ / 2))
            some(kt, s, j0, nj);
        else if (rows > 32 * J0)
            some(kt, s, j0, std::integral_constant<int, NJ / 2>{});
    };
    // this wavefront's loads but the last n, then everybody's
    const auto meet = [&](auto n) {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(decltype(n)::value) : "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    const auto block_scales = [&](int kt) {
        if ((kt & 63) == 0)
#pragma unroll
            for (int h = 0; h < H; h++) {
                wsv[h] = ws[h][min(kt + lane, KB - 1)];
                asm volatile("" : "+v"(wsv[h]));    // waited for here, not at each use
            }
#pragma unroll
        for (int h = 0; h < H; h++)
            f[h] = block_scale<XF32>(__int_as_float(
                __builtin_amdgcn_readlane(__float_as_int(wsv[h]), kt & 63)));
    };
    typedef std::integral_constant<int, 0> zero;
    issue_s(0);
    if constexpr (S == 2) {
        // Two stages, and a barrier in the middle of a tile.  The rows of tile kt+1
        // are loaded from the start of tile kt on, its weights from the middle of
        // tile kt-1, whose own went to registers before: the first half of the rows
        // has a whole tile's time to arrive, the second and the weights a half more.
        issue_w(0, stage[0]);
        issue_x(0, stage[0]);
        issue_w(1, stage[1]);
        meet(std::integral_constant<int, LT + LW>{});
        read_w(stage[0]);
        for (int kt = 0; kt < KB; kt++) {
            Stage &s = stage[kt & 1], &o = stage[(kt + 1) & 1];
            block_scales(kt);
            meet(std::integral_constant<int, LT / 2 + LW>{});
            if (kt % SB == 0)
                issue_s(kt / SB + 1);
            issue_x(kt + 1, o);
            part(kt, s, zero{}, std::integral_constant<int, TB / 2>{});
            meet(std::integral_constant<int, LT>{});
            issue_w(kt + 2, s);
            part(kt, s, std::integral_constant<int, TB / 2>{}, std::integral_constant<int, TB / 2>{});
            read_w(o);
        }
    } else {
        // S stages, one barrier a tile, loads S - 1 tiles ahead
#pragma unroll
        for (int t = 0; t < S - 1; t++) {
            issue_w(t, stage[t]);
            issue_x(t, stage[t]);
        }
        int at = 0;
        for (int kt = 0; kt < KB; kt++) {
            block_scales(kt);
            meet(std::integral_constant<int, (S - 2) * (LW + LT)>{});
            // (before the loads where four wavefronts leave nobody else to go on: 37
            // tokens of 4096 x 14336 13.0 -> 12.5 us; eight gain nothing, 293 -> 295)
            if (NW == 4)
                read_w(stage[at]);
            if (kt % SB == 0)
                issue_s(kt / SB + 1);
            Stage &o = stage[at == 0 ? S - 1 : at - 1];
            issue_w(kt + S - 1, o);
            issue_x(kt + S - 1, o);
            if (NW != 4)
                read_w(stage[at]);
            part(kt, stage[at], zero{}, std::integral_constant<int, TB>{});
            at = at + 1 == S ? 0 : at + 1;
        }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

    // ---- out: accumulator e of block (i, j) is output 4 * RUN * q + 4i + e of the
    // wavefront's, token 32j + 16th + l % 16
#pragma unroll
    for (int j = 0; j < TB; j++) {
        const int r = 32 * j + 16 * th + r16;
        const bool in = r < rows;
        const int64_t p = p0 + r;
        int slot = 0;
        if (MODE != kDense && in)
            slot = a.p.order[p];
        const bool fine = in && (uint32_t)slot < (uint32_t)(MODE == kDense ? 1 : a.p.slots);
        if (MODE != kDense && in && !fine)
            raise(a.p.err, ENGRAM_DEVERR_ROUTE);
        if (MODE == kUp) {
            float v[2][4], amax = 0.0f;
#pragma unroll
            for (int i = 0; i < 2; i++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    v[i][e] = gated(acc[i][j][e], acc[2 + i][j][e]);
                    amax = fmaxf(amax, finite_abs(v[i][e]));
                }
            const int k = e4m3_scale_exp(max_x16(amax));
            const float inv = exp2_int(-k);
            if (!fine)
                continue;
            const int n = n0 + 32 * oq;
            *(u32x2 *)((uint8_t *)a.y + p * a.N + n + 8 * q) =
                u32x2{e4m3x4(v[0][0] * inv, v[0][1] * inv, v[0][2] * inv, v[0][3] * inv),
                      e4m3x4(v[1][0] * inv, v[1][1] * inv, v[1][2] * inv, v[1][3] * inv)};
            if (q == 0)
                a.hs[p * (a.N / 32) + n / 32] = (uint8_t)(k + 127);
            continue;
        }
        // products leave as f16 under a power of two per 64 of a row: half the bytes of
        // f32, twice over memory (4096 tokens of eight of 64 experts 455 us, with f32 583;
        // 1024 tokens 174 and 201, 512 140 and 153).  Each is off by 2^-11 of itself, or
        // 2^-39 of the 64's largest: an eighth of what the sum's own rounding to bf16 is
        // off by, but where a token's products cancel.  Few rows (f8_rows.hip) stay f32.
        int k16 = 0;
        if (MODE == kDown) {
            float amax = 0.0f;
#pragma unroll
            for (int i = 0; i < WB; i++)
#pragma unroll
                for (int e = 0; e < 4; e++)
                    amax = fmaxf(amax, finite_abs(acc[i][j][e]));
            k16 = f16_scale_exp(max_x16(amax));
        }
        const int n = n0 + 16 * WB * oq + 4 * RUN * q;
        if (!fine || n >= a.N)
            continue;
        const float inv = exp2_int(-k16);
        uint32_t o[2 * WB];
#pragma unroll
        for (int i = 0; i < WB; i++) {
            const f32x4 v = acc[i][j];
            o[2 * i] = MODE == kDense ? cvt_bf16x2(v[0], v[1]) : cvt_f16x2(v[0] * inv, v[1] * inv);
            o[2 * i + 1] = MODE == kDense ? cvt_bf16x2(v[2], v[3]) : cvt_f16x2(v[2] * inv, v[3] * inv);
        }
        uint16_t *y = (uint16_t *)a.y + (MODE == kDense ? p : (int64_t)slot) * a.N + n;
#pragma unroll
        for (int i = 0; i < WB; i += 2)
            *(u32x4 *)(y + 4 * i) = u32x4{o[2 * i], o[2 * i + 1], o[2 * i + 2], o[2 * i + 3]};
        if (MODE == kDown && q == 0)
            a.hs[(int64_t)slot * ((a.N + 63) / 64) + n / 64] = (uint8_t)k16;
    }
}

template <F8Mode MODE, int BM, int BN, int S, int OQ>
int32_t launch_size(const F8Args &a, bool f32, bool last, const Launch &l)
{
    constexpr int NT = MODE == kUp ? BN / 2 : BN;
    // (of an experts' call, the tiles that any plan of it can ask for)
    const int64_t tiles_m = MODE == kDense ? (a.T + BM - 1) / BM : f8_most_tiles(a.p, BM);
    const int64_t tiles = tiles_m * ((a.N + NT - 1) / NT);
    if (tiles >= (int64_t)1 << 23)                   // a grid counts its threads in 32 bits
        return fail(ENGRAM_E_RANGE, "engram f8 tiles: %lld workgroups exceed 2^23-1", (long long)tiles);
    const dim3 grid((unsigned)tiles);
    if (f32)
        dispatch(tiles_kernel<MODE, true, BM, BN, S, OQ>, grid, dim3(128 * OQ), l, true, last, a);
    else
        dispatch(tiles_kernel<MODE, false, BM, BN, S, OQ>, grid, dim3(128 * OQ), l, true, last, a);
    return launch_status("engram f8 tiles kernel");
}

}  // namespace

template <F8Mode MODE>
int32_t launch_f8_tiles(const F8Args &a, bool f32, bool last, const Launch &l)
{
    if constexpr (MODE == kDense) {
        const int64_t cus = device_cus();
        const int64_t *const each =
            a.T <= kStreamedRows && (int64_t)a.N * a.K >= kStreamedBytes ? kEachStreamed : kEach;
        const int64_t size[5][2] = {{256, 256}, {128, 256}, {128, 128}, {64, 128}, {64, 64}};
        int pick = 0;
        int64_t least = INT64_MAX;
        for (int i = 0; i < 5; i++) {
            const int64_t tiles = ((a.T + size[i][0] - 1) / size[i][0]) * ((a.N + size[i][1] - 1) / size[i][1]);
            const int64_t rounds = (tiles + cus - 1) / cus;
            const int64_t cost = rounds == 1 ? kAlone[i] : rounds * each[i];
            if (cost < least) {
                least = cost;
                pick = i;
            }
        }
        return pick == 0   ? launch_size<kDense, 256, 256, 2, 4>(a, f32, last, l)
               : pick == 1 ? launch_size<kDense, 128, 256, 3, 4>(a, f32, last, l)
               : pick == 2 ? launch_size<kDense, 128, 128, 2, 4>(a, f32, last, l)
               : pick == 3 ? launch_size<kDense, 64, 128, 3, 2>(a, f32, last, l)
                           : launch_size<kDense, 64, 64, 3, 2>(a, f32, last, l);
    } else {
        const int64_t rows = a.p.slots / a.p.E;
        return rows >= kRows8   ? launch_size<MODE, 256, 256, 2, 4>(a, f32, last, l)
               : rows >= kRows4 ? launch_size<MODE, 128, 256, 3, 4>(a, f32, last, l)
                                : launch_size<MODE, 64, 256, 3, 4>(a, f32, last, l);
    }
}

template int32_t launch_f8_tiles<kDense>(const F8Args &, bool, bool, const Launch &);
template int32_t launch_f8_tiles<kUp>(const F8Args &, bool, bool, const Launch &);
template int32_t launch_f8_tiles<kDown>(const F8Args &, bool, bool, const Launch &);

}  // namespace engram
