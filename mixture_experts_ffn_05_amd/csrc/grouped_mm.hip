// Grouped matrix products by expert, ragged segments, and their gradients.
//
// Expert e owns the sorted rows [offsets[e], offsets[e+1]); row s reads input
// row r(s) = pairs[s] / k (or s).  The three products
//   forward   c[s][n]    = sum_k a[r(s)][k] b[e][n][k] + bias[e][n]
//   dgrad     da[s][k]   = sum_n dc[s][n] b[e][n][k]
//   wgrad     db[e][n][k] (+)= sum_{s in e} dc[s][n] a[r(s)][k]
// are one tiled kernel, D[r][c] = sum_j P[r][j] Q[c][j] per tile, on
// v_mfma_f32_32x32x16_{bf16,f16} with fp32 accumulation:
//   forward: P = weight rows n,         Q = token rows s,      j = k
//   dgrad:   P = weight columns k,      Q = rows of dc,        j = n
//   wgrad:   P = columns k of a,        Q = columns n of dc,   j = the segment's rows
// P's index is the output's contiguous one in all three, so a lane's four
// consecutive accumulator rows are one vector store.
//
// Operands whose memory is contiguous along j are staged as [rows][32 j] LDS
// tiles.  Operands contiguous along r or c (the weights of dgrad, both
// operands of wgrad) are staged as they lie, [32 j][columns], and
// ds_read_b64_tr_b16 transposes them on the way to the registers: no
// transposed copy of the weights or of the activations is ever written.
// Both kinds give a lane the j values 16 s + 8 (lane / 32) + 0..7 in order, so
// either kind can meet either in one MFMA.
//
// The tile loop is a ring of 4 LDS stages of 32 j filled by direct-to-LDS loads
// two to three stages ahead, one barrier a stage, after the first half of the
// stage's MFMAs.  The loads are spread among the MFMAs (issued together, eight
// waves' MFMAs wait behind the address unit), their addresses are a uniform base
// per stage and fixed 32-bit offsets, and the loop is unrolled by the ring so
// that LDS addresses are constants: it holds no address arithmetic.  P's
// fragments are replaced in place as their MFMAs are issued, Q's are double.
// Only the last stages check bounds; what they find past the contracted length,
// or past the matrix's width in a transposed tile, reads as zeros.
// Rows and widths that are not multiples of 8 elements (or bases not 16-byte
// aligned) cannot use the direct loads (VEC = false): they go through
// registers, with unaligned 16-byte loads and an element loop only in a row's
// last chunk.
//
// Bound by the matrix cores at the clock that their load allows: 1116 us for
// 32768 rows, 32 experts of Zipf shares, 2880 -> 5760 bf16 (0.97 PFLOP/s; the
// library's dense product of those sizes 1.23), 1299 us for both gradients at
// 2880 x 2880 with the bias gradient (0.84 PFLOP/s; dense 1.11 and 0.73).  What each part gave: loads
// among the MFMAs 1201 -> 1125 us, no address arithmetic 1242 -> 1171.
#include <string.h>

#include <type_traits>
#include <utility>

#include "elem16.h"
#include "moe_ops.h"
#include "tile_sched.h"

namespace moe {

namespace {

constexpr int GP_BK = 32;
constexpr int GP_NBUF = 4;

enum { GP_FWD = 0, GP_DGRAD = 1, GP_WGRAD = 2 };

// Tile shapes: WR x WC waves, each WB x TB blocks of 32 x 32.
template <int WR_, int WC_, int WB_, int TB_>
struct TileCfg {
    static constexpr int WR = WR_, WC = WC_, WB = WB_, TB = TB_;
    static constexpr int NW = WR * WC, THREADS = NW * WAVE;
    static constexpr int BR = WR * WB * 32, BC = WC * TB * 32;
};
using TileLarge = TileCfg<2, 4, 4, 2>;  // 256 x 256, 8 waves
using TileWide = TileCfg<2, 4, 5, 2>;   // 320 x 256, 8 waves
using TileSmall = TileCfg<2, 2, 2, 1>;  // 128 x 64, 4 waves

__device__ uint32_t gp_zeros[4] __attribute__((aligned(16)));  // never written

struct GpArgs {
    int M, N, K, E, a_rows;
    unsigned long long k_magic;  // p / k = (p * k_magic) >> k_shift for 0 <= p < 2^31
    int k_shift;
    long long lda, ldc;
    const int32_t* offsets;
    const int32_t* pairs;
    const void* a;
    const void* b;
    const void* bias;
    const void* dc;
    void* out;
    int splits;
    int accumulate;
};

// Input row of sorted position s; a pair outside [0, a_rows * k) gives -1 (a
// row of zeros).
__device__ __forceinline__ int input_row(const GpArgs& g, int p)
{
    const int r = (int)(((unsigned long long)(unsigned)p * g.k_magic) >> g.k_shift);
    return ((p >= 0) & (r < g.a_rows)) ? r : -1;
}

// The schedule puts each expert's ragged last tile after its full ones: dealt
// out at the very end instead, so that the last round is of short tiles, they lose
// the L2's copies of their expert's rows (prefill product 1188 -> 1258 us).
// M-tile `tile` of the schedule in which expert e owns ceil(len_e / BC) * nt
// consecutive tiles; every wave computes the same.  Also returns the number of
// tiles of all experts.
template <int BC>
__device__ __forceinline__ int gp_total(const GpArgs& g, int nt)
{
    int n = 0;
    for (int base = 0; base < g.E; base += WAVE) {
        const int e = base + lane_id();
        int mt = 0;
        if (e < g.E) {
            const Segment sg = segment_of(g.offsets, e, g.M);
            mt = (sg.end - sg.begin + BC - 1) / BC;
        }
        n += wave_sum(mt);
    }
    return n * nt;
}

template <int BC>
__device__ __forceinline__ int gp_locate(const GpArgs& g, int nt, int tile, int* local, int* mtiles)
{
    const int lane = lane_id();
    int before = 0;
    for (int base = 0; base < g.E; base += WAVE) {
        const int e = base + lane;
        int mt = 0;
        if (e < g.E) {
            const Segment sg = segment_of(g.offsets, e, g.M);
            mt = (sg.end - sg.begin + BC - 1) / BC;
        }
        const int n = mt * nt;
        const int excl = wave_excl_scan(n) + before;
        const uint64_t hm = ballot(n > 0 && tile >= excl && tile < excl + n);
        if (hm) {
            const int src = (int)__builtin_ctzll(hm);
            *local = tile - __shfl(excl, src, WAVE);
            *mtiles = __shfl(mt, src, WAVE);
            return base + src;
        }
        before = __shfl(excl + n, WAVE - 1, WAVE);
    }
    return -1;
}

// The expert whose segment has rank `rank` by descending length (ties: lower
// index first).  E <= 256: lane l holds experts l, l + 64, ...
__device__ __forceinline__ int gp_ranked_expert(const GpArgs& g, int rank)
{
    const int lane = lane_id();
    int len[4], rk[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = lane + WAVE * i;
        len[i] = -1;
        rk[i] = 0;
        if (e < g.E) {
            const Segment sg = segment_of(g.offsets, e, g.M);
            len[i] = sg.end - sg.begin;
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (WAVE * j >= g.E) break;  // uniform
        for (int o = 0; o < min(WAVE, g.E - WAVE * j); ++o) {
            const int lo = __builtin_amdgcn_readlane(len[j], o);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                rk[i] += (lo > len[i] || (lo == len[i] && WAVE * j + o < lane + WAVE * i)) ? 1 : 0;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t hit = ballot(lane + WAVE * i < g.E && rk[i] == rank);
        if (hit) return WAVE * i + (int)__builtin_ctzll(hit);
    }
    return -1;
}

typedef __attribute__((address_space(4))) const int32_t* gp_cptr;  // read through the scalar unit
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((address_space(3))) s16x4* gp_trptr;

// 8 elements from p on; those from element `left` on are 0.
template <typename T>
__device__ __forceinline__ u32x4 load8_masked(const T* p, int left)
{
    if (left >= 8) return load16_any(p);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) w[i >> 1] |= (uint32_t)p[i].v << (16 * (i & 1));
    return u32x4{w[0], w[1], w[2], w[3]};
}

template <typename F, int... I>
__device__ __forceinline__ void for_constants(F f, std::integer_sequence<int, I...>)
{
    (f(std::integral_constant<int, I>{}), ...);
}

// GATHER (wgrad): rows of a through pairs.  The forward gathers by `pairs`
// itself, once per tile.
template <typename T, typename O, int MODE, bool VEC, bool GATHER, typename Cfg>
__global__ __launch_bounds__(Cfg::THREADS, Cfg::THREADS / 256) void gmm_kernel(GpArgs g)
{
    constexpr int BR = Cfg::BR, BC = Cfg::BC, NW = Cfg::NW, WB = Cfg::WB, TB = Cfg::TB;
    constexpr bool P_TR = MODE != GP_FWD, Q_TR = MODE == GP_WGRAD;
    // 1 KB loads per stage and wave; where the waves' shares of P differ, the
    // last of them is the first waves' only.
    constexpr int NLP = BR * 64 / 1024, DLP = (NLP + NW - 1) / NW, DLQ = BC * 64 / 1024 / NW;
    constexpr int FULL = NLP - (DLP - 1) * NW;  // waves with DLP loads
    static_assert(WB >= DLP && WB >= DLQ, "every load has its place among the MFMAs");
    static_assert(BR * 64 % 1024 == 0 && BC * 64 % (1024 * NW) == 0, "a stage is whole loads");
    __shared__ __attribute__((aligned(16))) uint8_t shp[GP_NBUF][BR * 64];
    __shared__ __attribute__((aligned(16))) uint8_t shq[GP_NBUF][BC * 64];

    const int R = MODE == GP_FWD ? g.N : g.K;  // the tile's row index runs over these
    const int nt = (R + BR - 1) / BR;

    // ---- tile of this block (uniform per block)
    int e, local, mtiles, split = 0;
    if constexpr (MODE == GP_WGRAD) {
        // An expert's tiles all contract over its own number of rows, so the
        // experts go out longest first; within an expert every XCD (blocks are
        // dealt round-robin over the 8) takes one contiguous run of the banded
        // tile order and shares its operand strips in its L2.
        mtiles = (g.N + BC - 1) / BC;
        const int tpe = mtiles * nt, tpe8 = (tpe + 7) / 8 * 8;
        const int t = (int)(blockIdx.x % tpe8);
        const int er = (int)(blockIdx.x / tpe8);
        local = (t % 8) * (tpe8 / 8) + t / 8;
        if (local >= tpe) return;
        split = er % g.splits;
        e = gp_ranked_expert(g, er / g.splits);
        if (e < 0) return;
    } else {
        // Blocks are dealt round-robin over the 8 XCDs; each XCD takes one
        // contiguous run of the tile order.
        const int total = gp_total<BC>(g, nt);
        const int per = (total + 7) / 8;
        if ((int)(blockIdx.x / 8) >= per) return;
        const int tile = (int)(blockIdx.x % 8) * per + (int)(blockIdx.x / 8);
        if (tile >= total) return;
        e = gp_locate<BC>(g, nt, tile, &local, &mtiles);
        if (e < 0) return;
    }
    int mt, ntile;
    e = __builtin_amdgcn_readfirstlane(e);
    gm_band(__builtin_amdgcn_readfirstlane(local), __builtin_amdgcn_readfirstlane(mtiles), nt, &mt, &ntile);
    const int r0 = ntile * BR;
    Segment seg = segment_of(g.offsets, e, g.M);
    seg.begin = __builtin_amdgcn_readfirstlane(seg.begin);
    seg.end = __builtin_amdgcn_readfirstlane(seg.end);
    int J;       // contracted length
    int c0, c1;  // the tile's first column-role index and the end of its range
    int j0 = 0;  // WGRAD: first row of the split, relative to the segment
    if constexpr (MODE == GP_WGRAD) {
        const int len = seg.end - seg.begin;
        const int per = ((len + g.splits - 1) / g.splits + GP_BK - 1) / GP_BK * GP_BK;
        j0 = min(split * per, len);
        J = min(per, len - j0);
        c0 = mt * BC;
        c1 = g.N;
    } else {
        J = MODE == GP_FWD ? g.K : g.N;
        c0 = seg.begin + mt * BC;
        c1 = seg.end;
    }
    const int nstages = (J + GP_BK - 1) / GP_BK;

    const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid / WAVE);
    // Waves w and w + 4 share a SIMD: they take column parts half a tile apart,
    // so that a tile with few valid columns keeps every SIMD busy.  A wave
    // without valid rows or columns still stages its share and meets every barrier.
    const int wr = wave / Cfg::WC, wc = (wave + (Cfg::WC / 2) * wr) % Cfg::WC;
    const bool live = c0 + 32 * TB * wc < c1 && r0 + 32 * WB * wr < R;

    // ---- sources of this wave's 1 KB loads: load i covers bytes 1024 (wave +
    // NW i) .. of the tile, lane l its 16-byte piece l.  Contiguous along j: tile
    // rows of 64 bytes; piece p of row r holds logical piece p ^ (r / 4 % 4).
    // Transposed: tile rows are j; a row of RB bytes holds its 64-byte segments
    // XORed with tr_xor(row), so that the four rows one transposing read
    // touches fall on different banks.
    const T* zeros = reinterpret_cast<const T*>(gp_zeros);
    constexpr int PRB = BR * 2, QRB = BC * 2;
    auto tr_xor = [](int row, int RB) { return RB % 256 == 0 ? row & 3 : (row >> 1) & 1; };
    const bool all_p = wave < FULL;

    const T* A = static_cast<const T*>(g.a);
    const T* B = static_cast<const T*>(g.b) + (size_t)e * g.N * g.K;
    const T* DC = static_cast<const T*>(g.dc);
    // Load i of an operand: this lane's tile row, and its first column (contiguous
    // along j: its first j).
    auto p_row = [&](int i) { return !P_TR ? 16 * (wave + NW * i) + (lane >> 2) : (WAVE * (wave + NW * i) + lane) / (PRB / 16); };
    auto q_row = [&](int i) { return !Q_TR ? 16 * (wave + NW * i) + (lane >> 2) : (WAVE * (wave + NW * i) + lane) / (QRB / 16); };
    auto p_first = [&](int i) {
        const int row = p_row(i), p = P_TR ? (WAVE * (wave + NW * i) + lane) % (PRB / 16) : lane & 3;
        return 8 * (P_TR ? (((p >> 2) ^ tr_xor(row, PRB)) << 2) | (p & 3) : p ^ ((row >> 2) & 3));
    };
    auto q_first = [&](int i) {
        const int row = q_row(i), p = Q_TR ? (WAVE * (wave + NW * i) + lane) % (QRB / 16) : lane & 3;
        return 8 * (Q_TR ? (((p >> 2) ^ tr_xor(row, QRB)) << 2) | (p & 3) : p ^ ((row >> 2) & 3));
    };
    // WGRAD with gathered rows: the pair ids of the next stage's rows, read
    // one stage early through the scalar unit (vector loads would have to be
    // waited for in order with the tiles in flight).
    constexpr int PROWS = (1024 + PRB - 1) / PRB + (1024 % PRB != 0 ? 1 : 0);  // rows that one load may touch
    [[maybe_unused]] int prow[DLP][PROWS];
    auto load_rows = [&](int st) {
        if constexpr (GATHER) {
            gp_cptr ids = (gp_cptr)(uintptr_t)g.pairs;
#pragma unroll
            for (int i = 0; i < DLP; ++i) {
                const int first = st * GP_BK + 1024 * (wave + NW * i) / PRB;  // uniform
#pragma unroll
                for (int q = 0; q < PROWS; ++q) prow[i][q] = ids[__builtin_amdgcn_readfirstlane(seg.begin + j0 + min(first + q, J - 1))];
            }
        }
    };

    // Source of load i at stage st with every bound checked: the zeros past the
    // operand's end (or, for the register path, null).  Branch-free: a branch
    // here makes the compiler wait for every load in flight at the join.
    auto pick = [&](bool ok, const T* src) {
        return reinterpret_cast<const T*>(ok ? reinterpret_cast<uintptr_t>(src)
                                             : VEC ? reinterpret_cast<uintptr_t>(zeros) : (uintptr_t)0);
    };
    auto p_at = [&](int i, int st) -> const T* {
        const int row = p_row(i), first = p_first(i);
        if constexpr (!P_TR) {
            const int j = st * GP_BK + first;
            return pick((r0 + row < R) & (j < J), B + (long long)(r0 + row) * g.K + j);
        } else {
            const int j = st * GP_BK + row, col = r0 + first;
            const bool ok = (col < R) & (j < J);
            if constexpr (MODE == GP_DGRAD) return pick(ok, B + (long long)j * g.K + col);
            int r = seg.begin + j0 + j;
            if constexpr (GATHER) {
                const int sub = row - 1024 * (wave + NW * i) / PRB;
                // read lane by lane: a plain choice among the array's elements
                // becomes an indexed load, and the array memory
                int p = __builtin_amdgcn_readfirstlane(prow[i][0]);
#pragma unroll
                for (int q = 1; q < PROWS; ++q) p = sub == q ? __builtin_amdgcn_readfirstlane(prow[i][q]) : p;
                r = input_row(g, p);
            }
            return pick(ok & ((unsigned)r < (unsigned)g.a_rows), A + (long long)r * g.lda + col);
        }
    };
    // The input row of column-role index c of the forward product (-1: zeros).
    auto fwd_row = [&](int c) {
        if (!g.pairs) return c;
        return c < c1 ? input_row(g, g.pairs[c]) : -1;
    };
    int qrow[MODE == GP_FWD ? DLQ : 1];  // forward: the rows of this wave's loads
    if constexpr (MODE == GP_FWD) {
#pragma unroll
        for (int i = 0; i < DLQ; ++i) qrow[i] = c0 + q_row(i) < c1 ? fwd_row(c0 + q_row(i)) : -1;
    }
    auto q_at = [&](int i, int st) -> const T* {
        const int row = q_row(i), first = q_first(i);
        if constexpr (MODE == GP_FWD) {
            const int j = st * GP_BK + first, r = qrow[i];
            return pick((r >= 0) & (j < J), A + (long long)r * g.lda + j);
        } else if constexpr (MODE == GP_DGRAD) {
            const int j = st * GP_BK + first;
            return pick((c0 + row < c1) & (j < J), DC + (long long)(c0 + row) * g.ldc + j);
        } else {
            const int j = st * GP_BK + row, col = c0 + first;
            return pick((col < c1) & (j < J), DC + (long long)(seg.begin + j0 + j) * g.ldc + col);
        }
    };

    // ---- VEC: direct-to-LDS loads.  Whole stages (32 valid j) use a uniform
    // base that moves with the stage and fixed 32-bit offsets, so a load costs no
    // vector arithmetic; rows and columns past the matrix's or the segment's end
    // read a valid one instead (their results are not stored).  Gathered rows
    // keep 64-bit addresses.  The last, partial stage checks every bound.
    constexpr bool Q64 = MODE == GP_FWD;  // q rows anywhere in `a`
    [[maybe_unused]] uint32_t poff[DLP], qoff[DLQ];
    [[maybe_unused]] const T* qptr[DLQ];
    const int nwhole = J / GP_BK;
    const T* pbase = nullptr;
    const T* qbase = nullptr;
    long long pstep = GP_BK, qstep = GP_BK;  // elements per stage
    if constexpr (VEC) {
        if constexpr (MODE == GP_FWD) {
            pbase = B + (size_t)r0 * g.K;
        } else if constexpr (MODE == GP_DGRAD) {
            pbase = B + r0;
            pstep = (long long)GP_BK * g.K;
            qbase = DC + (size_t)c0 * g.ldc;
        } else {
            pbase = A + (size_t)(seg.begin + j0) * g.lda + r0;
            pstep = GP_BK * g.lda;
            qbase = DC + (size_t)(seg.begin + j0) * g.ldc + c0;
            qstep = GP_BK * g.ldc;
        }
#pragma unroll
        for (int i = 0; i < DLP; ++i) {
            const int row = p_row(i), first = p_first(i);
            if constexpr (!P_TR)
                poff[i] = 2u * ((uint32_t)min(row, R - 1 - r0) * (uint32_t)g.K + first);
            else
                poff[i] = 2u * ((uint32_t)row * (uint32_t)(MODE == GP_DGRAD ? g.K : g.lda) + (r0 + first < R ? first : 0));
        }
#pragma unroll
        for (int i = 0; i < DLQ; ++i) {
            const int row = q_row(i), first = q_first(i);
            if constexpr (Q64)
                qptr[i] = A + (size_t)max(qrow[i], 0) * g.lda + first;
            else if constexpr (!Q_TR)
                qoff[i] = 2u * ((uint32_t)min(row, c1 - 1 - c0) * (uint32_t)g.ldc + first);
            else
                qoff[i] = 2u * ((uint32_t)row * (uint32_t)g.ldc + (c0 + first < c1 ? first : 0));
        }
    }
    const uint32_t lds_p = lds_address(shp[0]) + 1024 * wave, lds_q = lds_address(shq[0]) + 1024 * wave;
    // P's load i, Q's load i of the whole stage st into buffer BUF.
    auto issue_p = [&](auto buf_c, auto i_c, int st) {
        constexpr int BUF = decltype(buf_c)::value, i = decltype(i_c)::value, at = BUF * BR * 64 + 1024 * NW * i;
        if (FULL < NW && i == DLP - 1 && !all_p) return;  // uniform
        if constexpr (GATHER)
            dma16_at<at>(p_at(i, st), lds_p);
        else
            dma16_at<at>(pbase + st * pstep, poff[i], lds_p);
    };
    auto issue_q = [&](auto buf_c, auto i_c, int st) {
        constexpr int BUF = decltype(buf_c)::value, i = decltype(i_c)::value, at = BUF * BC * 64 + 1024 * NW * i;
        if constexpr (Q64)
            dma16_at<at>(qptr[i] + st * GP_BK, lds_q);
        else
            dma16_at<at>(qbase + st * qstep, qoff[i], lds_q);
    };
    // The loads that go with block row m's MFMAs: P's spread over the second
    // half of a stage, Q's over the first half of the next one.  (All at once
    // after the barrier, eight waves' MFMAs wait behind the address unit.)
    auto among_p = [&](auto buf_c, int st) {
        return [&, buf_c, st](auto m_c) {
            constexpr int m = decltype(m_c)::value;
            for_constants(
                [&](auto i_c) {
                    if constexpr (decltype(i_c)::value * WB / DLP == m) issue_p(buf_c, i_c, st);
                },
                std::make_integer_sequence<int, DLP>{});
            if constexpr (m == WB - 1) load_rows(st + 1);
        };
    };
    auto among_q = [&](auto buf_c, int st) {
        return [&, buf_c, st](auto m_c) {
            constexpr int m = decltype(m_c)::value;
            for_constants(
                [&](auto i_c) {
                    if constexpr (decltype(i_c)::value * WB / DLQ == m) issue_q(buf_c, i_c, st);
                },
                std::make_integer_sequence<int, DLQ>{});
        };
    };
    // Any stage, bounds checked; past the last one zeros.
    auto issue_any = [&](int st) {
        const int buf = st % GP_NBUF;
#pragma unroll
        for (int i = 0; i < DLP; ++i)
            if (FULL == NW || i < DLP - 1 || all_p) dma16_at<0>(p_at(i, st), lds_p + buf * BR * 64 + 1024 * NW * i);
#pragma unroll
        for (int i = 0; i < DLQ; ++i) dma16_at<0>(q_at(i, st), lds_q + buf * BC * 64 + 1024 * NW * i);
        load_rows(st + 1);
    };
    // ---- otherwise: through registers
    [[maybe_unused]] u32x4 rp[2][DLP], rq[2][DLQ];
    auto fetch = [&](int set, int st) {
        const u32x4 z = u32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < DLP; ++i) {
            const T* src = p_at(i, st);
            rp[set][i] = src ? load8_masked(src, P_TR ? R - (r0 + p_first(i)) : J - (st * GP_BK + p_first(i))) : z;
        }
#pragma unroll
        for (int i = 0; i < DLQ; ++i) {
            const T* src = q_at(i, st);
            rq[set][i] = src ? load8_masked(src, Q_TR ? c1 - (c0 + q_first(i)) : J - (st * GP_BK + q_first(i))) : z;
        }
        load_rows(st + 1);
    };
    auto store = [&](int set, int buf) {
#pragma unroll
        for (int i = 0; i < DLP; ++i)
            if (FULL == NW || i < DLP - 1 || all_p)
                *reinterpret_cast<u32x4*>(shp[buf] + 1024 * (wave + NW * i) + 16 * lane) = rp[set][i];
#pragma unroll
        for (int i = 0; i < DLQ; ++i)
            *reinterpret_cast<u32x4*>(shq[buf] + 1024 * (wave + NW * i) + 16 * lane) = rq[set][i];
    };

    f32x16_t acc[WB][TB];
#pragma unroll
    for (int m = 0; m < WB; ++m)
#pragma unroll
        for (int t = 0; t < TB; ++t) acc[m][t] = f32x16_t{};

    // ---- operand fragments of one 16-wide j step
    const int r32 = lane & 31, kg = lane >> 5;
    // Transposing read: lane l addresses row l % 16 / 4 (+ 8 for the upper half
    // wave) and columns 16 (l / 16 % 2) + 4 (l % 4) .. +3 of a 32-column block,
    // and receives four rows of its own column.
    const int tr_row = ((lane & 15) >> 2) + 8 * kg;
    const int tr_in = 32 * ((lane >> 4) & 1) + 8 * (lane & 3);
    auto read_tr = [&](const uint8_t* tile, int RB, int block, int s) {
        const int seg64 = block ^ tr_xor(tr_row, RB);
        const uint8_t* at = tile + (tr_row + 16 * s) * RB + seg64 * 64 + tr_in;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((gp_trptr)at);
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((gp_trptr)(at + 4 * RB));
        const uint2 l2 = __builtin_bit_cast(uint2, lo), h2 = __builtin_bit_cast(uint2, hi);
        return u32x4{l2.x, l2.y, h2.x, h2.y};
    };
    auto read_row = [&](const uint8_t* tile, int row, int s) {
        const int c = (2 * s + kg) ^ ((row >> 2) & 3);
        return *reinterpret_cast<const u32x4*>(tile + row * 64 + c * 16);
    };
    u32x4 p[WB], q[2][TB];
    auto load_p = [&](int buf, int s, int m) {
        if constexpr (P_TR)
            p[m] = read_tr(shp[buf], PRB, WB * wr + m, s);
        else
            p[m] = read_row(shp[buf], 32 * (WB * wr + m) + r32, s);
    };
    auto load_q = [&](int buf, int s) {
#pragma unroll
        for (int t = 0; t < TB; ++t) {
            if constexpr (Q_TR)
                q[s][t] = read_tr(shq[buf], QRB, TB * wc + t, s);
            else
                q[s][t] = read_row(shq[buf], 32 * (TB * wc + t) + r32, s);
        }
    };
    // The MFMAs of step s, with the fragments of the next step (1 - s of buffer
    // `next`) read among them: q into its other set first, p[m] in place once
    // its own MFMAs are issued.
    auto step = [&](auto s_c, int next, auto between) {
        constexpr int S = decltype(s_c)::value;
        load_q(next, 1 - S);
        for_constants(
            [&](auto m_c) {
                constexpr int m = decltype(m_c)::value;
#pragma unroll
                for (int t = 0; t < TB; ++t) acc[m][t] = mfma32_t(p[m], q[S][t], acc[m][t], T{});
                load_p(next, 1 - S, m);
                between(m_c);
                __builtin_amdgcn_sched_barrier(0);
            },
            std::make_integer_sequence<int, WB>{});
    };
    using S0 = std::integral_constant<int, 0>;
    using S1 = std::integral_constant<int, 1>;

    // ---- software pipeline: each stage is two 16-wide steps; the barrier that
    // publishes stage st+1 sits between them.
    if (nstages > 0) {
        // Stages st with st + 6 < nwhole run four at a time, buffers constant,
        // on whole stages only; the others check every bound.
        const bool main_loop = VEC && 6 < nwhole;
        load_rows(0);
        if constexpr (VEC) {
            issue_any(0);
            issue_any(1);
            if (main_loop)
                for_constants(among_p(std::integral_constant<int, 2>{}, 2), std::make_integer_sequence<int, WB>{});
            else
                issue_any(2);
            dma_wait<DLP + DLQ>();  // stage 0
        } else {
            fetch(0, 0);
            fetch(1, 1);
            store(0, 0);
            store(1, 1);
            fetch(0, 2);
            fetch(1, 3);
        }
        lds_barrier();
        if (live) {
            load_q(0, 0);
#pragma unroll
            for (int m = 0; m < WB; ++m) load_p(0, 0, m);
        }
        auto none = [](auto) {};
        // Stage st in buffer buf.  `load` runs after the barrier, first(m) and
        // second(m) with block row m's MFMAs before and after it.
        auto stage = [&](int buf, int next, auto load, auto first, auto second) {
            __builtin_amdgcn_sched_barrier(0);
            if (live)
                step(S0{}, buf, first);
            else
                for_constants(first, std::make_integer_sequence<int, WB>{});
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (VEC) {  // stage st+1 has landed; st+2's loads may be in flight
                if (FULL == NW || all_p)
                    dma_wait<DLP + DLQ>();
                else
                    dma_wait<DLP + DLQ - 1>();
            }
            lds_barrier();  // stage st+1 visible; the buffer of stage st-1 is free
            load();
            __builtin_amdgcn_sched_barrier(0);
            if (live)
                step(S1{}, next, second);
            else
                for_constants(second, std::make_integer_sequence<int, WB>{});
        };
        int st = 0;
        if constexpr (VEC) {
            if (main_loop) {
                for (; st + 6 < nwhole; st += 4)
                    for_constants(
                        [&](auto b_c) {
                            constexpr int BUF = decltype(b_c)::value;
                            stage(BUF, (BUF + 1) % GP_NBUF, [] {},
                                  among_q(std::integral_constant<int, (BUF + 2) % GP_NBUF>{}, st + BUF + 2),
                                  among_p(std::integral_constant<int, (BUF + 3) % GP_NBUF>{}, st + BUF + 3));
                        },
                        std::make_integer_sequence<int, 4>{});
                // Q's of the last stage begun (st is a multiple of 4)
                for_constants(among_q(std::integral_constant<int, 2>{}, st + 2), std::make_integer_sequence<int, WB>{});
            }
            for (; st + 1 < nstages; ++st)
                stage(st % GP_NBUF, (st + 1) % GP_NBUF, [&] { issue_any(st + 3); }, none, none);
        } else {
            auto pair = [&](int s, auto set_c) {  // set_c = s & 1, a constant so that the sets stay in registers
                constexpr int SET = decltype(set_c)::value;
                stage(
                    s % GP_NBUF, (s + 1) % GP_NBUF,
                    [&] {
                        store(SET, (s + 2) % GP_NBUF);
                        fetch(SET, s + 4);
                    },
                    none, none);
            };
            for (; st + 2 < nstages; st += 2) {
                pair(st, S0{});
                pair(st + 1, S1{});
            }
            if (st + 1 < nstages) {
                pair(st, S0{});
                ++st;
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        if (live) {
            step(S0{}, st % GP_NBUF, none);
#pragma unroll
            for (int m = 0; m < WB; ++m)
#pragma unroll
                for (int t = 0; t < TB; ++t) acc[m][t] = mfma32_t(p[m], q[1][t], acc[m][t], T{});
        }
        mfma_drain();
        dma_wait<0>();  // the surplus loads past the last stage
    }
    if (!live) return;

    // ---- epilogue: block (m, t) of the lane holds tile rows 32 (WB wr + m) +
    // 8 q + 4 (lane / 32) + 0..3 (q = 0..3) of column 32 (TB wc + t) + lane % 32.
    O* out;
    long long ldo;
    if constexpr (MODE == GP_WGRAD) {
        out = static_cast<O*>(g.out) + ((size_t)split * g.E + e) * g.N * g.K;
        ldo = g.K;
    } else {
        out = static_cast<O*>(g.out);
        ldo = MODE == GP_FWD ? g.ldc : g.lda;
    }
    bool zero_row[TB] = {};  // forward: a pair that names no input row
    if constexpr (MODE == GP_FWD) {
#pragma unroll
        for (int t = 0; t < TB; ++t) {
            const int c = c0 + 32 * (TB * wc + t) + r32;
            zero_row[t] = c < c1 && fwd_row(c) < 0;
        }
    }
    const T* bias = MODE == GP_FWD && g.bias ? static_cast<const T*>(g.bias) + (size_t)e * g.N : nullptr;
#pragma unroll
    for (int m = 0; m < WB; ++m) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int row = r0 + 32 * (WB * wr + m) + 8 * q + 4 * kg;
            if (row >= R) continue;
            const int nv = min(4, R - row);
            float bv[4] = {0.f, 0.f, 0.f, 0.f};
            if (MODE == GP_FWD && bias) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < nv) bv[i] = to_f32(bias[row + i]);
            }
#pragma unroll
            for (int t = 0; t < TB; ++t) {
                const int c = c0 + 32 * (TB * wc + t) + r32;
                if (c >= c1) continue;
                O* at = out + (size_t)c * ldo + row;
                float v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = (zero_row[t] ? 0.f : acc[m][t][4 * q + i]) + bv[i];
                if constexpr (std::is_same<O, float>::value) {
                    if (MODE == GP_WGRAD && g.accumulate) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (i < nv) v[i] += at[i];
                    }
                    if (nv == 4) {
                        store16_any(at, u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                              __float_as_uint(v[3])});
                        continue;
                    }
                } else if (nv == 4) {
                    store8_any(at, pack2<O>(v[0], v[1]), pack2<O>(v[2], v[3]));
                    continue;
                }
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    if (i < nv) at[i] = from_f32<O>(v[i]);
            }
        }
    }
}

// db[i] (+)= sum over the splits' partial sums, in split order.
template <typename O>
__global__ __launch_bounds__(256) void gmm_reduce_kernel(const float* __restrict__ part, long long n, int splits,
                                                         int accumulate, O* __restrict__ out)
{
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    float v = 0.f;
    for (int s = 0; s < splits; ++s) v += part[s * n + i];
    if constexpr (std::is_same<O, float>::value) {
        if (accumulate) v += out[i];
        out[i] = v;
    } else {
        out[i] = from_f32<O>(v);
    }
}

// ------------------------------------------------------------------ bias gradient
// dbias[e][n] = sum of dc's rows of segment e.  Pass 1: one workgroup per (range
// of DB_ROWS rows of an expert, 256 columns): 8 groups of 32 threads take every
// eighth row of the range, 8 columns (16 bytes) a thread, in fp32, and are added
// in order; pass 2 adds an expert's ranges in order, so the result does not
// depend on timing.
constexpr int DB_COLS = 256, DB_GROUPS = 8, DB_ROWS = 128;

// Ranges of the experts before e, and of e itself.
__device__ __forceinline__ int dbias_ranges(const GpArgs& g, int e, int* own)
{
    int before = 0;
    for (int base = 0; base <= e; base += WAVE) {
        const int j = base + lane_id();
        const Segment sg = j < g.E ? segment_of(g.offsets, j, g.M) : Segment{0, 0};
        const int n = (sg.end - sg.begin + DB_ROWS - 1) / DB_ROWS;
        before += wave_sum(j < e ? n : 0);
        if (e < base + WAVE) *own = __shfl(n, e - base, WAVE);
    }
    return before;
}

template <typename T>
__global__ __launch_bounds__(DB_COLS) void dbias_partial_kernel(GpArgs g, float* __restrict__ part)
{
    __shared__ float sh[DB_GROUPS][DB_COLS];
    const int cv = threadIdx.x & 31, grp = threadIdx.x >> 5;
    const int cols = (g.N + DB_COLS - 1) / DB_COLS, at = (int)(blockIdx.x / cols), c0 = (int)(blockIdx.x % cols) * DB_COLS;
    const int n = c0 + 8 * cv;
    // range `at` of the experts' consecutive ranges
    int e = -1, first = 0, before = 0;
    for (int base = 0; base < g.E && e < 0; base += WAVE) {
        const int j = base + lane_id();
        const Segment sg = j < g.E ? segment_of(g.offsets, j, g.M) : Segment{0, 0};
        const int k = (sg.end - sg.begin + DB_ROWS - 1) / DB_ROWS, excl = wave_excl_scan(k) + before;
        const uint64_t hit = ballot(at >= excl && at < excl + k);
        if (hit) {
            const int src = (int)__builtin_ctzll(hit);
            e = base + src;
            first = at - __shfl(excl, src, WAVE);
        }
        before = __shfl(excl + k, WAVE - 1, WAVE);
    }
    if (e < 0) return;  // uniform
    const Segment seg = segment_of(g.offsets, e, g.M);
    const int b = seg.begin + first * DB_ROWS, t = min(b + DB_ROWS, seg.end);
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (n < g.N) {
        const T* p = static_cast<const T*>(g.dc) + n;
        for (int s = b + grp; s < t; s += 8 * DB_GROUPS) {
            u32x4 x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = s + DB_GROUPS * i;
                x[i] = r < t ? load8_masked(p + (size_t)r * g.ldc, g.N - n) : u32x4{0, 0, 0, 0};
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[2 * j] += lo_f32<T>(x[i][j]);
                    v[2 * j + 1] += hi_f32<T>(x[i][j]);
                }
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sh[grp][8 * cv + j] = v[j];
    __syncthreads();
    const int c = c0 + (int)threadIdx.x;
    if (c >= g.N) return;
    float s = sh[0][threadIdx.x];
#pragma unroll
    for (int q = 1; q < DB_GROUPS; ++q) s += sh[q][threadIdx.x];
    part[(size_t)at * g.N + c] = s;
}

__global__ __launch_bounds__(256) void dbias_reduce_kernel(GpArgs g, const float* __restrict__ part,
                                                           float* __restrict__ dbias)
{
    const int e = blockIdx.y, n = blockIdx.x * 256 + threadIdx.x;
    int own = 0;
    // (offsets that decrease can count more ranges than there are: bounded)
    const int ranges = g.M / DB_ROWS + g.E, before = min(dbias_ranges(g, e, &own), ranges);
    own = min(own, ranges - before);
    if (n >= g.N) return;
    const float* p = part + (size_t)before * g.N + n;
    float s = 0.f;
    int i = 0;
    for (; i + 8 <= own; i += 8) {  // 8 loads in flight, added in order
        float x[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) x[q] = p[(size_t)(i + q) * g.N];
#pragma unroll
        for (int q = 0; q < 8; ++q) s += x[q];
    }
    for (; i < own; ++i) s += p[(size_t)i * g.N];
    float* out = dbias + (size_t)e * g.N + n;
    *out = g.accumulate ? *out + s : s;
}

__global__ __launch_bounds__(256) void zero16_kernel(uint16_t* __restrict__ p, long long n)
{
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) p[i] = 0;
}

template <typename T, typename O, int MODE, bool VEC, bool GATHER, typename Cfg>
hipError_t launch_gathered(const GpArgs& g, hipStream_t s)
{
    long long grid;
    if (MODE == GP_WGRAD) {
        const long long nt = (g.K + Cfg::BR - 1) / Cfg::BR, mt = (g.N + Cfg::BC - 1) / Cfg::BC;
        grid = (nt * mt + 7) / 8 * 8 * g.E * g.splits;
    } else {
        const long long nt = ((MODE == GP_FWD ? g.N : g.K) + Cfg::BR - 1) / Cfg::BR;
        grid = (nt * ((g.M + Cfg::BC - 1) / Cfg::BC + g.E) + 7) / 8 * 8;
    }
    if (grid * Cfg::THREADS > 0xFFFFFFFFll) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((gmm_kernel<T, O, MODE, VEC, GATHER, Cfg>), dim3((unsigned)grid), dim3(Cfg::THREADS), 0, s, g);
    return hipGetLastError();
}

template <typename T, typename O, int MODE, bool VEC, typename Cfg>
hipError_t launch_cfg(const GpArgs& g, hipStream_t s)
{
    if (MODE == GP_WGRAD && g.pairs) return launch_gathered<T, O, MODE, VEC, MODE == GP_WGRAD, Cfg>(g, s);
    return launch_gathered<T, O, MODE, VEC, false, Cfg>(g, s);
}

// Rows that the direct loads take: 16-byte aligned, and short enough that a
// tile's offsets (at most 320 rows) fit 32 bits.
bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }
bool vec_stride(long long ld) { return ld % 8 == 0 && ld <= 4ll << 20; }

// 320 or 256 tile rows: the one that covers the output's rows with fewer, and
// 320 where they tie (it loads a tenth less per product).  Measured on the Zipf
// prefill, 320 / 256 rows: 5760 columns 1188 / 1224 us, gradients at 2880 x 2880
// 1369 / 1404 us.  Counting rounds of 256 tiles instead (2592 tiles of 320 rows
// are 10.1 of them) predicts the opposite and is wrong.
template <int MODE>
bool wide_tile(const GpArgs& g)
{
    const int R = MODE == GP_FWD ? g.N : g.K;
    auto covered = [&](int BR) { return (R + BR - 1) / BR * BR; };
    return covered(TileWide::BR) <= covered(TileLarge::BR);
}

template <typename T, typename O, int MODE>
hipError_t launch_mode(const GpArgs& g, bool vec, bool small, hipStream_t s)
{
    if (vec) {
        if (small) return launch_cfg<T, O, MODE, true, TileSmall>(g, s);
        return wide_tile<MODE>(g) ? launch_cfg<T, O, MODE, true, TileWide>(g, s)
                                  : launch_cfg<T, O, MODE, true, TileLarge>(g, s);
    }
    return launch_cfg<T, O, MODE, false, TileSmall>(g, s);
}

GpArgs gp_args(const GmmArgs& a)
{
    GpArgs g;
    memset(&g, 0, sizeof g);
    g.M = a.M;
    g.N = a.N;
    g.K = a.K;
    g.E = a.E;
    g.a_rows = a.a_rows;
    g.k_shift = a.k > 1 ? 34 : 0;
    g.k_magic = a.k > 1 ? ((1ull << 34) + a.k - 1) / a.k : 1;
    g.lda = a.lda;
    g.ldc = a.ldc;
    g.offsets = a.offsets;
    g.pairs = a.pairs;
    g.a = a.a;
    g.b = a.b;
    g.bias = a.bias;
    g.dc = a.dc;
    g.out = a.out;
    g.splits = 1;
    return g;
}

template <int MODE>
hipError_t launch_types(const GmmArgs& a, const GpArgs& g, bool vec, bool small, hipStream_t s)
{
    if (a.dtype == DT_BF16)
        return a.out_dtype == DT_F32 ? launch_mode<bf16_t, float, MODE>(g, vec, small, s)
                                     : launch_mode<bf16_t, bf16_t, MODE>(g, vec, small, s);
    return a.out_dtype == DT_F32 ? launch_mode<f16_t, float, MODE>(g, vec, small, s)
                                 : launch_mode<f16_t, f16_t, MODE>(g, vec, small, s);
}

// The large tiles once an average expert's rows fill a third of one and there
// are tiles for a third of the CUs.  Small against large tiles, N = K = 2880
// unless said, in us:
//   32 experts, N 5760: 64 rows each 234 and 265, 96 rows each 311 and 271;
//   1 expert: 2048 rows (72 large tiles) 62 and 75, 2560 rows (90) 83 and 78;
//   8 experts: 2048 rows (72) 77 and 90, 2560 rows (90) 94 and 81.
bool use_small_tile(const GmmArgs& a, int cols)
{
    return (long long)a.M < 80ll * a.E || (long long)(a.M / TileWide::BC) * ((cols + TileWide::BR - 1) / TileWide::BR) < 85;
}

}  // namespace

hipError_t launch_zero16(void* p, int64_t n, hipStream_t s)
{
    if (!p || n <= 0) return hipSuccess;
    const long long blocks = (n + 255) / 256;
    hipLaunchKernelGGL(zero16_kernel, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), 0, s, static_cast<uint16_t*>(p),
                       (long long)n);
    return hipGetLastError();
}

hipError_t launch_gmm_forward(const GmmArgs& a, hipStream_t s)
{
    const GpArgs g = gp_args(a);
    const bool vec = aligned16(a.a) && aligned16(a.b) && a.K % 8 == 0 && vec_stride(a.lda);
    return launch_types<GP_FWD>(a, g, vec, use_small_tile(a, a.N), s);
}

hipError_t launch_gmm_dgrad(const GmmArgs& a, hipStream_t s)
{
    const GpArgs g = gp_args(a);
    const bool vec = aligned16(a.dc) && aligned16(a.b) && a.K % 8 == 0 && a.N % 8 == 0 && vec_stride(a.ldc);
    return launch_types<GP_DGRAD>(a, g, vec, use_small_tile(a, a.K), s);
}

// Ranges of rows whose partial sums are added up afterwards, where the small
// tiles alone would leave CUs without work: two tiles per CU, and at least 1024
// rows of an average expert per range.  Without and with, one expert, N = K =
// 1024 (128 tiles), in us: 2048 rows 14.4 and 15.9, 4096 rows 32 and 22, 65536
// rows 457 and 231.  From 256 tiles on the second pass costs more than it gives:
// 8 experts, N = K = 512, 65536 rows, 67 without and 79 with two ranges.
int gmm_wgrad_splits(int M, int N, int K, int E)
{
    const long long tiles = (long long)((N + TileSmall::BR - 1) / TileSmall::BR) *
                            ((K + TileSmall::BC - 1) / TileSmall::BC) * E;
    if (tiles >= 256) return 1;
    const long long by_rows = (long long)M / E / 1024, by_tiles = 512 / tiles;
    const long long sp = by_rows < by_tiles ? by_rows : by_tiles;
    return sp < 1 ? 1 : sp > 64 ? 64 : (int)sp;
}

// sum over experts of ceil(len / DB_ROWS)
int gmm_dbias_ranges(int M, int E) { return M / DB_ROWS + E; }

hipError_t launch_gmm_wgrad(const GmmArgs& a, hipStream_t s)
{
    GpArgs g = gp_args(a);
    g.splits = a.splits;
    g.accumulate = a.accumulate;
    const bool vec = aligned16(a.a) && aligned16(a.dc) && a.K % 8 == 0 && a.N % 8 == 0 && vec_stride(a.lda) &&
                     vec_stride(a.ldc);
    // The large tiles once every CU has one.  Small against large, in us: 4096
    // rows, 2 experts, 2880 x 2880 (288 large tiles) 91 and 71; 8192 rows, 8
    // experts, 1024 x 2048 (256) 52 and 42; 1 expert, 2880 x 2880 (144) 180 and 191.
    const bool small = (long long)((a.N + 255) / 256) * ((a.K + 255) / 256) * a.E * a.splits < 256;
    // The bias gradient first: after the weight gradient its reads would wait for
    // that kernel's writes to drain to HBM.
    hipError_t err;
    if (a.dbias) {
        const int cols = (a.N + DB_COLS - 1) / DB_COLS;
        const dim3 grid((unsigned)((long long)cols * gmm_dbias_ranges(a.M, a.E)));
        if (a.dtype == DT_BF16)
            hipLaunchKernelGGL(dbias_partial_kernel<bf16_t>, grid, dim3(DB_COLS), 0, s, g, a.dbias_part);
        else
            hipLaunchKernelGGL(dbias_partial_kernel<f16_t>, grid, dim3(DB_COLS), 0, s, g, a.dbias_part);
        if ((err = hipGetLastError()) != hipSuccess) return err;
        hipLaunchKernelGGL(dbias_reduce_kernel, dim3((a.N + 255) / 256, a.E), dim3(256), 0, s, g, a.dbias_part, a.dbias);
        if ((err = hipGetLastError()) != hipSuccess) return err;
    }
    if (a.splits > 1) {
        g.out = a.part;
        g.accumulate = 0;
        GmmArgs p = a;
        p.out_dtype = DT_F32;
        if ((err = launch_types<GP_WGRAD>(p, g, vec, small, s)) != hipSuccess) return err;
        const long long n = (long long)a.E * a.N * a.K;
        const dim3 grid((unsigned)((n + 255) / 256));
        if (a.out_dtype == DT_F32)
            hipLaunchKernelGGL(gmm_reduce_kernel<float>, grid, dim3(256), 0, s, a.part, n, a.splits, a.accumulate,
                               static_cast<float*>(a.out));
        else if (a.dtype == DT_BF16)
            hipLaunchKernelGGL(gmm_reduce_kernel<bf16_t>, grid, dim3(256), 0, s, a.part, n, a.splits, 0,
                               static_cast<bf16_t*>(a.out));
        else
            hipLaunchKernelGGL(gmm_reduce_kernel<f16_t>, grid, dim3(256), 0, s, a.part, n, a.splits, 0,
                               static_cast<f16_t*>(a.out));
        return hipGetLastError();
    }
    return launch_types<GP_WGRAD>(a, g, vec, small, s);
}

}  // namespace moe
