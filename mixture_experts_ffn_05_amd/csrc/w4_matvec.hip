// Products of few rows with 4-bit weights (decoding).
//
//   v[s][n] = sum_i x[r(s)][i] scale[n][i / group] (code[n][i] - zero[n][i / group]) + bias[n]
// and, for SwiGLU, y[s][n] = silu(v[s][n]) v[s][N/2 + n].  The codes are the
// traffic; every one is read once per XR rows of an expert.
//
// An item is 32 weight rows (for SwiGLU 16 gate rows and the matching 16 up
// rows) times up to XR rows of x.  A wave streams its items' K in chunks of 256
// (128) columns through its own ring of LDS slots, filled by direct-to-LDS loads
// that run on into the next item: no barrier, no bubble between items, and
// a slot's codes always in flight.  A slot holds 128 (64) bytes of each weight
// row and the x rows' same columns, a table beside it the scales and zero points
// of one or two chunks, so nothing but LDS is read in the loop.  With few items
// (KS = 4) the 4 waves of a workgroup share an item, every fourth chunk each,
// and add up through LDS.
//
// v_mfma_f32_16x16x32 takes x's rows as its A rows and weight rows as its B
// columns, so a lane's four results are rows of x for one n: a group's scale and
// zero point are one value per lane.  Codes become 16-bit floats without
// arithmetic: a code placed in the mantissa of 16.0 is exactly 16 + code (a
// shift and an and-or for two codes).  Per group the matrix cores sum D = sum
// (16 + code) x and, against a matrix of ones, S = sum x; then
// v += scale (D - (16 + zero) S) in fp32.  Nothing is rounded between the code
// and the fp32 sum.  The two codes of a word that share a register are 4 apart;
// x's fragments are permuted to match (four byte permutes, shared by both
// 16-row tiles).  With 4 or 8 rows of x the 16 A rows hold 4 or 2 groups side
// by side, so that one correction serves as many groups: the vector work per
// code, not the matrix cores, is what competes with the memory here.
//
// 16 tokens, 4 of 128 experts, 2880 -> 5760 with SwiGLU, groups of 64: 110 us for
// 463 MB (4.2 TB/s; 409 with slots filled through registers, 140 without the
// groups side by side, 117 with scales gathered for every chunk).  It is bound by
// the cache lines that the loads touch: with 64-byte pieces of the rows, twice the
// lines and the same bytes, it takes 150 us at two, three or four workgroups a CU.
#include <string.h>

#include <type_traits>

#include "elem16.h"
#include "moe_ops.h"
#include "tile_sched.h"

namespace moe {

namespace {

constexpr int WQ_NW = 4;     // waves per workgroup
constexpr int WQ_DEPTH = 2;  // ring slots per wave
constexpr int WQ_THREADS = WQ_NW * WAVE;

__device__ uint32_t wq_zeros[4] __attribute__((aligned(16)));  // never written

struct WqArgs {
    int M, N, K, E, x_rows, k;
    int group, swiglu, out_f32;
    const int32_t* offsets;
    const int32_t* pairs;
    const void* x;
    const uint8_t* codes;
    const void* scales;
    const uint8_t* zeros;
    const void* bias;
    void* out;
};

// Codes in the mantissa of 16.0: pairs (0,4)(1,5)(2,6)(3,7) of a word's eight.
// mask and base stay in registers, so that masking and joining are one
// instruction (two literals would not fit it).
template <typename T>
struct Code16 {
    static constexpr bool B = std::is_same<T, bf16_t>::value;
    static constexpr uint32_t one = B ? 0x3F803F80u : 0x3C003C00u;  // (1.0, 1.0)
    uint32_t mask = B ? 0x00780078u : 0x03C003C0u, base = B ? 0x41804180u : 0x4C004C00u;
    __device__ __forceinline__ Code16() { asm("" : "+v"(mask), "+s"(base)); }
    __device__ __forceinline__ u32x4 decode(uint32_t w) const
    {
        return B ? u32x4{((w << 3) & mask) | base, ((w >> 1) & mask) | base, ((w >> 5) & mask) | base,
                         ((w >> 9) & mask) | base}
                 : u32x4{((w << 6) & mask) | base, ((w << 2) & mask) | base, ((w >> 2) & mask) | base,
                         ((w >> 6) & mask) | base};
    }
};

// Elements (0,1)(2,3)(4,5)(6,7) -> (0,4)(1,5)(2,6)(3,7).
__device__ __forceinline__ u32x4 pair_by_four(u32x4 v)
{
    return u32x4{__builtin_amdgcn_perm(v.z, v.x, 0x05040100u), __builtin_amdgcn_perm(v.z, v.x, 0x07060302u),
                 __builtin_amdgcn_perm(v.w, v.y, 0x05040100u), __builtin_amdgcn_perm(v.w, v.y, 0x07060302u)};
}

typedef __attribute__((address_space(4))) const int32_t* wq_cptr;  // read through the scalar unit

// GB: 32-column blocks per group.  Z: zero points given (else 8).  XR: rows of
// x per item.  KS: waves that share an item's K.
template <int GB, bool Z, int XR, int KS>
struct WqShape {
    // Columns per chunk.  A wave that streams whole rows takes 128-byte pieces of
    // them; with 16 rows of x, or rows shared by four waves, 64-byte pieces, whose
    // slots leave room for two or more workgroups a CU.  64-byte against 128-byte
    // pieces: 13.6 and 17.5 us (1 row, 2 of 32 experts, 2880 -> 5760, KS = 4),
    // 14.6 and 21.8 us (64 rows, 2880 -> 2880).
    static constexpr int CK = XR < 16 && KS == 1 ? 256 : 128, ROWB = CK / 2;
    static constexpr int BPC = CK / 32, GPC = BPC / GB;  // 32-column blocks, groups per chunk
    static constexpr int WBYTES = 32 * ROWB, XBYTES = XR * 2 * CK;
    // Scales and zero points are gathered for SPAN chunks at once, into one of two
    // tables (one slot's, where SPAN is 1): a gather's cost is the cache lines it
    // touches, one a row.  Two chunks (110 us against 117 for one, 16 tokens as
    // above) where the tables leave room for two workgroups a CU and a wave's
    // chunks are adjacent.
    static constexpr int table(int span) { return span * GPC < 2 ? 256 : 32 * span * GPC * 4; }
    static constexpr int SPAN =
        KS == 1 && WQ_NW * 2 * (WBYTES + XBYTES + (Z ? 2 : 1) * table(2)) + 16 <= 80 * 1024 ? 2 : 1;
    static constexpr int SBYTES = table(SPAN), SLOT = WBYTES + XBYTES, TABLE = (Z ? 2 : 1) * SBYTES;
    static constexpr int RING = WQ_NW * WQ_DEPTH * (SLOT + TABLE), RED = KS > 1 ? WQ_NW * 2 * WAVE : 1;
    static_assert(WQ_DEPTH == 2, "a table per slot, or two chunks a table");
    // Two workgroups per CU where their LDS fits: asking for them also keeps
    // the matrix cores' results in ordinary registers.
    static constexpr int WAVES_PER_SIMD = RING + RED * 16 <= 80 * 1024 ? 2 : 1;
};

template <typename T, int GB, bool Z, int XR, int KS>
__global__ __launch_bounds__(WQ_THREADS, (WqShape<GB, Z, XR, KS>::WAVES_PER_SIMD)) void w4_matvec_kernel(WqArgs g)
{
    using S = WqShape<GB, Z, XR, KS>;
    static_assert(KS == 1 || KS == WQ_NW, "an item belongs to a wave or to a workgroup");
    constexpr int GPC = S::GPC, WBYTES = S::WBYTES, XBYTES = S::XBYTES, SBYTES = S::SBYTES, SLOT = S::SLOT;
    constexpr int SPAN = S::SPAN, TG = SPAN * GPC;  // chunks, groups per table
    constexpr int WQ_CK = S::CK, WQ_ROWB = S::ROWB;
    constexpr int WL = WBYTES / 1024, XL = XBYTES / 1024, SL = SBYTES / 256;  // loads per slot
    constexpr int NL = WL + XL, NT = (Z ? 2 : 1) * SL;  // of a slot, of a table
    static_assert(XL >= 1 && NL + NT < 64, "load count");
    __shared__ __attribute__((aligned(16))) uint8_t sh[S::RING];
    __shared__ f32x4 red[S::RED];

    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int l16 = lane & 15, kg = lane >> 4;
    const bool swiglu = g.swiglu;
    const int half = g.N / 2, G = (g.K + g.group - 1) / g.group;
    const int nchunks = (g.K + SPAN * WQ_CK - 1) / (SPAN * WQ_CK) * SPAN;  // whole tables; zeros past K
    const int tiles = swiglu ? (half + 15) / 16 : (g.N + 31) / 32;
    uint8_t* ring = sh + wave * WQ_DEPTH * (SLOT + S::TABLE);
    uint8_t* tables = ring + WQ_DEPTH * SLOT;
    const int cw = KS > 1 ? wave : 0;  // first chunk of this wave

    // ---- every expert's segment, one per lane (E <= 256), and its first item
    int seg_b[4], seg_n[4], first[4], items = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        seg_b[j] = seg_n[j] = first[j] = 0;
        if (WAVE * j >= g.E) continue;  // uniform
        const int e = lane + WAVE * j;
        if (e < g.E) {
            const Segment sg = segment_of(g.offsets, e, g.M);
            seg_b[j] = sg.begin;
            seg_n[j] = sg.end - sg.begin;
        }
        const int n = (seg_n[j] + XR - 1) / XR * tiles;
        const int excl = wave_excl_scan(n);
        first[j] = items + excl;
        items += __shfl(excl + n, WAVE - 1, WAVE);
    }
    items = __builtin_amdgcn_readfirstlane(items);
    const int stride = KS > 1 ? (int)gridDim.x : (int)gridDim.x * WQ_NW;

    struct Item {
        int e, s0, s1, n0;  // expert, rows [s0, s1) of x (at most XR), first output column
    };
    auto locate = [&](int it) {
        Item r{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (WAVE * j >= g.E) continue;
            const int n = (seg_n[j] + XR - 1) / XR * tiles;
            const uint64_t hit = ballot(n > 0 && it >= first[j] && it < first[j] + n);
            if (hit) {
                const int src = (int)__builtin_ctzll(hit);
                const int local = it - __builtin_amdgcn_readlane(first[j], src);
                const int pass = local / tiles;
                r.e = WAVE * j + src;
                r.s0 = __builtin_amdgcn_readlane(seg_b[j], src) + pass * XR;
                r.s1 = min(r.s0 + XR, __builtin_amdgcn_readlane(seg_b[j], src) + __builtin_amdgcn_readlane(seg_n[j], src));
                r.n0 = (local - pass * tiles) * (swiglu ? 16 : 32);
            }
        }
        return r;
    };
    // Weight row of an item's row i (0..31), clamped to the matrix.
    auto wrow = [&](const Item& t, int i) {
        const int n = min(t.n0 + (i & 15), half - 1);
        return swiglu ? (i < 16 ? n : half + n) : min(t.n0 + i, g.N - 1);
    };

    // ---- issue side: sources of the item being loaded.  Weights: a row's chunk
    // is WPP 16-byte pieces, piece p of row r lying at p ^ wswz(r); x: XPP pieces,
    // piece p of row r at p ^ (r % 16): the 16 rows that one fragment read touches
    // fall on different banks.
    constexpr int WPP = WQ_ROWB / 16, WRPL = WAVE / WPP;        // pieces a row, rows a load
    constexpr int XPP = 2 * WQ_CK / 16, XRPL = WAVE / XPP;
    auto wswz = [](int r) { return WPP == 8 ? (r >> 1) & 7 : (r >> 2) & 3; };
    const uintptr_t zeros = reinterpret_cast<uintptr_t>(wq_zeros);
    uintptr_t wsrc[WL], xsrc[XL], ssrc[SL], zsrc[Z ? SL : 1];
    int xlim[XL];
    auto open = [&](const Item& t) {
        const size_t erow = (size_t)t.e * g.N;
#pragma unroll
        for (int i = 0; i < WL; ++i) {
            const int r = WRPL * i + lane / WPP, p = (lane % WPP) ^ wswz(r);
            wsrc[i] = reinterpret_cast<uintptr_t>(g.codes) + (erow + wrow(t, r)) * (size_t)(g.K / 2) + 16 * p;
        }
#pragma unroll
        for (int i = 0; i < SL; ++i) {
            const int q = min(lane + WAVE * i, 32 * TG - 1);
            const size_t at = (erow + wrow(t, q / TG)) * G + q % TG;
            ssrc[i] = reinterpret_cast<uintptr_t>(g.scales) + 2 * at;
            if (Z) zsrc[i] = reinterpret_cast<uintptr_t>(g.zeros) + at;
        }
        wq_cptr ids = (wq_cptr)(uintptr_t)g.pairs;
#pragma unroll
        for (int i = 0; i < XL; ++i) {
            int src = -1;
#pragma unroll
            for (int h = 0; h < XRPL; ++h) {
                const int s = t.s0 + XRPL * i + h;
                int row = s < t.s1 ? s : -1;
                if (g.pairs) {  // uniform
                    const int p = ids[min(s, t.s1 - 1)];
                    row = s < t.s1 && p >= 0 ? p / g.k : -1;
                }
                if (row >= g.x_rows) row = -1;
                src = lane / XPP == h ? row : src;
            }
            const int r = XRPL * i + lane / XPP, p = (lane % XPP) ^ (r & 15);
            xlim[i] = src >= 0 ? g.K - 8 * p : 0;
            xsrc[i] = reinterpret_cast<uintptr_t>(g.x) + ((size_t)max(src, 0) * g.K + 8 * p) * 2;
        }
    };
    // Chunk c of the open item into a slot; chunks at or past nchunks read zeros only.
    int itab = 0, ctab = 0;  // table to fill, table in use
    auto issue = [&](int c, int slot) {
        uint8_t* at = ring + slot * SLOT;
        const int k0 = c * WQ_CK;
#pragma unroll
        for (int i = 0; i < WL; ++i) {
            const int k = 32 * ((lane % WPP) ^ wswz(WRPL * i + lane / WPP));
            dma16(reinterpret_cast<const void*>(k0 + k < g.K ? wsrc[i] + (size_t)c * WQ_ROWB : zeros), at + 1024 * i);
        }
#pragma unroll
        for (int i = 0; i < XL; ++i)
            dma16(reinterpret_cast<const void*>(k0 < xlim[i] ? xsrc[i] + 2 * (size_t)k0 : zeros), at + WBYTES + 1024 * i);
        if (SPAN > 1 && slot) return;  // an even chunk brings the table of two
        uint8_t* tab = tables + itab * S::TABLE;
        itab ^= 1;
#pragma unroll
        for (int i = 0; i < SL; ++i) {
            const bool ok = c * GPC + min(lane + WAVE * i, 32 * TG - 1) % TG < G;
            dma_u16(reinterpret_cast<const void*>(ok ? ssrc[i] + 2 * (size_t)(c * GPC) : zeros), tab + 256 * i);
            if constexpr (Z)
                dma_u8(reinterpret_cast<const void*>(ok ? zsrc[i] + (size_t)(c * GPC) : zeros), tab + SBYTES + 256 * i);
        }
    };

    int it = KS > 1 ? (int)blockIdx.x : (int)blockIdx.x * WQ_NW + wave;
    if (it >= items) return;  // uniform per item owner
    Item cur = locate(it), next_item = cur;
    int iit = it, ic = cw;  // item and chunk to load next
    open(cur);
    auto advance = [&](int slot) {  // load the next chunk of this wave's stream
        if (iit < items && ic >= nchunks) {
            iit += stride;
            ic = cw;
            if (iit < items) {
                next_item = locate(iit);
                open(next_item);
            }
        }
        issue(iit < items ? ic : nchunks, slot);
        ic += KS;
    };
#pragma unroll
    for (int d = 0; d < WQ_DEPTH; ++d) {
        if (cw < nchunks) advance(d);
    }

    // The 16 A rows of the matrix cores are XR rows of x times SLOTS groups: A
    // row XR u + r holds row r in the columns of the set's group u and zeros
    // elsewhere, so D's rows XR u + r are group u's sums alone, and a lane
    // scales the sums of its own group: one correction for SPC groups.
    constexpr int SLOTS = 16 / XR, SPC = SLOTS < GPC ? SLOTS : GPC;
    const int my_slot = l16 / XR, xr = l16 % XR;         // of the A row this lane supplies
    const int d_slot = min(4 * kg / XR, SPC - 1);        // of the D rows it receives
    const Code16<T> code;
    uint32_t mask[SLOTS];
#pragma unroll
    for (int u = 0; u < SLOTS; ++u) mask[u] = my_slot == u ? ~0u : 0u;
    const u32x4 ones = u32x4{Code16<T>::one, Code16<T>::one, Code16<T>::one, Code16<T>::one};
    int slot = 0;
    for (; it < items; it += stride) {
        cur = locate(it);
        f32x4 acc[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
        for (int c = cw; c < nchunks; c += KS) {
            // all but the next chunk's loads, which have a table's among them unless
            // this chunk's table is also the next one's
            if (SPAN > 1 && slot == 0)
                dma_wait<NL>();
            else
                dma_wait<NL + NT>();
            const uint8_t* at = ring + slot * SLOT;
            const uint32_t* st = reinterpret_cast<const uint32_t*>(tables + ctab * S::TABLE) + (SPAN > 1 ? slot * GPC : 0);
#pragma unroll
            for (int q = 0; q < GPC; q += SPC) {  // a set of groups
                f32x4 dsum[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}}, xsum = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int b = 0; b < GB; ++b) {
                    const int jx = (q + min(my_slot, SPC - 1)) * GB + b;  // block of this lane's A row
                    u32x4 a = pair_by_four(
                        *reinterpret_cast<const u32x4*>(at + WBYTES + xr * (2 * WQ_CK) + (((4 * jx + kg) ^ xr) << 4)));
                    xsum = mfma16_t(a, ones, xsum, T{});
#pragma unroll
                    for (int u = 0; u < SPC; ++u) {
                        const u32x4 am = SLOTS == 1 ? a : a & mask[u];
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            const int r = 16 * n + l16, j = (q + u) * GB + b;
                            const uint32_t w =
                                *reinterpret_cast<const uint32_t*>(at + r * WQ_ROWB + ((j ^ wswz(r)) << 4) + 4 * kg);
                            dsum[n] = mfma16_t(am, code.decode(w), dsum[n], T{});
                        }
                    }
                }
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const int si = (16 * n + l16) * TG + q + d_slot;
                    const float sc = to_f32(T{(uint16_t)st[si]});
                    const float z = Z ? 16.f + (float)(st[SBYTES / 4 + si] & 15u) : 24.f;
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[n][i] = fmaf(sc, fmaf(-z, xsum[i], dsum[n][i]), acc[n][i]);
                }
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // this slot's reads are done
            advance(slot);
            if (SPAN == 1 || slot) ctab ^= 1;
            slot ^= 1;
        }

        // ---- the item's results: rows 4 kg % XR + i, summed over the slots
        // (A rows of slots past SPC hold a copy of the last one's x: not summed)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (4 * kg / XR >= SPC) acc[n][i] = 0.f;
                if constexpr (XR <= 8) acc[n][i] += __shfl_xor(acc[n][i], 32, WAVE);
                if constexpr (XR <= 4) acc[n][i] += __shfl_xor(acc[n][i], 16, WAVE);
            }
        if constexpr (KS > 1) {
            if (it != (int)blockIdx.x) lds_barrier();  // the last item's sums have been read
#pragma unroll
            for (int n = 0; n < 2; ++n) red[(wave * 2 + n) * WAVE + lane] = acc[n];
            lds_barrier();
            if (wave >= (swiglu ? 1 : 2)) continue;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                if (!swiglu && n != wave) continue;
                acc[n] = red[n * WAVE + lane];
#pragma unroll
                for (int w = 1; w < WQ_NW; ++w) acc[n] += red[(w * 2 + n) * WAVE + lane];
            }
        }
        const T* bias = g.bias ? static_cast<const T*>(g.bias) + (size_t)cur.e * g.N : nullptr;
        const int cols = swiglu ? half : g.N;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            if (swiglu ? n > 0 : KS > 1 && n != wave) continue;
            const int col = cur.n0 + 16 * n + l16;
            if (col >= cols) continue;
            f32x4 v = acc[n];
            const float b = bias ? to_f32(bias[col]) : 0.f;
            if (swiglu) {
                const float bu = bias ? to_f32(bias[half + col]) : 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = silu(v[i] + b) * (acc[1][i] + bu);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] += b;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 4 * kg + i;  // the first slot's lanes store
                if (r >= XR || cur.s0 + r >= cur.s1) continue;
                const size_t at = (size_t)(cur.s0 + r) * cols + col;
                if (g.out_f32)
                    static_cast<float*>(g.out)[at] = v[i];
                else
                    static_cast<T*>(g.out)[at] = from_f32<T>(v[i]);
            }
        }
    }
    dma_wait<0>();  // loads past the last chunk
}

constexpr int WQ_CUS = 256;

template <typename T, int GB, bool Z, int XR>
hipError_t launch_xr(const WqArgs& g, hipStream_t s)
{
    const long long tiles = g.swiglu ? (g.N / 2 + 15) / 16 : (g.N + 31) / 32;
    const long long items = tiles * ((g.M + XR - 1) / XR + (g.E == 1 ? 0 : g.E < g.M ? g.E : g.M));  // at most
    // A wave per item once there are items for every wave of the chip (two workgroups a CU),
    // a workgroup per item before.  Wave and workgroup, 2880 columns, in us: 1 row,
    // 90 items 17 and 8, 1024 items 18 and 15, 2048 items 26 and 28; 32 experts'
    // SwiGLU, 4 of them 18 and 13, 16 of them (3600 items) 34 and 36.
    if (items >= 8 * WQ_CUS) {
        const long long blocks = (items + WQ_NW - 1) / WQ_NW, most = 2 * WQ_CUS;
        hipLaunchKernelGGL((w4_matvec_kernel<T, GB, Z, XR, 1>), dim3((unsigned)(blocks < most ? blocks : most)),
                           dim3(WQ_THREADS), 0, s, g);
    } else {
        hipLaunchKernelGGL((w4_matvec_kernel<T, GB, Z, XR, WQ_NW>), dim3((unsigned)items), dim3(WQ_THREADS), 0, s, g);
    }
    return hipGetLastError();
}

// Rows of x per item: twice an expert's average share (its share varies), so
// that a second pass over an expert's codes is rare, in the smallest form that
// holds them; a wider one costs LDS space, and with it loads in flight.  32
// experts' SwiGLU, 2880 -> 5760, in us: 2 rows each, 67 with 4 and 84 with 16; 4
// rows each, 68, 71 and 84 with 4, 8 and 16; 8 rows each, 115 with 4 and 88 with 16.
template <typename T, int GB, bool Z>
hipError_t launch_rows(const WqArgs& g, hipStream_t s)
{
    const int want = g.E == 1 ? g.M : 2 * ((g.M + g.E - 1) / g.E);
    if (want <= 4) return launch_xr<T, GB, Z, 4>(g, s);
    if (want <= 8) return launch_xr<T, GB, Z, 8>(g, s);
    return launch_xr<T, GB, Z, 16>(g, s);
}

template <typename T, int GB>
hipError_t launch_zeros(const WqArgs& g, hipStream_t s)
{
    return g.zeros ? launch_rows<T, GB, true>(g, s) : launch_rows<T, GB, false>(g, s);
}

template <typename T>
hipError_t launch_group(const WqArgs& g, hipStream_t s)
{
    return g.group == 32 ? launch_zeros<T, 1>(g, s) : g.group == 64 ? launch_zeros<T, 2>(g, s) : launch_zeros<T, 4>(g, s);
}

}  // namespace

hipError_t launch_w4_matvec(const W4Args& a, hipStream_t s)
{
    WqArgs g;
    memset(&g, 0, sizeof g);
    g.M = a.M;
    g.N = a.N;
    g.K = a.K;
    g.E = a.E;
    g.x_rows = a.x_rows;
    g.k = a.k;
    g.group = a.group;
    g.offsets = a.offsets;
    g.pairs = a.pairs;
    g.x = a.x;
    g.codes = a.codes;
    g.scales = a.scales;
    g.zeros = a.zeros;
    g.bias = a.bias;
    g.out = a.out;
    g.swiglu = a.swiglu;
    g.out_f32 = a.out_dtype == DT_F32;
    return a.dtype == DT_BF16 ? launch_group<bf16_t>(g, s) : launch_group<f16_t>(g, s);
}

}  // namespace moe
