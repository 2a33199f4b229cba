// Products of few rows with an expert's matrix (decoding): the weights are the
// traffic, and every one is read once per pass over the rows.
//
//   y[s][n] = sum_k x[r(s)][k] w[e][n][k] + bias[e][n]
// with w a 16-bit matrix (moe_grouped_mm with few rows) or 4-bit codes with a
// scale and a zero point per group of 32, 64 or 128 columns (moe_w4_matvec),
//   w[n][k] = scale[n][k / group] * (code[n][k] - zero[n][k / group]),
// whose result may be the SwiGLU of the first and second half of the columns n.
//
// A workgroup owns 32 weight rows (for SwiGLU 16 gate rows and the matching 16
// up rows) of one expert; its 4 waves split K in chunks and add up at the end.
// Each wave runs its own ring of LDS slots filled by direct-to-LDS loads, so
// there is no barrier in the loop and several KB per wave are always in
// flight: a chunk's weights (256 bytes a row for 16-bit, 128 bytes for 4-bit
// rows: whole cache lines) and the same columns of up to XR rows of x.
// v_mfma_f32_16x16x32 takes x's rows as its A rows and weight rows as its B
// columns, so a lane's four results are four rows of x for one n: a group's
// scale and zero point are one value per lane.
//
// 4-bit codes become 16-bit floats without arithmetic: a code placed in the
// mantissa of 16.0 is exactly 16 + code (one shift and one and-or for two
// codes).  Per group the matrix cores sum D = sum (16 + code) x and, against a
// matrix of ones, S = sum x; then y += scale * (D - (16 + zero) S) in fp32.
// Nothing is rounded between the code and the fp32 sum.  Two codes of a word
// that share a register are 4 apart, so x's fragments are permuted to match
// (four byte permutes, shared by all weight rows).
#include <string.h>

#include <type_traits>

#include "elem16.h"
#include "moe_ops.h"

namespace moe {

namespace {

constexpr int SK_NW = 4;                 // waves per workgroup
constexpr int SK_THREADS = SK_NW * WAVE;
constexpr int SK_NT = 2;                 // 16-row weight tiles per workgroup
constexpr int SK_DEPTH = 2;              // ring slots per wave
constexpr int SK_TABLE = 128;            // groups whose scales are held in LDS at a time

__device__ uint32_t sk_zeros[4] __attribute__((aligned(16)));  // never written

struct SkArgs {
    int M, N, K, E, x_rows, k;
    long long ldx, ldo;
    int group;
    const int32_t* offsets;
    const int32_t* pairs;
    const void* x;
    const void* w;
    const void* scales;
    const uint8_t* zeros;
    const void* bias;
    void* out;
};

// The a-th (0-based) expert with a non-empty segment; -1 if there are fewer.
__device__ __forceinline__ int sk_active_expert(const SkArgs& g, int a)
{
    if (!g.offsets) return a == 0 ? 0 : -1;
    const int lane = lane_id();
    for (int base = 0; base < g.E; base += WAVE) {
        const int e = base + lane;
        bool act = false;
        if (e < g.E) {
            const Segment sg = segment_of(g.offsets, e, g.M);
            act = sg.end > sg.begin;
        }
        const uint64_t m = ballot(act);
        const int cnt = __popcll(m);
        if (a < cnt) {
            const int before = __popcll(m & lanemask_lt());
            return base + (int)__builtin_ctzll(ballot(act && before == a));
        }
        a -= cnt;
    }
    return -1;
}

template <typename T>
struct Code16;  // codes in the mantissa of 16.0
template <>
struct Code16<bf16_t> {
    static constexpr uint32_t one = 0x3F803F80u;  // (1.0, 1.0)
    static __device__ __forceinline__ u32x4 decode(uint32_t w)
    {
        constexpr uint32_t m = 0x00780078u, b = 0x41804180u;
        return u32x4{((w << 3) & m) | b, ((w >> 1) & m) | b, ((w >> 5) & m) | b, ((w >> 9) & m) | b};
    }
};
template <>
struct Code16<f16_t> {
    static constexpr uint32_t one = 0x3C003C00u;
    static __device__ __forceinline__ u32x4 decode(uint32_t w)
    {
        constexpr uint32_t m = 0x03C003C0u, b = 0x4C004C00u;
        return u32x4{((w << 6) & m) | b, ((w << 2) & m) | b, ((w >> 2) & m) | b, ((w >> 6) & m) | b};
    }
};

// Elements (0,1)(2,3)(4,5)(6,7) -> (0,4)(1,5)(2,6)(3,7).
__device__ __forceinline__ u32x4 pair_by_four(u32x4 v)
{
    return u32x4{__builtin_amdgcn_perm(v.z, v.x, 0x05040100u), __builtin_amdgcn_perm(v.z, v.x, 0x07060302u),
                 __builtin_amdgcn_perm(v.w, v.y, 0x05040100u), __builtin_amdgcn_perm(v.w, v.y, 0x07060302u)};
}

template <bool W4, int XR>
struct SkShape {
    static constexpr int CK = W4 ? 256 : 128;          // columns per chunk
    static constexpr int WROW = W4 ? CK / 2 : CK * 2;  // bytes of a weight row's chunk
    static constexpr int XROW = CK * 2;                // bytes of an x row's chunk
    static constexpr int WBYTES = SK_NT * 16 * WROW, XBYTES = XR * XROW;
    static constexpr int SLOT = WBYTES + XBYTES;
    static constexpr int WL = WBYTES / 1024, XL = XBYTES / 1024;  // loads per wave and slot
    static constexpr int RING = SK_NW * SK_DEPTH * SLOT;
    static constexpr int TT = XR <= 16 ? 1 : XR / 16;  // 16-row tiles of x
    static_assert(XL >= 1 && (SK_DEPTH - 1) * (WL + XL) < 64, "load count");
    static_assert(SK_NW * SK_NT * TT * 1024 <= RING, "the reduction reuses the ring");
};

// GB: 32-column blocks per group (W4).  XR: rows of x per pass.
template <typename T, typename O, bool W4, int GB, bool SWIGLU, int XR>
__global__ __launch_bounds__(SK_THREADS) void skinny_mm_kernel(SkArgs g)
{
    using S = SkShape<W4, XR>;
    constexpr int TT = S::TT;
    __shared__ __attribute__((aligned(16))) uint8_t sh[S::RING + (W4 ? 32 * (SK_TABLE | 1) * 4 : 0)];
    uint32_t* table = reinterpret_cast<uint32_t*>(sh + S::RING);  // W4: [32 rows][ldt]

    const int e = sk_active_expert(g, blockIdx.y);
    if (e < 0) return;  // uniform
    const Segment seg = segment_of(g.offsets, e, g.M);
    const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid / WAVE);
    const int l16 = lane & 15, kg = lane >> 4;
    const int half = g.N / 2;
    // Weight row of tile row i (0..31), and its bound.
    const int n0 = blockIdx.x * (SWIGLU ? 16 : 32);
    auto wrow = [&](int i) {
        if constexpr (SWIGLU) {
            const int n = min(n0 + (i & 15), half - 1);
            return i < 16 ? n : half + n;
        } else {
            return min(n0 + i, g.N - 1);
        }
    };
    const int nchunks = (g.K + S::CK - 1) / S::CK;
    const T* zero16 = reinterpret_cast<const T*>(sk_zeros);
    const uint8_t* zero8 = reinterpret_cast<const uint8_t*>(sk_zeros);
    uint8_t* ring = sh + wave * SK_DEPTH * S::SLOT;

    // ---- weight sources.  W4: load i covers 8 rows of 128 bytes, 16-byte
    // piece p of row r lying at p ^ (r / 2 % 8); 16-bit: 4 rows of 256 bytes,
    // piece p at p ^ (r % 16): the 16 rows one fragment read touches then fall
    // on different banks.
    constexpr int WPR = S::WROW / 16, WRPL = 1024 / S::WROW;  // pieces per row, rows per load
    constexpr int XPR = S::XROW / 16, XRPL = 1024 / S::XROW;
    const uint8_t* wsrc[S::WL];
    int wk[S::WL];
#pragma unroll
    for (int i = 0; i < S::WL; ++i) {
        const int r = WRPL * i + lane / WPR;  // tile row 0..31
        const int p = (lane % WPR) ^ (W4 ? (r >> 1) & 7 : r & 15);
        const size_t row = (size_t)e * g.N + wrow(r);
        if constexpr (W4)
            wsrc[i] = static_cast<const uint8_t*>(g.w) + row * (g.K / 2) + 16 * p;
        else
            wsrc[i] = reinterpret_cast<const uint8_t*>(static_cast<const T*>(g.w) + row * g.K) + 16 * p;
        wk[i] = p * (W4 ? 32 : 8);
    }

    for (int s0 = seg.begin; s0 < seg.end; s0 += XR) {  // one pass over the weights per XR rows
        const T* xsrc[S::XL];
        int xk[S::XL], xlim[S::XL];
#pragma unroll
        for (int i = 0; i < S::XL; ++i) {
            const int r = XRPL * i + lane / XPR;
            const int p = (lane % XPR) ^ (r & 15);
            const int s = s0 + r;
            int row = s;
            bool ok = s < seg.end;
            if (ok && g.pairs) {
                row = g.pairs[s];
                ok = row >= 0;
                row /= g.k;
            }
            ok = ok && row < g.x_rows;
            xsrc[i] = static_cast<const T*>(g.x) + (ok ? (size_t)row * g.ldx : 0) + 8 * p;
            xk[i] = 8 * p;
            xlim[i] = ok ? g.K : 0;
        }
        auto issue = [&](int c, int slot) {  // chunk c; past the last one only zeros
            uint8_t* at = ring + slot * S::SLOT;
            const int k0 = c * S::CK;
#pragma unroll
            for (int i = 0; i < S::WL; ++i) {
                const uint8_t* src = wsrc[i] + (size_t)c * S::WROW;
                dma16(reinterpret_cast<const void*>(k0 + wk[i] < g.K ? reinterpret_cast<uintptr_t>(src)
                                                                     : reinterpret_cast<uintptr_t>(zero8)),
                      at + 1024 * i);
            }
#pragma unroll
            for (int i = 0; i < S::XL; ++i) {
                const T* src = xsrc[i] + k0;
                dma16(reinterpret_cast<const void*>(k0 + xk[i] < xlim[i] ? reinterpret_cast<uintptr_t>(src)
                                                                         : reinterpret_cast<uintptr_t>(zero16)),
                      at + S::WBYTES + 1024 * i);
            }
        };

        f32x4 acc[SK_NT][TT];
#pragma unroll
        for (int n = 0; n < SK_NT; ++n)
#pragma unroll
            for (int t = 0; t < TT; ++t) acc[n][t] = f32x4{0.f, 0.f, 0.f, 0.f};

        // x fragment: row (16 t + lane % 16) % XR, columns 32 j + 8 kg .. +7.
        auto x_frag = [&](const uint8_t* slot, int t, int j) {
            const int r = (16 * t + l16) & (XR - 1);
            return *reinterpret_cast<const u32x4*>(slot + S::WBYTES + r * S::XROW + (((4 * j + kg) ^ (r & 15)) << 4));
        };

        // Table super-blocks (W4): the scales of SK_TABLE groups at a time.
        const int G = W4 ? (g.K + g.group - 1) / g.group : 1;
        const int ldt = min(G, SK_TABLE) | 1;
        constexpr int CPS = W4 ? SK_TABLE * GB * 32 / S::CK : 0;  // chunks per super-block
        for (int cb = 0; cb < nchunks; cb += W4 ? CPS : nchunks) {
            const int ce = W4 ? min(cb + CPS, nchunks) : nchunks;
#pragma unroll
            for (int d = 0; d < SK_DEPTH; ++d) issue(cb + wave + SK_NW * d < ce ? cb + wave + SK_NW * d : nchunks, d);
            if constexpr (W4) {
                const int g0 = cb * S::CK / (32 * GB), gn = min(G - g0, SK_TABLE);
                for (int i = tid; i < 32 * gn; i += SK_THREADS) {
                    const int r = i / gn, q = i % gn;
                    const size_t at = ((size_t)e * g.N + wrow(r)) * G + g0 + q;
                    const uint32_t z = g.zeros ? g.zeros[at] & 15u : 8u;
                    table[r * ldt + q] = ((uint32_t) static_cast<const T*>(g.scales)[at].v << 16) | (16u + z);
                }
                __syncthreads();
            }
            int slot = 0;
            for (int c = cb + wave; c < ce; c += SK_NW) {
                dma_wait<(SK_DEPTH - 1) * (S::WL + S::XL)>();
                const uint8_t* at = ring + slot * S::SLOT;
                if constexpr (!W4) {
#pragma unroll
                    for (int j = 0; j < S::CK / 32; ++j) {
                        u32x4 a[TT];
#pragma unroll
                        for (int t = 0; t < TT; ++t) a[t] = x_frag(at, t, j);
#pragma unroll
                        for (int n = 0; n < SK_NT; ++n) {
                            const u32x4 b = *reinterpret_cast<const u32x4*>(at + (16 * n + l16) * S::WROW +
                                                                            (((4 * j + kg) ^ l16) << 4));
#pragma unroll
                            for (int t = 0; t < TT; ++t) acc[n][t] = mfma16_t(a[t], b, acc[n][t], T{});
                        }
                    }
                } else {
                    const u32x4 ones = u32x4{Code16<T>::one, Code16<T>::one, Code16<T>::one, Code16<T>::one};
#pragma unroll
                    for (int q = 0; q < 8 / GB; ++q) {  // the chunk's groups
                        f32x4 dsum[SK_NT][TT], xsum[TT];
#pragma unroll
                        for (int t = 0; t < TT; ++t) {
                            xsum[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                            for (int n = 0; n < SK_NT; ++n) dsum[n][t] = f32x4{0.f, 0.f, 0.f, 0.f};
                        }
#pragma unroll
                        for (int b = 0; b < GB; ++b) {
                            const int j = q * GB + b;
                            u32x4 a[TT];
#pragma unroll
                            for (int t = 0; t < TT; ++t) {
                                a[t] = pair_by_four(x_frag(at, t, j));
                                xsum[t] = mfma16_t(a[t], ones, xsum[t], T{});
                            }
#pragma unroll
                            for (int n = 0; n < SK_NT; ++n) {
                                const int r = 16 * n + l16;
                                const uint32_t w = *reinterpret_cast<const uint32_t*>(
                                    at + r * S::WROW + ((j ^ ((r >> 1) & 7)) << 4) + 4 * kg);
                                const u32x4 d = Code16<T>::decode(w);
#pragma unroll
                                for (int t = 0; t < TT; ++t) dsum[n][t] = mfma16_t(a[t], d, dsum[n][t], T{});
                            }
                        }
                        // a chunk's last groups may lie past K: their sums are 0 (x reads as zeros there)
                        const int gi = min(c * (8 / GB) + q, G - 1) - cb * (8 / GB);
#pragma unroll
                        for (int n = 0; n < SK_NT; ++n) {
                            const uint32_t sz = table[(16 * n + l16) * ldt + gi];
                            const float sc = to_f32(T{(uint16_t)(sz >> 16)}), z = (float)(sz & 0xFFu);
#pragma unroll
                            for (int t = 0; t < TT; ++t)
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    acc[n][t][i] = fmaf(sc, fmaf(-z, xsum[t][i], dsum[n][t][i]), acc[n][t][i]);
                        }
                    }
                }
                if constexpr (!W4) mfma_drain();
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // this slot's reads are done
                const int next = c + SK_NW * SK_DEPTH;
                issue(next < ce ? next : nchunks, slot);
                slot = slot + 1 == SK_DEPTH ? 0 : slot + 1;
            }
            dma_wait<0>();
            __syncthreads();  // the table and the ring are free
        }

        // ---- add up the waves' partial sums (in wave order) and store
        f32x4* red = reinterpret_cast<f32x4*>(sh);  // [wave][nt][tt][lane]
#pragma unroll
        for (int n = 0; n < SK_NT; ++n)
#pragma unroll
            for (int t = 0; t < TT; ++t) red[((wave * SK_NT + n) * TT + t) * WAVE + lane] = acc[n][t];
        __syncthreads();
        const T* bias = g.bias ? static_cast<const T*>(g.bias) + (size_t)e * g.N : nullptr;
        auto total = [&](int n, int t) {
            f32x4 v = red[(n * TT + t) * WAVE + lane];
#pragma unroll
            for (int w = 1; w < SK_NW; ++w) v += red[((w * SK_NT + n) * TT + t) * WAVE + lane];
            return v;
        };
        for (int u = wave; u < (SWIGLU ? 1 : SK_NT) * TT; u += SK_NW) {
            const int n = u / TT, t = u % TT;
            const int col = n0 + 16 * n + l16;
            if (col >= (SWIGLU ? half : g.N)) continue;
            f32x4 v = total(n, t);
            const float b = bias ? to_f32(bias[col]) : 0.f;
            if constexpr (SWIGLU) {
                const f32x4 up = total(1, t);
                const float bu = bias ? to_f32(bias[half + col]) : 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = silu(v[i] + b) * (up[i] + bu);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] += b;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 16 * t + 4 * kg + i, s = s0 + r;
                if (r < XR && s < seg.end) static_cast<O*>(g.out)[(size_t)s * g.ldo + col] = from_f32<O>(v[i]);
            }
        }
        __syncthreads();
    }
}

template <typename T, typename O, bool W4, int GB, bool SWIGLU, int XR>
hipError_t launch_one(const SkArgs& g, hipStream_t s)
{
    const int cols = SWIGLU ? g.N / 2 : g.N, per = SWIGLU ? 16 : 32;
    const dim3 grid((cols + per - 1) / per, g.offsets ? (g.E < g.M ? g.E : g.M) : 1);
    hipLaunchKernelGGL((skinny_mm_kernel<T, O, W4, GB, SWIGLU, XR>), grid, dim3(SK_THREADS), 0, s, g);
    return hipGetLastError();
}

// Rows of x per pass: twice an expert's average share (its share varies), so
// that a second pass over the weights is rare, in the smallest form that holds
// them; a wider form costs LDS space, and with it loads in flight.
template <typename T, typename O, bool W4, int GB, bool SWIGLU>
hipError_t launch_rows(const SkArgs& g, hipStream_t s)
{
    const int want = g.E == 1 ? g.M : 2 * ((g.M + g.E - 1) / g.E);
    if (want <= 4) return launch_one<T, O, W4, GB, SWIGLU, 4>(g, s);
    if (want <= 8) return launch_one<T, O, W4, GB, SWIGLU, 8>(g, s);
    if constexpr (W4) {
        return launch_one<T, O, W4, GB, SWIGLU, 16>(g, s);
    } else {
        if (want <= 16) return launch_one<T, O, W4, GB, SWIGLU, 16>(g, s);
        return launch_one<T, O, W4, GB, SWIGLU, 32>(g, s);
    }
}

template <typename T, typename O>
hipError_t launch_w4(const W4Args& a, const SkArgs& g, hipStream_t s)
{
    switch (a.group) {
    case 32: return a.swiglu ? launch_rows<T, O, true, 1, true>(g, s) : launch_rows<T, O, true, 1, false>(g, s);
    case 64: return a.swiglu ? launch_rows<T, O, true, 2, true>(g, s) : launch_rows<T, O, true, 2, false>(g, s);
    default: return a.swiglu ? launch_rows<T, O, true, 4, true>(g, s) : launch_rows<T, O, true, 4, false>(g, s);
    }
}

}  // namespace

bool gmm_use_skinny(const GmmArgs& a)
{
    return a.M <= 64 && a.K % 8 == 0 && a.lda % 8 == 0 && ((uintptr_t)a.a & 15) == 0 && ((uintptr_t)a.b & 15) == 0;
}

hipError_t launch_gmm_skinny(const GmmArgs& a, hipStream_t s)
{
    SkArgs g;
    memset(&g, 0, sizeof g);
    g.M = a.M;
    g.N = a.N;
    g.K = a.K;
    g.E = a.E;
    g.x_rows = a.a_rows;
    g.k = a.k;
    g.ldx = a.lda;
    g.ldo = a.ldc;
    g.offsets = a.offsets;
    g.pairs = a.pairs;
    g.x = a.a;
    g.w = a.b;
    g.bias = a.bias;
    g.out = a.out;
    if (a.dtype == DT_BF16)
        return a.out_dtype == DT_F32 ? launch_rows<bf16_t, float, false, 1, false>(g, s)
                                     : launch_rows<bf16_t, bf16_t, false, 1, false>(g, s);
    return a.out_dtype == DT_F32 ? launch_rows<f16_t, float, false, 1, false>(g, s)
                                 : launch_rows<f16_t, f16_t, false, 1, false>(g, s);
}

hipError_t launch_w4_matvec(const W4Args& a, hipStream_t s)
{
    SkArgs g;
    memset(&g, 0, sizeof g);
    g.M = a.M;
    g.N = a.N;
    g.K = a.K;
    g.E = a.E;
    g.x_rows = a.x_rows;
    g.k = a.k;
    g.ldx = a.K;
    g.ldo = a.swiglu ? a.N / 2 : a.N;
    g.group = a.group;
    g.offsets = a.offsets;
    g.pairs = a.pairs;
    g.x = a.x;
    g.w = a.codes;
    g.scales = a.scales;
    g.zeros = a.zeros;
    g.bias = a.bias;
    g.out = a.out;
    if (a.dtype == DT_BF16)
        return a.out_dtype == DT_F32 ? launch_w4<bf16_t, float>(a, g, s) : launch_w4<bf16_t, bf16_t>(a, g, s);
    return a.out_dtype == DT_F32 ? launch_w4<f16_t, float>(a, g, s) : launch_w4<f16_t, f16_t>(a, g, s);
}

}  // namespace moe
