// Grouped products of few rows with an expert's 16-bit matrix (decoding): the
// weights are the traffic, and every one is read once per pass over the rows.
//
// A workgroup owns 32 weight rows of one expert; its 4 waves split K in chunks
// and add up at the end.  Each wave runs its own ring of LDS slots filled by
// direct-to-LDS loads, so there is no barrier in the loop and several KB per
// wave are always in flight: a chunk's weights (256 bytes of each row: whole
// cache lines) and the same columns of up to XR rows of x.
// v_mfma_f32_16x16x32 takes x's rows as its A rows and weight rows as its B
// columns, so a lane's four results are four rows of x for one n.
// 16 tokens, 4 of 32 experts, 2880 -> 5760: 157 us for 937 MB, 6.0 TB/s (a pure
// read of the card reaches 6.15).
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

__device__ uint32_t sk_zeros[4] __attribute__((aligned(16)));  // never written

struct SkArgs {
    int M, N, K, E, x_rows, k;
    long long ldx, ldo;
    const int32_t* offsets;
    const int32_t* pairs;
    const void* x;
    const void* w;
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

template <int XR>
struct SkShape {
    static constexpr int CK = 128;         // columns per chunk
    static constexpr int ROWB = CK * 2;    // bytes of a row's chunk
    static constexpr int WBYTES = SK_NT * 16 * ROWB, XBYTES = XR * ROWB;
    static constexpr int SLOT = WBYTES + XBYTES;
    static constexpr int WL = WBYTES / 1024, XL = XBYTES / 1024;  // loads per wave and slot
    static constexpr int RING = SK_NW * SK_DEPTH * SLOT;
    static constexpr int TT = XR <= 16 ? 1 : XR / 16;  // 16-row tiles of x
    static_assert(XL >= 1 && (SK_DEPTH - 1) * (WL + XL) < 64, "load count");
    static_assert(SK_NW * SK_NT * TT * 1024 <= RING, "the reduction reuses the ring");
};

// XR: rows of x per pass.
template <typename T, typename O, int XR>
__global__ __launch_bounds__(SK_THREADS) void skinny_mm_kernel(SkArgs g)
{
    using S = SkShape<XR>;
    constexpr int TT = S::TT;
    __shared__ __attribute__((aligned(16))) uint8_t sh[S::RING];

    const int e = sk_active_expert(g, blockIdx.y);
    if (e < 0) return;  // uniform
    const Segment seg = segment_of(g.offsets, e, g.M);
    const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid / WAVE);
    const int l16 = lane & 15, kg = lane >> 4;
    const int n0 = blockIdx.x * 32;
    const int nchunks = (g.K + S::CK - 1) / S::CK;
    const uintptr_t zeros = reinterpret_cast<uintptr_t>(sk_zeros);
    uint8_t* ring = sh + wave * SK_DEPTH * S::SLOT;

    // ---- weight sources: load i covers 4 rows of 256 bytes, 16-byte piece p
    // of row r lying at p ^ (r % 16): the 16 rows that one fragment read touches
    // then fall on different banks.  Rows past N are read as the last one.
    const T* wsrc[S::WL];
    int wk[S::WL];
#pragma unroll
    for (int i = 0; i < S::WL; ++i) {
        const int r = 4 * i + (lane >> 4), p = l16 ^ (r & 15);
        wsrc[i] = static_cast<const T*>(g.w) + ((size_t)e * g.N + min(n0 + r, g.N - 1)) * g.K + 8 * p;
        wk[i] = 8 * p;
    }

    for (int s0 = seg.begin; s0 < seg.end; s0 += XR) {  // one pass over the weights per XR rows
        const T* xsrc[S::XL];
        int xlim[S::XL];
#pragma unroll
        for (int i = 0; i < S::XL; ++i) {
            const int r = 4 * i + (lane >> 4), p = l16 ^ (r & 15), s = s0 + r;
            int row = s;
            bool ok = s < seg.end;
            if (ok && g.pairs) {
                row = g.pairs[s];
                ok = row >= 0;
                row /= g.k;
            }
            ok = ok && row < g.x_rows;
            xsrc[i] = static_cast<const T*>(g.x) + (ok ? (size_t)row * g.ldx : 0) + 8 * p;
            xlim[i] = ok ? g.K - 8 * p : 0;
        }
        auto issue = [&](int c, int slot) {  // chunk c; past the last one only zeros
            uint8_t* at = ring + slot * S::SLOT;
            const int k0 = c * S::CK;
#pragma unroll
            for (int i = 0; i < S::WL; ++i)
                dma16(reinterpret_cast<const void*>(k0 + wk[i] < g.K ? reinterpret_cast<uintptr_t>(wsrc[i] + k0) : zeros),
                      at + 1024 * i);
#pragma unroll
            for (int i = 0; i < S::XL; ++i)
                dma16(reinterpret_cast<const void*>(k0 < xlim[i] ? reinterpret_cast<uintptr_t>(xsrc[i] + k0) : zeros),
                      at + S::WBYTES + 1024 * i);
        };

        f32x4 acc[SK_NT][TT];
#pragma unroll
        for (int n = 0; n < SK_NT; ++n)
#pragma unroll
            for (int t = 0; t < TT; ++t) acc[n][t] = f32x4{0.f, 0.f, 0.f, 0.f};

        // x fragment: row (16 t + lane % 16) % XR, columns 32 j + 8 kg .. +7.
        auto x_frag = [&](const uint8_t* slot, int t, int j) {
            const int r = (16 * t + l16) & (XR - 1);
            return *reinterpret_cast<const u32x4*>(slot + S::WBYTES + r * S::ROWB + (((4 * j + kg) ^ (r & 15)) << 4));
        };

#pragma unroll
        for (int d = 0; d < SK_DEPTH; ++d) issue(wave + SK_NW * d < nchunks ? wave + SK_NW * d : nchunks, d);
        int slot = 0;
        for (int c = wave; c < nchunks; c += SK_NW) {
            dma_wait<(SK_DEPTH - 1) * (S::WL + S::XL)>();
            const uint8_t* at = ring + slot * S::SLOT;
#pragma unroll
            for (int j = 0; j < S::CK / 32; ++j) {
                u32x4 a[TT];
#pragma unroll
                for (int t = 0; t < TT; ++t) a[t] = x_frag(at, t, j);
#pragma unroll
                for (int n = 0; n < SK_NT; ++n) {
                    const u32x4 b =
                        *reinterpret_cast<const u32x4*>(at + (16 * n + l16) * S::ROWB + (((4 * j + kg) ^ l16) << 4));
#pragma unroll
                    for (int t = 0; t < TT; ++t) acc[n][t] = mfma16_t(a[t], b, acc[n][t], T{});
                }
            }
            mfma_drain();
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // this slot's reads are done
            const int next = c + SK_NW * SK_DEPTH;
            issue(next < nchunks ? next : nchunks, slot);
            slot = slot + 1 == SK_DEPTH ? 0 : slot + 1;
        }
        dma_wait<0>();
        __syncthreads();  // the ring is free

        // ---- add up the waves' partial sums (in wave order) and store
        f32x4* red = reinterpret_cast<f32x4*>(sh);  // [wave][nt][tt][lane]
#pragma unroll
        for (int n = 0; n < SK_NT; ++n)
#pragma unroll
            for (int t = 0; t < TT; ++t) red[((wave * SK_NT + n) * TT + t) * WAVE + lane] = acc[n][t];
        __syncthreads();
        const T* bias = g.bias ? static_cast<const T*>(g.bias) + (size_t)e * g.N : nullptr;
        for (int u = wave; u < SK_NT * TT; u += SK_NW) {
            const int n = u / TT, t = u % TT;
            const int col = n0 + 16 * n + l16;
            if (col >= g.N) continue;
            f32x4 v = red[(n * TT + t) * WAVE + lane];
#pragma unroll
            for (int w = 1; w < SK_NW; ++w) v += red[((w * SK_NT + n) * TT + t) * WAVE + lane];
            const float b = bias ? to_f32(bias[col]) : 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 16 * t + 4 * kg + i, s = s0 + r;
                if (r < XR && s < seg.end) static_cast<O*>(g.out)[(size_t)s * g.ldo + col] = from_f32<O>(v[i] + b);
            }
        }
        __syncthreads();
    }
}

template <typename T, typename O, int XR>
hipError_t launch_one(const SkArgs& g, hipStream_t s)
{
    const dim3 grid((g.N + 31) / 32, g.offsets ? (g.E < g.M ? g.E : g.M) : 1);
    hipLaunchKernelGGL((skinny_mm_kernel<T, O, XR>), grid, dim3(SK_THREADS), 0, s, g);
    return hipGetLastError();
}

// Rows of x per pass: twice an expert's average share (its share varies), so
// that a second pass over the weights is rare, in the smallest form that holds
// them; a wider form costs LDS space, and with it loads in flight.  8 experts,
// 2880 -> 5760, in us: 2 rows each, 47 with 4, 58 with 16, 63 with 32; 8 rows each,
// 79 with 4, 60 with 16, 65 with 32.
template <typename T, typename O>
hipError_t launch_rows(const SkArgs& g, hipStream_t s)
{
    const int want = g.E == 1 ? g.M : 2 * ((g.M + g.E - 1) / g.E);
    if (want <= 4) return launch_one<T, O, 4>(g, s);
    if (want <= 8) return launch_one<T, O, 8>(g, s);
    if (want <= 16) return launch_one<T, O, 16>(g, s);
    return launch_one<T, O, 32>(g, s);
}

}  // namespace

// Few rows in all.  This kernel and the tiled one, in us: 1 expert, 2880 x 2880,
// 64 rows 16 and 24, 128 rows 28 and 24; 32 experts, 2880 -> 5760, 64 rows spread
// evenly 171 and 196, 96 rows spread unevenly (a second pass over the weights of
// the full experts) 111 and 107.
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
        return a.out_dtype == DT_F32 ? launch_rows<bf16_t, float>(g, s)
                                     : launch_rows<bf16_t, bf16_t>(g, s);
    return a.out_dtype == DT_F32 ? launch_rows<f16_t, float>(g, s)
                                 : launch_rows<f16_t, f16_t>(g, s);
}

}  // namespace moe
