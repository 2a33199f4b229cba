// Norms around a block, backward.  The statistics are taken again from the
// rows, which the backward reads anyway: nothing but the inputs is kept from
// the forward, and the dropout mask is drawn again from its counters.
//
// With xh = (x - mean) r, n = xh w + b and dn the gradient of n (norm_in: dy;
// norm_out: dout * gate * keep / (1 - p)), t = dn w:
//   dx = r (t - xh mean(t xh) [- mean(t) for the layer norm])
//        (+ res_scale * dres for norm_in: the gradient that passes the block)
//   dw = sum over rows of dn xh,   db = sum of dn,
//   dgate = dout * keep / (1 - p) * n, summed over rows (a gate per channel)
//        or over columns (a gate per token), or as it is (a full gate).
//
// A workgroup of as many waves as a row has 512-column pieces (at most 8; then
// NV vectors of 8 columns per thread) walks over its rows, the next row's loads
// in flight while one is worked on.  A thread's columns never change: their
// parameters and the sums for dw, db and dgate stay in its registers, in fp32.
// The workgroups' sums go to `part` and a second kernel adds them in order: the
// result does not depend on timing.  (With a row per wave, 6 vectors a thread at
// 2880 columns, those sums alone took 144 registers and spilled; four rows at
// once needed over 200 and left one workgroup a CU: 197 us for the two kernels
// on 8192 x 2880 bf16, against 106 us with one row and two workgroups.)
// HBM bound: 3 rows moved per row (4 with dres).  8192 x 2880 bf16: norm_in with
// dres 35 us, 5.6 TB/s; norm_out with dropout and a channel gate 43 us, 3.6 TB/s,
// where drawing the mask again and the sums take as long; column sums 4 us each.
#pragma once

#include <type_traits>

#include "norm_device.h"

namespace moe {

// Second pass: the workgroups' sums to dweight, dbias and the channel gate's gradient.
hipError_t launch_norm_reduce(const float* part, int blocks, int Q, int H, float* o0, float* o1, float* o2,
                              hipStream_t s);

namespace {

constexpr int NB_MAX_WAVES = 8;
inline int nb_nv(int H)  // vectors per thread
{
    const int waves = (H + 511) / 512;
    return waves <= NB_MAX_WAVES ? 1 : waves <= 2 * NB_MAX_WAVES ? 2 : 4;
}
inline int nb_waves(int H)
{
    const int nv = nb_nv(H);
    return (H + 512 * nv - 1) / (512 * nv);
}
// Workgroups: two of 6 waves a CU (more of narrower ones), each with the same
// number of rows but for the last.  Half, this many and twice as many, in us:
// 8192 x 2880 bf16 RMS norm_in 51, 36 and 34, norm_out 59, 43 and 57; norm_in as a
// layer norm 46 and 49 (fp32 54 and 66) for this many and twice as many.
inline int nb_blocks(int T, int H)
{
    int most = 12 * 256 / nb_waves(H);
    most = most < 1024 ? most : 1024;
    const int rows = (T + most - 1) / most;
    return rows ? (T + rows - 1) / rows : 0;
}

// L: layer norm.  B: sums of dn (the bias gradient) are wanted; G: the channel
// gate's are.
template <typename T, int NV, bool OUT, bool L, bool B, bool G>
__global__ __launch_bounds__(NB_MAX_WAVES* WAVE, NV == 1 ? 4 : 2) void norm_bwd_kernel(NormArgs a)
{
    // Sums per row, with c = x - mean, taken in one round before r is known: c^2,
    // t c, t (layer norm), and for a token's gate dk c w and dk b.
    constexpr int S_T = 2, S_G = S_T + L, NS = S_G + (OUT && !G ? 2 : 0);
    __shared__ float lds[8 * NS];
    const int nw = blockDim.x / WAVE, stride = blockDim.x, v0 = threadIdx.x, H = a.H;
    const bool wf32 = a.wdtype == DT_F32, full = OUT && a.gate_kind == NG_FULL;
    const T* gate = static_cast<const T*>(a.gate);
    uint64_t seed = 0, offset = 0;
    if (OUT && a.drop_threshold) {
        seed = a.rng[0];
        offset = a.rng[1];
    }
    float w[NV][8], b[OUT ? NV : 1][8], gc[OUT ? NV : 1][8];
    float aw[NV][8], ab[B ? NV : 1][8], ag[G ? NV : 1][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = v0 + stride * i;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            w[i][j] = 1.f;
            aw[i][j] = 0.f;
            if (OUT) b[OUT ? i : 0][j] = 0.f, gc[OUT ? i : 0][j] = 1.f;
            if (B) ab[B ? i : 0][j] = 0.f;
            if (G) ag[G ? i : 0][j] = 0.f;
        }
        if (8 * v >= H) continue;
        if (a.weight) load_param8<T>(a.weight, wf32, v, H, w[i]);
        if (OUT && a.bias) load_param8<T>(a.bias, wf32, v, H, b[OUT ? i : 0]);
        if (OUT && a.gate_kind == NG_CHANNEL) load_param8<T>(gate, sizeof(T) == 4, v, H, gc[OUT ? i : 0]);
    }
    const float inv_h = 1.f / (float)H;
    // Sums over the workgroup.
    auto block_sums = [&](auto& s) {
        wave_totals(s);
        if (nw > 1) group_totals(s, nw, lds);
    };
    struct Row {
        Vec8<T> x[NV], d[NV], e[NV];  // e: norm_in: dres; norm_out: a full gate
        float g;                      // the token's gate
    };
    const T* er = full ? gate : !OUT ? static_cast<const T*>(a.res) : nullptr;
    auto load = [&](int t, Row& r) {
        const size_t at = (size_t)t * H;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = v0 + stride * i;
            r.x[i] = r.d[i] = r.e[i] = Vec8<T>{};
            if (8 * v + 8 <= H) {
                r.x[i] = load_full8(static_cast<const T*>(a.x) + at + 8 * v);
                r.d[i] = load_full8(static_cast<const T*>(a.dout) + at + 8 * v);
                if (er) r.e[i] = load_full8(er + at + 8 * v);
            } else if (8 * v < H) {
                r.x[i] = load_tail8(static_cast<const T*>(a.x) + at, 8 * v, H);
                r.d[i] = load_tail8(static_cast<const T*>(a.dout) + at, 8 * v, H);
                if (er) r.e[i] = load_tail8(er + at, 8 * v, H);
            }
        }
        r.g = OUT && a.gate_kind == NG_TOKEN ? to_f32(gate[t]) : 1.f;
    };

    Row cur, next;
    load(blockIdx.x, next);
    for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
        cur = next;
        if (t + (int)gridDim.x < a.T) load(t + gridDim.x, next);
        const size_t at = (size_t)t * H;
        bool keep[NV][8];
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) keep[i][j] = true;
        if (OUT && a.drop_threshold) {
#pragma unroll
            for (int i = 0; i < NV; ++i) dropout_keep8(v0 + stride * i, t, seed, offset, a.drop_threshold, keep[i]);
        }
        // dout with the dropout's mask and scale, and the gate
        auto dropped = [&](int i, int j) {
            const float v = cur.d[i].get(j);
            if constexpr (!OUT) return v;
            return keep[i][j] ? v * a.drop_scale : 0.f;
        };
        auto gate_of = [&](int i, int j) {
            if constexpr (!OUT) return 1.f;
            return full ? cur.e[i].get(j) : cur.g * gc[OUT ? i : 0][j];
        };
        float mean = 0.f;
        auto centred = [&](int i, int j) {  // x is 0 past the row
            if constexpr (!L) return cur.x[i].get(j);
            return 8 * (v0 + stride * i) + j < H ? cur.x[i].get(j) - mean : 0.f;
        };
        if constexpr (L) {
            float s[1] = {0.f};
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) s[0] += cur.x[i].get(j);
            block_sums(s);
            mean = s[0] * inv_h;
        }
        float s[NS];
#pragma unroll
        for (int k = 0; k < NS; ++k) s[k] = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float c = centred(i, j), dk = dropped(i, j);
                const float t1 = dk * gate_of(i, j) * w[i][j];
                s[0] = fmaf(c, c, s[0]);
                s[1] = fmaf(t1, c, s[1]);
                if constexpr (L) s[S_T] += t1;
                if constexpr (OUT && !G) {  // dk: dout with the dropout
                    s[S_G] = fmaf(dk * w[i][j], c, s[S_G]);
                    s[S_G + 1] = fmaf(dk, b[i][j], s[S_G + 1]);
                }
            }
        block_sums(s);
        const float r = a.kind == NK_NONE ? 1.f : 1.f / sqrtf(s[0] * inv_h + a.eps);
        if constexpr (OUT && !G) {
            if (a.gate_kind == NG_TOKEN && a.dgate && v0 == 0)
                static_cast<float*>(a.dgate)[t] = fmaf(r, s[S_G], s[S_G + 1]);
        }
        const float m1 = a.kind == NK_NONE ? 0.f : r * s[1] * inv_h;  // mean of t xh
        const float m2 = L ? s[S_T] * inv_h : 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = v0 + stride * i;
            if (8 * v >= H) continue;
            float o[8], dg[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float xh = centred(i, j) * r;
                const float dk = dropped(i, j), dn = dk * gate_of(i, j);
                o[j] = a.kind == NK_NONE ? dn : r * (fmaf(dn, w[i][j], -m2) - xh * m1);
                aw[i][j] = fmaf(dn, xh, aw[i][j]);
                if (B) ab[B ? i : 0][j] += dn;
                if constexpr (OUT) {  // a dropped element has no part in the gate's gradient, whatever it was
                    dg[j] = keep[i][j] ? dk * fmaf(xh, w[i][j], b[i][j]) : 0.f;
                    if (G) ag[G ? i : 0][j] += dg[j];
                } else {
                    o[j] = fmaf(a.res_scale, cur.e[i].get(j), o[j]);  // e is 0 without dres
                }
            }
            if constexpr (OUT) {
                if (full && a.dgate) store_vec8(static_cast<T*>(a.dgate) + at, v, H, dg);
            }
            store_vec8(static_cast<T*>(a.dx) + at, v, H, o);
        }
    }

    // ---- this workgroup's column sums -> part[block][quantity][H]
    float* part = a.part + (size_t)blockIdx.x * (1 + B + G) * H;
    auto emit = [&](int q, const float(*acc)[8]) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = v0 + stride * i;
            if (8 * v < H) store_vec8(part + (size_t)q * H, v, H, acc[i]);
        }
    };
    emit(0, aw);
    if constexpr (B) emit(1, ab);
    if constexpr (G) emit(1 + B, ag);
}

template <typename T, bool OUT, bool L, bool B, bool G>
hipError_t launch_flags(const NormArgs& a, hipStream_t s)
{
    const int blocks = nb_blocks(a.T, a.H);
    const dim3 grid(blocks), threads(nb_waves(a.H) * WAVE);
    switch (nb_nv(a.H)) {
    case 1: hipLaunchKernelGGL((norm_bwd_kernel<T, 1, OUT, L, B, G>), grid, threads, 0, s, a); break;
    case 2: hipLaunchKernelGGL((norm_bwd_kernel<T, 2, OUT, L, B, G>), grid, threads, 0, s, a); break;
    default: hipLaunchKernelGGL((norm_bwd_kernel<T, 4, OUT, L, B, G>), grid, threads, 0, s, a); break;
    }
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess || (!a.dweight && !B && !G)) return err;
    float* dg = static_cast<float*>(a.dgate);
    return launch_norm_reduce(a.part, blocks, 1 + B + G, a.H, a.dweight, B ? a.dbias : dg, dg, s);
}

template <typename T, bool OUT, bool L>
hipError_t launch_kind(const NormArgs& a, hipStream_t s)
{
    if constexpr (OUT) {
        if (a.gate_kind == NG_CHANNEL && a.dgate)
            return a.dbias ? launch_flags<T, OUT, L, true, true>(a, s) : launch_flags<T, OUT, L, false, true>(a, s);
    }
    return a.dbias ? launch_flags<T, OUT, L, true, false>(a, s) : launch_flags<T, OUT, L, false, false>(a, s);
}

template <typename T, bool OUT>
hipError_t launch_type(const NormArgs& a, hipStream_t s)
{
    return a.kind == NK_LAYER ? launch_kind<T, OUT, true>(a, s) : launch_kind<T, OUT, false>(a, s);
}

}  // namespace

}  // namespace moe
