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
// NV vectors of 8 columns per thread) walks over the rows, R at a time, so
// that several rows' loads are in flight and one exchange through LDS serves
// R rows.  A thread's columns never change: their parameters and the sums for
// dw, db and dgate stay in its registers, in fp32.  The workgroups' sums go to
// `part` and a second kernel adds them in order: the result does not depend on
// timing.  (With a row per wave, 6 vectors a thread at 2880 columns, those
// sums alone took 144 registers and spilled.)  HBM bound: 3 rows moved per row.
#pragma once

#include <type_traits>

#include "norm_device.h"

namespace moe {

// Second pass: the workgroups' sums to dweight, dbias and the channel gate's gradient.
hipError_t launch_norm_reduce(const float* part, int blocks, int Q, int H, float* o0, float* o1, float* o2,
                              hipStream_t s);

namespace {

constexpr int NB_MAX_WAVES = 8;
constexpr int NB_ROWS = 4;  // rows x vectors per thread of one step

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
inline int nb_blocks(int T, int H)
{
    const int rows = NB_ROWS / nb_nv(H), need = (T + rows - 1) / rows;
    const int most = 2048 / nb_waves(H) < 1024 ? 2048 / nb_waves(H) : 1024;
    return need < most ? need : most;
}

// B: sums of dn (the bias gradient) are wanted; G: the channel gate's are.
template <typename T, int NV, bool OUT, bool B, bool G>
__global__ __launch_bounds__(NB_MAX_WAVES* WAVE) void norm_bwd_kernel(NormArgs a)
{
    constexpr int R = NB_ROWS / NV, NS = OUT ? 5 : 3;
    __shared__ float lds[NB_MAX_WAVES * R * NS];
    const int nw = blockDim.x / WAVE, stride = blockDim.x, v0 = threadIdx.x, wave = threadIdx.x / WAVE, H = a.H;
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
    // N sums per row of the step over the workgroup, waves added in order.
    auto block_sums = [&](auto& s, auto n_c) {
        constexpr int N = decltype(n_c)::value;
#pragma unroll
        for (int q = 0; q < R; ++q)
#pragma unroll
            for (int k = 0; k < N; ++k) s[q][k] = wave_sum(s[q][k]);
        if (nw == 1) return;  // uniform
        __syncthreads();      // the previous sums have been read
        if (lane_id() == 0) {
#pragma unroll
            for (int q = 0; q < R; ++q)
#pragma unroll
                for (int k = 0; k < N; ++k) lds[(wave * R + q) * N + k] = s[q][k];
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < R; ++q)
#pragma unroll
            for (int k = 0; k < N; ++k) {
                float v = lds[q * N + k];
                for (int u = 1; u < nw; ++u) v += lds[(u * R + q) * N + k];
                s[q][k] = v;
            }
    };

    for (int t0 = blockIdx.x * R; t0 < a.T; t0 += gridDim.x * R) {
        Vec8<T> x[R][NV], d[R][NV], e[R][NV];  // e: norm_in: dres; norm_out: a full gate
        float g_row[R];
        const T* er = full ? gate : !OUT ? static_cast<const T*>(a.res) : nullptr;
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const int t = min(t0 + q, a.T - 1);  // past the last row: read it again, write nothing
            const size_t at = (size_t)t * H;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = v0 + stride * i;
                x[q][i] = d[q][i] = e[q][i] = Vec8<T>{};
                if (8 * v + 8 <= H) {
                    x[q][i] = load_full8(static_cast<const T*>(a.x) + at + 8 * v);
                    d[q][i] = load_full8(static_cast<const T*>(a.dout) + at + 8 * v);
                    if (er) e[q][i] = load_full8(er + at + 8 * v);
                } else if (8 * v < H) {
                    x[q][i] = load_tail8(static_cast<const T*>(a.x) + at, 8 * v, H);
                    d[q][i] = load_tail8(static_cast<const T*>(a.dout) + at, 8 * v, H);
                    if (er) e[q][i] = load_tail8(er + at, 8 * v, H);
                }
            }
            g_row[q] = OUT && a.gate_kind == NG_TOKEN ? to_f32(gate[t]) : 1.f;
        }
        uint32_t keep[R][NV];
#pragma unroll
        for (int q = 0; q < R; ++q)
#pragma unroll
            for (int i = 0; i < NV; ++i)
                keep[q][i] = OUT && a.drop_threshold
                                 ? dropout_keep8(v0 + stride * i, t0 + q, seed, offset, a.drop_threshold)
                                 : 255u;
        // dout with the dropout's mask and scale, and the gate
        auto dropped = [&](int q, int i, int j) {
            const float v = d[q][i].get(j);
            if constexpr (!OUT) return v;
            return keep[q][i] >> j & 1u ? v * a.drop_scale : 0.f;
        };
        auto gate_of = [&](int q, int i, int j) {
            if constexpr (!OUT) return 1.f;
            return full ? e[q][i].get(j) : g_row[q] * gc[OUT ? i : 0][j];
        };
        auto centred = [&](int q, int i, int j, float mean) {
            return 8 * (v0 + stride * i) + j < H ? x[q][i].get(j) - mean : 0.f;
        };
        float mean[R];
#pragma unroll
        for (int q = 0; q < R; ++q) mean[q] = 0.f;
        if (a.kind == NK_LAYER) {
            float s[R][1];
#pragma unroll
            for (int q = 0; q < R; ++q) {
                s[q][0] = 0.f;
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) s[q][0] += x[q][i].get(j);
            }
            block_sums(s, std::integral_constant<int, 1>{});
#pragma unroll
            for (int q = 0; q < R; ++q) mean[q] = s[q][0] * inv_h;
        }
        // One round of sums with c = x - mean, before r is known: c^2, t c, t,
        // and for the gate dk c w and dk b (dk = dout with the dropout).
        float s[R][NS];
#pragma unroll
        for (int q = 0; q < R; ++q) {
#pragma unroll
            for (int k = 0; k < NS; ++k) s[q][k] = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float c = centred(q, i, j, mean[q]), dk = dropped(q, i, j);
                    const float t1 = dk * gate_of(q, i, j) * w[i][j];
                    s[q][0] = fmaf(c, c, s[q][0]);
                    s[q][1] = fmaf(t1, c, s[q][1]);
                    s[q][2] += t1;
                    if constexpr (OUT) {
                        s[q][3] = fmaf(dk * w[i][j], c, s[q][3]);
                        s[q][4] = fmaf(dk, b[i][j], s[q][4]);
                    }
                }
        }
        block_sums(s, std::integral_constant<int, NS>{});
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const int t = t0 + q;
            if (t >= a.T) break;  // uniform
            const size_t at = (size_t)t * H;
            const float r = a.kind == NK_NONE ? 1.f : 1.f / sqrtf(s[q][0] * inv_h + a.eps);
            if constexpr (OUT) {
                if (a.gate_kind == NG_TOKEN && a.dgate && v0 == 0)
                    static_cast<float*>(a.dgate)[t] = fmaf(r, s[q][3], s[q][4]);
            }
            const float m1 = a.kind == NK_NONE ? 0.f : r * s[q][1] * inv_h;  // mean of t xh
            const float m2 = a.kind == NK_LAYER ? s[q][2] * inv_h : 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = v0 + stride * i;
                if (8 * v >= H) continue;
                float o[8], dg[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float xh = centred(q, i, j, mean[q]) * r;
                    const float dk = dropped(q, i, j), dn = dk * gate_of(q, i, j);
                    o[j] = a.kind == NK_NONE ? dn : r * (fmaf(dn, w[i][j], -m2) - xh * m1);
                    aw[i][j] = fmaf(dn, xh, aw[i][j]);
                    if (B) ab[B ? i : 0][j] += dn;
                    if constexpr (OUT) {  // a dropped element has no part in the gate's gradient, whatever it was
                        dg[j] = keep[q][i] >> j & 1u ? dk * fmaf(xh, w[i][j], b[i][j]) : 0.f;
                        if (G) ag[G ? i : 0][j] += dg[j];
                    } else {
                        o[j] = fmaf(a.res_scale, e[q][i].get(j), o[j]);  // e is 0 without dres
                    }
                }
                if constexpr (OUT) {
                    if (full && a.dgate) store_vec8(static_cast<T*>(a.dgate) + at, v, H, dg);
                }
                store_vec8(static_cast<T*>(a.dx) + at, v, H, o);
            }
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

template <typename T, bool OUT, bool B, bool G>
hipError_t launch_flags(const NormArgs& a, hipStream_t s)
{
    const int blocks = nb_blocks(a.T, a.H);
    const dim3 grid(blocks), threads(nb_waves(a.H) * WAVE);
    switch (nb_nv(a.H)) {
    case 1: hipLaunchKernelGGL((norm_bwd_kernel<T, 1, OUT, B, G>), grid, threads, 0, s, a); break;
    case 2: hipLaunchKernelGGL((norm_bwd_kernel<T, 2, OUT, B, G>), grid, threads, 0, s, a); break;
    default: hipLaunchKernelGGL((norm_bwd_kernel<T, 4, OUT, B, G>), grid, threads, 0, s, a); break;
    }
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess || (!a.dweight && !B && !G)) return err;
    float* dg = static_cast<float*>(a.dgate);
    return launch_norm_reduce(a.part, blocks, 1 + B + G, a.H, a.dweight, B ? a.dbias : dg, dg, s);
}

template <typename T, bool OUT>
hipError_t launch_type(const NormArgs& a, hipStream_t s)
{
    if constexpr (OUT) {
        if (a.gate_kind == NG_CHANNEL && a.dgate)
            return a.dbias ? launch_flags<T, OUT, true, true>(a, s) : launch_flags<T, OUT, false, true>(a, s);
    }
    return a.dbias ? launch_flags<T, OUT, true, false>(a, s) : launch_flags<T, OUT, false, false>(a, s);
}

}  // namespace

}  // namespace moe
