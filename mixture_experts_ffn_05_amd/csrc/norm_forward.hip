// Norms around a block, forward.
//
//   norm_in   y = n(x) * w + b                       (before the block)
//   norm_out  o = res_scale * res + gate * drop(n(f) * w + b)   (after it)
// with n(x) = x / sqrt(mean(x^2) + eps) (RMS) or (x - mean) / sqrt(var + eps)
// (layer), statistics in fp32 from the values held in registers: every row is
// read once, whatever its kind (the layer norm's variance is the mean of the
// squared differences from the mean, a second pass over registers).  Bound by
// HBM: 2 rows moved per row of norm_in, 3 (4 with a full gate) of norm_out.  8192 x
// 2880 bf16: 20.6 and 30.2 us, 4.6 and 4.7 TB/s (a copy reaches 4.9).
//
// A row is held by one wave up to 2048 columns (no barrier, rows independent, 4
// of them in a workgroup), by 256 threads above, each thread keeping vectors of
// 8 columns (16 bytes), lanes adjacent.  norm_in with a wave and with 256 threads
// a row, bf16, in us: 8192 x 512 5.1 and 8.6, 8192 x 2048 12.4 and 14.1, 1024 x 2880
// 5.6 and 4.8, 8192 x 2880 19.6 and 19.1, 4096 x 4096 13.5 and 12.5.  Rows of odd
// length use unaligned vector accesses and an element loop in the last vector.
#include "norm_device.h"

namespace moe {

namespace {

template <typename T, int TPR, int NV, bool OUT>
__global__ __launch_bounds__(256) void norm_fwd_kernel(NormArgs a)
{
    __shared__ float lds[TPR > WAVE ? 8 : 1];
    constexpr int RPB = 256 / TPR;
    const int64_t row = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * RPB + (int)threadIdx.x / TPR;
    if (row >= a.T) return;  // uniform per wave; per block where a row spans waves
    const int t = (int)row;
    const int v0 = threadIdx.x % TPR, H = a.H;
    const size_t at = (size_t)t * H;
    const T* xr = static_cast<const T*>(a.x) + at;
    const T* rr = OUT && a.res ? static_cast<const T*>(a.res) + at : nullptr;
    const T* gate = static_cast<const T*>(a.gate);
    Vec8<T> x[NV], res[OUT ? NV : 1], gt[OUT ? NV : 1];
    const bool gate_vec = OUT && (a.gate_kind == NG_CHANNEL || a.gate_kind == NG_FULL);
    const T* gr = a.gate_kind == NG_FULL ? gate + at : gate;
    load_row<TPR>(xr, v0, H, x);
    if constexpr (OUT) {
        if (rr) load_row<TPR>(rr, v0, H, res);
        if (gate_vec) load_row<TPR>(gr, v0, H, gt);
    }
    const float g_row = OUT && a.gate_kind == NG_TOKEN ? to_f32(gate[t]) : 1.f;

    float mean = 0.f, r = 1.f;
    if (a.kind == NK_LAYER) {
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) s[0] += x[i].get(j);
        row_sums<TPR>(s, lds);
        mean = s[0] / (float)H;
    }
    if (a.kind != NK_NONE) {
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float d = 8 * (v0 + TPR * i) + j < H ? x[i].get(j) - mean : 0.f;
                s[0] = fmaf(d, d, s[0]);
            }
        row_sums<TPR>(s, lds);
        r = 1.f / sqrtf(s[0] / (float)H + a.eps);
    }

    const bool wf32 = a.wdtype == DT_F32;
    uint64_t seed = 0, offset = 0;
    if (OUT && a.drop_threshold) {
        seed = a.rng[0];
        offset = a.rng[1];
    }
    T* orow = static_cast<T*>(a.out) + at;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = v0 + TPR * i;
        if (8 * v >= H) continue;
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = (x[i].get(j) - mean) * r;
        if (a.weight) {
            float w[8];
            load_param8<T>(a.weight, wf32, v, H, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] *= w[j];
        }
        if (a.bias) {
            float b[8];
            load_param8<T>(a.bias, wf32, v, H, b);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] += b[j];
        }
        if constexpr (OUT) {
            if (a.drop_threshold) {  // a dropped element is 0, whatever it was
                bool keep[8];
                dropout_keep8(v, t, seed, offset, a.drop_threshold, keep);
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = keep[j] ? y[j] * a.drop_scale : 0.f;
            }
            if (gate_vec) {
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] *= gt[i].get(j);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] *= g_row;
            }
            if (rr) {
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = fmaf(a.res_scale, res[i].get(j), y[j]);
            }
        }
        store_vec8(orow, v, H, y);
    }
}

template <typename T, bool OUT>
hipError_t launch_type(const NormArgs& a, hipStream_t s)
{
    const int nv = (a.H + 7) / 8;
    constexpr unsigned most = 1u << 22;  // workgroups in x: fewer than 2^32 threads
#define MOE_NORM_LAUNCH(TPR, NV)                                                                          \
    if (nv <= (TPR) * (NV)) {                                                                             \
        constexpr int rpb = 256 / (TPR);                                                                  \
        const unsigned blocks = ((unsigned)a.T + rpb - 1) / rpb, x = blocks < most ? blocks : most;       \
        hipLaunchKernelGGL((norm_fwd_kernel<T, TPR, NV, OUT>), dim3(x, (blocks + x - 1) / x), dim3(256), 0, s, a); \
        return hipGetLastError();                                                                         \
    }
    MOE_NORM_LAUNCH(64, 1)
    MOE_NORM_LAUNCH(64, 2)
    MOE_NORM_LAUNCH(64, 4)
    MOE_NORM_LAUNCH(256, 2)
    MOE_NORM_LAUNCH(256, 4)
    MOE_NORM_LAUNCH(256, 8)
#undef MOE_NORM_LAUNCH
    return hipErrorInvalidValue;
}

template <bool OUT>
hipError_t launch_fwd(const NormArgs& a, hipStream_t s)
{
    return a.dtype == DT_BF16  ? launch_type<bf16_t, OUT>(a, s)
           : a.dtype == DT_F16 ? launch_type<f16_t, OUT>(a, s)
                               : launch_type<float, OUT>(a, s);
}

}  // namespace

hipError_t launch_norm_in(const NormArgs& a, hipStream_t s) { return launch_fwd<false>(a, s); }
hipError_t launch_norm_out(const NormArgs& a, hipStream_t s) { return launch_fwd<true>(a, s); }

}  // namespace moe
