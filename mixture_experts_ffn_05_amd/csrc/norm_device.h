// Device helpers of the block norms: rows as vectors of 8 columns held in
// registers, row sums, and the counter-based dropout.
#pragma once

#include <type_traits>

#include "elem16.h"
#include "moe_ops.h"

namespace moe {

// 8 neighbouring elements as stored.
template <typename T>
struct Vec8 {
    u32x4 w;
    __device__ __forceinline__ float get(int i) const
    {
        return i & 1 ? hi_f32<T>(w[i >> 1]) : lo_f32<T>(w[i >> 1]);
    }
};
template <>
struct Vec8<float> {
    u32x4 w, w2;
    __device__ __forceinline__ float get(int i) const { return __uint_as_float(i < 4 ? w[i & 3] : w2[i & 3]); }
};

// Elements first .. first+7 of a row of H, those past the row 0, one by one.
template <typename T>
__device__ __forceinline__ Vec8<T> load_tail8(const T* row, int first, int H)
{
    uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (first + i >= H) continue;
        if constexpr (sizeof(T) == 4)
            w[i] = __float_as_uint(row[first + i]);
        else
            w[i >> 1] |= (uint32_t)row[first + i].v << (16 * (i & 1));
    }
    Vec8<T> r;
    r.w = u32x4{w[0], w[1], w[2], w[3]};
    if constexpr (sizeof(T) == 4) r.w2 = u32x4{w[4], w[5], w[6], w[7]};
    return r;
}
template <typename T>
__device__ __forceinline__ Vec8<T> load_full8(const T* p)
{
    Vec8<T> r;
    r.w = load16_any(p);
    if constexpr (sizeof(T) == 4) r.w2 = load16_any(p + 4);
    return r;
}

// A thread's vectors v0, v0 + TPR, ... of a row of H elements (zeros past the
// row).  The row's last, partial vector is loaded once, apart from the loop.
template <int TPR, int NV, typename T>
__device__ __forceinline__ void load_row(const T* row, int v0, int H, Vec8<T> (&x)[NV])
{
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = v0 + TPR * i;
        x[i] = Vec8<T>{};
        if (8 * v + 8 <= H) x[i] = load_full8(row + 8 * v);
    }
    const int vt = H >> 3;
    if ((H & 7) && vt % TPR == v0) {
        const Vec8<T> tail = load_tail8(row, 8 * vt, H);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (v0 + TPR * i == vt) x[i] = tail;
    }
}

// The same for columns held as 8 floats per vector.
template <typename T>
__device__ __forceinline__ void store_full8(T* p, const float (&f)[8])
{
    if constexpr (sizeof(T) == 4) {
        store16_any(p, u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])});
        store16_any(p + 4,
                    u32x4{__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7])});
    } else {
        store16_any(p, u32x4{pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]), pack2<T>(f[6], f[7])});
    }
}
template <typename T>
__device__ __forceinline__ void store_vec8(T* row, int v, int H, const float (&f)[8])
{
    if (8 * v + 8 <= H) {
        store_full8(row + 8 * v, f);
        return;
    }
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (8 * v + i < H) row[8 * v + i] = from_f32<T>(f[i]);
}
template <typename T>
__device__ __forceinline__ Vec8<T> load_vec8(const T* row, int v, int H)
{
    return 8 * v + 8 <= H ? load_full8(row + 8 * v) : load_tail8(row, 8 * v, H);
}

// Weights, biases: fp32 or the activations' type (uniform per launch).
template <typename T>
__device__ __forceinline__ void load_param8(const void* p, bool f32, int v, int H, float (&f)[8])
{
    if (f32) {
        const Vec8<float> x = load_vec8(static_cast<const float*>(p), v, H);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = x.get(i);
    } else {
        const Vec8<T> x = load_vec8(static_cast<const T*>(p), v, H);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = x.get(i);
    }
}

// v of the lane that DPP control CTRL names.
template <int CTRL>
__device__ __forceinline__ float dpp(float v)
{
    return __uint_as_float(
        (uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ float lane_value(float v, int l)
{
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), l));
}

// Sums of N values over the 64 lanes in a fixed order, the same in every lane:
// within rows of 16 lanes by DPP (no LDS traffic; the values side by side, so
// that one's wait states are another's work), then the four rows' sums read as
// scalars.
template <int N>
__device__ __forceinline__ void wave_totals(float (&v)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += dpp<0xB1>(v[i]);  // quad_perm 1,0,3,2
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += dpp<0x4E>(v[i]);  // quad_perm 2,3,0,1
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += dpp<0x141>(v[i]);  // row_half_mirror
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += dpp<0x140>(v[i]);  // row_mirror
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = (lane_value(v[i], 0) + lane_value(v[i], 16)) + (lane_value(v[i], 32) + lane_value(v[i], 48));
}

// Sums of N values over the waves of a workgroup (NW <= 8; waves in order),
// after wave_totals: the waves leave theirs in LDS, [value][8 waves], and each
// group of 8 lanes adds one value's.
template <int N>
__device__ __forceinline__ void group_totals(float (&v)[N], int nw, float* lds)
{
    const int lane = lane_id(), wave = threadIdx.x / WAVE;
    __syncthreads();  // the previous sums have been read
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) lds[8 * i + wave] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; i += 8) {
        const int at = 8 * i + lane;
        float x = (lane & 7) < nw && at < 8 * N ? lds[at] : 0.f;
        x += dpp<0xB1>(x);
        x += dpp<0x4E>(x);
        x += dpp<0x141>(x);
#pragma unroll
        for (int k = 0; k < 8 && i + k < N; ++k) v[i + k] = lane_value(x, 8 * k);
    }
}

// Sums of N values over the TPR threads of a row (TPR 64: one wave; otherwise
// the whole workgroup).  Every thread gets the sums.
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* lds)
{
    wave_totals(v);
    if constexpr (TPR > WAVE) group_totals(v, TPR / WAVE, lds);
}

// Dropout's random bits: Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel
// random numbers: as easy as 1, 2, 3", 2011) at counter (column / 8, row,
// offset), key seed; 16 bits for each of the 8 columns, low halves first.
// keep[i]: column i is kept.
__device__ __forceinline__ void dropout_keep8(uint32_t v, uint32_t row, uint64_t seed, uint64_t offset,
                                              uint32_t threshold, bool (&keep)[8])
{
    uint32_t c0 = v, c1 = row, c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)b;
        c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    const uint32_t w[4] = {c0, c1, c2, c3};
#pragma unroll
    for (int i = 0; i < 8; ++i) keep[i] = (i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xFFFFu) >= threshold;
}

constexpr int NK_NONE = 0, NK_RMS = 1, NK_LAYER = 2;
constexpr int NG_NONE = 0, NG_CHANNEL = 1, NG_TOKEN = 2, NG_FULL = 3;

}  // namespace moe
