// Host-side launchers of the stand-alone operators (grouped products, 4-bit
// products, block norms).  Each returns the hipError_t of its launches;
// arguments are validated by the entry points (ops_api.hip) before any of
// these run.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

enum { DT_BF16 = 0, DT_F16 = 1, DT_F32 = 2 };  // MOE_DT_* of moe.h

// ------------------------------------------------------------------ grouped products
// One product of the grouped kernels.  Row s of expert e's segment
// [offsets[e], offsets[e+1]) (clamped to [0, M]; offsets null: one segment of
// M rows) is row pairs[s] / k of `a` (pairs null: row s), which has a_rows rows.
struct GmmArgs {
    int M, N, K, E;
    int a_rows, k;
    int dtype, out_dtype;
    int accumulate;             // weight gradient: add to what db and dbias hold
    long long lda, ldc;         // row strides of a / da and of c / dc, in elements
    const int32_t* offsets;
    const int32_t* pairs;
    const void* a;
    const void* b;              // [E][N][K]
    const void* bias;           // [E][N] or null
    const void* dc;
    void* out;                  // c, da or db
    float* dbias;               // [E][N] or null
    float* part;                // weight gradient: partial sums (null: unsplit)
    float* dbias_part;
    int splits;                 // weight gradient: row ranges per expert
};

hipError_t launch_gmm_forward(const GmmArgs& a, hipStream_t s);
hipError_t launch_gmm_dgrad(const GmmArgs& a, hipStream_t s);
hipError_t launch_gmm_wgrad(const GmmArgs& a, hipStream_t s);
// The decode form of the forward product (weights streamed once).
hipError_t launch_gmm_skinny(const GmmArgs& a, hipStream_t s);
bool gmm_use_skinny(const GmmArgs& a);
// Row ranges that the weight gradient cuts each segment into, and that the bias
// gradient cuts all of them into (at most).
int gmm_wgrad_splits(int M, int N, int K, int E);
int gmm_dbias_ranges(int M, int E);
// n 16-bit zeros at p (null or n <= 0: nothing).  A kernel, not a memset, so
// that it may be captured into a graph.
hipError_t launch_zero16(void* p, int64_t n, hipStream_t s);

// ------------------------------------------------------------------ 4-bit products
struct W4Args {
    int M, N, K, E;
    int x_rows, k;
    int group;                  // 32, 64 or 128
    int dtype, out_dtype;
    int swiglu;
    const int32_t* offsets;
    const int32_t* pairs;
    const void* x;              // [x_rows][K]
    const uint8_t* codes;       // [E][N][K/2]
    const void* scales;         // [E][N][ceil(K/group)]
    const uint8_t* zeros;       // same shape, or null (8)
    const void* bias;           // [E][N] or null
    void* out;                  // [M][N] or [M][N/2]
};
hipError_t launch_w4_matvec(const W4Args& a, hipStream_t s);

// ------------------------------------------------------------------ block norms
struct NormArgs {
    int T, H;
    int dtype, wdtype;
    int kind;                   // 0 none, 1 RMS, 2 layer
    int gate_kind;              // 0 none, 1 [H], 2 [T], 3 [T][H]
    float eps, res_scale;
    uint32_t drop_threshold;    // keep an element when its 16 random bits >= this; 0: no dropout
    float drop_scale;           // 1 / keep probability
    const void* x;              // the normalised rows
    const void* res;            // forward: residual; backward of the norm before: the residual's gradient (or null)
    const void* weight;
    const void* bias;
    const void* gate;
    const uint64_t* rng;        // {seed, offset}
    void* out;
    // backward
    const void* dout;
    void* dx;
    float* dweight;
    float* dbias;
    void* dgate;
    float* part;                // [blocks][quantities][H]
};
hipError_t launch_norm_in(const NormArgs& a, hipStream_t s);
hipError_t launch_norm_out(const NormArgs& a, hipStream_t s);
hipError_t launch_norm_in_backward(const NormArgs& a, hipStream_t s);
hipError_t launch_norm_out_backward(const NormArgs& a, hipStream_t s);
constexpr int NORM_MAX_H = 16384;  // 512 threads x 4 vectors of 8
// Floats of the partial sums of the weight, bias and channel-gate gradients.
size_t norm_partial_floats(int T, int H);

}  // namespace moe
