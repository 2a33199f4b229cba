// Norms around a block, backward: the entry by type, and the sums over the
// workgroups (the kernels are in norm_backward.h, compiled per type).
#include "norm_backward.h"

namespace moe {

hipError_t launch_norm_in_backward_bf16(const NormArgs& a, hipStream_t s);
hipError_t launch_norm_in_backward_f16(const NormArgs& a, hipStream_t s);
hipError_t launch_norm_in_backward_f32(const NormArgs& a, hipStream_t s);
hipError_t launch_norm_out_backward_bf16(const NormArgs& a, hipStream_t s);
hipError_t launch_norm_out_backward_f16(const NormArgs& a, hipStream_t s);
hipError_t launch_norm_out_backward_f32(const NormArgs& a, hipStream_t s);

namespace {

// out[q][h] = sum over the workgroups of part[block][q][h]: 64 columns per
// workgroup, 16 groups of blocks summed side by side and then in order.
__global__ __launch_bounds__(1024) void norm_reduce_kernel(const float* __restrict__ part, int blocks, int Q, int H,
                                                          float* o0, float* o1, float* o2)
{
    __shared__ float sh[16][64];
    const int c = threadIdx.x & 63, grp = threadIdx.x >> 6;
    const int h = blockIdx.x * 64 + c, q = blockIdx.y;
    const int per = (blocks + 15) / 16, b0 = grp * per, b1 = min(b0 + per, blocks);
    float v = 0.f;
    if (h < H) {
        const float* p = part + (size_t)q * H + h;
        int b = b0;
        for (; b + 8 <= b1; b += 8) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = p[(size_t)(b + i) * Q * H];
#pragma unroll
            for (int i = 0; i < 8; ++i) v += x[i];
        }
        for (; b < b1; ++b) v += p[(size_t)b * Q * H];
    }
    sh[grp][c] = v;
    __syncthreads();
    if (grp == 0 && h < H) {
#pragma unroll
        for (int i = 1; i < 16; ++i) v += sh[i][c];
        float* o = q == 0 ? o0 : q == 1 ? o1 : o2;
        if (o) o[h] = v;
    }
}

}  // namespace

hipError_t launch_norm_reduce(const float* part, int blocks, int Q, int H, float* o0, float* o1, float* o2,
                              hipStream_t s)
{
    hipLaunchKernelGGL(norm_reduce_kernel, dim3((H + 63) / 64, Q), dim3(1024), 0, s, part, blocks, Q, H, o0, o1, o2);
    return hipGetLastError();
}

size_t norm_partial_floats(int T, int H) { return (size_t)nb_blocks(T, H) * 3 * H; }

hipError_t launch_norm_in_backward(const NormArgs& a, hipStream_t s)
{
    return a.dtype == DT_BF16  ? launch_norm_in_backward_bf16(a, s)
           : a.dtype == DT_F16 ? launch_norm_in_backward_f16(a, s)
                               : launch_norm_in_backward_f32(a, s);
}
hipError_t launch_norm_out_backward(const NormArgs& a, hipStream_t s)
{
    return a.dtype == DT_BF16  ? launch_norm_out_backward_bf16(a, s)
           : a.dtype == DT_F16 ? launch_norm_out_backward_f16(a, s)
                               : launch_norm_out_backward_f32(a, s);
}

}  // namespace moe
