// Drives the entry points of the stand-alone operators (ops_api.hip, compiled
// as plain C++) with extreme and mixed-up descriptors against stand-ins of the
// kernel launchers, under AddressSanitizer and UndefinedBehaviorSanitizer on
// the host (test infrastructure).  The pointers are never followed: the
// stand-ins check only that what reaches a launcher is within the documented
// limits and within the workspace.  Prints "ok" and exits 0 on success.
#include <stdint.h>
#include <stdio.h>

#include "moe.h"
#include "moe_ops.h"

namespace {
long long launches = 0;
int failures = 0;
void expect(bool ok, const char* what)
{
    if (!ok && ++failures < 20) fprintf(stderr, "%s\n", what);
}
hipError_t gmm_ok(const moe::GmmArgs& a)
{
    ++launches;
    expect(a.M > 0 && a.N > 0 && a.K > 0 && a.E > 0 && a.E <= 256 && a.k >= 1 && a.k <= 8, "sizes of a product");
    expect(a.lda >= a.K && a.ldc >= a.N, "strides of a product");
    // tiles of 128 x 64, 256 threads each: fewer than 2^32 threads
    const long long wide = (a.N > a.K ? a.N : a.K) / 128 + 1;
    expect(wide * (a.M / 64 + a.E + 1) * 256 < (1ll << 32), "grid of a product");
    return hipSuccess;
}
hipError_t norm_ok(const moe::NormArgs& a)
{
    ++launches;
    expect(a.T >= 0 && a.H > 0 && a.H <= moe::NORM_MAX_H, "sizes of a norm");
    expect(a.drop_threshold < 65536 && a.drop_scale >= 1.f, "dropout");
    return hipSuccess;
}
}  // namespace

namespace moe {
void set_last_error(const char*) {}
hipError_t launch_gmm_forward(const GmmArgs& a, hipStream_t) { return gmm_ok(a); }
hipError_t launch_gmm_dgrad(const GmmArgs& a, hipStream_t) { return gmm_ok(a); }
hipError_t launch_gmm_wgrad(const GmmArgs& a, hipStream_t) { return gmm_ok(a); }
hipError_t launch_gmm_skinny(const GmmArgs& a, hipStream_t) { return gmm_ok(a); }
bool gmm_use_skinny(const GmmArgs& a) { return a.M <= 64; }
int gmm_wgrad_splits(int M, int, int, int E) { return M / E / 1024 > 64 ? 64 : M / E / 1024 < 1 ? 1 : M / E / 1024; }
int gmm_dbias_ranges(int M, int E) { return M / 128 + E; }
hipError_t launch_zero16(void*, int64_t n, hipStream_t)
{
    ++launches;
    expect(n >= 0, "zeros");
    return hipSuccess;
}
hipError_t launch_w4_matvec(const W4Args& a, hipStream_t)
{
    ++launches;
    expect(a.M > 0 && a.K % 32 == 0, "sizes of a 4-bit product");
    const long long rows = a.M <= 4 * a.E ? 4 : 16;
    expect(a.E * ((a.M + rows - 1) / rows) * ((a.N + 31) / 32 + 1ll) < (1ll << 31), "items of a 4-bit product");
    return hipSuccess;
}
hipError_t launch_norm_in(const NormArgs& a, hipStream_t) { return norm_ok(a); }
hipError_t launch_norm_out(const NormArgs& a, hipStream_t) { return norm_ok(a); }
hipError_t launch_norm_in_backward(const NormArgs& a, hipStream_t) { return norm_ok(a); }
hipError_t launch_norm_out_backward(const NormArgs& a, hipStream_t) { return norm_ok(a); }
size_t norm_partial_floats(int T, int H) { return (size_t)(T < 1024 ? T : 1024) * 3 * H; }
}  // namespace moe

namespace {
uint64_t state = 0x1234567;
uint32_t draw()
{
    state = state * 6364136223846793005ull + 1442695040888963407ull;
    return (uint32_t)(state >> 33);
}
const int32_t SIZES[] = {INT32_MIN, -1, 0, 1, 2, 3, 8, 32, 63, 64, 96, 256, 257, 2880, 5760, 1 << 20, 1 << 22, (1 << 22) + 1, INT32_MAX};
const int32_t SMALL[] = {-1, 0, 1, 2, 3, 4, 8, 9, 32, 64, 128};
const int64_t STRIDES[] = {0, 0, 0, -1, 8, 2880, 5761, 1ll << 31, (1ll << 31) + 1, INT64_MAX, INT64_MIN};
const float FLOATS[] = {0.f, 1e-5f, 1.f, -1.f, 0.1f, 0.999f, 0.99999f, 1e30f, __builtin_inff(), -__builtin_inff(), __builtin_nanf("")};
template <typename V, size_t n>
V pick(const V (&v)[n])
{
    return v[draw() % n];
}
const void* any_pointer()
{
    static const uintptr_t P[] = {4096, 4096, 4096, 4096, 0, 4097, 4098, 4100, 4104};
    return reinterpret_cast<const void*>(pick(P));
}
// A rejected call launches nothing.
void call(int rc, long long before, const char* what)
{
    expect(rc == MOE_OK || launches == before, what);
}
}  // namespace

extern "C" const char* hipGetErrorString(hipError_t) { return "stand-in"; }

int main()
{
    for (int i = 0; i < 400000; ++i) {
        const void *a = any_pointer(), *b = any_pointer(), *c = any_pointer(), *d = any_pointer(), *e = any_pointer();
        void *o = const_cast<void*>(any_pointer()), *w = const_cast<void*>(any_pointer());
        float *f0 = (float*)any_pointer(), *f1 = (float*)any_pointer();
        const int32_t *off = (const int32_t*)any_pointer(), *pairs = (const int32_t*)any_pointer();
        const size_t bytes = draw() % 2 ? SIZE_MAX : draw();
        moe_gmm g = {pick(SIZES), pick(SIZES), pick(SIZES), pick(SMALL), pick(SIZES), pick(SMALL),
                     (int32_t)(draw() % 4), (int32_t)(draw() % 4), (int32_t)(draw() % 3), 0, pick(STRIDES), pick(STRIDES)};
        if (draw() % 8 == 0) g.E = 256;
        if (draw() % 2) g.out_dtype = draw() % 2 ? g.dtype : (int)MOE_DT_F32;
        size_t n = 0;
        long long before = launches;
        call(moe_grouped_mm_workspace_size(&g, draw() % 8 ? &n : nullptr), before, "workspace size");
        call(moe_grouped_mm(&g, a, off, pairs, b, c, o, nullptr), before, "grouped_mm");
        before = launches;
        call(moe_grouped_mm_dgrad(&g, a, off, b, o, nullptr), before, "dgrad");
        before = launches;
        call(moe_grouped_mm_wgrad(&g, a, off, pairs, b, o, f0, w, bytes, nullptr), before, "wgrad");
        moe_w4 q = {g.M, g.N, g.K, g.E, g.T, g.k, pick(SMALL), g.dtype, g.out_dtype, (int32_t)(draw() % 3)};
        before = launches;
        call(moe_w4_matvec(&q, a, off, pairs, (const uint8_t*)b, c, (const uint8_t*)d, e, o, nullptr), before, "w4");
        moe_norm m = {pick(SIZES), pick(SIZES), (int32_t)(draw() % 4), (int32_t)(draw() % 4), (int32_t)(draw() % 5) - 1,
                      (int32_t)(draw() % 6) - 1, pick(FLOATS), pick(FLOATS), pick(FLOATS)};
        if (draw() % 2) m.wdtype = m.dtype;
        const uint64_t* rng = (const uint64_t*)any_pointer();
        before = launches;
        call(moe_norm_workspace_size(&m, &n), before, "norm workspace size");
        call(moe_norm_in(&m, a, b, c, o, nullptr), before, "norm_in");
        before = launches;
        call(moe_norm_out(&m, a, b, c, d, e, rng, o, nullptr), before, "norm_out");
        before = launches;
        call(moe_norm_in_backward(&m, a, b, c, d, o, f0, f1, w, bytes, nullptr), before, "norm_in_backward");
        before = launches;
        call(moe_norm_out_backward(&m, a, b, c, d, rng, e, o, f0, f1, w, o, bytes, nullptr), before, "norm_out_backward");
    }
    size_t n;
    expect(moe_grouped_mm(nullptr, 0, 0, 0, 0, 0, 0, 0) == MOE_ERR_INVALID_ARG, "null descriptor");
    expect(moe_w4_matvec(nullptr, 0, 0, 0, 0, 0, 0, 0, 0, 0) == MOE_ERR_INVALID_ARG, "null descriptor");
    expect(moe_norm_workspace_size(nullptr, &n) == MOE_ERR_INVALID_ARG, "null descriptor");
    expect(launches > 1000, "too few accepted calls");
    if (failures) return 1;
    puts("ok");
    return 0;
}
