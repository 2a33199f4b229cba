// 16- and 32-bit element types of the stand-alone operators: conversions,
// rounding and vector access that does not ask for alignment.
#pragma once

#include "moe_device.h"

namespace moe {

struct bf16_t {  // raw bfloat16
    uint16_t v;
};
struct f16_t {  // raw IEEE half
    uint16_t v;
};

typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;
typedef __attribute__((ext_vector_type(16))) float f32x16_t;

__device__ __forceinline__ float to_f32(bf16_t x) { return __uint_as_float((uint32_t)x.v << 16); }
__device__ __forceinline__ float to_f32(f16_t x) { return (float)__builtin_bit_cast(_Float16, x.v); }
__device__ __forceinline__ float to_f32(float x) { return x; }

// Round to nearest even.
template <typename T>
__device__ __forceinline__ T from_f32(float f);
template <>
__device__ __forceinline__ bf16_t from_f32<bf16_t>(float f)
{
    return bf16_t{__builtin_bit_cast(uint16_t, (__bf16)f)};
}
template <>
__device__ __forceinline__ f16_t from_f32<f16_t>(float f)
{
    return f16_t{__builtin_bit_cast(uint16_t, (_Float16)f)};
}
template <>
__device__ __forceinline__ float from_f32<float>(float f)
{
    return f;
}

// The value of the low / high half of a word of two 16-bit elements.
template <typename T>
__device__ __forceinline__ float lo_f32(uint32_t w)
{
    return to_f32(T{(uint16_t)w});
}
template <typename T>
__device__ __forceinline__ float hi_f32(uint32_t w)
{
    return to_f32(T{(uint16_t)(w >> 16)});
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    return (uint32_t)from_f32<T>(lo).v | ((uint32_t)from_f32<T>(hi).v << 16);
}
template <>
__device__ __forceinline__ uint32_t pack2<bf16_t>(float lo, float hi)  // one v_cvt_pk_bf16_f32
{
    typedef __attribute__((ext_vector_type(2))) float f32x2;
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
}

// 16 bytes at any element-aligned address: gfx950 serves unaligned vector
// accesses, so a row of odd length needs no element loop except in its tail.
struct __attribute__((packed, aligned(2))) raw16_t {
    u32x4 v;
};
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
struct __attribute__((packed, aligned(2))) raw8_t {
    u32x2 v;
};
__device__ __forceinline__ u32x4 load16_any(const void* p) { return static_cast<const raw16_t*>(p)->v; }
__device__ __forceinline__ void store16_any(void* p, u32x4 v) { static_cast<raw16_t*>(p)->v = v; }
__device__ __forceinline__ void store8_any(void* p, uint32_t x, uint32_t y) { static_cast<raw8_t*>(p)->v = u32x2{x, y}; }

__device__ __forceinline__ f32x16_t mfma32_t(u32x4 a, u32x4 b, f32x16_t c, bf16_t)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}
__device__ __forceinline__ f32x16_t mfma32_t(u32x4 a, u32x4 b, f32x16_t c, f16_t)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
}
__device__ __forceinline__ f32x4 mfma16_t(u32x4 a, u32x4 b, f32x4 c, bf16_t)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}
__device__ __forceinline__ f32x4 mfma16_t(u32x4 a, u32x4 b, f32x4 c, f16_t)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
}

// Direct-to-LDS load: 16 bytes of every lane, lane l landing at lds + 16 l (lds
// uniform).  Written as asm because the compiler, for the builtin, drains every
// load in flight before any LDS read that it cannot prove disjoint (measured on
// the transposing reads of the grouped products); completion is counted by the
// caller with dma_wait.  It has no register output.  (m0 is the
// compiler's scratch: it sets it right before each use of its own.)
__device__ __forceinline__ void dma16(const void* src, const void* lds)
{
    typedef __attribute__((address_space(3))) const void* lds_t;
    const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_t)lds);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(at), "v"(src) : "memory");
}
// The same from base + offset (base uniform, offset a lane's bytes) to the LDS
// address lds + AT (lds uniform, AT constant): no address arithmetic per load.
__device__ __forceinline__ uintptr_t uniform_address(const void* p)
{
    const uint64_t v = (uint64_t)(uintptr_t)p;
    return (uintptr_t)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v) |
                       (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32)) << 32);
}
template <int AT>
__device__ __forceinline__ void dma16_at(const void* base, uint32_t offset, uint32_t lds)
{
    asm volatile("s_add_u32 m0, %0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, %3" ::"s"(lds), "n"(AT), "v"(offset),
                 "s"(uniform_address(base))
                 : "memory", "scc");
}
template <int AT>
__device__ __forceinline__ void dma16_at(const void* src, uint32_t lds)
{
    asm volatile("s_add_u32 m0, %0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, off" ::"s"(lds), "n"(AT), "v"(src)
                 : "memory", "scc");
}
// LDS address of a shared object.
__device__ __forceinline__ uint32_t lds_address(const void* p)
{
    typedef __attribute__((address_space(3))) const void* lds_t;
    return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_t)p);
}

// The same for 2 and 1 bytes of every lane, each landing zero-extended in the
// 4-byte LDS word lds + 4 l.
__device__ __forceinline__ void dma_u16(const void* src, const void* lds)
{
    typedef __attribute__((address_space(3))) const void* lds_t;
    const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_t)lds);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_ushort %1, off" ::"s"(at), "v"(src) : "memory");
}
__device__ __forceinline__ void dma_u8(const void* src, const void* lds)
{
    typedef __attribute__((address_space(3))) const void* lds_t;
    const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_t)lds);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_ubyte %1, off" ::"s"(at), "v"(src) : "memory");
}
// Wait until at most N vector-memory operations of this wave are outstanding
// (they complete in order).
template <int N>
__device__ __forceinline__ void dma_wait()
{
    static_assert(N >= 0 && N < 64, "vmcnt range");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Segment e of the sorted rows, clamped to [0, M] whatever the offsets hold.
struct Segment {
    int begin, end;
};
__device__ __forceinline__ Segment segment_of(const int32_t* __restrict__ offsets, int e, int M)
{
    if (!offsets) return Segment{0, M};
    const int b = min(max(offsets[e], 0), M);
    return Segment{b, min(max(offsets[e + 1], b), M)};
}

}  // namespace moe
