// qb_mm_device.h -- device helpers of the products with 4-bit weights: operands of
// the MFMA instructions, and the dequantization of a lane's weights into them.
#pragma once
#include "qb_device.h"

namespace qb {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// Eight weights or activations of one MFMA operand, in the compute dtype.
template <int XDT>
struct Frag {
    uint32_t w[4];                           // 8 x 16 bits (bf16 / fp16)
};
template <>
struct Frag<DT_F32> {
    float w[8];
};

template <int XDT>
__device__ __forceinline__ void frag_zero(Frag<XDT>& f)
{
#pragma unroll
    for (int i = 0; i < (XDT == DT_F32 ? 8 : 4); ++i) f.w[i] = 0;
}

// A T at byte offset off (uint32) from a uniform base: the address is the
// scalar base plus one 32-bit lane offset.  Cached (the activations and the
// block constants are re-read by other workgroups).
template <class T>
__device__ __forceinline__ T ldo(const void* base, uint32_t off)
{
    const QB_G char* const b = (const QB_G char*)base;          // global address space first
    return *(const QB_G T*)(b + off);
}

// Eight activations at byte offset off from a uniform base.
template <int XDT>
__device__ __forceinline__ void load_frag_o(const void* base, uint32_t off, Frag<XDT>& f)
{
    if constexpr (XDT == DT_F32) {
        const f32x4 a = ldo<f32x4>(base, off), b = ldo<f32x4>(base, off + 16u);
        f.w[0] = a.x; f.w[1] = a.y; f.w[2] = a.z; f.w[3] = a.w;
        f.w[4] = b.x; f.w[5] = b.y; f.w[6] = b.z; f.w[7] = b.w;
    } else {
        const u32x4 a = ldo<u32x4>(base, off);
        f.w[0] = a.x; f.w[1] = a.y; f.w[2] = a.z; f.w[3] = a.w;
    }
}

// acc += A B over the 8 k of this lane's fragments (16x16 tile).
template <int XDT>
__device__ __forceinline__ void mma(const Frag<XDT>& a, const Frag<XDT>& b, f32x4& acc)
{
    if constexpr (XDT == DT_BF16) {
        bf16x8 av, bv;
        __builtin_memcpy(&av, a.w, 16);
        __builtin_memcpy(&bv, b.w, 16);
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, bv, acc, 0, 0, 0);
    } else if constexpr (XDT == DT_F16) {
        f16x8 av, bv;
        __builtin_memcpy(&av, a.w, 16);
        __builtin_memcpy(&bv, b.w, 16);
        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(av, bv, acc, 0, 0, 0);
    } else {
        // binary32: eight 16x16x4 products, one k per lane group each
#pragma unroll
        for (int i = 0; i < 8; ++i) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a.w[i], b.w[i], acc, 0, 0, 0);
    }
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Two binary32 values rounded to nearest even into one word of the compute
// dtype, a in the low half.
template <int XDT>
__device__ __forceinline__ uint32_t pack_two(float a, float b)
{
    if constexpr (XDT == DT_BF16) {
        const bf16x2 h = __builtin_convertvector((f32x2{a, b}), bf16x2);    // one v_cvt_pk_bf16_f32
        uint32_t u;
        __builtin_memcpy(&u, &h, 4);
        return u;
    } else {
        return pack2<XDT>(a, b);
    }
}

// Eight weights (the bytes 4q .. 4q+3 of a lane's 16-byte chunk): code value times the
// block absmax, one binary32 multiply, rounded once to the compute dtype (as
// qb_dequantize).  Byte j of a code word holds element 2j (high nibble) and 2j+1 (low);
// two masks per word turn all eight nibbles into byte offsets into the 16-entry table of
// code values in LDS.
template <int XDT>
__device__ __forceinline__ void dequant_frag(uint32_t word, float a, const float* s_val, Frag<XDT>& f)
{
    const char* const tv = reinterpret_cast<const char*>(s_val);
    uint32_t th = (word >> 2) & 0x3C3C3C3Cu;           // 4 * high nibbles
    uint32_t tl = (word << 2) & 0x3C3C3C3Cu;           // 4 * low nibbles
    // Opaque to the compiler (no instruction): it would otherwise fold the
    // masks into a shift and a mask per nibble, where one bit-field extract
    // per nibble suffices.
    asm("" : "+v"(th), "+v"(tl));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float hi = *reinterpret_cast<const float*>(tv + __builtin_amdgcn_ubfe(th, 8 * j, 8)) * a;
        const float lo = *reinterpret_cast<const float*>(tv + __builtin_amdgcn_ubfe(tl, 8 * j, 8)) * a;
        if constexpr (XDT == DT_F32) {
            f.w[2 * j] = hi;
            f.w[2 * j + 1] = lo;
        } else {
            f.w[j] = pack_two<XDT>(hi, lo);
        }
    }
}

// dequant_frag in two steps: the code values of eight weights, and their products.
__device__ __forceinline__ void code_values(uint32_t word, const float* s_val, float* v)
{
    const char* const tv = reinterpret_cast<const char*>(s_val);
    uint32_t th = (word >> 2) & 0x3C3C3C3Cu, tl = (word << 2) & 0x3C3C3C3Cu;
    asm("" : "+v"(th), "+v"(tl));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[2 * j] = *reinterpret_cast<const float*>(tv + __builtin_amdgcn_ubfe(th, 8 * j, 8));
        v[2 * j + 1] = *reinterpret_cast<const float*>(tv + __builtin_amdgcn_ubfe(tl, 8 * j, 8));
    }
}

template <int XDT>
__device__ __forceinline__ void scaled(const float* v, float a, Frag<XDT>& f)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (XDT == DT_F32) {
            f.w[2 * j] = v[2 * j] * a;
            f.w[2 * j + 1] = v[2 * j + 1] * a;
        } else {
            f.w[j] = pack_two<XDT>(v[2 * j] * a, v[2 * j + 1] * a);
        }
    }
}

// The 32 weights of a lane's chunk.
template <int XDT>
__device__ __forceinline__ void dequant_chunk(const u32x4& cw, float a, const float* s_val, Frag<XDT>* f)
{
    dequant_frag<XDT>(cw.x, a, s_val, f[0]);
    dequant_frag<XDT>(cw.y, a, s_val, f[1]);
    dequant_frag<XDT>(cw.z, a, s_val, f[2]);
    dequant_frag<XDT>(cw.w, a, s_val, f[3]);
}

// Waits until at most N loads of this wave are in flight.
template <int N>
__device__ __forceinline__ void wait_loads()
{
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}

// Workgroup barrier behind which this wave's LDS reads have returned.  Direct global-to-LDS
// loads stay in flight across it (a fence would wait for all of them): the caller waits for
// those that it needs.
__device__ __forceinline__ void pipeline_barrier()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (3 << 14));       // lgkmcnt(0), of which the compiler knows
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Pointers of a direct global-to-LDS load.
typedef const void __attribute__((address_space(1)))* gptr_t;
typedef void __attribute__((address_space(3)))* lptr_t;

}  // namespace qb
