// Operands of the LDS-tiled matrix-core kernels (gemm.hip, experts.hip): codes
// unpacked in the natural order of their columns, the 16 x 16 x 32 matrix
// product of either activation type, and the barrier of a DMA ring.
#pragma once

#include <type_traits>

#include "tq_device.h"

namespace tq {

template <class T> struct Mfma;
template <> struct Mfma<F16> {
    typedef f16x8 vec;
    static constexpr float kUnit = 1.0f;  // value of the operand bits of +1
    static __device__ __forceinline__ f32x4 mma(vec a, vec b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};
template <> struct Mfma<BF16> {
    typedef bf16x8 vec;
    static constexpr float kUnit = kBf16TernaryUnit;  // the operand bits of +1 read as bf16 are 2^-7
    static __device__ __forceinline__ f32x4 mma(vec a, vec b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};

// Two values rounded to the activation type by the hardware's conversion (to
// nearest even, infinities and NaN kept), in one word.
template <class T>
__device__ __forceinline__ uint32_t round_pair(float lo, float hi) {
    if constexpr (std::is_same<T, F16>::value) return __builtin_bit_cast(uint32_t, f16x2{(_Float16)lo, (_Float16)hi});
    else return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)lo, (__bf16)hi});
}
template <class T>
__device__ __forceinline__ uint16_t round_one(float v) {
    if constexpr (std::is_same<T, F16>::value) return __builtin_bit_cast(uint16_t, (_Float16)v);
    else return __builtin_bit_cast(uint16_t, (__bf16)v);
}

// Natural-order operand pairs of byte b of a code dword x (fields f_4b ..
// f_4b+3 at bits 0, 2, 4, 6 of the byte): one byte permute puts the byte in
// the low byte of both halves, a mask into 1024.0 keeps field 4b (low half)
// and 4b+1 (high half) at bits 0 and 2, or fields 4b+2 and 4b+3 at bits 4
// and 6, and one packed fp16 fma per pair scales each half by its own power
// of 4 and subtracts 1024/4^s + 1: (1024 + 4^s c) / 4^s - (1024/4^s + 1) =
// c - 1, exact.
struct NatConsts {
    f16x2 mul_lo, add_lo, mul_hi, add_hi;
};
__device__ __forceinline__ NatConsts nat_consts() {
    return NatConsts{f16x2{(_Float16)1.0f, (_Float16)0.25f}, f16x2{(_Float16)-1025.0f, (_Float16)-257.0f},
                     f16x2{(_Float16)0.0625f, (_Float16)0.015625f}, f16x2{(_Float16)-65.0f, (_Float16)-17.0f}};
}
__device__ __forceinline__ uint32_t nat_fma(uint32_t v, f16x2 mul, f16x2 add) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(f16x2, v), mul, add));
}
// Operand of fields 8h .. 8h+7 of x (bytes 2h and 2h+1) in natural order.
template <int H>
__device__ __forceinline__ uint4 nat_quad(uint32_t x, uint32_t magic_v, const NatConsts& k) {
    const uint32_t p0 = __builtin_amdgcn_perm(x, x, 0x0C000C00u | (uint32_t)(2 * H) * 0x00010001u);
    const uint32_t p1 = __builtin_amdgcn_perm(x, x, 0x0C000C00u | (uint32_t)(2 * H + 1) * 0x00010001u);
    const uint32_t mlo = sgpr_const<0x000C0003u>(), mhi = sgpr_const<0x00C00030u>();
    return make_uint4(nat_fma((p0 & mlo) | magic_v, k.mul_lo, k.add_lo), nat_fma((p0 & mhi) | magic_v, k.mul_hi, k.add_hi),
                      nat_fma((p1 & mlo) | magic_v, k.mul_lo, k.add_lo), nat_fma((p1 & mhi) | magic_v, k.mul_hi, k.add_hi));
}

// Workgroup barrier without a release fence: __syncthreads() would wait for
// every outstanding DMA, including the stages issued ahead.  LDS reads and
// writes issued before it are waited for here (the hardware barrier does not
// wait for them, and the compiler may place register-only work, with the
// waits that feed it, after the barrier): a slot read before the barrier may
// be refilled by another wave's DMA right after it, and pairs written before
// it are read by other waves after it.
__device__ __forceinline__ void stage_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// (q_2d - z, q_2d+1 - z) of code word x as exact fp16, natural order.
template <int D>
__device__ __forceinline__ uint32_t nat_w4_pair(uint32_t x, uint32_t mask_v, uint32_t magic_v, f16x2 mul, f16x2 add) {
    const uint32_t y = __builtin_amdgcn_perm(x, x, 0x0C000C00u | (uint32_t)D | ((uint32_t)D << 16));
    const f16x2 v = __builtin_bit_cast(f16x2, (y & mask_v) | magic_v);
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(v, mul, add));
}

template <class T>
__device__ __forceinline__ uint4 nat_w4_quad(uint32_t x, uint32_t mask_v, uint32_t magic_v, f16x2 mul, f16x2 add) {
    const uint4 h = make_uint4(nat_w4_pair<0>(x, mask_v, magic_v, mul, add), nat_w4_pair<1>(x, mask_v, magic_v, mul, add),
                               nat_w4_pair<2>(x, mask_v, magic_v, mul, add), nat_w4_pair<3>(x, mask_v, magic_v, mul, add));
    if constexpr (std::is_same<T, F16>::value) return h;
    else return make_uint4(f16x2_to_bf16x2(h.x), f16x2_to_bf16x2(h.y), f16x2_to_bf16x2(h.z), f16x2_to_bf16x2(h.w));
}

// -(1024 + z) in the low half, -(64 + z) in the high half
__device__ __forceinline__ f16x2 w4_nat_sub(uint32_t z) {
    return __builtin_bit_cast(f16x2, (0xE400u + z) | ((0xD400u + 16u * z) << 16));
}

}  // namespace tq
