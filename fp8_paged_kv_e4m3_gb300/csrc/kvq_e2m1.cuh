// kvq_e2m1.cuh -- the 4-bit (E2M1) cache's format: page layout, quantiser and
// decoder, shared by the append, read-back, decode and prefill kernels.
//
// A channel's value is E2M1(code) * b * S: S the layer's calibrated scale,
// b the E4M3 scale of its block of 16 channels of one token.  One page of one
// kv head is 9 * D / 4 bytes (D = 128: 288 = 9 sectors of 32 bytes):
//   codes  [4 tokens][D / 2]          channel 2i in the low nibble of byte i
//   scales [D / 16 blocks][4 tokens]  E4M3 bytes
// The scales are block-major so that a thread of the P V product, which holds
// one block of a page's four tokens, reads their four scales as one word.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

namespace kvq {

__host__ __device__ constexpr int e2m1_page_bytes(int head_dim) { return 9 * head_dim / 4; }
__host__ __device__ constexpr int e2m1_scale_off(int head_dim) { return 2 * head_dim; }   // first scale byte

// two fp32 -> two E2M1 codes in one byte (lo in the low nibble): round to
// nearest even, magnitudes beyond 6 to 6
__device__ __forceinline__ uint32_t e2m1_pack2(float lo, float hi)
{
    uint32_t d;
    asm("{\n\t.reg .b8 b, z;\n\tmov.b16 {z, b}, 0;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\tmov.b32 %0, {b, z, z, z};\n\t}"
        : "=r"(d) : "f"(lo), "f"(hi));
    return d;   // the other bytes are 0
}

// eight fp32 -> eight E2M1 codes (element 0 in the lowest nibble).  The bytes
// are joined by integer instructions: one asm block of four conversions and a
// mov of their bytes compiles (nvcc 13.0) to a store of zeros in some places.
__device__ __forceinline__ uint32_t e2m1_pack8(const float (&y)[8])
{
    const uint32_t a = __byte_perm(e2m1_pack2(y[0], y[1]), e2m1_pack2(y[2], y[3]), 0x0040);
    const uint32_t b = __byte_perm(e2m1_pack2(y[4], y[5]), e2m1_pack2(y[6], y[7]), 0x0040);
    return __byte_perm(a, b, 0x5410);
}

// byte Y of x (two codes) -> two fp16 values, the low nibble in the low half;
// exact (every E2M1 value is an fp16 value)
template <int Y>
__device__ __forceinline__ uint32_t e2m1_pair(uint32_t x)
{
    uint32_t d;
    if (Y == 0)
        asm("{\n\t.reg .b8 a, b, c, e;\n\tmov.b32 {a, b, c, e}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(d) : "r"(x));
    else if (Y == 1)
        asm("{\n\t.reg .b8 a, b, c, e;\n\tmov.b32 {a, b, c, e}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(d) : "r"(x));
    else if (Y == 2)
        asm("{\n\t.reg .b8 a, b, c, e;\n\tmov.b32 {a, b, c, e}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(d) : "r"(x));
    else
        asm("{\n\t.reg .b8 a, b, c, e;\n\tmov.b32 {a, b, c, e}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, e;\n\t}" : "=r"(d) : "r"(x));
    return d;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// one E4M3 byte -> fp32, exact
__device__ __forceinline__ float e4m3_value(uint32_t byte)
{
    return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3)));
}

// The scale byte of a block of 16 values whose largest magnitude has the
// binary32 bits `amax` (compared as integers, so that a NaN is the largest),
// and the factor its values are multiplied by before the rounding to E2M1:
//   b = E4M3(a / fl(6 S)),  r = fl(1 / fl(b S))  (0 for b = 0)
// Each quotient and product is one binary32 operation rounded to nearest
// even; b saturates at 448 and is NaN for a NaN, which makes the block NaN.
struct E2m1Block {
    uint32_t scale;
    float factor;
};

__device__ __forceinline__ E2m1Block e2m1_block(uint32_t amax, float six_s, float s)
{
    E2m1Block k;
    k.scale = __nv_cvt_float_to_fp8(__fdiv_rn(__uint_as_float(amax), six_s), __NV_SATFINITE, __NV_E4M3);
    k.factor = k.scale == 0u ? 0.f : __frcp_rn(__fmul_rn(e4m3_value(k.scale), s));
    return k;
}

}  // namespace kvq
