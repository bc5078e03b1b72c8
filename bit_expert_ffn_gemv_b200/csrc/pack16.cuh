// pack16.cuh -- conversions between fp32 and 16-bit vectors of either type.
#pragma once
#include "common.cuh"

namespace moe {

template <bool BF16>
MOE_DEV float2 unpack2(uint32_t u) {
    if (BF16) return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
}
template <bool BF16>
MOE_DEV uint32_t pack2(float lo, float hi) {
    if (BF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <bool BF16>
MOE_DEV uint16_t pack1(float v) {
    return BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
}
template <bool BF16>
MOE_DEV float unpack1(uint16_t v) {
    return BF16 ? bf16_bits_to_float(v) : __half2float(__ushort_as_half(v));
}
template <bool BF16>
MOE_DEV void unpack8(const uint4& v, float (&f)[8]) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = unpack2<BF16>(u[i]);
        f[2 * i] = p.x;
        f[2 * i + 1] = p.y;
    }
}
template <bool BF16>
MOE_DEV uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack2<BF16>(f[0], f[1]), pack2<BF16>(f[2], f[3]), pack2<BF16>(f[4], f[5]),
                      pack2<BF16>(f[6], f[7]));
}
template <bool BF16>
MOE_DEV void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (BF16) mma_bf16(d, a, b0, b1, d);
    else mma_f16(d, a, b0, b1, d);
}

// 16 bytes through the read-only path, or zeros: a predicated load, not a
// branch, so that independent loads stay together (not volatile: they may move
// ahead of earlier MMAs)
MOE_DEV uint4 load_or_zero(const void* p, bool take) {
    uint4 v;
    asm("{\n .reg .pred q;\n setp.ne.b32 q, %5, 0;\n mov.b32 %0, 0;\n mov.b32 %1, 0;\n mov.b32 %2, 0;\n"
        " mov.b32 %3, 0;\n @q ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];\n}\n"
        : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
        : "l"(p), "r"(take ? 1 : 0));
    return v;
}

}  // namespace moe
