// adapter.cuh -- the delta B_a v_t of 16 tokens by a warp's 32 features, as
// warp-MMA fragments.
//
// v is fp32; the MMA takes 16-bit operands, so v is split into terms of B's
// type (v = hi + lo [+ lower], each exact in what the ones before leave): two
// terms hold 16 bits of v in bf16 and 22 in fp16, three hold 24 in bf16, which
// fp32 results use.  fp16's range is too small for v: each token's values are
// first scaled by a power of two that brings the largest to [1, 2).
#pragma once
#include "common.cuh"
#include "kernels.h"
#include "pack16.cuh"

namespace moe {

// d[m][n][i]: feature 16 m + lane / 4 + 8 (i / 2), token 8 n + 2 (lane % 4) + i % 2
struct DeltaFrags {
    float d[2][2][4];
};
MOE_DEV int frag_feature(int m, int i) { return 16 * m + ((threadIdx.x & 31) >> 2) + 8 * (i >> 1); }
MOE_DEV int frag_token(int n, int i) { return 8 * n + 2 * (threadIdx.x & 3) + (i & 1); }

// The lane's four v values of rank j..j+3 of token t, summed over the slices.
MOE_DEV float4 adapter_v(const AdapterArgs& p, int t, int j) {
    const float* q = p.v + (int64_t)t * p.r + j;
    float4 s = *reinterpret_cast<const float4*>(q);
    for (int i = 1; i < p.slices; ++i) {
        const float4 u = *reinterpret_cast<const float4*>(q + (int64_t)i * p.T * p.r);
        s.x += u.x, s.y += u.y, s.z += u.z, s.w += u.w;
    }
    return s;
}

template <bool BF16>
MOE_DEV float next_term(float v, float term) {  // what the term leaves (an infinite term leaves nothing)
    return isinf(term) ? 0.f : v - term;
}

// Frags of B_a[f0 .. f0 + 31] . v of tokens t0 .. t0 + 15 that are in `used`
// (a bit per token; the others' columns hold nothing meaningful).
template <bool BF16, int TERMS>
MOE_DEV void adapter_delta(const AdapterArgs& p, int t0, uint32_t used, int a, int f0, DeltaFrags& out) {
    const int lane = threadIdx.x & 31, gq = lane >> 2, c = lane & 3;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) out.d[m][n][i] = 0.f;
    const uint16_t* B = static_cast<const uint16_t*>(p.b) + ((int64_t)a * p.N) * p.r;
    const uint16_t* row[4];  // features f0 + gq + 8 i (past N: any row, its results are not stored)
#pragma unroll
    for (int i = 0; i < 4; ++i) row[i] = B + (int64_t)min(f0 + gq + 8 * i, p.N - 1) * p.r;
    float back[2] = {1.f, 1.f};  // fp16: undoes the scale of token 8 n + gq
    float scale[2] = {1.f, 1.f};
    if (!BF16) {
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            float most = 0.f;
            if ((used >> (8 * n + gq)) & 1)
                for (int j = 4 * c; j < p.r; j += 16) {
                    const float4 v = adapter_v(p, t0 + 8 * n + gq, j);
                    most = fmaxf(fmaxf(fmaxf(most, fabsf(v.x)), fmaxf(fabsf(v.y), fabsf(v.z))), fabsf(v.w));
                }
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
            const int e = min(max((int)(__float_as_uint(most) >> 23), 1), 253);  // biased exponent
            scale[n] = __uint_as_float((uint32_t)(254 - e) << 23);
            back[n] = __uint_as_float((uint32_t)e << 23);
        }
    }
#pragma unroll 2
    for (int j0 = 0; j0 < p.r; j0 += 16) {
        const int j = j0 + 4 * c;
        uint2 w[4];
        float4 v[2];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = j < p.r ? __ldg(reinterpret_cast<const uint2*>(row[i] + j)) : make_uint2(0, 0);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            v[n] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (j < p.r && ((used >> (8 * n + gq)) & 1)) v[n] = adapter_v(p, t0 + 8 * n + gq, j);
            if (!BF16) v[n].x *= scale[n], v[n].y *= scale[n], v[n].z *= scale[n], v[n].w *= scale[n];
        }
        const uint32_t f0r[4] = {w[0].x, w[1].x, w[0].y, w[1].y}, f1r[4] = {w[2].x, w[3].x, w[2].y, w[3].y};
#pragma unroll
        for (int n = 0; n < 2; ++n) {
#pragma unroll
            for (int term = 0; term < TERMS; ++term) {
                const uint32_t b0 = pack2<BF16>(v[n].x, v[n].y), b1 = pack2<BF16>(v[n].z, v[n].w);
                mma16<BF16>(out.d[0][n], f0r, b0, b1);
                mma16<BF16>(out.d[1][n], f1r, b0, b1);
                if (term + 1 < TERMS) {
                    const float2 x0 = unpack2<BF16>(b0), x1 = unpack2<BF16>(b1);
                    v[n] = make_float4(next_term<BF16>(v[n].x, x0.x), next_term<BF16>(v[n].y, x0.y),
                                       next_term<BF16>(v[n].z, x1.x), next_term<BF16>(v[n].w, x1.y));
                }
            }
        }
    }
    if (!BF16) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float s = __shfl_sync(0xffffffffu, back[n], (2 * c + i) * 4);
                out.d[0][n][i] *= s, out.d[0][n][i + 2] *= s, out.d[1][n][i] *= s, out.d[1][n][i + 2] *= s;
            }
    }
}

// Adds the delta of tokens t0 .. t0 + n - 1 (n <= 16) to the fragments lo
// (features f0 .. f0 + 15) and hi (f0 + 16 .. f0 + 31): two of 8 tokens each,
// fp32 bits.  Whole warps; any order of ids, one pass per distinct adapter.
template <bool BF16, int TERMS>
MOE_DEV void add_delta(const AdapterArgs& p, int t0, int n, int f0, uint32_t* lo, uint32_t* hi) {
    const int lane = threadIdx.x & 31;
    int id = lane < n ? __ldg(&p.ids[t0 + lane]) : -1;
    if (id < 0 || id >= p.L) id = -1;
    const uint32_t mine = __match_any_sync(0xffffffffu, id);
    uint32_t todo = __ballot_sync(0xffffffffu, id >= 0);
    while (todo) {
        const int leader = __ffs(todo) - 1;
        const int a = __shfl_sync(0xffffffffu, id, leader);
        const uint32_t used = __shfl_sync(0xffffffffu, mine, leader);
        todo &= ~used;
        DeltaFrags fr;
        adapter_delta<BF16, TERMS>(p, t0, used, a, f0, fr);
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // (another adapter's infinities must not reach this token)
                if (!((used >> frag_token(q, i)) & 1)) continue;
                lo[4 * q + i] = __float_as_uint(__uint_as_float(lo[4 * q + i]) + fr.d[0][q][i]);
                hi[4 * q + i] = __float_as_uint(__uint_as_float(hi[4 * q + i]) + fr.d[1][q][i]);
            }
    }
}

}  // namespace moe
