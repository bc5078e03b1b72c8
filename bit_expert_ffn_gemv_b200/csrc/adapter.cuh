// adapter.cuh -- the inner values v of the tokens' adapters and their delta
// B_a v_t, as warp-MMA fragments of 32 features by 16 tokens.
//
// v is fp32; the MMA takes 16-bit operands, so v is split into terms of B's
// type (v = hi + lo [+ lower], each exact in what the ones before leave): two
// terms hold 16 bits of v in bf16 and 22 in fp16, three hold 24 in bf16, which
// fp32 results use.  The split is made once, where v is computed.  fp16's range
// is too small for v: a token whose largest value lies outside [2^-2, 2^15) is
// first scaled by a power of two that brings it into [1, 2), undone in the
// result (inside the range the two terms hold 2^-23 of that largest value).
#pragma once
#include "common.cuh"
#include "kernels.h"
#include "pack16.cuh"

namespace moe {

// Split v: `terms` row-major 16-bit matrices [T x r], then (fp16) the factor
// that undoes each token's scale.  fp32 v: [T x r].
MOE_DEV const uint16_t* adapter_term(const AdapterArgs& p, int term) {
    return static_cast<const uint16_t*>(p.v) + (int64_t)term * p.T * p.r;
}
MOE_DEV float* adapter_back(const AdapterArgs& p, int terms) {
    return reinterpret_cast<float*>(static_cast<uint16_t*>(p.v) + (int64_t)terms * p.T * p.r);
}

// the next term of a value, and what it leaves (an infinite term leaves nothing)
template <bool BF16>
MOE_DEV uint16_t take_term(float& v) {
    const uint16_t t = pack1<BF16>(v);
    const float x = unpack1<BF16>(t);
    v = isinf(x) ? 0.f : v - x;
    return t;
}

// d[m][n][i]: feature 16 m + lane / 4 + 8 (i / 2), token 8 n + 2 (lane % 4) + i % 2
struct DeltaFrags {
    float d[2][2][4];
};
MOE_DEV int frag_feature(int m, int i) { return 16 * m + ((threadIdx.x & 31) >> 2) + 8 * (i >> 1); }
MOE_DEV int frag_token(int n, int i) { return 8 * n + 2 * (threadIdx.x & 3) + (i & 1); }

// Frags of B_a[f0 .. f0 + 31] . v of tokens t0 .. t0 + 15 that are in `used`
// (a bit per token; the others' columns hold nothing meaningful).  Lane l / 4
// reads token l / 4 (+ 8) and feature rows l / 4 + 8 i; lane l % 4 takes four
// consecutive rank values of each, the same for both operands.
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
    const int quads = p.r >> 2;
    const bool use[2] = {((used >> gq) & 1) != 0, ((used >> (8 + gq)) & 1) != 0};
    const int64_t vrow = (int64_t)(t0 + gq) * p.r;
#pragma unroll 4
    for (int q0 = 0; q0 < quads; q0 += 4) {
        const int q = q0 + c;
        uint2 w[4], v[2][TERMS];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = q < quads ? __ldg(reinterpret_cast<const uint2*>(row[i] + 4 * q)) : make_uint2(0, 0);
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int k = 0; k < TERMS; ++k) {
                v[n][k] = make_uint2(0, 0);
                if (q < quads && use[n])
                    v[n][k] = *reinterpret_cast<const uint2*>(adapter_term(p, k) + vrow + (int64_t)n * 8 * p.r + 4 * q);
            }
        const uint32_t f0r[4] = {w[0].x, w[1].x, w[0].y, w[1].y}, f1r[4] = {w[2].x, w[3].x, w[2].y, w[3].y};
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int k = 0; k < TERMS; ++k) {
                mma16<BF16>(out.d[0][n], f0r, v[n][k].x, v[n][k].y);
                mma16<BF16>(out.d[1][n], f1r, v[n][k].x, v[n][k].y);
            }
    }
    if (!BF16) {
        const float* back = adapter_back(p, TERMS) + t0;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = 8 * n + 2 * c + i;
                const float s = (used >> t) & 1 ? back[t] : 1.f;
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
