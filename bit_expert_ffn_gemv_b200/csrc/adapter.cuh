// adapter.cuh -- the inner values v of the tokens' adapters and their delta
// B_a v_t, as warp-MMA fragments of 32 features by 16 tokens.
//
// v is fp32; the MMA takes 16-bit operands, so v is split into terms of B's
// type (v = hi + lo [+ lower], each exact in what the ones before leave): two
// terms hold 16 bits of v in bf16 and 22 in fp16, three hold 24 in bf16, which
// fp32 results use.  fp16's range is too small for v: each token's values are
// first scaled by a power of two that brings the largest into [1, 2), undone
// in the result.  The split is made once, where v is computed.
#pragma once
#include "common.cuh"
#include "kernels.h"
#include "pack16.cuh"

namespace moe {

// Split v, per token r / 4 quads of four rank values: 16 bytes {hi01, hi23,
// lo01, lo23}, and with three terms 16 more {lower01, lower23, -, -}; then
// (fp16) one factor per token.  fp32 v: [token][r].
MOE_DEV int quad_vectors(int terms) { return terms == 3 ? 2 : 1; }
MOE_DEV float* adapter_back(const AdapterArgs& p, int terms) {
    return reinterpret_cast<float*>(static_cast<uint4*>(p.v) + (int64_t)p.T * (p.r >> 2) * quad_vectors(terms));
}

// the next term of two values: packed, and what it leaves (an infinite term leaves nothing)
template <bool BF16>
MOE_DEV uint32_t take_term(float& a, float& b) {
    const uint32_t t = pack2<BF16>(a, b);
    const float2 x = unpack2<BF16>(t);
    a = isinf(x.x) ? 0.f : a - x.x;
    b = isinf(x.y) ? 0.f : b - x.y;
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
    constexpr int kVecs = TERMS == 3 ? 2 : 1;
    const int quads = p.r >> 2;
    const uint4* v0 = static_cast<const uint4*>(p.v) + (int64_t)(t0 + gq) * quads * kVecs;
    const bool use[2] = {((used >> gq) & 1) != 0, ((used >> (8 + gq)) & 1) != 0};
#pragma unroll 4
    for (int q0 = 0; q0 < quads; q0 += 4) {
        const int q = q0 + c;
        uint2 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = q < quads ? __ldg(reinterpret_cast<const uint2*>(row[i] + 4 * q)) : make_uint2(0, 0);
        uint4 v[2][kVecs];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int k = 0; k < kVecs; ++k) {
                v[n][k] = make_uint4(0, 0, 0, 0);
                if (q < quads && use[n]) v[n][k] = v0[((int64_t)n * 8 * quads + q) * kVecs + k];
            }
        const uint32_t f0r[4] = {w[0].x, w[1].x, w[0].y, w[1].y}, f1r[4] = {w[2].x, w[3].x, w[2].y, w[3].y};
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            mma16<BF16>(out.d[0][n], f0r, v[n][0].x, v[n][0].y);
            mma16<BF16>(out.d[1][n], f1r, v[n][0].x, v[n][0].y);
            mma16<BF16>(out.d[0][n], f0r, v[n][0].z, v[n][0].w);
            mma16<BF16>(out.d[1][n], f1r, v[n][0].z, v[n][0].w);
            if (TERMS == 3) {
                mma16<BF16>(out.d[0][n], f0r, v[n][kVecs - 1].x, v[n][kVecs - 1].y);
                mma16<BF16>(out.d[1][n], f1r, v[n][kVecs - 1].x, v[n][kVecs - 1].y);
            }
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
