// adapter.cuh -- the inner values v of the tokens' adapters as 16-bit terms, and
// their delta B_a v_t in warp-MMA fragments.
//
// v is fp32; the MMA takes 16-bit operands, so v is split into terms of B's
// type (v = hi + lo [+ lower], each exact in what the ones before leave): three
// bf16 terms hold all 24 bits of v, two fp16 terms 22.  Fewer would show: where
// W x, the old y or the other rank values cancel a delta, what v leaves out is
// the result.  (Two bf16 terms leave out 2^-17 of v, and 8192 tokens of eight
// requests beside 2048 x 2048 at rank 32 take 71.3 us with them, 73.4 with three;
// the delta alone at rank 16 36.7 and 43.9.)  The split is made once, where v is
// computed.  fp16's range is too small for v: a token whose largest value lies
// outside [2^-2, 2^15) is first scaled by a power of two that brings it into
// [1, 2), undone in the result.  Either way the two terms hold each value to
// 2^-23 of the token's largest.
#pragma once
#include "common.cuh"
#include "kernels.h"
#include "pack16.cuh"

namespace moe {

constexpr int adapter_terms(bool bf16) { return bf16 ? 3 : 2; }

// Split v: `terms` row-major 16-bit matrices [T x r], then (fp16) the factor
// that undoes each token's scale.  fp32 v: [T x r].
MOE_DEV const uint16_t* adapter_term(const AdapterArgs& p, int term) {
    return static_cast<const uint16_t*>(p.v) + (int64_t)term * p.T * p.r;
}
MOE_DEV float* adapter_back(const AdapterArgs& p) {  // (fp16)
    return reinterpret_cast<float*>(static_cast<uint16_t*>(p.v) + (int64_t)adapter_terms(false) * p.T * p.r);
}

// the next term of a value, and what it leaves (an infinite term leaves nothing)
template <bool BF16>
MOE_DEV uint16_t take_term(float& v) {
    const uint16_t t = pack1<BF16>(v);
    const float x = unpack1<BF16>(t);
    v = isinf(x) ? 0.f : v - x;
    return t;
}

// Adds the delta of tokens t0 .. t0 + n - 1 (n <= 16) to MMA fragments of fp32
// bits: lo[4 q + i] is feature f0 + lane / 4 + 8 (i / 2), token 8 q + 2 (lane %
// 4) + i % 2; hi the same 16 features further.  Whole warps, any order of ids.
//
// 32 rank values at a time: v's fragments of all 16 tokens are loaded once, then
// each distinct adapter among them takes one pass of MMAs whose columns are kept
// for its own tokens only (another adapter's infinities must not reach a token).
// The next adapter's rows of B load behind the pass, and those of the tokens
// after these (next .. next + n_next - 1) are fetched into L1.  Lane l / 4 reads
// token l / 4 (+ 8) and feature rows l / 4 + 8 i; lane l % 4 takes eight
// consecutive rank values of each, the same for both operands.
template <bool BF16>
MOE_DEV void add_delta(const AdapterArgs& p, int t0, int n, int next, int n_next, int f0, uint32_t* lo, uint32_t* hi) {
    constexpr int TERMS = adapter_terms(BF16);
    const int lane = threadIdx.x & 31, gq = lane >> 2, c = lane & 3;
    int id = lane < n ? __ldg(&p.ids[t0 + lane]) : -1;
    int id_next = lane < n_next ? __ldg(&p.ids[next + lane]) : -1;
    if (id < 0 || id >= p.L) id = -1;
    if (id_next < 0 || id_next >= p.L) id_next = -1;
    const uint16_t* B = static_cast<const uint16_t*>(p.b);
    const uint32_t mine = __match_any_sync(0xffffffffu, id), mine_next = __match_any_sync(0xffffffffu, id_next);
    if (id_next >= 0 && (mine_next & ((1u << lane) - 1)) == 0) {  // an adapter's first token: its 32 rows are contiguous
        const char* rows = reinterpret_cast<const char*>(B + ((int64_t)id_next * p.N + f0) * p.r);
        for (int i = 0; i < 64 * min(p.r, 64) && f0 + 32 <= p.N; i += 128) asm volatile("prefetch.global.L1 [%0];" ::"l"(rows + i));
    }
    const uint32_t all = __ballot_sync(0xffffffffu, id >= 0);
    if (!all) return;
    const bool use[2] = {((all >> gq) & 1) != 0, ((all >> (8 + gq)) & 1) != 0};
    float back[4];  // fp16: undoes the scale of tokens 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = 8 * (i >> 1) + 2 * c + (i & 1);
        back[i] = !BF16 && ((all >> t) & 1) ? adapter_back(p)[t0 + t] : 1.f;
    }
    int64_t at[4];  // offset of feature rows f0 + gq + 8 i in one adapter's B (past N: any row, not stored)
#pragma unroll
    for (int i = 0; i < 4; ++i) at[i] = (int64_t)min(f0 + gq + 8 * i, p.N - 1) * p.r + 8 * c;
    for (int j0 = 0; j0 < p.r; j0 += 32) {
        const bool in = j0 + 8 * c < p.r;
        uint4 v[2][TERMS], w[4], w_next[4];
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int k = 0; k < TERMS; ++k) {
                v[q][k] = make_uint4(0, 0, 0, 0);
                if (in && use[q])
                    v[q][k] = *reinterpret_cast<const uint4*>(adapter_term(p, k) + (int64_t)(t0 + gq + 8 * q) * p.r + j0 + 8 * c);
            }
        auto load = [&](int a, uint4 (&to)[4]) {
            const uint16_t* rows = B + (int64_t)a * p.N * p.r + j0;
#pragma unroll
            for (int i = 0; i < 4; ++i) to[i] = load_or_zero(rows + at[i], in);
        };
        uint32_t todo = all;
        int leader = __ffs(todo) - 1;
        load(__shfl_sync(0xffffffffu, id, leader), w);
        while (todo) {
            const uint32_t used = __shfl_sync(0xffffffffu, mine, leader);
            todo &= ~used;
            if (todo) {
                leader = __ffs(todo) - 1;
                load(__shfl_sync(0xffffffffu, id, leader), w_next);
            }
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                if (!((used >> (8 * q)) & 0xffu)) continue;
                float d[2][4] = {};
                const uint32_t lo0[4] = {w[0].x, w[1].x, w[0].y, w[1].y}, lo1[4] = {w[0].z, w[1].z, w[0].w, w[1].w};
                const uint32_t hi0[4] = {w[2].x, w[3].x, w[2].y, w[3].y}, hi1[4] = {w[2].z, w[3].z, w[2].w, w[3].w};
#pragma unroll
                for (int k = 0; k < TERMS; ++k) {
                    mma16<BF16>(d[0], lo0, v[q][k].x, v[q][k].y);
                    mma16<BF16>(d[1], hi0, v[q][k].x, v[q][k].y);
                    mma16<BF16>(d[0], lo1, v[q][k].z, v[q][k].w);
                    mma16<BF16>(d[1], hi1, v[q][k].z, v[q][k].w);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (!((used >> (8 * q + 2 * c + (i & 1))) & 1)) continue;
                    const float s = back[2 * q + (i & 1)];
                    lo[4 * q + i] = __float_as_uint(BF16 ? __uint_as_float(lo[4 * q + i]) + d[0][i] : fmaf(d[0][i], s, __uint_as_float(lo[4 * q + i])));
                    hi[4 * q + i] = __float_as_uint(BF16 ? __uint_as_float(hi[4 * q + i]) + d[1][i] : fmaf(d[1][i], s, __uint_as_float(hi[4 * q + i])));
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = w_next[i];
        }
    }
}

}  // namespace moe
