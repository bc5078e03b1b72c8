// adapters.cu -- low-rank adapters of many requests beside a shared projection.
//
//   v_t = scale[a] * A_a x_t            (rank values, fp32; a = ids[t])
//   y_t = [y_t +] [W x_t +] B_a v_t     (no delta where ids[t] is not in [0, L))
//
// Two launches.  The first computes v for every token; the second starts
// while the first still runs (programmatic dependent launch), streams W, and
// waits for v only before it adds the delta:
//   shrink_kernel   v, from windows of 8 or 32 tokens by slices of K
//   skinny_kernel   up to 64 tokens: W by warp MMAs, straight from HBM
//   grouped_kernel  more tokens: W on the tensor cores (grouped.cu), and with it the delta of runs
//                   of one adapter, as further steps; of mixed tokens it is added in the epilogue
//   expand_kernel   no W: the delta alone
// v is summed in fp32.  Up to 64 tokens with W the delta is fp32 arithmetic too;
// the other forms multiply v as 16-bit terms that hold all of it (bf16), or 2^-23
// of a token's largest value (fp16; adapter.cuh).  The result is rounded once.
#include <cuda_runtime.h>

#include <type_traits>

#include "adapter.cuh"
#include "common.cuh"
#include "kernels.h"
#include "pack16.cuh"
#include "tc.cuh"

namespace moe {

// ---------------------------------------------------------------- shrink
// A cluster of CTAs owns a window of WIN tokens and splits K; its CTAs' sums
// meet through distributed shared memory in rank order, so v is written once,
// already scaled, in the form its reader takes (adapter.cuh).  Inside a CTA the
// window's tokens are grouped by adapter with one match instruction, in any
// order of ids, into items of up to WIN tokens of one adapter, whose A rows
// are read once: MMAs of 16 A rows by 8 tokens, both operands loaded 16 bytes a
// lane in the same permuted order of k.  The eight warps take an item each;
// with fewer items several warps share one and split its K.  Bound by the A
// rows of a decode batch (every token another adapter) or the x of a prefill
// chunk.  8192 tokens of eight requests, K = 2048, x from HBM (5.1 us of it), with
// an expand_kernel of 8 features behind it: 15 us at rank 16, 17 at 32, 27 at 64.
constexpr int kShrinkThreads = 256;
// Values that one MMA accumulator sums (skinny.cu says why).  LONG: a CTA's share of K is
// more, and so may a warp's be, where adapters mix in the window; the items of a request's
// chunk are split over the warps and stay below it up to K = 4096.
constexpr int kShrinkPart = 512;

// Octets of tokens per item, 16-row tiles of A per pass, and the steps of 32 of K
// in flight.  Large windows keep theirs in a ring in shared memory, as many as leave
// room for two CTAs an SM (8192 tokens of rank 32 and K = 2048, x from HBM, v in two
// terms: 15.1 us with the ring, 16.1 with registers; of mixed adapters 46 against 72);
// small ones hold them in registers, as many as about 50 hold (512 tokens of 30
// adapters beside a projection, v in two terms: 36 us, 40 with a ring; in three 38).
template <int WIN, int TILES>
struct ShrinkCfg {
    static constexpr int kOctets = WIN / 8, kTiles = TILES, kRows = 16 * TILES, kPitch = kRows + 4;
    static constexpr int kVecs = kOctets + 2 * TILES, kDepth = WIN == 8 ? (kVecs <= 3 ? 4 : 2) : 27 / kVecs;
    static constexpr int kStep = kVecs * 512;  // bytes of a warp's step
    static constexpr int kRing = WIN == 8 ? 0 : 8 * kDepth * kStep;
    static constexpr int kRed = 8 * WIN * kPitch * 4;            // [warp][token of its item][row], in the ring's place
    static constexpr int kShared = kRing > kRed ? kRing : kRed;  // bytes
};

template <bool BF16, int WIN, int TERMS, int TILES, bool LONG>
__global__ void __launch_bounds__(kShrinkThreads, 2) shrink_kernel(const AdapterArgs p) {
    using C = ShrinkCfg<WIN, TILES>;
    extern __shared__ __align__(16) uint8_t shrink_smem[];
    float* red = reinterpret_cast<float*>(shrink_smem);                 // [8][WIN][kPitch]
    float* sums = reinterpret_cast<float*>(shrink_smem + C::kShared);   // [WIN][r]
    __shared__ int item_adapter[WIN], item_count[WIN];
    __shared__ int8_t item_tok[WIN][WIN];          // tokens of an item, in order
    __shared__ int8_t tok_item[WIN], tok_place[WIN];  // a token's item (-1: none) and place in it
    grid_wait();     // the kernel before may still write x and ids, or read v
    grid_release();  // (after the wait: the next kernel reads W, x and ids at once)
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, c = lane & 3;
    const int t0 = blockIdx.x * WIN, slice = blockIdx.y;
    const int per = ((p.K + p.slices - 1) / p.slices + 31) & ~31;  // K of a CTA
    const int sb = slice * per, se = min(p.K, sb + per);
    const int t = t0 + lane;
    int id = lane < WIN && t < p.T ? __ldg(&p.ids[t]) : -1;
    if (id < 0 || id >= p.L) id = -1;
    const uint32_t mine = __match_any_sync(0xffffffffu, id);
    const bool begins = id >= 0 && (mine & ((1u << lane) - 1)) == 0;  // the adapter's first token
    const uint32_t starts = __ballot_sync(0xffffffffu, begins);
    const int items = __popc(starts);
    if (items == 0) return;  // (the whole cluster)
    if (warp == 0 && lane < WIN) {
        const uint32_t below = (1u << lane) - 1;
        const int it = __popc(starts & ((1u << (__ffs(mine) - 1)) - 1)), place = __popc(mine & below);
        tok_item[lane] = (int8_t)(id >= 0 ? it : -1);
        tok_place[lane] = (int8_t)place;
        if (id >= 0) item_tok[it][place] = (int8_t)lane;
        if (begins) {
            item_adapter[it] = id;
            item_count[it] = __popc(mine);
        }
    }
    __syncthreads();
    const int share = items == 1 ? 8 : items == 2 ? 4 : items <= 4 ? 2 : 1;  // warps per item
    const int at_once = 8 / share, part = warp % share;
    const int kw = ((se - sb + share - 1) / share + 31) & ~31;
    const int kb = sb + part * kw, ke = min(se, kb + kw);
    const uint16_t* x = static_cast<const uint16_t*>(p.x);
    const uint16_t* A = static_cast<const uint16_t*>(p.a);
    for (int base = 0; base < items; base += at_once) {
        const int it = base + warp / share;
        const int n = it < items ? item_count[it] : 0, a = n ? item_adapter[it] : 0;
        const int octets = (n + 7) >> 3;
        // (columns and rows past the item's end repeat its first: their sums are not read)
        const uint16_t* xr[C::kOctets];
#pragma unroll
        for (int o = 0; o < C::kOctets; ++o)
            xr[o] = x + (int64_t)(t0 + (8 * o + gq < n ? item_tok[it][8 * o + gq] : n ? item_tok[it][0] : 0)) * p.ldx + 8 * c;
        for (int j0 = 0; j0 < p.r; j0 += C::kRows) {
            const int rows = min(C::kRows, p.r - j0), tiles = (rows + 15) >> 4;
            float acc[C::kTiles][C::kOctets][4] = {};
            if (n) {
                const uint16_t* ar[2 * C::kTiles];
#pragma unroll
                for (int q = 0; q < 2 * C::kTiles; ++q)
                    ar[q] = A + ((int64_t)a * p.r + j0 + (q * 8 + gq < rows ? q * 8 + gq : gq)) * p.K + 8 * c;
                // The warp's share of K.  IN_PARTS: more than kShrinkPart of it, summed in parts of that many, the item's
                // octets (of which a window of many adapters has one each) one after the other, o0 first to last
                auto walk = [&](auto in_parts, int o0) {
                    constexpr bool IN_PARTS = decltype(in_parts)::value;
                    constexpr int OCT = IN_PARTS ? 1 : C::kOctets;
                    float now[C::kTiles][OCT][4] = {}, before[C::kTiles][OCT][4] = {};
                    const uint16_t* xs[OCT];
#pragma unroll
                    for (int o = 0; o < C::kOctets; ++o)
                        if (!IN_PARTS || o == o0) xs[IN_PARTS ? 0 : o] = xr[o];
                    auto source = [&](int v) { return v < OCT ? xs[v] : ar[v - OCT]; };
                    auto multiply = [&](auto operand) {
                        uint4 bv[OCT];
#pragma unroll
                        for (int o = 0; o < OCT; ++o)
                            if (o == 0 || o < octets) bv[o] = operand(o);
#pragma unroll
                        for (int q = 0; q < C::kTiles; ++q) {
                            const uint4 lo = operand(OCT + 2 * q), hi = operand(OCT + 2 * q + 1);
                            const uint32_t f0[4] = {lo.x, hi.x, lo.y, hi.y}, f1[4] = {lo.z, hi.z, lo.w, hi.w};
#pragma unroll
                            for (int o = 0; o < OCT; ++o) {
                                if (o > 0 && o >= octets) break;
                                mma16<BF16>(now[q][o], f0, bv[o].x, bv[o].y);
                                mma16<BF16>(now[q][o], f1, bv[o].z, bv[o].w);
                            }
                        }
                    };
                    auto end_part = [&] {
#pragma unroll
                        for (int q = 0; q < C::kTiles; ++q)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                before[q][0][i] += now[q][0][i];
                                now[q][0][i] = 0.f;
                            }
                    };
                    constexpr int VECS = OCT + 2 * C::kTiles;
                    if constexpr (C::kRing > 0) {
                        // a lane copies what it will multiply itself: the ring needs no barrier
                        uint8_t* ring = shrink_smem + warp * C::kDepth * C::kStep + lane * 16;
                        auto fetch = [&](uint8_t* to, int k) {
                            const uint32_t bytes = k + 8 * c < ke ? 16 : 0;
#pragma unroll
                            for (int v = 0; v < VECS; ++v)
                                if (v == 0 || v < octets || v >= OCT) tc::cp16_or_zero(to + v * 512, source(v) + k, bytes);
                        };
#pragma unroll
                        for (int b = 0; b < C::kDepth - 1; ++b) {
                            if (kb + 32 * b < ke) fetch(ring + b * C::kStep, kb + 32 * b);
                            tc::cp_commit();
                        }
                        int in = C::kDepth - 1, out = 0;  // the ring's places to fill and to read
                        for (int k = kb; k < ke; k += 32) {
                            if (IN_PARTS && ((k - kb) & (kShrinkPart - 1)) == 0) end_part();
                            const int ahead = k + 32 * (C::kDepth - 1);
                            if (ahead < ke) fetch(ring + in * C::kStep, ahead);
                            tc::cp_commit();
                            tc::cp_wait<C::kDepth - 1>();
                            const uint8_t* from = ring + out * C::kStep;
                            multiply([&](int v) { return *reinterpret_cast<const uint4*>(from + v * 512); });
                            in = in + 1 == C::kDepth ? 0 : in + 1;
                            out = out + 1 == C::kDepth ? 0 : out + 1;
                        }
                    } else {
                        // (only a last, partial step looks at the end of K)
                        uint4 held[C::kDepth][VECS];
                        auto fetch = [&](int b, int k) {
                            if (k + 32 <= ke) {
#pragma unroll
                                for (int v = 0; v < VECS; ++v) held[b][v] = __ldg(reinterpret_cast<const uint4*>(source(v) + k));
                            } else {
                                const bool in = k + 8 * c < ke;
#pragma unroll
                                for (int v = 0; v < VECS; ++v) held[b][v] = load_or_zero(source(v) + k, in);
                            }
                        };
#pragma unroll
                        for (int b = 0; b < C::kDepth - 1; ++b)
                            if (kb + 32 * b < ke) fetch(b, kb + 32 * b);
                        for (int k0 = kb; k0 < ke; k0 += 32 * C::kDepth) {
                            if (IN_PARTS && ((k0 - kb) & (kShrinkPart - 1)) == 0) end_part();
#pragma unroll
                            for (int b = 0; b < C::kDepth; ++b) {
                                const int k = k0 + 32 * b, ahead = k + 32 * (C::kDepth - 1);
                                if (ahead < ke) fetch((b + C::kDepth - 1) % C::kDepth, ahead);
                                if (k < ke) multiply([&](int v) { return held[b][v]; });
                            }
                        }
                    }
#pragma unroll
                    for (int o = 0; o < C::kOctets; ++o) {
                        if (IN_PARTS && o != o0) continue;
#pragma unroll
                        for (int q = 0; q < C::kTiles; ++q)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int own = IN_PARTS ? 0 : o;
                                acc[q][o][i] = IN_PARTS ? before[q][own][i] + now[q][own][i] : now[q][own][i];
                            }
                    }
                };
                // (both loops in one kernel only with large windows, whose chunks of a request stay below a part: with
                // small ones they spill, 1000 mixed tokens of rank 64, K = 4096: 154 us against 76)
                if constexpr (LONG && WIN == 8) {
                    walk(std::true_type{}, 0);
                } else if constexpr (LONG) {
                    if (ke - kb > kShrinkPart)
                        for (int o = 0; o < octets; ++o) walk(std::true_type{}, o);
                    else walk(std::false_type{}, 0);
                } else {
                    walk(std::false_type{}, 0);
                }
            }
            __syncthreads();  // every warp is through with its ring, or the last pass's sums
            float* mr = red + warp * WIN * C::kPitch;
#pragma unroll
            for (int q = 0; q < C::kTiles; ++q)
#pragma unroll
                for (int o = 0; o < C::kOctets; ++o) {
                    if (q >= tiles || o >= octets) break;
                    float* m = mr + (8 * o + 2 * c) * C::kPitch + q * 16 + gq;
                    m[0] = acc[q][o][0];
                    m[C::kPitch] = acc[q][o][1];
                    m[8] = acc[q][o][2];
                    m[C::kPitch + 8] = acc[q][o][3];
                }
            __syncthreads();
            // each token's sums, the shares added in order
#pragma unroll
            for (int i = tid; i < WIN * C::kRows; i += kShrinkThreads) {
                const int m = i / C::kRows, j = i % C::kRows, slot = tok_item[m] - base;
                if (j >= rows || tok_item[m] < 0 || slot < 0 || slot >= at_once) continue;
                const float* src = red + (slot * share * WIN + tok_place[m]) * C::kPitch + j;
                float s = src[0];
#pragma unroll
                for (int q = 1; q < 8; ++q)
                    if (q < share) s += src[q * WIN * C::kPitch];
                sums[m * p.r + j0 + j] = s;
            }
            if (C::kRing > 0 && (j0 + C::kRows < p.r || base + at_once < items)) __syncthreads();  // the next pass fills the ring
        }
    }
    if (p.slices > 1) tc::cluster_sync();
    else __syncthreads();
    // each CTA finishes its share of the tokens: a warp a token, a lane every 32nd rank value
    for (int m = slice * 8 + warp; m < WIN; m += 8 * p.slices) {
        const int a = __shfl_sync(0xffffffffu, id, m);
        if (a < 0) continue;
        const float sc = p.scale ? __ldg(&p.scale[a]) : 1.0f;
        constexpr int kPer = kMaxAdapterRank / 32;
        float v[kPer], most = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int j = lane + 32 * i;
            v[i] = 0.f;
            if (32 * i >= p.r) break;
            if (j < p.r) {
                const float* at = sums + m * p.r + j;
                if (p.slices == 1) v[i] = *at;
                else
                    for (int s = 0; s < p.slices; ++s) v[i] += tc::ld_cluster(tc::cluster_addr(at, s));
                v[i] *= sc;
            }
            most = fmaxf(most, fabsf(v[i]));
        }
        const int64_t row = (int64_t)(t0 + m) * p.r;
        if (TERMS == 0) {
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (lane + 32 * i < p.r) static_cast<float*>(p.v)[row + lane + 32 * i] = v[i];
            continue;
        }
        float scale = 1.f;
        if (!BF16) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
            float back = 1.f;
            if (most != 0.f && !(most >= 0.25f && most < 32768.f)) {
                const int e = min(max((int)(__float_as_uint(most) >> 23), 1), 253);  // biased exponent
                scale = __uint_as_float((uint32_t)(254 - e) << 23);
                back = __uint_as_float((uint32_t)e << 23);
            }
            if (lane == 0) adapter_back(p)[t0 + m] = back;
        }
        uint16_t* out = static_cast<uint16_t*>(p.v) + row + lane;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (32 * i >= p.r) break;
            if (lane + 32 * i >= p.r) continue;
            float u = BF16 ? v[i] : v[i] * scale;
#pragma unroll
            for (int k = 0; k < TERMS; ++k) out[(int64_t)k * p.T * p.r + 32 * i] = take_term<BF16>(u);
        }
    }
    if (p.slices > 1) tc::cluster_sync();  // no CTA leaves while another reads its sums
}

// ---------------------------------------------------------------- the delta alone
// CTA: 16 tokens by 256 features, a warp 64 of them.  Tokens are the MMA's M, so
// that v's fragments serve all 64 features; the features' order over the MMA's
// columns gives a lane four adjacent ones of a pair of column tiles, so y moves
// 16 (fp32) or 8 bytes a lane, and both operands load 16 bytes a lane (32 rank
// values a row) in the same permuted order.  y and the ids are read before the
// wait for v.
template <bool BF16, bool OUT32>
__global__ void __launch_bounds__(128) expand_kernel(const AdapterArgs p) {
    constexpr int TERMS = adapter_terms(BF16), PAIRS = 4;  // pairs of column tiles: 16 features each
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, c = lane & 3;
    const int f0 = (blockIdx.y * 4 + warp) * 16 * PAIRS, t0 = blockIdx.x * 16, n = min(16, p.T - t0);
    if (f0 >= p.N) return;
    int id = lane < n ? __ldg(&p.ids[t0 + lane]) : -1;
    if (id < 0 || id >= p.L) id = -1;
    const uint32_t mine = __match_any_sync(0xffffffffu, id);
    uint32_t todo = __ballot_sync(0xffffffffu, id >= 0);
    // y[pair][h][i]: token gq + 8 h, feature f0 + 16 pair + 4 c + i
    float y[PAIRS][2][4];
#pragma unroll
    for (int t = 0; t < PAIRS; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int f = f0 + 16 * t + 4 * c;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (p.accumulate && gq + 8 * h < n && f < p.N) {
                const int64_t o = (int64_t)(t0 + gq + 8 * h) * p.ldy + f;
                if (OUT32) {
                    v = *reinterpret_cast<const float4*>(static_cast<const float*>(p.y) + o);
                } else {
                    const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.y) + o);
                    const float2 a = unpack2<BF16>(u.x), b = unpack2<BF16>(u.y);
                    v = make_float4(a.x, a.y, b.x, b.y);
                }
            }
            y[t][h][0] = v.x, y[t][h][1] = v.y, y[t][h][2] = v.z, y[t][h][3] = v.w;
        }
    grid_wait();
    const int fl = 4 * (gq >> 1) + (gq & 1);  // column gq of a pair's first tile is this feature, of the second 2 more
    while (todo) {  // one pass per distinct adapter of the 16 tokens
        const int leader = __ffs(todo) - 1;
        const int a = __shfl_sync(0xffffffffu, id, leader);
        const uint32_t used = __shfl_sync(0xffffffffu, mine, leader);
        todo &= ~used;
        const bool use[2] = {((used >> gq) & 1) != 0, ((used >> (8 + gq)) & 1) != 0};
        const uint16_t* B = static_cast<const uint16_t*>(p.b) + ((int64_t)a * p.N + f0 + fl) * p.r + 8 * c;
        const int64_t vrow = (int64_t)(t0 + gq) * p.r + 8 * c;
        float d[2 * PAIRS][4] = {};
        for (int j0 = 0; j0 < p.r; j0 += 32) {
            const bool in = j0 + 8 * c < p.r;
            uint4 v[2][TERMS], w[2 * PAIRS];
#pragma unroll
            for (int t = 0; t < 2 * PAIRS; ++t) {
                const int f = 16 * (t >> 1) + 2 * (t & 1);
                w[t] = load_or_zero(B + (int64_t)f * p.r + j0, in && f0 + fl + f < p.N);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int k = 0; k < TERMS; ++k) {
                    v[h][k] = make_uint4(0, 0, 0, 0);
                    if (in && use[h]) v[h][k] = *reinterpret_cast<const uint4*>(adapter_term(p, k) + vrow + (int64_t)h * 8 * p.r + j0);
                }
#pragma unroll
            for (int k = 0; k < TERMS; ++k) {
                const uint32_t a0[4] = {v[0][k].x, v[1][k].x, v[0][k].y, v[1][k].y};
                const uint32_t a1[4] = {v[0][k].z, v[1][k].z, v[0][k].w, v[1][k].w};
#pragma unroll
                for (int t = 0; t < 2 * PAIRS; ++t) {
                    mma16<BF16>(d[t], a0, w[t].x, w[t].y);
                    mma16<BF16>(d[t], a1, w[t].z, w[t].w);
                }
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (!use[h]) continue;  // (another adapter's infinities must not reach this token)
            const float back = BF16 ? 1.f : adapter_back(p)[t0 + gq + 8 * h];
#pragma unroll
            for (int t = 0; t < PAIRS; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float v = d[2 * t + (i >> 1)][2 * h + (i & 1)];
                    y[t][h][i] = BF16 ? y[t][h][i] + v : fmaf(v, back, y[t][h][i]);
                }
        }
    }
    grid_release();
#pragma unroll
    for (int t = 0; t < PAIRS; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int f = f0 + 16 * t + 4 * c;
            if (gq + 8 * h < n && f < p.N) {
                const int64_t o = (int64_t)(t0 + gq + 8 * h) * p.ldy + f;
                const float* v = y[t][h];
                if (OUT32) *reinterpret_cast<float4*>(static_cast<float*>(p.y) + o) = make_float4(v[0], v[1], v[2], v[3]);
                else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.y) + o) = make_uint2(pack2<BF16>(v[0], v[1]), pack2<BF16>(v[2], v[3]));
            }
        }
}

// ---------------------------------------------------------------- launcher
// A window is 8 tokens while such windows fit the 148 SMs once, else 32.  Small
// windows share a mixed batch's A rows out over more CTAs (512 tokens of 30
// adapters, rank 16, v in two terms: 22 us against 29), large ones read the A rows of a long
// run less often (8192 tokens of one adapter, rank 64, v in two terms: 25 us against 39).
constexpr int kSmallWindowTokens = 148 * 8;

// CTAs that split a window's K: a power of two up to 8, so that the windows'
// CTAs fill the GPU once while each keeps at least 256 of K (as many as run two an
// SM, powers of two or not: 1500 tokens of rank 16, K = 2048, 13.8 us against 9.5).
static int shrink_slices(int T, int K) {
    const int win = T <= kSmallWindowTokens ? 8 : 32, windows = (T + win - 1) / win;
    int s = 1;
    while (s < 8 && windows * s < 148 && 2 * s * 256 <= K) s *= 2;
    return s;
}

size_t adapter_workspace(int T, int r) {
    // the largest form: three 16-bit terms per rank value, and a factor per token
    return (size_t)T * r * 6 + (((size_t)T * 4 + 15) & ~size_t(15));
}

template <bool BF16, int WIN, int TERMS, int TILES>
static cudaError_t shrink_tiles(const AdapterArgs& p, cudaStream_t s) {
    auto kern = (p.K + p.slices - 1) / p.slices > kShrinkPart ? shrink_kernel<BF16, WIN, TERMS, TILES, true>
                                                              : shrink_kernel<BF16, WIN, TERMS, TILES, false>;
    const int smem = ShrinkCfg<WIN, TILES>::kShared + WIN * p.r * 4;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchAttribute at[2] = {};
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 1;
    at[0].val.clusterDim.y = (unsigned)p.slices;
    at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((p.T + WIN - 1) / WIN, p.slices);
    cfg.blockDim = kShrinkThreads;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

// as many rows of A a pass as the rank fills (32 tokens: two tiles leave room for the octets' accumulators)
template <bool BF16, int WIN, int TERMS>
static cudaError_t shrink(const AdapterArgs& p, cudaStream_t s) {
    if (p.r <= 16) return shrink_tiles<BF16, WIN, TERMS, 1>(p, s);
    if constexpr (WIN == 8)
        if (p.r > 32) return shrink_tiles<BF16, WIN, TERMS, 4>(p, s);
    return shrink_tiles<BF16, WIN, TERMS, 2>(p, s);
}

template <bool BF16, bool OUT32>
static cudaError_t adapters(AdapterArgs p, cudaStream_t s) {
    constexpr int kTerms = adapter_terms(BF16);
    p.slices = shrink_slices(p.T, p.K);
    const bool skinny = p.w && p.T <= kSkinnyMaxRows;
    const cudaError_t e = skinny                        ? shrink<BF16, 8, 0>(p, s)
                          : p.T <= kSmallWindowTokens ? shrink<BF16, 8, kTerms>(p, s)
                                                        : shrink<BF16, 32, kTerms>(p, s);
    if (e != cudaSuccess) return e;
    if (skinny) return launch_skinny_adapter(p, BF16, OUT32, s);
    if (p.w) return launch_grouped_adapter(p, BF16, OUT32, s);
    return launch_behind(expand_kernel<BF16, OUT32>, dim3((p.T + 15) / 16, (p.N + 255) / 256), 128, 0, s, p);
}

cudaError_t launch_adapters(const AdapterArgs& p, bool bf16, bool out32, cudaStream_t s) {
    if (bf16) return out32 ? adapters<true, true>(p, s) : adapters<true, false>(p, s);
    return out32 ? adapters<false, true>(p, s) : adapters<false, false>(p, s);
}

}  // namespace moe
