// grouped.cu -- matrix products of ragged row groups with 16-bit matrices
// (tcgen05, pairs of SMs), and their gradients.
//
// Group e owns rows o[e] <= r < o[e+1] and a matrix W_e [N x K]:
//   forward   y[r, n]    = sum_k x[r, k] W_e[n, k]
//   rows      dx[r, k]   = sum_n dy[r, n] W_e[n, k]
//   weights   dW_e[n, k] = sum_r dy[r, n] x[r, k]
// The unquantised counterpart of the expert GEMMs of gemm_sm100.cu: the
// products a token's selected experts are (tech.okbari.net guide, section
// "Strata, Qwen and GSQ-RCO are different components").
//
// One tile is 256 features by up to 256 columns, held by a cluster of two CTAs
// (cta_group::2, M = 256): each CTA stages its own 128 features and half of the
// columns' operand, which halves the column operand's shared-memory traffic per
// SM against one-SM tiles.  For the forward and rows products the features are
// the MMA's M and the group's rows its N (rounded up to 32): a group of few
// rows costs few columns, not a padded 128-row tile.  For the weight gradient
// M is n, N is k and the contraction runs over the group's rows; both operands
// are read MN-major, straight from row-major memory.
//
// Warp roles (every role walks the same tile sequence; persistent):
//   warps 0, 3  loaders (one lane each): TMA of this CTA's half of A and of B
//               into a ring of K = 64 steps, completing on the leader's
//               full[stage]
//   warp 1      MMA issuer (leader CTA, one thread)
//   warp 2      tensor-memory allocation; weight gradient: zeroes the rows of
//               the last step that belong to the next group (a product with
//               zero would let their infinities and NaN through, so both
//               operands are cleared)
//   warps 4-11  (weights: 4-7) epilogue: TMEM -> registers -> shared transpose -> 16-byte
//               stores; two accumulators, so it overlaps the next tile's MMAs
// Every wait is bounded, and covers at most kLongPart steps, or is given their number.
//
// What bounds it, and what it measures: a steady tile takes 530 cycles a K = 64
// step where the tensor pipe alone needs 512, so large groups run at the tensor
// core's rate under the 1000 W cap (64 even groups of 640 rows by 2048 x 768:
// 140 us, a batched library product 140; their weights' gradient at 1536 x 2048:
// 231 to 267 us against 247).  Small groups are bound by reading the matrices:
// 64 tokens' 640 rows over 512 experts of 1536 x 2048 (some 204 in use, 1.29 GB)
// take 190 us, the measured copy's rate; 81920 rows over 512 even ones 590 us, 98%
// of it.  Below about 10 us a call is its start-up: offsets, tensor memory, the
// cluster's barrier and the first load, 3 us each way with up to 64 groups.  Sorting
// the groups by cost compares all pairs of them and grows with their square: the
// weights' gradient of 64 x 64 matrices, two rows a group, takes 5.6 us for 16
// groups, 11 for 128, 49 for 512 and 135 for 1024, a product of 256 rows a group
// 18 us for 64, 36 for 256, 112 for 512 and 326 for 1024 (products of fewer rows a
// group are not sorted: 14 and 25 us for 512 and 1024).  A group's contraction is
// never split: one of 40003 rows by 256 x 256 takes 187 us on one pair of SMs.
#include <cuda.h>
#include <cuda_runtime.h>

#include "adapter.cuh"
#include "common.cuh"
#include "kernels.h"
#include "pack16.cuh"
#include "tc.cuh"

namespace moe {

constexpr int kEpiWarps = 8;  // two for each quarter of the TMEM lanes, taking turns at the columns (weights: one, with two buffers)
constexpr int kGroupedThreads = (4 + kEpiWarps) * 32;
constexpr int kHalfTile = 128 * 128;            // bytes of one CTA's half of an operand, one K = 64 step
constexpr int kPanel = 64 * 128;                // MN-major: 64 contraction rows x 64 values
constexpr int kRowPitch = 36;                   // floats: fp32 rows of 32 features, padded
constexpr int kEpiWarpBytes = 2560;             // epilogue transpose buffer of one warp (16 fp32 rows, or 2 KB)
static_assert(16 * kRowPitch * 4 <= kEpiWarpBytes && kEpiWarpBytes % 512 == 0, "buffer; tile stores need 512-byte starts");
// Ring of (A half, B half): six steps of 256-row tiles, or nine of tiles of at
// most 64 rows, whose B half is a quarter: where groups are that small reading
// the matrices is the cost, and three more steps in flight cover HBM's latency.
constexpr int grouped_stage(bool small) { return kHalfTile + (small ? kHalfTile / 4 : kHalfTile); }
constexpr int grouped_stages(bool small) { return small ? 9 : 6; }
constexpr int grouped_smem(bool small) { return grouped_stages(small) * grouped_stage(small) + kEpiWarps * kEpiWarpBytes + 1024; }
// fp32 results: the tensor core rounds its accumulator towards zero at every
// 16-wide step, an error that grows with the number of steps (measured: 3.5e-5
// relative after 1875 steps), so the contraction is cut into parts of this
// many K = 64 steps, each summed from zero and added in fp32 (round to nearest)
// by the epilogue: 6e-7.  16-bit results round at 2^-9 or 2^-12 and take one part
// up to kLongPart steps (8192 values, whose rounding of equal signs stays under an
// eighth of fp16's half step); longer contractions are summed in parts of that many
// in one accumulator, and the epilogue adds them in fp32 in the other.
constexpr int kPartSteps = 8;
constexpr int kLongPart = 128;
static_assert(grouped_smem(false) + 12 * (kGroupedMaxGroups + 16) <= 227 * 1024, "shared memory");

struct GroupedMaps {
    CUtensorMap a, b, c;  // c: forward and rows, b in 32-row boxes; weights, the result
};

// 16-bit pair in the requested type
MOE_DEV uint32_t pack16(float lo, float hi, bool bf16) { return bf16 ? pack2<true>(lo, hi) : pack2<false>(lo, hi); }

struct GroupedTile {
    int e, row0, n;  // group; first row and rows of the tile (weights: of the group)
    int f0, g0;      // first feature (of the pair); weights: first k column
};

// The tile list.  Forward and rows products cut a group into blocks of equal
// size (at most g.block rows, 256 or less where that fills the GPU; multiples of 32, so that no block is a sliver) and
// enumerate (group, band of blocks, features, block); the weight gradient, with
// 256-wide k columns in the blocks' place, the same.
struct TileList {
    const int* start;  // [E + 1] first row of each group
    const int* pre;    // [E + 1] forward, rows: blocks of the groups before this place
    const int* order;  // [E] group at each place
    int E;
};

// blocks of a group of c rows, and the rows of each
MOE_DEV int block_count(int c, int most) { return (c + most - 1) / most; }
MOE_DEV int block_rows(int c, int most) {
    const int blocks = block_count(c, most);
    return blocks <= 1 ? c : (((c + blocks - 1) / blocks) + 31) & ~31;
}

// Tile t of a group's JT x blocks tiles: bands of 8 blocks, features outside,
// blocks inside.  The tiles in flight then form a square of the product, whose
// two operands L2 holds, whatever the number of features.
MOE_DEV void band(int t, int JT, int blocks, int& jt, int& block) {
    const int b = t / (8 * JT), in = t - b * 8 * JT, height = min(8, blocks - 8 * b);
    jt = in / height;
    block = 8 * b + in - jt * height;
}

template <int MODE>
MOE_DEV GroupedTile tile_at(const GroupedArgs& g, int t, const TileList& l, int JT) {
    GroupedTile r;
    if (MODE == kGroupedWeights) {
        const int KT = (g.C + 255) >> 8, per = JT * KT;
        const int place = t / per;
        int jt, kt;
        band(t - place * per, JT, KT, jt, kt);
        r.e = l.order[place];
        r.f0 = jt << 8;
        r.g0 = kt << 8;
        r.row0 = l.start[r.e];
        r.n = l.start[r.e + 1] - r.row0;
        return r;
    }
    const int q = t / JT;
    r.g0 = 0;
    int lo = 0, hi = l.E - 1;  // last place with pre <= q
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (l.pre[mid] <= q) lo = mid;
        else hi = mid - 1;
    }
    int jt, at;
    band(t - l.pre[lo] * JT, JT, l.pre[lo + 1] - l.pre[lo], jt, at);
    r.f0 = jt << 8;
    r.e = l.order[lo];
    const int c = l.start[r.e + 1] - l.start[r.e], rows = block_rows(c, g.block);
    at *= rows;
    r.row0 = l.start[r.e] + at;
    r.n = min(rows, c - at);
    return r;
}

// The i-th tile of pair p of P, back and forth over the pairs: with costs that
// fall along the list every pair gets about the same sum.
MOE_DEV int tile_index(int i, int p, int P) { return i * P + ((i & 1) ? P - 1 - p : p); }

// Exclusive prefix sum of one value per thread over the CTA, and the total;
// every thread calls it.
MOE_DEV int block_exclusive(int v, int* wsum, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    int before = inc - v;
    total = 0;
#pragma unroll
    for (int w = 0; w < kGroupedThreads / 32; ++w) {
        if (w < warp) before += wsum[w];
        total += wsum[w];
    }
    __syncthreads();  // (wsum may be written again)
    return before;
}

// Adapters (one "group" per run of tokens of one adapter, below): the maps of B
// [L][N][r] and of v's terms [term][T][r], in boxes of 128 and of 32 tokens.
template <bool ADAPT>
struct GroupedExtra {};
template <>
struct GroupedExtra<true> {
    AdapterArgs args;
    CUtensorMap b, v, v_small;
};

// Tokens [row0, row0 + n) whose v's terms are unscaled (fp16; adapter.cuh); a warp.
MOE_DEV bool unscaled(const AdapterArgs& p, int row0, int n) {
    const float* back = adapter_back(p) + row0;
    bool ok = true;
    for (int i = threadIdx.x & 31; i < n; i += 32) ok = ok && back[i] == 1.f;
    return __all_sync(0xffffffffu, ok);
}
MOE_DEV int adapter_of(const AdapterArgs& p, int t) {
    const int id = __ldg(&p.ids[t]);
    return id >= 0 && id < p.L ? id : -1;
}

// The two accumulators' turns, the same for the MMA issuer and the epilogue: each
// part of a contraction takes the other one, but a long tile of a 16-bit result
// (stay) keeps one for all its parts, and the tile after it takes that one once
// more: once it has been drained the epilogue is through with the other too,
// where it holds the parts' sum.
struct AccTurn {
    uint32_t s = 0;  // bit 0: whose turn; 1, 2: parity of each one's uses; 3, 4: whether it has been used
    MOE_DEV uint32_t b() const { return s & 1; }
    MOE_DEV uint32_t parity() const { return (s >> (1 + b())) & 1; }
    MOE_DEV bool used() const { return ((s >> (3 + b())) & 1) != 0; }
    MOE_DEV void next(bool stay) { s = ((s ^ (2u << b())) | (8u << b())) ^ (stay ? 0u : 1u); }
};

template <int MODE, bool OUT32, bool ADAPT, bool SMALL>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGroupedThreads, 1)
    grouped_kernel(const GroupedArgs g, const __grid_constant__ GroupedExtra<ADAPT> ex, const __grid_constant__ CUtensorMap amap,
                   const __grid_constant__ CUtensorMap bmap, const __grid_constant__ CUtensorMap cmap) {
    constexpr bool WG = MODE == kGroupedWeights;
    constexpr int kGroupedStage = grouped_stage(SMALL), kGroupedStages = grouped_stages(SMALL);
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full_bar[kGroupedStages], empty_bar[kGroupedStages], tail_bar[kGroupedStages];
    __shared__ __align__(8) uint64_t accf_bar[2], acce_bar[2];
    __shared__ uint32_t tmem_slot;
    __shared__ int start[kGroupedMaxGroups + 1], pre[WG ? 1 : kGroupedMaxGroups + 1], order[kGroupedMaxGroups];
    __shared__ int wsum[kGroupedThreads / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t rank = tc::cta_rank();
    const int JT = (g.F + 255) >> 8;

    if (tid == 0) {
        for (int i = 0; i < kGroupedStages; ++i) {
            mbar_init(&full_bar[i], 4);
            mbar_init(&empty_bar[i], 1);
            mbar_init(&tail_bar[i], 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&accf_bar[i], 1);
            mbar_init(&acce_bar[i], 2 * (WG ? 4 : kEpiWarps));
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) tc::tmem_alloc_pair(&tmem_slot, 512);
    if (warp == 3 && lane < 3) tc::prefetch_map(lane == 0 ? &amap : lane == 1 ? &bmap : &cmap);

    if (!ADAPT) grid_wait();  // (adapters: W, x and ids are older than the kernel before, which only makes v)
    // (the loops below stay rolled: this part runs once, and its instructions come from memory)
    int E = g.E;
    bool runs = false;  // adapters: every tile has one adapter
    if constexpr (ADAPT) {
        // Groups are the runs of tokens of one adapter (or of none), so that the
        // tensor core can add a tile's delta: worth it while runs are 32 tokens
        // long on average.  Otherwise one group, and the epilogue adds the deltas.
        const int seg = (g.M + kGroupedThreads - 1) / kGroupedThreads;
        const int i0 = min(tid * seg, g.M), i1 = min(i0 + seg, g.M);
        int n = 0, was = i0 > 0 && i0 < i1 ? adapter_of(ex.args, i0 - 1) : -2;
        const int before0 = was;
#pragma unroll 8
        for (int i = i0; i < i1; ++i) {
            const int id = adapter_of(ex.args, i);
            n += id != was;
            was = id;
        }
        int found;
        int at = block_exclusive(n, wsum, found);
        runs = found <= kGroupedMaxGroups && (int64_t)found * 32 <= g.M;
        E = runs ? found : 1;
        if (runs) {
            was = before0;
            for (int i = i0; i < i1; ++i) {
                const int id = adapter_of(ex.args, i);
                if (id != was) start[at++] = i;
                was = id;
            }
        }
        if (tid == 0) {
            if (!runs) start[0] = 0;
            start[E] = g.M;
        }
    } else {
        // Group starts: clamped into [0, rows] and made ascending, so that a bad
        // table reads and writes nothing out of range.
        bool rising = true;
#pragma unroll 1
        for (int e = tid; e < E; e += kGroupedThreads) {
            const int a = min(max(__ldg(&g.offsets[e]), 0), g.M), b = min(max(__ldg(&g.offsets[e + 1]), 0), g.M);
            start[e] = a;
            if (e == E - 1) start[E] = b;
            rising = rising && a <= b;
        }
        if (!__syncthreads_and(rising)) {
            if (tid == 0)
                for (int e = 0; e < E; ++e) start[e + 1] = max(start[e + 1], start[e]);
        }
    }
    __syncthreads();
    // Places by falling tile cost, so that the long tiles come first and the
    // pairs end together.  Where the groups are so small that reading their
    // matrices is the cost (under 256 rows on average), the groups' own order,
    // which mixes short and long tiles and keeps HBM busy throughout.
    const bool sorted = !ADAPT && (WG || start[E] - start[0] >= 256 * E);
    if (sorted) {
        auto key = [&](int e) {
            const int c = start[e + 1] - start[e];
            return WG ? c : block_rows(c, g.block);
        };
#pragma unroll 1
        for (int e = tid; e < E; e += kGroupedThreads) {
            const int mine = key(e);
            int n = 0;
#pragma unroll 1
            for (int o = 0; o < E; ++o) {
                const int k = key(o);
                n += k > mine || (k == mine && o < e);
            }
            order[n] = e;
        }
    } else {
#pragma unroll 1
        for (int e = tid; e < E; e += kGroupedThreads) order[e] = e;
    }
    __syncthreads();
    int total;
    if (WG) {
        total = E * JT * ((g.C + 255) >> 8);
    } else {
        int all = 0;
#pragma unroll 1
        for (int base = 0; base < E; base += kGroupedThreads) {
            const int at = base + tid, e = at < E ? order[at] : 0;
            int sum;
            const int before = block_exclusive(at < E ? block_count(start[e + 1] - start[e], g.block) : 0, wsum, sum);
            if (at < E) pre[at] = all + before;
            all += sum;
        }
        if (tid == 0) pre[E] = all;
        total = all * JT;
    }
    const TileList list{start, pre, order, E};
    tc::fence_before();
    __syncthreads();
    tc::cluster_sync();  // both CTAs' barriers are initialised, both halves of tensor memory allocated
    tc::fence_after();
    const uint32_t tmem = tmem_slot;
    const int pair = (int)blockIdx.x >> 1, pairs = (int)gridDim.x >> 1;
    const int KC = (g.C + 63) >> 6;  // steps per tile (forward, rows)
    // Adapters: steps that add a tile's delta, v's terms times B in 64-wide
    // blocks of the rank; 0 where there is none or the epilogue adds it.  Whole
    // warps.  (fp16: v must be there to see whether it was scaled.)
    int rank_blocks = 0, terms = 0, one_adapter = -1;
    if constexpr (ADAPT) {
        rank_blocks = (ex.args.r + 63) >> 6;
        terms = adapter_terms(g.bf16 != 0);
    }
    auto delta_steps = [&](const GroupedTile& tl) -> int {
        if constexpr (ADAPT) {
            one_adapter = runs ? adapter_of(ex.args, tl.row0) : -1;
            if (one_adapter < 0) return 0;
            if (!g.bf16) {
                grid_wait();
                if (!unscaled(ex.args, tl.row0, tl.n)) return 0;
            }
            return terms * rank_blocks;
        }
        return 0;
    };

    if (warp == 0 || warp == 3) {
        // ======================= loaders (the whole warp walks, one lane issues): warp 0 A, warp 3 B
        const bool is_a = warp == 0, one = tc::elect_one();
        const uint32_t full_leader = tc::cluster_addr(&full_bar[0], 0), tail_own = tc::cluster_addr(&tail_bar[0], rank);
        bool ok = true, filled = false;  // filled: every stage has been used once
        int st = 0;
        uint32_t phase = 1;  // parity of the stage's last "empty" (0 once every stage has been used)
        for (int i = 0, t = pair; t < total && ok; t = tile_index(++i, pair, pairs)) {
            const GroupedTile tl = tile_at<MODE>(g, t, list, JT);
            const int KS = WG ? (tl.n + 63) >> 6 : KC + delta_steps(tl);
            const int nh = WG ? 128 : ((tl.n + 31) & ~31) >> 1;
            const int brow = tl.row0 + (int)rank * nh;
            const int f = tl.f0 + (int)rank * 128, gc = tl.g0 + (int)rank * 128;
            const int nbox = nh > 64 ? 0 : (nh + 31) >> 5;  // 32-row boxes (0: one of 128 rows)
            const uint32_t bytes = is_a || WG || nbox == 0 ? kHalfTile : nbox * 32 * 128;
            for (int s = 0; s < KS; ++s) {
                if (filled) ok = tc::bar_wait(&empty_bar[st], phase, g.status);
                if (!ok) break;
                uint8_t* As = smem + st * kGroupedStage;
                uint8_t* Bs = As + kHalfTile;
                // a last step that ends inside 16 rows is completed by warp 2 once it is cleared
                const bool tail = WG && s == KS - 1 && (tl.n & 15);
                const uint32_t bar = (tail ? tail_own : full_leader) + (uint32_t)st * 8u;
                if (ADAPT && s == KC) {
                    grid_wait();  // v, from the kernel before
                    fence_proxy_async_global();
                }
                if (one) {
                    if (tail) mbar_arrive_expect_tx(&tail_bar[st], bytes);
                    else tc::arrive_expect_cluster(bar, bytes);
                    if (WG) {
                        const int r = tl.row0 + s * 64;
                        if (is_a) {
                            tc::tma_2d_pair(As, &amap, f, r, bar);
                            tc::tma_2d_pair(As + kPanel, &amap, f + 64, r, bar);
                        } else {
                            tc::tma_2d_pair(Bs, &bmap, gc, r, bar);
                            tc::tma_2d_pair(Bs + kPanel, &bmap, gc + 64, r, bar);
                        }
                    } else if (ADAPT && s >= KC) {
                        if constexpr (ADAPT) {
                            const int term = (s - KC) / rank_blocks, j = (s - KC) % rank_blocks * 64;
                            if (is_a) tc::tma_3d_pair(As, &ex.b, j, f, one_adapter, bar);
                            else if (nbox == 0) tc::tma_3d_pair(Bs, &ex.v, j, brow, term, bar);
                            else
                                for (int x = 0; x < nbox; ++x)
                                    tc::tma_3d_pair(Bs + x * 32 * 128, &ex.v_small, j, brow + x * 32, term, bar);
                        }
                    } else if (is_a) {
                        if (MODE == kGroupedForward) {
                            tc::tma_3d_pair(As, &amap, s * 64, f, ADAPT ? 0 : tl.e, bar);  // (adapters: one W)
                        } else {
                            tc::tma_3d_pair(As, &amap, f, s * 64, tl.e, bar);
                            tc::tma_3d_pair(As + kPanel, &amap, f + 64, s * 64, tl.e, bar);
                        }
                    } else {
                        if (nbox == 0) tc::tma_2d_pair(Bs, &bmap, s * 64, brow, bar);
                        else
                            for (int x = 0; x < nbox; ++x)
                                tc::tma_2d_pair(Bs + x * 32 * 128, &cmap, s * 64, brow + x * 32, bar);
                    }
                }
                __syncwarp();
                if (++st == kGroupedStages) {
                    st = 0;
                    phase ^= 1;
                    filled = true;
                }
            }
        }
        grid_release();  // (late: the next kernel's CTAs then find most SMs free, not the first few)
        if (!ok) tc::settle();
    } else if (warp == 1) {
        if (rank == 0) {
            // ======================= MMA issuer (the whole warp walks, one lane issues)
            const bool one = tc::elect_one();
            // descriptors of stage 0, A and B; a stage or a 16-wide step further is an addition to the address
            const uint32_t a0 = smem_addr(smem), b0 = a0 + kHalfTile;
            const uint64_t adesc = MODE == kGroupedForward ? tc::sdesc(a0) : tc::sdesc_mn(a0, kPanel);
            const uint64_t bdesc = WG ? tc::sdesc_mn(b0, kPanel) : tc::sdesc(b0);
            constexpr uint32_t kA16 = (MODE == kGroupedForward ? 32 : 2048) >> 4, kB16 = (WG ? 2048 : 32) >> 4;
            bool ok = true;
            int st = 0;
            AccTurn turn;
            uint32_t phase = 0;
            for (int i = 0, t = pair; t < total && ok; t = tile_index(++i, pair, pairs)) {
                const GroupedTile tl = tile_at<MODE>(g, t, list, JT);
                const int KS = WG ? (tl.n + 63) >> 6 : KC + delta_steps(tl);
                const uint32_t idesc = tc::idesc_f16_major(256, WG ? 256 : (tl.n + 31) & ~31, g.bf16 != 0,
                                                           MODE != kGroupedForward, WG);
                const bool stay = !OUT32 && KS > kLongPart;
                for (int s = 0; s < KS; ++s) {
                    constexpr int kPart = OUT32 ? kPartSteps : kLongPart;
                    const int ps = s % kPart;
                    if (ps == 0 && turn.used()) {  // a new part: the accumulator, once the epilogue has drained it
                        ok = tc::bar_wait(&acce_bar[turn.b()], turn.parity() ^ 1, g.status);
                        if (!ok) break;
                    }
                    ok = tc::bar_wait(&full_bar[st], phase, g.status);
                    if (!ok) break;
                    tc::fence_after();
                    const uint32_t acc = tmem + turn.b() * 256;
                    const uint64_t ad = adesc + (uint32_t)(st * (kGroupedStage >> 4)), bd = bdesc + (uint32_t)(st * (kGroupedStage >> 4));
                    int kks = WG && s == KS - 1 ? (tl.n - s * 64 + 15) >> 4 : 4;
                    if constexpr (ADAPT) {
                        if (s >= KC) kks = (min(64, ex.args.r - (s - KC) % rank_blocks * 64) + 15) >> 4;
                    }
                    const bool done = s == KS - 1 || ps == kPart - 1;
                    if (one) {
                        tc::mma_pair(acc, ad, bd, idesc, ps > 0 ? 1u : 0u);
#pragma unroll
                        for (int kk = 1; kk < 4; ++kk)
                            if ((!WG && !ADAPT) || kk < kks) tc::mma_pair(acc, ad + kk * kA16, bd + kk * kB16, idesc, 1u);
                        tc::commit_pair(&empty_bar[st]);
                        if (done) tc::commit_pair(&accf_bar[turn.b()]);
                    }
                    __syncwarp();
                    if (done) turn.next(stay);
                    if (++st == kGroupedStages) {
                        st = 0;
                        phase ^= 1;
                    }
                }
            }
            if (!ok) tc::settle();
        }
    } else if (WG && warp == 2) {
        // ======================= rows of a group's last step that are not its own
        bool ok = true;
        int j = 0;
        uint32_t phases = 0;  // per stage: parity of its next cleared step
        for (int i = 0, t = pair; t < total && ok; t = tile_index(++i, pair, pairs)) {
            const GroupedTile tl = tile_at<MODE>(g, t, list, JT);
            const int KS = (tl.n + 63) >> 6;
            j += KS;
            if (!(tl.n & 15)) continue;
            const int st = (j - 1) % kGroupedStages;
            ok = true;
            // (the whole contraction passes before its last step: one limit, 0.5 s, more for every 65536 steps, 18 ms)
            if (lane == 0) ok = tc::bar_wait(&tail_bar[st], (phases >> st) & 1, g.status, 1 + (KS >> 16));
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
            if (!ok) break;
            phases ^= 1u << st;
            const int r0 = tl.n - (KS - 1) * 64, nz = ((r0 + 15) & ~15) - r0;
            // 4 panels x 8 pieces: a row a turn
            uint8_t* base = smem + st * kGroupedStage + (lane >> 3) * kPanel + r0 * 128 + (lane & 7) * 16;
            for (int i = 0; i < nz; ++i) *reinterpret_cast<uint4*>(base + i * 128) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tc::arrive_cluster(tc::cluster_addr(&full_bar[st], 0), 2);  // for both loaders
        }
    } else if (warp >= 4 && (!WG || warp < 8)) {
        // ======================= epilogue: lane = feature, register = column
        const int q = warp & 3, turn = (warp - 4) >> 2;
        uint8_t* stg = smem + kGroupedStages * kGroupedStage + (warp - 4) * (WG ? 2 : 1) * kEpiWarpBytes;
        const bool one = tc::elect_one();
        bool ok = true;
        AccTurn acc;
        uint32_t stores = 0;  // weights: tile stores issued; their number, not the column, says whose turn a buffer is
        const bool bf16 = g.bf16 != 0;
        if (ADAPT) grid_wait();  // v, from the kernel before
        for (int i = 0, t = pair; t < total && ok; t = tile_index(++i, pair, pairs)) {
            const GroupedTile tl = tile_at<MODE>(g, t, list, JT);
            const bool empty = WG && tl.n == 0;
            if (empty && g.accumulate) continue;
            const int KS = WG ? (tl.n + 63) >> 6 : KC + delta_steps(tl);
            const bool by_hand = ADAPT && KS == KC && (!runs || one_adapter >= 0);  // deltas to add here
            constexpr int kPart = OUT32 ? kPartSteps : kLongPart;
            const int parts = empty ? 1 : (KS + kPart - 1) / kPart;
            for (int part = 0; part < parts; ++part) {
                const uint32_t b = acc.b();
                const bool add = OUT32 && (part > 0 || g.accumulate);
                if (!empty) {
                    if (lane == 0) ok = tc::bar_wait(&accf_bar[b], acc.parity(), g.status);
                    ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
                    if (!ok) break;
                    acc.next(!OUT32 && parts > 1);
                    tc::fence_after();
                }
                const uint32_t tb = tmem + ((uint32_t)(32 * q) << 16) + b * 256;
                const int f = tl.f0 + (int)rank * 128 + 32 * q;  // the warp's first feature
                if (!OUT32 && parts > 1) {
                    // A part of a long contraction: the sum so far is in the other accumulator's columns of this
                    // warp, which it has read before (the MMAs leave them alone until this tile's last part is
                    // drained).  The last part's sum goes back where the code below reads it
                    const uint32_t other = tb ^ 256u, to = part == parts - 1 ? tb : other;
                    const int most = WG ? min(256, g.C - tl.g0) : tl.n, step = WG ? 32 : 64;
                    for (int c0 = WG ? 0 : 32 * turn; c0 < most; c0 += step)
#pragma unroll
                        for (int h = 0; h < 32; h += 16) {
                            uint32_t v[16], sum[16];
                            tc::ld16_nowait(tb + c0 + h, v);
                            if (part > 0) tc::ld16_nowait(other + c0 + h, sum);
                            tc::ld_wait();
                            if (part > 0)
#pragma unroll
                                for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(sum[i]));
                            tc::st16(to + c0 + h, v);
                        }
                    tc::st_wait();
                    if (part < parts - 1) {
                        tc::fence_before();
                        __syncwarp();
                        if (lane == 0) tc::arrive_cluster_relaxed(tc::cluster_addr(&acce_bar[b], 0));
                        continue;
                    }
                }
                if (!WG) {
                    // 32 rows at a time.  TMEM is read as warp-MMA fragments, so an adapter's delta is added in
                    // registers; 16-bit results are packed in pairs and transposed by stmatrix into [row][32
                    // features] (16-byte pieces permuted against bank conflicts), then leave as whole pieces of
                    // the rows
                    const int seg = lane & 3, vr = lane >> 2;
                    const bool in = f + seg * 8 < g.F;
                    const int64_t at = (int64_t)tl.row0 * g.ldo + f;
                    // stmatrix: this lane's row of matrix lane / 8: token, 16-byte piece
                    const int mrow = (lane & 7) + 8 * (lane >> 4), mpiece = (lane >> 3) & 1;
                    uint32_t r[2][16];  // [16 features][fragment of 8 rows]
                    if (32 * turn < tl.n) {
                        tc::ld_frags_nowait(tb + 32 * turn, r[0]);
                        tc::ld_frags_nowait(tb + (16u << 16) + 32 * turn, r[1]);
                        tc::ld_wait();
                    }
                    for (int c0 = 32 * turn; c0 < tl.n; c0 += 64) {
                        if constexpr (ADAPT) {
                            if (by_hand && part == (OUT32 ? 0 : parts - 1))
#pragma unroll
                                for (int h = 0; h < 2; ++h)
                                    if (c0 + 16 * h < tl.n) {
                                        const int t0 = tl.row0 + c0 + 16 * h, left = tl.n - c0 - 16 * h;
                                        const int skip = h ? 48 : 16;  // to the warp's next 16 rows
                                        const int m = min(16, left), mn = min(16, left - skip);
                                        if (bf16) add_delta<true>(ex.args, t0, m, t0 + skip, mn, f, &r[0][8 * h], &r[1][8 * h]);
                                        else add_delta<false>(ex.args, t0, m, t0 + skip, mn, f, &r[0][8 * h], &r[1][8 * h]);
                                    }
                        }
                        if (ADAPT && !OUT32 && g.accumulate) {  // y's values, added before the one rounding
                            const uint16_t* y = static_cast<const uint16_t*>(g.out) + at + (int64_t)c0 * g.ldo;
#pragma unroll
                            for (int m = 0; m < 2; ++m)
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    const int row = 8 * (i >> 2) + 2 * (lane & 3) + (i & 1);
                                    const int ff = 16 * m + (lane >> 2) + 8 * ((i >> 1) & 1);
                                    if (c0 + row < tl.n && f + ff < g.F) {
                                        const uint16_t was = y[(int64_t)row * g.ldo + ff];
                                        r[m][i] = __float_as_uint(__uint_as_float(r[m][i]) +
                                                                  (bf16 ? unpack1<true>(was) : unpack1<false>(was)));
                                    }
                                }
                        }
                        const bool more = c0 + 64 < tl.n;
                        if (OUT32) {
                            // 16 rows at a time through shared memory (rows of 32 features, padded against bank
                            // conflicts), 16 bytes a lane.  Later parts are added in L2, no old value is waited
                            // for: one lane owns an address, so its additions keep their order
                            const int fr = lane >> 3, fs = (lane & 7) * 4;
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                if (c0 + 16 * h >= tl.n) break;
                                float* buf = reinterpret_cast<float*>(stg);
                                __syncwarp();  // the last 16 rows have been read
#pragma unroll
                                for (int m = 0; m < 2; ++m)
#pragma unroll
                                    for (int i = 0; i < 8; ++i)
                                        buf[(8 * (i >> 2) + 2 * (lane & 3) + (i & 1)) * kRowPitch + 16 * m + (lane >> 2) +
                                            8 * ((i >> 1) & 1)] = __uint_as_float(r[m][8 * h + i]);
                                __syncwarp();
#pragma unroll
                                for (int q4 = 0; q4 < 4; ++q4) {
                                    const int row = c0 + 16 * h + 4 * q4 + fr;
                                    if (row < tl.n && f + fs < g.F) {
                                        const float4 v = *reinterpret_cast<const float4*>(buf + (4 * q4 + fr) * kRowPitch + fs);
                                        float* dst = static_cast<float*>(g.out) + at + (int64_t)row * g.ldo + fs;
                                        if (add) tc::add_global4(dst, v);
                                        else *reinterpret_cast<float4*>(dst) = v;
                                    }
                                }
                            }
                            if (more) {
                                tc::ld_frags_nowait(tb + c0 + 64, r[0]);
                                tc::ld_frags_nowait(tb + (16u << 16) + c0 + 64, r[1]);
                                tc::ld_wait();
                            }
                        } else {
                            uint8_t* buf = stg;
                            __syncwarp();  // the last 32 rows have been read
#pragma unroll
                            for (int m = 0; m < 2; ++m)
#pragma unroll
                                for (int n = 0; n < 4; n += 2) {
                                    const uint32_t* v = &r[m][4 * n];
                                    const int token = 8 * n + mrow, piece = 2 * m + mpiece;
                                    tc::stmatrix4_trans(smem_addr(buf) + token * 64 + ((piece ^ ((token >> 1) & 3)) << 4),
                                                        pack16(__uint_as_float(v[0]), __uint_as_float(v[1]), bf16),
                                                        pack16(__uint_as_float(v[2]), __uint_as_float(v[3]), bf16),
                                                        pack16(__uint_as_float(v[4]), __uint_as_float(v[5]), bf16),
                                                        pack16(__uint_as_float(v[6]), __uint_as_float(v[7]), bf16));
                                }
                            if (more) {  // in flight while this block leaves
                                tc::ld_frags_nowait(tb + c0 + 64, r[0]);
                                tc::ld_frags_nowait(tb + (16u << 16) + c0 + 64, r[1]);
                            }
                            __syncwarp();
                            uint16_t* out = static_cast<uint16_t*>(g.out) + at + seg * 8;
#pragma unroll
                            for (int p = 0; p < 4; ++p) {
                                const int row = 8 * p + vr;
                                if (in && c0 + row < tl.n) {
                                    const uint4 v = *reinterpret_cast<const uint4*>(buf + row * 64 + ((seg ^ ((row >> 1) & 3)) << 4));
                                    uint4* dst = reinterpret_cast<uint4*>(out + (int64_t)(c0 + row) * g.ldo);
                                    *dst = v;
                                }
                            }
                            if (more) tc::ld_wait();
                        }
                    }
                } else {
                    // 32 features x 64 bytes at a time, through two swizzled buffers and tile stores (which
                    // clip at the matrix's edges).  The buffers take turns across tiles too: after the wait
                    // for all stores but the last, that last one reads the other buffer, whatever number of
                    // blocks a tile has.  Later parts, and MOE_ACCUMULATE, are added in L2 by the
                    // store itself, each part once the one before has landed: a fixed order of additions
                    constexpr int kCols = OUT32 ? 16 : 32;
                    if (part > 0) {
                        if (one) tc::store_wait_done();
                        __syncwarp();
                    }
                    if (f < g.F) {
                        uint32_t r[kCols];
                        auto load = [&](int c0) {
#pragma unroll
                            for (int h = 0; h < kCols; h += 16)
                                tc::ld16_nowait(tb + c0 + h, *reinterpret_cast<uint32_t(*)[16]>(&r[h]));
                        };
                        if (!empty) load(0);
                        for (int c0 = 0; c0 < 256 && tl.g0 + c0 < g.C; c0 += kCols) {
                            uint8_t* buf = stg + (stores++ & 1) * kEpiWarpBytes;
                            if (one) tc::store_wait_read<1>();
                            if (!empty) tc::ld_wait();
                            __syncwarp();
#pragma unroll
                            for (int p = 0; p < 4; ++p) {  // 16-byte pieces of the lane's row
                                uint4 v = make_uint4(0, 0, 0, 0);
                                if (!empty) {
                                    if (OUT32) {
                                        v = make_uint4(r[4 * p], r[4 * p + 1], r[4 * p + 2], r[4 * p + 3]);
                                    } else {
                                        uint32_t w[4];
#pragma unroll
                                        for (int i = 0; i < 4; ++i)
                                            w[i] = pack16(__uint_as_float(r[(8 * p + 2 * i) % kCols]),
                                                          __uint_as_float(r[(8 * p + 2 * i + 1) % kCols]), bf16);
                                        v = make_uint4(w[0], w[1], w[2], w[3]);
                                    }
                                }
                                *reinterpret_cast<uint4*>(buf + lane * 64 + ((p ^ ((lane >> 1) & 3)) << 4)) = v;
                            }
                            if (!empty && c0 + kCols < 256) load(c0 + kCols);  // in flight while this block leaves
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (one) {
                                if (add) tc::add_3d(&cmap, tl.g0 + c0, f, tl.e, buf);
                                else tc::store_3d(&cmap, tl.g0 + c0, f, tl.e, buf);
                                tc::store_commit();
                            }
                        }
                        if (!empty) tc::ld_wait();
                    }
                }
                if (!empty) {
                    tc::fence_before();
                    __syncwarp();
                    // (relaxed: the accumulator has been read into registers, and the release of the
                    // stores above, which no one waits for here, would take ~700 cycles)
                    if (lane == 0) tc::arrive_cluster_relaxed(tc::cluster_addr(&acce_bar[b], 0));
                }
            }
        }
        if (WG && one) tc::store_wait_done();
        if (!ok) tc::settle();
    }
    tc::fence_before();
    __syncthreads();
    tc::cluster_sync();  // neither CTA leaves while the other may still signal it or read its operands
    tc::fence_after();
    if (warp == 2) tc::tmem_dealloc_pair(tmem, 512);
}

// ---------------------------------------------------------------- launcher
static int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 148;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 148;
    return sms;
}

// Rows per block: 256, less where that leaves SMs without a tile (a matrix read
// by more blocks comes from L2).
static int block_limit(int rows, int features) {
    const int64_t JT = (features + 255) / 256, pairs = sm_count() / 2;
    const int64_t even = (rows * JT / pairs + 31) / 32 * 32;
    return (int)(even < 32 ? 32 : even > 256 ? 256 : even);
}

// map of a row-major 16-bit matrix [rows x cols], rows `ld` values apart; boxes of 64 columns x box_rows
static Elem elem16(bool bf16) { return bf16 ? Elem::kBf16 : Elem::kFp16; }
static cudaError_t map_2d(CUtensorMap* m, bool bf16, const void* base, int64_t rows, int64_t cols, int64_t ld,
                          int box_rows) {
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, str[1] = {(cuuint64_t)ld * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
    return encode_tiles(m, elem16(bf16), base, 2, dims, str, box, 128);
}

template <int MODE, bool OUT32, bool SMALL>
static cudaError_t grouped_launch(const GroupedArgs& g, const GroupedMaps& m, int64_t most_tiles, cudaStream_t s) {
    auto kern = grouped_kernel<MODE, OUT32, false, SMALL>;
    constexpr int smem = grouped_smem(SMALL);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int pairs = (int)(most_tiles < sm_count() / 2 ? most_tiles : sm_count() / 2);
    return launch_behind(kern, 2 * pairs, kGroupedThreads, smem, s, g, GroupedExtra<false>{}, m.a, m.b, m.c);
}

// maps of the forward and rows products: W as [E][N][K], whose rows (forward) or columns are the features
static cudaError_t product_maps(GroupedMaps* m, bool forward, bool bf, int E, int N, int K, const void* w,
                                const void* rows, int64_t M, int64_t ld) {
    const cuuint64_t dims[3] = {(cuuint64_t)K, (cuuint64_t)N, (cuuint64_t)E};
    const cuuint64_t str[2] = {(cuuint64_t)K * 2, (cuuint64_t)N * K * 2};
    const cuuint32_t box[3] = {64, forward ? 128u : 64u, 1};
    cudaError_t e = encode_tiles(&m->a, elem16(bf), w, 3, dims, str, box, 128);
    if (e == cudaSuccess) e = map_2d(&m->b, bf, rows, M, forward ? K : N, ld, 128);
    if (e == cudaSuccess) e = map_2d(&m->c, bf, rows, M, forward ? K : N, ld, 32);
    return e;
}

template <bool OUT32, bool SMALL>
static cudaError_t adapter_launch(const AdapterArgs& p, bool bf16, cudaStream_t s) {
    GroupedMaps m;
    cudaError_t e = product_maps(&m, true, bf16, 1, p.N, p.K, p.w, p.x, p.T, p.ldx);
    if (e != cudaSuccess) return e;
    GroupedArgs g{};
    g.E = 1;
    g.M = p.T;
    g.F = p.N;
    g.C = p.K;
    g.out = p.y;
    g.ldo = p.ldy;
    g.bf16 = bf16 ? 1 : 0;
    g.accumulate = p.accumulate;
    g.status = p.status;
    g.block = block_limit(p.T, p.N);
    GroupedExtra<true> ex;
    ex.args = p;
    {
        const cuuint64_t bd[3] = {(cuuint64_t)p.r, (cuuint64_t)p.N, (cuuint64_t)p.L};
        const cuuint64_t bs[2] = {(cuuint64_t)p.r * 2, (cuuint64_t)p.N * p.r * 2};
        const cuuint64_t vd[3] = {(cuuint64_t)p.r, (cuuint64_t)p.T, (cuuint64_t)adapter_terms(bf16)};
        const cuuint64_t vs[2] = {(cuuint64_t)p.r * 2, (cuuint64_t)p.T * p.r * 2};
        const cuuint32_t big[3] = {64, 128, 1}, small[3] = {64, 32, 1};
        e = encode_tiles(&ex.b, elem16(bf16), p.b, 3, bd, bs, big, 128);
        if (e == cudaSuccess) e = encode_tiles(&ex.v, elem16(bf16), p.v, 3, vd, vs, big, 128);
        if (e == cudaSuccess) e = encode_tiles(&ex.v_small, elem16(bf16), p.v, 3, vd, vs, small, 128);
        if (e != cudaSuccess) return e;
    }
    auto kern = grouped_kernel<kGroupedForward, OUT32, true, SMALL>;
    constexpr int smem = grouped_smem(SMALL);
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    // (runs cut blocks off: at most one block more per run of 32 tokens)
    const int64_t tiles = (int64_t)((p.T + g.block - 1) / g.block + p.T / 32) * ((p.N + 255) / 256);
    const int pairs = (int)(tiles < sm_count() / 2 ? tiles : sm_count() / 2);
    return launch_behind(kern, 2 * pairs, kGroupedThreads, smem, s, g, ex, m.a, m.b, m.c);
}

cudaError_t launch_grouped_adapter(const AdapterArgs& p, bool bf16, bool out32, cudaStream_t s) {
    if (block_limit(p.T, p.N) <= 64)
        return out32 ? adapter_launch<true, true>(p, bf16, s) : adapter_launch<false, true>(p, bf16, s);
    return out32 ? adapter_launch<true, false>(p, bf16, s) : adapter_launch<false, false>(p, bf16, s);
}

cudaError_t launch_grouped(int mode, const GroupedArgs& args, const void* w, const void* x, int64_t ldx, const void* dy,
                           int64_t lddy, bool out_fp32, cudaStream_t s) {
    GroupedMaps m{};
    GroupedArgs g = args;
    g.block = block_limit(g.M, g.F);
    const bool bf = g.bf16 != 0;
    cudaError_t e;
    const int JT = (g.F + 255) / 256;
    if (mode == kGroupedWeights) {
        e = map_2d(&m.a, bf, dy, g.M, g.F, lddy, 64);
        if (e == cudaSuccess) e = map_2d(&m.b, bf, x, g.M, g.C, ldx, 64);
        const int bytes = out_fp32 ? 4 : 2;
        const cuuint64_t dims[3] = {(cuuint64_t)g.C, (cuuint64_t)g.F, (cuuint64_t)g.E};
        const cuuint64_t str[2] = {(cuuint64_t)g.C * bytes, (cuuint64_t)g.F * g.C * bytes};
        const cuuint32_t box[3] = {(cuuint32_t)(64 / bytes), 32, 1};
        if (e == cudaSuccess) e = encode_tiles(&m.c, out_fp32 ? Elem::kFp32 : elem16(bf), g.out, 3, dims, str, box, 64);
        if (e != cudaSuccess) return e;
        const int64_t tiles = (int64_t)g.E * JT * ((g.C + 255) / 256);
        return out_fp32 ? grouped_launch<kGroupedWeights, true, false>(g, m, tiles, s)
                        : grouped_launch<kGroupedWeights, false, false>(g, m, tiles, s);
    }
    const bool forward = mode == kGroupedForward;
    // Few rows: the warp-MMA kernel while the tiles would not give every pair of SMs one, which costs the
    // tensor-core kernel its start-up and leaves SMs idle (64 rows of one 2048 x 2048 matrix: 6.9 us against
    // 12.5; of 64 such matrices: 78 us against 58, its CTAs living too short for HBM).
    if (forward && g.M <= kSkinnyMaxRows && (g.E < g.M ? g.E : g.M) * JT < sm_count() / 2)
        return launch_skinny_grouped(g, w, x, ldx, out_fp32, s);
    e = product_maps(&m, forward, bf, g.E, forward ? g.F : g.C, forward ? g.C : g.F, w, forward ? x : dy, g.M,
                     forward ? ldx : lddy);
    if (e != cudaSuccess) return e;
    const int64_t tiles = ((int64_t)(g.M + g.block - 1) / g.block + (g.E < g.M ? g.E : g.M)) * JT;
    const bool small = g.block <= 64;
    if (forward) {
        if (small) return out_fp32 ? grouped_launch<kGroupedForward, true, true>(g, m, tiles, s)
                                   : grouped_launch<kGroupedForward, false, true>(g, m, tiles, s);
        return out_fp32 ? grouped_launch<kGroupedForward, true, false>(g, m, tiles, s)
                        : grouped_launch<kGroupedForward, false, false>(g, m, tiles, s);
    }
    if (small) return out_fp32 ? grouped_launch<kGroupedRows, true, true>(g, m, tiles, s)
                               : grouped_launch<kGroupedRows, false, true>(g, m, tiles, s);
    return out_fp32 ? grouped_launch<kGroupedRows, true, false>(g, m, tiles, s)
                    : grouped_launch<kGroupedRows, false, false>(g, m, tiles, s);
}

}  // namespace moe
