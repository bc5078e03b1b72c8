// skinny.cu -- products of few rows with 16-bit matrices: every matrix value is
// read once from HBM, straight into the registers of a warp-level MMA.
//
// One CTA: 16 features of one matrix by the (at most 64) rows that use it; its
// eight warps split K.  Features are the MMA's M, rows its N in blocks of 8;
// both operands load 16 bytes a lane in the same permuted order of k, so no
// shared memory sits between HBM and the tensor core and no padded row tile is
// computed.  The warps' sums meet in shared memory in warp order
// (deterministic).  Bound by HBM, 2 N K bytes per matrix, and by the latency of
// a CTA's few loads: ten rows of ten 1536 x 2048 matrices take 13.8 us, 70% of
// the measured copy; one row-block of 64 rows by 2048 x 2048 6.9 us.  With 17 to
// 64 rows and two CTAs an SM the eight row blocks do not fit 128 registers: 300
// bytes a thread are read back from local memory (8 matrices by 64 rows 14.5 us).
//
// Grouped form: a CTA finds the group it works for in the offsets (one round of
// loads and a prefix count of those that hold rows), so no list of groups is
// built beforehand.  Adapter form: one matrix, then the tokens' deltas.
#include <cuda_runtime.h>

#include "common.cuh"
#include "kernels.h"
#include "pack16.cuh"

namespace moe {

constexpr int kSkinnyThreads = 256;

struct SkinnyArgs {
    const void* w;       // [groups x F x K]
    const void* x;       // rows, pitch ldx
    int64_t ldx;
    int F, K;
    const int32_t* offsets;  // grouped form
    int E, M;
    void* y;
    int64_t ldy;
    AdapterArgs ad;      // adapter form
};

// A warp MMA rounds its accumulator towards zero at each step, like the tensor
// core's tiles (grouped.cu), so a warp's sum is cut into parts of this many values,
// added in fp32 in the place in shared memory where the warps' sums meet.  A warp's
// share of K is an eighth, so up to K = 4096 there is one part, and a kernel that
// looks for none (LONG false; K = 2048: 64 rows of one matrix 6.9 us, 7.25 looking;
// one token's product 13.8 and 14.0).  K = 2^17, values of one sign: 7.6e-5 off in
// one part, 3e-7 in parts.
constexpr int kSkinnyPart = 512;

template <bool BF16, int NB, bool LONG>
MOE_DEV void skinny_sums(const uint16_t* w0, const uint16_t* w1, const uint16_t* x, int64_t ldx, int n, int kb, int ke,
                         float* red, int pitch) {
    const int lane = threadIdx.x & 31, gq = lane >> 2, c = lane & 3;
    float acc[NB][4] = {};
    const uint16_t* xr[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) xr[b] = x + (int64_t)min(b * 8 + gq, n - 1) * ldx + 8 * c;
    w0 += 8 * c;
    w1 += 8 * c;
    constexpr int U = NB <= 2 ? 8 : 4;  // 32-wide steps in flight
    uint4 lo[U], hi[U];
    auto multiply = [&](int u, const uint4 (&bv)[NB]) {
        const uint32_t f0[4] = {lo[u].x, hi[u].x, lo[u].y, hi[u].y}, f1[4] = {lo[u].z, hi[u].z, lo[u].w, hi[u].w};
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            mma16<BF16>(acc[b], f0, bv[b].x, bv[b].y);
            mma16<BF16>(acc[b], f1, bv[b].z, bv[b].w);
        }
    };
    auto each = [&](auto use) {  // this lane's sums, [feature][row]
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            use(red[gq * pitch + b * 8 + 2 * c], acc[b][0]);
            use(red[gq * pitch + b * 8 + 2 * c + 1], acc[b][1]);
            use(red[(gq + 8) * pitch + b * 8 + 2 * c], acc[b][2]);
            use(red[(gq + 8) * pitch + b * 8 + 2 * c + 1], acc[b][3]);
        }
    };
    int k0 = kb, part = kb;  // part: where the part in acc began
    for (; k0 + 32 * U <= ke; k0 += 32 * U) {
        if (LONG && k0 - part == kSkinnyPart) {
            if (part == kb) each([](float& sum, float& a) { sum = a; a = 0.f; });
            else each([](float& sum, float& a) { sum += a; a = 0.f; });
            part = k0;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            lo[u] = __ldcs(reinterpret_cast<const uint4*>(w0 + k0 + 32 * u));
            hi[u] = __ldcs(reinterpret_cast<const uint4*>(w1 + k0 + 32 * u));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            uint4 bv[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b) bv[b] = __ldg(reinterpret_cast<const uint4*>(xr[b] + k0 + 32 * u));
            multiply(u, bv);
        }
    }
    if (k0 < ke) {  // the rest, zeros past the end
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool in = k0 + 32 * u + 8 * c < ke;
            lo[u] = load_or_zero(w0 + k0 + 32 * u, in);
            hi[u] = load_or_zero(w1 + k0 + 32 * u, in);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (k0 + 32 * u >= ke) break;
            uint4 bv[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b) bv[b] = load_or_zero(xr[b] + k0 + 32 * u, k0 + 32 * u + 8 * c < ke);
            multiply(u, bv);
        }
    }
    if (LONG && part != kb) each([](float& sum, float& a) { sum += a; });
    else each([](float& sum, float& a) { sum = a; });
}

// MAXNB: blocks of 8 rows that a group can have (the call's rows, rounded up).
// PER_SM: CTAs an SM must hold; one, where there is no second, leaves registers
// for all of x's loads in flight.
template <bool BF16, bool OUT32, bool ADAPT, bool LONG, int MAXNB, int PER_SM = 2>
__global__ void __launch_bounds__(kSkinnyThreads, PER_SM) skinny_kernel(const SkinnyArgs p) {
    constexpr int kPitch = 8 * MAXNB + 1;
    __shared__ __align__(16) float red[8][16 * kPitch];
    __shared__ int found[3], counts[8];
    if (!ADAPT) grid_wait();  // (adapters: W, x and ids are older than the kernel before, which only makes v)
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2;
    int e = 0, row0 = 0, n = ADAPT ? p.ad.T : 0;
    if (!ADAPT) {
        // this CTA's group: the blockIdx.y-th that holds rows (a thread looks at up to four)
        constexpr int kMost = kGroupedMaxGroups / kSkinnyThreads;
        const int each = (p.E + kSkinnyThreads - 1) / kSkinnyThreads, first = tid * each;
        int lo[kMost], hi[kMost], mine = 0;
        constexpr int kFalls = 1 << 16;  // added, above the counts, where an offset is below the one before it
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
            lo[i] = hi[i] = 0;
            if (i < each && first + i < p.E) {
                lo[i] = min(max(__ldg(&p.offsets[first + i]), 0), p.M);
                hi[i] = min(max(__ldg(&p.offsets[first + i + 1]), 0), p.M);
            }
            mine += hi[i] > lo[i] ? 1 : hi[i] < lo[i] ? kFalls : 0;
        }
        int before = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before += u;
        }
        if (lane == 31) counts[warp] = before;
        if (tid == 0) found[1] = -1;
        __syncthreads();
        before -= mine;
        int all = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int c = counts[q];
            if (q < warp) before += c;
            all += c;
        }
        if (all < kFalls) {
#pragma unroll
            for (int i = 0; i < kMost; ++i) {
                if (hi[i] <= lo[i]) continue;
                if (before == (int)blockIdx.y) {
                    found[0] = first + i;
                    found[1] = lo[i];
                    found[2] = hi[i] - lo[i];
                }
                ++before;
            }
        } else if (tid == 0) {
            // made ascending, as in the tensor-core kernel, so that no two groups share a row
            int at = min(max(__ldg(&p.offsets[0]), 0), p.M), left = blockIdx.y;
            for (int g = 0; g < p.E && left >= 0; ++g) {
                const int to = max(at, min(__ldg(&p.offsets[g + 1]), p.M));
                if (to > at && left-- == 0) {
                    found[0] = g;
                    found[1] = at;
                    found[2] = to - at;
                }
                at = to;
            }
        }
        __syncthreads();
        if (found[1] < 0) return;
        e = found[0];
        row0 = found[1];
        n = found[2];
    }
    const int f0 = blockIdx.x * 16;
    const uint16_t* w = static_cast<const uint16_t*>(p.w) + ((int64_t)e * p.F + f0) * p.K;
    const uint16_t* w0 = w + (int64_t)gq * p.K;
    const uint16_t* w1 = w + (int64_t)(f0 + gq + 8 < p.F ? gq + 8 : gq) * p.K;
    const uint16_t* x = static_cast<const uint16_t*>(p.x) + (int64_t)row0 * p.ldx;
    const int kw = (((p.K + 7) >> 3) + 31) & ~31, kb = warp * kw, ke = min(p.K, kb + kw);
    if (n <= 8) skinny_sums<BF16, 1, LONG>(w0, w1, x, p.ldx, n, kb, ke, red[warp], kPitch);
    else if (MAXNB == 2 || (MAXNB > 2 && n <= 16)) skinny_sums<BF16, 2, LONG>(w0, w1, x, p.ldx, n, kb, ke, red[warp], kPitch);
    else if (MAXNB == 8 && n <= 32) skinny_sums<BF16, 4, LONG>(w0, w1, x, p.ldx, n, kb, ke, red[warp], kPitch);
    // (a decode batch of 48 requests with adapters: 9.7 us, 10.7 as 64 rows.  The products' kernel would gain as much,
    // 48 rows of one 2048 x 2048 matrix 6.3 to 5.7 us, and spill more: 64 rows of 8 matrices 14.5 to 15.6)
    else if (ADAPT && MAXNB == 8 && n <= 48) skinny_sums<BF16, 6, LONG>(w0, w1, x, p.ldx, n, kb, ke, red[warp], kPitch);
    else if (MAXNB == 8) skinny_sums<BF16, 8, LONG>(w0, w1, x, p.ldx, n, kb, ke, red[warp], kPitch);
    __syncthreads();
    grid_release();  // (late: the next kernel's CTAs then spread over the SMs as evenly as this one's)
    // thread: feature tid % 16, rows tid / 16 + 16 i
    constexpr int kOut = (16 * 8 * MAXNB + kSkinnyThreads - 1) / kSkinnyThreads;
    const int j = tid & 15, f = f0 + j, m0 = tid >> 4;
    float s[kOut];
#pragma unroll
    for (int i = 0; i < kOut; ++i) {
        s[i] = 0.f;
        if (m0 + 16 * i < n) {
#pragma unroll
            for (int q = 0; q < 8; ++q) s[i] += red[q][j * kPitch + m0 + 16 * i];
        }
    }
    if (ADAPT) {
        const AdapterArgs& ad = p.ad;
        int id[kOut];
        const uint16_t* br[kOut];
        uint4 ahead[kOut][2];  // the first 16 of each token's row of B, read before v is there
#pragma unroll
        for (int i = 0; i < kOut; ++i) {
            const int m = m0 + 16 * i;
            id[i] = m < n && f < p.F ? __ldg(&ad.ids[m]) : -1;
            if (id[i] >= ad.L) id[i] = -1;
            br[i] = static_cast<const uint16_t*>(ad.b) + ((int64_t)max(id[i], 0) * ad.N + min(f, p.F - 1)) * ad.r;
            ahead[i][0] = ahead[i][1] = make_uint4(0, 0, 0, 0);
            if (id[i] >= 0) {
                ahead[i][0] = __ldg(reinterpret_cast<const uint4*>(br[i]));
                if (ad.r > 8) ahead[i][1] = __ldg(reinterpret_cast<const uint4*>(br[i] + 8));
            }
        }
        grid_wait();
        constexpr int kBlock = 64;  // rank values per pass
        float* v = &red[0][0];      // [row][kBlock]: the sums above are in registers
        static_assert(8 * MAXNB * kBlock <= 8 * 16 * kPitch, "v fits over the sums");
        for (int j0 = 0; j0 < ad.r; j0 += kBlock) {
            const int nj = min(kBlock, ad.r - j0), quads = nj >> 2;
            __syncthreads();
            for (int i = tid; i < n * quads; i += kSkinnyThreads) {
                const int m = i / quads, jq = (i - m * quads) * 4;
                const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(ad.v) + (int64_t)m * ad.r + j0 + jq);
                *reinterpret_cast<float4*>(v + m * kBlock + jq) = a;
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kOut; ++i) {
                if (id[i] < 0) continue;
                const float* vm = v + (m0 + 16 * i) * kBlock;
                for (int q = 0; q < nj; q += 8) {
                    float b[8];
                    unpack8<BF16>(j0 + q == 0 ? ahead[i][0] : j0 + q == 8 ? ahead[i][1]
                                  : __ldg(reinterpret_cast<const uint4*>(br[i] + j0 + q)), b);
#pragma unroll
                    for (int z = 0; z < 8; ++z) s[i] = fmaf(b[z], vm[q + z], s[i]);
                }
            }
        }
    }
    if (f >= p.F) return;
#pragma unroll
    for (int i = 0; i < kOut; ++i) {
        const int m = m0 + 16 * i;
        if (m >= n) continue;
        const int64_t o = (int64_t)(row0 + m) * p.ldy + f;
        if (ADAPT && p.ad.accumulate)
            s[i] += OUT32 ? static_cast<const float*>(p.y)[o] : unpack1<BF16>(static_cast<const uint16_t*>(p.y)[o]);
        if (OUT32) static_cast<float*>(p.y)[o] = s[i];
        else static_cast<uint16_t*>(p.y)[o] = pack1<BF16>(s[i]);
    }
}

template <bool BF16, bool OUT32, bool ADAPT, bool LONG>
static cudaError_t skinny_k(const SkinnyArgs& p, int rows, dim3 grid, cudaStream_t s) {
    auto kern = rows <= 8    ? skinny_kernel<BF16, OUT32, ADAPT, LONG, 1>
                : rows <= 16 ? skinny_kernel<BF16, OUT32, ADAPT, LONG, 2>
                             : skinny_kernel<BF16, OUT32, ADAPT, LONG, 8>;
    // at most a CTA an SM (64 rows of one 2048 x 2048 matrix: 6.9 us against 8.7; of 8 matrices, 18.1 against 14.4)
    if constexpr (!ADAPT)
        if (rows > 16 && grid.x * grid.y <= 148) kern = skinny_kernel<BF16, OUT32, false, LONG, 8, 1>;
    return launch_behind(kern, grid, kSkinnyThreads, 0, s, p);
}

template <bool BF16, bool OUT32, bool ADAPT>
static cudaError_t skinny(const SkinnyArgs& p, int rows, dim3 grid, cudaStream_t s) {
    return p.K > 8 * kSkinnyPart ? skinny_k<BF16, OUT32, ADAPT, true>(p, rows, grid, s)
                                 : skinny_k<BF16, OUT32, ADAPT, false>(p, rows, grid, s);
}

cudaError_t launch_skinny_grouped(const GroupedArgs& g, const void* w, const void* x, int64_t ldx, bool out32,
                                  cudaStream_t s) {
    SkinnyArgs p{};
    p.w = w;
    p.x = x;
    p.ldx = ldx;
    p.F = g.F;
    p.K = g.C;
    p.offsets = g.offsets;
    p.E = g.E;
    p.M = g.M;
    p.y = g.out;
    p.ldy = g.ldo;
    const dim3 grid((g.F + 15) / 16, g.E < g.M ? g.E : g.M);  // (groups that hold rows, at most)
    if (g.bf16) return out32 ? skinny<true, true, false>(p, g.M, grid, s) : skinny<true, false, false>(p, g.M, grid, s);
    return out32 ? skinny<false, true, false>(p, g.M, grid, s) : skinny<false, false, false>(p, g.M, grid, s);
}

cudaError_t launch_skinny_adapter(const AdapterArgs& a, bool bf16, bool out32, cudaStream_t s) {
    SkinnyArgs p{};
    p.w = a.w;
    p.x = a.x;
    p.ldx = a.ldx;
    p.F = a.N;
    p.K = a.K;
    p.y = a.y;
    p.ldy = a.ldy;
    p.ad = a;
    const dim3 grid((a.N + 15) / 16);
    if (bf16) return out32 ? skinny<true, true, true>(p, a.T, grid, s) : skinny<true, false, true>(p, a.T, grid, s);
    return out32 ? skinny<false, true, true>(p, a.T, grid, s) : skinny<false, false, true>(p, a.T, grid, s);
}

}  // namespace moe
