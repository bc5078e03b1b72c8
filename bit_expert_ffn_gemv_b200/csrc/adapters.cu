// adapters.cu -- low-rank adapters of many requests beside a shared projection.
//
//   v_t = scale[a] * A_a x_t            (rank values, fp32; a = ids[t])
//   y_t = [y_t +] [W x_t +] B_a v_t     (no delta where ids[t] is not in [0, L))
//
// Two launches.  The first computes v for every token; the second starts
// while the first still runs (programmatic dependent launch), streams W, and
// waits for v only before it adds the delta:
//   shrink_kernel   v, from windows of 32 tokens by slices of K
//   skinny_kernel   up to 64 tokens: W by warp MMAs, straight from HBM
//   grouped_kernel  more tokens: W on the tensor cores (grouped.cu), the delta in its epilogue
//   expand_kernel   no W: the delta alone
// v and the delta stay in fp32, so the result is rounded once.
#include <cuda_runtime.h>

#include "adapter.cuh"
#include "common.cuh"
#include "kernels.h"
#include "pack16.cuh"

namespace moe {

// ---------------------------------------------------------------- shrink
// One CTA: a window of WIN tokens, one slice of K.  The window's tokens are
// grouped by adapter with one match instruction, in any order of ids, and cut
// into items of up to eight tokens of one adapter, whose A rows are read once:
// MMAs of 16 A rows by 8 tokens, both operands loaded 16 bytes a lane in the
// same permuted order of k.  The eight warps take an item each; with fewer
// items several warps share one and split its K.  Bound by the A rows of a
// decode batch (every token another adapter) or the x of a prefill chunk.
constexpr int kShrinkThreads = 256;
constexpr int kShrinkRows = 64;  // A rows per pass

template <bool BF16, int WIN>
__global__ void __launch_bounds__(kShrinkThreads) shrink_kernel(const AdapterArgs p) {
    __shared__ float red[8][8][kShrinkRows + 4];  // [warp][token of its item][row]
    __shared__ int item_adapter[WIN], item_tok[WIN][8];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, c = lane & 3;
    const int t0 = blockIdx.x * WIN, slice = blockIdx.y;
    const int per = ((p.K + p.slices - 1) / p.slices + 31) & ~31;  // K of a slice
    const int sb = slice * per, se = min(p.K, sb + per);
    const int t = t0 + lane;
    int id = lane < WIN && t < p.T ? __ldg(&p.ids[t]) : -1;
    if (id < 0 || id >= p.L) id = -1;
    const uint32_t mine = __match_any_sync(0xffffffffu, id);
    // this lane's token is number `order` of its group; every eighth begins an item
    const int order = __popc(mine & ((1u << lane) - 1));
    const bool begins = id >= 0 && (order & 7) == 0;
    const uint32_t starts = __ballot_sync(0xffffffffu, begins);
    const int items = __popc(starts);
    if (items == 0) return;
    if (warp == 0) {
        if (begins) {
            const int it = __popc(starts & ((1u << lane) - 1));
            item_adapter[it] = id;
            uint32_t rest = mine & ~((1u << lane) - 1);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                item_tok[it][i] = rest ? __ffs(rest) - 1 : -1;
                rest &= rest - 1;
            }
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
        const bool live = it < items;
        const int a = live ? item_adapter[it] : 0, tok = live ? item_tok[it][gq] : -1;
        const uint16_t* xr = x + (int64_t)(t0 + (tok < 0 ? 0 : tok)) * p.ldx;
        for (int j0 = 0; j0 < p.r; j0 += kShrinkRows) {
            const int rows = min(kShrinkRows, p.r - j0), tiles = (rows + 15) >> 4;
            float acc[4][4] = {};
            const uint16_t* ar = A + ((int64_t)a * p.r + j0) * p.K;
            if (live) {
#pragma unroll 4
                for (int k0 = kb; k0 < ke; k0 += 32) {
                    const int k = k0 + 8 * c;
                    const bool in = k < ke;
                    uint4 bv = make_uint4(0, 0, 0, 0);
                    if (in && tok >= 0) bv = __ldg(reinterpret_cast<const uint4*>(xr + k));
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        if (q >= tiles) break;
                        const int r0 = q * 16 + gq;
                        uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
                        if (in && r0 < rows) lo = __ldg(reinterpret_cast<const uint4*>(ar + (int64_t)r0 * p.K + k));
                        if (in && r0 + 8 < rows) hi = __ldg(reinterpret_cast<const uint4*>(ar + (int64_t)(r0 + 8) * p.K + k));
                        const uint32_t f0[4] = {lo.x, hi.x, lo.y, hi.y}, f1[4] = {lo.z, hi.z, lo.w, hi.w};
                        mma16<BF16>(acc[q], f0, bv.x, bv.y);
                        mma16<BF16>(acc[q], f1, bv.z, bv.w);
                    }
                }
            }
            __syncthreads();  // the last pass's sums have been read
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (q >= tiles) break;
                red[warp][2 * c][q * 16 + gq] = acc[q][0];
                red[warp][2 * c + 1][q * 16 + gq] = acc[q][1];
                red[warp][2 * c][q * 16 + gq + 8] = acc[q][2];
                red[warp][2 * c + 1][q * 16 + gq + 8] = acc[q][3];
            }
            __syncthreads();
            // each warp writes one token of each of the items in turn, the shares added in order
            for (int i = warp; i < at_once * 8; i += 8) {
                const int w = (i >> 3) * share, m = i & 7, ii = base + (i >> 3);
                const int at = ii < items ? item_tok[ii][m] : -1;
                if (at < 0) continue;
                const float sc = p.scale ? __ldg(&p.scale[item_adapter[ii]]) : 1.0f;
                for (int j = lane; j < rows; j += 32) {
                    float s = red[w][m][j];
                    for (int q = 1; q < share; ++q) s += red[w + q][m][j];
                    p.v[((int64_t)slice * p.T + t0 + at) * p.r + j0 + j] = sc * s;
                }
            }
        }
    }
}

// ---------------------------------------------------------------- the delta alone
// CTA: 128 features (32 a warp) by 32 tokens, 16 at a time, in fragments.
template <bool BF16, bool OUT32>
__global__ void __launch_bounds__(128) expand_kernel(const AdapterArgs p) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int f0 = blockIdx.x * 128 + warp * 32;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (f0 >= p.N) return;
    const int end = min(p.T, ((int)blockIdx.y + 1) * 32);
    for (int t0 = blockIdx.y * 32; t0 < end; t0 += 16) {
        const int n = min(16, end - t0);
        uint32_t r[2][8];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int t = frag_token(i >> 2, i), f = f0 + frag_feature(m, i & 3);
                float v = 0.f;
                if (p.accumulate && t < n && f < p.N) {
                    const int64_t o = (int64_t)(t0 + t) * p.ldy + f;
                    v = OUT32 ? static_cast<const float*>(p.y)[o] : unpack1<BF16>(static_cast<const uint16_t*>(p.y)[o]);
                }
                r[m][i] = __float_as_uint(v);
            }
        add_delta<BF16, BF16 && OUT32 ? 3 : 2>(p, t0, n, f0, r[0], r[1]);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int t = frag_token(i >> 2, i), f = f0 + frag_feature(m, i & 3);
                if (t < n && f < p.N) {
                    const int64_t o = (int64_t)(t0 + t) * p.ldy + f;
                    if (OUT32) static_cast<float*>(p.y)[o] = __uint_as_float(r[m][i]);
                    else static_cast<uint16_t*>(p.y)[o] = pack1<BF16>(__uint_as_float(r[m][i]));
                }
            }
    }
}

// ---------------------------------------------------------------- launcher
// Up to this many tokens a window is 8 tokens: a decode batch is mostly
// tokens of different adapters, and more windows share its A rows out.
constexpr int kSmallWindowTokens = 256;

int adapter_slices(int T, int K) {
    // slices of K: CTAs for every SM as long as a slice keeps 256 of K
    const int win = T <= kSmallWindowTokens ? 8 : 32;
    const int windows = (T + win - 1) / win, most = (K + 255) / 256;
    const int want = (148 + windows - 1) / windows;
    return want < most ? want : most;
}

template <bool BF16>
static cudaError_t adapters(const AdapterArgs& p, bool out32, cudaStream_t s) {
    if (p.T <= kSmallWindowTokens)
        shrink_kernel<BF16, 8><<<dim3((p.T + 7) / 8, p.slices), kShrinkThreads, 0, s>>>(p);
    else
        shrink_kernel<BF16, 32><<<dim3((p.T + 31) / 32, p.slices), kShrinkThreads, 0, s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (p.w) return p.T <= kSkinnyMaxRows ? launch_skinny_adapter(p, BF16, out32, s)
                                          : launch_grouped_adapter(p, BF16, out32, s);
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((p.N + 127) / 128, (p.T + 31) / 32);
    cfg.blockDim = 128;
    cfg.stream = s;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return out32 ? cudaLaunchKernelEx(&cfg, expand_kernel<BF16, true>, p)
                 : cudaLaunchKernelEx(&cfg, expand_kernel<BF16, false>, p);
}

cudaError_t launch_adapters(const AdapterArgs& p, bool bf16, bool out32, cudaStream_t s) {
    return bf16 ? adapters<true>(p, out32, s) : adapters<false>(p, out32, s);
}

}  // namespace moe
