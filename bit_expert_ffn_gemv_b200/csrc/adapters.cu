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
// One CTA: 32 tokens, one slice of K; its eight warps split the slice and add
// their sums in warp order.  The window's tokens are grouped by adapter with
// one match instruction, in any order of ids, and each group's A rows are read
// once per eight of its tokens: MMAs of 16 A rows by 8 tokens, both operands
// loaded 16 bytes a lane in the same permuted order of k.
constexpr int kShrinkThreads = 256;
constexpr int kShrinkRows = 64;  // A rows per pass

template <bool BF16>
__global__ void __launch_bounds__(kShrinkThreads) shrink_kernel(const AdapterArgs p) {
    __shared__ float red[8][8][kShrinkRows + 4];  // [warp][token][row]
    __shared__ int pos[8];                        // window positions of the eight tokens
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, c = lane & 3;
    const int t0 = blockIdx.x * 32, slice = blockIdx.y;
    const int per = ((p.K + p.slices - 1) / p.slices + 255) & ~255;  // K of a slice: 32-wide steps for eight warps
    const int kb = slice * per + warp * (per >> 3), ke = min(p.K, kb + (per >> 3));
    const int t = t0 + lane;
    int id = t < p.T ? __ldg(&p.ids[t]) : -1;
    if (id < 0 || id >= p.L) id = -1;
    const uint32_t mine = __match_any_sync(0xffffffffu, id);
    uint32_t todo = __ballot_sync(0xffffffffu, id >= 0);
    const uint16_t* x = static_cast<const uint16_t*>(p.x);
    const uint16_t* A = static_cast<const uint16_t*>(p.a);
    while (todo) {
        const int leader = __ffs(todo) - 1;
        const int a = __shfl_sync(0xffffffffu, id, leader);
        // the group's next eight tokens, in order
        const uint32_t group = __shfl_sync(0xffffffffu, mine, leader) & todo;
        uint32_t rest = group;
        int tok = -1, n = 0;  // window position of this lane's token (gq-th of the eight)
        for (; n < 8 && rest; ++n) {
            const int w = __ffs(rest) - 1;
            if (n == gq) tok = w;
            rest &= rest - 1;
        }
        todo &= ~(group & ~rest);
        const uint16_t* xr = x + (int64_t)(t0 + (tok < 0 ? leader : tok)) * p.ldx;
        for (int j0 = 0; j0 < p.r; j0 += kShrinkRows) {
            const int tiles = (min(kShrinkRows, p.r - j0) + 15) >> 4;
            float acc[4][4] = {};
            const uint16_t* ar = A + ((int64_t)a * p.r + j0) * p.K;
#pragma unroll 2
            for (int k = kb + 8 * c; k < ke + 8 * c; k += 32) {
                const bool in = k < ke;
                uint4 bv = make_uint4(0, 0, 0, 0);
                if (in) bv = __ldg(reinterpret_cast<const uint4*>(xr + k));
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (q >= tiles) break;
                    const int r0 = q * 16 + gq;
                    uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
                    if (in && j0 + r0 < p.r) lo = __ldg(reinterpret_cast<const uint4*>(ar + (int64_t)r0 * p.K + k));
                    if (in && j0 + r0 + 8 < p.r)
                        hi = __ldg(reinterpret_cast<const uint4*>(ar + (int64_t)(r0 + 8) * p.K + k));
                    const uint32_t f0[4] = {lo.x, hi.x, lo.y, hi.y}, f1[4] = {lo.z, hi.z, lo.w, hi.w};
                    mma16<BF16>(acc[q], f0, bv.x, bv.y);
                    mma16<BF16>(acc[q], f1, bv.z, bv.w);
                }
            }
            __syncthreads();  // the last pass's sums have been read
            if (warp == 0 && c == 0) pos[gq] = tok;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (q >= tiles) break;
                red[warp][2 * c][q * 16 + gq] = acc[q][0];
                red[warp][2 * c + 1][q * 16 + gq] = acc[q][1];
                red[warp][2 * c][q * 16 + gq + 8] = acc[q][2];
                red[warp][2 * c + 1][q * 16 + gq + 8] = acc[q][3];
            }
            __syncthreads();
            const float sc = p.scale ? __ldg(&p.scale[a]) : 1.0f;
            const int rows = min(kShrinkRows, p.r - j0);
            for (int i = tid; i < n * rows; i += kShrinkThreads) {
                const int m = i / rows, j = i - m * rows;
                float s = 0.f;
#pragma unroll
                for (int w = 0; w < 8; ++w) s += red[w][m][j];
                p.v[((int64_t)slice * p.T + t0 + pos[m]) * p.r + j0 + j] = sc * s;
            }
        }
    }
}

// ---------------------------------------------------------------- the delta alone
// CTA: 128 features by 64 tokens; lane = feature, 16 tokens at a time.
template <bool BF16, bool OUT32>
__global__ void __launch_bounds__(128) expand_kernel(const AdapterArgs p) {
    __shared__ __align__(16) float vbuf[4][kAdapterV];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int f = blockIdx.x * 128 + warp * 32 + lane;
    AdapterRow row;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int end = min(p.T, ((int)blockIdx.y + 1) * 64);
    for (int t0 = blockIdx.y * 64; t0 < end; t0 += 16) {
        const int n = min(16, end - t0);
        float acc[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            acc[i] = 0.f;
            if (p.accumulate && i < n && f < p.N) {
                const int64_t o = (int64_t)(t0 + i) * p.ldy + f;
                acc[i] = OUT32 ? static_cast<const float*>(p.y)[o] : unpack1<BF16>(static_cast<const uint16_t*>(p.y)[o]);
            }
        }
        adapter_delta<BF16>(p, t0, n, f, vbuf[warp], row, acc);
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (i < n && f < p.N) {
                const int64_t o = (int64_t)(t0 + i) * p.ldy + f;
                if (OUT32) static_cast<float*>(p.y)[o] = acc[i];
                else static_cast<uint16_t*>(p.y)[o] = pack1<BF16>(acc[i]);
            }
    }
}

// ---------------------------------------------------------------- launcher
int adapter_slices(int T, int K) {
    // slices of K: enough CTAs for the GPU while every warp keeps at least 64 of K; one for large batches, whose
    // windows fill the GPU by themselves
    const int windows = (T + 31) / 32, most = (K + 511) / 512;
    const int want = (148 + windows - 1) / windows;
    return want < most ? want : most;
}

template <bool BF16>
static cudaError_t adapters(const AdapterArgs& p, bool out32, cudaStream_t s) {
    shrink_kernel<BF16><<<dim3((p.T + 31) / 32, p.slices), kShrinkThreads, 0, s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (p.w) return p.T <= kSkinnyMaxRows ? launch_skinny_adapter(p, BF16, out32, s)
                                          : launch_grouped_adapter(p, BF16, out32, s);
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((p.N + 127) / 128, (p.T + 63) / 64);
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
