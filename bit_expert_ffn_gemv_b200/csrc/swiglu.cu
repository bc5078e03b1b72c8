// swiglu.cu -- the activation between an expert's two products, and its gradient.
//
//   h   = rw * g s u                      s = 1 / (1 + e^-g), gu = [g | u] per row
//   dg  = rw * dh u s (1 + g (1 - s))     du = rw * dh g s
//   drw = sum_j dh_j g_j s_j u_j          (the routing weight's gradient)
// rw: an optional fp32 weight per row (a token's routing weight, folded into h
// so that the down product needs no epilogue and its gradient stays local).
//
// Bound by HBM: every value is read once and written once, 16 bytes per lane;
// loads are issued before the arithmetic of the values before them.  One warp owns a row
// when there are enough rows to fill the GPU (drw is then a shuffle), eight
// warps share one otherwise.  81920 rows of f = 768: the gradient with h and drw
// 112 us, 6.7 TB/s or the measured copy; 640 rows forward 2.5 us.
#include <cuda_runtime.h>

#include "common.cuh"
#include "kernels.h"
#include "pack16.cuh"

namespace moe {

// s and 1 - s, from e^-|g|: the quotient's denominator lies in [1, 2], where the
// fast division holds (it gives zero for denominators above 2^126, and with
// e^-g those are the gates below -87.3, whose h a large u keeps from being
// small), and neither value cancels.
struct Sigmoid {
    float s, rest;
};
MOE_DEV Sigmoid sigmoid(float g) {
    const float z = __expf(-fabsf(g)), big = __fdividef(1.0f, 1.0f + z), small = z * big;
    return g >= 0.0f ? Sigmoid{big, small} : Sigmoid{small, big};
}

constexpr int kSwigluThreads = 256;
constexpr int kSwigluFewRows = 148 * 8 * 4;  // below this many rows a whole block takes each row

template <bool BF16, int WARPS>
__global__ void __launch_bounds__(kSwigluThreads) swiglu_kernel(const SwigluArgs a) {
    grid_release();
    grid_wait();
    const int per = 8 / WARPS, lanes = WARPS * 32;
    const int r = blockIdx.x * per + (WARPS == 1 ? threadIdx.x >> 5 : 0);
    const int lane = threadIdx.x & (lanes - 1);
    const int rows = a.n_rows ? min(__ldg(a.n_rows), a.M) : a.M;
    if (r >= rows) return;
    const uint16_t* gu = static_cast<const uint16_t*>(a.gu) + (int64_t)r * a.ldgu;
    uint16_t* h = static_cast<uint16_t*>(a.h) + (int64_t)r * a.ldh;
    const float rw = a.rw ? __ldg(&a.rw[r]) : 1.0f;
#pragma unroll 4
    for (int c = lane * 8; c < a.f; c += lanes * 8) {
        const uint4 gv = __ldg(reinterpret_cast<const uint4*>(gu + c));
        const uint4 uv = __ldg(reinterpret_cast<const uint4*>(gu + a.f + c));
        float g[8], u[8];
        unpack8<BF16>(gv, g);
        unpack8<BF16>(uv, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = rw * (g[i] * sigmoid(g[i]).s * u[i]);
        *reinterpret_cast<uint4*>(h + c) = pack8<BF16>(g);
    }
}

// (four blocks an SM, 64 registers, two blocks of a row ahead: 112 us at 81920 rows; four ahead in 100 registers 133)
template <bool BF16, int WARPS>
__global__ void __launch_bounds__(kSwigluThreads, 4) swiglu_grad_kernel(const SwigluArgs a) {
    __shared__ float part[8];
    grid_release();
    grid_wait();
    const int per = 8 / WARPS, lanes = WARPS * 32;
    const int r = blockIdx.x * per + (WARPS == 1 ? threadIdx.x >> 5 : 0);
    const int lane = threadIdx.x & (lanes - 1);
    const int rows = a.n_rows ? min(__ldg(a.n_rows), a.M) : a.M;
    if (r >= rows) return;  // the whole warp, and with eight warps per row the whole block
    const uint16_t* gu = static_cast<const uint16_t*>(a.gu) + (int64_t)r * a.ldgu;
    const uint16_t* dhp = static_cast<const uint16_t*>(a.dh) + (int64_t)r * a.lddh;
    uint16_t* dgu = static_cast<uint16_t*>(a.dgu) + (int64_t)r * a.lddgu;
    uint16_t* h = a.h ? static_cast<uint16_t*>(a.h) + (int64_t)r * a.ldh : nullptr;
    const float rw = a.rw ? __ldg(&a.rw[r]) : 1.0f;
    float dot = 0.f;
    // dgu may be gu itself: the loads are plain ones, and a lane loads its next two blocks before it stores either
    constexpr int kAhead = 2;
    for (int c0 = lane * 8; c0 < a.f; c0 += kAhead * lanes * 8) {
        uint4 gv[kAhead], uv[kAhead], dv[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int c = c0 + j * lanes * 8;
            if (c >= a.f) break;
            gv[j] = *reinterpret_cast<const uint4*>(gu + c);
            uv[j] = *reinterpret_cast<const uint4*>(gu + a.f + c);
            dv[j] = *reinterpret_cast<const uint4*>(dhp + c);
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int c = c0 + j * lanes * 8;
            if (c >= a.f) break;
            float g[8], u[8], d[8], hh[8];
            unpack8<BF16>(gv[j], g);
            unpack8<BF16>(uv[j], u);
            unpack8<BF16>(dv[j], d);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const Sigmoid sg = sigmoid(g[i]);
                const float act = g[i] * sg.s, act_u = act * u[i], dw = rw * d[i];
                hh[i] = rw * act_u;
                dot = fmaf(d[i], act_u, dot);
                g[i] = dw * (sg.s * (1.0f + g[i] * sg.rest)) * u[i];  // (dh u may overflow where the product does not)
                u[i] = dw * act;
            }
            *reinterpret_cast<uint4*>(dgu + c) = pack8<BF16>(g);
            *reinterpret_cast<uint4*>(dgu + a.f + c) = pack8<BF16>(u);
            if (h) *reinterpret_cast<uint4*>(h + c) = pack8<BF16>(hh);
        }
    }
    if (!a.drw) return;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (WARPS > 1) {
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = dot;
        __syncthreads();
        dot = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) dot += part[w];
    }
    if (lane == 0) a.drw[r] = dot;
}

template <bool BF16>
static cudaError_t launch(const SwigluArgs& a, bool grad, cudaStream_t s) {
    const bool few = a.M < kSwigluFewRows;
    const int blocks = few ? a.M : (a.M + 7) / 8;
    auto kern = grad ? (few ? swiglu_grad_kernel<BF16, 8> : swiglu_grad_kernel<BF16, 1>)
                     : (few ? swiglu_kernel<BF16, 8> : swiglu_kernel<BF16, 1>);
    return launch_behind(kern, blocks, kSwigluThreads, 0, s, a);
}

cudaError_t launch_swiglu(const SwigluArgs& a, bool bf16, bool grad, cudaStream_t s) {
    return bf16 ? launch<true>(a, grad, s) : launch<false>(a, grad, s);
}

}  // namespace moe
