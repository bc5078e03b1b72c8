// adapter.cuh -- the delta B_a v_t of a token's adapter, added to fp32 values
// held as lane = feature, register = token (the layout the tensor core's
// accumulators are read in).
#pragma once
#include "common.cuh"
#include "kernels.h"
#include "pack16.cuh"

namespace moe {

constexpr int kAdapterBlock = 64;                     // rank values per pass
constexpr int kAdapterPitch = 20;                     // floats per rank value: 16 tokens, padded
constexpr int kAdapterV = kAdapterBlock * kAdapterPitch;  // floats of one warp's buffer

// a lane's row B_a[f][0..64) as it was last loaded, packed
struct AdapterRow {
    int a = -1;
    uint4 b[kAdapterBlock / 8];
};

MOE_DEV void fma2(float2& d, float2 a, float2 b) {
    asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%0, %1};\n"
        " fma.rn.f32x2 z, x, y, z;\n mov.b64 {%0, %1}, z;\n}\n"
        : "+f"(d.x), "+f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
}

// acc[i] += B_a[f] . v of token t0 + i, i < n <= 16; called by whole warps
// (f may lie past N: its lane adds nothing).  vbuf: kAdapterV floats of shared
// memory private to the warp.  When the 16 tokens share an adapter its row
// stays in registers from one call to the next; otherwise every token reads
// its own.
template <bool BF16>
MOE_DEV void adapter_delta(const AdapterArgs& p, int t0, int n, int f, float* vbuf, AdapterRow& row, float (&acc)[16]) {
    const int lane = threadIdx.x & 31;
    int id = lane < n ? __ldg(&p.ids[t0 + lane]) : -1;
    if (id < 0 || id >= p.L) id = -1;
    const uint32_t used = __ballot_sync(0xffffffffu, id >= 0);
    if (!used) return;
    const int first = __shfl_sync(0xffffffffu, id, __ffs(used) - 1);
    const bool same = __all_sync(0xffffffffu, id == first || id < 0);
    const uint16_t* B = static_cast<const uint16_t*>(p.b);
    const bool in = f < p.N;
    for (int j0 = 0; j0 < p.r; j0 += kAdapterBlock) {
        const int nj = min(kAdapterBlock, p.r - j0);
        __syncwarp();  // the last pass's values have been read
        for (int i = lane; i < 16 * nj; i += 32) {
            const int m = i / nj, j = i - m * nj;
            float v = 0.f;
            if ((used >> m) & 1) {
                const float* q = p.v + (int64_t)(t0 + m) * p.r + j0 + j;
                for (int s = 0; s < p.slices; ++s) v += q[(int64_t)s * p.T * p.r];
            }
            vbuf[j * kAdapterPitch + m] = v;
        }
        __syncwarp();
        if (same) {
            if (row.a != first || p.r > kAdapterBlock) {
                const uint16_t* br = B + ((int64_t)first * p.N + (in ? f : 0)) * p.r + j0;
#pragma unroll
                for (int q = 0; q < kAdapterBlock / 8; ++q)
                    row.b[q] = q * 8 < nj && in ? __ldg(reinterpret_cast<const uint4*>(br + q * 8)) : make_uint4(0, 0, 0, 0);
                row.a = first;
            }
            float2 d[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] = make_float2(acc[2 * i], acc[2 * i + 1]);
#pragma unroll
            for (int q = 0; q < kAdapterBlock / 8; ++q) {
                if (q * 8 < nj) {
                    float b[8];
                    unpack8<BF16>(row.b[q], b);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float4* v4 = reinterpret_cast<const float4*>(vbuf + (q * 8 + j) * kAdapterPitch);
                        const float2 bb = make_float2(b[j], b[j]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float4 v = v4[i];
                            fma2(d[2 * i], bb, make_float2(v.x, v.y));
                            fma2(d[2 * i + 1], bb, make_float2(v.z, v.w));
                        }
                    }
                }
            }
            // (a token without an adapter keeps its value even where B holds infinities)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if ((used >> (2 * i)) & 1) acc[2 * i] = d[i].x;
                if ((used >> (2 * i + 1)) & 1) acc[2 * i + 1] = d[i].y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int a = __shfl_sync(0xffffffffu, id, i);
                if (a < 0) continue;
                const uint16_t* br = B + ((int64_t)a * p.N + (in ? f : 0)) * p.r + j0;
                float s = 0.f;
                for (int q = 0; q < nj; q += 8) {
                    float b[8];
                    unpack8<BF16>(__ldg(reinterpret_cast<const uint4*>(br + q)), b);
#pragma unroll
                    for (int j = 0; j < 8; ++j) s = fmaf(b[j], vbuf[(q + j) * kAdapterPitch + i], s);
                }
                if (in) acc[i] += s;
            }
        }
    }
}

}  // namespace moe
