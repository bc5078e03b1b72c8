// api_ops.cu -- C entries of the 16-bit expert operators (include/moe.h):
// argument checks and launches.  No handle, no allocation: every call works on
// the caller's buffers on the caller's stream, so calls on different streams
// are independent.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"
#include "moe.h"

// Device-side errors of the operators (bounded waits), one word per device.
__device__ uint32_t g_op_status;

namespace {

constexpr int kMaxGroups = moe::kGroupedMaxGroups;
constexpr int32_t kMaxRows = 1 << 27;  // row blocks of all groups and their tiles stay inside 32 bits
constexpr int32_t kMaxCols = 1 << 17;
constexpr int32_t kMaxRank = moe::kMaxAdapterRank;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool good(const void* p) { return p && aligned16(p); }
bool good_cols(int32_t n) { return n >= 8 && n % 8 == 0 && n <= kMaxCols; }
// row pitch in values: whole 16-byte pieces, room for the row
bool good_ld(int64_t ld, int64_t cols) { return ld >= cols && ld % 8 == 0 && ld <= (int64_t(1) << 32); }

cudaError_t status_word(uint32_t** p) {
    void* v = nullptr;
    const cudaError_t e = cudaGetSymbolAddress(&v, g_op_status);
    *p = static_cast<uint32_t*>(v);
    return e;
}

moe_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

}  // namespace

extern "C" {

moe_status moe_grouped_matmul(const void* x, int64_t ldx, int32_t rows, const void* w, const int32_t* offsets,
                              int32_t n_groups, int32_t n, int32_t k, void* y, int64_t ldy, uint32_t flags,
                              void* stream) {
    if (flags & ~(MOE_OUT_FP32 | MOE_OP_FP16 | MOE_OP_TRANSPOSE)) return MOE_ERR_INVALID_ARG;
    if (rows < 0 || rows > kMaxRows || n_groups < 1 || n_groups > kMaxGroups || !good_cols(n) || !good_cols(k))
        return MOE_ERR_INVALID_ARG;
    const bool tr = (flags & MOE_OP_TRANSPOSE) != 0;
    if (!good_ld(ldx, tr ? n : k) || !good_ld(ldy, tr ? k : n)) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!good(x) || !good(w) || !good(y) || x == y || w == y || !offsets || !aligned4(offsets)) return MOE_ERR_INVALID_ARG;
    moe::GroupedArgs g{};
    g.offsets = offsets;
    g.E = n_groups;
    g.M = rows;
    g.F = tr ? k : n;
    g.C = tr ? n : k;
    g.out = y;
    g.ldo = ldy;
    g.bf16 = (flags & MOE_OP_FP16) ? 0 : 1;
    if (status_word(&g.status) != cudaSuccess) return MOE_ERR_CUDA;
    return cuda_status(moe::launch_grouped(tr ? moe::kGroupedRows : moe::kGroupedForward, g, w, x, ldx, x, ldx,
                                           (flags & MOE_OUT_FP32) != 0, static_cast<cudaStream_t>(stream)));
}

moe_status moe_grouped_wgrad(const void* dy, int64_t lddy, const void* x, int64_t ldx, int32_t rows,
                             const int32_t* offsets, int32_t n_groups, int32_t n, int32_t k, void* dw,
                             uint32_t flags, void* stream) {
    if (flags & ~(MOE_OUT_FP32 | MOE_ACCUMULATE | MOE_OP_FP16)) return MOE_ERR_INVALID_ARG;
    const bool f32 = (flags & MOE_OUT_FP32) != 0, acc = (flags & MOE_ACCUMULATE) != 0;
    if (acc && !f32) return MOE_ERR_INVALID_ARG;
    if (rows < 0 || rows > kMaxRows || n_groups < 1 || n_groups > kMaxGroups || !good_cols(n) || !good_cols(k) ||
        !good_ld(lddy, n) || !good_ld(ldx, k) || !good(dw))
        return MOE_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (rows == 0) {  // every group is empty
        if (acc) return MOE_OK;
        return cuda_status(cudaMemsetAsync(dw, 0, (size_t)n_groups * n * k * (f32 ? 4 : 2), s));
    }
    if (!good(dy) || !good(x) || dw == dy || dw == x || !offsets || !aligned4(offsets)) return MOE_ERR_INVALID_ARG;
    moe::GroupedArgs g{};
    g.offsets = offsets;
    g.E = n_groups;
    g.M = rows;
    g.F = n;
    g.C = k;
    g.out = dw;
    g.ldo = k;
    g.bf16 = (flags & MOE_OP_FP16) ? 0 : 1;
    g.accumulate = acc ? 1 : 0;
    if (status_word(&g.status) != cudaSuccess) return MOE_ERR_CUDA;
    return cuda_status(moe::launch_grouped(moe::kGroupedWeights, g, nullptr, x, ldx, dy, lddy, f32, s));
}

moe_status moe_swiglu(const void* gu, int64_t ldgu, int32_t rows, int32_t f, const float* row_weights,
                      const int32_t* n_rows, void* h, int64_t ldh, uint32_t flags, void* stream) {
    if (flags & ~MOE_OP_FP16) return MOE_ERR_INVALID_ARG;
    if (rows < 0 || rows > kMaxRows || !good_cols(f) || !good_ld(ldgu, 2 * (int64_t)f) || !good_ld(ldh, f))
        return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!good(gu) || !good(h) || !aligned4(row_weights) || !aligned4(n_rows) || h == gu) return MOE_ERR_INVALID_ARG;
    moe::SwigluArgs a{};
    a.gu = gu;
    a.ldgu = ldgu;
    a.M = rows;
    a.f = f;
    a.rw = row_weights;
    a.n_rows = n_rows;
    a.h = h;
    a.ldh = ldh;
    return cuda_status(moe::launch_swiglu(a, !(flags & MOE_OP_FP16), false, static_cast<cudaStream_t>(stream)));
}

moe_status moe_swiglu_backward(const void* gu, int64_t ldgu, const void* dh, int64_t lddh, int32_t rows, int32_t f,
                               const float* row_weights, const int32_t* n_rows, void* dgu, int64_t lddgu, void* h,
                               int64_t ldh, float* d_row_weights, uint32_t flags, void* stream) {
    if (flags & ~MOE_OP_FP16) return MOE_ERR_INVALID_ARG;
    if (rows < 0 || rows > kMaxRows || !good_cols(f) || !good_ld(ldgu, 2 * (int64_t)f) || !good_ld(lddh, f) ||
        !good_ld(lddgu, 2 * (int64_t)f) || (h && !good_ld(ldh, f)))
        return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!good(gu) || !good(dh) || !good(dgu) || (h && !aligned16(h)) || !aligned4(row_weights) || !aligned4(n_rows) ||
        !aligned4(d_row_weights))
        return MOE_ERR_INVALID_ARG;
    // in place only as the kernel can: every value of dgu by the lane that has read gu's at its address
    if ((dgu == gu && lddgu != ldgu) || dgu == dh || (h && (h == gu || h == dh || h == dgu)) ||
        (d_row_weights && d_row_weights == row_weights))
        return MOE_ERR_INVALID_ARG;
    moe::SwigluArgs a{};
    a.gu = gu;
    a.ldgu = ldgu;
    a.M = rows;
    a.f = f;
    a.rw = row_weights;
    a.n_rows = n_rows;
    a.dh = dh;
    a.lddh = lddh;
    a.dgu = dgu;
    a.lddgu = lddgu;
    a.h = h;
    a.ldh = ldh;
    a.drw = d_row_weights;
    return cuda_status(moe::launch_swiglu(a, !(flags & MOE_OP_FP16), true, static_cast<cudaStream_t>(stream)));
}

size_t moe_adapter_workspace(int32_t tokens, int32_t rank) {
    if (tokens <= 0 || tokens > kMaxRows || rank <= 0 || rank > kMaxRank) return 0;
    return moe::adapter_workspace(tokens, rank);
}

moe_status moe_adapter_check(const moe_adapter_args* args, uint32_t flags) {
    if (!args || (flags & ~(MOE_OUT_FP32 | MOE_ACCUMULATE | MOE_OP_FP16))) return MOE_ERR_INVALID_ARG;
    const moe_adapter_args& q = *args;
    if (q.tokens < 0 || q.tokens > kMaxRows || !good_cols(q.n) || !good_cols(q.k) || q.n_adapters < 1 ||
        q.rank < 8 || q.rank % 8 || q.rank > kMaxRank || !good_ld(q.ldx, q.k) || !good_ld(q.ldy, q.n))
        return MOE_ERR_INVALID_ARG;
    if (q.tokens == 0) return MOE_OK;
    if (!good(q.x) || !good(q.a) || !good(q.b) || !good(q.y) || !good(q.workspace) || (q.w && !aligned16(q.w)) ||
        !q.ids || !aligned4(q.ids) || !aligned4(q.scale) ||
        q.workspace_bytes < moe_adapter_workspace(q.tokens, q.rank) || q.y == q.x || q.y == q.w || q.y == q.a ||
        q.y == q.b || q.y == q.workspace || q.workspace == q.x)
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

moe_status moe_adapter_project(const moe_adapter_args* args, uint32_t flags, void* stream) {
    const moe_status st = moe_adapter_check(args, flags);
    if (st != MOE_OK || args->tokens == 0) return st;
    const moe_adapter_args& q = *args;
    moe::AdapterArgs a{};
    a.x = q.x;
    a.ldx = q.ldx;
    a.T = q.tokens;
    a.N = q.n;
    a.K = q.k;
    a.L = q.n_adapters;
    a.r = q.rank;
    a.w = q.w;
    a.a = q.a;
    a.b = q.b;
    a.scale = q.scale;
    a.ids = q.ids;
    a.y = q.y;
    a.ldy = q.ldy;
    a.v = q.workspace;
    a.accumulate = (flags & MOE_ACCUMULATE) ? 1 : 0;
    if (status_word(&a.status) != cudaSuccess) return MOE_ERR_CUDA;
    return cuda_status(moe::launch_adapters(a, !(flags & MOE_OP_FP16), (flags & MOE_OUT_FP32) != 0,
                                            static_cast<cudaStream_t>(stream)));
}

moe_status moe_check_op_status(void) {
    if (cudaDeviceSynchronize() != cudaSuccess) return MOE_ERR_CUDA;
    uint32_t v = 0;
    if (cudaMemcpyFromSymbol(&v, g_op_status, sizeof(v)) != cudaSuccess) return MOE_ERR_CUDA;
    const uint32_t zero = 0;
    if (v && cudaMemcpyToSymbol(g_op_status, &zero, sizeof(zero)) != cudaSuccess) return MOE_ERR_CUDA;
    return (v & moe::kStatusTimeout) ? MOE_ERR_TIMEOUT : MOE_OK;
}

}  // extern "C"
