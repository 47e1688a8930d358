// layer.hpp -- what the kernels around the expert products share (rmsnorm.cu,
// moe_gate.cu, moe_combine.cu, gemv_nvfp4.cu): their launchers, for the C ABI,
// and the device helpers that only they use.  A file of its own, as the
// recorded profiles of the other kernels are keyed by the contents of the
// headers that those include.
#pragma once

#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "sm100.cuh"

namespace fpq {

// RMS norm (rmsnorm.cu): fmt FPQ_FP8_1x128 or FPQ_MXFP8 when q is given;
// residual, h, y, q + scales and rstd may be nullptr.  ld_x in elements.
cudaError_t launch_rmsnorm_quantize(int fmt, const void* x, int64_t ld_x, const void* residual, const void* weight,
                                    int64_t rows, int64_t cols, float eps, void* h, void* y, void* q, void* scales,
                                    float* rstd, int sms, cudaStream_t st);
size_t rmsnorm_backward_workspace_bytes(int64_t rows, int64_t cols, int sms);
cudaError_t launch_rmsnorm_backward(const void* dy, const void* x, int64_t ld_x, const void* weight,
                                    const float* rstd, const void* dres, int64_t rows, int64_t cols, void* dx,
                                    float* dweight, void* workspace, uint32_t* err, int sms, cudaStream_t st);

// Expert gate (moe_gate.cu): f32 selects fp32 logits, else bf16.
cudaError_t launch_moe_gate(const void* logits, int f32, const float* bias, int64_t tokens, int experts, int sigmoid,
                            int n_group, int topk_group, int group_top, int topk, int renormalize, float scale,
                            int32_t* ids, float* weights, cudaStream_t st);
cudaError_t launch_moe_gate_backward(const void* logits, int f32, const int32_t* ids, const float* dweights,
                                     int64_t tokens, int experts, int sigmoid, int topk, int renormalize,
                                     float scale, void* dlogits, uint32_t* err, cudaStream_t st);

// Combination of the experts' rows (moe_combine.cu); rows may be nullptr
// (pair p is row p).  launch_moe_pair_rows reads the route workspace.
cudaError_t launch_moe_pair_rows(const int32_t* ids, int64_t tokens, int topk, int experts, const void* workspace,
                                 const int64_t* dst_row0, int32_t* rows, cudaStream_t st);
cudaError_t launch_moe_combine(const void* y, int y_f32, int64_t y_rows, const int32_t* rows, const float* weights,
                               int64_t tokens, int topk, int64_t hidden, const void* add, void* out, int out_f32,
                               uint32_t* err, cudaStream_t st);
cudaError_t launch_moe_combine_backward(const void* dout, int dout_f32, const void* y, int y_f32, int64_t y_rows,
                                        const int32_t* rows, const float* weights, int64_t tokens, int topk,
                                        int64_t hidden, void* dy, float* dweights, int32_t* owner, uint32_t* err,
                                        int sms, cudaStream_t st);
// Zeros into the rows of dy that no pair names; owner as written by the
// backward call (unused without rows).
cudaError_t launch_moe_clear_rows(const int32_t* rows, int64_t pairs, int64_t y_rows, const int32_t* owner,
                                  int64_t row_bytes, void* dy, cudaStream_t st);

// Few rows times NVFP4 weights (gemv_nvfp4.cu): row m of y [m, n] is row
// m / x_div of x times the matrix (ids == nullptr) or expert ids[m]'s.
cudaError_t launch_gemv_nvfp4(const void* x, int64_t m, int x_div, int tokens, const int32_t* ids, int experts,
                              const void* wq, const void* ws, const float* wg, int64_t n, int64_t k, void* y,
                              int y_f32, uint32_t* err, int sms, cudaStream_t st);

// Lets the kernel take up to `Bytes` of dynamic shared memory on the current
// device, once.  The attribute is the function's, not the launch's: it is a
// constant, so that host threads with calls of different sizes cannot take
// from each other what they need.
template <auto Kernel, int Bytes>
cudaError_t allow_shared_memory() {
    static std::atomic<bool> done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Bytes);
    if (e == cudaSuccess) done[dev].store(true, std::memory_order_release);
    return e;
}

// two E4M3 codes (bits 0..15) -> packed f16x2, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t c2) {
    uint32_t h2;
    const uint16_t in = (uint16_t)(c2 & 0xFFFFu);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(in));
    return h2;
}

// Contiguous copy global -> shared; both addresses and the size multiples of
// 16 bytes.
__device__ __forceinline__ void bulk_load(void* smem_dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 :: "r"(sm100::smem_u32(smem_dst)), "l"(src), "r"(bytes), "r"(sm100::smem_u32(bar)) : "memory");
}

// Wait for the phase with the given parity to complete, giving up after
// about two seconds (a copy takes microseconds).
__device__ __forceinline__ bool mbar_wait_seconds(uint64_t* bar, uint32_t parity) {
    if (sm100::mbar_try_wait(bar, parity)) return true;
    uint64_t t0, t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
    do {
        for (int i = 0; i < 64; ++i)
            if (sm100::mbar_try_wait(bar, parity)) return true;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    } while (t - t0 < 2000000000ull);
    return false;
}

}  // namespace fpq
