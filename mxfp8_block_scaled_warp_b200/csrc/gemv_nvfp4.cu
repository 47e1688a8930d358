// gemv_nvfp4.cu -- products of a few bf16 rows with NVFP4 weights, the form
// that decoding takes: y[m, n] = g sum_k x[m, k] e2m1(W[n, k]) e4m3(S[n, k/16]),
// the weights of one matrix, or for row m those of expert ids[m].
//
// A weight is decoded exactly (an E2M1 code times an E4M3 scale has at most
// six significant bits), sums are fp32, g multiplies the sum once.
//
// Bound by HBM: 9/16 byte per weight.
#include <cuda_runtime.h>

#include "common.cuh"
#include "internal.h"

namespace fpq {

namespace {

constexpr int kGemvWarps = 8;
constexpr int kGemvRows = 16;             // rows of x per pass over the weights

struct GemvArgs {
    const uint16_t* x;          // row m at x + (m / x_div) k
    int64_t m;
    int x_div;
    const int32_t* ids;         // [m], or nullptr
    int experts;
    const uint8_t* wq;          // [experts, n, k / 2]
    const uint8_t* ws;          // [experts, n, k / 16]
    const float* wg;            // [experts]
    int64_t n, k;
    void* y;                    // [m, n]
    uint32_t* err;
};

__device__ __forceinline__ void put(void* y, int64_t at, float v, bool f32) {
    if (f32) static_cast<float*>(y)[at] = v;
    else static_cast<uint16_t*>(y)[at] = (uint16_t)f32_to_bf16(v);
}

// Warp per weight row; blockIdx.y: up to 16 rows of x, or one with ids.
template <bool F32>
__global__ void __launch_bounds__(32 * kGemvWarps)
gemv_nvfp4_kernel(const GemvArgs a) {
    pdl_trigger();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * kGemvWarps + warp;
    if (row >= a.n) return;
    const int64_t m0 = a.ids ? blockIdx.y : (int64_t)blockIdx.y * kGemvRows;
    const int count = a.ids ? 1 : (int)min64(kGemvRows, a.m - m0);
    int64_t e = 0;
    if (a.ids) {
        e = a.ids[m0];
        if (e < 0 || e >= a.experts) {
            if (lane == 0) {
                raise_device_error(a.err, FPQ_ERR_DEVICE_BAD_INPUT);
                put(a.y, m0 * a.n + row, 0.0f, F32);
            }
            return;
        }
    }
    const uint8_t* wq = a.wq + (e * a.n + row) * (a.k / 2);
    const uint8_t* ws = a.ws + (e * a.n + row) * (a.k / 16);
    float acc[kGemvRows] = {};
    for (int64_t c = lane; c < a.k / 32; c += 32) {           // 32 weights: 16 bytes of codes, two scales
        const uint4 codes = ld_stream(wq + 16 * c);
        const float2 s = e4m3x2_to_f32x2(*reinterpret_cast<const uint16_t*>(ws + 2 * c));
        const uint32_t cw[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float w[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 v = e2m1x2_to_f32x2(cw[i] >> (8 * j));
                w[2 * j] = v.x * (i < 2 ? s.x : s.y);
                w[2 * j + 1] = v.y * (i < 2 ? s.x : s.y);
            }
#pragma unroll
            for (int m = 0; m < kGemvRows; ++m) {
                if (m >= count) break;
                const uint4 xv = __ldg(reinterpret_cast<const uint4*>(a.x + (m0 + m) / a.x_div * a.k + 32 * c) + i);
                const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[m] = fmaf(bf16_hi(xw[j]), w[2 * j + 1], fmaf(bf16_lo(xw[j]), w[2 * j], acc[m]));
            }
        }
    }
    const float g = a.wg[e];
#pragma unroll
    for (int m = 0; m < kGemvRows; ++m) {
        if (m >= count) break;
        float v = acc[m];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        if (lane == 0) put(a.y, (m0 + m) * a.n + row, v * g, F32);
    }
}

}  // namespace

cudaError_t launch_gemv_nvfp4(const void* x, int64_t m, int x_div, const int32_t* ids, int experts, const void* wq,
                              const void* ws, const float* wg, int64_t n, int64_t k, void* y, int y_f32,
                              uint32_t* err, int sms, cudaStream_t st) {
    const GemvArgs a{(const uint16_t*)x, m, x_div, ids, experts, (const uint8_t*)wq, (const uint8_t*)ws, wg, n, k,
                     y, err};
    const dim3 grid((unsigned)((n + kGemvWarps - 1) / kGemvWarps),
                    (unsigned)(ids ? m : (m + kGemvRows - 1) / kGemvRows));
    return y_f32 ? launch_pdl(gemv_nvfp4_kernel<true>, grid, dim3(32 * kGemvWarps), 0, st, a)
                 : launch_pdl(gemv_nvfp4_kernel<false>, grid, dim3(32 * kGemvWarps), 0, st, a);
}

}  // namespace fpq
