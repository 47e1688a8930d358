// rmsnorm.cu -- RMS norm with the residual's addition and a block-scaled
// 8-bit output, and its backward pass.
//
// Forward, per row of `cols` elements, all in fp32:
//   s = x + residual (x alone without one),  rstd = 1 / sqrt(sum s^2 / cols + eps)
//   y = (s rstd) w
// with the outputs h = bf16(s) (the residual stream), bf16(y), and the codes
// and scales of y under the 1x128 or MXFP8 rules.  The codes are taken from
// the fp32 y, not from bf16(y): one rounding instead of two.
//
// Backward for the gradient dy of y (the quantizer passes gradients
// unchanged, as in the QAT backward) and dres of h:
//   dx = dres + rstd g - x (rstd^3 / cols) sum(g x),   g = dy w
//   dw = sum over rows of dy x rstd
//
// Both are bound by HBM: a row is read once into registers, reduced over the
// threads that hold it, and written from the registers.  A thread holds V
// vectors of 8 elements (16 bytes of bf16); rows of at most 1024 elements
// take one warp each (no block barrier), longer rows one CTA each.
#include <cuda_runtime.h>

#include "common.cuh"
#include "internal.h"
#include "quant_unit.cuh"

namespace fpq {

namespace {

enum { kNormNone = 0, kNormFp8 = 1, kNormMx = 2 };
constexpr int kRowWarps = 8;             // rows (warps) per CTA in the warp-per-row form

// 16-byte load of data that is read once.  Not the non-coherent form: h may
// be written over the residual it is read from.
__device__ __forceinline__ uint4 ld_once(const uint4* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
    f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x); f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z); f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(f32x2_to_bf16x2(f[0], f[1]), f32x2_to_bf16x2(f[2], f[3]), f32x2_to_bf16x2(f[4], f[5]),
                      f32x2_to_bf16x2(f[6], f[7]));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Sum over the threads of a row: a warp, or the CTA through `red` (one slot
// per warp; the caller alternates two arrays so that one barrier suffices).
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float* red) {
    v = warp_sum(v);
    if (WARP) return v;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    return warp_sum(lane < warps ? red[lane] : 0.0f);
}

// MXFP8 exponent of an fp32 magnitude pattern: as mx_exponent for bf16 ones.
__device__ __forceinline__ int mx_exponent_f32(uint32_t a) {
    if (a > 0x7F800000u) return 128;
    if (a == 0x7F800000u) return 127;
    const int E = (int)(a >> 23);
    if (E == 0) return -127;
    return max(-127, min(127, E - 127 - 8 + ((a & 0x7FFFFFu) > 0x600000u ? 1 : 0)));
}

struct NormArgs {
    const uint4* x;        // row r at x + r ld
    int64_t ld;            // in vectors of 8 elements
    const uint4* res;      // dense, or nullptr
    const uint4* w;
    int64_t rows;
    int nvec;
    float cols, eps;
    uint4* h;              // dense outputs; each may be nullptr
    uint4* y;
    uint2* q;
    void* scales;
    float* rstd;
};

template <int FMT, int V, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kRowWarps : V <= 2 ? 1024 : 512)
rmsnorm_quant_kernel(const NormArgs a) {
    __shared__ float red[32];
    pdl_trigger();
    pdl_wait();
    const int t = WARP ? (threadIdx.x & 31) : threadIdx.x, T = WARP ? 32 : blockDim.x;
    const int64_t row = WARP ? (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= a.rows) return;                              // whole warps (the row's threads) leave together
    const uint4* xr = a.x + row * a.ld;
    const int64_t dense = row * a.nvec;

    uint4 xv[V], rv[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int v = t + i * T;
        xv[i] = rv[i] = make_uint4(0, 0, 0, 0);
        if (v < a.nvec) {
            xv[i] = ld_once(xr + v);
            if (a.res) rv[i] = ld_once(a.res + dense + v);
        }
    }
    float s[V][8], sq = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float r[8];
        unpack8(xv[i], s[i]);
        if (a.res) {
            unpack8(rv[i], r);
#pragma unroll
            for (int j = 0; j < 8; ++j) s[i][j] += r[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) sq = fmaf(s[i][j], s[i][j], sq);
        const int v = t + i * T;
        if (a.h && v < a.nvec) st_v4(a.h + dense + v, pack8(s[i]));
    }
    sq = row_sum<WARP>(sq, red);
    const float rstd = __frcp_rn(__fsqrt_rn(__fdiv_rn(sq, a.cols) + a.eps));
    if (a.rstd && t == 0) a.rstd[row] = rstd;

#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int v = t + i * T;
        const bool in = v < a.nvec;
        float w[8];
        unpack8(in ? __ldg(a.w + v) : make_uint4(0, 0, 0, 0), w);
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            s[i][j] = s[i][j] * rstd * w[j];
            top = max(top, __float_as_uint(s[i][j]) & 0x7FFFFFFFu);   // NaN patterns order above infinity
        }
        if (a.y && in) st_v4(a.y + dense + v, pack8(s[i]));
        if (FMT == kNormFp8) {
            top = group_max<16>(in ? top : 0u);             // the 16 lanes of a 128-element tile, in or out together
            const float sc = top ? __fdiv_rn(__uint_as_float(top), 448.0f) : 1.0f;
            uint32_t c[4];
            if (reciprocal_ok(sc)) {
                const QuotientBracket b = quotient_bracket(sc);
#pragma unroll
                for (int j = 0; j < 4; ++j) c[j] = e4m3x2_of_quotients(s[i][2 * j], s[i][2 * j + 1], b);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    c[j] = f32x2_to_e4m3x2(__fdiv_rn(s[i][2 * j], sc), __fdiv_rn(s[i][2 * j + 1], sc));
            }
            if (in) {
                st_v2(a.q + dense + v, make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16)));
                if ((v & 15) == 0) static_cast<float*>(a.scales)[(dense + v) >> 4] = sc;
            }
        } else if (FMT == kNormMx) {
            top = group_max<4>(in ? top : 0u);
            const int e = mx_exponent_f32(top);
            const float mul = pow2_neg(e == 128 ? 127 : e);
            uint32_t c[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) c[j] = f32x2_to_e4m3x2(s[i][2 * j] * mul, s[i][2 * j + 1] * mul);
            uint2 q = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
            if (e == 128) q = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
            if (in) {
                st_v2(a.q + dense + v, q);
                if ((v & 3) == 0) static_cast<uint8_t*>(a.scales)[(dense + v) >> 2] = (uint8_t)(e + 127);
            }
        }
    }
}

template <int FMT>
cudaError_t launch_norm(const NormArgs& a, int sms, cudaStream_t st) {
    const int nv = a.nvec;
    if (nv <= 128) {
        const dim3 grid((unsigned)((a.rows + kRowWarps - 1) / kRowWarps)), block(32 * kRowWarps);
        if (nv <= 32) return launch_pdl(rmsnorm_quant_kernel<FMT, 1, true>, grid, block, 0, st, a);
        if (nv <= 64) return launch_pdl(rmsnorm_quant_kernel<FMT, 2, true>, grid, block, 0, st, a);
        return launch_pdl(rmsnorm_quant_kernel<FMT, 4, true>, grid, block, 0, st, a);
    }
    // Few rows: latency counts, so a row is spread over as many threads as
    // it has vectors.  Many rows: V = 4 keeps four loads per operand in
    // flight per thread and the barrier among fewer warps.
    const dim3 grid((unsigned)a.rows);
    const auto threads = [&](int v) { return dim3((unsigned)(((nv + v - 1) / v + 31) / 32 * 32)); };
    const bool few = a.rows < 2 * sms;
    if (few && nv <= 1024) return launch_pdl(rmsnorm_quant_kernel<FMT, 1, false>, grid, threads(1), 0, st, a);
    if (few && nv <= 2048) return launch_pdl(rmsnorm_quant_kernel<FMT, 2, false>, grid, threads(2), 0, st, a);
    if (nv <= 2048) return launch_pdl(rmsnorm_quant_kernel<FMT, 4, false>, grid, threads(4), 0, st, a);
    return launch_pdl(rmsnorm_quant_kernel<FMT, 8, false>, grid, threads(8), 0, st, a);
}

// ------------------------------------------------------------------ backward

struct NormBwdArgs {
    const uint4* dy;
    const uint4* x;        // row r at x + r ld
    int64_t ld;            // in vectors of 8 elements
    const uint4* w;
    const float* rstd;
    const uint4* dres;     // or nullptr
    int64_t rows;
    int nvec;
    float cols;
    uint4* dx;
    float* partial;        // [grid, cols] sums of dw over a CTA's rows, or nullptr
};

// CTAs (or warps) take rows r, r + grid, ...; a thread's columns are the
// same for every row, so dw stays in its registers until the end.
template <int V, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kRowWarps : 512)
rmsnorm_bwd_kernel(const NormBwdArgs a) {
    __shared__ float red[2][32];
    __shared__ __align__(16) float acc_s[WARP ? 1024 : 4];
    pdl_trigger();
    pdl_wait();
    const int t = WARP ? (threadIdx.x & 31) : threadIdx.x, T = WARP ? 32 : blockDim.x;
    const int64_t step = WARP ? (int64_t)gridDim.x * kRowWarps : gridDim.x;
    uint4 wv[V];
    float acc[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        wv[i] = t + i * T < a.nvec ? __ldg(a.w + t + i * T) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = 0.0f;
    }
    int turn = 0;
    for (int64_t row = WARP ? (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5) : blockIdx.x; row < a.rows;
         row += step, turn ^= 1) {
        const int64_t dense = row * a.nvec;
        const uint4* xr = a.x + row * a.ld;
        uint4 dv[V], xv[V], ev[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = t + i * T;
            dv[i] = xv[i] = ev[i] = make_uint4(0, 0, 0, 0);
            if (v < a.nvec) {
                dv[i] = ld_once(a.dy + dense + v);
                xv[i] = ld_once(xr + v);
                if (a.dres) ev[i] = ld_once(a.dres + dense + v);
            }
        }
        const float rstd = a.rstd[row];
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float d[8], x[8], w[8];
            unpack8(dv[i], d);
            unpack8(xv[i], x);
            unpack8(wv[i], w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                dot = fmaf(d[j] * w[j], x[j], dot);
                acc[i][j] = fmaf(d[j], x[j] * rstd, acc[i][j]);
            }
        }
        dot = row_sum<WARP>(dot, red[turn]);
        const float c = -__fdiv_rn(dot * rstd, a.cols) * rstd * rstd;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = t + i * T;
            float d[8], x[8], w[8], e[8];
            unpack8(dv[i], d);
            unpack8(xv[i], x);
            unpack8(wv[i], w);
            unpack8(ev[i], e);
#pragma unroll
            for (int j = 0; j < 8; ++j) e[j] += fmaf(x[j], c, d[j] * w[j] * rstd);
            if (v < a.nvec) st_v4(a.dx + dense + v, pack8(e));
        }
    }
    if (!a.partial) return;
    float4* out = reinterpret_cast<float4*>(a.partial) + (int64_t)blockIdx.x * a.nvec * 2;
    if (WARP) {
        // the CTA's eight warps add their sums in order
        for (int wi = 0; wi < kRowWarps; ++wi) {
            if ((int)(threadIdx.x >> 5) == wi) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (t + i * T < a.nvec)
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            float* p = &acc_s[(t + i * T) * 8 + j];
                            *p = wi ? *p + acc[i][j] : acc[i][j];
                        }
            }
            __syncthreads();
        }
        for (int v = threadIdx.x; v < 2 * a.nvec; v += blockDim.x) out[v] = reinterpret_cast<float4*>(acc_s)[v];
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = t + i * T;
            if (v < a.nvec) {
                out[2 * v] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
                out[2 * v + 1] = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
            }
        }
    }
}

// dweight[c] = sum of the partial rows, in a fixed order: warp i of a CTA
// adds rows i, i + 32, ... of its 128 columns, then the warps' sums are added.
__global__ void __launch_bounds__(1024)
rmsnorm_dweight_kernel(const float4* __restrict__ partial, int parts, int nvec4, float4* __restrict__ dweight) {
    __shared__ float4 sum[32][32];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int v = blockIdx.x * 32 + lane;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (v < nvec4) {
#pragma unroll 4
        for (int p = warp; p < parts; p += 32) {
            const float4 u = partial[(int64_t)p * nvec4 + v];
            s.x += u.x; s.y += u.y; s.z += u.z; s.w += u.w;
        }
    }
    sum[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && v < nvec4) {
        for (int i = 1; i < 32; ++i) {
            const float4 u = sum[i][lane];
            s.x += u.x; s.y += u.y; s.z += u.z; s.w += u.w;
        }
        dweight[v] = s;
    }
}

int bwd_vectors(int nvec) { return nvec <= 32 ? 1 : nvec <= 64 ? 2 : nvec <= 2048 ? 4 : 8; }

int bwd_threads(int nvec) {
    if (nvec <= 128) return 32 * kRowWarps;
    const int v = bwd_vectors(nvec);
    return ((nvec + v - 1) / v + 31) / 32 * 32;
}

// About 1024 threads per SM: the registers of more do not fit.
int bwd_grid(int64_t rows, int nvec, int sms) {
    const int64_t tasks = nvec <= 128 ? (rows + kRowWarps - 1) / kRowWarps : rows;
    return (int)min64(tasks, (int64_t)sms * (nvec <= 128 ? 4 : max64(1, 1024 / bwd_threads(nvec))));
}

}  // namespace

cudaError_t launch_rmsnorm_quantize(int fmt, const void* x, int64_t ld_x, const void* residual, const void* weight,
                                    int64_t rows, int64_t cols, float eps, void* h, void* y, void* q, void* scales,
                                    float* rstd, int sms, cudaStream_t st) {
    const NormArgs a{(const uint4*)x, ld_x / 8, (const uint4*)residual, (const uint4*)weight, rows, (int)(cols / 8),
                     (float)cols, eps, (uint4*)h, (uint4*)y, (uint2*)q, scales, rstd};
    if (!q) return launch_norm<kNormNone>(a, sms, st);
    return fmt == FPQ_FP8_1x128 ? launch_norm<kNormFp8>(a, sms, st) : launch_norm<kNormMx>(a, sms, st);
}

size_t rmsnorm_backward_workspace_bytes(int64_t rows, int64_t cols, int sms) {
    return (size_t)bwd_grid(rows, (int)(cols / 8), sms) * (size_t)cols * sizeof(float);
}

cudaError_t launch_rmsnorm_backward(const void* dy, const void* x, int64_t ld_x, const void* weight,
                                    const float* rstd, const void* dres, int64_t rows, int64_t cols, void* dx,
                                    float* dweight, void* workspace, int sms, cudaStream_t st) {
    const int nvec = (int)(cols / 8), grid = bwd_grid(rows, nvec, sms);
    const NormBwdArgs a{(const uint4*)dy, (const uint4*)x, ld_x / 8, (const uint4*)weight, rstd, (const uint4*)dres,
                        rows, nvec, (float)cols, (uint4*)dx, dweight ? (float*)workspace : nullptr};
    cudaError_t e = cudaSuccess;
    if (grid > 0) {
        const dim3 g((unsigned)grid), b((unsigned)bwd_threads(nvec));
        if (nvec <= 32) e = launch_pdl(rmsnorm_bwd_kernel<1, true>, g, b, 0, st, a);
        else if (nvec <= 64) e = launch_pdl(rmsnorm_bwd_kernel<2, true>, g, b, 0, st, a);
        else if (nvec <= 128) e = launch_pdl(rmsnorm_bwd_kernel<4, true>, g, b, 0, st, a);
        else if (nvec <= 2048) e = launch_pdl(rmsnorm_bwd_kernel<4, false>, g, b, 0, st, a);
        else e = launch_pdl(rmsnorm_bwd_kernel<8, false>, g, b, 0, st, a);
    }
    if (e != cudaSuccess || !dweight) return e;
    return launch_pdl(rmsnorm_dweight_kernel, dim3((unsigned)((2 * nvec + 31) / 32)), dim3(1024), 0, st,
                      (const float4*)workspace, grid, 2 * nvec, (float4*)dweight);
}

}  // namespace fpq
