// moe_combine.cu -- the way back of a mixture-of-experts layer: each token's
// expert rows, weighted and added, and the backward pass; and the row of
// every (token, choice) pair in the dispatched buffer.
//
//   out[t]    = add[t] + sum_j weights[t, j] y[row(t, j)]      j ascending, fp32, one rounding
//   dy[row]   = weights[t, j] dout[t]
//   dweights[t, j] = sum_h dout[t, h] y[row(t, j), h]          fp32
//
// A pair's row is rows[t, j], or its own index t topk + j without a row map;
// -1 means the pair was dropped: it adds nothing, and its dweight is 0.
// Rows are gathered, never scattered with atomics: every output has one
// writer and a fixed order of additions.
//
// Bound by HBM: the forward reads topk rows and writes one per token, the
// backward reads and writes topk rows.  A thread keeps eight loads of 16
// bytes in flight: one vector of eight rows, two of four or four of two
// (with one vector of two rows 16000 tokens x 2048, two choices took 61 us
// forward and 152 back; with four of two 39 and 53).  Measured, bf16: 8192
// tokens x 7168, eight choices and an addend 185 us (6.34 TB/s), back 338 us
// (5.91 TB/s); 16 tokens 2.6 and 5.7 us, which is latency.  Zeros in the rows
// that no pair names, where they are asked for, take 2 to 4 us more.
#include <type_traits>

#include <cuda_runtime.h>

#include "common.cuh"
#include "layer.hpp"

namespace fpq {

namespace {

constexpr int kInFlight = 8;              // vectors per thread: KB rows of kInFlight / KB vectors each
constexpr int kCombineThreads = 256;

// Eight consecutive elements as fp32; index in units of eight.
template <bool F32> struct Vec8;
template <> struct Vec8<false> {
    uint4 a;
    __device__ __forceinline__ void load(const void* p, int64_t v) { a = ld_stream(static_cast<const uint4*>(p) + v); }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        f[0] = bf16_lo(a.x); f[1] = bf16_hi(a.x); f[2] = bf16_lo(a.y); f[3] = bf16_hi(a.y);
        f[4] = bf16_lo(a.z); f[5] = bf16_hi(a.z); f[6] = bf16_lo(a.w); f[7] = bf16_hi(a.w);
    }
    static __device__ __forceinline__ void store(void* p, int64_t v, const float (&f)[8]) {
        st_v4(static_cast<uint4*>(p) + v, make_uint4(f32x2_to_bf16x2(f[0], f[1]), f32x2_to_bf16x2(f[2], f[3]),
                                                     f32x2_to_bf16x2(f[4], f[5]), f32x2_to_bf16x2(f[6], f[7])));
    }
};
template <> struct Vec8<true> {
    uint4 a, b;
    __device__ __forceinline__ void load(const void* p, int64_t v) {
        a = ld_stream(static_cast<const uint4*>(p) + 2 * v);
        b = ld_stream(static_cast<const uint4*>(p) + 2 * v + 1);
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y); f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
        f[4] = __uint_as_float(b.x); f[5] = __uint_as_float(b.y); f[6] = __uint_as_float(b.z); f[7] = __uint_as_float(b.w);
    }
    static __device__ __forceinline__ void store(void* p, int64_t v, const float (&f)[8]) {
        uint4* o = static_cast<uint4*>(p) + 2 * v;
        st_v4(o, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])));
        st_v4(o + 1, make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7])));
    }
};

struct CombineArgs {
    const void* y;
    int64_t y_rows;
    const int32_t* rows;        // [tokens, topk], or nullptr
    const float* weights;       // [tokens, topk]
    int64_t tokens;
    int topk, nvec;
    const void* add;            // forward: bf16 [tokens, hidden], or nullptr
    const void* dout;           // backward
    void* out;                  // forward: [tokens, hidden]; backward: dy
    float* dweights;
    uint32_t* err;
    int32_t* owner;             // backward: [y_rows], or nullptr; a named row's gets its pair
};

// Row of pair p, -1 if it is dropped or outside the buffer.
__device__ __forceinline__ int64_t pair_row(const CombineArgs& a, int64_t p, bool report) {
    if (!a.rows) return p;
    const int32_t r = __ldg(a.rows + p);
    if (r >= -1 && r < a.y_rows) return r;
    if (report) raise_device_error(a.err, FPQ_ERR_DEVICE_BAD_INPUT);
    return -1;
}

// CTA (x, y): the y-th part of token x's row, kInFlight / KB vectors per thread.
template <bool Y32, bool OUT32, int KB>
__global__ void __launch_bounds__(kCombineThreads)
moe_combine_kernel(const CombineArgs a) {
    constexpr int VB = kInFlight / KB;
    pdl_trigger();
    pdl_wait();
    const int64_t tok = blockIdx.x;
    const int v0 = blockIdx.y * blockDim.x * VB + threadIdx.x, step = blockDim.x;
    if (v0 >= a.nvec) return;
    float acc[VB][8];
#pragma unroll
    for (int i = 0; i < VB; ++i) {
        if (a.add && v0 + i * step < a.nvec) {
            Vec8<false> u;
            u.load(a.add, tok * a.nvec + v0 + i * step);
            u.get(acc[i]);
        } else {
#pragma unroll
            for (int c = 0; c < 8; ++c) acc[i][c] = 0.0f;
        }
    }
    for (int j0 = 0; j0 < a.topk; j0 += KB) {
        Vec8<Y32> u[KB][VB];
        float w[KB];
        bool ok[KB];
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            ok[j] = j0 + j < a.topk;
            if (!ok[j]) continue;
            const int64_t p = tok * a.topk + j0 + j, r = pair_row(a, p, threadIdx.x == 0);
            ok[j] = r >= 0;
            if (!ok[j]) continue;
            w[j] = __ldg(a.weights + p);
#pragma unroll
            for (int i = 0; i < VB; ++i)
                if (v0 + i * step < a.nvec) u[j][i].load(a.y, r * a.nvec + v0 + i * step);
        }
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            if (!ok[j]) continue;
#pragma unroll
            for (int i = 0; i < VB; ++i) {
                if (v0 + i * step >= a.nvec) continue;
                float f[8];
                u[j][i].get(f);
#pragma unroll
                for (int c = 0; c < 8; ++c) acc[i][c] = fmaf(w[j], f[c], acc[i][c]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < VB; ++i)
        if (v0 + i * step < a.nvec) Vec8<OUT32>::store(a.out, tok * a.nvec + v0 + i * step, acc[i]);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// A token per warp where there are many (no barrier), else per CTA.  dout's
// vectors are read once per KB choices (from L1 after the first), each y
// vector once; the dots are reduced at the end.
template <bool Y32, bool D32, int KB, bool WARP>
__global__ void __launch_bounds__(kCombineThreads)
moe_combine_bwd_kernel(const CombineArgs a) {
    constexpr int VB = kInFlight / KB;
    __shared__ float red[kCombineThreads / 32][KB];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int64_t tok = WARP ? (int64_t)blockIdx.x * warps + warp : blockIdx.x;
    if (tok >= a.tokens) return;                             // whole warps; with a CTA per token never
    const int t = WARP ? lane : threadIdx.x, T = WARP ? 32 : blockDim.x;
    for (int j0 = 0; j0 < a.topk; j0 += KB) {
        int64_t r[KB];
        float w[KB], dot[KB];
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            const int64_t p = tok * a.topk + j0 + j;
            r[j] = j0 + j < a.topk ? pair_row(a, p, t == 0) : -1;
            if (a.owner && t == 0 && r[j] >= 0) a.owner[r[j]] = (int32_t)p;
            w[j] = r[j] >= 0 ? __ldg(a.weights + p) : 0.0f;
            dot[j] = 0.0f;
        }
        for (int v0 = t; v0 < a.nvec; v0 += T * VB) {
            Vec8<D32> d[VB];
            Vec8<Y32> u[KB][VB];
#pragma unroll
            for (int i = 0; i < VB; ++i) {
                const int v = v0 + i * T;
                if (v >= a.nvec) continue;
                d[i].load(a.dout, tok * a.nvec + v);
#pragma unroll
                for (int j = 0; j < KB; ++j)
                    if (r[j] >= 0) u[j][i].load(a.y, r[j] * a.nvec + v);
            }
#pragma unroll
            for (int i = 0; i < VB; ++i) {
                const int v = v0 + i * T;
                if (v >= a.nvec) continue;
                float df[8];
                d[i].get(df);
#pragma unroll
                for (int j = 0; j < KB; ++j) {
                    if (r[j] < 0) continue;
                    float f[8];
                    u[j][i].get(f);
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        dot[j] = fmaf(df[c], f[c], dot[j]);
                        f[c] = w[j] * df[c];
                    }
                    Vec8<Y32>::store(a.out, r[j] * a.nvec + v, f);
                }
            }
        }
        if (WARP) {
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                const float s = warp_sum(dot[j]);
                if (lane == 0 && j0 + j < a.topk) a.dweights[tok * a.topk + j0 + j] = s;
            }
        } else {
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                const float s = warp_sum(dot[j]);
                if (lane == 0) red[warp][j] = s;
            }
            __syncthreads();
            if (threadIdx.x < KB && j0 + (int)threadIdx.x < a.topk) {
                float s = 0.0f;
                for (int i = 0; i < warps; ++i) s += red[i][threadIdx.x];
                a.dweights[tok * a.topk + j0 + threadIdx.x] = s;
            }
            __syncthreads();
        }
    }
}

// Zeros into the rows of dy that no pair names.  A row is named if its owner is
// a pair that names it, so the owners need no initial value: what an unnamed
// row's memory holds is no pair, or one with another row.  A row per thread,
// the unnamed ones written by the whole warp; with none a launch, 2 us.
constexpr int kClearThreads = 256;

__global__ void __launch_bounds__(kClearThreads)
moe_clear_rows_kernel(const int32_t* rows, int64_t pairs, int64_t y_rows, const int32_t* owner, int64_t row_vecs,
                      uint4* dy) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t r = (int64_t)blockIdx.x * kClearThreads + threadIdx.x, first = r - lane;
    bool unnamed = false;
    if (r < y_rows) {
        const int64_t p = rows ? owner[r] : r;
        unnamed = p < 0 || p >= pairs || (rows && rows[p] != r);
    }
    for (uint32_t left = __ballot_sync(0xFFFFFFFFu, unnamed); left; left &= left - 1) {
        uint4* const row = dy + (first + __ffs(left) - 1) * row_vecs;
        for (int64_t v = lane; v < row_vecs; v += 32) st_v4(row + v, make_uint4(0, 0, 0, 0));
    }
}

// rows[t, j] of every pair: dst_row0 of its expert + its slot, the slot as
// the dispatch kernel counts it (one warp per chunk of tokens, from the
// chunk's slot bases, in token then choice order).  -1 for an id out of range.
constexpr int kRowWarps = 8;

__global__ void __launch_bounds__(32 * kRowWarps)
moe_pair_rows_kernel(const int32_t* __restrict__ ids, int64_t tokens, int topk, int experts,
                     const int32_t* __restrict__ base, int64_t tpc, int64_t chunks,
                     const int64_t* __restrict__ dst_row0, int32_t* __restrict__ rows) {
    extern __shared__ int32_t run_all[];                    // [kRowWarps][experts] running slots
    pdl_trigger();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t c = (int64_t)blockIdx.x * kRowWarps + warp;
    if (c >= chunks) return;
    int32_t* run = run_all + warp * experts;
    const int64_t p0 = c * tpc * topk, p1 = min64(tokens, (c + 1) * tpc) * topk;
    for (int e = lane; e < experts; e += 32) run[e] = base[(int64_t)e * chunks + c];
    __syncwarp();
    for (int64_t p = p0; p < p1; p += 32) {
        // 32 pairs at a time: a pair's slot is its expert's running slot plus
        // the earlier lanes with the same expert
        const bool in = p + lane < p1;
        const int e = in ? ids[p + lane] : -1;
        const bool ok = e >= 0 && e < experts;
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, ok ? e : -1);
        const int before = __popc(same & ((1u << lane) - 1u));
        const int slot = ok ? run[e] + before : 0;
        __syncwarp();
        if (ok && (same >> lane) == 1u) run[e] = slot + 1;   // the last lane of the expert
        __syncwarp();
        if (in) rows[p + lane] = ok ? (int32_t)(dst_row0[e] + slot) : -1;
    }
}

}  // namespace

cudaError_t launch_moe_pair_rows(const int32_t* ids, int64_t tokens, int topk, int experts, const void* workspace,
                                 const int64_t* dst_row0, int32_t* rows, cudaStream_t st) {
    const int64_t tpc = moe_tokens_per_chunk(tokens), chunks = moe_chunks(tokens);
    if (chunks == 0) return cudaSuccess;
    const int32_t* base = static_cast<const int32_t*>(workspace) + (size_t)experts * (size_t)chunks;
    return launch_pdl(moe_pair_rows_kernel, dim3((unsigned)((chunks + kRowWarps - 1) / kRowWarps)),
                      dim3(32 * kRowWarps), kRowWarps * experts * sizeof(int32_t), st, ids, tokens, topk, experts,
                      base, tpc, chunks, dst_row0, rows);
}

namespace {

template <bool Y32, bool OUT32, int KB>
cudaError_t combine(const CombineArgs& a, cudaStream_t st) {
    const int per = (a.nvec + kInFlight / KB - 1) / (kInFlight / KB);      // threads that a row takes
    const int threads = per >= kCombineThreads ? kCombineThreads : (per + 31) / 32 * 32;
    return launch_pdl(moe_combine_kernel<Y32, OUT32, KB>, dim3((unsigned)a.tokens, (unsigned)((per + threads - 1) / threads)),
                      dim3((unsigned)threads), 0, st, a);
}

template <bool Y32, bool D32, int KB>
cudaError_t combine_backward(const CombineArgs& a, int sms, cudaStream_t st) {
    // A warp per token needs tokens for sixteen warps per SM: 16000 tokens x
    // 2048, two choices 53 us (a CTA per token 98), 8000 x 512 x 8 24 us (25),
    // 8192 x 7168 x 8 337 us (329); with fewer, a CTA per token is done sooner:
    // 16 tokens x 7168, eight choices 5.7 us (a warp per token 24).
    if (a.tokens >= 16 * (int64_t)sms)
        return launch_pdl(moe_combine_bwd_kernel<Y32, D32, KB, true>,
                          dim3((unsigned)((a.tokens + kCombineThreads / 32 - 1) / (kCombineThreads / 32))),
                          dim3(kCombineThreads), 0, st, a);
    const int threads = a.nvec >= kCombineThreads ? kCombineThreads : (a.nvec + 31) / 32 * 32;
    return launch_pdl(moe_combine_bwd_kernel<Y32, D32, KB, false>, dim3((unsigned)a.tokens), dim3((unsigned)threads), 0,
                      st, a);
}

template <typename F>
cudaError_t by_types(bool y32, bool o32, int topk, F&& f) {
    const auto by_topk = [&](auto y, auto o) {
        if (topk <= 2) return f(y, o, std::integral_constant<int, 2>());
        if (topk <= 4) return f(y, o, std::integral_constant<int, 4>());
        return f(y, o, std::integral_constant<int, 8>());
    };
    if (y32) return o32 ? by_topk(std::true_type(), std::true_type()) : by_topk(std::true_type(), std::false_type());
    return o32 ? by_topk(std::false_type(), std::true_type()) : by_topk(std::false_type(), std::false_type());
}

}  // namespace

cudaError_t launch_moe_combine(const void* y, int y_f32, int64_t y_rows, const int32_t* rows, const float* weights,
                               int64_t tokens, int topk, int64_t hidden, const void* add, void* out, int out_f32,
                               uint32_t* err, cudaStream_t st) {
    const CombineArgs a{y, y_rows, rows, weights, tokens, topk, (int)(hidden / 8), add, nullptr, out, nullptr, err,
                        nullptr};
    return by_types(y_f32 != 0, out_f32 != 0, topk, [&](auto y32, auto o32, auto kb) {
        return combine<decltype(y32)::value, decltype(o32)::value, decltype(kb)::value>(a, st);
    });
}

cudaError_t launch_moe_combine_backward(const void* dout, int dout_f32, const void* y, int y_f32, int64_t y_rows,
                                        const int32_t* rows, const float* weights, int64_t tokens, int topk,
                                        int64_t hidden, void* dy, float* dweights, int32_t* owner, uint32_t* err,
                                        int sms, cudaStream_t st) {
    const CombineArgs a{y, y_rows, rows, weights, tokens, topk, (int)(hidden / 8), nullptr, dout, dy, dweights, err,
                        owner};
    return by_types(y_f32 != 0, dout_f32 != 0, topk, [&](auto y32, auto d32, auto kb) {
        return combine_backward<decltype(y32)::value, decltype(d32)::value, decltype(kb)::value>(a, sms, st);
    });
}

cudaError_t launch_moe_clear_rows(const int32_t* rows, int64_t pairs, int64_t y_rows, const int32_t* owner,
                                  int64_t row_bytes, void* dy, cudaStream_t st) {
    return launch_pdl(moe_clear_rows_kernel, dim3((unsigned)((y_rows + kClearThreads - 1) / kClearThreads)),
                      dim3(kClearThreads), 0, st, rows, pairs, y_rows, owner, row_bytes / 16, (uint4*)dy);
}

}  // namespace fpq
