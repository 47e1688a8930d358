// gemv_nvfp4.cu -- products of a few bf16 rows with NVFP4 weights, the form
// that decoding takes: y[m, n] = g sum_k x[m, k] e2m1(W[n, k]) e4m3(S[n, k/16]),
// the weights of one matrix, or for row m those of expert ids[m].
//
// Bound by HBM (9/16 byte per weight) and, close behind, by the instructions
// that decode the codes: at the copy peak an SM has about three instruction
// slots per weight.  So the products run on the tensor cores' register form
// (mma.m16n8k16, weights as the 16-row operand, rows of x as columns), which
// leaves the slots to the decoding and serves 8 rows of x at the price of
// one.  A tcgen05 product would need the decoded weights in shared memory:
// four bytes written there per byte read from HBM.
//
// Weights are decoded exactly: one conversion makes two f16 numbers of two
// codes, one f16x2 multiplication applies the block scale (a code times an
// E4M3 scale has at most six significant bits).  The operands of a product
// have one type, so x becomes f16 too: per row and block of 128 it is
// multiplied by the power of two that takes the block's largest magnitude to
// [2^14, 2^15), and the block's fp32 sum is multiplied back.  That is exact
// for every element within 2^-31 of the block's largest (eight bits above
// f16's smallest step, 2^-24); a smaller one is rounded by at most half a
// step, 2^-39 of the largest, far below what the fp32 sum keeps
// of it.  (With bf16 as the common type nothing of x is rounded, but a pair
// of codes takes four instructions instead of two: 60 us against 37 for one
// row, 32768 x 7168, at that step.)
//
// A CTA takes 16 weight rows per row warp, WR row warps by WK warps along k
// (sixteen warps per SM, in one CTA or two).  A warp walks along k in groups
// of four blocks of 128 weights; a lane holds 32 codes of two rows per block
// (16-byte loads), and loads a block of the next group into the registers of
// the one it has just used, so that three to four blocks are always on their
// way.  x is converted into shared memory once per CTA, or in chunks along k
// where it is too large.  WK and WR follow from n, k and the form alone, so
// a row's result does not depend on what else is in the call.
//
// Measured (weights of HBM, none in L2): one row x 32768 x 7168 29 us (4.6
// TB/s), 8 rows 35.5, 16 rows 45; 2048 x 7168, one row 5.2; 8 tokens x 8 of
// 64 experts, 2048 x 7168, 83 us, 32 tokens 159.  Bound by the data pipe of
// the L1 (70% busy for 8 tokens, 80 for 16 rows): a load of codes takes a
// cycle for each of the eight rows that it touches, so does each of a block's
// two 16-bit loads of scales, an eighth of the bytes, and x is read from
// shared memory in the width of the decoded weights for every eight columns,
// those past the last too.  Its conversion is another 8 us of the 45; the
// sixteen-column kernels spill 40 bytes at 128 registers.  One token through
// one expert takes 11.6 us, where the launch rule's eight experts leave most
// SMs without a CTA.  Not better, and not here: loads
// of 32 bytes, half as many for the pipe (8 tokens 82 us, but 16 rows 48 and
// one 31: fewer, larger pieces on their way); 24 or 32 warps of fewer
// registers (16 rows 49 and 59, 8 tokens 88 and 92); the blocks through a
// ring in shared memory, by asynchronous copies (45 instead of 37 for one
// row: more instructions) or by TMA and a warp of its own (34.5, 16 rows 48,
// but 8.7 instead of 5.3 and 100 instead of 85); two row tiles per warp,
// which halves the reads of x (16 rows 55: registers).
#include <cuda_runtime.h>

#include "common.cuh"
#include "layer.hpp"
#include "quant_unit.cuh"

namespace fpq {

namespace {

constexpr int kGemvWarps = 16;             // of an SM, in one CTA or two
constexpr int kBlock = 128;               // weights of a row per warp and step
constexpr int kGroup = 4;                 // blocks per group
constexpr int kXBytes = 112 * 1024;       // of an SM for x

struct GemvArgs {
    const uint16_t* x;          // row m at x + (m / x_div) k
    int m, x_div;
    const int32_t* ids;         // [m], or nullptr
    int experts;
    const uint8_t* wq;          // [experts, n, k / 2]
    const uint8_t* ws;          // [experts, n, k / 16]
    const float* wg;            // [experts]
    int64_t n;
    int k;
    void* y;                    // [m, n]
    uint32_t* err;
    int y_f32;
    int cap;                    // pairs of an expert that a CTA takes (at most the columns)
    int wk, wr;                 // warps along k, row tiles per CTA
    int cols, chunk;            // columns and groups of x in shared memory at a time
};

__device__ __forceinline__ void put(void* y, int64_t at, float v, bool f32) {
    if (f32) static_cast<float*>(y)[at] = v;
    else static_cast<uint16_t*>(y)[at] = (uint16_t)f32_to_bf16(v);
}

template <bool FIRST>                      // FIRST: c = a b, else c += a b
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    if (FIRST)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%10,%10,%10,%10};"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t f32x2_to_f16x2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// Eight codes times the scale pair sc: out[i] = elements (2 i, 2 i + 1).
__device__ __forceinline__ void decode8(uint32_t w, uint32_t sc, uint32_t (&out)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(out[0]), "=r"(out[1]), "=r"(out[2]), "=r"(out[3]) : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = mul_f16x2(out[i], sc);
}

struct Block {                             // a lane's 32 codes and two scales of rows g and g + 8
    uint4 q[2];
    uint32_t s[2];
};

// TILES: column tiles of eight (rows of x); CTAS: CTAs per SM; EXPERTS: ids
// are given.
template <int TILES, int CTAS, bool EXPERTS>
__global__ void __launch_bounds__(32 * kGemvWarps / CTAS, CTAS)
gemv_nvfp4_kernel(const GemvArgs a) {
    constexpr int COLS = 8 * TILES;
    extern __shared__ __align__(16) uint8_t smem[];         // per column a chunk of x, then the blocks' factors
    __shared__ float red[kGemvWarps / CTAS][32][COLS / 2];
    __shared__ int member[COLS], xrow[COLS];
    __shared__ uint32_t same[32];                            // of each 32 pairs, those of this CTA's expert
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int threads = blockDim.x, WK = a.wk, WR = a.wr, wk = warp % WK, wr = warp / WK;
    const int64_t tile0 = (int64_t)blockIdx.x * WR;          // the CTA's first 16-row tile
    int64_t e = 0;
    int count;
    if (EXPERTS) {
        // blockIdx.y is a pair; every cap-th pair of an expert takes itself and
        // the next cap - 1, the others have nothing to do and find that out
        // in one latency of memory: all parts of ids are loaded at once (one
        // part after the other: 181 us instead of 159 for 32 tokens x 8)
        const int p = blockIdx.y, id = a.ids[p], parts = (a.m + 31) / 32;
        for (int c = warp; c < parts; c += threads / 32) {   // whole warps
            const uint32_t mask = __ballot_sync(0xFFFFFFFFu, c * 32 + lane < a.m && a.ids[min(c * 32 + lane, a.m - 1)] == id);
            if (lane == 0) same[c] = mask;
        }
        e = id;
        if (id < 0 || id >= a.experts) {
            if (tid == 0) raise_device_error(a.err, FPQ_ERR_DEVICE_BAD_INPUT);
            for (int i = tid; i < 16 * WR; i += threads)
                if (tile0 * 16 + i < a.n) put(a.y, (int64_t)p * a.n + tile0 * 16 + i, 0.0f, a.y_f32);
            return;
        }
        __syncthreads();
        // every warp counts the pairs of the expert before this one, the first
        // lists it and the next ones; lane c has part c
        const uint32_t mask = lane < parts ? same[lane] : 0u;
        const uint32_t earlier = lane < (p >> 5) ? mask : lane == (p >> 5) ? mask & ((1u << (p & 31)) - 1u) : 0u;
        if (__reduce_add_sync(0xFFFFFFFFu, (unsigned)__popc(earlier)) % (unsigned)a.cap) return;
        uint32_t later = mask & ~earlier;
        int at = __popc(later);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xFFFFFFFFu, at, o);
            if (lane >= o) at += u;
        }
        count = min(__shfl_sync(0xFFFFFFFFu, at, 31), a.cap);
        at -= __popc(later);
        if (warp == 0)
            for (; later && at < count; later &= later - 1, ++at) {
                member[at] = lane * 32 + __ffs(later) - 1;
                xrow[at] = member[at] / a.x_div;
            }
        __syncthreads();
    } else {
        count = a.m;
        if (tid < COLS) member[tid] = xrow[tid] = tid;
        __syncthreads();
    }

    const int groups = (a.k + kGroup * kBlock - 1) / (kGroup * kBlock), whole = a.k / (kGroup * kBlock);
    // rows past the last read the last row; their sums are not written
    const int64_t r0 = min64((tile0 + wr) * 16 + g, a.n - 1), r1 = min64((tile0 + wr) * 16 + g + 8, a.n - 1);
    const uint8_t* q0 = a.wq + (e * a.n + r0) * (a.k / 2) + 16 * t;
    const uint8_t* q1 = a.wq + (e * a.n + r1) * (a.k / 2) + 16 * t;
    const uint8_t* s0 = a.ws + (e * a.n + r0) * (a.k / 16) + 2 * t;
    const uint8_t* s1 = a.ws + (e * a.n + r1) * (a.k / 16) + 2 * t;
    const auto load = [&](Block& b, int group, int i) {      // block i of the group
        const int at = (group * kGroup + i) * kBlock;
        if (group < whole || at + 32 * t < a.k) {
            b.q[0] = ld_stream(q0 + (at >> 1));
            b.q[1] = ld_stream(q1 + (at >> 1));
            b.s[0] = __ldg(reinterpret_cast<const uint16_t*>(s0 + (at >> 4)));
            b.s[1] = __ldg(reinterpret_cast<const uint16_t*>(s1 + (at >> 4)));
        } else {
            b.q[0] = b.q[1] = make_uint4(0, 0, 0, 0);
            b.s[0] = b.s[1] = 0;
        }
    };
    Block blk[kGroup];
#pragma unroll
    for (int i = 0; i < kGroup; ++i) load(blk[i], wk, i);    // zeros if there is no such group

    // x in shared memory: column c at c x_stride; in it block b at 256 b, word
    // j of lane t at 64 j + 16 t.  The stride is 64 bytes past a multiple of
    // 128, so that the eight columns of a read fall on different banks.
    // Behind the columns one fp32 factor per block and column.
    const int chunk_blocks = a.chunk * kGroup;
    const int x_stride = chunk_blocks * 256 + 64;
    float* const factors = reinterpret_cast<float*>(smem + a.cols * x_stride);
    // A unit is 64 bytes, the 32 elements of a lane's block; four adjacent
    // threads hold a block.
    const int col_units = chunk_blocks * 4, step_col = threads / col_units, step_u = threads % col_units;
    const auto stage = [&](int group0) {
        int col = tid / col_units, u = tid % col_units;
        for (int i = warp * 32; i < count * col_units; i += threads) {      // whole warps: there are shuffles
            const int k0 = group0 * (kGroup * kBlock) + u * 32;
            const bool in = col < count;
            uint4 v[4] = {};
            if (in && k0 < a.k) {
                const uint4* src = reinterpret_cast<const uint4*>(a.x + (int64_t)xrow[col] * a.k + k0);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = __ldg(src + j);
            }
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                top = absmax_bf16x2(top, absmax_bf16x2(absmax_bf16x2(v[j].x, v[j].y), absmax_bf16x2(v[j].z, v[j].w)));
            top = group_max<4>(hmax2(abs2(top)));
            // 2^f takes the block's largest to [2^14, 2^15); f within what one
            // bf16 factor holds (largest below 2^-112), -112 with an infinity
            // or a NaN (the finite elements stay finite), 0 for a zero block
            const int f = top >= 0x7F80u ? -112 : top == 0 ? 0 : min(127, 141 - (int)(top >> 7));
            const uint32_t s1 = (uint32_t)(127 + f) << 7, s2 = s1 | (s1 << 16);
            if (in) {
                uint8_t* const dst = smem + col * x_stride + (u >> 2) * 256 + (u & 3) * 16;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        w[h] = mul_bf16x2(w[h], s2);
                        w[h] = f32x2_to_f16x2(bf16_lo(w[h]), bf16_hi(w[h]));
                    }
                    *reinterpret_cast<uint4*>(dst + 64 * j) = make_uint4(w[0], w[1], w[2], w[3]);
                }
                if ((u & 3) == 0) factors[(u >> 2) * COLS + col] = pow2_neg(f);
            }
            col += step_col;
            u += step_u;
            if (u >= col_units) { u -= col_units; ++col; }
        }
    };

    float acc[TILES][4] = {};
    // columns past the last read the last one, and factors that nobody wrote;
    // their sums are not written
    uint32_t xb[TILES];
#pragma unroll
    for (int h = 0; h < TILES; ++h) xb[h] = min(8 * h + g, count - 1) * x_stride + 16 * t;
    for (int group0 = 0; group0 < groups; group0 += a.chunk) {
        if (group0) __syncthreads();
        stage(group0);
        __syncthreads();
        const int last = min(groups - group0, a.chunk);
        for (int gl = (wk - group0 % WK + WK) % WK; gl < last; gl += WK) {   // groups wk, wk + WK, ... of all
#pragma unroll
            for (int i = 0; i < kGroup; ++i) {
                uint32_t sc[2][2];                           // [row][scale]
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint32_t h = e4m3x2_to_f16x2(blk[i].s[r]);
                    sc[r][0] = __byte_perm(h, h, 0x1010);
                    sc[r][1] = __byte_perm(h, h, 0x3232);
                }
                const uint32_t w0[4] = {blk[i].q[0].x, blk[i].q[0].y, blk[i].q[0].z, blk[i].q[0].w};
                const uint32_t w1[4] = {blk[i].q[1].x, blk[i].q[1].y, blk[i].q[1].z, blk[i].q[1].w};
                float sum[TILES][2][4];                      // two chains per column tile
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t d0[4], d1[4];
                    decode8(w0[j], sc[0][j >> 1], d0);
                    decode8(w1[j], sc[1][j >> 1], d1);
#pragma unroll
                    for (int h = 0; h < TILES; ++h) {
                        const uint4 b = *reinterpret_cast<const uint4*>(smem + xb[h] + gl * (kGroup * 256) + i * 256 + j * 64);
                        if (j == 0) {
                            mma_f16<true>(sum[h][0], d0[0], d1[0], d0[1], d1[1], b.x, b.y);
                            mma_f16<true>(sum[h][1], d0[2], d1[2], d0[3], d1[3], b.z, b.w);
                        } else {
                            mma_f16<false>(sum[h][0], d0[0], d1[0], d0[1], d1[1], b.x, b.y);
                            mma_f16<false>(sum[h][1], d0[2], d1[2], d0[3], d1[3], b.z, b.w);
                        }
                    }
                }
                load(blk[i], group0 + gl + WK, i);
#pragma unroll
                for (int h = 0; h < TILES; ++h) {
                    const float2 f = *reinterpret_cast<const float2*>(factors + (gl * kGroup + i) * COLS + 8 * h + 2 * t);
#pragma unroll
                    for (int c = 0; c < 4; ++c) acc[h][c] = fmaf(sum[h][0][c] + sum[h][1][c], c & 1 ? f.y : f.x, acc[h][c]);
                }
            }
        }
    }

    // sums of the WK warps of a row tile, in order
#pragma unroll
    for (int h = 0; h < TILES; ++h)
#pragma unroll
        for (int f = 0; f < 4; ++f) red[warp][lane][4 * h + f] = acc[h][f];
    __syncthreads();
    const float scale = __ldg(a.wg + e);
    const int rows = 16 * WR;
    for (int o = tid; o < rows * count; o += threads) {
        const int r = o % rows, col = o / rows;              // consecutive threads: consecutive weight rows
        const int64_t row = tile0 * 16 + r;
        if (row >= a.n) continue;
        // fragment: row g (+ 8 for entries 2, 3), columns 2 t, 2 t + 1 of its tile
        const int from = (r & 7) * 4 + ((col & 7) >> 1), at = (col >> 3) * 4 + ((r >> 3) & 1) * 2 + (col & 1);
        float v = 0.0f;
        for (int w = 0; w < WK; ++w) v += red[(r >> 4) * WK + w][from][at];
        put(a.y, (int64_t)member[col] * a.n + row, v * scale, a.y_f32);
    }
}

template <int TILES, int CTAS, bool EXPERTS>
cudaError_t gemv(GemvArgs a, cudaStream_t st) {
    const int groups = (a.k + kGroup * kBlock - 1) / (kGroup * kBlock);
    a.cols = EXPERTS ? a.cap : a.m;
    const int fit = kXBytes / CTAS / (a.cols * kGroup * 256);
    a.chunk = fit < groups ? fit : groups;
    const int blocks = a.chunk * kGroup;
    const int smem = a.cols * (blocks * 256 + 64) + blocks * 8 * TILES * (int)sizeof(float);
    // x and the columns' padding, and a factor per block and column of a tile:
    // the most blocks are those of a single column
    constexpr int most = kXBytes / CTAS + 64 * 8 * TILES + kXBytes / CTAS / 256 * 8 * TILES * (int)sizeof(float);
    static_assert(CTAS * (most + 20 * 1024) <= 227 * 1024, "with the static arrays, an SM's shared memory");
    constexpr auto kernel = gemv_nvfp4_kernel<TILES, CTAS, EXPERTS>;
    const cudaError_t e = allow_shared_memory<kernel, most>();
    if (e != cudaSuccess) return e;
    const int64_t tiles = (a.n + 15) / 16;
    return launch_pdl(kernel, dim3((unsigned)((tiles + a.wr - 1) / a.wr), (unsigned)(EXPERTS ? a.m : 1)),
                      dim3(32u * a.wk * a.wr), smem, st, a);
}

}  // namespace

cudaError_t launch_gemv_nvfp4(const void* x, int64_t m, int x_div, int tokens, const int32_t* ids, int experts,
                              const void* wq, const void* ws, const float* wg, int64_t n, int64_t k, void* y,
                              int y_f32, uint32_t* err, int sms, cudaStream_t st) {
    // As many warps along k as leave one wave of an SM's sixteen, up to one for
    // each group (2048 x 7168, one row: 16 warps for 14 groups 5.2 us, 8 warps
    // 6.8), then as many row tiles per CTA as bring the CTAs into one
    // wave: with 148 SMs and two CTAs each, 2048 tiles become 293 CTAs of
    // seven warps; 128 tiles become 128 CTAs of sixteen.  The expert form
    // counts on eight experts per call.
    const int64_t tiles = (n + 15) / 16, waves = tiles * (ids ? 8 : 1), groups = (k + kGroup * kBlock - 1) / (kGroup * kBlock);
    int wk = kGemvWarps;
    while (wk > 1 && (waves * wk > kGemvWarps * (int64_t)sms || wk / 2 >= groups)) wk /= 2;
    // Sixteen columns for more than eight rows, or where an expert can be
    // expected to have more than eight pairs.  Then one CTA per SM: x fills
    // its shared memory, and is converted once for twice the weights.
    const bool wide = ids ? m > 8 && m > 4 * (int64_t)experts : m > 8;
    const int ctas = wide || wk == kGemvWarps ? 1 : 2;
    const int64_t wr = max64(1, min64(kGemvWarps / ctas / wk, (waves + ctas * sms - 1) / (ctas * sms)));
    // An expert has at most a pair of each token (of a token that names it
    // twice, two).  Four where that is far above the average: they take half
    // of the shared memory of eight, which is the loads' cache.
    const int cap = wide ? 16 : tokens < 4 ? tokens : m <= 2 * (int64_t)experts ? 4 : 8;
    const GemvArgs a{(const uint16_t*)x, (int)m, x_div, ids, experts, (const uint8_t*)wq, (const uint8_t*)ws, wg, n,
                     (int)k, y, err, y_f32, cap, wk, (int)wr, 0, 0};
    if (ids) return wide ? gemv<2, 1, true>(a, st) : ctas == 1 ? gemv<1, 1, true>(a, st) : gemv<1, 2, true>(a, st);
    return wide ? gemv<2, 1, false>(a, st) : ctas == 1 ? gemv<1, 1, false>(a, st) : gemv<1, 2, false>(a, st);
}

}  // namespace fpq
