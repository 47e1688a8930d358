// gemv_nvfp4.cu -- products of a few bf16 rows with NVFP4 weights, the form
// that decoding takes: y[m, n] = g sum_k x[m, k] e2m1(W[n, k]) e4m3(S[n, k/16]),
// the weights of one matrix, or for row m those of expert ids[m].
//
// Bound by HBM (9/16 byte per weight) and, close behind, by the instructions
// that decode the codes: at the copy peak an SM has about three instruction
// slots per weight.  So the products run on the tensor cores' register form
// (mma.m16n8k16, weights as the 16-row operand, up to 16 rows of x as
// columns), which leaves the slots to the decoding and serves 8 rows of x at
// the price of one.  A tcgen05 product would need the decoded weights in
// shared memory: four bytes written there per byte read from HBM.
//
// Decoding is exact.  A code times its block scale has at most six
// significant bits, so it is a bf16 number:  the code's three magnitude bits
// at the bottom of a bf16's exponent field and the top of its mantissa are
// the value times 2^-126 (0.5 as a subnormal), and one bf16x2 multiplication
// by the scale times 2^117 gives code * scale * 2^-9.  The sum is fp32; 2^9
// and g multiply it at the end.  Element i and i + 4 of a 32-bit word of
// eight codes decode as a pair, so x's elements are paired the same way.
//
// A CTA of eight warps takes 16 weight rows per row warp, WR row warps by WK
// warps along k (WR WK = 8).  A warp's step is a block of 128 weights of its
// 16 rows: each lane copies 32 consecutive codes of two rows to the warp's own
// shared-memory ring, kStages - 1 steps ahead, with no barrier.  x's next
// chunk travels through registers, where its elements are paired, into a
// double buffer; one block barrier per chunk.  WK and WR follow from n and k
// alone, so a row's result does not depend on what else is in the call.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "internal.h"
#include "sm100.cuh"

namespace fpq {

namespace {

constexpr int kGemvThreads = 256;
constexpr int kBlock = 128;               // weights of a row per step
constexpr int kStages = 4;                // steps in a warp's ring
constexpr int kStageBytes = 16 * (kBlock / 2 + kBlock / 16);   // 16 rows: codes, then scales

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
    uint32_t mul_lo, mul_hi;    // 0x1040 and 0x0104 (see decode8)
};

__device__ __forceinline__ void put(void* y, int64_t at, float v, bool f32) {
    if (f32) static_cast<float*>(y)[at] = v;
    else static_cast<uint16_t*>(y)[at] = (uint16_t)f32_to_bf16(v);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
    const int bytes = in ? 16 : 0;                          // 0: the 16 bytes are filled with zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void sts32(uint32_t dst, uint32_t v) {
    asm volatile("st.shared.u32 [%0], %1;" :: "r"(dst), "r"(v) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Eight codes times the scale pair sc (scale 2^117 in both halves): out[i] =
// elements (i, i + 4).  One multiplication copies a nibble to the sign's and
// to the magnitude's place (by 2^12 + 2^6, or 2^8 + 2^2 for the second nibble
// of a byte; kept as kernel arguments so that it stays one multiplication).
__device__ __forceinline__ void decode8(uint32_t w, uint32_t sc, uint32_t mul_lo, uint32_t mul_hi,
                                        uint32_t (&out)[4]) {
    const uint32_t v = w >> 8;
    out[0] = mul_bf16x2(((w & 0x000F000Fu) * mul_lo) & 0x81C081C0u, sc);
    out[1] = mul_bf16x2(((w & 0x00F000F0u) * mul_hi) & 0x81C081C0u, sc);
    out[2] = mul_bf16x2(((v & 0x000F000Fu) * mul_lo) & 0x81C081C0u, sc);
    out[3] = mul_bf16x2(((v & 0x00F000F0u) * mul_hi) & 0x81C081C0u, sc);
}

// Eight consecutive bf16 as the pairs (i, i + 4).
__device__ __forceinline__ uint4 pair8(const uint4& x) {
    return make_uint4(__byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632), __byte_perm(x.y, x.w, 0x5410),
                      __byte_perm(x.y, x.w, 0x7632));
}

// COLS: 8 or 16 columns of the product (rows of x); WK as above.
template <int COLS, int WK>
struct Shape {
    static constexpr int WR = 8 / WK;
    static constexpr int chunk_blocks = WK == 8 ? 8 : 4;             // blocks of 128 per chunk of x
    static constexpr int steps = chunk_blocks / WK;                  // per warp and chunk
    static constexpr int pieces = chunk_blocks * 16;                 // 16-byte pieces per column and chunk
    static constexpr int per_thread = COLS * pieces / kGemvThreads;
    static constexpr int x_bytes = COLS * pieces * 16;               // one chunk
    static constexpr int smem = 2 * x_bytes + 8 * kStages * kStageBytes;
};

template <int COLS, int WK>
__global__ void __launch_bounds__(kGemvThreads, 2)
gemv_nvfp4_kernel(const GemvArgs a) {
    using S = Shape<COLS, WK>;
    extern __shared__ __align__(16) uint8_t smem[];         // two chunks of x, then the warps' rings
    __shared__ float red[8][32][COLS / 2];
    __shared__ int member[COLS], xrow[COLS], info[2];       // info: members, occurrences before this pair
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int wk = warp % WK, wr = warp / WK;
    const int64_t tile0 = (int64_t)blockIdx.x * S::WR;       // the CTA's first 16-row tile
    int64_t e = 0;
    int count;
    if (a.ids) {
        // blockIdx.y is a pair; every COLS-th pair of an expert takes itself
        // and the next COLS - 1, the others have nothing to do
        const int p = blockIdx.y, id = a.ids[p];
        e = id;
        if (id < 0 || id >= a.experts) {
            if (tid == 0) raise_device_error(a.err, FPQ_ERR_DEVICE_BAD_INPUT);
            for (int i = tid; i < 16 * S::WR; i += kGemvThreads)
                if (tile0 * 16 + i < a.n) put(a.y, (int64_t)p * a.n + tile0 * 16 + i, 0.0f, a.y_f32);
            return;
        }
        if (warp == 0) {
            int found = 0;
            for (int q = p; q < a.m && found < COLS; q += 32) {
                const bool same = q + lane < a.m && a.ids[q + lane] == id;
                const uint32_t mask = __ballot_sync(0xFFFFFFFFu, same);
                const int at = found + __popc(mask & ((1u << lane) - 1u));
                if (same && at < COLS) {
                    member[at] = q + lane;
                    xrow[at] = (q + lane) / a.x_div;
                }
                found += __popc(mask);
            }
            if (lane == 0) info[0] = min(found, COLS);
        } else if (warp == 1) {
            int before = 0;
            for (int q = 0; q < p; q += 32)
                before += __popc(__ballot_sync(0xFFFFFFFFu, q + lane < p && a.ids[q + lane] == id));
            if (lane == 0) info[1] = before;
        }
        __syncthreads();
        if (info[1] % COLS) return;
        count = info[0];
    } else {
        count = a.m;
        if (tid < COLS) member[tid] = xrow[tid] = tid;
        __syncthreads();
    }

    const uint32_t ring = sm100::smem_u32(smem) + 2 * S::x_bytes + warp * kStages * kStageBytes;
    const int blocks = (a.k + kBlock - 1) / kBlock, chunks = (blocks + S::chunk_blocks - 1) / S::chunk_blocks;
    const int total = chunks * S::steps;                     // the warp's steps; past the last block: zeros

    // Step i of the warp is block i WK + wk.  Codes: lane (g, t) copies its own
    // 32 of rows g and g + 8.  Scales: lane l loads four of row l / 2 into a
    // register and stores them to the ring at the next call (rows of k / 16
    // bytes are four-byte aligned only for k % 64 == 0, too little for an
    // asynchronous copy).
    const int64_t tile_row = (tile0 + wr) * 16, base = e * a.n + tile_row;
    const bool in0 = tile_row + g < a.n, in1 = tile_row + g + 8 < a.n, ins = tile_row + (lane >> 1) < a.n;
    const uint8_t* q0 = a.wq + (base + (in0 ? g : 0)) * (a.k / 2) + 16 * t;
    const uint8_t* q1 = a.wq + (base + (in1 ? g + 8 : 0)) * (a.k / 2) + 16 * t;
    const uint8_t* sp = a.ws + (base + (ins ? lane >> 1 : 0)) * (a.k / 16) + 4 * (lane & 1);
    const bool whole = a.k % 64 == 0;
    uint32_t scales = 0;
    const auto load = [&](int i) {
        if (i > 0 && i <= total) sts32(ring + ((i - 1) % kStages) * kStageBytes + 1024 + lane * 4, scales);
        if (i < total) {
            const int kb = i * WK + wk;
            const uint32_t st = ring + (i % kStages) * kStageBytes;
            const bool in = kb * kBlock + 32 * t < a.k;
            cp_async16(st + lane * 16, q0 + (in ? kb * (kBlock / 2) : 0), in && in0);
            cp_async16(st + 512 + lane * 16, q1 + (in ? kb * (kBlock / 2) : 0), in && in1);
            const int left = a.k / 16 - kb * 8 - 4 * (lane & 1);          // scales from here to the row's end
            scales = 0;
            if (ins && left > 0) {
                if (whole) {
                    scales = __ldg(reinterpret_cast<const uint32_t*>(sp + kb * 8));
                } else {
                    scales = __ldg(reinterpret_cast<const uint16_t*>(sp + kb * 8));
                    if (left > 2) scales |= (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(sp + kb * 8 + 2)) << 16;
                }
            }
        }
        cp_async_commit();                                   // empty past the end: the counts stay the same
    };
    // x: piece q = 16 block + 4 t + j of a column, at ((4 block + j) COLS + column) 4
    // + t, so that a warp reads word j of all lanes in one row of banks
    uint4 xr[S::per_thread];
    const auto fetch = [&](int c) {
#pragma unroll
        for (int p = 0; p < S::per_thread; ++p) {
            const int i = tid + p * kGemvThreads, col = i / S::pieces, k0 = (c * S::pieces + i % S::pieces) * 8;
            if (col < count && k0 < a.k)
                xr[p] = __ldg(reinterpret_cast<const uint4*>(a.x + (int64_t)xrow[col] * a.k + k0));
            else
                xr[p] = make_uint4(0, 0, 0, 0);
        }
    };
    const auto store = [&](int buf) {
#pragma unroll
        for (int p = 0; p < S::per_thread; ++p) {
            const int i = tid + p * kGemvThreads, col = i / S::pieces, q = i % S::pieces;
            reinterpret_cast<uint4*>(smem + buf * S::x_bytes)[(((q >> 4) * 4 + (q & 3)) * COLS + col) * 4 +
                                                             ((q >> 2) & 3)] = pair8(xr[p]);
        }
    };

    float acc[COLS / 8][2][4] = {};                          // [column tile][alternating][fragment]
    const auto multiply = [&](int i, int u, int buf) {       // step i, the u-th of its chunk
        const uint8_t* st = smem + 2 * S::x_bytes + (warp * kStages + i % kStages) * kStageBytes;
        const uint4* qs = reinterpret_cast<const uint4*>(st);
        const uint4 qa = qs[lane], qb = qs[32 + lane];
        uint32_t sc[2][2];                                   // [row][scale]
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float2 f = e4m3x2_to_f32x2(*reinterpret_cast<const uint16_t*>(st + 1024 + (g + 8 * r) * 8 + 2 * t));
            sc[r][0] = f32x2_to_bf16x2(f.x * 0x1p117f, f.x * 0x1p117f);
            sc[r][1] = f32x2_to_bf16x2(f.y * 0x1p117f, f.y * 0x1p117f);
        }
        const uint4* xb = reinterpret_cast<const uint4*>(smem + buf * S::x_bytes) + (u * WK + wk) * 16 * COLS + lane;
        const uint32_t w0[4] = {qa.x, qa.y, qa.z, qa.w}, w1[4] = {qb.x, qb.y, qb.z, qb.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t d0[4], d1[4];
            decode8(w0[j], sc[0][j >> 1], a.mul_lo, a.mul_hi, d0);
            decode8(w1[j], sc[1][j >> 1], a.mul_lo, a.mul_hi, d1);
#pragma unroll
            for (int h = 0; h < COLS / 8; ++h) {
                const uint4 b = xb[j * COLS * 4 + h * 32];
                mma_bf16(acc[h][0], d0[0], d1[0], d0[1], d1[1], b.x, b.y);
                mma_bf16(acc[h][1], d0[2], d1[2], d0[3], d1[3], b.z, b.w);
            }
        }
    };

#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) load(i);
    fetch(0);
    store(0);
    __syncthreads();
    int i = 0;
    for (int c = 0; c < chunks; ++c) {
        if (c + 1 < chunks) fetch(c + 1);
#pragma unroll
        for (int u = 0; u < S::steps; ++u, ++i) {
            cp_async_wait<kStages - 2>();
            __syncwarp();                                    // the other lanes' scales
            multiply(i, u, c & 1);
            load(i + kStages - 1);
        }
        // the buffer written here was last read before the previous barrier
        if (c + 1 < chunks) store((c + 1) & 1);
        __syncthreads();
    }

    // sums of the WK warps of a row tile, in order
    float part[COLS / 2];
#pragma unroll
    for (int h = 0; h < COLS / 8; ++h)
#pragma unroll
        for (int f = 0; f < 4; ++f) part[4 * h + f] = acc[h][0][f] + acc[h][1][f];
#pragma unroll
    for (int f = 0; f < COLS / 2; ++f) red[warp][lane][f] = part[f];
    __syncthreads();
    const float scale = __ldg(a.wg + e);
    constexpr int rows = 16 * S::WR;
    for (int o = tid; o < rows * count; o += kGemvThreads) {
        const int r = o % rows, col = o / rows;              // consecutive threads: consecutive weight rows
        const int64_t row = tile0 * 16 + r;
        if (row >= a.n) continue;
        // fragment: row g (+ 8 for entries 2, 3), columns 2 t, 2 t + 1 of its tile
        const int from = (r & 7) * 4 + ((col & 7) >> 1), at = (col >> 3) * 4 + ((r >> 3) & 1) * 2 + (col & 1);
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < WK; ++w) v += red[(r >> 4) * WK + w][from][at];
        put(a.y, (int64_t)member[col] * a.n + row, v * 512.0f * scale, a.y_f32);
    }
}

template <int COLS, int WK>
cudaError_t gemv(const GemvArgs& a, cudaStream_t st) {
    using S = Shape<COLS, WK>;
    const auto kernel = gemv_nvfp4_kernel<COLS, WK>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::smem);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (a.n + 15) / 16;
    return launch_pdl(kernel, dim3((unsigned)((tiles + S::WR - 1) / S::WR), (unsigned)(a.ids ? a.m : 1)),
                      dim3(kGemvThreads), S::smem, st, a);
}

}  // namespace

cudaError_t launch_gemv_nvfp4(const void* x, int64_t m, int x_div, const int32_t* ids, int experts, const void* wq,
                              const void* ws, const float* wg, int64_t n, int64_t k, void* y, int y_f32,
                              uint32_t* err, int sms, cudaStream_t st) {
    const GemvArgs a{(const uint16_t*)x, (int)m, x_div, ids, experts, (const uint8_t*)wq, (const uint8_t*)ws, wg, n,
                     (int)k, y, err, y_f32, 0x1040u, 0x0104u};
    // Warps along k where there are few rows: as many row tiles per CTA as
    // leave two CTAs per SM, and two steps per warp at least.
    const int64_t tiles = (n + 15) / 16, blocks = (k + kBlock - 1) / kBlock;
    int wk = 8;
    while (wk > 1 && (tiles / (16 / wk) >= 2 * sms || blocks < 2 * wk)) wk /= 2;
    // Sixteen columns where an expert can be expected to have more than eight pairs.
    const bool wide = ids ? m > 8 && m > 4 * (int64_t)experts : m > 8;
    switch (wk) {
    case 8: return wide ? gemv<16, 8>(a, st) : gemv<8, 8>(a, st);
    case 4: return wide ? gemv<16, 4>(a, st) : gemv<8, 4>(a, st);
    case 2: return wide ? gemv<16, 2>(a, st) : gemv<8, 2>(a, st);
    default: return wide ? gemv<16, 1>(a, st) : gemv<8, 1>(a, st);
    }
}

}  // namespace fpq
