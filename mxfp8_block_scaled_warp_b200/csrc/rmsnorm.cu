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
// Both are bound by HBM.  Rows of at most 1024 elements take one warp each
// (no block barrier), longer rows one CTA each; a thread has V vectors of 8
// elements (16 bytes of bf16).  The forward reads a row into registers,
// reduces it over the threads that hold it and writes from the registers;
// several CTAs per SM hide each other's reduction.  The backward keeps its
// CTAs for the whole call (their columns' sums of dw stay in registers) and
// so has few of them: rows travel through a ring in shared memory, bulk
// copies three to four stages ahead (8192 x 7168: 78 us; with the rows loaded
// into registers 101).
//
// Measured at 8192 x 7168: residual, bf16 and MXFP8 out 81 us (6.53 TB/s, the
// rate of a copy), FP8 without bf16 68.5 us; backward with dres 77.5 us (6.06
// TB/s), 3 to 4 of them the second kernel's; without dres, a quarter less to
// move, 74.3: a row's two passes set the pace.  16384 x 1024 backward 26.4 us
// (5.1 TB/s).  A row of 7168 2.3 us, backward 5.
#include <type_traits>

#include <cuda_runtime.h>

#include "common.cuh"
#include "layer.hpp"
#include "quant_unit.cuh"
#include "sm100.cuh"

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

// Eight bf16 as four pairs of fp32 (paired fp32 instructions do two IEEE
// operations each) and back.
__device__ __forceinline__ void unpack4(const uint4& v, uint64_t (&p)[4]) {
    p[0] = bf16x2_pair(v.x); p[1] = bf16x2_pair(v.y); p[2] = bf16x2_pair(v.z); p[3] = bf16x2_pair(v.w);
}
__device__ __forceinline__ uint4 pack4(const uint64_t (&p)[4]) {
    return make_uint4(f32x2_to_bf16x2(lo_of(p[0]), hi_of(p[0])), f32x2_to_bf16x2(lo_of(p[1]), hi_of(p[1])),
                      f32x2_to_bf16x2(lo_of(p[2]), hi_of(p[2])), f32x2_to_bf16x2(lo_of(p[3]), hi_of(p[3])));
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// The larger magnitude with the product of the signs, NaN if either is NaN.
__device__ __forceinline__ float absmax_f32(float a, float b) {
    float d;
    asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
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

// -fp32(y / s) of a pair, for the codes, from n = fp32(-1 / s): the product
// y n and one correction by its remainder, which the fused multiply-add
// leaves exact (Markstein's division).  Its E4M3 code is the negated code of
// the correctly rounded quotient: for every mantissa of s and the nine values
// of y around each midpoint of codes, 1.2e9 cases, the quotients were compared
// and are equal; away from midpoints the last place decides nothing.  Negated,
// so that a zero keeps its sign.  For 2^-92 <= s < infinity: the remainder is
// exact for |y| >= 2^-103, and a smaller y is below half the smallest code.
// Two more paired instructions per pair than the product alone (8192 x 7168
// with a residual 68.5 us instead of 67.2, without one 47.8 instead of 44.8).
__device__ __forceinline__ bool corrected_quotients_ok(float s) { return s >= 0x1p-92f && s < INFINITY; }
__device__ __forceinline__ uint64_t negated_quotients(uint64_t y, uint64_t s, uint64_t n) {
    const uint64_t q = mul2(y, n);
    return fma2(fma2(q, s, y), n, q);
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

// RES: a residual is given.  Without one a thread has half as many bytes on
// their way, so fewer registers and more CTAs count: 8192 x 7168 to MXFP8 48 us
// with the residual tested for in the kernel, 43 compiled apart, 40 with room
// for a third CTA of 512 threads (rows of 1280 to 3584 0 to 6 % slower).  With
// one, two such CTAs: 8192 x 7168 to FP8 67 us, 74 where the compiler chooses
// (before the codes took the correction of negated_quotients).
template <int FMT, int V, bool WARP, bool RES>
__global__ void __launch_bounds__(WARP ? 32 * kRowWarps : V <= 2 ? 1024 : 512, WARP || V != 4 ? 0 : RES ? 2 : 3)
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
            if (RES) rv[i] = ld_once(a.res + dense + v);
        }
    }
    uint64_t s[V][4], sq2 = 0;                              // pairs
#pragma unroll
    for (int i = 0; i < V; ++i) {
        unpack4(xv[i], s[i]);
        if (RES) {
            uint64_t r[4];
            unpack4(rv[i], r);
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] = add2(s[i][j], r[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) sq2 = fma2(s[i][j], s[i][j], sq2);
        const int v = t + i * T;
        if (a.h && v < a.nvec) st_v4(a.h + dense + v, pack4(s[i]));
    }
    const float sq = row_sum<WARP>(lo_of(sq2) + hi_of(sq2), red);
    const float rstd = __frcp_rn(__fsqrt_rn(__fdiv_rn(sq, a.cols) + a.eps));
    if (a.rstd && t == 0) a.rstd[row] = rstd;
    const uint64_t rstd2 = pack2(rstd, rstd);

#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int v = t + i * T;
        const bool in = v < a.nvec;
        uint64_t w[4];
        unpack4(in ? __ldg(a.w + v) : make_uint4(0, 0, 0, 0), w);
        float most = 0.0f;                                   // largest magnitude, but for its sign; NaN if there is one
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            s[i][j] = mul2(mul2(s[i][j], rstd2), w[j]);
            most = absmax_f32(most, absmax_f32(lo_of(s[i][j]), hi_of(s[i][j])));
        }
        uint32_t top = __float_as_uint(most) & 0x7FFFFFFFu;  // NaN patterns order above infinity
        if (a.y && in) st_v4(a.y + dense + v, pack4(s[i]));
        if (FMT == kNormFp8) {
            top = group_max<16>(in ? top : 0u);             // the 16 lanes of a 128-element tile, in or out together
            // up to 224 steps of the smallest number the quotient rounds to 0
            const float sc = top > 224u ? __fdiv_rn(__uint_as_float(top), 448.0f) : 1.0f;
            uint64_t d[4];
            uint32_t flip = 0;
            if (corrected_quotients_ok(sc)) {
                const float n = -__frcp_rn(sc);
                const uint64_t n2 = pack2(n, n), sc2 = pack2(sc, sc);
#pragma unroll
                for (int j = 0; j < 4; ++j) d[j] = negated_quotients(s[i][j], sc2, n2);
                flip = 0x80808080u;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) d[j] = pack2(__fdiv_rn(lo_of(s[i][j]), sc), __fdiv_rn(hi_of(s[i][j]), sc));
            }
            const uint32_t c[2] = {e4m3x4_of_pairs(d[0], d[1]) ^ flip, e4m3x4_of_pairs(d[2], d[3]) ^ flip};
            if (in) {
                st_v2(a.q + dense + v, make_uint2(c[0], c[1]));
                if ((v & 15) == 0) static_cast<float*>(a.scales)[(dense + v) >> 4] = sc;
            }
        } else if (FMT == kNormMx) {
            top = group_max<4>(in ? top : 0u);
            const int e = mx_exponent_f32(top);
            const float mul = pow2_neg(e == 128 ? 127 : e);
            const uint64_t mul_2 = pack2(mul, mul);
            uint2 q = make_uint2(e4m3x4_of_pairs(mul2(s[i][0], mul_2), mul2(s[i][1], mul_2)),
                                 e4m3x4_of_pairs(mul2(s[i][2], mul_2), mul2(s[i][3], mul_2)));
            if (e == 128) q = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
            if (in) {
                st_v2(a.q + dense + v, q);
                if ((v & 3) == 0) static_cast<uint8_t*>(a.scales)[(dense + v) >> 2] = (uint8_t)(e + 127);
            }
        }
    }
}

template <int FMT, bool RES>
cudaError_t launch_norm(const NormArgs& a, int sms, cudaStream_t st) {
    const int nv = a.nvec;
    if (nv <= 128) {
        const dim3 grid((unsigned)((a.rows + kRowWarps - 1) / kRowWarps)), block(32 * kRowWarps);
        if (nv <= 32) return launch_pdl(rmsnorm_quant_kernel<FMT, 1, true, RES>, grid, block, 0, st, a);
        if (nv <= 64) return launch_pdl(rmsnorm_quant_kernel<FMT, 2, true, RES>, grid, block, 0, st, a);
        return launch_pdl(rmsnorm_quant_kernel<FMT, 4, true, RES>, grid, block, 0, st, a);
    }
    // Few rows: latency counts, so a row is spread over as many threads as
    // it has vectors.  Many rows: V = 4 keeps four loads per operand in
    // flight per thread and the barrier among fewer warps.
    const dim3 grid((unsigned)a.rows);
    const auto threads = [&](int v) { return dim3((unsigned)(((nv + v - 1) / v + 31) / 32 * 32)); };
    const bool few = a.rows < 2 * sms;
    if (few && nv <= 1024) return launch_pdl(rmsnorm_quant_kernel<FMT, 1, false, RES>, grid, threads(1), 0, st, a);
    if (few && nv <= 2048) return launch_pdl(rmsnorm_quant_kernel<FMT, 2, false, RES>, grid, threads(2), 0, st, a);
    if (nv <= 2048) return launch_pdl(rmsnorm_quant_kernel<FMT, 4, false, RES>, grid, threads(4), 0, st, a);
    return launch_pdl(rmsnorm_quant_kernel<FMT, 8, false, RES>, grid, threads(8), 0, st, a);
}

// ------------------------------------------------------------------ backward

struct NormBwdArgs {
    const uint8_t* dy;
    const uint8_t* x;      // row r at x + r ld
    int64_t ld;            // in bytes
    const uint4* w;
    const float* rstd;
    const uint8_t* dres;   // or nullptr
    int64_t rows;
    int nvec;
    float cols;
    uint4* dx;
    float* partial;        // [grid, cols] sums of dw over a CTA's rows, or nullptr
    int stages, batch;     // stages of a ring; rows per stage (1 for a CTA)
    uint32_t* err;
};

constexpr int kBwdMaxWarps = 16;          // rows (warps) per CTA in the warp-per-row form
constexpr int kBwdMaxStages = 4;
constexpr int kBwdSmem = 216 * 1024;        // rings of the CTAs of an SM

// A team (the CTA, or a warp) takes batches of consecutive rows, every
// grid-th; a thread's columns are the same for every row.
template <int V, bool WARP>
__global__ void __launch_bounds__(512, 1)
rmsnorm_bwd_kernel(const NormBwdArgs a) {
    extern __shared__ __align__(128) uint8_t smem[];         // w, then the rings: stages of dy, x, dres rows
    __shared__ uint64_t bars[WARP ? kBwdMaxWarps : 1][kBwdMaxStages];
    __shared__ __align__(16) float red[2][32];
    const int t = WARP ? (threadIdx.x & 31) : threadIdx.x, T = WARP ? 32 : blockDim.x;
    const int team = WARP ? threadIdx.x >> 5 : 0, cta_teams = WARP ? blockDim.x >> 5 : 1;
    const uint32_t row_bytes = (uint32_t)a.nvec * 16, part = row_bytes * a.batch;
    uint4* const wsm = reinterpret_cast<uint4*>(smem);
    uint8_t* const ring = smem + (row_bytes + 127) / 128 * 128 + team * a.stages * 3 * part;
    uint64_t* const bar = bars[team];
    if (!WARP && t < 32) red[0][t] = red[1][t] = 0.0f;       // slots past the last warp stay 0
    if (t == 0) {
        for (int i = 0; i < a.stages; ++i) sm100::mbar_init(&bar[i], 1);
        sm100::fence_barrier_init();
    }
    pdl_wait();
    for (int v = threadIdx.x; v < a.nvec; v += blockDim.x) wsm[v] = __ldg(a.w + v);
    __syncthreads();

    const int64_t teams = (int64_t)gridDim.x * cta_teams, first = (int64_t)blockIdx.x * cta_teams + team;
    const int64_t batches = (a.rows + a.batch - 1) / a.batch;
    const auto fill = [&](int64_t b, int stage) {            // one thread of the team
        if (b >= batches) return;
        const int64_t row = b * a.batch;
        const uint32_t n = (uint32_t)min64(a.batch, a.rows - row), bytes = n * row_bytes;
        uint8_t* dst = ring + stage * 3 * part;
        sm100::mbar_arrive_expect_tx(&bar[stage], bytes * (a.dres ? 3 : 2));
        bulk_load(dst, a.dy + row * row_bytes, bytes, &bar[stage]);
        if (a.ld == row_bytes) {
            bulk_load(dst + part, a.x + row * row_bytes, bytes, &bar[stage]);
        } else {
            for (uint32_t i = 0; i < n; ++i)
                bulk_load(dst + part + i * row_bytes, a.x + (row + i) * a.ld, row_bytes, &bar[stage]);
        }
        if (a.dres) bulk_load(dst + 2 * part, a.dres + row * row_bytes, bytes, &bar[stage]);
    };
    if (t == 0)
        for (int i = 0; i < a.stages; ++i) fill(first + i * teams, i);

    // KEEP: the row stays in registers between the two passes, so that its
    // stage is refilled between them; rows too long for that are read twice
    constexpr bool KEEP = V <= 2;
    // WREG: the weights stay there too (8192 x 7168 80.6 -> 78.2 us)
    constexpr bool WREG = KEEP && !WARP;
    uint64_t wr[WREG ? V : 1][4];
    if (WREG)
#pragma unroll
        for (int i = 0; i < V; ++i) unpack4(t + i * T < a.nvec ? wsm[t + i * T] : make_uint4(0, 0, 0, 0), wr[WREG ? i : 0]);
    uint64_t acc[V][4];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0;
    int turn = 0, stage = 0;
    uint32_t phase = 0;
    float next_rstd = first < batches ? __ldg(a.rstd + first * a.batch) : 0.0f;
    for (int64_t b = first; b < batches; b += teams) {
        if (!mbar_wait_seconds(&bar[stage], phase)) {     // after this long no copy is in flight
            raise_device_error(a.err, FPQ_ERR_DEVICE_TIMEOUT);
            return;
        }
        const int64_t row0 = b * a.batch;
        const int n = (int)min64(a.batch, a.rows - row0);
        for (int r = 0; r < n; ++r, turn ^= 1) {
            const uint8_t* at = ring + stage * 3 * part + r * row_bytes;
            const uint4* dv = reinterpret_cast<const uint4*>(at);
            const uint4* xv = reinterpret_cast<const uint4*>(at + part);
            const uint4* ev = reinterpret_cast<const uint4*>(at + 2 * part);
            const float rstd = next_rstd;                    // loaded a row ahead
            if (r + 1 < n) next_rstd = __ldg(a.rstd + row0 + r + 1);
            else if (b + teams < batches) next_rstd = __ldg(a.rstd + (b + teams) * a.batch);
            const uint64_t rstd2 = pack2(rstd, rstd);
            uint64_t gw[KEEP ? V : 1][4], x[KEEP ? V : 1][4], dot2 = 0;   // dy w and x
            uint4 e[KEEP ? V : 1];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int v = t + i * T, k = KEEP ? i : 0;
                if (KEEP) e[k] = make_uint4(0, 0, 0, 0);
                if (v >= a.nvec) continue;
                uint64_t d[4], w[4];
                unpack4(dv[v], d);
                unpack4(xv[v], x[k]);
                if (WREG) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[j] = wr[WREG ? i : 0][j];
                } else {
                    unpack4(wsm[v], w);
                }
                if (KEEP && a.dres) e[k] = ev[v];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    gw[k][j] = mul2(d[j], w[j]);
                    dot2 = fma2(gw[k][j], x[k][j], dot2);
                    acc[i][j] = fma2(d[j], mul2(x[k][j], rstd2), acc[i][j]);
                }
            }
            float dot = warp_sum(lo_of(dot2) + hi_of(dot2));
            if (!WARP) {
                // every thread adds the warps' sums itself: one latency, where a
                // second round of shuffles has five (8192 x 7168: 0.4 us)
                if ((t & 31) == 0) red[turn][t >> 5] = dot;
                __syncthreads();
                const float4* r = reinterpret_cast<const float4*>(red[turn]);
                const float4 s0 = r[0], s1 = r[1], s2 = r[2], s3 = r[3];
                dot = (((s0.x + s0.y) + (s0.z + s0.w)) + ((s1.x + s1.y) + (s1.z + s1.w))) +
                      (((s2.x + s2.y) + (s2.z + s2.w)) + ((s3.x + s3.y) + (s3.z + s3.w)));
            }
            if (!WARP && t == 0) {
                // every thread of the CTA is past its reads of this row (KEEP)
                // or has left the previous one
                if (KEEP) fill(b + a.stages * teams, stage);
                else if (b != first) fill(b + (a.stages - 1) * teams, stage == 0 ? a.stages - 1 : stage - 1);
            }
            const float c = -__fdiv_rn(dot * rstd, a.cols) * rstd * rstd;
            const uint64_t c2 = pack2(c, c);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int v = t + i * T, k = KEEP ? i : 0;
                if (v >= a.nvec) continue;
                if (!KEEP) {
                    uint64_t d[4], w[4];
                    unpack4(dv[v], d);
                    unpack4(xv[v], x[k]);
                    unpack4(wsm[v], w);
#pragma unroll
                    for (int j = 0; j < 4; ++j) gw[k][j] = mul2(d[j], w[j]);
                    e[k] = a.dres ? ev[v] : make_uint4(0, 0, 0, 0);
                }
                uint64_t out[4];
                unpack4(e[k], out);
#pragma unroll
                for (int j = 0; j < 4; ++j) out[j] = fma2(x[k][j], c2, fma2(gw[k][j], rstd2, out[j]));
                st_v4(a.dx + (row0 + r) * a.nvec + v, pack4(out));
            }
        }
        if (WARP) {
            __syncwarp();
            if (t == 0) fill(b + a.stages * teams, stage);
        }
        if (++stage == a.stages) { stage = 0; phase ^= 1; }
    }
    // Only now: CTAs of the next kernel on this one's SMs, and of the next
    // call's beside those, would keep some of a wave's CTAs waiting for a
    // whole wave (16384 x 2048, call after call: 68 us instead of 47).  For
    // the same reason the kernel that adds the sums triggers by its end.
    pdl_trigger();
    if (!a.partial) return;
    float4* out = reinterpret_cast<float4*>(a.partial) + (int64_t)blockIdx.x * a.nvec * 2;
    if (WARP) {
        // the warps' sums side by side in the rings' place (a ring has at least
        // 96 bytes per vector, they take 32), then added in the warps' order
        float4* const sums = reinterpret_cast<float4*>(smem);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = t + i * T;
            if (v < a.nvec) {
                float4* p = sums + (team * a.nvec + v) * 2;
                p[0] = make_float4(lo_of(acc[i][0]), hi_of(acc[i][0]), lo_of(acc[i][1]), hi_of(acc[i][1]));
                p[1] = make_float4(lo_of(acc[i][2]), hi_of(acc[i][2]), lo_of(acc[i][3]), hi_of(acc[i][3]));
            }
        }
        __syncthreads();
        for (int v = threadIdx.x; v < 2 * a.nvec; v += blockDim.x) {
            float4 s = sums[v];
#pragma unroll 4
            for (int wi = 1; wi < cta_teams; ++wi) {
                const float4 u = sums[wi * 2 * a.nvec + v];
                s.x += u.x; s.y += u.y; s.z += u.z; s.w += u.w;
            }
            out[v] = s;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = t + i * T;
            if (v < a.nvec) {
                out[2 * v] = make_float4(lo_of(acc[i][0]), hi_of(acc[i][0]), lo_of(acc[i][1]), hi_of(acc[i][1]));
                out[2 * v + 1] = make_float4(lo_of(acc[i][2]), hi_of(acc[i][2]), lo_of(acc[i][3]), hi_of(acc[i][3]));
            }
        }
    }
}

// Rows of which no two fit in shared memory (more than 15360 elements): read
// from global memory, four vectors at a time; with V = 8 a second time, from
// L2, as the registers hold the sums of dw.
template <int V>
__global__ void __launch_bounds__(512)
rmsnorm_bwd_long_kernel(const NormBwdArgs a) {
    __shared__ float red[2][32];
    pdl_wait();
    const int t = threadIdx.x, T = blockDim.x;
    uint64_t acc[V][4];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        const uint4* dv = reinterpret_cast<const uint4*>(a.dy) + row * a.nvec;
        const uint4* xv = reinterpret_cast<const uint4*>(a.x + row * a.ld);
        const float rstd = __ldg(a.rstd + row);
        const uint64_t rstd2 = pack2(rstd, rstd);
        uint4 d[4], x[4];
        const auto load = [&](int i0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int v = t + (i0 + i) * T;
                d[i] = x[i] = make_uint4(0, 0, 0, 0);
                if (v < a.nvec) {
                    d[i] = ld_once(dv + v);
                    x[i] = ld_once(xv + v);
                }
            }
        };
        uint64_t dot2 = 0;
#pragma unroll
        for (int i0 = 0; i0 < V; i0 += 4) {
            load(i0);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int v = t + (i0 + i) * T;
                uint64_t dp[4], xp[4], w[4];
                unpack4(d[i], dp);
                unpack4(x[i], xp);
                unpack4(v < a.nvec ? __ldg(a.w + v) : make_uint4(0, 0, 0, 0), w);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    dot2 = fma2(mul2(dp[j], w[j]), xp[j], dot2);
                    acc[i0 + i][j] = fma2(dp[j], mul2(xp[j], rstd2), acc[i0 + i][j]);
                }
            }
        }
        const float dot = row_sum<false>(lo_of(dot2) + hi_of(dot2), red[turn]);
        const float c = -__fdiv_rn(dot * rstd, a.cols) * rstd * rstd;
        const uint64_t c2 = pack2(c, c);
#pragma unroll
        for (int i0 = 0; i0 < V; i0 += 4) {
            if (V > 4) load(i0);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int v = t + (i0 + i) * T;
                if (v >= a.nvec) continue;
                uint64_t dp[4], xp[4], w[4], out[4];
                unpack4(d[i], dp);
                unpack4(x[i], xp);
                unpack4(__ldg(a.w + v), w);
                unpack4(a.dres ? ld_once(reinterpret_cast<const uint4*>(a.dres) + row * a.nvec + v) : make_uint4(0, 0, 0, 0), out);
#pragma unroll
                for (int j = 0; j < 4; ++j) out[j] = fma2(xp[j], c2, fma2(mul2(dp[j], w[j]), rstd2, out[j]));
                st_v4(a.dx + row * a.nvec + v, pack4(out));
            }
        }
    }
    pdl_trigger();
    if (!a.partial) return;
    float4* out = reinterpret_cast<float4*>(a.partial) + (int64_t)blockIdx.x * a.nvec * 2;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int v = t + i * T;
        if (v < a.nvec) {
            out[2 * v] = make_float4(lo_of(acc[i][0]), hi_of(acc[i][0]), lo_of(acc[i][1]), hi_of(acc[i][1]));
            out[2 * v + 1] = make_float4(lo_of(acc[i][2]), hi_of(acc[i][2]), lo_of(acc[i][3]), hi_of(acc[i][3]));
        }
    }
}

// dweight[c] = sum of the partial rows, in a fixed order: a CTA takes 16
// columns; thread (i, j) adds rows i, i + 128, ... of its four, all loads in
// flight at once (there are at most four rows per SM), then the threads of a
// column are added, in a warp and across the warps.  Latency alone, about 3
// us of the call (4 us with 32 rows of threads).
constexpr int kSumRows = 128, kSumVecs = 4, kSumWarps = kSumRows * kSumVecs / 32;

__device__ __forceinline__ float4 sum_rows(float4 s) {       // over the lanes of a vector
#pragma unroll
    for (int o = kSumVecs; o < 32; o <<= 1) {
        s.x += __shfl_xor_sync(0xFFFFFFFFu, s.x, o);
        s.y += __shfl_xor_sync(0xFFFFFFFFu, s.y, o);
        s.z += __shfl_xor_sync(0xFFFFFFFFu, s.z, o);
        s.w += __shfl_xor_sync(0xFFFFFFFFu, s.w, o);
    }
    return s;
}

__global__ void __launch_bounds__(kSumRows * kSumVecs)
rmsnorm_dweight_kernel(const float4* __restrict__ partial, int parts, int nvec4, float4* __restrict__ dweight) {
    __shared__ float4 sum[kSumWarps][kSumVecs];
    pdl_wait();
    const int i = threadIdx.x / kSumVecs, j = threadIdx.x % kSumVecs, v = blockIdx.x * kSumVecs + j;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (v < nvec4) {
#pragma unroll 8
        for (int p = i; p < parts; p += kSumRows) {
            const float4 u = partial[(int64_t)p * nvec4 + v];
            s.x += u.x; s.y += u.y; s.z += u.z; s.w += u.w;
        }
    }
    s = sum_rows(s);
    if (lane < kSumVecs) sum[warp][lane] = s;
    __syncthreads();
    if (warp == 0) {
        // lane (w, j) adds warps w and w + 8
        static_assert(kSumWarps == 16 && kSumVecs == 4, "two warps' sums per lane");
        const float4 c = sum[lane >> 2][j], d = sum[(lane >> 2) + 8][j];
        s = sum_rows(make_float4(c.x + d.x, c.y + d.y, c.z + d.z, c.w + d.w));
        if (lane < kSumVecs && v < nvec4) dweight[v] = s;
    }
}

// How the backward of rows of nvec vectors is launched.
struct BwdPlan {
    int v, threads, ctas;      // vectors per thread, threads per CTA, CTAs per SM
    int batch, stages, smem;   // rows per stage (warps), stages and bytes of shared memory per CTA
};

// Longest row of the ring: w and two stages of three rows fit in kBwdSmem.
constexpr int kRingVectors = kBwdSmem / 16 / 7 / 128 * 128;
static_assert(kRingVectors * 16 + 2 * 3 * kRingVectors * 16 <= kBwdSmem, "a ring has two stages");

BwdPlan bwd_plan(int64_t rows, int nvec, int sms) {
    BwdPlan p{};
    const bool warp = nvec <= 128;
    p.v = warp ? (nvec <= 32 ? 1 : nvec <= 64 ? 2 : 4) : nvec <= 1024 ? 2 : nvec <= 2048 ? 4 : 8;
    // Short rows are copied several at a time, up to 2 KB per operand, unless
    // that leaves warps without any (505 x 144: 5.9 us with seven rows per
    // copy).
    p.batch = warp ? (int)max64(1, min64(128 / nvec, rows / (8 * (int64_t)sms))) : 1;
    // Sixteen warps hide each other's latency where there are rows for them
    // (16384 x 1024 27.6 us, eight warps 30.3); few rows are spread over more
    // CTAs (300 x 1024 5.2 us, sixteen warps 6.0).
    const int warps = (rows + p.batch - 1) / p.batch > 8 * (int64_t)sms ? kBwdMaxWarps : kBwdMaxWarps / 2;
    p.threads = warp ? 32 * warps : ((nvec + p.v - 1) / p.v + 31) / 32 * 32;
    // About 512 threads per SM: with 8192 x 7168 (448 threads) one CTA of four
    // stages takes 78 us and two of two stages 85, with 16384 x 2048 (128
    // threads) four CTAs 46 us, seven of two stages 50.
    p.ctas = warp ? 1 : 512 / p.threads > 4 ? 4 : 512 / p.threads;
    if (nvec > kRingVectors) return p;
    const int row = nvec * 16, stage = 3 * row * p.batch * (warp ? warps : 1), w = (row + 127) / 128 * 128;
    p.stages = (kBwdSmem / p.ctas - w) / stage;
    if (p.stages > kBwdMaxStages) p.stages = kBwdMaxStages;
    p.smem = w + p.stages * stage;
    return p;
}

int bwd_grid(int64_t rows, const BwdPlan& p, int nvec, int sms) {
    const int warps = p.threads / 32;
    const int64_t tasks = nvec <= 128 ? ((rows + p.batch - 1) / p.batch + warps - 1) / warps : rows;
    return (int)min64(tasks, (int64_t)sms * p.ctas);
}

template <int V, bool WARP>
cudaError_t launch_bwd(const NormBwdArgs& a, const BwdPlan& p, int grid, cudaStream_t st) {
    constexpr auto kernel = rmsnorm_bwd_kernel<V, WARP>;
    const cudaError_t e = allow_shared_memory<kernel, kBwdSmem>();
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3((unsigned)grid), dim3((unsigned)p.threads), p.smem, st, a);
}

}  // namespace

cudaError_t launch_rmsnorm_quantize(int fmt, const void* x, int64_t ld_x, const void* residual, const void* weight,
                                    int64_t rows, int64_t cols, float eps, void* h, void* y, void* q, void* scales,
                                    float* rstd, int sms, cudaStream_t st) {
    const NormArgs a{(const uint4*)x, ld_x / 8, (const uint4*)residual, (const uint4*)weight, rows, (int)(cols / 8),
                     (float)cols, eps, (uint4*)h, (uint4*)y, (uint2*)q, scales, rstd};
    const auto launch = [&](auto res) {
        constexpr bool RES = decltype(res)::value;
        if (!q) return launch_norm<kNormNone, RES>(a, sms, st);
        return fmt == FPQ_FP8_1x128 ? launch_norm<kNormFp8, RES>(a, sms, st) : launch_norm<kNormMx, RES>(a, sms, st);
    };
    return residual ? launch(std::true_type()) : launch(std::false_type());
}

size_t rmsnorm_backward_workspace_bytes(int64_t rows, int64_t cols, int sms) {
    const int nvec = (int)(cols / 8);
    return (size_t)bwd_grid(rows, bwd_plan(rows, nvec, sms), nvec, sms) * (size_t)cols * sizeof(float);
}

cudaError_t launch_rmsnorm_backward(const void* dy, const void* x, int64_t ld_x, const void* weight,
                                    const float* rstd, const void* dres, int64_t rows, int64_t cols, void* dx,
                                    float* dweight, void* workspace, uint32_t* err, int sms, cudaStream_t st) {
    const int nvec = (int)(cols / 8);
    const BwdPlan p = bwd_plan(rows, nvec, sms);
    const int grid = bwd_grid(rows, p, nvec, sms);
    const NormBwdArgs a{(const uint8_t*)dy, (const uint8_t*)x, ld_x * 2, (const uint4*)weight, rstd,
                        (const uint8_t*)dres, rows, nvec, (float)cols, (uint4*)dx,
                        dweight ? (float*)workspace : nullptr, p.stages, p.batch, err};
    cudaError_t e = cudaSuccess;
    if (grid > 0) {
        const dim3 g((unsigned)grid), b((unsigned)p.threads);
        if (nvec <= 32) e = launch_bwd<1, true>(a, p, grid, st);
        else if (nvec <= 64) e = launch_bwd<2, true>(a, p, grid, st);
        else if (nvec <= 128) e = launch_bwd<4, true>(a, p, grid, st);
        else if (nvec <= 1024) e = launch_bwd<2, false>(a, p, grid, st);
        else if (nvec <= kRingVectors) e = launch_bwd<4, false>(a, p, grid, st);
        else if (nvec <= 2048) e = launch_pdl(rmsnorm_bwd_long_kernel<4>, g, b, 0, st, a);
        else e = launch_pdl(rmsnorm_bwd_long_kernel<8>, g, b, 0, st, a);
    }
    if (e != cudaSuccess || !dweight) return e;
    return launch_pdl(rmsnorm_dweight_kernel, dim3((unsigned)((2 * nvec + kSumVecs - 1) / kSumVecs)),
                      dim3(kSumRows * kSumVecs), 0, st,
                      (const float4*)workspace, grid, 2 * nvec, (float4*)dweight);
}

}  // namespace fpq
