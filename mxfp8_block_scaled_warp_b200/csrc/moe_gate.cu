// moe_gate.cu -- the expert gate of a mixture-of-experts layer and its
// backward pass: scores of the gate's logits, an optional balance bias,
// optional group-limited choice, top-k, and the routing weights.
//
//   score p_e = softmax(l)_e or 1 / (1 + exp(-l_e))
//   key     k_e = l_e without a bias (both scores grow with the logit) and
//               where l_e is -inf, p_e + b_e with one
//   groups: E / n_group consecutive experts each; a group's rank is the sum
//           of its `group_top` largest p_e + b_e (p_e without a bias);
//           experts outside the topk_group best groups are not chosen
//   ids     the topk largest keys, in order; equal keys by lowest index
//   weights scale p_e, divided by the sum of the chosen p with `renormalize`
//
// Which expert is chosen must not depend on rounding.  Without a bias the
// keys are the inputs themselves.  With one, and for the groups, a choice is
// made on fp32 keys whose error is below half of `slack`: if only one
// candidate lies within `slack` of the largest key, it is the largest in
// exact arithmetic too; otherwise (under one row in a hundred for spread
// logits, and every exact tie) the candidates' keys are recomputed in fp64.
//
// A logit of -inf has score 0.  A NaN key orders below every number.  A row
// whose chosen scores sum to 0 gets zero weights.
//
// One warp per token, expert e = 32 i + lane in register i: the row is read
// once, coalesced.  The traffic (a logit read per expert) is a few
// microseconds at most; what bounds the kernel is its instructions, about
// 200 per token and 64 experts.  So the topk largest are not taken one after
// the other: the topk-th largest of the 32 lane maxima bounds them from
// below, the few keys at or above it (ten for eight of 256) are gathered, one
// per lane, and each counts how many are before it, which is its place in
// the output.  The bound itself and the choice of groups are counted too, not
// taken one maximum after the other: for a few tokens the kernel is the
// latency of one warp's steps (16 tokens of 256 experts in groups 3.8 us
// instead of 5.4).  One maximum after the other remains for rows with more
// than 32 such keys, which take equal logits, and for groups too near to
// tell; throughout it took 51 us for 16384 tokens.  Measured for eight of 256,
// 16384 tokens, fp32: 13.0 us without a bias (1.4 TB/s), sigmoid with one
// 18.4, in eight groups 27.4 (at 78% of the issue slots), softmax with a bias
// 26.4.
#include <type_traits>

#include <cuda_runtime.h>

#include "common.cuh"
#include "layer.hpp"

namespace fpq {

namespace {

constexpr int kGateWarps = 4;
constexpr uint32_t kFull = 0xFFFFFFFFu;

// Order-preserving patterns: larger key, larger pattern.  Below every number
// (-inf is kMasked): NaN 2, outside the chosen groups 1, taken or past
// the last expert 0.
constexpr uint32_t kTaken = 0, kOutside = 1, kNaN = 2, kMasked = 0x007FFFFF;

__device__ __forceinline__ uint32_t pattern(float f) {
    if (f != f) return kNaN;
    const uint32_t b = __float_as_uint(f + 0.0f);           // -0 to +0
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value(uint32_t p) {
    if (p <= kNaN) return -INFINITY;
    return __uint_as_float((p & 0x80000000u) ? p ^ 0x80000000u : ~p);
}

template <typename T> __device__ __forceinline__ float load_logit(const T* p);
template <> __device__ __forceinline__ float load_logit<float>(const float* p) { return __ldg(p); }
template <> __device__ __forceinline__ float load_logit<uint16_t>(const uint16_t* p) {
    return __uint_as_float((uint32_t)__ldg(p) << 16);
}

__device__ __forceinline__ float sigmoid(float x) { return __fdiv_rn(1.0f, 1.0f + expf(-x)); }
// For keys: within 2^-21 (the fast exponential's error grows with its
// argument, which the sigmoid's slope outweighs).
__device__ __forceinline__ float sigmoid_key(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

struct GateArgs {
    const void* logits;
    const float* bias;          // or nullptr
    int64_t tokens;
    int experts, topk, n_group, topk_group, group_top;
    int renormalize;
    float scale;
    int32_t* ids;
    float* weights;
};

// The fp64 score of a logit, for the rows that need it: mx and sum are the
// row's softmax maximum and sum.
template <bool SIGMOID>
__device__ __noinline__ double score64(float l, float mx, double sum) {
    if (SIGMOID) return 1.0 / (1.0 + exp(-(double)l));
    return mx == -INFINITY ? 0.0 : exp((double)l - (double)mx) / sum;
}

// Best of the warp's candidates (lanes with has) in fp64, the lowest index
// among equals; a NaN orders below every number.
__device__ __forceinline__ int best64(double key, int index, bool has) {
    if (!(key == key)) key = -INFINITY;
    if (!has) index = 0x7FFFFFFF;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const double k = __shfl_xor_sync(kFull, key, o);
        const int e = __shfl_xor_sync(kFull, index, o);
        if (e != 0x7FFFFFFF && (index == 0x7FFFFFFF || k > key || (k == key && e < index))) { key = k; index = e; }
    }
    return index;
}

template <typename T, bool SIGMOID, int VPT>
__global__ void __launch_bounds__(32 * kGateWarps)
moe_gate_kernel(const GateArgs a) {
    extern __shared__ float sh[];                           // per warp: keys of the row, padded per 32 (groups only)
    __shared__ uint2 gathered[kGateWarps][32];               // key pattern, expert
    __shared__ uint4 tops[kGateWarps][8];                    // the lanes' largest keys
    pdl_trigger();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = a.experts;
    const int64_t tok = (int64_t)blockIdx.x * kGateWarps + warp;
    if (tok >= a.tokens) return;
    const T* row = static_cast<const T*>(a.logits) + tok * E;

    float l[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) l[i] = 32 * i + lane < E ? load_logit<T>(row + 32 * i + lane) : -INFINITY;
    float b[VPT];                                            // loaded with the logits: one latency
#pragma unroll
    for (int i = 0; i < VPT; ++i) b[i] = a.bias && 32 * i + lane < E ? __ldg(a.bias + 32 * i + lane) : 0.0f;

    // softmax maximum and sum, where the scores themselves are needed (the
    // weights take the sum only without renormalize)
    const bool scores = a.bias || a.n_group > 1;
    float mx = -INFINITY, sum = 0.0f;
    if (!SIGMOID && (scores || !a.renormalize)) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) mx = fmaxf(mx, l[i]);
        mx = warp_max(mx);
        if (mx != -INFINITY) {
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                sum += 32 * i + lane < E ? (a.renormalize ? __expf(l[i] - mx) : expf(l[i] - mx)) : 0.0f;
            sum = warp_sum(sum);
        }
    }
    const auto score_key = [&](float x) {
        if (SIGMOID) return sigmoid_key(x);
        if (mx == -INFINITY) return x == x ? 0.0f : x;
        return __fdividef(__expf(x - mx), sum);
    };
    // At least twice the error of an fp32 key: a sigmoid is within 2^-20; a
    // softmax within 2^-18 of the row's largest (1 / sum), as its sum of up to
    // 1024 terms goes through at most 37 additions in a row; adding the bias
    // costs half a step.
    const float error = SIGMOID ? 0x1p-20f : sum > 0.0f ? __fdividef(0x1p-18f, sum) : 0.0f;
    const auto slack = [&](float key) {
        return fabsf(key) < INFINITY ? 2.0f * (error + 0x1p-23f * fabsf(key)) : 0.0f;
    };
    double sum64 = 0.0;
    const auto need64 = [&]() {                             // warp-uniform
        if (!SIGMOID && sum64 == 0.0 && mx != -INFINITY) {
#pragma unroll 1
            for (int e = lane; e < E; e += 32) sum64 += exp((double)load_logit<T>(row + e) - (double)mx);
            sum64 = warp_sum(sum64);
        }
    };
    const auto key64 = [&](int e) {                         // of p + b, or p
        const double p = score64<SIGMOID>(load_logit<T>(row + e), mx, sum64);
        return a.bias ? p + (double)__ldg(a.bias + e) : p;
    };

    float* const s = sh + warp * (E + E / 32 + 1);          // entry e at e + e / 32: a group's scan is free of conflicts
    uint32_t key[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int e = 32 * i + lane;
        float k = l[i];
        if (scores && e < E) {
            float r = score_key(l[i]);
            if (a.bias) r += b[i];
            if (a.bias && l[i] != -INFINITY) k = r;          // a masked expert gains nothing by its bias
            if (a.n_group > 1) s[e + i] = r == r ? r : -INFINITY;
        }
        key[i] = e >= E ? kTaken : pattern(k);
    }

    if (a.n_group > 1) {
        __syncwarp();
        // `split` adjacent lanes share a group; lane `split` g holds its rank:
        // its largest key, or the sum of its two largest
        const int size = E / a.n_group, shift = __clz(a.n_group - 1) - 27, split = 1 << shift, g = lane >> shift;
        float first = -INFINITY, second = -INFINITY;
        if (g < a.n_group)
#pragma unroll 4
            for (int e = g * size + (lane & (split - 1)); e < (g + 1) * size; e += split) {
                const float v = s[e + (e >> 5)];
                second = fmaxf(second, fminf(first, v));
                first = fmaxf(first, v);
            }
        for (int o = 1; o < split; o <<= 1) {
            const float f = __shfl_xor_sync(kFull, first, o), n = __shfl_xor_sync(kFull, second, o);
            second = fmaxf(fmaxf(second, n), fminf(first, f));
            first = fmaxf(first, f);
        }
        const float rank = a.group_top == 2 ? first + second : first;
        const bool holds = g < a.n_group && (lane & (split - 1)) == 0;
        uint32_t gkey = holds ? pattern(rank) : kTaken;
        // twice the rank's error: each key has its own, by its own magnitude,
        // which the sum may fall far below; the addition's step is within them
        const float own = value(gkey);
        const float reach = fabsf(own) < INFINITY ? slack(first) + (a.group_top == 2 ? slack(second) : 0.0f) : 0.0f;
        // each group counts the ranks above its own; only where two are too
        // near to tell are the best taken one after the other
        int above = 0;
        bool close = false;
#pragma unroll 4
        for (int j = 0; j < a.n_group; ++j) {
            const int holder = j << shift;
            const uint32_t k = __shfl_sync(kFull, gkey, holder);
            above += k > gkey || (k == gkey && holder < lane);
            close |= holder != lane && k > kNaN && gkey > kNaN && (k == gkey || fabsf(value(k) - own) <= reach);
        }
        const bool apart = !__any_sync(kFull, holds && close);
        uint32_t open = __ballot_sync(kFull, holds && above < a.topk_group);   // lanes of the chosen groups
        if (!apart) open = 0;
        for (int c = apart ? a.topk_group : 0; c < a.topk_group; ++c) {
            const uint32_t m = __reduce_max_sync(kFull, gkey);
            const float most_reach = __uint_as_float(__reduce_max_sync(kFull, gkey == m ? __float_as_uint(reach) : 0u));
            const bool near = gkey != kTaken && (gkey == m || (gkey > kNaN && value(m) - own <= fmaxf(reach, most_reach)));
            const uint32_t cand = __ballot_sync(kFull, near);
            int best = __ffs(cand) - 1;
            if (cand & (cand - 1)) {
                // the near groups' ranks in fp64, one after the other, over the warp
                need64();
                double most = 0.0;
                best = -1;
                for (uint32_t left = cand; left; left &= left - 1) {
                    const int holder = __ffs(left) - 1, at = (holder >> shift) * size;
                    double f = -INFINITY, n = -INFINITY;
#pragma unroll 1
                    for (int e = at + lane; e < at + size; e += 32) {
                        const double v = key64(e);
                        if (v > f) { n = f; f = v; }
                        else if (v > n) n = v;
                    }
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) {
                        const double F = __shfl_xor_sync(kFull, f, o), N = __shfl_xor_sync(kFull, n, o);
                        n = fmax(fmax(n, N), fmin(f, F));
                        f = fmax(f, F);
                    }
                    double r = a.group_top == 2 ? f + n : f;
                    if (!(r == r)) r = -INFINITY;
                    if (best < 0 || r > most) { best = holder; most = r; }   // equal ones: the lowest group
                }
            }
            open |= 1u << best;
            if (lane == best) gkey = kTaken;
        }
        // e / size for e < 1024: the reciprocal is off by less than e / 2^20 < 1 / size
        const uint32_t inverse = ((1u << 20) + size - 1) / size;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int e = 32 * i + lane;
            if (e < E && !((open >> (((e * inverse) >> 20) << shift)) & 1u)) key[i] = kOutside;
        }
    }

    // the topk-th largest lane maximum (or below it: equal ones count at once)
    uint32_t top = key[0];
#pragma unroll
    for (int i = 1; i < VPT; ++i) top = max(top, key[i]);
    reinterpret_cast<uint32_t*>(tops[warp])[lane] = top;
    __syncwarp();
    int from = 0;                                            // lanes whose largest is not below this one's
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint4 u = tops[warp][i];
        from += (u.x >= top) + (u.y >= top) + (u.z >= top) + (u.w >= top);
    }
    uint32_t bound = __reduce_max_sync(kFull, from >= a.topk ? top : 0u);
    if (a.bias && bound > kNaN) bound = pattern(value(bound) - slack(value(bound)));
    bound = max(bound, kNaN);                                // there are topk experts inside the chosen groups
    int count = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const bool in = key[i] >= bound;
        const uint32_t mask = __ballot_sync(kFull, in);
        const int at = count + __popc(mask & ((1u << lane) - 1u));
        if (in && at < 32) gathered[warp][at] = make_uint2(key[i], (uint32_t)(32 * i + lane));
        count += __popc(mask);
    }
    __syncwarp();

    int mine = 0, place = 32;                                // this lane's expert and its place in the output
    if (count <= 32) {
        // in order of the expert's index: an equal key before this one's goes first
        const uint2 c = lane < count ? gathered[warp][lane] : make_uint2(kTaken, 0);
        mine = (int)c.y;
        place = lane < count ? 0 : 32;
        bool near = false;
        if (a.bias) {
            const float v = value(c.x), reach = slack(v);
#pragma unroll 4
            for (int j = 0; j < count; ++j) {
                const uint32_t k = __shfl_sync(kFull, c.x, j);
                place += (k > c.x || (k == c.x && j < lane)) ? 1 : 0;
                near |= j != lane && c.x > kNaN && k > kNaN && fabsf(value(k) - v) <= reach;
            }
        } else {
#pragma unroll 4
            for (int j = 0; j < count; ++j) {
                const uint32_t k = __shfl_sync(kFull, c.x, j);
                place += (k > c.x || (k == c.x && j < lane)) ? 1 : 0;
            }
        }
        if (__any_sync(kFull, near && lane < count)) {
            need64();
            double k64 = c.x > kMasked ? key64(mine) : -INFINITY;
            if (!(k64 == k64)) k64 = -INFINITY;
            // NaN patterns are behind every number
            const int group = c.x > kNaN;
            place = lane < count ? 0 : 32;
            for (int j = 0; j < count; ++j) {
                const double k = __shfl_sync(kFull, k64, j);
                const int other = __shfl_sync(kFull, group, j);
                place += (other > group || (other == group && (k > k64 || (k == k64 && j < lane)))) ? 1 : 0;
            }
        }
    } else {
        // one maximum after the other
        for (int j = 0; j < a.topk; ++j) {
            uint32_t t = key[0];
#pragma unroll
            for (int i = 1; i < VPT; ++i) t = max(t, key[i]);
            const uint32_t m = __reduce_max_sync(kFull, t);
            uint32_t least = m;
            if (a.bias && m > kNaN) least = pattern(value(m) - slack(value(m)));
            int n = 0;
#pragma unroll
            for (int i = 0; i < VPT; ++i) n += key[i] >= least;
            int best;
            if (least < m && __reduce_add_sync(kFull, (unsigned)n) > 1) {
                need64();
                double bk = -INFINITY;
                int be = 0;
                bool has = false;
#pragma unroll
                for (int i = 0; i < VPT; ++i)
                    if (key[i] >= least) {
                        const double k = key64(32 * i + lane);
                        if (!has || k > bk) { bk = k; be = 32 * i + lane; has = true; }
                    }
                best = best64(bk, be, has);
            } else {
                uint32_t e = 0xFFFFFFFFu;
#pragma unroll
                for (int i = VPT - 1; i >= 0; --i)
                    if (key[i] == m) e = 32 * i + lane;
                best = (int)__reduce_min_sync(kFull, e);
            }
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (32 * i + lane == best) key[i] = kTaken;
            if (lane == j) {
                mine = best;
                place = j;
            }
        }
    }

    // weights of the chosen experts
    const bool have = place < a.topk;
    const float x = have ? load_logit<T>(row + mine) : -INFINITY;
    float p;
    if (SIGMOID) {
        p = sigmoid(x);
    } else if (a.renormalize) {                              // softmax over the chosen logits
        const float cm = warp_max(x);
        p = cm == -INFINITY && !(x != x) ? 0.0f : expf(x - cm);
    } else {
        p = mx == -INFINITY ? (x == x ? 0.0f : x) : __fdiv_rn(expf(x - mx), sum);
    }
    if (!have) p = 0.0f;
    if (a.renormalize) {
        const float total = warp_sum(p);
        p = total == 0.0f ? 0.0f : __fdiv_rn(p, total);
    }
    if (have) {
        a.ids[tok * a.topk + place] = mine;
        a.weights[tok * a.topk + place] = p * a.scale;
    }
}

// Up to eight of few experts, without a bias: LANES lanes per token, expert
// e = LANES i + s in register i of the token's lane s, 32 / LANES tokens per
// warp.  Each lane sorts its eight keys, and log2 LANES times two lanes merge
// their lists: the larger of element i of one and 7 - i of the other are the
// eight largest of both, in bitonic order.  No step waits for the one before
// as in taking maxima one after the other, and the four tokens of a warp
// share the instructions: 110 per token for 64 bf16 logits (16384 tokens:
// 4.3 us; as the kernel above 9.7; 256 logits 10.9).  A key carries its
// index, so that equal logits compare by it: in the lower half of a bf16
// logit's pattern (which is the type's own width), else in a second word.
template <int LANES, typename T> struct MergeKey;
template <int LANES> struct MergeKey<LANES, uint16_t> {
    using K = uint32_t;
    // NaN (2) becomes 0, below -inf (0x007F....)
    static __device__ __forceinline__ K make(uint32_t p, int e) { return (p & 0xFFFF0000u) | (uint32_t)(8 * LANES - e); }
    static __device__ __forceinline__ int index(K k) { return 8 * LANES - (int)(k & 0xFFFFu); }
};
template <int LANES> struct MergeKey<LANES, float> {
    using K = unsigned long long;
    static __device__ __forceinline__ K make(uint32_t p, int e) { return ((K)p << 32) | (uint32_t)(8 * LANES - e); }
    static __device__ __forceinline__ int index(K k) { return 8 * LANES - (int)(uint32_t)k; }
};

template <typename K>
__device__ __forceinline__ void order2(K& hi, K& lo) {
    const K a = hi, b = lo;
    hi = max(a, b);
    lo = min(a, b);
}

template <typename T, bool SIGMOID, int LANES>
__global__ void __launch_bounds__(32 * kGateWarps)
moe_gate_merge_kernel(const GateArgs a) {
    using M = MergeKey<LANES, T>;
    using K = typename M::K;
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, s = lane % LANES, E = a.experts;
    const int64_t tok = ((int64_t)blockIdx.x * kGateWarps + (threadIdx.x >> 5)) * (32 / LANES) + lane / LANES;
    const bool live = tok < a.tokens;                        // the warp's other tokens go on
    const T* row = static_cast<const T*>(a.logits) + (live ? tok : 0) * E;
    float l[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) l[i] = LANES * i + s < E ? load_logit<T>(row + LANES * i + s) : -INFINITY;
    float mx = -INFINITY, sum = 0.0f;
    if (!SIGMOID && !a.renormalize) {
#pragma unroll
        for (int i = 0; i < 8; ++i) mx = fmaxf(mx, l[i]);
#pragma unroll
        for (int o = 1; o < LANES; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
        if (mx != -INFINITY)
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += LANES * i + s < E ? expf(l[i] - mx) : 0.0f;
#pragma unroll
        for (int o = 1; o < LANES; o <<= 1) sum += __shfl_xor_sync(kFull, sum, o);
    }
    K k[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) k[i] = LANES * i + s < E ? M::make(pattern(l[i]), LANES * i + s) : (K)0;
    // Batcher's network for eight
    order2(k[0], k[1]); order2(k[2], k[3]); order2(k[4], k[5]); order2(k[6], k[7]);
    order2(k[0], k[2]); order2(k[1], k[3]); order2(k[4], k[6]); order2(k[5], k[7]);
    order2(k[1], k[2]); order2(k[5], k[6]);
    order2(k[0], k[4]); order2(k[1], k[5]); order2(k[2], k[6]); order2(k[3], k[7]);
    order2(k[2], k[4]); order2(k[3], k[5]);
    order2(k[1], k[2]); order2(k[3], k[4]); order2(k[5], k[6]);
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) {
        K other[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) other[i] = __shfl_xor_sync(kFull, k[7 - i], o);
#pragma unroll
        for (int i = 0; i < 8; ++i) k[i] = max(k[i], other[i]);
#pragma unroll
        for (int d = 4; d > 0; d >>= 1)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if ((i & d) == 0) order2(k[i], k[i + d]);
    }
    // every lane holds the token's list; lane j < topk takes choice j
    K own = k[0];
#pragma unroll
    for (int j = 1; j < 8; ++j)
        if (s == j) own = k[j];
    const bool have = live && s < a.topk;
    const int mine = M::index(own);
    const float x = have ? load_logit<T>(row + mine) : -INFINITY;
    float p;
    if (SIGMOID) {
        p = sigmoid(x);
    } else if (a.renormalize) {                              // softmax over the chosen logits
        float cm = x;
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) cm = fmaxf(cm, __shfl_xor_sync(kFull, cm, o));
        p = cm == -INFINITY && !(x != x) ? 0.0f : expf(x - cm);
    } else {
        p = mx == -INFINITY ? (x == x ? 0.0f : x) : __fdiv_rn(expf(x - mx), sum);
    }
    if (!have) p = 0.0f;
    if (a.renormalize) {
        float total = p;
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) total += __shfl_xor_sync(kFull, total, o);
        p = total == 0.0f ? 0.0f : __fdiv_rn(p, total);
    }
    if (have) {
        a.ids[tok * a.topk + s] = mine;
        a.weights[tok * a.topk + s] = p * a.scale;
    }
}

// ------------------------------------------------------------------ backward

struct GateBwdArgs {
    const void* logits;
    const int32_t* ids;
    const float* dweights;
    int64_t tokens;
    int experts, topk, renormalize;
    float scale;
    void* dlogits;
    uint32_t* err;
};

// With w_j = scale p_j (/ sum of the chosen p) and v_j = scale dw_j:
//   sigmoid:              dl_j = ds_j p_j (1 - p_j), 0 where not chosen,
//     ds_j = v_j, or with renormalize (v_j - sum_i v_i p_i / P) / P, P = sum p
//   softmax, renormalize: dl_j = c_j (v_j - sum_i v_i c_i), 0 where not
//     chosen, c = softmax over the chosen logits
//   softmax:              dl_e = p_e (ds_e - sum_i v_i p_i), ds_e = v_j at id j
// Only the last one reads every logit.
__device__ __forceinline__ int checked_id(const GateBwdArgs& a, int64_t tok, int choice, bool in) {
    if (!in) return -1;
    const int id = a.ids[tok * a.topk + choice];
    if (id >= 0 && id < a.experts) return id;
    raise_device_error(a.err, FPQ_ERR_DEVICE_BAD_INPUT);     // its gradient is dropped
    return -1;
}

// The first three: LANES lanes per token (at least topk), choice j in lane j.
// They write zeros, 16 bytes at a time, and then the few values.  Bound by
// those writes and by the latency of a token's chain (its ids, their logits,
// the sums): 16384 x 256 fp32 6.1 us, of which the zeros are 2.6; a warp per
// token 7.8.
template <typename T, bool SIGMOID, int LANES>
__global__ void __launch_bounds__(32 * kGateWarps)
moe_gate_bwd_kernel(const GateBwdArgs a) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, s = lane % LANES, E = a.experts;
    const int64_t tok = ((int64_t)blockIdx.x * kGateWarps + (threadIdx.x >> 5)) * (32 / LANES) + lane / LANES;
    const bool live = tok < a.tokens;                        // the warp's other tokens go on
    const int id = checked_id(a, tok, s, live && s < a.topk);
    const bool have = id >= 0;
    const float x = have ? load_logit<T>(static_cast<const T*>(a.logits) + tok * E + id) : -INFINITY;
    const float v = have ? a.scale * a.dweights[tok * a.topk + s] : 0.0f;
    T* out = static_cast<T*>(a.dlogits) + tok * E;
    const auto put = [&](int e, float f) {
        if (sizeof(T) == 4) reinterpret_cast<float*>(out)[e] = f;
        else reinterpret_cast<uint16_t*>(out)[e] = (uint16_t)f32_to_bf16(f);
    };
    if (live) {
        constexpr int per = 16 / (int)sizeof(T);
        if (E % per == 0) {
            for (int i = s; i < E / per; i += LANES) st_v4(reinterpret_cast<uint4*>(out) + i, make_uint4(0, 0, 0, 0));
        } else {
            for (int e = s; e < E; e += LANES) put(e, 0.0f);
        }
    }
    const auto token_sum = [&](float f) {
#pragma unroll
        for (int o = 1; o < LANES; o <<= 1) f += __shfl_xor_sync(kFull, f, o);
        return f;
    };
    float g;                                                 // what the choice adds at its id
    if (SIGMOID) {
        const float p = have ? sigmoid(x) : 0.0f, q = have ? sigmoid(-x) : 0.0f;   // q = 1 - p without cancellation
        g = v;
        if (a.renormalize) {
            const float P = token_sum(p), vp = token_sum(v * p);
            g = P == 0.0f ? 0.0f : __fdiv_rn(v - __fdiv_rn(vp, P), P);
        }
        g = g * p * q;
    } else {
        float mx = x;
#pragma unroll
        for (int o = 1; o < LANES; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
        const float c = have && mx != -INFINITY ? expf(x - mx) : 0.0f;
        const float total = token_sum(c), vc = token_sum(v * c);
        g = total == 0.0f ? 0.0f : __fdiv_rn(c, total) * (v - __fdiv_rn(vc, total));
    }
    // an id named twice gets the sum, in the order of the choices, with its
    // first choice
    const uint32_t same = __match_any_sync(kFull, have ? id | (lane / LANES) << 16 : -1 - lane);
    const bool first = have && __ffs(same) - 1 == lane;
    if (__any_sync(kFull, have && !first)) {
        float total = 0.0f;
        for (int j = 0; j < 32; ++j) {
            const float gj = __shfl_sync(kFull, g, j);
            if ((same >> j) & 1u) total += gj;
        }
        g = total;
    }
    __syncwarp();                                            // after the zeros
    if (first) put(id, g);
}

// The softmax over all experts: a warp per token, the row read once into
// registers and one exponential per logit; every entry is written as one that
// was not chosen, then the chosen ones again.  16384 x 256 fp32 8.6 us (3.9
// TB/s), 8192 x 512 6.6; read three times, with the chosen entries added in
// shared memory, 13.6 and 14.6.
template <typename T, int VPT>
__global__ void __launch_bounds__(32 * kGateWarps)
moe_gate_bwd_dense_kernel(const GateBwdArgs a) {
    pdl_trigger();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = a.experts;
    const int64_t tok = (int64_t)blockIdx.x * kGateWarps + warp;
    if (tok >= a.tokens) return;
    const T* row = static_cast<const T*>(a.logits) + tok * E;
    float l[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) l[i] = 32 * i + lane < E ? load_logit<T>(row + 32 * i + lane) : -INFINITY;
    const int id = checked_id(a, tok, lane, lane < a.topk);
    const bool have = id >= 0;
    const float v = have ? a.scale * a.dweights[tok * a.topk + lane] : 0.0f;
    const float x = have ? load_logit<T>(row + id) : -INFINITY;
    float mx = -INFINITY, sum = 0.0f, inverse = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) mx = fmaxf(mx, l[i]);
    mx = warp_max(mx);
    const bool some = mx != -INFINITY;                       // else every score is 0
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        l[i] = some && 32 * i + lane < E ? expf(l[i] - mx) : 0.0f;
        sum += l[i];
    }
    sum = warp_sum(sum);
    if (some) inverse = __fdiv_rn(1.0f, sum);
    const float p = have && some ? expf(x - mx) * inverse : 0.0f;
    const float dot = warp_sum(v * p), other = -dot * inverse;
    T* out = static_cast<T*>(a.dlogits) + tok * E;
    const auto put = [&](int e, float f) {
        if (sizeof(T) == 4) reinterpret_cast<float*>(out)[e] = f;
        else reinterpret_cast<uint16_t*>(out)[e] = (uint16_t)f32_to_bf16(f);
    };
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        if (32 * i + lane < E) put(32 * i + lane, l[i] * other);
    // an id named twice gets the sum, in the order of the choices
    const uint32_t same = __match_any_sync(kFull, have ? id : -1 - lane);
    const bool first = have && __ffs(same) - 1 == lane;
    float mine = v;
    if (__any_sync(kFull, have && !first)) {
        mine = 0.0f;
        for (int j = 0; j < 32; ++j) {
            const float vj = __shfl_sync(kFull, v, j);
            if ((same >> j) & 1u) mine += vj;
        }
    }
    __syncwarp();                                            // after the others
    if (first) put(id, p * (mine - dot));
}

// By the registers that a row of E takes at 32 lanes.
template <typename F>
cudaError_t by_registers(int E, F&& f) {
    if (E <= 32) return f(std::integral_constant<int, 1>());
    if (E <= 64) return f(std::integral_constant<int, 2>());
    if (E <= 128) return f(std::integral_constant<int, 4>());
    if (E <= 256) return f(std::integral_constant<int, 8>());
    if (E <= 512) return f(std::integral_constant<int, 16>());
    return f(std::integral_constant<int, 32>());
}

template <typename T, bool SIGMOID>
cudaError_t gate(const GateArgs& a, cudaStream_t st) {
    const dim3 grid((unsigned)((a.tokens + kGateWarps - 1) / kGateWarps)), block(32 * kGateWarps);
    const size_t smem = a.n_group > 1 ? (size_t)kGateWarps * (a.experts + a.experts / 32 + 1) * sizeof(float) : 0;
    const int E = a.experts;
    // Merging lists: without a bias, up to eight choices; 256 bf16 logits, 64
    // fp32 ones (whose two-word keys cost three times the instructions).
    if (!a.bias && a.n_group == 1 && a.topk <= 8 && E <= (sizeof(T) == 2 ? 256 : 64)) {
        const auto merge = [&](auto kernel, int lanes) {
            const int64_t per = kGateWarps * 32 / lanes;
            return launch_pdl(kernel, dim3((unsigned)((a.tokens + per - 1) / per)), block, 0, st, a);
        };
        if (E <= 64) return merge(moe_gate_merge_kernel<T, SIGMOID, 8>, 8);
        if constexpr (sizeof(T) == 2) {
            if (E <= 128) return merge(moe_gate_merge_kernel<T, SIGMOID, 16>, 16);
            return merge(moe_gate_merge_kernel<T, SIGMOID, 32>, 32);
        }
    }
    return by_registers(E, [&](auto n) {
        return launch_pdl(moe_gate_kernel<T, SIGMOID, decltype(n)::value>, grid, block, smem, st, a);
    });
}

}  // namespace

cudaError_t launch_moe_gate(const void* logits, int f32, const float* bias, int64_t tokens, int experts, int sigmoid,
                            int n_group, int topk_group, int group_top, int topk, int renormalize, float scale,
                            int32_t* ids, float* weights, cudaStream_t st) {
    const GateArgs a{logits, bias, tokens, experts, topk, n_group, topk_group, group_top, renormalize, scale, ids,
                     weights};
    if (f32) return sigmoid ? gate<float, true>(a, st) : gate<float, false>(a, st);
    return sigmoid ? gate<uint16_t, true>(a, st) : gate<uint16_t, false>(a, st);
}

cudaError_t launch_moe_gate_backward(const void* logits, int f32, const int32_t* ids, const float* dweights,
                                     int64_t tokens, int experts, int sigmoid, int topk, int renormalize,
                                     float scale, void* dlogits, uint32_t* err, cudaStream_t st) {
    const GateBwdArgs a{logits, ids, dweights, tokens, experts, topk, renormalize, scale, dlogits, err};
    const auto launch = [&](auto kernel, int per_warp) {
        const int64_t per = kGateWarps * per_warp;
        return launch_pdl(kernel, dim3((unsigned)((tokens + per - 1) / per)), dim3(32 * kGateWarps), 0, st, a);
    };
    if (!sigmoid && !renormalize)
        return by_registers(experts, [&](auto n) {
            constexpr int VPT = decltype(n)::value;
            return f32 ? launch(moe_gate_bwd_dense_kernel<float, VPT>, 1) : launch(moe_gate_bwd_dense_kernel<uint16_t, VPT>, 1);
        });
    // four tokens per warp where their choices fit: a quarter of the instructions
    if (topk <= 8) {
        if (f32)
            return sigmoid ? launch(moe_gate_bwd_kernel<float, true, 8>, 4) : launch(moe_gate_bwd_kernel<float, false, 8>, 4);
        return sigmoid ? launch(moe_gate_bwd_kernel<uint16_t, true, 8>, 4) : launch(moe_gate_bwd_kernel<uint16_t, false, 8>, 4);
    }
    if (f32)
        return sigmoid ? launch(moe_gate_bwd_kernel<float, true, 32>, 1) : launch(moe_gate_bwd_kernel<float, false, 32>, 1);
    return sigmoid ? launch(moe_gate_bwd_kernel<uint16_t, true, 32>, 1) : launch(moe_gate_bwd_kernel<uint16_t, false, 32>, 1);
}

}  // namespace fpq
