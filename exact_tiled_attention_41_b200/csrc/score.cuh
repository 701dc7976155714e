// score.cuh -- scores that are capped by a tanh and / or biased by the distance of query and key.
//
// With a cap (softcapping: flash-attention README, changelog 2.6) and slopes (ALiBi: README,
// flash_attn_func docstring) the score of query i and key j of a sequence is
//     x_ij = cap tanh(scale q_i.k_j / cap) - slope_h |i + Lk - Lq - j|
// (either part may be absent), and softmax, output and LSE are those of x.  The derivative of the cap is
// 1 - tanh^2, so with t = tanh(scale q.k / cap) the gradient of the raw score is
//     dS = P (dP - Delta) (1 - t^2);
// the bias is data and has none.  The kernels work in log2 units: x log2(e) = t (cap log2(e)) + bias log2(e).
#pragma once

#include "internal.h"
#include "sm100.cuh"

#include <type_traits>

namespace fa {

// Score mode of a kernel instance, a bit mask; 0 leaves the kernels as they are without modifiers.
constexpr int kScorePlain = 0, kScoreCap = 1, kScoreBias = 2;
constexpr int kScoreWide = 4;          // a cap beyond kNarrowCap: another softmax reference and tanh
constexpr float kNarrowCap = 55.f;     // 55 log2(e) < 80

// Coefficients of the tanh polynomials, see cap_pair below.
#define FA_TANH2 {0.12841614f, -0.33321908f, 0.9999996f}
#define FA_TANH4 {0.0171350036f, -0.0529860742f, 0.133247793f, -0.333330691f, 1.0f}
#define FA_TANH6 {0.0010410226f, -0.00620337902f, 0.0202899799f, -0.0534570292f, 0.13325204f, -0.333328396f, 0.99999994f}

struct ScoreParams {
    float in;             // scale / cap: raw score -> argument of the tanh
    float out_log2;       // cap * log2(e): tanh -> score in log2 units
    const float* slopes;  // [Hq] (slope_sB = 0) or [B][Hq] (slope_sB = Hq)
    int slope_sB;
    // The tanh polynomials (kTanh2, kTanh4) in the raw score, with both factors in the coefficients (each
    // doubled for the packed FMA): out_log2 tanh(in s) = s (fold[0] w^n + ... + fold[n]), w = s^2, for |s| up to
    // limit[range]; limit[2]: |in s| <= 1.
    float2 fold2[3], fold4[5];
    float limit[3];
    // log2 of the factor by which a row's reference lies above its largest bias (the forward's fixed reference): P is at
    // most 2^8 up to a cap of 33 (as against a running maximum), and at most 2^71 at 55, its least 2^-88
    float ref_log2;
};

inline ScoreParams score_params(float scale, float softcap, const float* slopes, int slope_sB) {
    ScoreParams sc = {softcap > 0.f ? scale / softcap : 0.f, softcap * 1.4426950408889634f, slopes, slope_sB};
    if (softcap > 0.f) {
        // the folded form serves while its coefficients (in^9 out_log2 the extreme one) are normal floats: one that became 0
        // would make NaN of a masked score's infinite square.  No usual scale and cap goes beyond.
        bool fits = sc.in >= 0x1p-13f && sc.in <= 0x1p13f;
        const double in = sc.in, c2[3] = FA_TANH2, c4[5] = FA_TANH4;
        double f = in * sc.out_log2;
        for (int k = 0; k < 5; ++k, f *= in * in) {
            if (k < 3) sc.fold2[2 - k] = make_float2(static_cast<float>(c2[2 - k] * f), static_cast<float>(c2[2 - k] * f));
            sc.fold4[4 - k] = make_float2(static_cast<float>(c4[4 - k] * f), static_cast<float>(c4[4 - k] * f));
            fits = fits && fabs(c4[4 - k] * f) >= 0x1p-126 && fabs(c4[4 - k] * f) < 0x1p127;
        }
        sc.limit[0] = fits ? 0.25f / sc.in : -1.f;
        sc.limit[1] = fits ? 0.5f / sc.in : -1.f;
        sc.limit[2] = 1.f / sc.in;
        const float top = 2.f * sc.out_log2 - 88.f;
        sc.ref_log2 = sc.out_log2 - (top > 8.f ? top : 8.f);
    }
    return sc;
}
inline ScoreParams score_params(const Problem& pr) {
    return score_params(pr.scale, pr.softcap, pr.slopes, pr.slope_sB);
}

// Calls run(std::integral_constant<int, mode>) for the modifiers given; the mode has kScoreWide where the cap asks for it.
template <typename F>
int with_score_mode(float softcap, const float* slopes, F&& run) {
    const bool wide = softcap > kNarrowCap;
    switch (score_mode(softcap, slopes)) {
        case kScorePlain: return run(std::integral_constant<int, kScorePlain>{});
        case kScoreBias: return run(std::integral_constant<int, kScoreBias>{});
        case kScoreCap:
            return wide ? run(std::integral_constant<int, kScoreCap | kScoreWide>{})
                        : run(std::integral_constant<int, kScoreCap>{});
        default:
            return wide ? run(std::integral_constant<int, kScoreCap | kScoreBias | kScoreWide>{})
                        : run(std::integral_constant<int, kScoreCap | kScoreBias>{});
    }
}

__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// tanh(x) = 1 - 2 / (1 + e^(2x)); absolute error about 2e-7 (ex2 and rcp on the multi-function unit are
// good to 2 ulp; near 0 the difference cancels, so the error is relative to 1, not to x, and a score is off by 2e-7 of
// the cap).  Large |x| gives exactly +-1: e^(2x) becomes inf or 0.
__device__ __forceinline__ float tanh_mufu(float x) {
    const float e = ex2_approx(x * 2.885390081777927f);   // 2 log2(e)
    return fmaf(-2.f, rcp_approx(1.f + e), 1.f);
}

__device__ __forceinline__ float2 splat2(float v) { return make_float2(v, v); }

// tanh(x) of a pair by the range of the arguments: x p(x^2) on the FMA pipe, with p of the smallest maximum relative
// error on its range (exact_tiled_attention_41_b200/fit_tanh_poly.py prints the coefficients; within 5e-7 relative for
// |x| <= 1/4, 2e-7 up to 1).  The polynomials' leading coefficients are positive: -inf stays -inf.
static __constant__ float kTanh2[3] = FA_TANH2;
static __constant__ float kTanh4[5] = FA_TANH4;
static __constant__ float kTanh6[7] = FA_TANH6;
enum TanhRange { kTanhQuarter, kTanhHalf, kTanhOne, kTanhAny };

template <int RANGE>
__device__ __forceinline__ float2 tanh_poly(float2 x) {
    static_assert(RANGE != kTanhAny, "no polynomial reaches that far");
    const float2 u = fmul2(x, x);
    constexpr int DEG = RANGE == kTanhQuarter ? 2 : RANGE == kTanhHalf ? 4 : 6;
    const float* c = RANGE == kTanhQuarter ? kTanh2 : RANGE == kTanhHalf ? kTanh4 : kTanh6;
    float2 p = ffma2(splat2(c[0]), u, splat2(c[1]));
#pragma unroll
    for (int i = 2; i <= DEG; ++i) p = ffma2(p, u, splat2(c[i]));
    return fmul2(p, x);
}

// tanh(x) of a pair, each within 3e-7 of its value whatever the other elements are: the polynomial up to 1, the
// multi-function unit beyond, where its error relative to 1 is one relative to the value.  (The unit alone was off by 3 %
// of the output at a cap of 1e6 and scores of a few units.)
__device__ __forceinline__ float2 tanh_pair(float2 x) {
    const float2 p = tanh_poly<kTanhOne>(x);
    return make_float2(fabsf(x.x) <= 1.f ? p.x : tanh_mufu(x.x), fabsf(x.y) <= 1.f ? p.y : tanh_mufu(x.y));
}

// tanh(in * s) of a pair of raw scores, all of a warp's within RANGE.  Where some lie beyond 1 the unit serves all of them
// for caps up to kNarrowCap, whose scores are then off by 1.1e-5 at most; WIDE, a larger cap, takes each by its size (in
// the gradient kernels 9 % of the time at scores around the cap, and 3 % at small ones, which is why the narrow caps do
// without).  A raw score beyond float32, +-inf, gives +-1: masks come later.
template <int RANGE, bool WIDE = false>
__device__ __forceinline__ float2 cap_pair(float2 s, float2 in) {
    const float2 x = fmul2(s, in);
    if constexpr (RANGE != kTanhAny) return tanh_poly<RANGE>(x);
    else if constexpr (WIDE) return tanh_pair(x);
    else return make_float2(tanh_mufu(x.x), tanh_mufu(x.y));
}

// The same for a pair without a vote: the kernels whose tanh is little of their work.
__device__ __forceinline__ float2 cap_pair_alone(float2 s, const ScoreParams& sc) {
    const float2 x = fmul2(s, splat2(sc.in));
    if (sc.out_log2 > kNarrowCap * 1.4426950408889634f) return tanh_pair(x);
    return make_float2(tanh_mufu(x.x), tanh_mufu(x.y));
}

// The larger of two, NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// out_log2 tanh(in s) + b of a pair of raw scores of a narrow cap: the folded polynomials where they reach.  Where some
// scores of the tile are masked, -inf is their mark and stays -inf.
template <int RANGE>
__device__ __forceinline__ float2 cap_pair_log2(float2 s, const ScoreParams& sc, float2 b, bool masked) {
    if constexpr (RANGE == kTanhQuarter || RANGE == kTanhHalf) {
        const float2 w = fmul2(s, s);
        float2 p;
        if constexpr (RANGE == kTanhQuarter) {
            p = ffma2(ffma2(sc.fold2[0], w, sc.fold2[1]), w, sc.fold2[2]);
        } else {
            p = ffma2(sc.fold4[0], w, sc.fold4[1]);
#pragma unroll
            for (int i = 2; i < 5; ++i) p = ffma2(p, w, sc.fold4[i]);
        }
        return ffma2(s, p, b);
    } else {
        float2 t = cap_pair<RANGE>(s, splat2(sc.in));
        if constexpr (RANGE == kTanhAny)
            t = make_float2(masked && s.x == -INFINITY ? -INFINITY : t.x, masked && s.y == -INFINITY ? -INFINITY : t.y);
        return ffma2(t, splat2(sc.out_log2), b);
    }
}

// Calls run(std::integral_constant<int, range>) for the smallest range that holds every argument of the warp
// (most: the largest |raw score| of the thread).  The softmax already keeps the multi-function unit busy with one
// exponential per score, and a tanh there costs two more results, while the FMA pipe has room; with a cap
// well above the scores, as caps are chosen, every block of scores takes one of the first ranges.
template <typename F>
__device__ __forceinline__ void with_tanh_range(float most, const ScoreParams& sc, F&& run) {
    if (__all_sync(0xffffffffu, most <= sc.limit[0])) run(std::integral_constant<int, kTanhQuarter>{});
    else if (__all_sync(0xffffffffu, most <= sc.limit[1])) run(std::integral_constant<int, kTanhHalf>{});
    else if (__all_sync(0xffffffffu, most <= sc.limit[2])) run(std::integral_constant<int, kTanhOne>{});
    else run(std::integral_constant<int, kTanhAny>{});
}

template <int N>
__device__ __forceinline__ float max_abs(const float (&s)[N]) {
    float m[2] = {fabsf(s[0]), fabsf(s[1])};
#pragma unroll
    for (int e = 2; e < N; e += 2) m[(e >> 1) & 1] = max3f(m[(e >> 1) & 1], fabsf(s[e]), fabsf(s[e + 1]));
    return fmaxf(m[0], m[1]);
}

// s <- tanh(in * s) for a thread's block of raw scores; a thread that is not valid (a row past its sequence) has no
// part in the warp's choice of polynomial
template <bool WIDE, int N>
__device__ __forceinline__ void cap_scores(float (&s)[N], const ScoreParams& sc, bool valid = true) {
    with_tanh_range(valid ? max_abs(s) : 0.f, sc, [&](auto range) {
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            const float2 t = cap_pair<decltype(range)::value, WIDE>(make_float2(s[e], s[e + 1]), splat2(sc.in));
            s[e] = t.x;
            s[e + 1] = t.y;
        }
    });
}
template <bool WIDE, int N>
__device__ __forceinline__ void cap_scores(uint32_t (&s)[N], const ScoreParams& sc, bool valid = true) {
    cap_scores<WIDE>(reinterpret_cast<float (&)[N]>(s), sc, valid);
}

// slope * log2(e) of query head h of sequence b
__device__ __forceinline__ float slope_log2(const ScoreParams& sc, int b, int h) {
    return __ldg(sc.slopes + static_cast<size_t>(b) * sc.slope_sB + h) * 1.4426950408889634f;
}

// bias (log2 units) at signed distance d: -slope |d|.  Distances are formed in fp32, exact up to 2^24 tokens.
__device__ __forceinline__ float bias_log2(float d, float slope) { return -slope * fabsf(d); }

// Adds the bias to a thread's row of scores, column c at distance d0 - c; slope in the unit of s.  Where the
// warp's columns all lie on one side of the diagonal (past: every column that the mask keeps does) the bias is
// linear in c, so only its column part is added, one FMA per score, and the row's part is returned; across
// the diagonal the whole bias is added and 0 returned.
template <int N>
__device__ __forceinline__ float bias_scores(float (&s)[N], float slope, float d0, bool past) {
    const bool behind = past || __all_sync(0xffffffffu, d0 >= N - 1);
    if (behind || __all_sync(0xffffffffu, d0 <= 0.f)) {
        const float step = behind ? slope : -slope;
#pragma unroll
        for (int c = 1; c < N; ++c) s[c] = fmaf(step, static_cast<float>(c), s[c]);
        return -step * d0;
    }
#pragma unroll
    for (int c = 0; c < N; ++c) s[c] = fmaf(-slope, fabsf(d0 - c), s[c]);
    return 0.f;
}

// gradient of the raw scores from that of the capped ones: ds (1 - t^2), t the tanh
__device__ __forceinline__ float2 cap_gradient(float2 ds, float2 t) {
    return fmul2(ds, ffma2(make_float2(-t.x, -t.y), t, make_float2(1.f, 1.f)));
}

}  // namespace fa
