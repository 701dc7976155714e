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

struct ScoreParams {
    float in;             // scale / cap: raw score -> argument of the tanh
    float out_log2;       // cap * log2(e): tanh -> score in log2 units
    const float* slopes;  // [Hq] (slope_sB = 0) or [B][Hq] (slope_sB = Hq)
    int slope_sB;
};

inline ScoreParams score_params(float scale, float softcap, const float* slopes, int slope_sB) {
    return {softcap > 0.f ? scale / softcap : 0.f, softcap * 1.4426950408889634f, slopes, slope_sB};
}
inline ScoreParams score_params(const Problem& pr) {
    return score_params(pr.scale, pr.softcap, pr.slopes, pr.slope_sB);
}

// Calls run(std::integral_constant<int, mode>) for the mode asked for.
template <typename F>
int with_score_mode(int mode, F&& run) {
    switch (mode) {
        case kScorePlain: return run(std::integral_constant<int, kScorePlain>{});
        case kScoreCap: return run(std::integral_constant<int, kScoreCap>{});
        case kScoreBias: return run(std::integral_constant<int, kScoreBias>{});
        default: return run(std::integral_constant<int, kScoreCap | kScoreBias>{});
    }
}

__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// tanh(x) = 1 - 2 / (1 + e^(2x)); absolute error about 2e-7 (ex2 and rcp on the multi-function unit are
// good to 2 ulp; near 0 the difference cancels, so the error is relative to 1, not to x).  Large |x|
// gives exactly +-1: e^(2x) becomes inf or 0.
__device__ __forceinline__ float tanh_mufu(float x) {
    const float e = ex2_approx(x * 2.885390081777927f);   // 2 log2(e)
    return fmaf(-2.f, rcp_approx(1.f + e), 1.f);
}

// tanh of a pair on the FMA pipe, x p(x^2) with p of the smallest maximum relative error on its range
// (exact_tiled_attention_41_b200/fit_tanh_poly.py prints the coefficients): within 2e-7 relative.
__device__ __forceinline__ float2 splat2(float v) { return make_float2(v, v); }

__device__ __forceinline__ float2 tanh_half(float2 x) {   // |x| <= 1/2
    const float2 u = fmul2(x, x);
    float2 p = ffma2(splat2(0.0171350036f), u, splat2(-0.0529860742f));
    p = ffma2(p, u, splat2(0.133247793f));
    p = ffma2(p, u, splat2(-0.333330691f));
    p = ffma2(p, u, splat2(1.0f));
    return fmul2(p, x);
}

__device__ __forceinline__ float2 tanh_one(float2 x) {    // |x| <= 1
    const float2 u = fmul2(x, x);
    float2 p = ffma2(splat2(0.0010410226f), u, splat2(-0.00620337902f));
    p = ffma2(p, u, splat2(0.0202899799f));
    p = ffma2(p, u, splat2(-0.0534570292f));
    p = ffma2(p, u, splat2(0.13325204f));
    p = ffma2(p, u, splat2(-0.333328396f));
    p = ffma2(p, u, splat2(0.99999994f));
    return fmul2(p, x);
}

// s <- tanh(in * s) for a thread's block of raw scores.  The softmax already keeps the multi-function unit busy with
// one exponential per score, and a tanh there costs two more results; the FMA pipe has room.  So the warp takes
// a polynomial whenever all its arguments are within its range (with a cap well above the scores, as caps are
// chosen, that is every block), and the multi-function unit otherwise.
template <int N>
__device__ __forceinline__ void cap_scores(float (&s)[N], float in) {
    float m[2] = {fabsf(s[0]), fabsf(s[1])};
#pragma unroll
    for (int e = 2; e < N; e += 2) m[(e >> 1) & 1] = max3f(m[(e >> 1) & 1], fabsf(s[e]), fabsf(s[e + 1]));
    const float most = fmaxf(m[0], m[1]) * in;
    const float2 in2 = splat2(in);
    if (__all_sync(0xffffffffu, most <= 0.5f)) {
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            const float2 t = tanh_half(fmul2(make_float2(s[e], s[e + 1]), in2));
            s[e] = t.x;
            s[e + 1] = t.y;
        }
    } else if (__all_sync(0xffffffffu, most <= 1.0f)) {
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            const float2 t = tanh_one(fmul2(make_float2(s[e], s[e + 1]), in2));
            s[e] = t.x;
            s[e + 1] = t.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) s[e] = tanh_mufu(s[e] * in);
    }
}
template <int N>
__device__ __forceinline__ void cap_scores(uint32_t (&s)[N], float in) {
    cap_scores(reinterpret_cast<float (&)[N]>(s), in);
}

// slope * log2(e) of query head h of sequence b
__device__ __forceinline__ float slope_log2(const ScoreParams& sc, int b, int h) {
    return __ldg(sc.slopes + static_cast<size_t>(b) * sc.slope_sB + h) * 1.4426950408889634f;
}

// bias (log2 units) at signed distance d: -slope |d|.  Distances are formed in fp32, exact up to 2^24 tokens.
__device__ __forceinline__ float bias_log2(float d, float slope) { return -slope * fabsf(d); }

// s <- mul s + bias for a thread's row of scores, column c at distance d0 - c.  Where the warp's columns all lie on one
// side of the diagonal (past: every column that the mask keeps does) the bias is one FMA, without it three
// operations.
template <int N>
__device__ __forceinline__ void bias_scores(float (&s)[N], float mul, float slope, float d0, bool past) {
    const bool behind = past || __all_sync(0xffffffffu, d0 >= N - 1);
    if (behind || __all_sync(0xffffffffu, d0 <= 0.f)) {
        const float step = behind ? slope : -slope, base = -step * d0;
#pragma unroll
        for (int c = 0; c < N; ++c) s[c] = fmaf(s[c], mul, fmaf(step, static_cast<float>(c), base));
    } else {
#pragma unroll
        for (int c = 0; c < N; ++c) s[c] = fmaf(s[c], mul, bias_log2(d0 - c, slope));
    }
}

// gradient of the raw scores from that of the capped ones: ds (1 - t^2), t the tanh
__device__ __forceinline__ float2 cap_gradient(float2 ds, float2 t) {
    return fmul2(ds, ffma2(make_float2(-t.x, -t.y), t, make_float2(1.f, 1.f)));
}

}  // namespace fa
