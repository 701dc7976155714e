// bwd_delta.cu -- Delta of the backward from the probabilities themselves, for rows that see few keys.
//
// The preprocess forms Delta_i = sum_d dO_id O_id with the stored, rounded O.  O's rounding (2^-9 relative on
// average) reaches every dS_ij = P_ij (dP_ij - Delta_i) of the row with the factor P_ij.  Over many keys that is small
// beside dS.  A row that a window, a steep bias or a short sequence leaves with two or three keys puts most of its
// weight on one of them, whose dP_ij nearly equals Delta_i, and there the error is a percent of dS: dq and dk of a
// window of 2 keys were 7e-3 off (Frobenius), 2.6e-3 with the sum below, most of it their own rounding.
//     Delta_i = sum_j P_ij dP_ij,   P_ij = exp2(x_ij - LSE2_i),   dP_ij = dO_i . v_j      (fp32)
// Only calls with score modifiers use it (the others keep the bits they had), and of them those where it costs
// little (delta_pays below); for rows of many keys the preprocess's sum stands.
//
// A block takes 16 query rows of a head; its four warps take every fourth tile of 16 keys and form the 16 x 16 scores
// and dP with bf16 mma.sync (16 rows could not fill a 128-row tcgen05 tile, and the work is small by the rule).
// A lane loads 16 bytes of a row at a time, 8 consecutive values: the products contract over the head dimension in
// whatever order both operands agree on, so values 8t .. 8t + 7 of each 32 serve lane t of a quad in two steps.
#include "internal.h"
#include "score.cuh"
#include "sm100.cuh"

namespace fa {

namespace {

struct DeltaParams {
    const __nv_bfloat16 *q, *k, *v, *dout;
    const float* lse2;      // [Hq][Tq]
    float* delta;           // [Hq][Tq]
    const int32_t* cu_q;
    const int32_t* cu_k;
    int Sq, Sk, Tq, Tk, Hq, Hkv, group, blocks;
    float scale_log2;
    int wl, wr;             // window sides, -1 = unbounded; a causal mask is wr = 0
    ScoreParams sc;
};

template <int D, int MODE>
__global__ void __launch_bounds__(128) bwd_delta_kernel(const __grid_constant__ DeltaParams p) {
    constexpr int KP = D / 32;
    __shared__ float part[4][16];
    const int u = blockIdx.x;
    const int q0 = (u % p.blocks) * 16, h = u / p.blocks % p.Hq, b = u / p.blocks / p.Hq;
    int q_start = b * p.Sq, Lq = p.Sq, k_start = b * p.Sk, Lk = p.Sk;
    if (p.cu_q != nullptr) {
        q_start = max(__ldg(p.cu_q + b), 0);
        k_start = max(__ldg(p.cu_k + b), 0);
        Lq = __ldg(p.cu_q + b + 1) - __ldg(p.cu_q + b);
        Lk = __ldg(p.cu_k + b + 1) - __ldg(p.cu_k + b);
        Lq = max(min(min(Lq, p.Tq - q_start), 1 << 30), 0);   // malformed offsets can only shrink the work
        Lk = max(min(min(Lk, p.Tk - k_start), 1 << 30), 0);
    }
    if (q0 >= Lq) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = lane >> 2, t = lane & 3;
    const int off = Lk - Lq, hk = h / p.group;
    const int row[2] = {q0 + quad, q0 + quad + 8};
    // keys that some row of the block sees
    const int lo = p.wl >= 0 ? max(0, q0 + off - p.wl) : 0;
    const int hi = p.wr >= 0 ? min(Lk - 1, min(q0 + 15, Lq - 1) + off + p.wr) : Lk - 1;
    uint4 qf[2][KP], df[2][KP];
    int key_lo[2], key_hi[2];
    float l2[2], slope = 0.f, acc[2] = {0.f, 0.f};
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int in = min(row[r], Lq - 1);   // rows past the sequence repeat its last one and are not written
        const size_t at = (static_cast<size_t>(q_start + in) * p.Hq + h) * D + t * 8;
#pragma unroll
        for (int kp = 0; kp < KP; ++kp) {
            qf[r][kp] = __ldg(reinterpret_cast<const uint4*>(p.q + at + kp * 32));
            df[r][kp] = __ldg(reinterpret_cast<const uint4*>(p.dout + at + kp * 32));
        }
        l2[r] = p.lse2[static_cast<size_t>(h) * p.Tq + q_start + in];
        key_lo[r] = p.wl >= 0 ? in + off - p.wl : 0;
        key_hi[r] = p.wr >= 0 ? min(Lk - 1, in + off + p.wr) : Lk - 1;
    }
    if constexpr ((MODE & kScoreBias) != 0) slope = slope_log2(p.sc, b, h);
    for (int k0 = lo / 16 * 16 + warp * 16; k0 <= hi; k0 += 64) {
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int kn = k0 + 8 * n;
            const size_t at = (static_cast<size_t>(k_start + min(kn + quad, Lk - 1)) * p.Hkv + hk) * D + t * 8;
            float s[4] = {0.f, 0.f, 0.f, 0.f}, dp[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int kp = 0; kp < KP; ++kp) {
                const uint4 kf = __ldg(reinterpret_cast<const uint4*>(p.k + at + kp * 32));
                const uint4 vf = __ldg(reinterpret_cast<const uint4*>(p.v + at + kp * 32));
                const uint32_t qa[4] = {qf[0][kp].x, qf[1][kp].x, qf[0][kp].y, qf[1][kp].y};
                const uint32_t qb[4] = {qf[0][kp].z, qf[1][kp].z, qf[0][kp].w, qf[1][kp].w};
                const uint32_t da[4] = {df[0][kp].x, df[1][kp].x, df[0][kp].y, df[1][kp].y};
                const uint32_t db[4] = {df[0][kp].z, df[1][kp].z, df[0][kp].w, df[1][kp].w};
                mma_bf16_16816(s, qa, kf.x, kf.y);
                mma_bf16_16816(s, qb, kf.z, kf.w);
                mma_bf16_16816(dp, da, vf.x, vf.y);
                mma_bf16_16816(dp, db, vf.z, vf.w);
            }
            if constexpr ((MODE & kScoreCap) != 0) {
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    const float2 x = cap_pair_alone(make_float2(s[e], s[e + 1]), p.sc);
                    s[e] = x.x;
                    s[e + 1] = x.y;
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = e >> 1, key = kn + 2 * t + (e & 1);
                float x = s[e] * ((MODE & kScoreCap) ? p.sc.out_log2 : p.scale_log2);
                if constexpr ((MODE & kScoreBias) != 0) x += bias_log2(static_cast<float>(row[r] + off - key), slope);
                const bool keep = key >= key_lo[r] && key <= key_hi[r];
                acc[r] += keep ? ex2_approx(x - l2[r]) * dp[e] : 0.f;
            }
        }
    }
    // a row's sum: the quad, then the warps in order
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        acc[r] += __shfl_xor_sync(0xffffffffu, acc[r], 1);
        acc[r] += __shfl_xor_sync(0xffffffffu, acc[r], 2);
        if (t == 0) part[warp][quad + 8 * r] = acc[r];
    }
    __syncthreads();
    const int i = threadIdx.x;
    if (i < 16 && q0 + i < Lq)
        p.delta[static_cast<size_t>(h) * p.Tq + q_start + q0 + i] = part[0][i] + part[1][i] + part[2][i] + part[3][i];
}

// Rows of at most 16 keys always (two or three tiles a block, some 5 % of the backward), and other problems up to
// 32,768 tiles in all, which take a few us: gradients of few rows, whose error nothing averages out.
bool delta_pays(const Problem& pr, long long blocks) {
    const bool banded = pr.wl >= 0 && pr.wr >= 0;
    if (banded && static_cast<long long>(pr.wl) + pr.wr + 1 <= 16) return true;
    long long keys = pr.Sk;
    if (banded && static_cast<long long>(pr.wl) + pr.wr + 16 < keys) keys = static_cast<long long>(pr.wl) + pr.wr + 16;
    return blocks * ((keys + 15) / 16) <= 32768;
}

}  // namespace

int launch_bwd_delta(const Problem& pr, const void* dout, const float* lse2, float* delta, cudaStream_t stream) {
    const int mode = score_mode(pr.softcap, pr.slopes);
    if (mode == kScorePlain) return 0;
    DeltaParams p;
    p.blocks = (pr.Sq + 15) / 16;
    const long long blocks = static_cast<long long>(p.blocks) * pr.Hq * pr.num_seqs;
    if (!delta_pays(pr, blocks) || blocks > 0x7fffffffLL) return 0;
    p.q = static_cast<const __nv_bfloat16*>(pr.q);
    p.k = static_cast<const __nv_bfloat16*>(pr.k);
    p.v = static_cast<const __nv_bfloat16*>(pr.v);
    p.dout = static_cast<const __nv_bfloat16*>(dout);
    p.lse2 = lse2;
    p.delta = delta;
    p.cu_q = pr.cu_q;
    p.cu_k = pr.cu_k;
    p.Sq = pr.Sq;
    p.Sk = pr.Sk;
    p.Tq = pr.Tq;
    p.Tk = pr.Tk;
    p.Hq = pr.Hq;
    p.Hkv = pr.Hkv;
    p.group = pr.Hq / pr.Hkv;
    p.scale_log2 = pr.scale * 1.4426950408889634f;
    p.wl = pr.wl;
    p.wr = pr.wr;
    p.sc = score_params(pr);
    auto run = [&](auto m) {
        constexpr int MODE = decltype(m)::value & ~kScoreWide;   // the kernel looks at the cap itself
        if constexpr (MODE != kScorePlain) {
            const unsigned grid = static_cast<unsigned>(blocks);
            switch (pr.D) {
                case 64: bwd_delta_kernel<64, MODE><<<grid, 128, 0, stream>>>(p); break;
                case 128: bwd_delta_kernel<128, MODE><<<grid, 128, 0, stream>>>(p); break;
                case 256: bwd_delta_kernel<256, MODE><<<grid, 128, 0, stream>>>(p); break;
                default: return 2;
            }
        }
        return cudaPeekAtLastError() == cudaSuccess ? 0 : 5;
    };
    return with_score_mode(pr.softcap, pr.slopes, run);
}

}  // namespace fa
