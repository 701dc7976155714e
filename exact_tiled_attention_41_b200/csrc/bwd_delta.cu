// bwd_delta.cu -- Delta of the backward from the probabilities themselves, for rows that see few keys.
//
// The preprocess forms Delta_i = sum_d dO_id O_id with the stored, rounded O.  O's rounding (2^-9 relative on
// average) reaches every dS_ij = P_ij (dP_ij - Delta_i) of the row with the factor P_ij.  Over many keys that is small
// beside dS.  A row that a window, a steep bias or a short sequence leaves with a few keys puts most of its
// weight on one of them, whose dP_ij nearly equals Delta_i, and there the error is a percent of dS.
//     Delta_i = sum_j P_ij dP_ij,   P_ij = exp2(x_ij - LSE2_i),   dP_ij = dO_i . v_j      (fp32)
// Only calls with score modifiers use it (the others keep the bits they had), and of their rows those that see few keys;
// for the others the preprocess's sum stands.  The choice follows from a row's own sequence, mask and slope, so the
// gradients of a sequence do not depend on the batch that it stands in:
//  * its rows see at most 16 keys (of a window, or of the sequence), or at most 64 where the sequence has at most 512
//    queries, since a gradient of few rows averages less: all of a row's keys;
//  * a head with a steep slope: the 48 keys with the largest bias, for the rows that put all but 2^-12 of their weight
//    there (what is left out is then below the rounding that this replaces).
// Error of dq (relative Frobenius norm) and time of the whole backward, without and with it (B200, 2 x 2048 causal tokens,
// 16 heads of 128, cap 30): windows of 17 keys 3.4e-3, 72 us and 2.4e-3, some 95 us, so they do without; slopes of
// 4 in all heads 1.1e-2, 162 us and 2.3e-3, 198 us; 0.5: 4.2e-3 and 2.3e-3; a slope of 0.25, left as it is, 3.7e-3.  The
// look at the blocks alone, where no head is steep, costs 5 us.  Short sequences pay most, for Q, K, V and dO are read once
// more: 512 packed ones of 64 tokens 578 us without, 749 with it (dq off by 3.0e-3 and 2.4e-3); 150 queries on 97 keys
// through a window of 41, cap and bias: 3.7e-3 and 2.4e-3 in some 4 us.
//
// A warp takes 16 query rows of a head and their keys 8 at a time: 16 x 8 scores and dP with bf16 mma.sync (16 rows could
// not fill a 128-row tcgen05 tile, and the work is small by the rule).  Bound by the latency of its loads, so many warps
// are wanted: with four warps to a block of rows, each with every fourth tile of 16 keys, windows of 2 to 16 keys took 32 us
// of the backward above, and take 22 to 24 so.  A warp looks at 32 blocks of rows at once for those that are to be summed.
// A lane loads 16 bytes of a row at a time, 8 consecutive values: the products contract over the head dimension in
// whatever order both operands agree on, so values 8t .. 8t + 7 of each 32 serve lane t of a quad in two steps.
#include "internal.h"
#include "score.cuh"
#include "sm100.cuh"

namespace fa {

namespace {

constexpr int kDeltaBand = 48;
constexpr float kDeltaSteep = 0.5f;   // natural units: exp(-0.5 * 17) < 2^-12

// The rows of a sequence see few keys whatever the slope.
__host__ __device__ constexpr bool delta_whole(int Lq, int Lk, int wl, int wr) {
    const int keys = wl >= 0 && wr >= 0 && wl < Lk && wr < Lk - wl ? wl + wr + 1 : Lk;   // that a row can see
    return keys <= 16 || (Lq <= 512 && keys <= 64);
}

struct DeltaParams {
    const __nv_bfloat16 *q, *k, *v, *dout;
    const float* lse2;      // [Hq][Tq]
    float* delta;           // [Hq][Tq]
    const int32_t* cu_q;
    const int32_t* cu_k;
    int Sq, Sk, Tq, Tk, Hq, Hkv, group, blocks, units;
    float scale_log2;
    int wl, wr;             // window sides, -1 = unbounded; a causal mask is wr = 0
    ScoreParams sc;
};

// 16 query rows of a head, and the keys to sum over: lo .. hi of the sequence
struct DeltaUnit {
    int h, q0, q_start, Lq, k_start, Lk, lo, hi;
    float slope;            // log2 units
    bool run, whole;        // whole: the rows see no other keys
};

template <int MODE>
__device__ __forceinline__ DeltaUnit delta_unit(const DeltaParams& p, int u) {
    DeltaUnit t;
    const int b = u / p.blocks / p.Hq;
    t.h = u / p.blocks % p.Hq;
    t.q0 = u % p.blocks * 16;
    t.q_start = b * p.Sq;
    t.k_start = b * p.Sk;
    t.Lq = p.Sq;
    t.Lk = p.Sk;
    if (p.cu_q != nullptr) {
        t.q_start = max(__ldg(p.cu_q + b), 0);
        t.k_start = max(__ldg(p.cu_k + b), 0);
        t.Lq = __ldg(p.cu_q + b + 1) - __ldg(p.cu_q + b);
        t.Lk = __ldg(p.cu_k + b + 1) - __ldg(p.cu_k + b);
        t.Lq = max(min(min(t.Lq, p.Tq - t.q_start), 1 << 30), 0);   // malformed offsets can only shrink the work
        t.Lk = max(min(min(t.Lk, p.Tk - t.k_start), 1 << 30), 0);
    }
    // keys that some row of the block sees
    const int off = t.Lk - t.Lq;
    const int at0 = t.q0 + off, at1 = min(t.q0 + 15, t.Lq - 1) + off;   // places of its rows among the keys
    t.lo = p.wl >= 0 ? max(0, at0 - p.wl) : 0;
    t.hi = p.wr >= 0 ? min(t.Lk - 1, at1 + p.wr) : t.Lk - 1;
    t.slope = (MODE & kScoreBias) ? slope_log2(p.sc, b, t.h) : 0.f;
    t.whole = delta_whole(t.Lq, t.Lk, p.wl, p.wr);
    t.run = t.q0 < t.Lq && (t.whole || fabsf(t.slope) >= kDeltaSteep * 1.4426950408889634f);
    if (!t.whole) {
        // the keys with the largest bias: around the diagonal, or the end that lies farther from it
        int first = min(at0 - (kDeltaBand - 16) / 2, t.hi - kDeltaBand + 1);
        if (t.slope < 0.f) first = at1 - t.lo >= t.hi - at0 ? t.lo : t.hi - kDeltaBand + 1;
        t.lo = max(t.lo, first);
        t.hi = min(t.hi, t.lo + kDeltaBand - 1);
    }
    return t;
}

template <int D, int MODE>
__device__ __forceinline__ void delta_rows(const DeltaParams& p, const DeltaUnit& u) {
    constexpr int KP = D / 32;
    const int lane = threadIdx.x & 31, quad = lane >> 2, t = lane & 3;
    const int off = u.Lk - u.Lq, hk = u.h / p.group;
    const int row[2] = {u.q0 + quad, u.q0 + quad + 8};
    uint4 qf[2][KP], df[2][KP];
    int key_lo[2], key_hi[2];
    float l2[2], acc[2] = {0.f, 0.f}, mass[2] = {0.f, 0.f};
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int in = min(row[r], u.Lq - 1);   // rows past the sequence repeat its last one and are not written
        const size_t at = (static_cast<size_t>(u.q_start + in) * p.Hq + u.h) * D + t * 8;
#pragma unroll
        for (int kp = 0; kp < KP; ++kp) {
            qf[r][kp] = __ldg(reinterpret_cast<const uint4*>(p.q + at + kp * 32));
            df[r][kp] = __ldg(reinterpret_cast<const uint4*>(p.dout + at + kp * 32));
        }
        l2[r] = p.lse2[static_cast<size_t>(u.h) * p.Tq + u.q_start + in];
        key_lo[r] = max(u.lo, p.wl >= 0 ? in + off - p.wl : 0);
        key_hi[r] = min(u.hi, p.wr >= 0 ? in + off + p.wr : u.hi);
    }
#pragma unroll 1
    for (int kn = u.lo / 8 * 8; kn <= u.hi; kn += 8) {
        const size_t at = (static_cast<size_t>(u.k_start + min(kn + quad, u.Lk - 1)) * p.Hkv + hk) * D + t * 8;
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
            if constexpr ((MODE & kScoreBias) != 0) x += bias_log2(static_cast<float>(row[r] + off - key), u.slope);
            // masked keys may hold anything
            const bool keep = key >= key_lo[r] && key <= key_hi[r];
            const float pr = keep ? ex2_approx(x - l2[r]) : 0.f;
            acc[r] += keep ? pr * dp[e] : 0.f;
            mass[r] += pr;
        }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        acc[r] += __shfl_xor_sync(0xffffffffu, acc[r], 1);
        acc[r] += __shfl_xor_sync(0xffffffffu, acc[r], 2);
        mass[r] += __shfl_xor_sync(0xffffffffu, mass[r], 1);
        mass[r] += __shfl_xor_sync(0xffffffffu, mass[r], 2);
        if (t == 0 && row[r] < u.Lq && (u.whole || mass[r] >= 1.f - 0x1p-12f))
            p.delta[static_cast<size_t>(u.h) * p.Tq + u.q_start + row[r]] = acc[r];
    }
}

template <int D, int MODE>
__global__ void __launch_bounds__(128) bwd_delta_kernel(const __grid_constant__ DeltaParams p) {
    const int lane = threadIdx.x & 31;
    const int warps = gridDim.x * 4, first = blockIdx.x * 4 + (threadIdx.x >> 5);
    // launched with programmatic serialization: LSE2 and the Delta that this replaces are settled after the wait
    grid_dep_wait();
    grid_dep_launch();
    for (long long u0 = first; u0 < p.units; u0 += 32LL * warps) {
        const long long mine = u0 + static_cast<long long>(lane) * warps;
        const bool run = mine < p.units && delta_unit<MODE>(p, static_cast<int>(mine)).run;
        for (unsigned todo = __ballot_sync(0xffffffffu, run); todo != 0; todo &= todo - 1)
            delta_rows<D, MODE>(p, delta_unit<MODE>(p, static_cast<int>(u0 + static_cast<long long>(__ffs(todo) - 1) * warps)));
    }
}

}  // namespace

int launch_bwd_delta(const Problem& pr, const void* dout, const float* lse2, float* delta, const Device& dev,
                     cudaStream_t stream) {
    const int mode = score_mode(pr.softcap, pr.slopes);
    if (mode == kScorePlain) return 0;
    DeltaParams p;
    p.blocks = (pr.Sq + 15) / 16;
    if (pr.cu_q == nullptr && !(mode & kScoreBias) && !delta_whole(pr.Sq, pr.Sk, pr.wl, pr.wr)) return 0;
    const long long units = static_cast<long long>(p.blocks) * pr.Hq * pr.num_seqs;
    if (units > 0x7fffffffLL) return 0;   // some 10^10 rows
    p.units = static_cast<int>(units);
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
            auto launch = [&](auto kern) {
                const long long blocks = (units + 3) / 4, most = 16LL * dev.num_sms;
                return launch_dependent(kern, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), dim3(128), 0, stream,
                                        p) == cudaSuccess ? 0 : 5;
            };
            switch (pr.D) {
                case 64: return launch(bwd_delta_kernel<64, MODE>);
                case 128: return launch(bwd_delta_kernel<128, MODE>);
                case 256: return launch(bwd_delta_kernel<256, MODE>);
                default: return 2;
            }
        }
        return 0;
    };
    return with_score_mode(pr.softcap, pr.slopes, run);
}

}  // namespace fa
