// rotary.cu -- rotary positions applied to queries or keys (and, with `inverse`, to their gradients), and the
// cosine / sine tables of those positions, scaled for long contexts.  See rotary.cuh for the rotation.
#include "../../include/fa.h"
#include "internal.h"
#include "rotary.cuh"

#include <math.h>

namespace fa {

struct RotaryParams {
    const __nv_bfloat16* x;
    __nv_bfloat16* y;
    const float* cos;
    const float* sin;
    const int32_t* cu;        // [num_seqs + 1], or NULL: equal lengths S
    const int32_t* offsets;   // first position of each sequence, or NULL: `offset` for all
    int offset;
    int num_seqs, S, H, rd, rows;   // rows of the tables
    long long tokens;
    long long x_sB, x_sT, x_sH, y_sB, y_sT, y_sH;   // strides in values; sB unused with cu
    int inverse;
    int zero_tail;            // rows of y outside every sequence of a packed batch: zeros, or left as they were
    int items;                // threads per row: pieces (interleaved) or pairs of pieces (halves), and copied pieces
    int* status;
};

// The sequence of token `tok` of a packed batch: the last b with cu[b] <= tok, -1 before the first; the whole warp
// searches together, 32 entries at a time.
__device__ __forceinline__ int find_seq(const int32_t* cu, int n, long long tok) {
    const int lane = threadIdx.x & 31;
    int lo = 0, len = n + 1;
    for (;;) {
        const int step = (len + 31) / 32;
        const bool below = lane * step < len && __ldg(cu + lo + lane * step) <= tok;
        const int count = __popc(__ballot_sync(0xffffffffu, below));
        if (count == 0) return -1;
        lo += (count - 1) * step;
        len = min(step, len - (count - 1) * step);
        if (step == 1) return lo;
    }
}

// n / d with a 32-bit division where n allows it: a 64-bit one takes as many instructions as the rest of a row
__device__ __forceinline__ long long div_small(long long n, int d) {
    if (n <= 0xffffffffLL) return static_cast<unsigned>(n) / static_cast<unsigned>(d);
    return n / d;
}

// A row is one head of one token.  p.items threads share a row: a thread takes the 16-byte piece of four
// interleaved pairs, the two pieces of eight pairs of halves, or a piece that is only copied.  A block takes
// consecutive rows (token by token, head by head), kRotRows of them per thread, whose loads are all in flight before
// the first store: bound by HBM, it needs about 35 KB in flight per SM.  The cosines and sines of a
// token are read once per head from L1 / L2, which is a third of the wavefronts and no HBM traffic.
// B200, 8192 tokens x 32 heads x 128 (134 MB): 23.5 us, 5.7 TB/s, 87 % of the copy rate; 1 row a thread 27 us, 4 rows
// 30, 256 threads 25, streaming loads and stores 24.
constexpr int kRotThreads = 128;
constexpr int kRotRows = 2;

template <bool INTER>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const __grid_constant__ RotaryParams p) {
    const int slots = kRotThreads / p.items;            // rows side by side
    const int slot = threadIdx.x / p.items, item = threadIdx.x % p.items;
    const long long row0 = static_cast<long long>(blockIdx.x) * (slots * kRotRows);
    const long long tok0 = div_small(row0, p.H);
    const int h0 = static_cast<int>(row0 - tok0 * p.H);
    const int half = p.rd / 2;
    const int turned = INTER ? p.rd / 8 : p.rd / 16;    // items of a row that rotate
    const bool turn = item < turned;
    const int d = turn ? item * 8 : p.rd + (item - turned) * 8;
    const int ci = INTER ? d / 2 : d;                   // column of the tables
    // the sequence and place of the block's first token; a row's own is at most a few further on
    int b0 = 0;
    long long pos0 = tok0;
    if (p.cu != nullptr) {
        b0 = find_seq(p.cu, p.num_seqs, tok0);
    } else {
        b0 = static_cast<int>(div_small(tok0, p.S));
        pos0 = tok0 - static_cast<long long>(b0) * p.S;
    }

    uint4 u[kRotRows], v[kRotRows];
    const float *cr[kRotRows], *sr[kRotRows];
    __nv_bfloat16* y[kRotRows];
    bool live[kRotRows], bad[kRotRows];
#pragma unroll
    for (int k = 0; k < kRotRows; ++k) {
        const int r = h0 + slot + k * slots;
        const int dt = r / p.H, h = r - dt * p.H;
        const long long tok = tok0 + dt;
        live[k] = slot < slots && tok < p.tokens;
        bad[k] = false;
        if (!live[k]) continue;
        int b;
        long long pos, xo, yo;
        if (p.cu != nullptr) {
            b = b0;
            while (b < p.num_seqs && __ldg(p.cu + b + 1) <= tok) ++b;
            if (b < 0 || b >= p.num_seqs) {              // outside every sequence
                live[k] = false;
                if (p.zero_tail) {
                    __nv_bfloat16* z = p.y + tok * p.y_sT + h * p.y_sH + d;
                    *reinterpret_cast<uint4*>(z) = make_uint4(0, 0, 0, 0);
                    if (!INTER && turn) *reinterpret_cast<uint4*>(z + half) = make_uint4(0, 0, 0, 0);
                }
                continue;
            }
            pos = tok - __ldg(p.cu + b);
            xo = tok * p.x_sT;
            yo = tok * p.y_sT;
        } else {
            b = b0;
            pos = pos0 + dt;
            if (pos >= p.S) {
                const unsigned k_seqs = static_cast<unsigned>(pos) / static_cast<unsigned>(p.S);   // pos < 2^30 + 512
                b += k_seqs;
                pos -= static_cast<long long>(k_seqs) * p.S;
            }
            xo = b * p.x_sB + pos * p.x_sT;
            yo = b * p.y_sB + pos * p.y_sT;
        }
        pos += p.offsets != nullptr ? __ldg(p.offsets + b) : p.offset;
        bad[k] = pos < 0 || pos >= p.rows;
        const size_t t = static_cast<size_t>(bad[k] ? 0 : pos) * half + ci;
        cr[k] = p.cos + t;
        sr[k] = p.sin + t;
        const __nv_bfloat16* x = p.x + xo + h * p.x_sH + d;
        y[k] = p.y + yo + h * p.y_sH + d;
        u[k] = *reinterpret_cast<const uint4*>(x);
        if (!INTER && turn) v[k] = *reinterpret_cast<const uint4*>(x + half);
    }
    const float sign = p.inverse ? -1.f : 1.f;
#pragma unroll
    for (int k = 0; k < kRotRows; ++k) {
        if (!live[k]) continue;
        if (turn) {
            if (bad[k]) {
                if (item == 0) atomicCAS(p.status, 0, FA_ERR_INVALID_ARG);
                u[k] = v[k] = make_uint4(0, 0, 0, 0);
            } else if constexpr (INTER) {
                const float4 c = __ldg(reinterpret_cast<const float4*>(cr[k]));
                const float4 s = __ldg(reinterpret_cast<const float4*>(sr[k]));
                u[k] = rot_interleaved(u[k], c, make_float4(s.x * sign, s.y * sign, s.z * sign, s.w * sign));
            } else {
                float c[8], s[8];
                load8(cr[k], c);
                load8(sr[k], s);
#pragma unroll
                for (int e = 0; e < 8; ++e) s[e] *= sign;
                rot_halves(u[k], v[k], c, s);
            }
            if (!INTER) *reinterpret_cast<uint4*>(y[k] + half) = v[k];
        }
        *reinterpret_cast<uint4*>(y[k]) = u[k];
    }
}

int launch_rotary(const RotaryCall& c, const Device& dev, cudaStream_t stream) {
    RotaryParams p;
    p.x = static_cast<const __nv_bfloat16*>(c.x);
    p.y = static_cast<__nv_bfloat16*>(c.y);
    p.cos = c.cos;
    p.sin = c.sin;
    p.cu = c.cu_seqlens;
    p.offsets = c.offsets;
    p.offset = c.offset;
    p.num_seqs = c.num_seqs;
    p.S = c.S;
    p.H = c.H;
    p.rd = c.rotary_dim;
    p.rows = c.seqlen_ro;
    p.tokens = c.tokens;
    p.x_sB = c.x_stride[0];
    p.x_sT = c.x_stride[1];
    p.x_sH = c.x_stride[2];
    p.y_sB = c.y_stride[0];
    p.y_sT = c.y_stride[1];
    p.y_sH = c.y_stride[2];
    p.inverse = c.inverse;
    p.zero_tail = c.zero_tail;
    p.items = (c.interleaved ? c.rotary_dim / 8 : c.rotary_dim / 16) + (c.x != c.y ? (c.D - c.rotary_dim) / 8 : 0);
    p.status = dev.status;
    const long long per_block = kRotThreads / p.items * kRotRows;
    const long long blocks = (p.tokens * p.H + per_block - 1) / per_block;
    if (blocks > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
    if (c.interleaved) {
        rotary_kernel<true><<<static_cast<unsigned>(blocks), kRotThreads, 0, stream>>>(p);
    } else {
        rotary_kernel<false><<<static_cast<unsigned>(blocks), kRotThreads, 0, stream>>>(p);
    }
    return cudaPeekAtLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// ------------------------------------------------------------------------------------------ tables
// The angle of row `pos` and pair i is pos * f_i.  An fp32 product would be off by pos * f * 2^-24 radians
// (0.008 at position 131072), so the angle is formed in turns as an integer: turn_i = f_i / 2 pi as a 64-bit
// fraction, and pos * turn_i modulo 2^64 is the fraction of a turn, off by at most pos * 2^-53 turns (f_i is
// a double): 1e-15 radians a position.  Its upper bits give the nearest quarter turn, and what is left, as a signed number
// of all 64 bits, is an angle y within pi / 4 (slow pairs turn little at small positions, and their sines keep their
// relative accuracy), whose sine and cosine are polynomials in y^2 (of the smallest maximum relative error;
// exact_tiled_attention_41_b200/fit_trig_poly.py prints the coefficients).
struct TableParams {
    uint64_t turn[128];   // rd / 2 <= 128 pairs
    float* cos;
    float* sin;
    int rows, half;
    float amplitude;
};

// sine and cosine of a fraction of a turn, in units of 2^-64
__device__ __forceinline__ void sin_cos_turn(uint64_t frac, float& sn, float& cs) {
    const uint32_t quarter = (static_cast<uint32_t>(frac >> 32) + 0x20000000u) >> 30;
    const int64_t left = static_cast<int64_t>(frac - (static_cast<uint64_t>(quarter) << 62));
    const float y = static_cast<float>(left) * 3.4061215800865545e-19f;   // 2 pi 2^-64
    const float u = y * y;
    float s = fmaf(-0.00019501822f, u, 0.00833201688f);
    s = fmaf(s, u, -0.166666508f);
    s = fmaf(s, u, 1.0f) * y;
    float c = fmaf(2.4372679e-05f, u, -0.00138865295f);
    c = fmaf(c, u, 0.041666612f);
    c = fmaf(c, u, -0.5f);
    c = fmaf(c, u, 1.0f);
    // a quarter turn takes (cos, sin) to (-sin, cos)
    const bool odd = quarter & 1;
    sn = __uint_as_float(__float_as_uint(odd ? c : s) ^ ((quarter & 2) << 30));
    cs = __uint_as_float(__float_as_uint(odd ? s : c) ^ (((quarter + 1) & 2) << 30));
}

// A thread owns four neighbouring pairs of a column block and walks down the rows: one 16-byte store to each table
// per row, and the angles advance by an addition.  Written once, nothing read: bound by the stores, or by issue
// slots (51 % busy).  B200, 131072 x 64 pairs (67 MB): 12 us; 4 or 16 rows a thread 16 and 15 us.
constexpr int kTableRows = 8;   // rows per thread

__global__ void __launch_bounds__(256) rotary_table_kernel(const __grid_constant__ TableParams p) {
    const int groups = p.half >> 2;                    // rotary_dim % 16 == 0: half is a multiple of 8
    const int per_block = 256 / groups;                // rows side by side in a block
    const int r = threadIdx.x / groups, k = (threadIdx.x % groups) * 4;
    if (r >= per_block) return;
    long long pos = static_cast<long long>(blockIdx.x) * per_block * kTableRows + r;
    uint64_t frac[4], step[4];   // fraction of a turn at pos, and from one row of the thread to its next
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        frac[e] = static_cast<uint32_t>(pos) * p.turn[k + e];
        step[e] = static_cast<uint32_t>(per_block) * p.turn[k + e];
    }
#pragma unroll
    for (int i = 0; i < kTableRows; ++i, pos += per_block) {
        if (pos >= p.rows) return;
        float s[4], c[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            sin_cos_turn(frac[e], s[e], c[e]);
            frac[e] += step[e];
        }
        const float a = p.amplitude;
        *reinterpret_cast<float4*>(p.cos + pos * p.half + k) = make_float4(c[0] * a, c[1] * a, c[2] * a, c[3] * a);
        *reinterpret_cast<float4*>(p.sin + pos * p.half + k) = make_float4(s[0] * a, s[1] * a, s[2] * a, s[3] * a);
    }
}

int launch_rotary_table(float* cos, float* sin, int rows, int rotary_dim, const double* freq, float amplitude,
                        cudaStream_t stream) {
    TableParams p;
    p.cos = cos;
    p.sin = sin;
    p.rows = rows;
    p.half = rotary_dim / 2;
    p.amplitude = amplitude;
    for (int i = 0; i < p.half; ++i) {
        const double t = freq[i] * 0.15915494309189533577;            // turns per position
        p.turn[i] = static_cast<uint64_t>(llrint(ldexp(t - rint(t), 63))) << 1;   // modulo one turn
    }
    const int rows_per_block = 256 / (p.half / 4) * kTableRows;
    rotary_table_kernel<<<(rows + rows_per_block - 1) / rows_per_block, 256, 0, stream>>>(p);
    return cudaPeekAtLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace fa
