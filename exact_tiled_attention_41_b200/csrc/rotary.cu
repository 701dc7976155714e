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
    int inverse, copy_rest;
    int* status;
};

// The sequence of token `tok` of a packed batch: the last b with cu[b] <= tok (-1 before the first).
__device__ __forceinline__ int find_seq(const int32_t* cu, int n, long long tok) {
    int lo = -1, hi = n + 1;   // cu[lo] <= tok < cu[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(cu + mid) <= tok) lo = mid;
        else hi = mid;
    }
    return lo;
}

// One warp per token and block of heads; a lane takes one piece (or, for halves, the two pieces of 8 pairs).
template <int D, bool INTER>
__global__ void __launch_bounds__(256) rotary_kernel(const __grid_constant__ RotaryParams p) {
    const int lane = threadIdx.x & 31;
    const long long tok = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (tok >= p.tokens) return;
    long long xt, yt;
    long long pos;
    int b;
    if (p.cu != nullptr) {
        b = find_seq(p.cu, p.num_seqs, tok);
        if (b < 0 || b >= p.num_seqs) return;   // behind the last sequence: left as it was
        pos = tok - __ldg(p.cu + b);
        xt = tok * p.x_sT;
        yt = tok * p.y_sT;
    } else {
        b = static_cast<int>(tok / p.S);
        pos = tok % p.S;
        xt = b * p.x_sB + pos * p.x_sT;
        yt = b * p.y_sB + pos * p.y_sT;
    }
    pos += p.offsets != nullptr ? __ldg(p.offsets + b) : p.offset;
    const bool bad = pos < 0 || pos >= p.rows;
    if (bad && lane == 0) atomicCAS(p.status, 0, FA_ERR_INVALID_ARG);
    const int half = p.rd / 2;
    const float* cr = p.cos + static_cast<size_t>(bad ? 0 : pos) * half;
    const float* sr = p.sin + static_cast<size_t>(bad ? 0 : pos) * half;
    const float sign = p.inverse ? -1.f : 1.f;
    constexpr int PIECES = D / 8;
    for (int idx = lane; idx < p.H * PIECES; idx += 32) {
        const int h = idx / PIECES, d = (idx % PIECES) * 8;
        const __nv_bfloat16* xr = p.x + xt + h * p.x_sH;
        __nv_bfloat16* yr = p.y + yt + h * p.y_sH;
        if (d >= p.rd) {
            if (p.copy_rest) *reinterpret_cast<uint4*>(yr + d) = *reinterpret_cast<const uint4*>(xr + d);
            continue;
        }
        if (bad) {
            *reinterpret_cast<uint4*>(yr + d) = make_uint4(0, 0, 0, 0);
            continue;
        }
        if constexpr (INTER) {
            float4 c = __ldg(reinterpret_cast<const float4*>(cr + d / 2));
            float4 s = __ldg(reinterpret_cast<const float4*>(sr + d / 2));
            s = make_float4(s.x * sign, s.y * sign, s.z * sign, s.w * sign);
            *reinterpret_cast<uint4*>(yr + d) = rot_interleaved(*reinterpret_cast<const uint4*>(xr + d), c, s);
        } else if (d < half) {
            float c[8], s[8];
            load8(cr + d, c);
            load8(sr + d, s);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] *= sign;
            uint4 u = *reinterpret_cast<const uint4*>(xr + d), v = *reinterpret_cast<const uint4*>(xr + d + half);
            rot_halves(u, v, c, s);
            *reinterpret_cast<uint4*>(yr + d) = u;
            *reinterpret_cast<uint4*>(yr + d + half) = v;
        }
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
    p.copy_rest = c.x != c.y;
    p.status = dev.status;
    const long long blocks = (p.tokens + 7) / 8;
    if (blocks > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
    auto run = [&](auto kern) { kern<<<static_cast<unsigned>(blocks), 256, 0, stream>>>(p); };
    switch (c.D) {
        case 64: c.interleaved ? run(rotary_kernel<64, true>) : run(rotary_kernel<64, false>); break;
        case 128: c.interleaved ? run(rotary_kernel<128, true>) : run(rotary_kernel<128, false>); break;
        case 256: c.interleaved ? run(rotary_kernel<256, true>) : run(rotary_kernel<256, false>); break;
        default: return FA_ERR_UNSUPPORTED;
    }
    return cudaPeekAtLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// ------------------------------------------------------------------------------------------ tables
// The angle of row `pos` and pair i is pos * f_i.  An fp32 product would be off by pos * f * 2^-24 radians
// (0.008 at position 131072), so the angle is formed in turns as an integer: turn_i = f_i / 2 pi as a 64-bit
// fraction, and pos * turn_i modulo 2^64 is the fraction of a turn, off by at most pos * 2^-53 turns (f_i is
// a double).  Its upper 32 bits as a signed number are the angle in half turns times 2^31; sincospif does the rest.
struct TableParams {
    uint64_t turn[128];   // rd / 2 <= 128 pairs
    float* cos;
    float* sin;
    int rows, half;
    float amplitude;
};

__global__ void __launch_bounds__(256) rotary_table_kernel(const __grid_constant__ TableParams p) {
    const long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= static_cast<long long>(p.rows) * p.half) return;
    const unsigned pos = static_cast<unsigned>(i / p.half);
    const int k = static_cast<int>(i % p.half);
    const uint64_t frac = pos * p.turn[k];
    const float x = static_cast<float>(static_cast<int32_t>(frac >> 32)) * 4.656612873077393e-10f;   // 2^-31
    float s, c;
    sincospif(x, &s, &c);
    p.cos[i] = c * p.amplitude;
    p.sin[i] = s * p.amplitude;
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
    const long long n = static_cast<long long>(rows) * p.half;
    rotary_table_kernel<<<static_cast<unsigned>((n + 255) / 256), 256, 0, stream>>>(p);
    return cudaPeekAtLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace fa
