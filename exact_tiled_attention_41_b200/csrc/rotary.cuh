// rotary.cuh -- rotary position embedding of one 16-byte piece (8 values) of a head, shared by the
// stand-alone kernel (rotary.cu) and the cache call (decode.cu), so that both give the same bits.
//
// The first rd of a head's D values are rotated, in pairs (2i, 2i + 1) (interleaved) or (i, i + rd / 2)
// (halves), by the angle whose cosine and sine stand in row `position` of the [seqlen_ro][rd / 2] tables
// (flash-attention README, flash_attn_with_kvcache docstring):
//     y_a = x_a c - x_b s,     y_b = x_b c + x_a s.
// The gradient is the rotation by the opposite angle.  rd is a multiple of 16, so a piece lies on one side of
// every boundary (halves: rd / 2 is a multiple of 8).  fp32 arithmetic, one rounding to bf16.
#pragma once

#include "sm100.cuh"

namespace fa {

// the two values of a pair; sn is negated by the caller for the opposite rotation
__device__ __forceinline__ float rot_first(float a, float b, float c, float sn) { return __fmaf_rn(-b, sn, __fmul_rn(a, c)); }
__device__ __forceinline__ float rot_second(float a, float b, float c, float sn) { return __fmaf_rn(a, sn, __fmul_rn(b, c)); }

__device__ __forceinline__ float2 unpack_bf16x2(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// interleaved pairs: piece x at value d, cosines and sines of pairs d / 2 .. d / 2 + 3
__device__ __forceinline__ uint4 rot_interleaved(uint4 x, float4 c, float4 s) {
    auto pair = [](uint32_t w, float cc, float ss) {
        const float2 v = unpack_bf16x2(w);
        return pack_bf16x2(rot_first(v.x, v.y, cc, ss), rot_second(v.x, v.y, cc, ss));
    };
    return make_uint4(pair(x.x, c.x, s.x), pair(x.y, c.y, s.y), pair(x.z, c.z, s.z), pair(x.w, c.w, s.w));
}

// halves: piece a at value d < rd / 2 and b at d + rd / 2 with the cosines and sines of pairs d .. d + 7;
// y_a and y_b replace them
__device__ __forceinline__ void rot_halves(uint4& a, uint4& b, const float (&c)[8], const float (&s)[8]) {
    uint32_t* wa = reinterpret_cast<uint32_t*>(&a);
    uint32_t* wb = reinterpret_cast<uint32_t*>(&b);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 u = unpack_bf16x2(wa[e]), v = unpack_bf16x2(wb[e]);
        wa[e] = pack_bf16x2(rot_first(u.x, v.x, c[2 * e], s[2 * e]), rot_first(u.y, v.y, c[2 * e + 1], s[2 * e + 1]));
        wb[e] = pack_bf16x2(rot_second(u.x, v.x, c[2 * e], s[2 * e]), rot_second(u.y, v.y, c[2 * e + 1], s[2 * e + 1]));
    }
}

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    *reinterpret_cast<float4*>(v) = __ldg(reinterpret_cast<const float4*>(p));
    *reinterpret_cast<float4*>(v + 4) = __ldg(reinterpret_cast<const float4*>(p) + 1);
}

}  // namespace fa
