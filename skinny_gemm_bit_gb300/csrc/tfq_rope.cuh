// What the kernels of norm, rotation and store share: their parameters, the angles, and the launch into a cache of 8 bits.
#pragma once

#include "tfq_cache.h"
#include "tfq_ptx.cuh"

namespace tfq {

struct RopeParams {
    const uint16_t* qkv;
    int64_t ld, M;
    int n_q;
    const uint16_t *q_gamma, *k_gamma;
    float eps;
    const int32_t* positions;
    const uint64_t* turns;
    int rot16;  // rot_dim / 16: lanes of a head whose chunks are rotated
    int interleaved;
    uint16_t* q;
    CacheView c;
    int layer;
    const int32_t* slots;
    int* status;
    int parts;  // warps (8 bits: CTAs) that share a row's heads
    int step;   // 8 bits: a CTA's rows begin at or behind every step-th
};

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8])
{
    f[0] = bf16lo_f32(v.x), f[1] = bf16hi_f32(v.x), f[2] = bf16lo_f32(v.y), f[3] = bf16hi_f32(v.y);
    f[4] = bf16lo_f32(v.z), f[5] = bf16hi_f32(v.z), f[6] = bf16lo_f32(v.w), f[7] = bf16hi_f32(v.w);
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8])
{
    return make_uint4(f32x2_to_bf16x2(f[0], f[1]), f32x2_to_bf16x2(f[2], f[3]), f32x2_to_bf16x2(f[4], f[5]),
                      f32x2_to_bf16x2(f[6], f[7]));
}

// Sine and cosine of hi + lo / 2^32 units of 2^-32 turn: less the nearest quarter turn, exactly, x is within
// [-pi / 4, pi / 4] and as near as fp32 has it however small it is; there the Taylor polynomials' own error is
// x^8 / 9! and x^10 / 10! at most (2^-21, 2^-25), so both are within 2^-20 of their own values at every angle.
__device__ __forceinline__ void turn_sincos(uint32_t hi, uint32_t lo, float& sn, float& cs)
{
    const uint32_t quarter = (hi + 0x20000000u) >> 30;
    const float x = fmaf((float)lo, 0x1p-32f, (float)(int32_t)(hi - (quarter << 30))) * 1.4629180792671596e-9f;  // 2 pi / 2^32
    const float y = x * x;
    const float s = fmaf(x * y, fmaf(y, fmaf(y, -1.f / 5040.f, 1.f / 120.f), -1.f / 6.f), x);
    const float c = fmaf(y, fmaf(y, fmaf(y, fmaf(y, 1.f / 40320.f, -1.f / 720.f), 1.f / 24.f), -0.5f), 1.f);
    const bool odd = quarter & 1;
    sn = __uint_as_float(__float_as_uint(odd ? c : s) ^ (quarter & 2) << 30);
    cs = __uint_as_float(__float_as_uint(odd ? s : c) ^ (quarter + 1 & 2) << 30);
}

// tfq_rope8.cu: the same pass with keys and values stored as e4m3 codes
cudaError_t launch_rope8(const RopeParams& p, bool pdl, cudaStream_t stream);

}  // namespace tfq
