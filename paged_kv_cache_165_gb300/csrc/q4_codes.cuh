// q4_codes.cuh -- the 4-bit cache format, shared by every kernel that writes or reads it (not
// part of the ABI).
//
// A row of d elements is held as 4-bit codes in groups of `group` elements (32, 64 or 128),
// each group with an fp16 scale and an fp16 zero: value = zero + scale * code (the low-bit
// cache trade-off of zwjcode.cn "KV Cache 的增量解码" §14).  The page of one (block, KV head)
// is bs * (d/2 + 4*G) contiguous bytes, G = d / group: the codes [bs][d/2] (byte j: element
// 2j in the low nibble, 2j+1 in the high one), then the parameters [bs][G] as (scale, zero)
// pairs.  One contiguous run, so a page is a single bulk copy.
//
// Quantising a group x_0 .. x_{n-1}, each clamped to +-65504 (fp16's range):
//   zero = fp16(min x) rounded towards -inf, so that no element lies below it,
//   scale = fp16((max x - zero) / 15) rounded to nearest,
//   code = clamp(round half to even((x - zero) / scale), 0, 15), 0 where scale is 0,
// every quotient exact before its one rounding.  The kernels compute in fp32, whose error
// could move a quotient across a rounding boundary: a quotient closer to a boundary than
// that error is decided in fp64, where the comparison is exact (fp64 is slow on this part,
// and about one element in 10^5 gets there).  A group that holds a NaN stores zero = NaN,
// scale 0 and codes 0, so every value read back from it is NaN.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

namespace pkv {

constexpr float kQ4Max = 65504.f;   // fp16's largest finite value

__host__ __device__ constexpr int q4_row_bytes(int d, int group) { return d / 2 + 4 * (d / group); }

// Scale of a group: fp16 nearest to (hi - zero) / 15.  The fp32 quotient is within 2^-22 of
// the exact one; unless both ends of that interval round to the same fp16 the exact quotient
// is compared with the value halfway between the two candidates.
__device__ __forceinline__ __half q4_scale(float hi, __half zero) {
    const float z = __half2float(zero);
    const float r = (hi - z) * (1.f / 15.f);
    const __half a = __float2half_rn(r * (1.f - 0x1p-21f)), b = __float2half_rn(r * (1.f + 0x1p-21f));
    if (__half_as_ushort(a) == __half_as_ushort(b)) return a;
    const double exact = static_cast<double>(hi) - static_cast<double>(z);   // 24- and 11-bit terms
    const double mid = 0.5 * (static_cast<double>(__half2float(a)) + static_cast<double>(__half2float(b)));
    const double cut = 15.0 * mid;
    if (exact != cut) return exact < cut ? a : b;
    return (__half_as_ushort(a) & 1) == 0 ? a : b;
}

// Code of x (already clamped, x >= zero) for scale s > 0 with inv = 1 / s in fp32.
__device__ __forceinline__ uint32_t q4_code(float x, float z, float s, float inv) {
    const float t = (x - z) * inv;
    float k = rintf(t);
    if (fabsf(t - k) > 0.5f - 1e-5f) {   // fp32 may be on the wrong side of k +- 1/2
        const float lo = floorf(t);
        const double edge = (static_cast<double>(lo) + 0.5) * static_cast<double>(s);   // exact
        const double dx = static_cast<double>(x) - static_cast<double>(z);
        if (dx != edge) k = dx > edge ? lo + 1.f : lo;
        else k = (static_cast<int>(lo) & 1) ? lo + 1.f : lo;
    }
    return static_cast<uint32_t>(fminf(fmaxf(k, 0.f), 15.f));
}

// Eight consecutive elements of a group spread over `lanes` consecutive lanes of the warp
// (4, 8 or 16: group / 8), every lane of the warp taking part.  Returns the lane's eight codes
// (element i in bits 4i .. 4i+3) and the group's (scale, zero).
__device__ __forceinline__ uint32_t q4_quantise8(const float (&in)[8], int lanes, __half2 &par) {
    float x[8];
    float lo = INFINITY, hi = -INFINITY;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        nan |= in[i] != in[i];
        x[i] = fminf(fmaxf(in[i], -kQ4Max), kQ4Max);
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
    }
    if (nan) lo = -INFINITY;   // below every clamped value: marks the group
    for (int sh = lanes >> 1; sh > 0; sh >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, sh));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, sh));
    }
    if (lo == -INFINITY) {
        par = __halves2half2(__ushort_as_half(0), __ushort_as_half(0x7fff));
        return 0;
    }
    const __half zero = __float2half_rd(lo);
    const __half scale = q4_scale(hi, zero);
    par = __halves2half2(scale, zero);
    const float s = __half2float(scale), z = __half2float(zero);
    if (!(s > 0.f)) return 0;
    const float inv = 1.f / s;
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) w |= q4_code(x[i], z, s, inv) << (4 * i);
    return w;
}

template <typename T>
__device__ __forceinline__ float q4_in(T x);
template <>
__device__ __forceinline__ float q4_in<float>(float x) { return x; }
template <>
__device__ __forceinline__ float q4_in<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

// Eight elements from p (16-byte loads where the caller has checked the alignment).
template <typename T, bool VEC>
__device__ __forceinline__ void q4_load8(const T *p, float (&x)[8]) {
    if constexpr (VEC && sizeof(T) == 2) {
        const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // a bf16 is the top half of an fp32
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else if constexpr (VEC) {
        const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = q4_in(p[i]);
    }
}

}  // namespace pkv
