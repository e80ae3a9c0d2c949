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
// every quotient exact before its one rounding.  The kernels compute in fp32: with d = x - zero
// exact and the quotient t = d / scale correctly rounded (a reciprocal and a quotient refined by
// their exact remainders, after Markstein), t is k + 1/2 only where the exact quotient is, and
// never on the other side of it: the boundary p = (k + 1/2) scale has 16 bits, d != p differ by
// at least d's last place, and that is more than half of t's last place away from k + 1/2.  Where
// d is not exact its error decides a t of k + 1/2 (bf16 rows sit on a lattice: ties are common,
// about one element in a thousand).  A group that holds a NaN stores zero = NaN, scale 0 and
// codes 0, so every value read back from it is NaN.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "common.cuh"

namespace pkv {

constexpr float kQ4Max = 65504.f;   // fp16's largest finite value

__host__ __device__ constexpr int q4_row_bytes(int d, int group) { return d / 2 + 4 * (d / group); }

// The sign of (x - z) - c for c near x - z, c a number of at most 16 bits, exactly: the difference d
// of x and z in fp32 and its error e (Knuth's two-sum); d - c is exact (c is within a factor of two
// of d) and, when it is not 0, a multiple of d's last place, which |e| stays below.
__device__ __forceinline__ float q4_side(float x, float z, float c) {
    const float d = x - z, y = d - x;
    const float r = d - c;
    return r != 0.f ? r : (x - (d - y)) + (-z - y);
}

// Scale of a group: fp16 nearest to (hi - zero) / 15.  The fp32 quotient is within 2^-22 of
// the exact one; unless both ends of a wider interval round to the same fp16 the exact quotient
// is compared with the value halfway between the two candidates.
__device__ __forceinline__ __half q4_scale(float hi, __half zero) {
    const float z = __half2float(zero), r = (hi - z) * (1.f / 15.f);
    __half a = __float2half_rn(r * (1.f - 0x1p-21f));
    const __half b = __float2half_rn(r * (1.f + 0x1p-21f));
    if (__half_as_ushort(a) != __half_as_ushort(b)) {
        const float side = q4_side(hi, z, 7.5f * (__half2float(a) + __half2float(b)));
        if (side > 0.f || (side == 0.f && (__half_as_ushort(a) & 1))) a = b;
    }
    return a;
}

__device__ __forceinline__ float q4_min_nan(float a, float b) {   // NaN if either is
    float d;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// The least and the largest of a group spread over LANES consecutive lanes, each with N elements; lo is
// NaN if an element is.
template <int LANES, int N>
__device__ __forceinline__ void q4_extremes(const float (&x)[N], float &lo, float &hi) {
    lo = hi = x[0];
#pragma unroll
    for (int i = 1; i < N; ++i) {
        lo = q4_min_nan(lo, x[i]);
        hi = fmaxf(hi, x[i]);
    }
#pragma unroll
    for (int sh = LANES / 2; sh > 0; sh >>= 1) {
        lo = q4_min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, sh));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, sh));
    }
}
// The same of bf16 elements, two to a word: pairs at a time, then (lo, -hi) in one word.
template <int LANES, int N>
__device__ __forceinline__ void q4_extremes(const uint32_t (&w)[N], float &lo, float &hi) {
    auto bf = [](uint32_t u) { return *reinterpret_cast<const __nv_bfloat162 *>(&u); };
    auto bits = [](__nv_bfloat162 v) { return *reinterpret_cast<const uint32_t *>(&v); };
    __nv_bfloat162 l = bf(w[0]), h = l;
#pragma unroll
    for (int i = 1; i < N; ++i) {
        l = __hmin2_nan(l, bf(w[i]));
        h = __hmax2_nan(h, bf(w[i]));
    }
    const uint32_t least = bits(l), most = bits(h) ^ 0x80008000u;
    uint32_t m = bits(__hmin2_nan(bf(__byte_perm(least, most, 0x5410)), bf(__byte_perm(least, most, 0x7632))));
#pragma unroll
    for (int sh = LANES / 2; sh > 0; sh >>= 1) m = bits(__hmin2_nan(bf(m), bf(__shfl_xor_sync(0xffffffffu, m, sh))));
    lo = __uint_as_float(m << 16);
    hi = -__uint_as_float(m & 0xffff0000u);
}

// N consecutive elements of a group with extremes lo and hi (BF16: they are bf16 values): their codes
// (element 8 w + i in bits 4i .. 4i+3 of word w) and the group's (scale, zero).  Quotients are rounded by
// adding and taking away 1.5 * 2^23 and packed as fp32 integers, four codes (below 2^16) at a time.
template <bool BF16, int N>
__device__ __forceinline__ void q4_quantise(float (&x)[N], float lo, float hi, __half2 &par, uint32_t (&code)[N / 8]) {
#pragma unroll
    for (int w = 0; w < N / 8; ++w) code[w] = 0;
    if (lo != lo) {
        par = __halves2half2(__ushort_as_half(0), __ushort_as_half(0x7fff));
        return;
    }
    if (lo < -kQ4Max || hi > kQ4Max) {
        lo = fminf(fmaxf(lo, -kQ4Max), kQ4Max);
        hi = fminf(fmaxf(hi, -kQ4Max), kQ4Max);
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = fminf(fmaxf(x[i], -kQ4Max), kQ4Max);
    }
    const __half zero = __float2half_rd(lo);
    const __half scale = q4_scale(hi, zero);
    par = __halves2half2(scale, zero);
    const float s = __half2float(scale), z = __half2float(zero);
    if (!(s > 0.f)) return;
    if (s < 0x1p-14f) {
        // a subnormal scale may be rounded by more than a part in 2^11: quotients can pass 15.5
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = fminf(x[i], fmaf(15.f, s, z));
    }
    float inv;   // 1 / s, correctly rounded: one Newton step from within a last place, checked for all 11-bit s
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    inv = fmaf(inv, fmaf(-s, inv, 1.f), inv);
    constexpr float kMagic = 12582912.f;
    const float2 mz = make_float2(-z, -z), ms = make_float2(-s, -s), i2 = make_float2(inv, inv);
    const float2 up = make_float2(kMagic, kMagic), down = make_float2(-kMagic, -kMagic);
    auto quotient = [&](int i) {   // of elements i and i + 1
        const float2 d = add2(make_float2(x[i], x[i + 1]), mz);   // never below 0
        const float2 q = make_float2(d.x * inv, d.y * inv);
        return fma2(fma2(q, ms, d), i2, q);
    };
    float k[N], worst = 0.f;
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float2 t = quotient(i), r = add2(add2(t, up), down);
        const float2 o = add2(t, make_float2(-r.x, -r.y));
        worst = fmaxf(worst, fmaxf(fabsf(o.x), fabsf(o.y)));
        k[i] = r.x, k[i + 1] = r.y;
    }
    bool inexact = worst == 0.5f;   // a tie in fp32: the error of x - z, where there is one, decides
    if (BF16 && inexact) {
        // 8- and 11-bit terms: exact unless one of them lies far below the difference
        float least = INFINITY;
#pragma unroll
        for (int i = 0; i < N; ++i) least = fminf(least, x[i] != 0.f ? fabsf(x[i]) : INFINITY);
        inexact = least < s * 0x1p-9f || (z != 0.f && fabsf(z) < s * 0x1p-7f);   // differences are below 16 s
    }
    if (inexact) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float2 t = quotient(i & ~1);
            const float off = (i & 1 ? t.y : t.x) - k[i];
            const float d = x[i] - z, y = d - x[i], e = (x[i] - (d - y)) + (-z - y);   // Knuth's two-sum
            if (off == 0.5f && e > 0.f) k[i] += 1.f;       // t = k + 1/2 went down to k
            if (off == -0.5f && e < 0.f) k[i] -= 1.f;      // t = k - 1/2 went up to k
        }
    }
#pragma unroll
    for (int w = 0; w < N; w += 8) {
        const float a = fmaf(fmaf(fmaf(k[w + 3], 16.f, k[w + 2]), 16.f, k[w + 1]), 16.f, k[w]);
        const float b = fmaf(fmaf(fmaf(k[w + 7], 16.f, k[w + 6]), 16.f, k[w + 5]), 16.f, k[w + 4]);
        // the integers below 2^16 stand in the low halves of a + 2^23 and b + 2^23
        code[w / 8] = __byte_perm(__float_as_uint(a + 8388608.f), __float_as_uint(b + 8388608.f), 0x5410);
    }
}

// 8 W elements at p as loaded, zeros where p is null.  VEC: p is on a 16-byte boundary.
template <bool VEC, int W>
__device__ __forceinline__ void q4_load(const __nv_bfloat16 *p, uint32_t (&w)[4 * W]) {
#pragma unroll
    for (int i = 0; i < 4 * W; ++i) w[i] = 0;
    if (p == nullptr) return;
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p) + i);
            w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
        }
    } else {
        const uint16_t *q = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
        for (int i = 0; i < 4 * W; ++i) w[i] = q[2 * i] | static_cast<uint32_t>(q[2 * i + 1]) << 16;
    }
}
template <bool VEC, int W>
__device__ __forceinline__ void q4_load(const float *p, float (&x)[8 * W]) {
#pragma unroll
    for (int i = 0; i < 8 * W; ++i) x[i] = 0.f;
    if (p == nullptr) return;
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < 2 * W; ++i) {
            const float4 a = __ldg(reinterpret_cast<const float4 *>(p) + i);
            x[4 * i] = a.x, x[4 * i + 1] = a.y, x[4 * i + 2] = a.z, x[4 * i + 3] = a.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8 * W; ++i) x[i] = p[i];
    }
}

// The codes and parameters of what every lane of a warp has loaded, a group over LANES lanes.
template <int LANES, int W>
__device__ __forceinline__ void q4_quantise_loaded(const uint32_t (&w)[4 * W], __half2 &par, uint32_t (&code)[W]) {
    float lo, hi, x[8 * W];
    q4_extremes<LANES>(w, lo, hi);
#pragma unroll
    for (int i = 0; i < 4 * W; ++i) {   // a bf16 is the top half of an fp32
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    q4_quantise<true>(x, lo, hi, par, code);
}
template <int LANES, int W>
__device__ __forceinline__ void q4_quantise_loaded(float (&x)[8 * W], __half2 &par, uint32_t (&code)[W]) {
    float lo, hi;
    q4_extremes<LANES>(x, lo, hi);
    q4_quantise<false>(x, lo, hi, par, code);
}

// How 8 W elements of type T are held between the two.
template <typename T, int W>
struct Q4Loaded;
template <int W>
struct Q4Loaded<__nv_bfloat16, W> {
    uint32_t v[4 * W];
};
template <int W>
struct Q4Loaded<float, W> {
    float v[8 * W];
};

}  // namespace pkv
