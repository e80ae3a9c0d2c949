// decode_q4.cuh -- what the attention kernels over a 4-bit cache share: their parameters, a
// sequence's query rows and keys, and f16 splits (not part of the ABI).
#pragma once

#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "decode_kparams.cuh"
#include "internal.h"
#include "q4_codes.cuh"

namespace pkv {

struct AttendQ4Params {
    DecodeKParams k;     // head_tiles: tiles of (query row, head) pairs per sequence and KV head (4, 8 or 64 each)
    uint8_t *kc, *vc;
    int new_bf16;        // type of the step's new rows
    float q_sign;        // the queries are taken times the scale's sign (0, 1, -1) and k.scale_log2 is positive, so
                         // that masked scores of -inf stay what they are when they are scaled
    int balanced;        // the thread blocks share all sequences' keys evenly (else grid (splits x tiles, Hkv, B))
};

constexpr int kMaxBalanced = 1024;   // sequences of a balanced launch
template <typename Kernel>
cudaError_t set_smem_once(Kernel kernel, int bytes, std::atomic<unsigned long long> &done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(done.load() & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit);
    }
    return cudaSuccess;
}

// x ~= hi + lo, hi = rn_f16(x), lo = rn_f16(x - hi); the low half holds x.x.
__device__ __forceinline__ void split2(float2 x, uint32_t &hi, uint32_t &lo) {
    const __half2 h = __floats2half2_rn(x.x, x.y);
    const float2 f = __half22float2(h);
    const float2 r = add2(x, make_float2(-f.x, -f.y));
    const __half2 l = __floats2half2_rn(r.x, r.y);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = *reinterpret_cast<const uint32_t *>(&l);
}

__device__ __forceinline__ void split2(float x0, float x1, uint32_t &hi, uint32_t &lo) {
    split2(make_float2(x0, x1), hi, lo);
}

// V's codes less 8 (their scale then belongs to zero + 8 * scale): sums of weights times codes that
// average out.  Codes 0 and 4 of w's eight as (c - 8) * 2^-9 in `even`, codes 1 and 5 in `odd`,
// exactly.  The tensor core aligns the products by their operands' exponents, and a subnormal's is
// the smallest normal one: as c * 2^-24 the sums would lose the last 7 of their 24 bits.
__device__ __forceinline__ void centre(uint32_t w, uint32_t &even, uint32_t &odd) {
    // f16: 2^15, 2^11, -2^-6
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(even) : "r"(w & 0x000f000fu), "r"(0x78007800u), "r"(0xa400a400u));
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(odd) : "r"(w & 0x00f000f0u), "r"(0x68006800u), "r"(0xa400a400u));
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "mul.rn.f32x2 rd, ra, rb;\n\t"
        "mov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// 2^e as a float, e clamped to the normal range.
__device__ __forceinline__ float pow2i(int e) {
    return __uint_as_float(static_cast<uint32_t>(min(max(e, -126), 127) + 127) << 23);
}

// A sequence's query rows r0 .. r0 + nq - 1 (checked), its length L and the pages [first, first +
// pages) that any of them sees; rows [z0, z1) see nothing and are written as out = 0, lse = -inf.
struct SeqRows {
    int r0, nq, L, first, pages, z0, z1, z2, z3;
    bool ok;
};

__device__ __forceinline__ SeqRows seq_rows(const AttendQ4Params &P, int b, int bs, bool report) {
    const DecodeKParams &p = P.k;
    SeqRows s{};
    s.L = checked_len(p, b, bs, report);
    s.ok = true;
    if (p.cu_q == nullptr) {
        s.r0 = b;
        s.nq = 1;
        if (s.L == 0) s.z0 = b, s.z1 = b + 1;
    } else {
        const int c0 = __ldg(p.cu_q + b), c1 = __ldg(p.cu_q + b + 1);
        s.r0 = c0;
        s.nq = c1 - c0;
        s.ok = query_rows_ok(p, c0, c1, s.L);
        if (!s.ok) s.z0 = min(max(c0, 0), p.rows), s.z1 = min(max(c1, 0), p.rows);
        // rows before the first sequence or behind the last one belong to none
        if (b == 0 && c0 > 0) s.z2 = 0, s.z3 = min(c0, p.rows);
        if (b == p.B - 1 && c1 < p.rows) s.z2 = max(c1, 0), s.z3 = p.rows;
        if (report && (!s.ok || s.z3 > s.z2)) raise_error(p.err, PKV_DEVERR_CU_SEQLENS);
    }
    s.first = p.window > 0 ? max(0, s.L - s.nq + 1 - p.window) / bs : 0;
    s.pages = s.L > 0 && s.ok ? (s.L + bs - 1) / bs - s.first : 0;
    return s;
}

__device__ __forceinline__ void clear_rows(const AttendQ4Params &P, const SeqRows &s, int kvh, int d) {
    const DecodeKParams &p = P.k;
    for (int part = 0; part < 2; ++part) {
        const int z0 = part ? s.z2 : s.z0, z1 = part ? s.z3 : s.z1;
        for (int r = z0; r < z1; ++r) {
            const size_t at = static_cast<size_t>(r) * p.Hq + kvh * p.m;
            for (int i = threadIdx.x; i < p.m * d; i += blockDim.x) p.out[at * d + i] = 0.f;
            if (p.lse != nullptr)
                for (int i = threadIdx.x; i < p.m; i += blockDim.x) p.lse[at + i] = -INFINITY;
        }
    }
}

// Row v of a tile's (query row, head) pairs: head kvh * m + v % m of the sequence's query row
// v / m, which sees tokens [lo, len).  A row past the sequence's last repeats that one's span,
// with bi = -1.
struct RowSpan {
    int bi;        // (query row) * Hq + head
    int lo, len;
};
__device__ __forceinline__ RowSpan tile_row(const AttendQ4Params &P, const SeqRows &s, int kvh, int v) {
    const DecodeKParams &p = P.k;
    const int i = min(v / p.m, s.nq - 1);
    RowSpan r;
    r.len = s.L - s.nq + i + 1;
    r.lo = p.window > 0 ? max(0, r.len - p.window) : 0;
    r.bi = v < s.nq * p.m ? (s.r0 + i) * p.Hq + kvh * p.m + v % p.m : -1;
    return r;
}

// The parts of a unit (the rows of a tile over ranges of its keys).
struct Parts {
    int first;   // balanced: the warp that holds part 0; warp first + i holds part i
    int own, n;  // this part and their number
    unsigned *counter;
};

// The warp-MMA kernel, tiles of `rows` 4 or 8, for head sizes of 32, 96, 160 (groups of 32), 192 (32, 64) and
// 256 (64, 128) with pages of 16 or 32 tokens (decode_q4_wide.cu), and for pages of eight (decode_q4_bs8.cu).
bool q4_wide_shape(int d, int group);
cudaError_t launch_attend_q4_wide(const AttendQ4Params &P, int rows, int d, int bs, int G, dim3 grid, cudaStream_t stream);
cudaError_t launch_attend_q4_bs8(const AttendQ4Params &P, int rows, int d, int G, dim3 grid, cudaStream_t stream);

// The tcgen05 kernel (decode_q4_umma.cu): more query rows x heads for each KV head than the warp-MMA kernel
// is faster for (24 with one scale group a row, 32 with two; q4_mma_slots in decode_q4.cu).
constexpr int kQ4UmmaSlots = 64;   // (query row, head) pairs of a tile
bool q4_umma_shape(int d, int group, int bs);
cudaError_t launch_attend_q4_umma(const AttendQ4Params &P, int d, int bs, int G, dim3 grid, cudaStream_t stream);

}  // namespace pkv
