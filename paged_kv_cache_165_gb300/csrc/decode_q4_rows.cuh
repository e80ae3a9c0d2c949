// decode_q4_rows.cuh -- the arithmetic of the warp-MMA kernel (decode_q4_mma.cuh) for a tile of query
// rows: how eight (query row, head) pairs, or up to four, are laid out over a warp, and what they do
// with a stage of 32 keys in shared memory.  Layouts and ranges: decode_q4_mma.cuh.
#pragma once

#include "common.cuh"
#include "decode_q4.cuh"

namespace pkv {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kStageKeys = 32;

// Blocks of an SM for tiles of 4 or 8 rows: what registers (128, 168, 255 a thread) and the stages of wider
// heads leave.
__host__ __device__ constexpr int mma_blocks_per_sm(int rows, int d) {
    return rows == 4 ? (d <= 128 ? 4 : d <= 192 ? 3 : 2) : d <= 128 ? 3 : 2;
}

// D = A(16x16, f16, row) * B(16x8, f16, col) + D, fp32 accumulate.
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with C = 0, so that no registers are cleared first.
__device__ __forceinline__ void mma16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// The transpose of an 8 x 8 matrix of 16-bit elements held as an MMA fragment.
__device__ __forceinline__ uint32_t transposed(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// Words per thread and group of `N` consecutive 32-bit words from shared memory.
template <int N>
__device__ __forceinline__ void lds_words(const uint8_t *p, uint32_t (&w)[N]) {
    if constexpr (N == 4) {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
        w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
    } else if constexpr (N == 2) {
        const uint2 u = *reinterpret_cast<const uint2 *>(p);
        w[0] = u.x, w[1] = u.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = reinterpret_cast<const uint32_t *>(p)[i];
    }
}

// The parameters of the stage's key `lane`, widened to fp32 and handed to put(group, scale, zero +
// centred * scale); 0 for a key that is not seen.  Returns the largest |scale|.
template <int BS, int G, typename Put>
__device__ __forceinline__ float widen(const uint8_t *params, int page_bytes, float centred, bool seen, int lane, Put put) {
    uint32_t v[G];
    lds_words<G>(params + (lane / BS) * page_bytes + (lane % BS) * G * 4, v);
    float top = 0.f;
#pragma unroll
    for (int gi = 0; gi < G; ++gi) {
        const uint32_t raw = seen ? v[gi] : 0u;
        const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&raw));
        put(gi, y.x, fmaf(centred, y.x, y.y));
        top = fmaxf(top, fabsf(y.x));
    }
    return top;
}

// The largest V scale (by magnitude) seen so far and its exponent rounded up; `top`: a lane's of this stage.
struct ScaleTop {
    float most = 0.f, exponent = -24.f;
    __device__ __forceinline__ void take(float top) {
        if (__any_sync(kFull, top > most)) {   // rarely after the first stage: the next power of two
            // non-negative floats order like their bits
            most = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(fmaxf(top, most))));
            exponent = fmaxf(static_cast<float>(static_cast<int>((__float_as_uint(most) + 0x7fffffu) >> 23) - 127), -24.f);
        }
    }
};

// The factor that brings |q| of a row (amax) to [2^13, 2^14); a row of zeros (or of subnormals) keeps
// it finite.
__device__ __forceinline__ int q_exponent(float amax) { return min(13 - (static_cast<int>(__float_as_uint(amax) >> 23) - 127), 126); }

// ---- eight rows.  Lane (g, t4) = (lane / 4, lane % 4) holds the scores and weights of row g and the outputs of
// rows 2 t4 and 2 t4 + 1.
template <int D, int BS, int G>
struct EightRows {
    static constexpr int ROWS = 8, OUT = 2;
    static constexpr int WORDS = D / 8, WPT = WORDS / (4 * G);   // code words per row; per lane and group
    static constexpr int HPG = D / 32 / G;                       // 32-dimension columns per group
    static constexpr int NT = kStageKeys / 8;
    static constexpr int kCodeBytes = BS * D / 2, kPageBytes = BS * (D / 2 + 4 * G);
    static constexpr int kQBytes = (D / 16) * 512;   // a warp's query fragments
    // Three blocks (12 warps, 168 registers a thread) against four (128, with spills): 70B-shaped step 91.4
    // against 94.2 us, four sequences of 131072 tokens 142 against 139 (before V's codes were centred).
    // 16 rows a warp in two blocks (255 registers) take 10% less from 25 rows on and more below: not kept.
    static constexpr int kBlocksPerSm = mma_blocks_per_sm(8, D);
    static_assert(WPT >= 1 && HPG >= 1, "a group has at least 32 elements");

    uint4 *qfrag;    // [step][lane] of the warp, in shared memory
    float f, qsum[G];   // score (base 2) = MMA sum * f; the groups' sums of q in the MMAs' units
    float v[G * WPT][8];
    float oT[D / 16][4];
    float2 zo[G];             // sums of weight * zero over this lane's keys
    float m_run, l, ref;      // the running max; ref = m_run + E - 14, and l relative to it
    ScaleTop vs;

    static __device__ __forceinline__ int row(int lane) { return lane >> 2; }         // of the lane's scores
    static __device__ __forceinline__ int query_row(int lane) { return lane >> 2; }   // of the query words it lays out
    static __device__ __forceinline__ bool owner(int lane) { return (lane & 3) == 0; }
    static __device__ __forceinline__ int out_row(int r, int lane) { return 2 * (lane & 3) + r; }
    template <typename T>
    static __device__ __forceinline__ T of_out_row(T x, int r, int lane) { return __shfl_sync(kFull, x, 8 * (lane & 3) + 4 * r); }
    template <typename T>
    static __device__ __forceinline__ T of_merge_row(T x, int lane) { return __shfl_sync(kFull, x, 4 * (lane & 7)); }

    __device__ __forceinline__ void load(const float *q, int lane) {
#pragma unroll
        for (int u = 0; u < G * WPT; ++u) {
            const float2 *src = reinterpret_cast<const float2 *>(q + 8 * ((u / WPT) * (WORDS / G) + (lane & 3) * WPT + u % WPT));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 y = q != nullptr ? __ldg(src + e) : make_float2(0.f, 0.f);
                v[u][2 * e] = y.x;
                v[u][2 * e + 1] = y.y;
            }
        }
    }

    __device__ __forceinline__ void begin(float scale_log2, float q_sign, int lane) {
        // MMA steps 2u and 2u + 1 of word u = gi * WPT + i:
        // elements 8 * word + {0, 4}, {2, 6}, and their odd neighbours / 16
        float amax = 0.f;
#pragma unroll
        for (int u = 0; u < G * WPT; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(v[u][e]));
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
        const int up = q_exponent(amax);
        const float scale = pow2i(up) * q_sign;
        f = (scale_log2 * 0x1p24f) * pow2i(-up);
#pragma unroll
        for (int gi = 0; gi < G; ++gi) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < WPT; ++i) {
                const int u = gi * WPT + i;
                uint4 e, o;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[u][j] *= scale;
                    sum += v[u][j];
                }
#pragma unroll
                for (int j = 1; j < 8; j += 2) v[u][j] *= 0.0625f;
                split2(v[u][0], v[u][4], e.x, e.y);
                split2(v[u][2], v[u][6], e.z, e.w);
                split2(v[u][1], v[u][5], o.x, o.y);
                split2(v[u][3], v[u][7], o.z, o.w);
                qfrag[(2 * u) * 32] = e;
                qfrag[(2 * u + 1) * 32] = o;
            }
            sum += __shfl_xor_sync(kFull, sum, 1);
            sum += __shfl_xor_sync(kFull, sum, 2);
            qsum[gi] = sum * 0x1p-24f;
        }
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) oT[mt][0] = oT[mt][1] = oT[mt][2] = oT[mt][3] = 0.f;
#pragma unroll
        for (int gi = 0; gi < G; ++gi) zo[gi] = make_float2(0.f, 0.f);
        m_run = ref = -INFINITY;
        l = 0.f;
        vs = ScaleTop{};
    }

    // 32 keys from position tok0 on; end < 0: every row sees them all.  par: the warp's [group][scale, zero][key]
    __device__ __forceinline__ void stage(const uint8_t *kpages, const uint8_t *vpages, float *par, bool seen, int tok0, int end,
                                          const RowSpan &me, int lane) {
        const int g = lane >> 2, t4 = lane & 3;
        auto put = [&](int gi, float scale, float zero) {
            par[gi * 64 + lane] = scale;
            par[gi * 64 + 32 + lane] = zero;
        };
        // ---- scores of row g for keys 8 * nt + 2 * t4 + {0, 1}
        widen<BS, G>(kpages + kCodeBytes, kPageBytes, 0.f, seen, lane, put);
        __syncwarp();
        float2 s[NT];
#pragma unroll
        for (int gi = 0; gi < G; ++gi) {
            float a[NT][4];
            uint32_t c[NT][WPT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                lds_words<WPT>(kpages + (nt * 8 / BS) * kPageBytes + (nt * 8 % BS + g) * (D / 2) + gi * (D / 2 / G) +
                                   t4 * WPT * 4,
                               c[nt]);
            }
#pragma unroll
            for (int i = 0; i < WPT; ++i) {
                const uint4 e = qfrag[(2 * (gi * WPT + i)) * 32], o = qfrag[(2 * (gi * WPT + i) + 1) * 32];
                // the tiles' chains side by side
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint32_t x = c[nt][i] & 0x000f000fu, y = (c[nt][i] >> 8) & 0x000f000fu;
                    if (i == 0) mma16_first(a[nt], e.x, e.y, e.z, e.w, x, y);
                    else mma16(a[nt], e.x, e.y, e.z, e.w, x, y);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma16(a[nt], o.x, o.y, o.z, o.w, c[nt][i] & 0x00f000f0u, (c[nt][i] >> 8) & 0x00f000f0u);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float2 sc = *reinterpret_cast<const float2 *>(par + gi * 64 + nt * 8 + 2 * t4);
                const float2 ze = *reinterpret_cast<const float2 *>(par + gi * 64 + 32 + nt * 8 + 2 * t4);
                const float2 qz = make_float2(qsum[gi], qsum[gi]);
                const float2 y = gi == 0 ? mul2(ze, qz) : fma2(ze, qz, s[nt]);
                s[nt] = fma2(sc, add2(make_float2(a[nt][0], a[nt][1]), make_float2(a[nt][2], a[nt][3])), y);
            }
        }
        if (end >= 0) {   // some row does not see all of them
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int tok = tok0 + nt * 8 + 2 * t4, stop = min(me.len, end);
                if (tok < me.lo || tok >= stop) s[nt].x = -INFINITY;
                if (tok + 1 < me.lo || tok + 1 >= stop) s[nt].y = -INFINITY;
            }
        }
        __syncwarp();   // K's parameters have been read

        // ---- the running reference: the rows' maxima and the largest V scale
        const float top = widen<BS, G>(vpages + kCodeBytes, kPageBytes, 8.f, seen, lane, put);
        float mx = fmaxf(s[0].x, s[0].y);
#pragma unroll
        for (int nt = 1; nt < NT; ++nt) mx = fmaxf(mx, fmaxf(s[nt].x, s[nt].y));
        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
        m_run = fmaxf(m_run, mx * f);   // the scores are in the MMAs' units
        vs.take(top);
        const float ref_new = m_run + (vs.exponent - 14.f);
        // a row that has seen no key yet has ref -inf: its weights are 0 whatever the base
        const float base = ref_new == -INFINITY ? 0.f : ref_new;
        const float alpha = ref == -INFINITY ? 1.f : ex2_approx(ref - base);   // nothing to rescale yet
        ref = ref_new;
        float2 psum = make_float2(0.f, 0.f), w[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float2 e = fma2(s[nt], make_float2(f, f), make_float2(-base, -base));
            w[nt] = make_float2(ex2_approx(e.x), ex2_approx(e.y));
            psum = add2(psum, w[nt]);
        }
        l = l * alpha + (psum.x + psum.y);
        const float2 rescale = make_float2(__shfl_sync(kFull, alpha, 8 * t4), __shfl_sync(kFull, alpha, 8 * t4 + 4));
#pragma unroll
        for (int gi = 0; gi < G; ++gi) zo[gi] = mul2(zo[gi], make_float2(alpha, alpha));
        __syncwarp();   // V's parameters have been written
        if (end >= 0) {   // a key that only another row sees may hold a NaN: the zeros' part here, past it
#pragma unroll
            for (int gi = 0; gi < G; ++gi)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float2 z = *reinterpret_cast<const float2 *>(par + gi * 64 + 32 + nt * 8 + 2 * t4);
                    zo[gi] = fma2(w[nt], make_float2(w[nt].x != 0.f ? z.x : 0.f, w[nt].y != 0.f ? z.y : 0.f), zo[gi]);
                }
            __syncwarp();
#pragma unroll
            for (int gi = 0; gi < G; ++gi) par[gi * 64 + 32 + lane] = 0.f;
            __syncwarp();
        }

        // ---- O^T = O^T alpha + V^T P^T, 16 keys per step.  ldmatrix with transposition over 16-bit
        // units (four codes of a key) hands lane (g, t4) the units 8 * c + g of keys 2 * t4, 2 * t4 + 1
        // in one register: the pairs along the keys that the A operand wants.  N columns of 32
        // dimensions at a time; four matrices per load: two columns of 16 keys, or one of 32
        constexpr int KT = kStageKeys / 16, N = HPG >= 2 ? 2 : 1;
        const int vkey = N == 2 ? lane & 15 : lane;
        const uint32_t vrow = smem_addr(vpages) + vkey / BS * kPageBytes + vkey % BS * (D / 2) + (N == 2 ? (lane >> 4) * 16 : 0);
#pragma unroll
        for (int gi = 0; gi < G; ++gi) {
            uint32_t ph[KT][2], pl[KT][2];
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                const float *src = par + gi * 64 + kt * 16 + 2 * t4;
                const float2 wa = w[2 * kt], wb = w[2 * kt + 1];
                split2(mul2(wa, *reinterpret_cast<const float2 *>(src)), ph[kt][0], pl[kt][0]);
                split2(mul2(wb, *reinterpret_cast<const float2 *>(src + 8)), ph[kt][1], pl[kt][1]);
                zo[gi] = fma2(wa, *reinterpret_cast<const float2 *>(src + 32),
                              fma2(wb, *reinterpret_cast<const float2 *>(src + 40), zo[gi]));
            }
#pragma unroll
            for (int h = 0; h < HPG; h += N) {
                const int c = gi * HPG + h;
                float sum[2 * N][4];   // even and odd elements of each column
                uint32_t u[4];
                if constexpr (N == 1) ldsm_x4_trans(vrow + c * 16, u[0], u[1], u[2], u[3]);   // keys 0..7, 8..15, ...
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) {
                    uint32_t e[2 * N][2], o[2 * N][2];
                    // units 8 * c of keys 0..7, of keys 8..15, units 8 * (c + 1) likewise
                    if constexpr (N == 2)
                        ldsm_x4_trans(vrow + (kt * 16 / BS) * kPageBytes + (kt * 16 % BS) * (D / 2) + c * 16, u[0], u[1], u[2], u[3]);
#pragma unroll
                    for (int i = 0; i < 2 * N; ++i) {
                        centre(u[N == 2 ? i : 2 * kt + i], e[i][0], o[i][0]);
                        centre(u[N == 2 ? i : 2 * kt + i] >> 8, e[i][1], o[i][1]);
                    }
#pragma unroll
                    for (int lo = 0; lo < 2; ++lo) {   // the weights' high parts, then their low ones
                        const uint32_t b0 = lo ? pl[kt][0] : ph[kt][0], b1 = lo ? pl[kt][1] : ph[kt][1];
#pragma unroll
                        for (int i = 0; i < N; ++i) {
                            if (kt == 0 && lo == 0) {
                                mma16_first(sum[2 * i], e[2 * i][0], e[2 * i][1], e[2 * i + 1][0], e[2 * i + 1][1], b0, b1);
                                mma16_first(sum[2 * i + 1], o[2 * i][0], o[2 * i][1], o[2 * i + 1][0], o[2 * i + 1][1], b0, b1);
                            } else {
                                mma16(sum[2 * i], e[2 * i][0], e[2 * i][1], e[2 * i + 1][0], e[2 * i + 1][1], b0, b1);
                                mma16(sum[2 * i + 1], o[2 * i][0], o[2 * i][1], o[2 * i + 1][0], o[2 * i + 1][1], b0, b1);
                            }
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 2 * N; ++i)
#pragma unroll
                    for (int r = 0; r < 4; r += 2) {
                        float(&acc)[4] = oT[2 * c + i];
                        const float2 y = fma2(make_float2(acc[r], acc[r + 1]), rescale, make_float2(sum[i][r], sum[i][r + 1]));
                        acc[r] = y.x;
                        acc[r + 1] = y.y;
                    }
            }
        }
    }

    __device__ __forceinline__ void end() {
        l += __shfl_xor_sync(kFull, l, 1);
        l += __shfl_xor_sync(kFull, l, 2);
#pragma unroll
        for (int gi = 0; gi < G; ++gi) {
            zo[gi].x += zo[gi].y;
            zo[gi].x += __shfl_xor_sync(kFull, zo[gi].x, 1);
            zo[gi].x += __shfl_xor_sync(kFull, zo[gi].x, 2);
        }
    }
    // row out_row(r): dimensions 32 * c + 4 * g + {0, 1, 2, 3}
    __device__ __forceinline__ float4 output(int c, int r, int lane) const {
        const float z = __shfl_sync(kFull, zo[c / HPG].x, 8 * (lane & 3) + 4 * r);
        const float(&e)[4] = oT[2 * c], (&o)[4] = oT[2 * c + 1];
        return make_float4(fmaf(e[r], 0x1p9f, z), fmaf(o[r], 0x1p9f, z), fmaf(e[2 + r], 0x1p9f, z), fmaf(o[2 + r], 0x1p9f, z));
    }
};

// ---- up to four rows.  The MMAs' roles change places in the scores: the codes are the A operand (16 keys
// by 16 dimensions), the queries B, each row's hi and lo parts two neighbouring columns, so that a
// lane's two sums are those of one row: lane (g, t4) holds row t4's scores for keys g, g + 8, .. and its outputs.
// The weights' (hi, lo) pairs, transposed 8 x 8 at a time, are the columns of P^T.  Half the MMAs
// of eight rows, half the exponentials, the query fragments in registers.
template <int D, int BS, int G>
struct FourRows {
    static constexpr int ROWS = 4, OUT = 1;
    static constexpr int WORDS = D / 8, WPT = WORDS / (4 * G), HPG = D / 32 / G, NT = kStageKeys / 8;
    static constexpr int kCodeBytes = BS * D / 2, kPageBytes = BS * (D / 2 + 4 * G);
    static constexpr int kQBytes = 0;
    static constexpr int kBlocksPerSm = mma_blocks_per_sm(4, D);
    static_assert(WPT >= 1 && HPG >= 1, "a group has at least 32 elements");

    float f, qsum[G];
    float v[G * WPT][8];
    uint32_t q[G * WPT][2][2];   // B operands: [word][even, odd elements][k half]
    float oT[D / 16][2];
    float zo[G], m_run, l, ref;
    ScaleTop vs;

    static __device__ __forceinline__ int row(int lane) { return lane & 3; }
    static __device__ __forceinline__ int query_row(int lane) { return lane >> 3; }   // columns 2 r and 2 r + 1 belong to row r
    static __device__ __forceinline__ bool owner(int lane) { return lane < 4; }
    static __device__ __forceinline__ int out_row(int, int lane) { return lane & 3; }
    template <typename T>
    static __device__ __forceinline__ T of_out_row(T x, int, int) { return x; }
    template <typename T>
    static __device__ __forceinline__ T of_merge_row(T x, int) { return x; }

    __device__ __forceinline__ void load(const float *src, int lane) {
#pragma unroll
        for (int u = 0; u < G * WPT; ++u) {
            const float2 *p = reinterpret_cast<const float2 *>(src + 8 * ((u / WPT) * (WORDS / G) + (lane & 3) * WPT + u % WPT));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 y = src != nullptr ? __ldg(p + e) : make_float2(0.f, 0.f);
                v[u][2 * e] = y.x;
                v[u][2 * e + 1] = y.y;
            }
        }
    }

    __device__ __forceinline__ void begin(float scale_log2, float q_sign, int lane) {
        float amax = 0.f;
#pragma unroll
        for (int u = 0; u < G * WPT; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(v[u][e]));
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
        const int up = q_exponent(amax);
        const float scale = pow2i(up) * q_sign;
        const int from = 8 * (lane & 3);   // a lane that laid out this lane's row
        f = __shfl_sync(kFull, (scale_log2 * 0x1p24f) * pow2i(-up), from);
        const bool low = lane >> 2 & 1;    // an odd column: the lo parts
#pragma unroll
        for (int gi = 0; gi < G; ++gi) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < WPT; ++i) {
                const int u = gi * WPT + i;
                float x[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    x[j] = v[u][j] * scale;
                    sum += x[j];
                }
#pragma unroll
                for (int j = 1; j < 8; j += 2) x[j] *= 0.0625f;
#pragma unroll
                for (int odd = 0; odd < 2; ++odd)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {   // elements (0, 4), (2, 6); (1, 5), (3, 7)
                        uint32_t hi, lo;
                        split2(x[2 * h + odd], x[2 * h + odd + 4], hi, lo);
                        q[u][odd][h] = low ? lo : hi;
                    }
            }
            sum += __shfl_xor_sync(kFull, sum, 1);
            sum += __shfl_xor_sync(kFull, sum, 2);
            qsum[gi] = __shfl_sync(kFull, sum, from) * 0x1p-24f;
            zo[gi] = 0.f;
        }
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) oT[mt][0] = oT[mt][1] = 0.f;
        m_run = ref = -INFINITY;
        l = 0.f;
        vs = ScaleTop{};
    }

    // par: the warp's [group][key] pairs (scale, zero)
    __device__ __forceinline__ void stage(const uint8_t *kpages, const uint8_t *vpages, float *par, bool seen, int tok0, int end,
                                          const RowSpan &me, int lane) {
        const int g = lane >> 2, t4 = lane & 3;
        float2 *pairs = reinterpret_cast<float2 *>(par);
        auto put = [&](int gi, float scale, float zero) { pairs[gi * 32 + lane] = make_float2(scale, zero); };
        widen<BS, G>(kpages + kCodeBytes, kPageBytes, 0.f, seen, lane, put);
        __syncwarp();
        float s[NT];   // keys g + 8 j
#pragma unroll
        for (int gi = 0; gi < G; ++gi) {
            float a[NT / 2][2][4];   // [16 keys][even, odd elements]
            uint32_t c[NT][WPT];
#pragma unroll
            for (int j = 0; j < NT; ++j)
                lds_words<WPT>(kpages + (j * 8 / BS) * kPageBytes + (j * 8 % BS + g) * (D / 2) + gi * (D / 2 / G) + t4 * WPT * 4, c[j]);
#pragma unroll
            for (int i = 0; i < WPT; ++i)
#pragma unroll
                for (int odd = 0; odd < 2; ++odd) {
                    const uint32_t mask = odd ? 0x00f000f0u : 0x000f000fu;
                    const uint32_t(&b)[2] = q[gi * WPT + i][odd];
#pragma unroll
                    for (int mt = 0; mt < NT / 2; ++mt) {
                        const uint32_t x = c[2 * mt][i], y = c[2 * mt + 1][i];
                        if (i == 0) mma16_first(a[mt][odd], x & mask, y & mask, (x >> 8) & mask, (y >> 8) & mask, b[0], b[1]);
                        else mma16(a[mt][odd], x & mask, y & mask, (x >> 8) & mask, (y >> 8) & mask, b[0], b[1]);
                    }
                }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const float2 p = pairs[gi * 32 + 8 * j + g];
                const float(&e)[4] = a[j / 2][0], (&o)[4] = a[j / 2][1];
                const float2 t = add2(make_float2(e[2 * (j & 1)], e[2 * (j & 1) + 1]), make_float2(o[2 * (j & 1)], o[2 * (j & 1) + 1]));
                const float y = gi == 0 ? p.y * qsum[gi] : fmaf(p.y, qsum[gi], s[j]);
                s[j] = fmaf(p.x, t.x + t.y, y);
            }
        }
        if (end >= 0) {
            const int stop = min(me.len, end);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int tok = tok0 + 8 * j + g;
                if (tok < me.lo || tok >= stop) s[j] = -INFINITY;
            }
        }
        __syncwarp();   // K's parameters have been read

        vs.take(widen<BS, G>(vpages + kCodeBytes, kPageBytes, 8.f, seen, lane, put));
        float mx = s[0];
#pragma unroll
        for (int j = 1; j < NT; ++j) mx = fmaxf(mx, s[j]);
#pragma unroll
        for (int sh = 4; sh < 32; sh *= 2) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, sh));
        m_run = fmaxf(m_run, mx * f);   // the scores are in the MMAs' units
        const float ref_new = m_run + (vs.exponent - 14.f);
        // a row that has seen no key yet has ref -inf: its weights are 0 whatever the base
        const float base = ref_new == -INFINITY ? 0.f : ref_new;
        const float alpha = ref == -INFINITY ? 1.f : ex2_approx(ref - base);   // nothing to rescale yet
        ref = ref_new;
        float w[NT], sum_w = 0.f;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            w[j] = ex2_approx(fmaf(s[j], f, -base));
            sum_w += w[j];
        }
        l = fmaf(l, alpha, sum_w);
#pragma unroll
        for (int gi = 0; gi < G; ++gi) zo[gi] *= alpha;
        __syncwarp();   // V's parameters have been written
        if (end >= 0) {   // a key that only another row sees may hold a NaN: the zeros' part here, past it
#pragma unroll
            for (int gi = 0; gi < G; ++gi)
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    if (w[j] != 0.f) zo[gi] = fmaf(w[j], pairs[gi * 32 + 8 * j + g].y, zo[gi]);
            __syncwarp();
#pragma unroll
            for (int gi = 0; gi < G; ++gi) pairs[gi * 32 + lane].y = 0.f;
            __syncwarp();
        }

        // O^T = O^T alpha + V^T P^T as for eight rows, N columns of 32 dimensions at a time
        constexpr int KT = kStageKeys / 16, N = HPG >= 2 ? 2 : 1;
        const int vkey = N == 2 ? lane & 15 : lane;
        const uint32_t vrow = smem_addr(vpages) + vkey / BS * kPageBytes + vkey % BS * (D / 2) + (N == 2 ? (lane >> 4) * 16 : 0);
#pragma unroll
        for (int gi = 0; gi < G; ++gi) {
            uint32_t b[NT];   // B operand of 8 keys
#pragma unroll
            for (int j = 0; j < NT; j += 2) {
                const float2 p = pairs[gi * 32 + 8 * j + g], r = pairs[gi * 32 + 8 * j + 8 + g];
                uint32_t hi, lo;
                split2(w[j] * p.x, w[j + 1] * r.x, hi, lo);
                b[j] = transposed(__byte_perm(hi, lo, 0x5410));
                b[j + 1] = transposed(__byte_perm(hi, lo, 0x7632));
                zo[gi] = fmaf(w[j], p.y, fmaf(w[j + 1], r.y, zo[gi]));
            }
#pragma unroll
            for (int h = 0; h < HPG; h += N) {
                const int c = gi * HPG + h;
                float sum[2 * N][4];   // even and odd elements of each column
                uint32_t u4[4];
                if constexpr (N == 1) ldsm_x4_trans(vrow + c * 16, u4[0], u4[1], u4[2], u4[3]);
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) {
                    if constexpr (N == 2)
                        ldsm_x4_trans(vrow + (kt * 16 / BS) * kPageBytes + (kt * 16 % BS) * (D / 2) + c * 16, u4[0], u4[1], u4[2], u4[3]);
                    uint32_t e[2 * N][2], o[2 * N][2];
#pragma unroll
                    for (int i = 0; i < 2 * N; ++i) {
                        const uint32_t u = u4[N == 2 ? i : 2 * kt + i];
                        centre(u, e[i][0], o[i][0]);
                        centre(u >> 8, e[i][1], o[i][1]);
                    }
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        float(&y)[4] = sum[2 * i], (&z)[4] = sum[2 * i + 1];
                        if (kt == 0) {
                            mma16_first(y, e[2 * i][0], e[2 * i][1], e[2 * i + 1][0], e[2 * i + 1][1], b[0], b[1]);
                            mma16_first(z, o[2 * i][0], o[2 * i][1], o[2 * i + 1][0], o[2 * i + 1][1], b[0], b[1]);
                        } else {
                            mma16(y, e[2 * i][0], e[2 * i][1], e[2 * i + 1][0], e[2 * i + 1][1], b[2], b[3]);
                            mma16(z, o[2 * i][0], o[2 * i][1], o[2 * i + 1][0], o[2 * i + 1][1], b[2], b[3]);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 2 * N; ++i) {
                    float(&acc)[2] = oT[2 * c + i];
                    acc[0] = fmaf(acc[0], alpha, sum[i][0] + sum[i][1]);
                    acc[1] = fmaf(acc[1], alpha, sum[i][2] + sum[i][3]);
                }
            }
        }
    }

    __device__ __forceinline__ void end() {
#pragma unroll
        for (int sh = 4; sh < 32; sh *= 2) {
            l += __shfl_xor_sync(kFull, l, sh);
#pragma unroll
            for (int gi = 0; gi < G; ++gi) zo[gi] += __shfl_xor_sync(kFull, zo[gi], sh);
        }
    }
    __device__ __forceinline__ float4 output(int c, int, int) const {
        const float z = zo[c / HPG];
        return make_float4(fmaf(oT[2 * c][0], 0x1p9f, z), fmaf(oT[2 * c + 1][0], 0x1p9f, z), fmaf(oT[2 * c][1], 0x1p9f, z),
                           fmaf(oT[2 * c + 1][1], 0x1p9f, z));
    }
};

}  // namespace
}  // namespace pkv
