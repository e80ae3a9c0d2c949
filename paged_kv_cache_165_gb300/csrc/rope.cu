// rope.cu -- rotary positions of new tokens' q and K rows, with K and V written into the cache.
//
// Dimension pair j of a head at position p turns by the angle phi = p * f_j:
//   (a, b) -> mscale * (a cos phi - b sin phi, a sin phi + b cos phi),
// pairs (j, j + rot/2) or neighbours (2j, 2j + 1), dimensions from rot on as they are.  The attention's
// scores then depend on the distance of the two positions.  The inverse turns by -phi (the gradient).
//
// The angle: f_j comes as a fraction of a turn in 2^-64 units, so that p * f_j modulo a turn is one 64-bit
// product that wraps -- an exact range reduction for every 32-bit position, where an fp32 angle would be off
// by p * 2^-24.  Its nearest quarter turn goes into signs, the rest (at most an eighth of a turn) into one
// sincospif.  The cosines and sines of a token are computed once, into shared memory, for all its heads.
//
// Every element is read and written once, in 16-byte units where pointers and strides allow: bound by HBM for
// prompts and by launch latency for a decode step.  17153 tokens of 64 + 8 + 8 heads of 128 in bf16: 115 us, 6.09 TB/s
// (90% of the measured copy rate), at eight blocks an SM (122 us at six, then); cache hints and units dealt over a block's
// tokens by number, two at a time, measured slower (122 and 147 against 118), rows fetched towards L2 ahead of the angles
// too (126 to 150); 64 tokens 3 us.
#include <algorithm>
#include <cmath>

#include <cuda_bf16.h>

#include "common.cuh"
#include "internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 4;   // of a block

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void narrow(float x, float &y) { y = x; }
__device__ __forceinline__ void narrow(float x, __nv_bfloat16 &y) { y = __float2bfloat16_rn(x); }

// N elements moved together: in 16 (or, of the narrower type, 8) aligned bytes when N > 2, else one by one.
template <typename T, int N>
struct alignas(N <= 2 ? sizeof(T) : sizeof(T) * N > 16 ? 16 : sizeof(T) * N) Piece {
    T x[N];
};

template <typename T, int N>
__device__ __forceinline__ Piece<T, N> load_piece(const T *p) {
    return *reinterpret_cast<const Piece<T, N> *>(p);
}

template <typename To, int N>
__device__ __forceinline__ void store_piece(To *p, const float (&y)[N]) {
    Piece<To, N> r;
#pragma unroll
    for (int i = 0; i < N; ++i) narrow(y[i], r.x[i]);
    *reinterpret_cast<Piece<To, N> *>(p) = r;
}

// The cosine and sine (times mscale) of position pos for one pair.
__device__ __forceinline__ float2 turned(int pos, unsigned long long turns, bool inverse, float mscale) {
    unsigned long long phase = static_cast<unsigned long long>(static_cast<long long>(pos)) * turns;
    if (inverse) phase = 0ull - phase;
    const unsigned quarter = static_cast<unsigned>((phase + (1ull << 61)) >> 62);
    const long long rest = static_cast<long long>(phase - (static_cast<unsigned long long>(quarter) << 62));
    float s, c;
    sincospif(__ll2float_rn(rest) * 0x1p-63f, &s, &c);   // half turns, at most a quarter of one
    const float x = quarter & 1 ? -s : c, y = quarter & 1 ? c : s;
    return quarter & 2 ? make_float2(-x * mscale, -y * mscale) : make_float2(x * mscale, y * mscale);
}

// Units of a head: N pairs (two pieces rot/2 apart; neighbours that pair up: one piece of N elements) up to
// rot, N elements past it.  N = 2 (neighbours, unaligned) may leave one element of an odd d.
template <bool INTER, int N>
__host__ __device__ __forceinline__ int units_that_turn(int rot) { return INTER ? rot / N : rot / 2 / N; }
template <int N>
__host__ __device__ __forceinline__ int units_past(int d, int rot) { return (d - rot + N - 1) / N; }

// Unit u of a token is (head u / uh, piece u % uh), uh units a head, heads in the order q, K, V.
template <typename T, typename Tq, bool INTER, int N>
__global__ void __launch_bounds__(kThreads, 8) rope_kernel(const RopeArgs a) {
    extern __shared__ float2 s_cs[];   // [tokens of the block][rot / 2]
    __shared__ long long s_row[kMaxTokens];   // K/V row of head 0, -1: none
    pdl_wait();
    const int pairs = a.rot / 2;
    const long long t0 = static_cast<long long>(blockIdx.x) * a.block_tokens;
    const int nt = static_cast<int>(min(static_cast<long long>(a.block_tokens), a.T - t0));
    for (int i = threadIdx.x; i < nt * pairs; i += kThreads) {
        const int t = i / pairs, j = i - t * pairs;
        s_cs[i] = turned(a.positions[t0 + t], a.turns[j], a.inverse, a.mscale);
    }
    if (threadIdx.x < nt) {
        long long row = (t0 + threadIdx.x) * a.Hkv;
        if (a.slots != nullptr) {
            const long long slot = a.slots[t0 + threadIdx.x];
            const bool ok = slot >= 0 && slot < a.n_slots;   // < 0: padding
            if (slot >= a.n_slots && blockIdx.y == 0) raise_error(a.err, PKV_DEVERR_SLOT);
            row = ok ? slot / a.bs * a.Hkv * a.bs + slot % a.bs : -1;
        }
        s_row[threadIdx.x] = row;
    }
    __syncthreads();
    const int turning = units_that_turn<INTER, N>(a.rot), uh = turning + units_past<N>(a.d, a.rot);
    const int heads = a.Hq + (a.k != nullptr ? a.Hkv : 0) + (a.v != nullptr ? a.Hkv : 0);
    const int head_rows = a.slots != nullptr ? a.bs : 1;   // rows from one KV head to the next
    const int first = blockIdx.y * kThreads + threadIdx.x, step = gridDim.y * kThreads;
    const int step_h = step / uh, step_p = step - step_h * uh;
    for (int t = 0; t < nt; ++t) {
        const long long tok = t0 + t;
        const float2 *cs = s_cs + t * pairs;
        int h = first / uh, piece = first - h * uh;
        for (; h < heads; h += step_h, piece += step_p) {
            if (piece >= uh) {
                piece -= uh;
                if (++h >= heads) break;
            }
            const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hkv;
            const T *src;
            T *dst_kv = nullptr;
            Tq *dst_q = nullptr;
            if (is_q) {
                src = static_cast<const T *>(a.q) + tok * a.q_stride + static_cast<long long>(h) * a.d;
                dst_q = static_cast<Tq *>(a.q_out) + (tok * a.Hq + h) * a.d;
            } else {
                const long long row = s_row[t];
                if (row < 0) continue;
                const int kvh = is_v ? h - a.Hq - a.Hkv : h - a.Hq;
                src = static_cast<const T *>(is_v ? a.v : a.k) + tok * (is_v ? a.v_stride : a.k_stride) +
                      static_cast<long long>(kvh) * a.d;
                dst_kv = static_cast<T *>(is_v ? a.v_dst : a.k_dst) +
                         (row + static_cast<long long>(kvh) * head_rows) * a.d;
            }
            const bool turns = piece < turning, two = !INTER && turns;
            const int e0 = turns ? piece * N : a.rot + (piece - turning) * N;
            if (N == 2 && e0 + 1 == a.d) {   // the last element of an odd d
                if (is_q) narrow(widen(src[e0]), dst_q[e0]);
                else dst_kv[e0] = src[e0];
                continue;
            }
            const Piece<T, N> x0 = load_piece<T, N>(src + e0);
            Piece<T, N> x1 = x0;
            if (two) x1 = load_piece<T, N>(src + e0 + pairs);
            if (!is_q && (is_v || !turns)) {   // as they are, bit by bit
                *reinterpret_cast<Piece<T, N> *>(dst_kv + e0) = x0;
                if (two) *reinterpret_cast<Piece<T, N> *>(dst_kv + e0 + pairs) = x1;
                continue;
            }
            float y0[N], y1[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                y0[i] = widen(x0.x[i]);
                y1[i] = widen(x1.x[i]);
            }
            if (turns) {
#pragma unroll
                for (int i = 0; i < N; i += INTER ? 2 : 1) {
                    const float2 c = cs[INTER ? (e0 + i) / 2 : e0 + i];
                    float &p = y0[i], &q = INTER ? y0[(i + 1) % N] : y1[i];
                    const float was = p;
                    // one rounding less than two products and a sum, and the same for every cut into pieces
                    p = __fmaf_rn(was, c.x, -__fmul_rn(q, c.y));
                    q = __fmaf_rn(was, c.y, __fmul_rn(q, c.x));
                }
            }
            if (is_q) {
                store_piece(dst_q + e0, y0);
                if (two) store_piece(dst_q + e0 + pairs, y1);
            } else {
                store_piece(dst_kv + e0, y0);
                if (two) store_piece(dst_kv + e0 + pairs, y1);
            }
        }
    }
}

template <typename T, typename Tq, bool INTER, int N>
cudaError_t launch(const RopeArgs &given, int sm_count, cudaStream_t stream) {
    RopeArgs a = given;
    const int pairs = a.rot / 2;
    const int uh = units_that_turn<INTER, N>(a.rot) + units_past<N>(a.d, a.rot);
    const long long heads = a.Hq + (a.k != nullptr ? a.Hkv : 0) + (a.v != nullptr ? a.Hkv : 0);
    const long long units = heads * uh;
    // a token's units over several blocks while there are too few tokens to fill the GPU
    const long long want = 4ll * std::max(sm_count, 1);
    const long long split = std::max(1ll, std::min((units + kThreads - 1) / kThreads, want / std::max(1, a.T)));
    // tokens of a block by a model of the time: a wave of blocks (eight an SM) takes as long as a block's tokens and 192
    // units.  (17153 tokens of 640 units, 1 to 4 a block: 121, 120, 115 and 118 us; 4900: 39, 42, 42 and 49.)
    const long long slots = 8ll * std::max(sm_count, 1);
    double best = 0;
    for (int n = 1; n <= kMaxTokens; ++n) {
        const long long blocks = (a.T + n - 1ll) / n * split;
        const double cost = static_cast<double>((blocks + slots - 1) / slots) * (n + 192.0 / units);
        if (n == 1 || cost < best) {
            best = cost;
            a.block_tokens = n;
        }
    }
    const dim3 grid(static_cast<unsigned>((a.T + static_cast<long long>(a.block_tokens) - 1) / a.block_tokens),
                    static_cast<unsigned>(split));
    return launch_dependent(rope_kernel<T, Tq, INTER, N>, grid, dim3(kThreads),
                            static_cast<size_t>(a.block_tokens) * pairs * sizeof(float2), stream, a);
}

template <typename T, typename Tq, bool INTER>
cudaError_t launch_pieces(const RopeArgs &a, int sm_count, cudaStream_t stream) {
    constexpr int kWide = 16 / sizeof(T);
    // 16-byte pieces: of every row and pointer, of the part that turns and of the rest
    auto bits = [](const void *p) { return static_cast<unsigned long long>(reinterpret_cast<uintptr_t>(p)); };
    const unsigned long long at = bits(a.q) | bits(a.q_out) | bits(a.k) | bits(a.v) | bits(a.k_dst) | bits(a.v_dst);
    const long long strides = a.q_stride | a.k_stride | a.v_stride;
    const int cut = INTER ? a.rot : a.rot / 2;
    if (at % 16 == 0 && strides % kWide == 0 && a.d % kWide == 0 && cut % kWide == 0)
        return launch<T, Tq, INTER, kWide>(a, sm_count, stream);
    constexpr int kNarrow = INTER ? 2 : 1;
    return launch<T, Tq, INTER, kNarrow>(a, sm_count, stream);
}

template <typename T>
cudaError_t launch_types(const RopeArgs &a, pkv_dtype q_out_dt, bool interleaved, int sm_count, cudaStream_t stream) {
    if (q_out_dt == PKV_F32)
        return interleaved ? launch_pieces<T, float, true>(a, sm_count, stream)
                           : launch_pieces<T, float, false>(a, sm_count, stream);
    return interleaved ? launch_pieces<T, __nv_bfloat16, true>(a, sm_count, stream)
                       : launch_pieces<T, __nv_bfloat16, false>(a, sm_count, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, pkv_dtype dt, pkv_dtype q_out_dt, bool interleaved, int sm_count,
                        cudaStream_t stream) {
    if (a.T == 0) return cudaSuccess;
    return dt == PKV_BF16 ? launch_types<__nv_bfloat16>(a, q_out_dt, interleaved, sm_count, stream)
                          : launch_types<float>(a, q_out_dt, interleaved, sm_count, stream);
}

// The angles per position of every pair, as fractions of a turn in 2^-64 units (host arithmetic in fp64).  False: one is
// not finite.
bool rope_turns(uint64_t *turns, int rot, double base, int scaling, double factor, double original, double low, double high) {
    constexpr double kTurn = 6.283185307179586476925286766559;
    if (scaling == PKV_ROPE_BASE) base *= std::pow(factor, static_cast<double>(rot) / (rot - 2));
    for (int j = 0; j < rot / 2; ++j) {
        double f = std::pow(base, -2.0 * j / rot) / kTurn;   // turns per position
        if (scaling == PKV_ROPE_LINEAR) f /= factor;
        if (scaling == PKV_ROPE_PARTS) {
            const double r = std::min(1.0, std::max(0.0, (original * f - low) / (high - low)));
            f *= r + (1.0 - r) / factor;
        }
        if (!std::isfinite(f)) return false;
        f -= std::floor(f);
        turns[j] = static_cast<uint64_t>(std::ldexp(f, 63)) << 1;   // f < 1; below 2^-11 its last bits are cut, by less than 2^-63
    }
    return true;
}

}  // namespace pkv
