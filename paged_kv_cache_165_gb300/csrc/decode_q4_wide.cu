// decode_q4_wide.cu -- the warp-MMA kernel of decode_q4_mma.cuh for head sizes other than 64 and 128.
// 64 x 2048 tokens, one query row: 32 heads on 8 of 96 41 us (3.1 TB/s; the CUDA-core kernel 252), 16 on
// 4 of 160 40 us (2.7; 251), 16 on 4 of 256 48 us (3.0; 234).
#include "decode_q4_mma.cuh"

namespace pkv {

bool q4_wide_shape(int d, int group) {
    return ((d == 32 || d == 96 || d == 160) && group == 32) || (d == 192 && group <= 64) || (d == 256 && group >= 64);
}

namespace {
template <template <int, int, int> class Rows, int BS>
cudaError_t launch_as(const AttendQ4Params &P, int d, int G, dim3 grid, cudaStream_t stream) {
#define PKV_Q4_WIDE(DD, GG) \
    if (d == DD && G == GG) return launch_mma_as<DD, BS, GG, Rows<DD, BS, GG>>(P, grid, stream)
    PKV_Q4_WIDE(32, 1);
    PKV_Q4_WIDE(96, 3);
    PKV_Q4_WIDE(160, 5);
    PKV_Q4_WIDE(192, 3);
    PKV_Q4_WIDE(192, 6);
    PKV_Q4_WIDE(256, 2);
    PKV_Q4_WIDE(256, 4);
#undef PKV_Q4_WIDE
    return cudaErrorInvalidValue;
}
}  // namespace

cudaError_t launch_attend_q4_wide(const AttendQ4Params &P, int rows, int d, int bs, int G, dim3 grid, cudaStream_t stream) {
    if (rows == 4) return bs == 16 ? launch_as<FourRows, 16>(P, d, G, grid, stream) : launch_as<FourRows, 32>(P, d, G, grid, stream);
    return bs == 16 ? launch_as<EightRows, 16>(P, d, G, grid, stream) : launch_as<EightRows, 32>(P, d, G, grid, stream);
}

}  // namespace pkv
