// decode_q4_bs8.cu -- the warp-MMA kernel of decode_q4_mma.cuh for pages of eight tokens: four bulk
// copies a side and stage.
#include "decode_q4_mma.cuh"

namespace pkv {
namespace {
template <template <int, int, int> class Rows>
cudaError_t launch_as(const AttendQ4Params &P, int d, int G, dim3 grid, cudaStream_t stream) {
#define PKV_Q4_BS8(DD, GG) \
    if (d == DD && G == GG) return launch_mma_as<DD, 8, GG, Rows<DD, 8, GG>>(P, grid, stream)
    PKV_Q4_BS8(32, 1);
    PKV_Q4_BS8(64, 1);
    PKV_Q4_BS8(64, 2);
    PKV_Q4_BS8(96, 3);
    PKV_Q4_BS8(128, 1);
    PKV_Q4_BS8(128, 2);
    PKV_Q4_BS8(128, 4);
    PKV_Q4_BS8(160, 5);
    PKV_Q4_BS8(192, 3);
    PKV_Q4_BS8(192, 6);
    PKV_Q4_BS8(256, 2);
    PKV_Q4_BS8(256, 4);
#undef PKV_Q4_BS8
    return cudaErrorInvalidValue;
}
}  // namespace

cudaError_t launch_attend_q4_bs8(const AttendQ4Params &P, int rows, int d, int G, dim3 grid, cudaStream_t stream) {
    return rows == 4 ? launch_as<FourRows>(P, d, G, grid, stream) : launch_as<EightRows>(P, d, G, grid, stream);
}

}  // namespace pkv
