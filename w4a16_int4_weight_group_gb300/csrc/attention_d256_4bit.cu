// The streaming attention kernel for heads of 256 elements with 4-bit codes (a translation unit of its own, to
// compile in parallel).
#include "attention_stream.cuh"

namespace w4a16 {
namespace attention {

template cudaError_t launch_stream<256, 4>(const Params &, int, int, cudaStream_t);

}  // namespace attention
}  // namespace w4a16
