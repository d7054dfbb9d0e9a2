// The attention kernel on the fifth-generation tensor cores for heads of 128 elements (a translation unit of its own,
// to compile in parallel).
#include "attention_tiles.cuh"

namespace w4a16 {
namespace attention {

template cudaError_t launch_tiles<128>(const Params &, int, int, cudaStream_t);

}  // namespace attention
}  // namespace w4a16
