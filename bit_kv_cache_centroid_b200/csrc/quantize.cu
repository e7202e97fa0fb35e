// quantize.cu — the append of consecutive tokens at one slot of every sequence.
#include "quantize.cuh"

namespace kv2 {

cudaError_t launch_quantize(const QuantizeArgs& a, cudaStream_t s) { return launch<false>(a, s); }

}  // namespace kv2
