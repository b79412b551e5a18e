// decode_own.cu -- the grouped-query split kernel over the pages past a shared
// prefix, for the shared-prefix decode, whose join merges its pieces.
#include "decode_gqa.cuh"

namespace pfkv {

int launch_gqa_split(DecodeArgs &a, cudaStream_t s) { return dispatch_split<true>(a, s); }

}  // namespace pfkv
