// decode_own.cu -- the grouped-query split kernel over the pages past a shared
// prefix, for the shared-prefix decode, whose join merges its pieces.
#include "decode_gqa.cuh"

namespace pfkv {

int prepare_gqa_split(const DecodeArgs &a, SplitLaunch &launch) { return dispatch_split<true>(a, launch); }

int launch_gqa_split(SplitLaunch &launch, cudaStream_t s) { return enqueue_split(launch, s); }

}  // namespace pfkv
