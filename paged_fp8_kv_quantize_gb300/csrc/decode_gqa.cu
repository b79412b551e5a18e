// decode_gqa.cu -- the grouped-query decode: split kernel and merge
// (decode_gqa.cuh).
#include "decode_gqa.cuh"

namespace pfkv {

int launch_gqa_decode(const DecodeArgs &a, cudaStream_t s) {
  SplitLaunch l;
  return dispatch_split<false>(a, l, s);
}

}  // namespace pfkv
