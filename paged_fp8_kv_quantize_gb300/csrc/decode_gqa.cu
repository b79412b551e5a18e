// decode_gqa.cu -- the grouped-query decode: split kernel and merge
// (decode_gqa.cuh).
#include "decode_gqa.cuh"

namespace pfkv {

int launch_gqa_decode(const DecodeArgs &a, cudaStream_t s) {
  DecodeArgs own = a;
  return dispatch_split<false>(own, s);
}

}  // namespace pfkv
