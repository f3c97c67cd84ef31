// Split-K decode attention on the tensor cores over 4-bit codes: the
// instantiations of the kernel in decode_heads.cuh for every group size.
#include "decode_heads.cuh"

namespace okv {

template <int NGQ>
static okv_status launch_int4(const DecodeArgs& a, cudaStream_t s, bool early) {
  switch (a.g) {
    case 1: return launch_decode_heads<1, NGQ, 1, 4>(a, s, early);
    case 2: return launch_decode_heads<2, NGQ, 1, 4>(a, s, early);
    case 4: return launch_decode_heads<4, NGQ, 1, 4>(a, s, early);
    case 8:
      if constexpr (NGQ == 1) return launch_decode_heads<8, 1, 1, 4>(a, s, early);
      else return launch_decode_heads<4, NGQ, 2, 4>(a, s, early);  // G = 8 as two halves
    default: return launch_decode_heads<4, NGQ, 4, 4>(a, s, early);  // G = 16 as four quarters
  }
}

okv_status launch_decode_heads_int4(const DecodeArgs& a, cudaStream_t s, bool early) {
  return a.ng == 1 ? launch_int4<1>(a, s, early) : a.ng == 2 ? launch_int4<2>(a, s, early) : launch_int4<4>(a, s, early);
}

}  // namespace okv
