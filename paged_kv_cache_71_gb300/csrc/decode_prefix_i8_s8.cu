// decode_prefix_i8_s8.cu -- instantiations of the shared-prefix decode (decode_mma.cuh) for an INT8 K/V
// cache and 8-token blocks.  (One file per cache dtype and block size, so that the instantiations compile in parallel.)
#include "decode_mma.cuh"

namespace pkv {

#define PKV_INST(G_, HP_)                                                                                   \
    template cudaError_t launch_paged_decode_prefix<G_, 8, KvI8, HP_>(const CUtensorMap&, const CUtensorMap&, \
                                                                       const DecodeArgs&, const PrefixArgs&, int, int, \
                                                                       size_t, cudaStream_t);
PKV_INST(1, 1)
PKV_INST(1, 2)
PKV_INST(2, 1)
PKV_INST(2, 2)
PKV_INST(4, 1)
PKV_INST(4, 2)
PKV_INST(8, 1)
#undef PKV_INST

}  // namespace pkv
