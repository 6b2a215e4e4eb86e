// decode_quant_cluster.cu -- k_decode_quant's instances of small calls, whose clusters join their partials.
#include "decode_quant.cuh"

namespace ddt {

#define DDT_QUANT_INSTANCE(T, D, HP, GH, QP, PP) \
    template cudaError_t quant_launch<T, D, HP, GH, QP, PP, true>(const DecodeParams&, const DecQuantArgs&, const CUtensorMap*, cudaStream_t);
DDT_QUANT_INSTANCES(DDT_QUANT_INSTANCE)

}  // namespace ddt
