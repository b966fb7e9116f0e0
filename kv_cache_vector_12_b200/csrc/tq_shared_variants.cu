// Instantiations of the decode attention kernel's build for groups that share
// a prefix (SHARED), for one head dimension and one K width, chosen by
// TQ_DECODE_DH and TQ_DECODE_BK on the compiler's command line as in
// tq_decode_variants.cu.  Without the two macros the object is empty.
#include "tq_decode_kernel.cuh"

#if defined(TQ_DECODE_DH) && defined(TQ_DECODE_BK)
namespace tq {

template <int DH, int BK>
DecodeVariant shared_variant(int bits_v, bool qjl, int nt) {
  return variant_k<BK, DH, true>(bits_v, qjl, nt, kShared);
}

template DecodeVariant shared_variant<TQ_DECODE_DH, TQ_DECODE_BK>(int, bool, int);

}  // namespace tq
#endif
