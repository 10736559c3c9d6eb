// Products of few int8 rows an expert with int8 weights: the kernels of product.hpp
// for this format.
#include "product.hpp"

namespace epk {

hipError_t launch_product_int8(const ProductArgs& a, int epilogue, hipStream_t s)
{
    return epilogue == kSwigluBf16 ? prod::launch_kind<kInt8, kSwigluBf16>(a, s)
                                   : prod::launch_kind<kInt8, kStoreBf16>(a, s);
}

}  // namespace epk
