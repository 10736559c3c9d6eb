// Products with MXFP4 weights: the kernels of product.hpp for this format.
#include "product.hpp"

namespace epk {

hipError_t launch_product_mxfp4(const ProductArgs& a, int epilogue, hipStream_t s)
{
    return prod::launch_epilogue<kMxfp4>(a, epilogue, s);
}

}  // namespace epk
