// Products with MXFP4 weights: the kernels of product.hpp for this format.
#include "product.hpp"

namespace epk {

hipError_t launch_product_mxfp4(const ProductArgs& a, int epilogue, hipStream_t s)
{
    return prod::launch_epilogue<kMxfp4>(a, epilogue, s);
}

hipError_t launch_down_few_mxfp4(const ProductArgs& a, bool* done, hipStream_t s)
{
    return prod::launch_down_few<kMxfp4>(a, done, s);
}

}  // namespace epk
