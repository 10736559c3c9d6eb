// Products with INT4 weights with a scale per 32 columns: the kernels of product.hpp for this format.
#include "product.hpp"

namespace epk {

hipError_t launch_product_int4_g32(const ProductArgs& a, int epilogue, hipStream_t s)
{
    return prod::launch_epilogue<kInt4G32>(a, epilogue, s);
}

hipError_t launch_down_few_int4_g32(const ProductArgs& a, bool* done, hipStream_t s)
{
    return prod::launch_down_few<kInt4G32>(a, done, s);
}

}  // namespace epk
