// Products with bf16 weights: the kernels of product.hpp for this format.
#include "product.hpp"

namespace epk {

hipError_t launch_product_bf16(const ProductArgs& a, int epilogue, hipStream_t s)
{
    return prod::launch_epilogue<kBf16>(a, epilogue, s);
}

}  // namespace epk
