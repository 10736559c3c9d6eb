// Products with bf16 weights: the kernels of product.hpp for this format.
#include "product.hpp"

namespace epk {

hipError_t launch_product_bf16(const ProductArgs& a, int epilogue, hipStream_t s)
{
    return prod::launch_epilogue<kBf16>(a, epilogue, s);
}

hipError_t launch_down_few_bf16(const ProductArgs& a, bool* done, hipStream_t s)
{
    return prod::launch_down_few<kBf16>(a, done, s);
}

}  // namespace epk
