// Whole-layer pieces around the expert products on gfx950: the choice of the
// product kernels by weight format, and the sum over a token's experts.
#include "experts.hpp"

namespace epk {

hipError_t launch_product_bf16(const ProductArgs& a, int epilogue, hipStream_t s);
hipError_t launch_product_mxfp4(const ProductArgs& a, int epilogue, hipStream_t s);
hipError_t launch_product_int4_g32(const ProductArgs& a, int epilogue, hipStream_t s);
hipError_t launch_product_int4_g64(const ProductArgs& a, int epilogue, hipStream_t s);
hipError_t launch_product_int4_g128(const ProductArgs& a, int epilogue, hipStream_t s);

hipError_t launch_down_few_bf16(const ProductArgs& a, bool* done, hipStream_t s);
hipError_t launch_down_few_mxfp4(const ProductArgs& a, bool* done, hipStream_t s);
hipError_t launch_down_few_int4_g32(const ProductArgs& a, bool* done, hipStream_t s);
hipError_t launch_down_few_int4_g64(const ProductArgs& a, bool* done, hipStream_t s);
hipError_t launch_down_few_int4_g128(const ProductArgs& a, bool* done, hipStream_t s);

hipError_t launch_down_few(const ProductArgs& a, bool* done, hipStream_t s)
{
    switch (a.w.kind) {
        case kBf16: return launch_down_few_bf16(a, done, s);
        case kMxfp4: return launch_down_few_mxfp4(a, done, s);
        case kInt4G32: return launch_down_few_int4_g32(a, done, s);
        case kInt4G64: return launch_down_few_int4_g64(a, done, s);
        default: return launch_down_few_int4_g128(a, done, s);
    }
}

hipError_t launch_product(ProductArgs a, int epilogue, hipStream_t s)
{
    switch (a.w.kind) {
        case kBf16: return launch_product_bf16(a, epilogue, s);
        case kMxfp4: return launch_product_mxfp4(a, epilogue, s);
        case kInt4G32: return launch_product_int4_g32(a, epilogue, s);
        case kInt4G64: return launch_product_int4_g64(a, epilogue, s);
        default: return launch_product_int4_g128(a, epilogue, s);
    }
}

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// out[t] = bf16(sum over the token's live entries, k ascending, of y[t,k]).
// Reads P rows of fp32 and writes N of bf16, a small share of the weights'
// bytes; four columns a thread.
__global__ __launch_bounds__(256) void k_layer_reduce(ReduceArgs a)
{
    const int h = (blockIdx.x * 256 + threadIdx.x) * 4;
    const int t = blockIdx.y;
    if (h >= a.H) return;
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < a.K; ++k) {
        const int e = a.topk[t * a.K + k];
        if ((uint32_t)e >= (uint32_t)a.E) continue;
        const f32x4 v = *reinterpret_cast<const f32x4*>(a.y + ((int64_t)t * a.K + k) * a.H + h);
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] += v[i];
    }
    const u32x2 d = {
        __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{sum[0], sum[1]}, bf16x2)),
        __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{sum[2], sum[3]}, bf16x2))};
    *reinterpret_cast<u32x2*>(a.out + (int64_t)t * a.H + h) = d;
}

}  // namespace

hipError_t launch_layer_reduce(const ReduceArgs& a, hipStream_t s)
{
    hipLaunchKernelGGL(k_layer_reduce, dim3((a.H / 4 + 255) / 256, a.N), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace epk
