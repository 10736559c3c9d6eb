// Interface of the expert-product kernels (experts.hip, experts_*.hip) and
// the router kernels (gate.hip) to their host side (moe_api.cpp).
#pragma once

#include "ep_internal.hpp"
#include "product_shape.hpp"

namespace epk {

// Pairs (token, k) of one whole-layer call: 256 tokens x 16.
constexpr int kMaxPairs = 4096;

struct WeightArgs {
    const uint8_t* data;
    const uint8_t* scales;      // kInt8: fp32, one a row
    const uint8_t* zeros;       // nullptr: 8 everywhere
    int kind;
    int rows, cols;             // M, C (kInt8: C / 2)
    int64_t row_bytes;          // of data
    int64_t row_groups;         // scales per row
};

// What a product kernel does with its sums.
enum Epilogue {
    kStoreBf16 = 0,             // y = bf16(sum)
    kSwigluBf16 = 1,            // y = bf16(silu(gate) * up)
    kSwigluSplit = 2,           // y + y_lo = w * silu(gate) * up, two bf16 terms
    kStoreF32 = 3               // y = sum, fp32
};

struct ProductArgs {
    WeightArgs w;
    int E;
    int units;                  // outputs per row: M, or M/2 with a gate
    // Rows.  Dense (topk and count null): rows [0, num_rows) of expert 0.
    // Received rows (count): expert e's rows are [psum[e], psum[e] + count[e])
    // below num_rows, at most cap of them if cap > 0.
    // Pairs (topk): pair p belongs to expert topk[p]; its output row is p.
    int64_t num_rows;
    const int32_t* psum;
    const int32_t* count;
    int cap;
    const int32_t* topk;
    int P, K;                   // pairs, and pairs per token
    bool x_per_pair;            // pairs: x row = p (else the token p / K)
    const float* weights;       // pairs: [P] or null
    const uint16_t* x;          // bf16 [.., ldx]; kInt8: int8 [.., 2 ldx]
    const float* x_scales;      // kInt8: of each row of x
    const uint16_t* x_lo;       // its second term (kStoreF32), or null
    int64_t ldx;
    void* y;
    uint16_t* y_lo;
    int64_t ldy;
    uint32_t* flags;
    // launch shape (set by launch_product)
    int kw;                     // waves of a block that share a tile's columns
    int x_rows, x_bytes;        // rows of x in LDS at a time, and their bytes
    int pass_rows;              // rows of an expert that are multiplied at once
    uint32_t pass_magic;        // div_magic(pass_rows)
    int dense_passes;           // ceil(num_rows / pass_rows)
};

struct ReduceArgs {
    const float* y;             // [P, H]
    const int32_t* topk;        // [P]
    int N, K, E, H;
    uint16_t* out;              // bf16 [N, H]
};

struct GateArgs {
    const void* logits;
    bool bf16;
    const float* bias;
    const uint8_t* mask;
    int64_t N;
    int E, K, scoring, groups, topk_groups, group_top;
    int per;                    // experts of a group
    uint32_t per_magic;         // div_magic(per)
    bool renorm, limit;
    bool vec;                   // backward: rows of the gradient take vectors of four
    float scale;
    const int32_t* idx_in;      // backward
    const float* grad_w;
    int32_t* idx;
    float* w;
    void* grad_logits;
};

// What ProductArgs asks for; one kernel.
hipError_t launch_product(ProductArgs a, int epilogue, hipStream_t s);
// The same as kStoreF32 and launch_layer_reduce in one kernel, y = bf16 [N, H],
// where the batch is small enough for it (*done).
hipError_t launch_down_few(const ProductArgs& a, bool* done, hipStream_t s);
// Products in 8-bit integers (kInt8): y = bf16, gated or not.
// part: room for matmul_workspace bytes of sums, or null (one kernel then).
hipError_t launch_matmul(const ProductArgs& a, bool gate, int32_t* part, hipStream_t s);
int64_t matmul_workspace(bool gate, int64_t cols, int64_t units, int64_t rows);
hipError_t launch_layer_reduce(const ReduceArgs& a, hipStream_t s);
hipError_t launch_gate(const GateArgs& a, hipStream_t s);
hipError_t launch_gate_backward(const GateArgs& a, hipStream_t s);

}  // namespace epk
