// Interface of the balance loss (balance.hip) to its host side (moe_api.cpp).
#pragma once

#include "ep_internal.hpp"

namespace epk {

struct BalanceArgs {
    const void* logits;         // [N, E]
    bool bf16;
    bool vec;                   // logits (and their gradient) move as vectors of four
    const int32_t* topk;        // [N, K]
    const uint8_t* mask;        // [N] or null
    const int32_t* start;       // [Q+1] or null: one sequence
    int64_t N;
    int E, K, Q;
    int scoring;
    bool normalize;
    uint32_t k_magic;           // div_magic(K)
    int chunk;                  // tokens of a block
    int64_t slots;              // of partial sums: ceil(N / chunk) + Q
    // forward: partial sums by slot, the sequences' shares of the loss
    float* part_sum;            // [slots, E]
    int32_t* part_count;        // [slots, E]
    int32_t* part_tokens;       // [slots]
    double* part_loss;          // [blocks of the second kernel]
    uint32_t* ticket;
    double factor;              // coefficient / Q * E / K
    float* loss;
    int32_t* counts;            // [Q, E]
    int32_t* tokens;            // [Q]
    float* sums;                // [Q, E]
    // backward
    const int32_t* counts_in;
    const int32_t* tokens_in;
    const float* grad_loss;
    void* grad_logits;
};

// Workspace of the forward kernels, in bytes from its start.
struct BalanceCarve {
    int chunk;
    int64_t slots;
    // of the second kernel: blocks, items of a block at a time, waves of an item
    int64_t blocks;
    int at_once, join;
    int64_t sum, count, tokens, loss, ticket, total;
};
BalanceCarve carve_balance(int64_t N, int E, int Q);

hipError_t launch_balance(const BalanceArgs& a, const BalanceCarve& c, hipStream_t s);
hipError_t launch_balance_backward(const BalanceArgs& a, hipStream_t s);

}  // namespace epk
