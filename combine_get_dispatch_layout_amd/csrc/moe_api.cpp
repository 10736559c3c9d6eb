// C-ABI host side of include/ep_moe.h: validation and launches.  As in
// api.cpp, arguments are checked before any HIP call and no device memory is
// allocated.
#include "ep_moe.h"

#include <hip/hip_runtime.h>

#include <cmath>

#include "ep_host.hpp"
#include "experts.hpp"

namespace {

#define EP_FAIL(st, ...) epk::host_fail((st), __FILE__, __LINE__, __VA_ARGS__)
#define EP_HIP(call)                                                                          \
    do {                                                                                      \
        hipError_t e_ = (call);                                                               \
        if (e_ != hipSuccess) return EP_FAIL(EP_ERR_HIP, "%s: %s", #call, hipGetErrorString(e_)); \
    } while (0)

constexpr int kMaxDim = 1 << 24;    // rows and columns of a weight matrix

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int64_t align_up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

ep_status check_gate(const ep_gate_config* c, int64_t num_tokens, epk::GateArgs* out)
{
    if (!c) return EP_FAIL(EP_ERR_INVALID_ARG, "config is NULL");
    if (c->num_experts < 1 || c->num_experts > epk::kMaxExperts)
        return EP_FAIL(EP_ERR_INVALID_ARG, "num_experts=%d outside [1,%d]", c->num_experts,
                       epk::kMaxExperts);
    if (c->num_topk < 1 || c->num_topk > epk::kMaxTopk || c->num_topk > c->num_experts)
        return EP_FAIL(EP_ERR_INVALID_ARG, "num_topk=%d outside [1,%d] or above num_experts=%d",
                       c->num_topk, epk::kMaxTopk, c->num_experts);
    if (c->scoring != EP_SCORE_SOFTMAX && c->scoring != EP_SCORE_SIGMOID)
        return EP_FAIL(EP_ERR_INVALID_ARG, "scoring=%d unknown", c->scoring);
    if (c->logits_type != EP_LOGITS_FP32 && c->logits_type != EP_LOGITS_BF16)
        return EP_FAIL(EP_ERR_INVALID_ARG, "logits_type=%d unknown", c->logits_type);
    if ((c->renormalize != 0 && c->renormalize != 1) || (c->group_limit != 0 && c->group_limit != 1))
        return EP_FAIL(EP_ERR_INVALID_ARG, "renormalize=%d and group_limit=%d must be 0 or 1",
                       c->renormalize, c->group_limit);
    if (!std::isfinite(c->scale)) return EP_FAIL(EP_ERR_INVALID_ARG, "scale is not finite");
    if (c->num_groups < 0 || c->num_groups > 64)
        return EP_FAIL(EP_ERR_INVALID_ARG, "num_groups=%d outside [0,64]", c->num_groups);
    if (c->num_groups > 1) {
        if (c->num_experts % c->num_groups != 0)
            return EP_FAIL(EP_ERR_INVALID_ARG, "num_groups=%d must divide num_experts=%d",
                           c->num_groups, c->num_experts);
        const int per = c->num_experts / c->num_groups;
        if (c->topk_groups < 1 || c->topk_groups > c->num_groups)
            return EP_FAIL(EP_ERR_INVALID_ARG, "topk_groups=%d outside [1,%d]", c->topk_groups,
                           c->num_groups);
        if (c->group_top < 1 || c->group_top > per)
            return EP_FAIL(EP_ERR_INVALID_ARG, "group_top=%d outside [1,%d]", c->group_top, per);
        if (c->topk_groups * (c->group_limit ? c->group_top : per) < c->num_topk)
            return EP_FAIL(EP_ERR_INVALID_ARG, "%d groups of %d experts cannot hold num_topk=%d",
                           c->topk_groups, c->group_limit ? c->group_top : per, c->num_topk);
    }
    if (num_tokens < 0 || num_tokens >= (int64_t)1 << 31)
        return EP_FAIL(EP_ERR_INVALID_ARG, "num_tokens=%lld outside [0, 2^31)", (long long)num_tokens);
    epk::GateArgs& a = *out;
    a = epk::GateArgs{};
    a.bf16 = c->logits_type == EP_LOGITS_BF16;
    a.N = num_tokens;
    a.E = c->num_experts;
    a.K = c->num_topk;
    a.scoring = c->scoring;
    a.renorm = c->renormalize == 1;
    a.groups = c->num_groups;
    a.topk_groups = c->topk_groups;
    a.group_top = c->group_top;
    a.per = c->num_groups > 1 ? c->num_experts / c->num_groups : 1;
    a.per_magic = epk::div_magic((uint32_t)a.per);
    a.limit = c->group_limit == 1;
    a.scale = c->scale;
    return EP_OK;
}

// Checks a weight stack without its pointers (sizes only) or with them.
ep_status check_weights(const ep_weights* w, const char* name, bool pointers)
{
    if (!w) return EP_FAIL(EP_ERR_INVALID_ARG, "%s is NULL", name);
    if (w->format < EP_WEIGHT_BF16 || w->format > EP_WEIGHT_INT4)
        return EP_FAIL(EP_ERR_INVALID_ARG, "%s: format=%d unknown", name, w->format);
    if (w->num_experts < 1 || w->num_experts > epk::kMaxExperts)
        return EP_FAIL(EP_ERR_INVALID_ARG, "%s: num_experts=%d outside [1,%d]", name, w->num_experts,
                       epk::kMaxExperts);
    if (w->rows < 1 || w->rows > kMaxDim || w->cols < 1 || w->cols > kMaxDim)
        return EP_FAIL(EP_ERR_INVALID_ARG, "%s: rows=%d and cols=%d must be in [1,%d]", name, w->rows,
                       w->cols, kMaxDim);
    if (w->reserved != 0) return EP_FAIL(EP_ERR_INVALID_ARG, "%s: reserved must be 0", name);
    if (w->format == EP_WEIGHT_BF16) {
        if (w->group != 0) return EP_FAIL(EP_ERR_INVALID_ARG, "%s: bf16 weights have no group", name);
        if (w->cols % 8 != 0)
            return EP_FAIL(EP_ERR_INVALID_ARG, "%s: cols=%d must be a multiple of 8", name, w->cols);
    } else {
        const bool mx = w->format == EP_WEIGHT_MXFP4;
        if (mx ? w->group != 32 : (w->group != 32 && w->group != 64 && w->group != 128))
            return EP_FAIL(EP_ERR_INVALID_ARG, "%s: group=%d must be %s", name, w->group,
                           mx ? "32" : "32, 64 or 128");
        if (w->cols % w->group != 0)
            return EP_FAIL(EP_ERR_INVALID_ARG, "%s: cols=%d must be a multiple of group=%d", name,
                           w->cols, w->group);
    }
    if (!pointers) return EP_OK;
    if (!w->d_data || !aligned(w->d_data, 16))
        return EP_FAIL(EP_ERR_INVALID_ARG, "%s: data must be 16-byte aligned and not NULL", name);
    if (w->format == EP_WEIGHT_BF16 ? w->d_scales != nullptr
                                    : (!w->d_scales || !aligned(w->d_scales, 16)))
        return EP_FAIL(EP_ERR_INVALID_ARG, "%s: scales must be %s", name,
                       w->format == EP_WEIGHT_BF16 ? "NULL for bf16 weights"
                                                   : "16-byte aligned and not NULL");
    if (w->d_zeros && w->format != EP_WEIGHT_INT4)
        return EP_FAIL(EP_ERR_INVALID_ARG, "%s: only INT4 weights have zeros", name);
    if (!aligned(w->d_zeros, 16))
        return EP_FAIL(EP_ERR_INVALID_ARG, "%s: zeros must be 16-byte aligned", name);
    return EP_OK;
}

epk::WeightArgs weight_args(const ep_weights* w)
{
    epk::WeightArgs a;
    a.data = static_cast<const uint8_t*>(w->d_data);
    a.scales = static_cast<const uint8_t*>(w->d_scales);
    a.zeros = static_cast<const uint8_t*>(w->d_zeros);
    a.kind = w->format == EP_WEIGHT_BF16 ? epk::kBf16
             : w->format == EP_WEIGHT_MXFP4 ? epk::kMxfp4
             : w->group == 32 ? epk::kInt4G32 : w->group == 64 ? epk::kInt4G64 : epk::kInt4G128;
    a.rows = w->rows;
    a.cols = w->cols;
    a.row_bytes = w->format == EP_WEIGHT_BF16 ? 2 * (int64_t)w->cols : w->cols / 2;
    a.row_groups = w->group ? w->cols / w->group : 0;
    return a;
}

ep_status check_activation(const ep_weights* w, int32_t activation)
{
    if (activation != EP_ACT_NONE && activation != EP_ACT_SWIGLU)
        return EP_FAIL(EP_ERR_INVALID_ARG, "activation=%d unknown", activation);
    if (activation == EP_ACT_SWIGLU && w->rows % 2 != 0)
        return EP_FAIL(EP_ERR_INVALID_ARG, "SWIGLU needs an even number of weight rows (rows=%d)",
                       w->rows);
    return EP_OK;
}

ep_status check_rows(const ep_weights* w, const void* d_x, int64_t rows, const void* d_y)
{
    // the kernels number (row, 16 outputs) tiles in 32 bits
    if (rows < 0 || rows >= (int64_t)1 << 31 || rows * ((w->rows + 15) / 16) >= (int64_t)1 << 31)
        return EP_FAIL(EP_ERR_INVALID_ARG, "%lld rows times %d outputs outside [0, 2^35)",
                       (long long)rows, w->rows);
    if (rows == 0) return EP_OK;
    if (!d_x || !d_y) return EP_FAIL(EP_ERR_INVALID_ARG, "x or y is NULL");
    if (!aligned(d_x, 16) || !aligned(d_y, 2))
        return EP_FAIL(EP_ERR_INVALID_ARG, "x must be 16-byte aligned, y 2-byte aligned");
    return EP_OK;
}

// The two stacks of a layer against the handle's configuration.
ep_status check_layer(const ep_handle* h, const ep_weights* up, const ep_weights* down,
                      int64_t num_tokens, bool pointers, epk::HandleInfo* info)
{
    if (!h) return EP_FAIL(EP_ERR_INVALID_ARG, "handle is NULL");
    ep_status st = check_weights(up, "w_up", pointers);
    if (st == EP_OK) st = check_weights(down, "w_down", pointers);
    if (st != EP_OK) return st;
    *info = epk::handle_info(h);
    const ep_config& c = *info->cfg;
    if (up->num_experts != c.num_experts || down->num_experts != c.num_experts)
        return EP_FAIL(EP_ERR_INVALID_ARG, "w_up has %d experts, w_down %d, the handle %d",
                       up->num_experts, down->num_experts, c.num_experts);
    if (up->cols != c.hidden || down->rows != c.hidden)
        return EP_FAIL(EP_ERR_INVALID_ARG, "w_up's cols=%d and w_down's rows=%d must be hidden=%d",
                       up->cols, down->rows, c.hidden);
    if (up->rows % 2 != 0 || down->cols != up->rows / 2)
        return EP_FAIL(EP_ERR_INVALID_ARG, "w_up's rows=%d must be twice w_down's cols=%d", up->rows,
                       down->cols);
    if (num_tokens < 0 || num_tokens > EP_MOE_MAX_TOKENS)
        return EP_FAIL(EP_ERR_INVALID_ARG, "num_tokens=%lld outside [0,%d]", (long long)num_tokens,
                       EP_MOE_MAX_TOKENS);
    // the kernels number (row, 16 outputs) tiles in 32 bits
    const int64_t outputs = up->rows > down->rows ? up->rows : down->rows;
    if (num_tokens * c.num_topk * ((outputs + 15) / 16) >= (int64_t)1 << 31)
        return EP_FAIL(EP_ERR_INVALID_ARG, "%lld pairs times %lld outputs above 2^35",
                       (long long)(num_tokens * c.num_topk), (long long)outputs);
    return EP_OK;
}

// Workspace of a layer: a in two bf16 terms, and each pair's output.
struct LayerCarve {
    int64_t act, act_lo, y, total;
};

LayerCarve carve_layer(int64_t pairs, int64_t inter, int64_t hidden)
{
    LayerCarve c;
    c.act = 0;
    c.act_lo = align_up(2 * pairs * inter, 256);
    c.y = 2 * c.act_lo;
    c.total = c.y + align_up(4 * pairs * hidden, 256);
    if (c.total < 256) c.total = 256;
    return c;
}

}  // namespace

extern "C" {

ep_status ep_gate(const ep_gate_config* cfg, const void* d_logits, const float* d_bias,
                  const uint8_t* d_token_mask, int64_t num_tokens, int32_t* d_topk_idx,
                  float* d_topk_weights, void* stream)
{
    epk::GateArgs a;
    ep_status st = check_gate(cfg, num_tokens, &a);
    if (st != EP_OK || num_tokens == 0) return st;
    if (!d_logits || !d_topk_idx || !d_topk_weights)
        return EP_FAIL(EP_ERR_INVALID_ARG, "logits, topk_idx or topk_weights is NULL");
    if (!aligned(d_logits, a.bf16 ? 2 : 4) || !aligned(d_bias, 4) || !aligned(d_topk_idx, 4) ||
        !aligned(d_topk_weights, 4))
        return EP_FAIL(EP_ERR_INVALID_ARG, "logits, bias, topk_idx or topk_weights is not aligned to its type");
    a.logits = d_logits;
    a.bias = d_bias;
    a.mask = d_token_mask;
    a.idx = d_topk_idx;
    a.w = d_topk_weights;
    EP_HIP(epk::launch_gate(a, static_cast<hipStream_t>(stream)));
    return EP_OK;
}

ep_status ep_gate_backward(const ep_gate_config* cfg, const void* d_logits,
                           const int32_t* d_topk_idx, const float* d_grad_weights,
                           int64_t num_tokens, void* d_grad_logits, void* stream)
{
    epk::GateArgs a;
    ep_status st = check_gate(cfg, num_tokens, &a);
    if (st != EP_OK || num_tokens == 0) return st;
    if (!d_logits || !d_topk_idx || !d_grad_weights || !d_grad_logits)
        return EP_FAIL(EP_ERR_INVALID_ARG, "logits, topk_idx, grad_weights or grad_logits is NULL");
    if (!aligned(d_logits, a.bf16 ? 2 : 4) || !aligned(d_grad_logits, a.bf16 ? 2 : 4) ||
        !aligned(d_topk_idx, 4) || !aligned(d_grad_weights, 4))
        return EP_FAIL(EP_ERR_INVALID_ARG, "logits, topk_idx, grad_weights or grad_logits is not aligned to its type");
    a.logits = d_logits;
    a.idx_in = d_topk_idx;
    a.grad_w = d_grad_weights;
    a.grad_logits = d_grad_logits;
    a.vec = a.E % 4 == 0 && aligned(d_grad_logits, a.bf16 ? 8 : 16);
    EP_HIP(epk::launch_gate_backward(a, static_cast<hipStream_t>(stream)));
    return EP_OK;
}

ep_status ep_matvec(const ep_weights* w, const void* d_x, int64_t num_rows, int32_t activation,
                    void* d_y, void* stream)
{
    ep_status st = check_weights(w, "w", true);
    if (st == EP_OK) st = check_activation(w, activation);
    if (st == EP_OK) st = check_rows(w, d_x, num_rows, d_y);
    if (st != EP_OK) return st;
    if (w->num_experts != 1)
        return EP_FAIL(EP_ERR_INVALID_ARG, "ep_matvec takes one matrix (num_experts=%d)", w->num_experts);
    epk::ProductArgs a = {};
    a.w = weight_args(w);
    a.E = 1;
    a.units = activation == EP_ACT_SWIGLU ? w->rows / 2 : w->rows;
    a.num_rows = num_rows;
    a.x = static_cast<const uint16_t*>(d_x);
    a.ldx = w->cols;
    a.y = d_y;
    a.ldy = a.units;
    EP_HIP(epk::launch_product(a, activation == EP_ACT_SWIGLU ? epk::kSwigluBf16 : epk::kStoreBf16,
                               static_cast<hipStream_t>(stream)));
    return EP_OK;
}

ep_status ep_expert_matvec(const ep_handle* h, const ep_weights* w, const void* d_x,
                           int64_t x_rows, int32_t activation, void* d_y, void* stream)
{
    if (!h) return EP_FAIL(EP_ERR_INVALID_ARG, "handle is NULL");
    ep_status st = check_weights(w, "w", true);
    if (st == EP_OK) st = check_activation(w, activation);
    if (st == EP_OK) st = check_rows(w, d_x, x_rows, d_y);
    if (st != EP_OK) return st;
    const epk::HandleInfo info = epk::handle_info(h);
    if (info.cfg->non_expand)
        return EP_FAIL(EP_ERR_INVALID_ARG, "non-expand rows belong to ranks, not experts");
    if (w->num_experts != info.cfg->num_experts)
        return EP_FAIL(EP_ERR_INVALID_ARG, "w has %d experts, the handle %d", w->num_experts,
                       info.cfg->num_experts);
    if (info.num_tokens < 0) return EP_FAIL(EP_ERR_STATE, "ep_get_layout has not run on this handle");
    if (info.pending)
        return EP_FAIL(EP_ERR_STATE, "the handle's layout is waiting for ep_combine_overlap");
    epk::ProductArgs a = {};
    a.w = weight_args(w);
    a.E = w->num_experts;
    a.units = activation == EP_ACT_SWIGLU ? w->rows / 2 : w->rows;
    a.num_rows = x_rows;
    a.P = (int)(info.num_tokens * info.cfg->num_topk);
    a.psum = info.psum_expert;
    a.count = info.num_unaligned;
    a.cap = info.cfg->expert_capacity;
    a.x = static_cast<const uint16_t*>(d_x);
    a.ldx = w->cols;
    a.y = d_y;
    a.ldy = a.units;
    a.flags = info.flags;
    EP_HIP(epk::launch_product(a, activation == EP_ACT_SWIGLU ? epk::kSwigluBf16 : epk::kStoreBf16,
                               static_cast<hipStream_t>(stream)));
    return EP_OK;
}

ep_status ep_moe_workspace_size(const ep_handle* h, const ep_weights* w_up,
                                const ep_weights* w_down, int64_t num_tokens, int64_t* bytes)
{
    epk::HandleInfo info;
    ep_status st = check_layer(h, w_up, w_down, num_tokens, false, &info);
    if (st != EP_OK) return st;
    if (!bytes) return EP_FAIL(EP_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = carve_layer(num_tokens * info.cfg->num_topk, w_down->cols, info.cfg->hidden).total;
    return EP_OK;
}

ep_status ep_moe_layer(const ep_handle* h, const ep_weights* w_up, const ep_weights* w_down,
                       const void* d_x, const int32_t* d_topk_idx, const float* d_topk_weights,
                       int64_t num_tokens, void* d_out, void* d_workspace, int64_t workspace_bytes,
                       void* stream)
{
    epk::HandleInfo info;
    ep_status st = check_layer(h, w_up, w_down, num_tokens, true, &info);
    if (st != EP_OK || num_tokens == 0) return st;
    const ep_config& c = *info.cfg;
    if (!d_x || !d_topk_idx || !d_out)
        return EP_FAIL(EP_ERR_INVALID_ARG, "x, topk_idx or out is NULL");
    if (!aligned(d_x, 16) || !aligned(d_out, 16) || !aligned(d_topk_idx, 4) ||
        !aligned(d_topk_weights, 4))
        return EP_FAIL(EP_ERR_INVALID_ARG,
                       "x and out must be 16-byte aligned, topk_idx and topk_weights 4-byte aligned");
    const int64_t pairs = num_tokens * c.num_topk;
    const LayerCarve cv = carve_layer(pairs, w_down->cols, c.hidden);
    if (!d_workspace || !aligned(d_workspace, 256))
        return EP_FAIL(EP_ERR_WORKSPACE, "workspace must be 256-byte aligned and not NULL");
    if (workspace_bytes < cv.total)
        return EP_FAIL(EP_ERR_WORKSPACE, "workspace has %lld bytes, needs %lld",
                       (long long)workspace_bytes, (long long)cv.total);
    unsigned char* ws = static_cast<unsigned char*>(d_workspace);
    const hipStream_t s = static_cast<hipStream_t>(stream);

    epk::ProductArgs up = {};
    up.w = weight_args(w_up);
    up.E = c.num_experts;
    up.units = w_up->rows / 2;
    up.topk = d_topk_idx;
    up.P = (int)pairs;
    up.K = c.num_topk;
    up.x_per_pair = false;
    up.weights = d_topk_weights;
    up.x = static_cast<const uint16_t*>(d_x);
    up.ldx = c.hidden;
    up.y = ws + cv.act;
    up.y_lo = reinterpret_cast<uint16_t*>(ws + cv.act_lo);
    up.ldy = up.units;
    up.flags = info.flags;
    EP_HIP(epk::launch_product(up, epk::kSwigluSplit, s));

    epk::ProductArgs down = {};
    down.w = weight_args(w_down);
    down.E = c.num_experts;
    down.units = c.hidden;
    down.topk = d_topk_idx;
    down.P = (int)pairs;
    down.K = c.num_topk;
    down.x_per_pair = true;
    down.x = reinterpret_cast<const uint16_t*>(ws + cv.act);
    down.x_lo = reinterpret_cast<const uint16_t*>(ws + cv.act_lo);
    down.ldx = w_down->cols;
    down.ldy = c.hidden;
    down.flags = info.flags;
    down.y = d_out;
    bool done = false;
    EP_HIP(epk::launch_down_few(down, &done, s));
    if (done) return EP_OK;
    down.y = ws + cv.y;
    EP_HIP(epk::launch_product(down, epk::kStoreF32, s));

    epk::ReduceArgs r = {};
    r.y = reinterpret_cast<const float*>(ws + cv.y);
    r.topk = d_topk_idx;
    r.N = (int)num_tokens;
    r.K = c.num_topk;
    r.E = c.num_experts;
    r.H = c.hidden;
    r.out = static_cast<uint16_t*>(d_out);
    EP_HIP(epk::launch_layer_reduce(r, s));
    return EP_OK;
}

}  // extern "C"
