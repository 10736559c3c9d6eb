// The router on gfx950: scores, the (group-limited) choice of K experts, their
// weights, and the weights' gradient.
//
// What is computed, per token with logits l:
//   s = softmax(l) or sigmoid(l); choice = s + bias;
//   groups: score = the sum of a group's best group_top choices; the best
//   topk_groups groups keep their experts;
//   the K best choices, highest first, ties to the lower id;
//   w = scale * s[idx] (/ their sum).
// A choice is a whole number, so it has to be right where two experts all but
// tie: order is decided in fp64, or by the logits themselves where no bias
// enters (s is strictly increasing in l).
#include "experts.hpp"

namespace epk {
namespace {

constexpr int kGateWaves = 4;
constexpr double kNone = -__builtin_huge_val();

__device__ __forceinline__ float load_logit(const void* p, bool bf16, int64_t i)
{
    if (bf16) return __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(p)[i] << 16);
    return reinterpret_cast<const float*>(p)[i];
}

// NaN and -infinity: -infinity (not eligible); +infinity: the largest float.
__device__ __forceinline__ float clean_logit(float l)
{
    return l == l ? fminf(l, 3.402823466e38f) : -__builtin_huge_valf();
}

__device__ __forceinline__ double wave_sum(double v)
{
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

__device__ __forceinline__ float wave_max(float v)
{
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
    return v;
}

// Highest key of the wave, ties to the lower id; every lane gets both.
__device__ __forceinline__ void wave_best(double& key, int& id)
{
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) {
        const double k = __shfl_xor(key, d);
        const int i = __shfl_xor(id, d);
        if (k > key || (k == key && i < id)) {
            key = k;
            id = i;
        }
    }
}

// One wave per token; lane l holds experts l, l + 64, ...
template <int VPL>
__global__ __launch_bounds__(kGateWaves* kWave) void k_gate(GateArgs a)
{
    __shared__ double choice_lds[kGateWaves][VPL * kWave];
    __shared__ double key_lds[kGateWaves][VPL * kWave];
    __shared__ uint8_t out_lds[kGateWaves][VPL * kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int64_t t = (int64_t)blockIdx.x * kGateWaves + wave;
    if (t >= a.N) return;
    int32_t* const idx = a.idx + t * a.K;
    float* const w = a.w + t * a.K;
    if (a.mask && a.mask[t] == 0) {
        if (lane < a.K) {
            idx[lane] = -1;
            w[lane] = 0.f;
        }
        return;
    }
    float l[VPL];
    float top = -__builtin_huge_valf();
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = lane + kWave * i;
        l[i] = e < a.E ? clean_logit(load_logit(a.logits, a.bf16, t * a.E + e)) : -__builtin_huge_valf();
        top = fmaxf(top, l[i]);
    }
    top = wave_max(top);
    const bool any = top > -__builtin_huge_valf();

    // scores in 64 bits
    double s[VPL], key[VPL];
    double total = 0.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const bool ok = l[i] > -__builtin_huge_valf();
        s[i] = !ok ? 0.0
               : a.scoring == 0 ? exp((double)l[i] - (double)top) : 1.0 / (1.0 + exp(-(double)l[i]));
        total += s[i];
    }
    if (a.scoring == 0 && any) {
        total = wave_sum(total);
#pragma unroll
        for (int i = 0; i < VPL; ++i) s[i] /= total;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = lane + kWave * i;
        const bool ok = l[i] > -__builtin_huge_valf();
        double c = ok ? s[i] : kNone;
        if (a.bias && ok) c += (double)a.bias[e];
        if (!(c > kNone)) c = kNone;
        key[i] = a.bias ? c : ok ? (double)l[i] : kNone;
        if (a.groups > 1) {
            choice_lds[wave][e] = c;
            key_lds[wave][e] = key[i];
            out_lds[wave][e] = 1;
        }
    }
    if (a.groups > 1) {
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        const int per = a.E / a.groups;
        double score = kNone;
        if (lane < a.groups) {
            // the best group_top members in order: each the first after the last
            double lk = __builtin_huge_val();
            int li = -1;
            bool got = false;
            double sum = 0.0;
            for (int m = 0; m < a.group_top; ++m) {
                double bk = kNone;
                int bi = -1;
                for (int j = 0; j < per; ++j) {
                    const int e = lane * per + j;
                    const double k = key_lds[wave][e];
                    const bool after = li < 0 || k < lk || (k == lk && e > li);
                    if (after && k > bk) {
                        bk = k;
                        bi = e;
                    }
                }
                if (bi < 0) break;
                sum += choice_lds[wave][bi];
                if (a.limit) out_lds[wave][bi] = 2;
                got = true;
                lk = bk;
                li = bi;
            }
            if (got) score = sum;
        }
        uint64_t used = 0;      // the same in every lane
        for (int r = 0; r < a.topk_groups; ++r) {
            double k = lane < a.groups && !(used >> lane & 1) ? score : kNone;
            int id = lane;
            wave_best(k, id);
            if (k > kNone) used |= 1ull << id;
        }
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int e = lane + kWave * i;
            const int group = e < a.E ? e / per : 0;
            const uint32_t keeps = (uint32_t)(used >> group) & (a.limit ? out_lds[wave][e] >> 1 : 1u);
            key[i] = (keeps & 1u) != 0u ? key[i] : kNone;
        }
    }

    // K times the best that is left
    int my_id = -1;
    float my_l = 0.f;
    double my_s = 0.0;
    for (int k = 0; k < a.K; ++k) {
        double bk = kNone;
        int bi = kMaxExperts;
        float bl = 0.f;
        double bs = 0.0;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (key[i] > bk) {
                bk = key[i];
                bi = lane + kWave * i;
                bl = l[i];
                bs = s[i];
            }
        double wk = bk;
        int wi = bi;
        wave_best(wk, wi);
        if (!(wk > kNone)) break;
        const int from = wi & (kWave - 1);
        const float l_of = __shfl(bl, from);
        const double s_of = __shfl(bs, from);
        if (lane == k) {
            my_id = wi;
            my_l = l_of;
            my_s = s_of;
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (lane + kWave * i == wi) key[i] = kNone;
    }
    const bool live = my_id >= 0;
    double v = live ? my_s : 0.0;
    if (a.renorm) {
        // over the chosen alone; in the logits' differences where the scores
        // have run out of range
        const float lm = wave_max(live ? my_l : -__builtin_huge_valf());
        double sum = wave_sum(v);
        if (a.scoring == 0 || !(sum > 0.0)) {
            v = live ? exp((double)my_l - (double)lm) : 0.0;
            sum = wave_sum(v);
        }
        v = live ? v / sum : 0.0;
    }
    if (lane < a.K) {
        idx[lane] = my_id;
        w[lane] = live ? (float)(v * (double)a.scale) : 0.f;
    }
}

// Gradient: one wave per token.  With p the weights over scale,
//   softmax:              dl_e = p_e * (sum of g over entries with idx e - sum g p)
//   normalised softmax:   the same over the chosen entries alone
//   sigmoid:              dl_e = sum over entries of g * s (1 - s)
//   normalised sigmoid:   dl_e = sum over entries of p (1 - s) (g - sum g p)
// HBM-bound: one pass over the logits (only the raw softmax needs them all),
// one over the gradient.
template <int VPL>
__global__ __launch_bounds__(kGateWaves* kWave) void k_gate_backward(GateArgs a)
{
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int64_t t = (int64_t)blockIdx.x * kGateWaves + wave;
    if (t >= a.N) return;
    const int64_t base = t * a.E;
    const float kLow = -__builtin_huge_valf();
    int id = lane < a.K ? a.idx_in[t * a.K + lane] : -1;
    if ((uint32_t)id >= (uint32_t)a.E) id = -1;
    const float g = id >= 0 ? a.grad_w[t * a.K + lane] * a.scale : 0.f;
    const float lc = id >= 0 ? clean_logit(load_logit(a.logits, a.bf16, base + id)) : kLow;
    const bool full = a.scoring == 0 && !a.renorm;      // every expert's logit matters

    float p[VPL];
    float pc = 0.f;     // this entry's p
    if (full) {
        float top = kLow;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int e = lane + kWave * i;
            p[i] = e < a.E ? clean_logit(load_logit(a.logits, a.bf16, base + e)) : kLow;
            top = fmaxf(top, p[i]);
        }
        top = wave_max(top);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            p[i] = p[i] > kLow ? expf(p[i] - top) : 0.f;
            sum += p[i];
        }
        sum = wave_sum(sum);
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) p[i] *= inv;
        pc = lc > kLow ? expf(lc - top) * inv : 0.f;
    } else {
        // log of the score up to a constant: l, or log sigmoid(l)
        const float ls = !(lc > kLow) ? kLow
                         : a.scoring == 0 ? lc : fminf(lc, 0.f) - log1pf(expf(-fabsf(lc)));
        if (a.renorm) {
            const float top = wave_max(ls);
            pc = ls > kLow ? expf(ls - top) : 0.f;
            const float sum = wave_sum(pc);
            pc = sum > 0.f ? pc / sum : 0.f;
        } else {
            pc = ls > kLow ? expf(ls) : 0.f;
        }
    }
    const float dot = full || a.renorm ? wave_sum(g * pc) : 0.f;
    // this entry's share of its expert's gradient
    float d;
    if (full) d = g;
    else if (a.scoring == 0) d = pc * (g - dot);
    else {
        // 1 - s = sigmoid(-l)
        const float q = lc > 0.f ? expf(-lc) / (1.f + expf(-lc)) : 1.f / (1.f + expf(lc));
        d = pc * q * (a.renorm ? g - dot : g);
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = lane + kWave * i;
        float v = 0.f;
        for (int k = 0; k < a.K; ++k) {
            const int ik = __builtin_amdgcn_readlane(id, k);
            const float dk = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(d), k));
            if (ik == e) v += dk;
        }
        if (full) v = p[i] * (v - dot);
        if (e < a.E) {
            if (a.bf16) {
                typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
                typedef float f32x2 __attribute__((ext_vector_type(2)));
                reinterpret_cast<uint16_t*>(a.grad_logits)[base + e] = (uint16_t)__builtin_bit_cast(
                    uint32_t, __builtin_convertvector(f32x2{v, 0.f}, bf16x2));
            } else {
                reinterpret_cast<float*>(a.grad_logits)[base + e] = v;
            }
        }
    }
}

template <bool BACK, int VPL>
hipError_t launch_vpl(const GateArgs& a, hipStream_t s)
{
    const dim3 grid((unsigned)((a.N + kGateWaves - 1) / kGateWaves)), block(kGateWaves * kWave);
    if constexpr (BACK) hipLaunchKernelGGL(k_gate_backward<VPL>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(k_gate<VPL>, grid, block, 0, s, a);
    return hipGetLastError();
}

template <bool BACK>
hipError_t launch_any(const GateArgs& a, hipStream_t s)
{
    if (a.E <= 64) return launch_vpl<BACK, 1>(a, s);
    if (a.E <= 128) return launch_vpl<BACK, 2>(a, s);
    if (a.E <= 256) return launch_vpl<BACK, 4>(a, s);
    if (a.E <= 512) return launch_vpl<BACK, 8>(a, s);
    return launch_vpl<BACK, 16>(a, s);
}

}  // namespace

hipError_t launch_gate(const GateArgs& a, hipStream_t s) { return launch_any<false>(a, s); }
hipError_t launch_gate_backward(const GateArgs& a, hipStream_t s) { return launch_any<true>(a, s); }

}  // namespace epk
