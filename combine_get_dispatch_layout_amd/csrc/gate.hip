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
constexpr int kMaxGroups = 64;
constexpr double kNone = -__builtin_huge_val();

// Blocks of one row of the grid, which holds fewer than 2^32 threads: 2^26
// tokens and more take several rows.
constexpr int64_t kGridRow = 1 << 20;

// The block's first token.
__device__ __forceinline__ int64_t first_token()
{
    return ((int64_t)blockIdx.y * kGridRow + blockIdx.x) * kGateWaves;
}

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

template <int CTRL>
__device__ __forceinline__ float dpp(float x)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xF, 0xF, false));
}

__device__ __forceinline__ float lane_value(float v, int lane)
{
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

// Largest of the wave: four steps inside the rows of 16 lanes (quad_perm
// [1,0,3,2] and [2,3,0,1], row_half_mirror, row_mirror), then the four rows.
__device__ __forceinline__ float wave_max(float v)
{
    v = fmaxf(v, dpp<0xB1>(v));
    v = fmaxf(v, dpp<0x4E>(v));
    v = fmaxf(v, dpp<0x141>(v));
    v = fmaxf(v, dpp<0x140>(v));
    return fmaxf(fmaxf(lane_value(v, 0), lane_value(v, 16)), fmaxf(lane_value(v, 32), lane_value(v, 48)));
}

__device__ __forceinline__ float wave_sum(float v)
{
    v += dpp<0xB1>(v);
    v += dpp<0x4E>(v);
    v += dpp<0x141>(v);
    v += dpp<0x140>(v);
    return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}

__device__ __forceinline__ double wave_sum(double v)
{
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// The lane whose (key, id) is the wave's highest, ties to the lower id; -1 if
// every key is -infinity.  Rounding to fp32 keeps the order, so one fp32
// maximum decides unless several lanes round to it; those are compared in 64
// bits.
__device__ __forceinline__ int wave_best(double key, int id)
{
    const float k = (float)key;
    const float top = wave_max(k);
    const bool any = key > kNone;
    uint64_t with = __ballot(any && k == top);
    if (with == 0) with = __ballot(any);     // all below fp32's range
    if (with == 0) return -1;
    int best = (int)__builtin_ctzll(with);
    for (with &= with - 1; with != 0; with &= with - 1) {
        const int l = (int)__builtin_ctzll(with);
        const double kb = __shfl(key, best), kl = __shfl(key, l);
        const int ib = __builtin_amdgcn_readlane(id, best), il = __builtin_amdgcn_readlane(id, l);
        if (kl > kb || (kl == kb && il < ib)) best = l;
    }
    return __builtin_amdgcn_readfirstlane(best);
}

__device__ __forceinline__ double score_of(int scoring, float l, float top, double total)
{
    return scoring == 0 ? exp((double)l - (double)top) / total : 1.0 / (1.0 + exp(-(double)l));
}

// One wave per token; lane l holds experts l, l + 64, ...
// What bounds it: 64-bit arithmetic.  Every score in fp64 costs an exponential
// and a division, so they are made only where a choice needs them (a bias,
// groups) or the weights do (the softmax's sum); else the logits are the keys
// and only the chosen experts' scores are computed, one a lane.  8192 tokens,
// 256 experts in 32 groups, sigmoid and bias: 20.7 us (33.7 with 64-bit
// exchanges in every reduction and all experts in the last search); without
// groups 4096 tokens, 128 experts, softmax, 8.1 us, one token 4.9 us (9.9).
template <int VPL>
__global__ __launch_bounds__(kGateWaves* kWave) void k_gate(GateArgs a)
{
    // groups only; expert e at e + its group, so that the lanes of the search,
    // one a group, start in different banks
    constexpr int kSlots = VPL * kWave + kMaxGroups;
    __shared__ double choice_lds[kGateWaves][kSlots];
    __shared__ double key_lds[kGateWaves][kSlots];
    __shared__ float logit_lds[kGateWaves][kSlots];
    __shared__ uint8_t out_lds[kGateWaves][kSlots];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t t = first_token() + wave;
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
    constexpr float kLow = -__builtin_huge_valf();
    float l[VPL];
    float top = kLow;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = lane + kWave * i;
        l[i] = e < a.E ? clean_logit(load_logit(a.logits, a.bf16, t * a.E + e)) : kLow;
        top = fmaxf(top, l[i]);
    }
    const bool groups = a.groups > 1;
    const bool choose = a.bias != nullptr || groups;            // by scores
    double total = 1.0;
    if (a.scoring == 0 && (choose || !a.renorm)) {
        top = wave_max(top);
        total = 0.0;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (l[i] > kLow) total += exp((double)l[i] - (double)top);
        total = wave_sum(total);
    }

    auto group_of = [&](int e) { return a.per_magic ? (int)__umulhi((uint32_t)e, a.per_magic) : e; };
    double key[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = l[i] > kLow ? (double)l[i] : kNone;
    if (choose) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int e = lane + kWave * i;
            double c = kNone;
            if (l[i] > kLow) {
                c = score_of(a.scoring, l[i], top, total);
                if (a.bias) c += (double)a.bias[e];
                if (!(c > kNone)) c = kNone;
            }
            if (a.bias) key[i] = c;
            if (groups && e < a.E) {
                const int to = e + group_of(e);
                choice_lds[wave][to] = c;
                key_lds[wave][to] = key[i];
                logit_lds[wave][to] = l[i];
                out_lds[wave][to] = 1;
            }
        }
    }
    double bk = kNone;      // this lane's best, its expert and its logit
    int bi = kMaxExperts;
    float bl = 0.f;
    bool packed = false;    // the lane has that one candidate at most
    if (groups) {
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        const int per = a.per;
        double score = kNone;
        if (lane < a.groups) {
            // the best group_top members in order, two a pass: those after the
            // last pair.  Going up in e, a later equal key never comes first.
            double lk = __builtin_huge_val();
            int li = -1;
            double sum = 0.0;
            const int base = lane * (per + 1);
            for (int m = 0; m < a.group_top; m += 2) {
                double k1 = kNone, k2 = kNone;
                int i1 = -1, i2 = -1;
#pragma unroll 4
                for (int j = 0; j < per; ++j) {
                    const double kj = key_lds[wave][base + j];
                    const bool after = li < 0 || kj < lk || (kj == lk && j > li);
                    const double k = after ? kj : kNone;
                    const bool best = k > k1, second = k > k2;
                    k2 = best ? k1 : second ? k : k2;
                    i2 = best ? i1 : second ? j : i2;
                    k1 = best ? k : k1;
                    i1 = best ? j : i1;
                }
                if (i1 < 0) break;
                sum += choice_lds[wave][base + i1];
                if (a.limit) out_lds[wave][base + i1] = 2;
                score = sum;
                if (i2 < 0 || m + 1 == a.group_top) break;
                sum += choice_lds[wave][base + i2];
                if (a.limit) out_lds[wave][base + i2] = 2;
                score = sum;
                lk = k2;
                li = i2;
            }
        }
        uint64_t used = 0;      // the same in every lane
        for (int r = 0; r < a.topk_groups; ++r) {
            const int best = wave_best(used >> lane & 1 ? kNone : score, lane);
            if (best < 0) break;
            used |= 1ull << best;
        }
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        // if the used groups' members fit the wave, one a lane: in the order of
        // their groups, so of their ids
        packed = a.topk_groups * per <= kWave;
        if (packed) {
            const int r = group_of(lane), j = lane - r * per;
            int group = -1;
            uint64_t left = used;
            for (int q = 0; q < a.topk_groups && left != 0; ++q, left &= left - 1)
                group = r == q ? (int)__builtin_ctzll(left) : group;
            const int at = group >= 0 ? group * (per + 1) + j : 0;
            const bool in = group >= 0 && (!a.limit || out_lds[wave][at] == 2);
            const double k = key_lds[wave][at];
            bk = in ? k : kNone;
            bi = in ? group * per + j : kMaxExperts;
            bl = logit_lds[wave][at];
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                const int e = lane + kWave * i;
                const int at = e < a.E ? e : 0, group = group_of(at);
                const uint32_t keeps = (uint32_t)(used >> group) & (a.limit ? out_lds[wave][at + group] >> 1 : 1u);
                key[i] = (keeps & 1u) != 0u ? key[i] : kNone;
            }
        }
    }

    // K times the best that is left; lane k keeps the k-th
    int my_id = -1;
    float my_l = 0.f;
    auto local_best = [&] {
        bk = kNone;
        bi = kMaxExperts;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const bool more = key[i] > bk;
            bk = more ? key[i] : bk;
            bi = more ? lane + kWave * i : bi;
            bl = more ? l[i] : bl;
        }
    };
    if (!packed) local_best();
    for (int k = 0; k < a.K; ++k) {
        const int from = wave_best(bk, bi);
        if (from < 0) break;
        const int id = __builtin_amdgcn_readlane(bi, from);
        const float lv = lane_value(bl, from);
        my_id = lane == k ? id : my_id;
        my_l = lane == k ? lv : my_l;
        if (packed) {
            bk = lane == from ? kNone : bk;
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i) key[i] = lane + kWave * i == id ? kNone : key[i];
            local_best();
        }
    }
    const bool live = my_id >= 0;
    double v = 0.0;
    if (a.scoring != 0 || !a.renorm) v = live ? score_of(a.scoring, my_l, top, total) : 0.0;
    if (a.renorm) {
        // over the chosen alone; in the logits' differences for a softmax, and
        // where sigmoids have run out of range
        const float lm = wave_max(live ? my_l : kLow);
        double sum = a.scoring != 0 ? wave_sum(v) : 0.0;
        if (!(sum > 0.0)) {
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
// one over the gradient, in vectors of four experts where rows allow it.  8191
// tokens, 256 experts, fp32: 7.8 us as a graph (9.9 with single stores), 2.2
// TB/s; 8.3 to 8.5 us in a kernel trace.
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

template <int VPL>
__global__ __launch_bounds__(kGateWaves* kWave) void k_gate_backward(GateArgs a)
{
    constexpr int V = VPL < 4 ? VPL : 4;            // neighbours in a lane
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t t = first_token() + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    if (t >= a.N) return;
    const int64_t base = t * a.E;
    const float kLow = -__builtin_huge_valf();
    auto expert = [&](int i) { return i / V * (kWave * V) + lane * V + i % V; };
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
            const int e = expert(i);
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
    float v[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] = 0.f;
    for (int k = 0; k < a.K; ++k) {
        const int ik = __builtin_amdgcn_readlane(id, k);
        const float dk = lane_value(d, k);
#pragma unroll
        for (int i = 0; i < VPL; ++i) v[i] += ik == expert(i) ? dk : 0.f;
    }
    if (full)
#pragma unroll
        for (int i = 0; i < VPL; ++i) v[i] = p[i] * (v[i] - dot);
#pragma unroll
    for (int i = 0; i < VPL; i += V) {
        const int e = expert(i);
        if (V == 4 && a.vec) {       // E % 4 == 0: whole or not at all
            if (e >= a.E) continue;
            if (a.bf16)
                *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(a.grad_logits) + base + e) =
                    u32x2{pack_bf16(v[i], v[i + 1 < VPL ? i + 1 : i]),
                          pack_bf16(v[i + 2 < VPL ? i + 2 : i], v[i + 3 < VPL ? i + 3 : i])};
            else
                *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(a.grad_logits) + base + e) =
                    f32x4{v[i], v[i + 1 < VPL ? i + 1 : i], v[i + 2 < VPL ? i + 2 : i],
                          v[i + 3 < VPL ? i + 3 : i]};
            continue;
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (e + j >= a.E) continue;
            if (a.bf16)
                reinterpret_cast<uint16_t*>(a.grad_logits)[base + e + j] = (uint16_t)pack_bf16(v[i + j], 0.f);
            else
                reinterpret_cast<float*>(a.grad_logits)[base + e + j] = v[i + j];
        }
    }
}

template <bool BACK, int VPL>
hipError_t launch_vpl(const GateArgs& a, hipStream_t s)
{
    const int64_t blocks = (a.N + kGateWaves - 1) / kGateWaves, row = blocks < kGridRow ? blocks : kGridRow;
    const dim3 grid((unsigned)row, (unsigned)((blocks + row - 1) / row)), block(kGateWaves * kWave);
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
