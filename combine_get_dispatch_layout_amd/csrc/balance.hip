// The balance loss of a router on gfx950: per-expert counts, sums of scores,
// the loss they make, and its gradient with respect to the logits.
//
// With V_q the unmasked tokens of sequence q, T_q their number, count[q,e] the
// entries of their topk_idx that name e, and p the scores:
//   S[q,e] = sum over t in V_q of p[t,e]
//   loss   = coefficient / Q * sum_q E / (K T_q^2) * sum_e count[q,e] S[q,e]
//
// What bounds it: one reading of the logits (the gradient: and one writing),
// for small batches the launches.
//
// A token's experts lie in 16 lanes (64 above 256 experts), sixteen or fewer to
// a lane: a reduction over them is four steps inside a row of lanes, for four
// tokens at once, and sums over tokens stay in registers.
//
// Results do not depend on the order of blocks: a block writes what its chunk
// of tokens adds to each sequence it touches, a second kernel adds those pieces
// up in order, in 64 bits.  The piece of chunk c and sequence q has the slot
// c + q: along the batch one of the two grows from piece to piece, so no two
// pieces share a slot, and a sequence's slots are consecutive.
#include "balance.hpp"

#include "router.hpp"

namespace epk {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = kWaves * kWave;

// A chunk: at least 16 tokens (four waves of four), so many that some 1024
// blocks make the batch, at most 1024 (which bounds the fp32 sums' length).
constexpr int kMinChunk = 16, kMaxChunk = 1024, kChunks = 1024;

constexpr float kLow = -__builtin_huge_valf();

// exp(x) for x <= 0, off by an ulp or two: the rounding of x log2(e), which
// the hardware's exp2 would magnify, is put right to first order.
__device__ __forceinline__ float exp_neg(float x)
{
    constexpr float kHi = 1.44269502f, kLo = 1.92596299e-8f;      // log2(e)
    x = fmaxf(x, -200.f);
    const float y = x * kHi;
    const float rest = fmaf(x, kLo, fmaf(x, kHi, -y));
    const float r = __builtin_amdgcn_exp2f(y);
    return fmaf(r, rest * 0.693147181f, r);
}

__device__ __forceinline__ float reciprocal(float d)
{
    const float r = __builtin_amdgcn_rcpf(d);
    return fmaf(fmaf(-d, r, 1.f), r, r);
}

template <int LANES>
__device__ __forceinline__ float lanes_max(float v)
{
    if constexpr (LANES == 64) return wave_max(v);
    v = fmaxf(v, dpp<0xB1>(v));
    v = fmaxf(v, dpp<0x4E>(v));
    v = fmaxf(v, dpp<0x141>(v));
    return fmaxf(v, dpp<0x140>(v));
}

template <int LANES>
__device__ __forceinline__ float lanes_sum(float v)
{
    if constexpr (LANES == 64) return wave_sum(v);
    v += dpp<0xB1>(v);
    v += dpp<0x4E>(v);
    v += dpp<0x141>(v);
    return v + dpp<0x140>(v);
}

// How a token's experts lie in LANES lanes: vector v of lane l holds the four
// experts from 4 (v LANES + l) on.
template <int LANES, int VECS>
struct Experts {
    static constexpr int kEach = 4 * VECS;           // of a lane
    static constexpr int kTokens = kWave / LANES;    // of a wave at a time
    static constexpr int kMost = LANES * kEach;

    static __device__ __forceinline__ int first(int lane, int v) { return 4 * (v * LANES + lane % LANES); }

    // Logits of token t as they are; -infinity past the last expert.
    static __device__ __forceinline__ void load(const BalanceArgs& a, int64_t t, float (&z)[kEach])
    {
        const int lane = threadIdx.x & (kWave - 1);
#pragma unroll
        for (int v = 0; v < VECS; ++v) {
            const int e = first(lane, v);
            const int64_t at = t * a.E + e;
#pragma unroll
            for (int j = 0; j < 4; ++j) z[4 * v + j] = kLow;
            if (a.vec) {        // E % 4 == 0: whole or not at all
                if (e >= a.E) continue;
                if (a.bf16) {
                    const u32x2 d = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(a.logits) + at);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        z[4 * v + j] = __uint_as_float(j % 2 ? d[j / 2] & 0xFFFF0000u : d[j / 2] << 16);
                } else {
                    const f32x4 d = *reinterpret_cast<const f32x4*>(static_cast<const float*>(a.logits) + at);
#pragma unroll
                    for (int j = 0; j < 4; ++j) z[4 * v + j] = d[j];
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (e + j < a.E) z[4 * v + j] = load_logit(a.logits, a.bf16, at + j);
            }
        }
    }

    // Logits to scores; of a sigmoid also 1 - s where GRAD asks for it.
    template <bool GRAD>
    static __device__ __forceinline__ void scores(const BalanceArgs& a, float (&z)[kEach], float (&rest)[GRAD ? kEach : 1])
    {
        float top = kLow;
#pragma unroll
        for (int i = 0; i < kEach; ++i) z[i] = clean_logit(z[i]);
        const bool divide = a.scoring == 0 || a.normalize;
        if (divide) {
#pragma unroll
            for (int i = 0; i < kEach; ++i) top = fmaxf(top, z[i]);
            top = lanes_max<LANES>(top);
        }
        float total = 0.f;
        if (a.scoring == 0) {
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                z[i] = z[i] > kLow ? exp_neg(z[i] - top) : 0.f;
                total += z[i];
            }
        } else {
            // normalised sigmoids that have all but run out of range go in
            // proportion to their exponentials, from the largest one down
            const bool far = divide && top < -64.f;
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const bool in = z[i] > kLow;
                const float x = exp_neg(-fabsf(z[i]));
                const float r = reciprocal(1.f + x);
                if constexpr (GRAD) rest[i] = z[i] >= 0.f ? x * r : r;
                float s = z[i] >= 0.f ? r : x * r;
                if (far) s = exp_neg(z[i] - top);
                z[i] = in ? s : 0.f;
                total += z[i];
            }
        }
        if (divide) {
            total = lanes_sum<LANES>(total);
            const float inv = total > 0.f ? reciprocal(total) : 0.f;
#pragma unroll
            for (int i = 0; i < kEach; ++i) z[i] *= inv;
        }
    }
};

// start[i], held inside the batch.
__device__ __forceinline__ int64_t start_of(const BalanceArgs& a, int64_t i)
{
    const int64_t s = a.start[i];
    return s < 0 ? 0 : s < a.N ? s : a.N;
}

// The first sequence that ends behind token t (Q if none does): the wave
// probes 64 ends at a time.
__device__ __forceinline__ int first_sequence(const BalanceArgs& a, int64_t t)
{
    const int lane = threadIdx.x & (kWave - 1);
    int lo = 0, n = a.Q;        // it is in [lo, lo + n]
    while (n > 0) {
        const int step = (n + kWave - 1) / kWave;
        const int at = lo + min((lane + 1) * step, n) - 1;
        const uint64_t behind = __ballot(start_of(a, (int64_t)at + 1) > t);
        if (behind == 0) return lo + n;
        // the probe before the first hit ends at or before t
        const int hit = (int)__builtin_ctzll(behind);
        const int to = lo + min((hit + 1) * step, n) - 1;
        lo += hit * step;
        n = to - lo;
    }
    return lo;
}

// Adds up each piece of the block's chunk: scores, entries, tokens.
template <int LANES, int VECS>
__global__ __launch_bounds__(kThreads) void k_balance_pieces(BalanceArgs a)
{
    using X = Experts<LANES, VECS>;
    __shared__ float sums[kWaves][X::kMost];
    __shared__ int counts[X::kMost];
    __shared__ int tokens[kWaves];
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    if (blockIdx.x == 0 && tid == 0) *a.ticket = 0;
    const int64_t c0 = (int64_t)blockIdx.x * a.chunk;
    const int64_t c1 = c0 + a.chunk < a.N ? c0 + a.chunk : a.N;

    for (int q = a.start ? first_sequence(a, c0) : 0; q < a.Q; ++q) {
        const int64_t s0 = a.start ? start_of(a, q) : 0, s1 = a.start ? start_of(a, (int64_t)q + 1) : a.N;
        if (s0 >= c1) break;
        const int64_t t0 = s0 > c0 ? s0 : c0, t1 = s1 < c1 ? s1 : c1;
        if (t0 >= t1) continue;

        for (int e = tid; e < X::kMost; e += kThreads) counts[e] = 0;
        __syncthreads();
        const int entries = (int)(t1 - t0) * a.K;
        for (int i = tid; i < entries; i += kThreads) {
            const int t = a.k_magic ? (int)__umulhi((uint32_t)i, a.k_magic) : i;
            if (a.mask && a.mask[t0 + t] == 0) continue;
            const int e = a.topk[t0 * a.K + i];
            if ((uint32_t)e < (uint32_t)a.E) atomicAdd(&counts[e], 1);
        }

        float acc[X::kEach], z[X::kEach], next[X::kEach], none[1];
#pragma unroll
        for (int i = 0; i < X::kEach; ++i) acc[i] = 0.f;
        int live = 0;
        const int64_t mine = t0 + wave * X::kTokens + lane / LANES;
        auto counted = [&](int64_t t) { return t < t1 && (!a.mask || a.mask[t] != 0); };
        bool in = counted(mine);
        if (in) X::load(a, mine, next);
        for (int64_t t = mine; t - lane / LANES < t1; t += kWaves * X::kTokens) {
            const bool now = in;
#pragma unroll
            for (int i = 0; i < X::kEach; ++i) z[i] = next[i];
            in = counted(t + kWaves * X::kTokens);
            if (in) X::load(a, t + kWaves * X::kTokens, next);
            live += (int)__popcll(__ballot(now)) / LANES;
            if (now) {
                X::template scores<false>(a, z, none);
#pragma unroll
                for (int i = 0; i < X::kEach; ++i) acc[i] += z[i];
            }
        }
#pragma unroll
        for (int i = 0; i < X::kEach; ++i)
#pragma unroll
            for (int d = LANES; d < kWave; d *= 2) acc[i] += __shfl_xor(acc[i], d);
        if (lane < LANES)
#pragma unroll
            for (int i = 0; i < X::kEach; ++i) sums[wave][X::first(lane, i / 4) + i % 4] = acc[i];
        if (lane == 0) tokens[wave] = live;
        __syncthreads();
        const int64_t slot = (int64_t)blockIdx.x + q;
        for (int e = tid; e < a.E; e += kThreads) {
            a.part_sum[slot * a.E + e] = (sums[0][e] + sums[1][e]) + (sums[2][e] + sums[3][e]);
            a.part_count[slot * a.E + e] = counts[e];
        }
        if (tid == 0) a.part_tokens[slot] = (tokens[0] + tokens[1]) + (tokens[2] + tokens[3]);
        __syncthreads();
    }
}

// Adds up a sequence's pieces for `slice` experts; the last block to finish
// adds up the blocks' shares of the loss, in their order.
__global__ __launch_bounds__(kThreads) void k_balance_finish(BalanceArgs a, int slice, int slices)
{
    __shared__ double sums[kThreads];
    __shared__ int counts[kThreads];
    __shared__ bool last;
    const int tid = threadIdx.x;
    const int q = blockIdx.x / slices, e0 = (blockIdx.x % slices) * slice;
    const int64_t s0 = a.start ? start_of(a, q) : 0, s1 = a.start ? start_of(a, (int64_t)q + 1) : a.N;
    const int64_t first = s0 / a.chunk, pieces = s1 > s0 ? (s1 - 1) / a.chunk - first + 1 : 0;
    const int64_t slot0 = first + q;

    int live = 0;
    for (int64_t i = tid; i < pieces; i += kThreads) live += a.part_tokens[slot0 + i];
    const int e = e0 + tid % slice, at = tid / slice, step = kThreads / slice;
    double sum = 0.0;
    int count = 0;
    if (e < a.E)
#pragma unroll 4
        for (int64_t i = at; i < pieces; i += step) {
            sum += (double)a.part_sum[(slot0 + i) * a.E + e];
            count += a.part_count[(slot0 + i) * a.E + e];
        }
    counts[tid] = live;
    __syncthreads();
    for (int d = kThreads / 2; d > 0; d /= 2) {
        if (tid < d) counts[tid] += counts[tid + d];
        __syncthreads();
    }
    live = counts[0];
    __syncthreads();
    sums[tid] = sum;
    counts[tid] = count;
    __syncthreads();
    for (int d = kThreads / 2; d >= slice; d /= 2) {
        if (tid < d) {
            sums[tid] += sums[tid + d];
            counts[tid] += counts[tid + d];
        }
        __syncthreads();
    }
    if (tid < slice && e < a.E) {
        a.sums[(int64_t)q * a.E + e] = (float)sums[tid];
        a.counts[(int64_t)q * a.E + e] = counts[tid];
    }
    if (tid < slice) sums[tid] = e < a.E ? sums[tid] * (double)counts[tid] : 0.0;
    __syncthreads();
    for (int d = slice / 2; d > 0; d /= 2) {
        if (tid < d) sums[tid] += sums[tid + d];
        __syncthreads();
    }
    const int blocks = (int)gridDim.x;
    if (tid == 0) {
        if (e0 == 0) a.tokens[q] = live;
        const double share = live > 0 ? a.factor * sums[0] / ((double)live * (double)live) : 0.0;
        __hip_atomic_store(&a.part_loss[blockIdx.x], share, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        last = __hip_atomic_fetch_add(a.ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)blocks - 1;
    }
    __syncthreads();
    if (!last) return;
    sum = 0.0;
    for (int i = tid; i < blocks; i += kThreads)
        sum += __hip_atomic_load(&a.part_loss[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    sums[tid] = sum;
    __syncthreads();
    for (int d = kThreads / 2; d > 0; d /= 2) {
        if (tid < d) sums[tid] += sums[tid + d];
        __syncthreads();
    }
    if (tid == 0) *a.loss = (float)sums[0];
}

// The gradient.  With f[e] = g coefficient / Q * E / (K T^2) * count[e]:
//   softmax             p (f - sum f p)
//   sigmoid             s (1 - s) f
//   normalised sigmoid  p (1 - s) (f - sum f p)
// Scores that sum to one leave a constant in f without effect: K T / E, what
// every expert has of a balanced batch, is taken from the counts as an integer,
// so that the differences do not drown in the counts' own size.
template <int LANES, int VECS>
__global__ __launch_bounds__(kThreads) void k_balance_backward(BalanceArgs a)
{
    using X = Experts<LANES, VECS>;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t c0 = (int64_t)blockIdx.x * a.chunk;
    const int64_t c1 = c0 + a.chunk < a.N ? c0 + a.chunk : a.N;
    const bool divide = a.scoring == 0 || a.normalize;
    const double g = (double)*a.grad_loss * a.factor;

    float f[X::kEach];          // counts less the even share, of this lane's sequence
    float scale = 0.f;
    int q = a.start ? first_sequence(a, c0) : 0, loaded = -1;
    int64_t s0 = 0, s1 = 0;
    auto bounds = [&] {
        s0 = a.start ? (q < a.Q ? start_of(a, q) : a.N) : 0;
        s1 = a.start ? (q < a.Q ? start_of(a, (int64_t)q + 1) : a.N) : a.N;
    };
    bounds();
    for (int64_t t = c0 + wave * X::kTokens + lane / LANES; t - lane / LANES < c1; t += kWaves * X::kTokens) {
        if (t >= c1) continue;
        float z[X::kEach], rest[X::kEach];
        const bool masked = a.mask && a.mask[t] == 0;
        if (!masked) X::load(a, t, z);
        while (q < a.Q && s1 <= t) {
            ++q;
            bounds();
        }
        const bool in = !masked && q < a.Q && s0 <= t;
        if (in && q != loaded) {
            loaded = q;
            const int live = a.tokens_in[q];
            const int even = divide ? (int)((int64_t)a.K * live / a.E) : 0;
#pragma unroll
            for (int i = 0; i < X::kEach; ++i) {
                const int e = X::first(lane, i / 4) + i % 4;
                f[i] = e < a.E ? (float)(a.counts_in[(int64_t)q * a.E + e] - even) : 0.f;
            }
            scale = live > 0 ? (float)(g / ((double)live * (double)live)) : 0.f;
        }
        if (in) {
            X::template scores<true>(a, z, rest);
            float dot = 0.f;
            if (divide) {
#pragma unroll
                for (int i = 0; i < X::kEach; ++i) dot = fmaf(z[i], f[i], dot);
                dot = lanes_sum<LANES>(dot);
            }
#pragma unroll
            for (int i = 0; i < X::kEach; ++i) {
                z[i] *= (f[i] - dot) * scale;
                if (a.scoring != 0) z[i] *= rest[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < X::kEach; ++i) z[i] = 0.f;
        }
#pragma unroll
        for (int v = 0; v < VECS; ++v) {
            const int e = X::first(lane, v);
            const int64_t at = t * a.E + e;
            const float* d = z + 4 * v;
            if (a.vec) {
                if (e >= a.E) continue;
                if (a.bf16)
                    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.grad_logits) + at) =
                        u32x2{pack_bf16(d[0], d[1]), pack_bf16(d[2], d[3])};
                else
                    *reinterpret_cast<f32x4*>(static_cast<float*>(a.grad_logits) + at) = f32x4{d[0], d[1], d[2], d[3]};
                continue;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (e + j >= a.E) continue;
                if (a.bf16) static_cast<uint16_t*>(a.grad_logits)[at + j] = (uint16_t)pack_bf16(d[j], 0.f);
                else static_cast<float*>(a.grad_logits)[at + j] = d[j];
            }
        }
    }
}

template <bool BACK, int LANES, int VECS>
hipError_t launch_shape(const BalanceArgs& a, hipStream_t s)
{
    const int64_t chunks = (a.N + a.chunk - 1) / a.chunk;
    const dim3 grid((unsigned)(chunks > 0 ? chunks : 1)), block(kThreads);
    if constexpr (BACK) hipLaunchKernelGGL((k_balance_backward<LANES, VECS>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_balance_pieces<LANES, VECS>), grid, block, 0, s, a);
    return hipGetLastError();
}

template <bool BACK>
hipError_t launch_any(const BalanceArgs& a, hipStream_t s)
{
    if (a.E <= 64) return launch_shape<BACK, 16, 1>(a, s);
    if (a.E <= 128) return launch_shape<BACK, 16, 2>(a, s);
    if (a.E <= 256) return launch_shape<BACK, 16, 4>(a, s);
    if (a.E <= 512) return launch_shape<BACK, 64, 2>(a, s);
    return launch_shape<BACK, 64, 4>(a, s);
}

int chunk_of(int64_t N)
{
    const int64_t c = (N + kChunks - 1) / kChunks, up = (c + kMinChunk - 1) / kMinChunk * kMinChunk;
    return (int)(up < kMinChunk ? kMinChunk : up < kMaxChunk ? up : kMaxChunk);
}

}  // namespace

BalanceCarve carve_balance(int64_t N, int E, int Q)
{
    auto up = [](int64_t v) { return (v + 255) / 256 * 256; };
    BalanceCarve c;
    c.chunk = chunk_of(N);
    c.slots = (N + c.chunk - 1) / c.chunk + Q;
    // few sequences: many blocks for each, so that its pieces are read at once
    c.slice = Q <= 16 ? 16 : 64;
    c.blocks = (int64_t)Q * ((E + c.slice - 1) / c.slice);
    c.sum = 0;
    c.count = c.sum + up(4 * c.slots * E);
    c.tokens = c.count + up(4 * c.slots * E);
    c.loss = c.tokens + up(4 * c.slots);
    c.ticket = c.loss + up(8 * c.blocks);
    c.total = c.ticket + 256;
    return c;
}

hipError_t launch_balance(const BalanceArgs& a, const BalanceCarve& c, hipStream_t s)
{
    const hipError_t e = launch_any<false>(a, s);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_balance_finish, dim3((unsigned)c.blocks), dim3(kThreads), 0, s, a, c.slice,
                       (int)(c.blocks / a.Q));
    return hipGetLastError();
}

hipError_t launch_balance_backward(const BalanceArgs& a, hipStream_t s)
{
    BalanceArgs b = a;
    b.chunk = chunk_of(a.N);
    return launch_any<true>(b, s);
}

}  // namespace epk
