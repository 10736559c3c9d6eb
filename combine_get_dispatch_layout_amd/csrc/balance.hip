// The balance loss of a router on gfx950: per-expert counts, sums of scores,
// the loss they make, and its gradient with respect to the logits.
//
// With V_q the unmasked tokens of sequence q, T_q their number, count[q,e] the
// entries of their topk_idx that name e, and p the scores:
//   S[q,e] = sum over t in V_q of p[t,e]
//   loss   = coefficient / Q * sum_q E / (K T_q^2) * sum_e count[q,e] S[q,e]
//
// What bounds it: one reading of the logits (the gradient: and one writing) and
// some 17 instructions a score, two of them at a quarter of the rate, which take as
// long; for small batches the launches.  65536 tokens of 256 experts, fp32, sigmoid
// scores in 37 sequences: 19 us and 9 for the second kernel, 28 in all (the bytes
// at the rate of a large read: 9.6); the gradient 35 (a plain copy of the same
// bytes: 23).  In bf16, softmax scores: 25.6 in all, the gradient 21.  4096 tokens
// of 128 experts, bf16: 3.8, 6.4 and 4.0 us.
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

// The second kernel: waves of a block and blocks, at most.
constexpr int kFinishWaves = 16, kFinishBlocks = 256;

// A chunk: at least 16 tokens (four waves of four), so many that some 1024
// blocks make the batch, at most 1024 (which bounds the fp32 sums' length).
constexpr int kMinChunk = 16, kMaxChunk = 1024, kChunks = 1024;

// A batch that one block takes.
constexpr int kSmallWaves = 16, kSmallExperts = 256, kSmallTokens = 256, kSmallSequences = 4;

constexpr float kLow = -__builtin_huge_valf();

// exp(x) for |x| <= 150, off by an ulp or two: what the roundings of x log2(e) and
// of that constant leave of x, which the hardware's exp2 would magnify (65 units of
// 2^-24 at 87), is put right to first order, with log(2) in two parts.
__device__ __forceinline__ float exp_near(float x)
{
    const float y = x * 1.44269502f;
    const float r = __builtin_amdgcn_exp2f(y);
    return fmaf(r, fmaf(-y, -1.90465421e-9f, fmaf(-y, 0.693147182f, x)), r);
}

__device__ __forceinline__ float reciprocal(float d)
{
    const float r = __builtin_amdgcn_rcpf(d);
    return fmaf(fmaf(-d, r, 1.f), r, r);
}

// Below this a sigmoid is taken for 0 (it would be less than the smallest
// normal fp32, as softmax scores below that are).
constexpr float kFar = -87.25f;

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

// How logits lie in memory: rows of vectors of four (E % 4 == 0, aligned), or
// anything.
enum Form { kVecF32, kVecBf16, kAny };

// How a token's experts lie in LANES lanes: vector v of lane l holds the four
// experts from 4 (v LANES + l) on.
template <int LANES, int VECS, int FORM>
struct Experts {
    static constexpr int kEach = 4 * VECS;           // of a lane
    static constexpr int kTokens = kWave / LANES;    // of a wave at a time
    static constexpr int kMost = LANES * kEach;

    // Logits as they are loaded, to be in flight while others are worked on: no
    // branch and no conversion stands between the loads.
    static constexpr int kWords = FORM == kVecBf16 ? 2 : 4;
    struct Raw {
        uint32_t w[VECS][kWords];
    };

    static __device__ __forceinline__ int first(int lane, int v) { return 4 * (v * LANES + lane % LANES); }

    static __device__ __forceinline__ void load(const BalanceArgs& a, int64_t t, Raw& o)
    {
        const int lane = threadIdx.x & (kWave - 1);
#pragma unroll
        for (int v = 0; v < VECS; ++v) {
            const int e = first(lane, v);
            const int64_t at = t * a.E + (e < a.E ? e : 0);
            if constexpr (FORM == kVecF32) {
                const u32x4 d = *reinterpret_cast<const u32x4*>(static_cast<const float*>(a.logits) + at);
#pragma unroll
                for (int j = 0; j < 4; ++j) o.w[v][j] = d[j];
            } else if constexpr (FORM == kVecBf16) {
                const u32x2 d = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(a.logits) + at);
                o.w[v][0] = d[0];
                o.w[v][1] = d[1];
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    o.w[v][j] = __float_as_uint(load_logit(a.logits, a.bf16, t * a.E + (e + j < a.E ? e + j : 0)));
            }
        }
    }

    // -infinity past the last expert
    static __device__ __forceinline__ void unpack(const BalanceArgs& a, const Raw& r, float (&z)[kEach])
    {
        const int lane = threadIdx.x & (kWave - 1);
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int v = i / 4, j = i % 4;
            if constexpr (FORM == kVecBf16)
                z[i] = __uint_as_float(j % 2 ? r.w[v][j / 2] & 0xFFFF0000u : r.w[v][j / 2] << 16);
            else
                z[i] = __uint_as_float(r.w[v][j]);
        }
        if (a.E < kMost)
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                z[i] = first(lane, i / 4) + (FORM == kAny ? i % 4 : 0) < a.E ? z[i] : kLow;
    }

    // Logits to scores, up to the returned factor; of a sigmoid also 1 - s where
    // GRAD asks for it.
    template <bool GRAD>
    static __device__ __forceinline__ float scores(const BalanceArgs& a, float (&z)[kEach], float (&rest)[GRAD ? kEach : 1])
    {
        // (maxima pass over NaN, comparisons with it are false)
        const bool divide = a.scoring == 0 || a.normalize;
        float top = kLow;
        if (divide) {
#pragma unroll
            for (int i = 0; i < kEach; ++i) top = fmaxf(top, z[i]);
            top = lanes_max<LANES>(top);
        }
        constexpr float kHighest = 3.402823466e38f;
        if (a.scoring == 0 && top > kHighest) {     // +infinity: the largest float
            top = kHighest;
#pragma unroll
            for (int i = 0; i < kEach; ++i) z[i] = z[i] > kHighest ? kHighest : z[i];
        }
        // normalised sigmoids that have all but run out of range go in
        // proportion to their exponentials, as a softmax's (1 - s is 1 there)
        if (a.scoring == 0 || (divide && top < -64.f)) {
            // (a NaN, also -infinity less itself, becomes the least there is)
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                z[i] = exp_near(fmaxf(z[i] - top, -150.f));
                if constexpr (GRAD) rest[i] = 1.f;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const float x = exp_near(-__builtin_amdgcn_fmed3f(z[i], kFar, 150.f));
                const float r = __builtin_amdgcn_rcpf(1.f + x);
                if constexpr (GRAD) rest[i] = x * r;
                z[i] = z[i] > kFar ? r : 0.f;
            }
        }
        if (!divide) return 1.f;
        float total = 0.f;
#pragma unroll
        for (int i = 0; i < kEach; ++i) total += z[i];
        total = lanes_sum<LANES>(total);
        return total > 0.f ? reciprocal(total) : 0.f;
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

// What the tokens [t0, t1) add up to, by the block's W waves, in LDS.
template <typename X, int W>
struct Piece {
    float sums[W][X::kMost];    // of scores, a wave's share
    int counts[X::kMost];
    int tokens[W];              // unmasked ones, a wave's share
};

// Ends at a barrier; the caller places one before the next piece.
template <typename X, int W>
__device__ __forceinline__ void add_up(const BalanceArgs& a, int64_t t0, int64_t t1, Piece<X, W>& out)
{
    constexpr int kLanes = kWave / X::kTokens;
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    float acc[X::kEach], z[X::kEach], none[1];
#pragma unroll
    for (int i = 0; i < X::kEach; ++i) acc[i] = 0.f;
    int live = 0;
    typename X::Raw next;
    const int64_t mine = t0 + wave * X::kTokens + lane / kLanes;
    auto counted = [&](int64_t t) { return t < t1 && (!a.mask || a.mask[t] != 0); };
    auto held = [&](int64_t t) { return t < t1 ? t : t0; };     // a token of the piece
    bool in = counted(mine);
    // (before the counting, which waits for its own loads: 27.4 us against 28.4 for
    // 65536 tokens of 256 experts; two to four tokens ahead take registers that
    // four waves a SIMD need, 29 to 34)
    if (t0 < t1) X::load(a, held(mine), next);
    for (int e = tid; e < X::kMost; e += W * kWave) out.counts[e] = 0;
    __syncthreads();
    const int entries = (int)(t1 - t0) * a.K;
    for (int i = tid; i < entries; i += W * kWave) {
        const int t = a.k_magic ? (int)__umulhi((uint32_t)i, a.k_magic) : i;
        if (a.mask && a.mask[t0 + t] == 0) continue;
        const int e = a.topk[t0 * a.K + i];
        if ((uint32_t)e < (uint32_t)a.E) atomicAdd(&out.counts[e], 1);
    }
    for (int64_t t = mine; t - lane / kLanes < t1; t += W * X::kTokens) {
        const bool now = in;
        X::unpack(a, next, z);
        in = counted(t + W * X::kTokens);
        X::load(a, held(t + W * X::kTokens), next);
        live += (int)__popcll(__ballot(now)) / kLanes;
        const float by = X::template scores<false>(a, z, none);
        const float all = now ? by : 0.f;
#pragma unroll
        for (int i = 0; i < X::kEach; ++i) acc[i] = fmaf(z[i], all, acc[i]);
    }
#pragma unroll
    for (int i = 0; i < X::kEach; ++i)
#pragma unroll
        for (int d = kLanes; d < kWave; d *= 2) acc[i] += __shfl_xor(acc[i], d);
    if (lane < kLanes)
#pragma unroll
        for (int i = 0; i < X::kEach; ++i) out.sums[wave][X::first(lane, i / 4) + i % 4] = acc[i];
    if (lane == 0) out.tokens[wave] = live;
    __syncthreads();
}

// Adds up each piece of the block's chunk.
template <int LANES, int VECS, int FORM>
__global__ __launch_bounds__(kThreads) void k_balance_pieces(BalanceArgs a)
{
    using X = Experts<LANES, VECS, FORM>;
    __shared__ Piece<X, kWaves> piece;
    const int tid = threadIdx.x;
    if (blockIdx.x == 0 && tid == 0) *a.ticket = 0;
    const int64_t c0 = (int64_t)blockIdx.x * a.chunk;
    const int64_t c1 = c0 + a.chunk < a.N ? c0 + a.chunk : a.N;

    for (int q = a.start ? first_sequence(a, c0) : 0, next = q + 1; q < a.Q; q = next++) {
        const int64_t s0 = a.start ? start_of(a, q) : 0, s1 = a.start ? start_of(a, (int64_t)q + 1) : a.N;
        if (s0 >= c1) break;
        const int64_t t0 = s0 > c0 ? s0 : c0, t1 = s1 < c1 ? s1 : c1;
        if (t0 >= t1) {
            // empty, as its neighbours may be: on to the next that ends behind here
            // (one by one, 1000 that pad a batch cost 400 us)
            next = max(first_sequence(a, t0), next);
            continue;
        }
        add_up<X, kWaves>(a, t0, t1, piece);
        const int64_t slot = (int64_t)blockIdx.x + q;
        for (int e = tid; e < a.E; e += kThreads) {
            a.part_sum[slot * a.E + e] = (piece.sums[0][e] + piece.sums[1][e]) + (piece.sums[2][e] + piece.sums[3][e]);
            a.part_count[slot * a.E + e] = piece.counts[e];
        }
        if (tid == 0) a.part_tokens[slot] = (piece.tokens[0] + piece.tokens[1]) + (piece.tokens[2] + piece.tokens[3]);
        __syncthreads();
    }
}

// A small batch in one block, without the second kernel: what a call of few
// tokens costs is its launches.  128 tokens, 16 experts: 16.5 us as issued from
// Python in two kernels.
template <int LANES, int VECS, int FORM>
__global__ __launch_bounds__(kSmallWaves* kWave) void k_balance_small(BalanceArgs a)
{
    using X = Experts<LANES, VECS, FORM>;
    static_assert(X::kMost <= kSmallExperts && kSmallExperts <= kSmallWaves * kWave, "an expert a thread");
    __shared__ Piece<X, kSmallWaves> piece;
    __shared__ double shares[kSmallWaves];
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    double loss = 0.0;
    for (int q = 0; q < a.Q; ++q) {
        const int64_t s0 = a.start ? start_of(a, q) : 0, s1 = a.start ? start_of(a, (int64_t)q + 1) : a.N;
        add_up<X, kSmallWaves>(a, s0, s1 > s0 ? s1 : s0, piece);
        double dot = 0.0;
        int live = 0;
        for (int w = 0; w < kSmallWaves; ++w) live += piece.tokens[w];
        if (tid < a.E) {
            double sum = 0.0;
            for (int w = 0; w < kSmallWaves; ++w) sum += (double)piece.sums[w][tid];
            a.sums[(int64_t)q * a.E + tid] = (float)sum;
            a.counts[(int64_t)q * a.E + tid] = piece.counts[tid];
            dot = sum * (double)piece.counts[tid];
        }
        if (tid == 0) a.tokens[q] = live;
        dot = wave_sum(dot);
        if (lane == 0) shares[wave] = dot;
        __syncthreads();
        if (tid == 0 && live > 0) {
            for (int w = 1; w < kSmallWaves; ++w) dot += shares[w];
            loss += a.factor * dot / ((double)live * (double)live);
        }
    }
    if (tid == 0) *a.loss = (float)loss;
}

__device__ __forceinline__ int wave_total(int v)
{
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// Adds up the pieces: an item is a sequence's 64 experts, one a lane, by `join`
// waves, each every join-th piece.  A block has waves / join items at a time and
// goes on by the whole grid's; the last block to finish adds up the blocks' shares
// of the loss, in their order.  What bounds it is a chain of loads, and with many
// blocks their way past the one counter, 23 ns each: 65536 tokens of 256 experts in
// 1024 sequences took 131 us with a block an item, 29 with at most 256 blocks (both
// kernels), in 8192 sequences 807 and 60.  `join` goes by the mean of pieces a
// sequence, so one long sequence beside many others is walked by few waves: 65536
// tokens in one sequence 32 us, with 1024 empty ones beside it 98.
__global__ __launch_bounds__(kFinishWaves* kWave) void k_balance_finish(BalanceArgs a, int slices, int join)
{
    __shared__ double sums[kFinishWaves][kWave];
    __shared__ int counts[kFinishWaves][kWave];
    __shared__ double shares[kFinishWaves];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), waves = blockDim.x / kWave;
    const int part = wave % join, at_once = waves / join;
    const int items = a.Q * slices, stride = (int)gridDim.x * at_once;      // below 2^23
    double shared = 0.0;        // the wave's items' shares of the loss
    for (int i0 = (int)blockIdx.x * at_once; i0 < items; i0 += stride) {
        const int item = i0 + wave / join;
        const bool there = item < items;
        const int q = there ? item / slices : 0, slice = item % slices, e = slice * kWave + lane;
        // (tokens are below 2^31)
        const uint32_t s0 = a.start ? (uint32_t)start_of(a, q) : 0u;
        const uint32_t s1 = a.start ? (uint32_t)start_of(a, (int64_t)q + 1) : (uint32_t)a.N;
        const int first = (int)(s0 / (uint32_t)a.chunk);
        const int pieces = there && s1 > s0 ? (int)((s1 - 1) / (uint32_t)a.chunk) - first + 1 : 0;
        const int64_t slot0 = (int64_t)first + q;

        int live = 0;
        if (part == 0)
            for (int i = lane; i < pieces; i += kWave) live += a.part_tokens[slot0 + i];
        double sum = 0.0;
        int count = 0;
        if (e < a.E)
#pragma unroll 8
            for (int i = part; i < pieces; i += join) {
                sum += (double)a.part_sum[(slot0 + i) * a.E + e];
                count += a.part_count[(slot0 + i) * a.E + e];
            }
        if (join > 1) {
            sums[wave][lane] = sum;
            counts[wave][lane] = count;
            __syncthreads();
            if (part == 0)
                for (int w = 1; w < join; ++w) {
                    sum += sums[wave + w][lane];
                    count += counts[wave + w][lane];
                }
            if (i0 + stride < items) __syncthreads();
        }
        if (part != 0 || !there) continue;
        live = wave_total(live);
        if (e < a.E) {
            a.sums[(int64_t)q * a.E + e] = (float)sum;
            a.counts[(int64_t)q * a.E + e] = count;
        }
        if (slice == 0 && lane == 0) a.tokens[q] = live;
        const double dot = wave_sum(sum * (double)count);
        if (live > 0) shared += a.factor * dot / ((double)live * (double)live);
    }
    if (at_once > 1) {
        if (lane == 0) shares[wave] = shared;
        __syncthreads();
    }
    if (wave != 0) return;
    for (int w = join; w < waves; w += join) shared += shares[w];
    const int blocks = (int)gridDim.x;
    if (blocks == 1) {
        if (lane == 0) *a.loss = (float)shared;
        return;
    }
    uint32_t before = 0;
    if (lane == 0) {
        __hip_atomic_store(&a.part_loss[blockIdx.x], shared, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        before = __hip_atomic_fetch_add(a.ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (__builtin_amdgcn_readfirstlane((int)before) != blocks - 1) return;
    double sum = 0.0;
    for (int i = lane; i < blocks; i += kWave)
        sum += __hip_atomic_load(&a.part_loss[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    sum = wave_sum(sum);
    if (lane == 0) *a.loss = (float)sum;
}

// The gradient.  With f[e] = g coefficient / Q * E / (K T^2) * count[e]:
//   softmax             p (f - sum f p)
//   sigmoid             s (1 - s) f
//   normalised sigmoid  p (1 - s) (f - sum f p)
// Scores that sum to one leave a constant in f without effect: K T / E, what
// every expert has of a balanced batch, is taken from the counts as an integer,
// so that the differences do not drown in the counts' own size.  A token with most
// of its score on one expert measures the counts from that expert's: sum f p all but
// equals its f, and their difference, which the others' small scores make, would be
// the rounding of f.  (65536 tokens of 256 experts, fp32, softmax: 32.3 us, 31.7
// without; if most tokens are so sure 33.1.)
template <int LANES, int VECS, int FORM>
__global__ __launch_bounds__(kThreads) void k_balance_backward(BalanceArgs a)
{
    using X = Experts<LANES, VECS, FORM>;
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
    typename X::Raw next;
    const int64_t mine = c0 + wave * X::kTokens + lane / LANES;
    auto unmasked = [&](int64_t t) { return t < c1 && (!a.mask || a.mask[t] != 0); };
    auto held = [&](int64_t t) { return t < c1 ? t : c0; };         // a token of the chunk
    bool coming = unmasked(mine);
    X::load(a, held(mine), next);
    for (int64_t t = mine; t - lane / LANES < c1; t += kWaves * X::kTokens) {
        float z[X::kEach], rest[X::kEach];
        const bool live = coming;
        X::unpack(a, next, z);
        coming = unmasked(t + kWaves * X::kTokens);
        X::load(a, held(t + kWaves * X::kTokens), next);
        if (t >= c1) continue;
        if (q < a.Q && s1 <= t) {
            ++q;
            bounds();
            if (q < a.Q && s1 <= t) {       // empty ones: the next that ends behind t
                int lo = q + 1, hi = a.Q;
                while (lo < hi) {
                    const int mid = lo + (hi - lo) / 2;
                    if (start_of(a, (int64_t)mid + 1) > t) hi = mid;
                    else lo = mid + 1;
                }
                q = lo;
                bounds();
            }
        }
        const bool in = live && q < a.Q && s0 <= t;
        if (in && q != loaded) {
            loaded = q;
            const int tokens = a.tokens_in[q];
            const int even = divide ? (int)((int64_t)a.K * tokens / a.E) : 0;
#pragma unroll
            for (int i = 0; i < X::kEach; ++i) {
                const int e = X::first(lane, i / 4) + i % 4;
                f[i] = e < a.E ? (float)(a.counts_in[(int64_t)q * a.E + e] - even) : 0.f;
            }
            scale = tokens > 0 ? (float)(g / ((double)tokens * (double)tokens)) : 0.f;
        }
        if (in) {
            const float by = X::template scores<true>(a, z, rest);
            const float all = by * scale;
            // z becomes p (f - c - sum (f - c) p) for a number c of the token's
            auto slope = [&](auto from) {
                float dot = 0.f;
                if (divide) {
#pragma unroll
                    for (int i = 0; i < X::kEach; ++i) dot = fmaf(z[i], from(f[i]), dot);
                    dot = lanes_sum<LANES>(dot) * by;
                }
#pragma unroll
                for (int i = 0; i < X::kEach; ++i) {
                    z[i] *= (from(f[i]) - dot) * all;
                    if (a.scoring != 0) z[i] *= rest[i];
                }
            };
            // (scores before `by` are at most 1; one branch for the wave's tokens)
            const bool sure = divide && by > 0.5f;
            if (__builtin_expect(__any(sure), 0)) {
                float most = 0.f, c = kLow;
#pragma unroll
                for (int i = 0; i < X::kEach; ++i) most = fmaxf(most, z[i]);
                most = lanes_max<LANES>(most);
#pragma unroll
                for (int i = 0; i < X::kEach; ++i) c = fmaxf(c, z[i] == most ? f[i] : kLow);
                c = lanes_max<LANES>(c);
                if (!sure) c = 0.f;
                slope([c](float v) { return v - c; });
            } else {
                slope([](float v) { return v; });
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
            if constexpr (FORM == kVecF32) {
                if (e < a.E)
                    *reinterpret_cast<f32x4*>(static_cast<float*>(a.grad_logits) + at) = f32x4{d[0], d[1], d[2], d[3]};
            } else if constexpr (FORM == kVecBf16) {
                if (e < a.E)
                    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.grad_logits) + at) =
                        u32x2{pack_bf16(d[0], d[1]), pack_bf16(d[2], d[3])};
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (e + j >= a.E) continue;
                    if (a.bf16) static_cast<uint16_t*>(a.grad_logits)[at + j] = (uint16_t)pack_bf16(d[j], 0.f);
                    else static_cast<float*>(a.grad_logits)[at + j] = d[j];
                }
            }
        }
    }
}

bool is_small(const BalanceArgs& a)
{
    return a.N <= kSmallTokens && a.E <= kSmallExperts && a.Q <= kSmallSequences;
}

template <bool BACK, int LANES, int VECS, int FORM>
hipError_t launch_shape(const BalanceArgs& a, hipStream_t s)
{
    if constexpr (!BACK && LANES * VECS * 4 <= kSmallExperts) {
        if (is_small(a)) {
            hipLaunchKernelGGL((k_balance_small<LANES, VECS, FORM>), dim3(1), dim3(kSmallWaves * kWave), 0, s, a);
            return hipGetLastError();
        }
    }
    const int64_t chunks = (a.N + a.chunk - 1) / a.chunk;
    const dim3 grid((unsigned)(chunks > 0 ? chunks : 1)), block(kThreads);
    if constexpr (BACK) hipLaunchKernelGGL((k_balance_backward<LANES, VECS, FORM>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_balance_pieces<LANES, VECS, FORM>), grid, block, 0, s, a);
    return hipGetLastError();
}

template <bool BACK, int LANES, int VECS>
hipError_t launch_form(const BalanceArgs& a, hipStream_t s)
{
    if (!a.vec) return launch_shape<BACK, LANES, VECS, kAny>(a, s);
    return a.bf16 ? launch_shape<BACK, LANES, VECS, kVecBf16>(a, s) : launch_shape<BACK, LANES, VECS, kVecF32>(a, s);
}

template <bool BACK>
hipError_t launch_any(const BalanceArgs& a, hipStream_t s)
{
    if (a.E <= 64) return launch_form<BACK, 16, 1>(a, s);
    if (a.E <= 128) return launch_form<BACK, 16, 2>(a, s);
    if (a.E <= 256) return launch_form<BACK, 16, 4>(a, s);
    if (a.E <= 512) return launch_form<BACK, 64, 2>(a, s);
    return launch_form<BACK, 64, 4>(a, s);
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
    // as many waves join as a sequence has pieces to go round, eight each
    const int64_t join = (c.slots / Q + 7) / 8, items = (int64_t)Q * ((E + kWave - 1) / kWave);
    c.join = (int)(join < 1 ? 1 : join < kFinishWaves ? join : kFinishWaves);
    c.at_once = kFinishWaves / c.join;
    if (c.at_once > items) c.at_once = (int)items;
    c.blocks = (items + c.at_once - 1) / c.at_once;
    if (c.blocks > kFinishBlocks) c.blocks = kFinishBlocks;
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
    if (e != hipSuccess || is_small(a)) return e;
    hipLaunchKernelGGL(k_balance_finish, dim3((unsigned)c.blocks), dim3(c.at_once * c.join * kWave), 0, s, a,
                       (a.E + kWave - 1) / kWave, c.join);
    return hipGetLastError();
}

hipError_t launch_balance_backward(const BalanceArgs& a, hipStream_t s)
{
    BalanceArgs b = a;
    b.chunk = chunk_of(a.N);
    return launch_any<true>(b, s);
}

}  // namespace epk
