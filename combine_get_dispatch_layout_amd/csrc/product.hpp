// Products of a few rows with expert weights on gfx950: the kernel that
// experts_*.hip instantiate for each weight format.
//
// What is computed, for the rows x[m] of one expert and 16 (or 32) of its
// outputs n at a time:
//   sum[m][n] = sum over columns k of W[n][k] * x[m][k]
// on the matrix cores (v_mfma_f32_16x16x32_bf16, fp32 sums), with the rows of
// x as the A operand and the weight rows as B, so that a lane's weight codes,
// scales and sums all belong to one output n = lane % 16.
//
// What bounds it: the weights are read from HBM once and used for few rows,
// so everything serves keeping 16-byte weight loads in flight.  They go
// straight from memory to registers (no LDS round trip, nothing to share
// between waves), one stage of loads ahead of the arithmetic; only x, which
// every wave of a block reads, goes through LDS.
//
// A lane's 16 bytes and the order of the columns.  A sum over columns may run
// in any order as long as x and W agree, so the 16 bytes that a lane loads are
// always contiguous in its weight row ("span" = the 64 bytes that the four
// lanes of a row load together):
//   bf16:  8 columns, one matrix instruction per span;
//   MXFP4: 32 columns = one scale group, four instructions.  Codes become
//          bf16 with their scale in v_cvt_scalef32_pk_bf16_fp4 (exact);
//   INT4:  32 columns; the four words of the four lanes of a row are
//          transposed in registers (v_permlane16_swap, v_permlane32_swap), so
//          that instruction j covers the 32 consecutive columns 32*j.  Code q
//          becomes the bf16 value 128 + q by an OR; a second instruction with
//          the constant -(128 + zero) in B takes the offset away in fp32; the
//          group's scale multiplies the fp32 sum of the group, so no weight is
//          rounded.
#pragma once

#include "experts.hpp"

namespace epk {
namespace prod {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr int kWaves = 4;            // per block
constexpr int kThreads = kWaves * kWave;

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ uint16_t to_bf16(float v)
{
    return (uint16_t)(__builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{v, 0.f}, bf16x2)) &
                      0xFFFFu);
}

__device__ __forceinline__ float from_bf16(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// Barrier for LDS only: loads from global memory stay in flight across it.
__device__ __forceinline__ void lds_barrier()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

template <int KIND>
struct Format {
    static constexpr bool kInt4 = KIND >= kInt4G32;
    static constexpr int kSpan = KIND == kBf16 ? 32 : 128;      // columns of 64 bytes
    static constexpr int kParts = KIND == kBf16 ? 1 : 4;        // instructions of a span
    // parts that share a scale (INT4)
    static constexpr int kGroupParts = KIND == kInt4G32 ? 1 : KIND == kInt4G64 ? 2 : 4;
};

// One span of one weight row quarter: codes and, for the 4-bit formats, the
// scale word (MXFP4: the E8M0 byte; INT4: bf16 scale << 16 | bf16 -(128+zero)).
struct Frag {
    u32x4 q;
    uint32_t s;
};

// Per-lane addresses of a weight row.
struct Row {
    const uint8_t* data;       // + 16 * (lane / 16)
    const uint8_t* scales;
    const uint8_t* zeros;
};

template <int KIND>
__device__ __forceinline__ Frag load_frag(const Row& r, int span, int c, int64_t last, int last_group)
{
    Frag f;
    // lanes past the row's end read its last 16 bytes instead (and zero them)
    const int64_t off = min((int64_t)span * 64, last);
    f.q = *reinterpret_cast<const u32x4*>(r.data + off);
    f.s = 0;
    if constexpr (KIND == kMxfp4) {
        f.s = r.scales[min(span * 4 + c, last_group)];
    } else if constexpr (Format<KIND>::kInt4) {
        const int g = KIND == kInt4G32 ? span * 4 + c : KIND == kInt4G64 ? span * 2 + (c >> 1) : span;
        const int gi = min(g, last_group);
        const uint32_t sc = reinterpret_cast<const uint16_t*>(r.scales)[gi];
        const uint32_t z = r.zeros ? r.zeros[gi] : 8u;
        f.s = sc << 16 | 0xC300u | z;
    }
    return f;
}

__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b)
{
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}

__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b)
{
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}

// B operands of a span's instructions, from the loaded codes.
template <int KIND>
struct Operand {
    u32x4 b[Format<KIND>::kParts];
    uint32_t s[4 / Format<KIND>::kGroupParts];   // INT4: scale words of the span's groups
};

template <int KIND>
__device__ __forceinline__ void expand(Frag f, bool empty, Operand<KIND>& o)
{
    if (empty) {      // columns past the end: 0 * 0
        f.q = u32x4{0, 0, 0, 0};
        f.s = KIND == kMxfp4 ? 127u : 0u;
    }
    if constexpr (KIND == kBf16) {
        o.b[0] = f.q;
    } else if constexpr (KIND == kMxfp4) {
        // the conversion takes the scale's exponent bits alone, so byte 0 is
        // 2^-127 and byte 255 gives NaN
        const float sc = __uint_as_float(f.s << 23);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t w = f.q[j];
            o.b[j][0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 0));
            o.b[j][1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 1));
            o.b[j][2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 2));
            o.b[j][3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 3));
        }
    } else {
        uint32_t q[4] = {f.q[0], f.q[1], f.q[2], f.q[3]};
        swap16(q[0], q[1]);
        swap16(q[2], q[3]);
        swap32(q[0], q[2]);
        swap32(q[1], q[3]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) o.b[j][i] = ((q[j] >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
        if constexpr (KIND == kInt4G128) {
            o.s[0] = f.s;
        } else {
            // lane c of a row holds group c's word (or c / 2's): all to all
            uint32_t a = f.s, b = f.s;
            if constexpr (KIND == kInt4G64) {
                swap32(a, b);
                o.s[0] = a;
                o.s[1] = b;
            } else {
                swap16(a, b);
                uint32_t a2 = a, b2 = b;
                swap32(a, a2);
                swap32(b, b2);
                o.s[0] = a;
                o.s[1] = b;
                o.s[2] = a2;
                o.s[3] = b2;
            }
        }
    }
}

// Adds one span's products to acc.  xa: the lane's A operand address of part
// 0 in LDS; parts are kPartBytes apart.
template <int KIND, bool LO>
__device__ __forceinline__ void multiply(const Operand<KIND>& o, const unsigned char* xa,
                                         int lo_bytes, f32x4& acc)
{
    using F = Format<KIND>;
    constexpr int kPartBytes = KIND == kMxfp4 ? 16 : 64;
    if constexpr (!F::kInt4) {
#pragma unroll
        for (int j = 0; j < F::kParts; ++j) {
            acc = mfma(*reinterpret_cast<const u32x4*>(xa + j * kPartBytes), o.b[j], acc);
            if constexpr (LO)
                acc = mfma(*reinterpret_cast<const u32x4*>(xa + lo_bytes + j * kPartBytes), o.b[j], acc);
        }
    } else {
#pragma unroll
        for (int g = 0; g < 4 / F::kGroupParts; ++g) {
            const uint32_t z = (o.s[g] & 0xFFFFu) * 0x10001u;
            const u32x4 off = {z, z, z, z};
            f32x4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = g * F::kGroupParts; j < (g + 1) * F::kGroupParts; ++j) {
                const u32x4 x = *reinterpret_cast<const u32x4*>(xa + j * kPartBytes);
                sum = mfma(x, off, sum);
                sum = mfma(x, o.b[j], sum);
                if constexpr (LO) {
                    const u32x4 xl = *reinterpret_cast<const u32x4*>(xa + lo_bytes + j * kPartBytes);
                    sum = mfma(xl, off, sum);
                    sum = mfma(xl, o.b[j], sum);
                }
            }
            const float sc = __uint_as_float(o.s[g] & 0xFFFF0000u);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = fmaf(sc, sum[i], acc[i]);
        }
    }
}

// The i-th expert that has a row, and its rows.
struct Group {
    int expert;      // -1: there is none
    int64_t row0;
    int64_t rows;
};

// Bit e of the LDS bitmap is set where expert e has a row: finds the which-th.
__device__ __forceinline__ int nth_expert(const uint32_t* bits, int which)
{
    const int lane = threadIdx.x & (kWave - 1);
    const uint32_t word = lane < kMaxExperts / 32 ? bits[lane] : 0u;
    int upto = __popc(word);
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int v = __shfl_up(upto, d);
        if (lane >= d) upto += v;
    }
    const int before = upto - __popc(word);
    const uint64_t here = __ballot(lane < kMaxExperts / 32 && before <= which && which < upto);
    if (here == 0) return -1;
    const int l = (int)__builtin_ctzll(here);
    uint32_t w = (uint32_t)__builtin_amdgcn_readlane((int)word, l);
    int n = which - __builtin_amdgcn_readlane(before, l);
    while (n-- > 0) w &= w - 1;
    return 32 * l + (int)__builtin_ctz(w);
}

// Pairs: the which-th chosen expert and its pairs, ascending, in list.
__device__ __forceinline__ Group group_pairs(const ProductArgs& a, int which, uint32_t* bits,
                                             int* wave_counts, uint16_t* list, bool report)
{
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    constexpr int kPer = kMaxPairs / kThreads;
    if (tid < kMaxExperts / 32) bits[tid] = 0u;
    lds_barrier();
    // wave w holds the pairs [w*64*per, (w+1)*64*per) in order
    const int per = (a.P + kThreads - 1) / kThreads;
    int ids[kPer];
    uint32_t bad = 0u;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (i < per) {
            const int p = (wave * per + i) * kWave + lane;
            const int e = p < a.P ? a.topk[p] : -1;
            const bool ok = (uint32_t)e < (uint32_t)a.E;
            if (ok) atomicOr(&bits[e >> 5], 1u << (e & 31));
            else if (e != -1) bad = kFlagBadId;
            ids[i] = ok ? e : -1;
        }
    }
    if (report && bad) atomicOr(a.flags, bad);
    lds_barrier();
    const int e = __builtin_amdgcn_readfirstlane(nth_expert(bits, which));
    if (e < 0) return Group{-1, 0, 0};
    int mine = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        if (i < per) mine += __popcll(__ballot(ids[i] == e));
    if (lane == 0) wave_counts[wave] = mine;
    lds_barrier();
    int at = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (w < wave) at += wave_counts[w];
        total += wave_counts[w];
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (i < per) {
            const uint64_t m = __ballot(ids[i] == e);
            if (ids[i] == e)
                list[at + __popcll(m & ((1ull << lane) - 1))] =
                    (uint16_t)((wave * per + i) * kWave + lane);
            at += __popcll(m);
        }
    }
    lds_barrier();
    return Group{e, 0, total};
}

// Received rows: the which-th expert with a row.
__device__ __forceinline__ Group group_received(const ProductArgs& a, int which, uint32_t* bits,
                                                bool report)
{
    const int tid = threadIdx.x;
    if (tid < kMaxExperts / 32) bits[tid] = 0u;
    lds_barrier();
    for (int e = tid; e < a.E; e += kThreads)
        if (a.count[e] > 0) atomicOr(&bits[e >> 5], 1u << (e & 31));
    lds_barrier();
    const int e = __builtin_amdgcn_readfirstlane(nth_expert(bits, which));
    if (e < 0) return Group{-1, 0, 0};
    const int64_t row0 = a.psum[e];
    int64_t n = a.count[e];
    if (a.cap > 0 && n > a.cap) n = a.cap;
    if (row0 + n > a.num_rows) {
        if (report && tid == 0) atomicOr(a.flags, kFlagCapacity);
        n = row0 < a.num_rows ? a.num_rows - row0 : 0;
    }
    return Group{e, row0, n};
}

// RT: 16-output tiles of a wave (with a gate: its gate tile and its up tile);
// TT: 16-row tiles of x; U: spans in flight per wave and stage.
template <int KIND, int EPI, int RT, int TT, int U>
__global__ __launch_bounds__(kThreads) void k_product(ProductArgs a)
{
    using F = Format<KIND>;
    constexpr bool kGate = EPI == kSwigluBf16 || EPI == kSwigluSplit;
    constexpr bool kPairs = EPI == kSwigluSplit || EPI == kStoreF32;
    constexpr bool LO = EPI == kStoreF32;
    constexpr int kPlanes = LO ? 2 : 1;
    constexpr int kTileUnits = kGate ? 16 : 16 * RT;     // outputs of a wave
    static_assert(!kGate || RT == 2, "a gated wave holds a gate tile and an up tile");

    extern __shared__ __align__(16) unsigned char smem[];   // x, later the waves' sums
    __shared__ uint32_t bits[kMaxExperts / 32];
    __shared__ int wave_counts[kWaves];
    __shared__ uint16_t list[kPairs ? kMaxPairs : 1];

    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int n = lane & 15, c = lane >> 4;
    const int kw = a.kw, rw = kWaves / kw;
    const int kq = wave % kw, rg = wave / kw;

    const bool first_tile = blockIdx.x == 0;
    Group g;
    if constexpr (kPairs) g = group_pairs(a, blockIdx.y, bits, wave_counts, list, first_tile && blockIdx.y == 0);
    else if (a.count) g = group_received(a, blockIdx.y, bits, first_tile);
    else g = Group{0, 0, a.num_rows};
    if (g.expert < 0) return;

    // ---- this wave's weight rows
    const int unit0 = (blockIdx.x * rw + rg) * kTileUnits;
    const int64_t expert_rows = (int64_t)g.expert * a.w.rows;
    Row row[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int u = min(unit0 + (kGate ? 0 : 16 * r) + n, a.units - 1);
        const int64_t at = expert_rows + (kGate && r == 1 ? a.units + u : u);
        row[r].data = a.w.data + at * a.w.row_bytes + 16 * c;
        row[r].scales = a.w.scales + at * a.w.row_groups * (F::kInt4 ? 2 : 1);
        row[r].zeros = a.w.zeros ? a.w.zeros + at * a.w.row_groups : nullptr;
    }
    const int64_t last = a.w.row_bytes - 16 - 16 * c;
    const int last_group = (int)a.w.row_groups - 1;
    const int spans = (int)((a.w.row_bytes + 63) / 64);
    const int iters = (spans + kw - 1) / kw;
    const bool tail_lane = (int64_t)(spans - 1) * 64 + 16 * c >= a.w.row_bytes;

    const int64_t block_step = (kPairs || a.count) ? 16 * TT : 16 * TT * (int64_t)gridDim.y;
    const int64_t block0 = (kPairs || a.count) ? 0 : 16 * TT * (int64_t)blockIdx.y;
    for (int64_t m0 = block0; m0 < g.rows; m0 += block_step) {
        const int rows = (int)min(g.rows - m0, (int64_t)(16 * TT));
        // iterations whose columns of these rows fit LDS at once
        int chunk = (a.x_bytes / (rows * kPlanes) - 16) / (kw * F::kSpan * 2);
        chunk = min(chunk, iters);
        const int chunk_cols = chunk * kw * F::kSpan;
        const int stride = chunk_cols * 2 + 16;      // 16: rows start in different banks
        const int lo_bytes = rows * stride;

        f32x4 acc[RT][TT];
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int t = 0; t < TT; ++t) acc[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};

        Frag f[U][RT];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int r = 0; r < RT; ++r)
                f[u][r] = load_frag<KIND>(row[r], min(u * kw + kq, spans - 1), c, last, last_group);

        for (int i0 = 0; i0 < iters; i0 += chunk) {
            // ---- x to LDS: columns [i0 * kw * span, + chunk_cols) of every row
            lds_barrier();
            const int col0 = i0 * kw * F::kSpan;
            const int vecs = chunk_cols / 8;
            for (int v = tid; v < rows * vecs; v += kThreads) {
                const int m = v / vecs, k = (v - m * vecs) * 8;
                int64_t xr;
                if constexpr (kPairs) {
                    const int p = list[m0 + m];
                    xr = a.x_per_pair ? p : p / a.K;
                } else {
                    xr = g.row0 + m0 + m;
                }
                const bool in = col0 + k < a.w.cols;
                const int64_t at = xr * a.ldx + col0 + k;
#pragma unroll
                for (int pl = 0; pl < kPlanes; ++pl) {
                    u32x4 d = {0, 0, 0, 0};
                    if (in) d = *reinterpret_cast<const u32x4*>((pl ? a.x_lo : a.x) + at);
                    if constexpr (F::kInt4)     // columns i and i+4 side by side, as the codes come out
                        d = u32x4{__builtin_amdgcn_perm(d[2], d[0], 0x05040100u),
                                  __builtin_amdgcn_perm(d[2], d[0], 0x07060302u),
                                  __builtin_amdgcn_perm(d[3], d[1], 0x05040100u),
                                  __builtin_amdgcn_perm(d[3], d[1], 0x07060302u)};
                    *reinterpret_cast<u32x4*>(smem + pl * lo_bytes + m * stride + 2 * k) = d;
                }
            }
            lds_barrier();

            // ---- this wave's spans of the chunk
            const int end = min(i0 + chunk, iters);
            const unsigned char* xa[TT];
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const int m = 16 * t + n < rows ? 16 * t + n : 0;     // others: any row
                xa[t] = smem + m * stride + (KIND == kMxfp4 ? 64 : 16) * c;
            }
            for (int i = i0; i < end; i += U) {
                const int next = i + U < end ? i + U : end;
                Frag fn[U][RT];
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int r = 0; r < RT; ++r)
                        fn[u][r] = load_frag<KIND>(row[r], min((next + u) * kw + kq, spans - 1), c,
                                                   last, last_group);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int span = (i + u) * kw + kq;
                    if (i + u < end && span < spans) {
                        const bool empty = span == spans - 1 && tail_lane;
#pragma unroll
                        for (int r = 0; r < RT; ++r) {
                            Operand<KIND> o;
                            expand<KIND>(f[u][r], empty, o);
#pragma unroll
                            for (int t = 0; t < TT; ++t)
                                if (t == 0 || 16 * t < rows)
                                    multiply<KIND, LO>(o, xa[t] + (span - i0 * kw) * F::kSpan * 2,
                                                       lo_bytes, acc[r][t]);
                        }
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int r = 0; r < RT; ++r) f[u][r] = fn[u][r];
            }
        }

        // ---- the waves' shares of a sum, added in wave order
        if (kw > 1) {
            lds_barrier();
            f32x4* red = reinterpret_cast<f32x4*>(smem);
            if (kq > 0)
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int t = 0; t < TT; ++t)
                        red[((wave * RT + r) * TT + t) * kWave + lane] = acc[r][t];
            lds_barrier();
            if (kq == 0)
                for (int q = 1; q < kw; ++q)
#pragma unroll
                    for (int r = 0; r < RT; ++r)
#pragma unroll
                        for (int t = 0; t < TT; ++t)
                            acc[r][t] += red[(((wave + q) * RT + r) * TT + t) * kWave + lane];
        }

        // ---- store: this lane has output n of rows 4c .. 4c+3 of each tile
        if (kq == 0) {
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int m = 16 * t + 4 * c + i;
                    if (m >= rows) continue;
                    int64_t yr;
                    if constexpr (kPairs) yr = list[m0 + m];
                    else yr = g.row0 + m0 + m;
                    if constexpr (kGate) {
                        const int u = unit0 + n;
                        if (u >= a.units) continue;
                        const float ga = acc[0][t][i];
                        const float v = ga / (1.f + __expf(-ga)) * acc[1][t][i];
                        const int64_t at = yr * a.ldy + u;
                        if constexpr (EPI == kSwigluBf16) {
                            reinterpret_cast<uint16_t*>(a.y)[at] = to_bf16(v);
                        } else {
                            // two bf16 terms hold 16 bits of the fp32 value (an
                            // infinity or NaN stays in the first)
                            const float wv = a.weights ? a.weights[yr] * v : v;
                            const uint16_t hi = to_bf16(wv);
                            reinterpret_cast<uint16_t*>(a.y)[at] = hi;
                            a.y_lo[at] = (hi & 0x7F80u) == 0x7F80u ? (uint16_t)0
                                                                   : to_bf16(wv - from_bf16(hi));
                        }
                    } else {
#pragma unroll
                        for (int r = 0; r < RT; ++r) {
                            const int u = unit0 + 16 * r + n;
                            if (u >= a.units) continue;
                            const int64_t at = yr * a.ldy + u;
                            if constexpr (EPI == kStoreBf16)
                                reinterpret_cast<uint16_t*>(a.y)[at] = to_bf16(acc[r][t][i]);
                            else
                                reinterpret_cast<float*>(a.y)[at] = acc[r][t][i];
                        }
                    }
                }
        }
    }
}

// ---- launch -------------------------------------------------------------

template <int KIND, int EPI, int RT, int TT, int U>
hipError_t launch_shape(ProductArgs a, int slots, int64_t max_rows, hipStream_t s)
{
    using F = Format<KIND>;
    constexpr int kPlanes = EPI == kStoreF32 ? 2 : 1;
    constexpr bool kGate = EPI == kSwigluBf16 || EPI == kSwigluSplit;
    const int kw = kWaves;
    const int rows = (int)(max_rows < 16 * TT ? max_rows : 16 * TT);
    const int64_t step = (int64_t)kw * F::kSpan * 2;
    const int64_t need = rows * kPlanes * (step + 16);
    const int64_t whole = rows * kPlanes * ((a.w.cols * 2 + step - 1) / step * step + 16);
    int64_t bytes = 32768;
    bytes = bytes < whole ? bytes : whole;
    bytes = bytes > need ? bytes : need;
    const int64_t red = (int64_t)kWaves * RT * TT * kWave * 16;
    bytes = bytes > red ? bytes : red;
    a.kw = kw;
    a.x_bytes = (int)bytes;
    const int per_block = (kWaves / kw) * (kGate ? 16 : 16 * RT);
    const dim3 grid((a.units + per_block - 1) / per_block, slots);
    if (bytes > 65536)
        (void)hipFuncSetAttribute(reinterpret_cast<const void*>(k_product<KIND, EPI, RT, TT, U>),
                                  hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    hipLaunchKernelGGL((k_product<KIND, EPI, RT, TT, U>), grid, dim3(kThreads), (size_t)bytes, s, a);
    return hipGetLastError();
}

// One kernel for the whole product.  Slots (blockIdx.y): experts that can have
// a row, or row blocks of the dense product.
template <int KIND, int EPI>
hipError_t launch_kind(const ProductArgs& a, hipStream_t s)
{
    constexpr bool kPairs = EPI == kSwigluSplit || EPI == kStoreF32;
    constexpr int U = KIND == kBf16 ? 4 : 2;
    const int64_t max_rows = kPairs || a.count ? a.P : a.num_rows;
    if (max_rows <= 0) return hipSuccess;
    const int64_t experts = kPairs || a.count ? (max_rows < a.E ? max_rows : a.E) : 0;
    const int64_t likely = experts ? max_rows / experts : max_rows;
    auto slots = [&](int tt) {
        if (experts) return (int)experts;
        const int64_t b = (max_rows + 16 * tt - 1) / (16 * tt);
        return (int)(b < 32768 ? b : 32768);
    };
    if (likely <= 16) return launch_shape<KIND, EPI, 2, 1, U>(a, slots(1), max_rows, s);
    return launch_shape<KIND, EPI, 2, 4, U>(a, slots(4), max_rows, s);
}

template <int KIND>
hipError_t launch_epilogue(const ProductArgs& a, int epilogue, hipStream_t s)
{
    switch (epilogue) {
        case kStoreBf16: return launch_kind<KIND, kStoreBf16>(a, s);
        case kSwigluBf16: return launch_kind<KIND, kSwigluBf16>(a, s);
        case kSwigluSplit: return launch_kind<KIND, kSwigluSplit>(a, s);
        default: return launch_kind<KIND, kStoreF32>(a, s);
    }
}

}  // namespace prod
}  // namespace epk
