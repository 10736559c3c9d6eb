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
// What bounds it: the weights are read from HBM once and used for few rows, so
// everything serves keeping 16-byte weight loads in flight.  They go straight
// from memory to registers (no LDS round trip, nothing to share between
// waves), a block of spans per tile ahead of the arithmetic: four, or two in
// the small blocks, with INT4 groups of 32 and with 4-bit weights beside x from
// memory.  Only x, which every wave of a block reads, goes through LDS.
//
// Scales come a block ahead too, as whole words, where a row has a multiple of
// four of them.  Other rows (and a row's last, partial block) load them span by
// span behind the ring's own loads, whose order they then wait for: 64 experts,
// 4096 outputs, 2816 columns of MXFP4 86 us, 2880 columns 141 us; INT4 in groups
// of 128, 1024 columns 44 us, 768 columns 59 us.
//
// A lane's 16 bytes and the order of the columns.  A sum over columns may run
// in any order as long as x and W agree.  A load takes 8 rows x 128 bytes
// (whole cache lines: with 16 rows x 64 bytes, the order of a matrix operand,
// every line is fetched in two loads; loads alone then take 770 us for the
// MXFP4 decode batch, 654 us so).  Two loads make a "line", 128 bytes of 16
// rows; lanes 0-7 and 8-15 of each row of 16 lanes trade one of the two (DPP),
// which leaves two operands ("spans"): lane (n, c) has bytes 32c + 16v of row n
// in span v.  That is
//   bf16:  8 columns, one matrix instruction per span;
//   MXFP4: 32 columns = one scale group, four instructions.  Codes become
//          bf16 with their scale in v_cvt_scalef32_pk_bf16_fp4 (exact);
//   INT8:  16 columns, whose products with int8 rows of x go through
//          v_mfma_i32_16x16x64_i8: the same bytes as bf16's 8 columns, exact
//          sums, scaled by row and output before the store;
//   INT4:  32 columns; the four words of the four lanes of a row are
//          transposed in registers (v_permlane16_swap, v_permlane32_swap), so
//          that instruction j covers the 32 consecutive columns of lane j.
//          Code q becomes the bf16 value 16 + q by an OR; a second
//          instruction with the constant -(16 + zero) in B takes the offset
//          away in fp32; the group's scale multiplies the fp32 sum, so no
//          weight is rounded.  16 is the smallest offset that leaves all codes
//          one exponent: what the fp32 sums lose and the x at which they
//          overflow go with it.  (The second instruction is an eighth of the
//          128-token layer's time: the price of exact codes.)
//
// Measured on MI355X (GPU time): the up projection of a decode batch (128
// tokens, 256 experts, top-8, 7168 columns, 2 x 2048 rows, MXFP4, 4.0 GB)
// 667 us, 5.9 TB/s; in bf16 2176 us, 6.8 TB/s; in INT4 (groups of 128) 809 us,
// 4.7 TB/s, where the arithmetic of two waves a SIMD no longer hides behind the
// loads: without any, the whole INT4 layer takes 1060 us of its 1350.  Twelve or
// sixteen waves a CU with shorter rings are slower (790 us and more for MXFP4):
// fewer bytes in flight.
#pragma once

#include "experts.hpp"

namespace epk {
namespace prod {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// The same on 64 bytes of a row; the sums are whole numbers, held in the bits
// of acc.
__device__ __forceinline__ f32x4 mfma_i8(u32x4 a, u32x4 b, f32x4 c)
{
    return __builtin_bit_cast(f32x4, __builtin_amdgcn_mfma_i32_16x16x64_i8(
                                         __builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b),
                                         __builtin_bit_cast(i32x4, c), 0, 0, 0));
}

// a + b of two such accumulators.
template <int KIND>
__device__ __forceinline__ f32x4 add_sums(f32x4 a, f32x4 b)
{
    if constexpr (KIND == kInt8)
        return __builtin_bit_cast(f32x4, __builtin_bit_cast(i32x4, a) + __builtin_bit_cast(i32x4, b));
    else return a + b;
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

// Orders one lane's writes to LDS before another's reads in the same wave.
__device__ __forceinline__ void wave_exchange()
{
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// Weights and scales are read through a buffer resource per tile (its first
// row as the base, its rows as the bound): the address of a load is one lane
// offset that never changes and one scalar, so the loop has no address
// arithmetic in vector registers.  (Offsets stay inside the tile: the bound
// is no substitute for that where the scalar offset passes it.)
typedef __amdgpu_buffer_rsrc_t Buffer;

__device__ __forceinline__ Buffer make_buffer(const uint8_t* base, int64_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, (int)bytes, 0x00020000);
}

// Weights are read once: the non-temporal hint (aux bit 1) keeps them from
// displacing x and the scales in the caches.
constexpr int kNonTemporal = 2;

__device__ __forceinline__ u32x4 load_weights(Buffer b, uint32_t lane_off, uint32_t off)
{
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, lane_off, off, kNonTemporal));
}

template <int KIND>
struct Format {
    static constexpr bool kInt4 = is_int4(KIND);
    static constexpr bool kPlain = is_plain(KIND);
    static constexpr int kLine = line_columns(KIND);
    static constexpr int kParts = kPlain ? 1 : 4;               // instructions of a span
    static constexpr int kGroup = KIND == kInt4G128 ? 128 : KIND == kInt4G64 ? 64 : 32;
    // INT4: parts of a span that share a scale
    static constexpr int kGroupParts = KIND == kInt4G128 ? 2 : 1;
    // bytes of x: a line, and from one span, part and lane c to the next
    static constexpr int kLineBytes = 2 * kLine;
    static constexpr int kSpanBytes = kPlain ? 16 : 64;
    static constexpr int kPartBytes = kInt4 ? 128 : 16;
    static constexpr int kLaneBytes = kInt4 ? 16 : KIND == kMxfp4 ? 128 : 32;
};

// Scales (and zeros) of one weight row for a block of U spans, as loaded.
template <int KIND, int U>
struct Scales {
    static constexpr int kGroups = U * 128 / Format<KIND>::kGroup;
    static constexpr int kWords = is_plain(KIND) ? 0 : (KIND == kMxfp4 ? kGroups : 2 * kGroups) / 4;
    static constexpr int kZeroWords = !is_int4(KIND) ? 0 : (kGroups + 3) / 4;
    uint32_t s[kWords > 0 ? kWords : 1];
    uint32_t z[kZeroWords > 0 ? kZeroWords : 1];
};

template <int WORDS>
__device__ __forceinline__ void load_words(uint32_t* to, Buffer b, uint32_t lane_off, uint32_t off)
{
    if constexpr (WORDS >= 4) {
        const u32x4 v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, lane_off, off, 0));
        to[0] = v[0], to[1] = v[1], to[2] = v[2], to[3] = v[3];
        if constexpr (WORDS == 8) load_words<4>(to + 4, b, lane_off, off + 16);
    } else if constexpr (WORDS == 2) {
        const u32x2 v = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(b, lane_off, off, 0));
        to[0] = v[0], to[1] = v[1];
    } else if constexpr (WORDS == 1) {
        to[0] = __builtin_amdgcn_raw_buffer_load_b32(b, lane_off, off, 0);
    }
}

// INT4: the scale group, within a line, of a span's q-th run of parts.
template <int KIND>
constexpr int group_in_line(int v, int q)
{
    return KIND == kInt4G32 ? 2 * q + v : q;
}

// INT4: bf16 -(16 + zero) in both halves, for a zero byte and for 8.
__device__ __forceinline__ uint32_t offset_of(uint32_t zero) { return (0xC180u | (zero & 15u) << 3) * 0x10001u; }
constexpr uint32_t kOffset8 = 0xC1C0C1C0u;

// What one span of a weight row multiplies with, from its scale words.
template <int KIND>
struct SpanScale {
    static constexpr int kGroups = Format<KIND>::kInt4 ? 4 / Format<KIND>::kGroupParts : 1;
    float s[kGroups];          // MXFP4: this lane's group alone
    uint32_t off[kGroups];     // INT4: bf16 -(16 + zero), twice
};

// Span v of the block's line ln.
template <int KIND, int U>
__device__ __forceinline__ SpanScale<KIND> span_scale(const Scales<KIND, U>& b, int ln, int v, int c, bool zeros)
{
    SpanScale<KIND> o;
    if constexpr (KIND == kMxfp4) {
        // byte 2c + v of the line's eight; the conversion takes the scale's
        // exponent bits alone: byte 0 is 2^-127, byte 255 gives NaN
        const uint64_t w = (uint64_t)b.s[2 * ln + 1] << 32 | b.s[2 * ln];
        o.s[0] = __uint_as_float((uint32_t)(w >> (16 * c + 8 * v)) << 23);
    } else if constexpr (Format<KIND>::kInt4) {
#pragma unroll
        for (int q = 0; q < SpanScale<KIND>::kGroups; ++q) {
            const int i = ln * (256 / Format<KIND>::kGroup) + group_in_line<KIND>(v, q);
            const uint32_t w = b.s[i / 2];
            o.s[q] = __uint_as_float(i % 2 ? w & 0xFFFF0000u : w << 16);
            o.off[q] = kOffset8;
            if (zeros)      // bytes 0x80 | zero << 3, 0xC1, and again
                o.off[q] = __builtin_amdgcn_perm((b.z[i / 4] << 3 & 0x78787878u) | 0x80808080u, 0xC1C1C1C1u,
                                                 0x00040004u + (uint32_t)(i % 4) * 0x00010001u);
        }
    }
    return o;
}

// Two loads of a line of 16 rows, each 8 rows of 128 bytes (lane: row l % 8,
// bytes 16 * (l / 8)), to two operands of 16 rows (lane: row l % 16; q0 bytes
// 32 * (l / 16), q1 the 16 behind): lanes 0-7 and 8-15 of a row of 16 trade.
__device__ __forceinline__ void trade_halves(const u32x4& a, const u32x4& b, u32x4& q0, u32x4& q1)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // row_ror:8, written in lanes 8-15 (banks 2, 3) or 0-7 (banks 0, 1)
        q0[i] = (uint32_t)__builtin_amdgcn_update_dpp((int)a[i], (int)b[i], 0x128, 0xF, 0xC, false);
        q1[i] = (uint32_t)__builtin_amdgcn_update_dpp((int)b[i], (int)a[i], 0x128, 0xF, 0x3, false);
    }
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
__device__ __forceinline__ void expand(u32x4 f, const SpanScale<KIND>& s, u32x4 (&b)[Format<KIND>::kParts])
{
    if constexpr (is_plain(KIND)) {
        b[0] = f;
    } else if constexpr (KIND == kMxfp4) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t w = f[j];
            b[j][0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s.s[0], 0));
            b[j][1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s.s[0], 1));
            b[j][2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s.s[0], 2));
            b[j][3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s.s[0], 3));
        }
    } else {
        uint32_t q[4] = {f[0], f[1], f[2], f[3]};
        swap16(q[0], q[1]);
        swap16(q[2], q[3]);
        swap32(q[0], q[2]);
        swap32(q[1], q[3]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                b[j][i] = ((i ? q[j] >> (4 * i - 3) : q[j] << 3) & 0x00780078u) | 0x41804180u;
    }
}

// Adds one span's products to acc.  x: the A operands of its parts, x_lo:
// their second terms (LO).
template <int KIND, bool LO>
__device__ __forceinline__ void multiply(const u32x4 (&b)[Format<KIND>::kParts],
                                         const SpanScale<KIND>& s,
                                         const u32x4 (&x)[(LO ? 2 : 1) * Format<KIND>::kParts],
                                         f32x4& acc)
{
    using F = Format<KIND>;
    if constexpr (KIND == kInt8) {
        acc = mfma_i8(x[0], b[0], acc);
    } else if constexpr (!F::kInt4) {
#pragma unroll
        for (int j = 0; j < F::kParts; ++j) {
            acc = mfma(x[j], b[j], acc);
            if constexpr (LO) acc = mfma(x[F::kParts + j], b[j], acc);
        }
    } else {
#pragma unroll
        for (int g = 0; g < SpanScale<KIND>::kGroups; ++g) {
            const u32x4 off = {s.off[g], s.off[g], s.off[g], s.off[g]};
            f32x4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = g * F::kGroupParts; j < (g + 1) * F::kGroupParts; ++j) {
                sum = mfma(x[j], off, sum);
                sum = mfma(x[j], b[j], sum);
                if constexpr (LO) {
                    sum = mfma(x[F::kParts + j], off, sum);
                    sum = mfma(x[F::kParts + j], b[j], sum);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = fmaf(s.s[g], sum[i], acc[i]);
        }
    }
}

// Eight columns of x in the order in which INT4 codes come out of a word:
// i and i + 4 side by side.
__device__ __forceinline__ u32x4 pair_columns(u32x4 d)
{
    return u32x4{__builtin_amdgcn_perm(d[2], d[0], 0x05040100u),
                 __builtin_amdgcn_perm(d[2], d[0], 0x07060302u),
                 __builtin_amdgcn_perm(d[3], d[1], 0x05040100u),
                 __builtin_amdgcn_perm(d[3], d[1], 0x07060302u)};
}

// __expf's argument is off by 2^-24 of itself, so silu by |gate| * 2^-24 of it:
// far below the 2^-17 that the two terms below hold for any |gate| whose silu
// does not vanish (< 88), and the 2^-9 of a bf16 result.
__device__ __forceinline__ float swiglu(float gate, float up) { return gate / (1.f + __expf(-gate)) * up; }

// y + y_lo = w * swiglu: two bf16 terms hold at least 16 bits of the fp32 value (an
// infinity or NaN stays in the first), so the down projection, which takes
// bf16 operands, loses 2^-17 of it and not 2^-9.
__device__ __forceinline__ void store_split(const ProductArgs& a, int64_t row, int u, float gate, float up)
{
    const float v = swiglu(gate, up);
    const float wv = a.weights ? a.weights[row] * v : v;
    const uint16_t hi = to_bf16(wv);
    const int64_t to = row * a.ldy + u;
    reinterpret_cast<uint16_t*>(a.y)[to] = hi;
    a.y_lo[to] = (hi & 0x7F80u) == 0x7F80u ? (uint16_t)0 : to_bf16(wv - from_bf16(hi));
}

// ---- which rows belong to which expert --------------------------------------
//
// Each expert's rows are taken in passes of up to pass_rows; the tiles of all
// passes form one sequence that is divided evenly over the blocks.

constexpr int kPerLane = kMaxExperts / kWave;

struct Groups {
    int count[kMaxExperts];      // rows of each expert
    int pass0[kWave];            // passes before lane l's 16 experts
    int passes;                  // of all experts
};

// Rows of expert e, of which row0 is the first (received rows).
__device__ __forceinline__ int received_rows(const ProductArgs& a, int e, int64_t* row0)
{
    int64_t n = a.count[e];
    *row0 = a.psum[e];
    if (a.cap > 0 && n > a.cap) n = a.cap;
    if (*row0 + n > a.num_rows) n = *row0 < a.num_rows ? a.num_rows - *row0 : 0;
    return (int)n;
}

// Passes that n rows take: ceil(n / pass_rows).
__device__ __forceinline__ int passes_of(const ProductArgs& a, int n)
{
    const uint32_t up = (uint32_t)(n + a.pass_rows - 1);
    return (int)(a.pass_magic ? __umulhi(up, a.pass_magic) : up);
}

// Counts the rows of every expert and numbers their passes.
template <bool PAIRS, int kThreads>
__device__ __forceinline__ void count_groups(const ProductArgs& a, Groups& g, uint16_t* ids)
{
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    if constexpr (PAIRS) {
        for (int e = tid; e < kMaxExperts; e += kThreads) g.count[e] = 0;
        lds_barrier();
        for (int p = tid; p < a.P; p += kThreads) {
            const int e = a.topk[p];
            const bool ok = (uint32_t)e < (uint32_t)a.E;
            if (ok) atomicAdd(&g.count[e], 1);
            else if (e != -1 && blockIdx.x == 0) atomicOr(a.flags, kFlagBadId);
            ids[p] = ok ? (uint16_t)e : (uint16_t)0xFFFFu;
        }
    } else {
        for (int e = tid; e < kMaxExperts; e += kThreads) {
            int n = 0;
            if (e < a.E) {
                int64_t row0;
                n = received_rows(a, e, &row0);
                if (blockIdx.x == 0) {
                    const int64_t all = a.cap > 0 && a.count[e] > a.cap ? a.cap : a.count[e];
                    if (all > n) atomicOr(a.flags, kFlagCapacity);
                }
            }
            g.count[e] = n;
        }
    }
    lds_barrier();
    if (tid < kWave) {
        int mine = 0;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i)
            mine += passes_of(a, g.count[lane * kPerLane + i]);
        int upto = mine;
#pragma unroll
        for (int d = 1; d < kWave; d *= 2) {
            const int v = __shfl_up(upto, d);
            if (lane >= d) upto += v;
        }
        g.pass0[lane] = upto - mine;
        if (lane == kWave - 1) g.passes = upto;
    }
    lds_barrier();
}

// Expert and first row (within it) of a pass.
__device__ __forceinline__ void find_pass(const ProductArgs& a, const Groups& g, int pass, int* expert,
                                          int* m0)
{
    const int lane = threadIdx.x & (kWave - 1);
    const uint64_t at = __ballot(g.pass0[lane] <= pass);
    const int l = 63 - (int)__builtin_clzll(at);        // lane 0 always is
    int left = pass - g.pass0[l];
    int e = l * kPerLane;
    for (;; ++e) {
        const int n = passes_of(a, g.count[e]);
        if (left < n || e == l * kPerLane + kPerLane - 1) break;
        left -= n;
    }
    *expert = __builtin_amdgcn_readfirstlane(e);
    *m0 = __builtin_amdgcn_readfirstlane(left) * a.pass_rows;
}

// A handful of pairs (one a lane): every wave groups them by itself, without
// LDS or a barrier; experts in the order of their first pairs.  e: the lane's
// expert or -1.  Returns a mask of the lanes that are their expert's first.
__device__ __forceinline__ uint64_t first_pairs(int e, int P)
{
    bool first = e >= 0;
    for (int j = 0; j < P - 1; ++j)
        first = first && !((int)(threadIdx.x & (kWave - 1)) > j && __builtin_amdgcn_readlane(e, j) == e);
    return __ballot(first);
}

// The which-th expert and its pairs, given first_pairs.
__device__ __forceinline__ void find_few(int e, uint64_t firsts, int which, int* expert, uint64_t* pairs)
{
    const int lane = threadIdx.x & (kWave - 1);
    const uint64_t at = __ballot((firsts >> lane & 1) && __popcll(firsts & ((1ull << lane) - 1)) == which);
    *expert = __builtin_amdgcn_readlane(e, (int)__builtin_ctzll(at | 1ull << 63));
    *pairs = __ballot(e == *expert);
}

// One wave: the pairs of an expert, ascending, from the m0-th on (up to most).
__device__ __forceinline__ void list_pairs(const ProductArgs& a, const uint16_t* ids, int expert, int m0,
                                           int most, int32_t* list)
{
    const int lane = threadIdx.x & (kWave - 1);
    int at = -m0;
    for (int p0 = 0; p0 < a.P && at < most; p0 += kWave) {
        const int p = p0 + lane;
        const bool hit = p < a.P && ids[p] == expert;
        const uint64_t m = __ballot(hit);
        const int to = at + __popcll(m & ((1ull << lane) - 1));
        if (hit && to >= 0 && to < most) list[to] = p;
        at += __popcll(m);
    }
}

// ---- the kernel ------------------------------------------------------------------

constexpr int kSegments = 8;        // passes whose x is in LDS at a time
constexpr int kListRows = 128;      // ... and their rows, at most

// A block takes an even share of the tiles and walks it a batch at a time: the
// tiles of as many passes ("segments") as have their rows in LDS together.
// Its kWaves waves form kWaves / kw teams; a team takes every (kWaves / kw)-th
// tile of the batch, and its kw waves every kw-th block of kU spans of the
// tile's columns.  RT = 2: 16-output tiles of a wave (with a gate: its gate
// tile and its up tile); TT: 16-row tiles of x.
// DIRECT: x is read from memory, a block ahead, not through LDS.  With 4-bit
// weights and two terms of x (a layer's down projection) the compiler keeps that
// block in private memory (272 bytes a lane), so the loads ahead gain little
// there: 64 tokens, 8 experts, 4096 x 14336, INT4: 977 us for a floor of 100.
template <int KIND, int EPI, int TT, bool DIRECT, int kU, int kWaves>
__global__ __launch_bounds__(kWaves* kWave, TT == 2 && is_int4(KIND) ? 1 : kWaves == 4 ? (is_int4(KIND) ? 2 : 3) : kWaves / 4) void k_product(ProductArgs a)
{
    constexpr int kThreads = kWaves * kWave;
    using F = Format<KIND>;
    constexpr int RT = 2;
    constexpr int kL = kU / 2;                           // lines of a block
    constexpr bool kGate = EPI == kSwigluBf16 || EPI == kSwigluSplit;
    constexpr bool kPairs = EPI == kSwigluSplit || EPI == kStoreF32;
    constexpr bool LO = EPI == kStoreF32;
    constexpr int kPlanes = LO ? 2 : 1;
    constexpr int kParts = F::kParts;
    constexpr int kTileUnits = kGate ? 16 : 32;          // outputs of a tile
    static_assert(!DIRECT || TT == 1, "x from memory: one row tile");
    constexpr int kScaleBytes = F::kInt4 ? 2 : 1;

    extern __shared__ __align__(16) unsigned char smem[];   // x, then the waves' sums
    __shared__ Groups groups;
    __shared__ uint16_t ids[kPairs ? kMaxPairs : 1];
    __shared__ int32_t list[kListRows];                  // rows of x in LDS: their output rows
    __shared__ int seg_expert[kSegments], seg_rows[kSegments], seg_first[kSegments];
    f32x4* const red = reinterpret_cast<f32x4*>(smem + a.x_bytes);

    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int n = lane & 15, c = lane >> 4;
    const int kw = a.kw, rw = kWaves / kw;
    const int kq = wave % kw, rg = wave / kw;
    const bool grouped = kPairs || a.count != nullptr;

    int passes;
    const bool few = kPairs && a.P <= kWave && a.P <= a.pass_rows;
    int my_expert = -1;      // few: of pair `lane`
    uint64_t firsts = 0;
    if (few) {
        if (lane < a.P) my_expert = a.topk[lane];
        if ((uint32_t)my_expert >= (uint32_t)a.E) {
            if (my_expert != -1 && blockIdx.x == 0) atomicOr(a.flags, kFlagBadId);
            my_expert = -1;
        }
        firsts = first_pairs(my_expert, a.P);
        passes = __popcll(firsts);
    } else if (grouped) {
        count_groups<kPairs, kThreads>(a, groups, ids);
        passes = groups.passes;
    } else {
        passes = a.dense_passes;
    }
    const int tiles = (a.units + kTileUnits - 1) / kTileUnits;
    // this block's share [at, stop) of all tiles (fewer than 2^31)
    const uint32_t all = (uint32_t)passes * (uint32_t)tiles;
    const uint32_t share = all / gridDim.x, more = all - share * gridDim.x;
    uint32_t at = blockIdx.x * share + min(blockIdx.x, more);
    const uint32_t stop = at + share + (blockIdx.x < more ? 1u : 0u);

    const int row_bytes = (int)a.w.row_bytes, row_groups = (int)a.w.row_groups;
    const bool has_zeros = F::kInt4 && a.w.zeros != nullptr;
    const int full = row_bytes / 128;                // whole lines
    const bool tail = row_bytes % 128 != 0;          // columns behind them
    const int blocks = (full + kL - 1) / kL;
    const int mine = (blocks - kq + kw - 1) / kw;    // blocks of this wave per tile
    // lines whose scales are loaded a block at a time, as whole words
    const int quick = row_groups % 4 == 0 ? full : 0;
    const int cols_up = (a.w.cols + F::kLine - 1) / F::kLine * F::kLine;
    const int stride = (int)x_stride(KIND, a.w.cols);           // of x in LDS

    while (at < stop) {
        // ---- a batch: tiles [at, batch_stop) of passes pass0, pass0 + 1, ...
        const int pass0 = (int)(at / (uint32_t)tiles);
        int segments = 0, lds_rows = 0;
        for (int pass = pass0; segments < kSegments && (uint32_t)pass * (uint32_t)tiles < stop; ++pass) {
            int expert = 0, m0 = 0, rows;
            int64_t row0 = 0;
            uint64_t pairs = 0;
            if (few) {
                find_few(my_expert, firsts, pass, &expert, &pairs);
                rows = (int)__popcll(pairs);
            } else if (grouped) {
                find_pass(a, groups, pass, &expert, &m0);
                rows = min(groups.count[expert] - m0, a.pass_rows);
                if constexpr (!kPairs) row0 = (int64_t)a.psum[expert] + m0;
            } else {
                row0 = (int64_t)pass * a.pass_rows;
                rows = (int)min(a.num_rows - row0, (int64_t)a.pass_rows);
            }
            rows = __builtin_amdgcn_readfirstlane(rows);
            if (segments > 0 && lds_rows + rows > a.x_rows) break;
            // every wave writes the same values, but for long lists of pairs
            if (few) {
                if (pairs >> lane & 1) list[lds_rows + __popcll(pairs & ((1ull << lane) - 1))] = lane;
            } else if constexpr (kPairs) {
                if (wave == segments % kWaves) list_pairs(a, ids, expert, m0, rows, list + lds_rows);
            } else {
                if (lane < rows) list[lds_rows + lane] = (int32_t)(row0 + lane);
            }
            if (lane == 0) {
                seg_expert[segments] = expert;
                seg_rows[segments] = rows;
                seg_first[segments] = lds_rows;
            }
            lds_rows += rows;
            ++segments;
        }
        const uint32_t batch_stop = min(stop, (uint32_t)(pass0 + segments) * (uint32_t)tiles);
        // the lists: of several waves, or the same from every wave for itself
        if (kPairs && !few) lds_barrier();
        else wave_exchange();

        // ---- loads: where the next block comes from
        Buffer data[RT], scales[RT], zeros[RT];
        uint32_t data_off[RT][2], scale_off[RT], zero_off[RT];
        // of a tile of the batch: its segment, its first output
        auto segment_of = [&](uint32_t t) { return (int)(t / (uint32_t)tiles) - pass0; };
        auto unit_of = [&](uint32_t t, int seg) { return (int)(t - (uint32_t)(pass0 + seg) * (uint32_t)tiles) * kTileUnits; };
        auto aim = [&](uint32_t t) {      // past the batch: at nothing
            const bool there = t < batch_stop && mine > 0;
            if (!there) t = at;
            const int seg = segment_of(t), unit0 = unit_of(t, seg);
            const int64_t expert_row = (int64_t)__builtin_amdgcn_readfirstlane(seg_expert[seg]) * a.w.rows;
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                // idle lanes repeat the last output
                const int t0 = min(unit0 + (kGate ? 0 : 16 * r), a.units - 1);
                const int have = min(16, a.units - t0);
                const int64_t first = expert_row + (kGate && r == 1 ? a.units : 0) + t0;
                data[r] = make_buffer(a.w.data + first * row_bytes, there ? (int64_t)have * row_bytes : 0);
#pragma unroll
                for (int v = 0; v < 2; ++v)
                    data_off[r][v] = (uint32_t)min(8 * v + (lane & 7), have - 1) * (uint32_t)row_bytes +
                                     16u * (lane >> 3);
                if constexpr (!F::kPlain) {
                    scales[r] = make_buffer(a.w.scales + first * row_groups * kScaleBytes,
                                            there ? (int64_t)have * row_groups * kScaleBytes : 0);
                    scale_off[r] = (uint32_t)min(n, have - 1) * (uint32_t)(row_groups * kScaleBytes);
                }
                if constexpr (F::kInt4) {
                    zeros[r] = make_buffer(a.w.zeros + first * row_groups, there ? (int64_t)have * row_groups : 0);
                    zero_off[r] = (uint32_t)min(n, have - 1) * (uint32_t)row_groups;
                }
            }
        };
        auto load_half = [&](int r, int v, int line) {
            return load_weights(data[r], data_off[r][v], (uint32_t)line * 128u);
        };
        auto load_scales = [&](int r, int block, Scales<KIND, kU>& o) {
            constexpr uint32_t kG = Scales<KIND, kU>::kGroups;
            if constexpr (!F::kPlain)
                load_words<Scales<KIND, kU>::kWords>(o.s, scales[r], scale_off[r], block * kG * kScaleBytes);
            if constexpr (F::kInt4) {
                if (has_zeros) {
                    if constexpr (kG == 2)
                        o.z[0] = __builtin_amdgcn_raw_buffer_load_b16(zeros[r], zero_off[r], block * kG, 0);
                    else
                        load_words<Scales<KIND, kU>::kZeroWords>(o.z, zeros[r], zero_off[r], block * kG);
                }
            }
        };

        // one block of weights ahead: a line's registers are loaded again as
        // soon as they are used
        u32x4 f[kU][RT];
        Scales<KIND, kU> next[RT];
        aim(at + rg);
        {
            const int l0 = at + rg < batch_stop && mine > 0 ? kq * kL : 0;
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                if (l0 + kL <= quick) load_scales(r, l0 / kL, next[r]);
#pragma unroll
                for (int u = 0; u < kU; ++u) f[u][r] = load_half(r, u % 2, max(min(l0 + u / 2, full - 1), 0));
            }
        }

        // ---- x to LDS
        auto x_row = [&](int m) -> int64_t {
            const int row = list[m];
            if constexpr (kPairs) return a.x_per_pair ? row : row / a.K;
            else return row;
        };
        const int lo_bytes = DIRECT ? 0 : a.x_rows * stride;
        if constexpr (!DIRECT) {
            const int vecs = cols_up / 8;
            for (int m = wave; m < lds_rows; m += kWaves) {
                const uint16_t* from = a.x + x_row(m) * a.ldx;
                const uint16_t* from_lo = LO ? a.x_lo + x_row(m) * a.ldx : nullptr;
#pragma unroll 4
                for (int v = lane; v < vecs; v += kWave)
#pragma unroll
                    for (int pl = 0; pl < kPlanes; ++pl) {
                        u32x4 d = {0, 0, 0, 0};
                        if (v * 8 < a.w.cols) d = *reinterpret_cast<const u32x4*>((pl ? from_lo : from) + v * 8);
                        if constexpr (F::kInt4) d = pair_columns(d);
                        *reinterpret_cast<u32x4*>(smem + pl * lo_bytes + m * stride + 16 * v) = d;
                    }
            }
            lds_barrier();
        }

        const int64_t lo_elems = LO ? a.x_lo - a.x : 0;
        int seg = -1, rows = 0, first_row = 0;
        int64_t expert_row = 0;
        const uint16_t* xg = nullptr;      // this lane's row of x, in memory
        const unsigned char* xa[TT];       // ... in LDS
        auto enter = [&](int to) {
            seg = to;
            rows = __builtin_amdgcn_readfirstlane(seg_rows[to]);
            first_row = __builtin_amdgcn_readfirstlane(seg_first[to]);
            expert_row = (int64_t)__builtin_amdgcn_readfirstlane(seg_expert[to]) * a.w.rows;
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const int m = first_row + (16 * t + n < rows ? 16 * t + n : 0);     // others: any row
                xa[t] = smem + m * stride + c * F::kLaneBytes;
                if constexpr (DIRECT) xg = a.x + x_row(m) * a.ldx + c * (F::kLaneBytes / 2);
            }
        };
        // A operands of span v of a line, for row tile t: from LDS, or from
        // memory (of a last, partial line with zeros past the end)
        auto x_lds = [&](int t, int line, int v, u32x4 (&x)[kPlanes * kParts]) {
            const unsigned char* p = xa[t] + line * F::kLineBytes + v * F::kSpanBytes;
#pragma unroll
            for (int pl = 0; pl < kPlanes; ++pl)
#pragma unroll
                for (int j = 0; j < kParts; ++j)
                    x[pl * kParts + j] = *reinterpret_cast<const u32x4*>(p + pl * lo_bytes + j * F::kPartBytes);
        };
        auto x_memory = [&](int line, int v, bool partial, u32x4 (&x)[kPlanes * kParts]) {
            const uint16_t* p = xg + (int64_t)line * F::kLine + v * (F::kSpanBytes / 2);
#pragma unroll
            for (int pl = 0; pl < kPlanes; ++pl)
#pragma unroll
                for (int j = 0; j < kParts; ++j) {
                    const int k = j * (F::kPartBytes / 2);
                    if (partial && line * F::kLine + v * (F::kSpanBytes / 2) + k + c * (F::kLaneBytes / 2) >= a.w.cols)
                        x[pl * kParts + j] = u32x4{0, 0, 0, 0};
                    else
                        x[pl * kParts + j] = *reinterpret_cast<const u32x4*>(p + pl * lo_elems + k);
                }
        };
        // scales of a single span: groups past the row's end read the last one
        auto load_span_scale = [&](int unit0, int r, int line, int v) {
            SpanScale<KIND> o;
            const int u = min(unit0 + (kGate ? 0 : 16 * r) + n, a.units - 1);
            const int64_t base = (expert_row + (kGate && r == 1 ? a.units : 0) + u) * row_groups;
            if constexpr (KIND == kMxfp4) {
                const int gi = min(line * 8 + 2 * c + v, row_groups - 1);
                o.s[0] = __uint_as_float((uint32_t)a.w.scales[base + gi] << 23);
            } else if constexpr (F::kInt4) {
#pragma unroll
                for (int q = 0; q < SpanScale<KIND>::kGroups; ++q) {
                    const int want = line * (256 / F::kGroup) + group_in_line<KIND>(v, q);
                    const int gi = min(want, row_groups - 1);
                    const uint32_t w = reinterpret_cast<const uint16_t*>(a.w.scales)[base + gi];
                    o.s[q] = want == gi ? __uint_as_float(w << 16) : 0.f;
                    o.off[q] = has_zeros ? offset_of(a.w.zeros[base + gi]) : kOffset8;
                }
            }
            return o;
        };

        u32x4 xr[DIRECT ? kU : 1][kPlanes * kParts];
        if (at + rg < batch_stop) enter(segment_of(at + rg));
        if constexpr (DIRECT) {
#pragma unroll
            for (int u = 0; u < kU; ++u)
                if (full > 0 && seg >= 0) x_memory(min(kq * kL + u / 2, full - 1), u % 2, false, xr[u]);
        }
        const int steps = (int)((batch_stop - at + rw - 1) / rw);
        for (int step = 0; step < steps; ++step) {
            const uint32_t tile = at + step * rw + rg;
            const bool here = tile < batch_stop;
            f32x4 acc[RT][TT];
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int t = 0; t < TT; ++t) acc[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};
            int unit0 = 0;
            [[maybe_unused]] float ws[RT], xs[TT][4];
            // A operands of a span; x0: the ones that were loaded ahead, if any
            auto x_of = [&](int t, int line, int v, bool partial, u32x4 (*x0)[kPlanes * kParts],
                            u32x4 (&x)[kPlanes * kParts]) {
                if constexpr (!DIRECT) {
                    x_lds(t, line, v, x);
                } else if (x0 != nullptr) {
#pragma unroll
                    for (int i = 0; i < kPlanes * kParts; ++i) x[i] = (*x0)[i];
                } else {
                    x_memory(line, v, partial, x);
                }
                if constexpr (DIRECT && F::kInt4)
#pragma unroll
                    for (int i = 0; i < kPlanes * kParts; ++i) x[i] = pair_columns(x[i]);
            };
            // adds a span
            auto use = [&](const u32x4 (&q)[RT], const SpanScale<KIND> (&s)[RT], int line, int v, bool partial,
                           u32x4 (*x0)[kPlanes * kParts]) {
                if constexpr (TT == 1) {
                    u32x4 x[kPlanes * kParts];
                    x_of(0, line, v, partial, x0, x);
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        u32x4 b[kParts];
                        expand<KIND>(q[r], s[r], b);
                        multiply<KIND, LO>(b, s[r], x, acc[r][0]);
                    }
                } else {
                    u32x4 b[RT][kParts];
#pragma unroll
                    for (int r = 0; r < RT; ++r) expand<KIND>(q[r], s[r], b[r]);
#pragma unroll
                    for (int t = 0; t < TT; ++t)
                        if (t == 0 || 16 * t < rows) {
                            u32x4 x[kPlanes * kParts];
                            x_of(t, line, v, partial, x0, x);
#pragma unroll
                            for (int r = 0; r < RT; ++r) multiply<KIND, LO>(b[r], s[r], x, acc[r][t]);
                        }
                }
            };

            if (here) {
                const int to = segment_of(tile);
                if (to != seg) {
                    enter(to);
                    // x of the first block of another pass's tile
                    if constexpr (DIRECT) {
#pragma unroll
                        for (int u = 0; u < kU; ++u)
                            if (full > 0) x_memory(min(kq * kL + u / 2, full - 1), u % 2, false, xr[u]);
                    }
                }
                unit0 = unit_of(tile, seg);
                if constexpr (KIND == kInt8) {
                    // scales of this lane's outputs and rows, for the store
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        const int u = min(unit0 + (kGate ? 0 : 16 * r) + n, a.units - 1);
                        ws[r] = reinterpret_cast<const float*>(a.w.scales)[expert_row + (kGate && r == 1 ? a.units : 0) + u];
                    }
#pragma unroll
                    for (int t = 0; t < TT; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int m = 16 * t + 4 * c + i;
                            xs[t][i] = m < rows ? a.x_scales[list[first_row + m]] : 0.f;
                        }
                }
                for (int j = 0; j < mine; ++j) {
                    const int line0 = (kq + j * kw) * kL;
                    // the block after this one: of this tile, of the next, or none
                    int next0 = line0 + kw * kL;
                    if (j + 1 == mine) {
                        aim(tile + rw);
                        next0 = tile + rw < batch_stop ? kq * kL : 0;
                    }
                    // both spans of line ln: codes from load order to row
                    // order, the registers loaded again, then the products
                    auto take = [&](int ln, u32x4 (&q0)[RT], u32x4 (&q1)[RT]) {
#pragma unroll
                        for (int r = 0; r < RT; ++r) {
                            trade_halves(f[2 * ln][r], f[2 * ln + 1][r], q0[r], q1[r]);
                            f[2 * ln][r] = load_half(r, 0, min(next0 + ln, full - 1));
                            f[2 * ln + 1][r] = load_half(r, 1, min(next0 + ln, full - 1));
                        }
                    };
                    auto refill_x = [&](int ln) {
                        if constexpr (DIRECT) {
                            x_memory(min(next0 + ln, full - 1), 0, false, xr[2 * ln]);
                            x_memory(min(next0 + ln, full - 1), 1, false, xr[2 * ln + 1]);
                        }
                    };
                    if (line0 + kL <= quick) {
                        Scales<KIND, kU> cur[RT];
#pragma unroll
                        for (int r = 0; r < RT; ++r) {
                            cur[r] = next[r];
                            if (next0 + kL <= quick) load_scales(r, next0 / kL, next[r]);
                        }
#pragma unroll
                        for (int ln = 0; ln < kL; ++ln) {
                            u32x4 q0[RT], q1[RT];
                            SpanScale<KIND> s[RT];
                            take(ln, q0, q1);
#pragma unroll
                            for (int r = 0; r < RT; ++r) s[r] = span_scale<KIND, kU>(cur[r], ln, 0, c, has_zeros);
                            use(q0, s, line0 + ln, 0, false, &xr[DIRECT ? 2 * ln : 0]);
#pragma unroll
                            for (int r = 0; r < RT; ++r) s[r] = span_scale<KIND, kU>(cur[r], ln, 1, c, has_zeros);
                            use(q1, s, line0 + ln, 1, false, &xr[DIRECT ? 2 * ln + 1 : 0]);
                            refill_x(ln);
                            __builtin_amdgcn_sched_barrier(0);
                        }
                    } else {
                        // the row's last, partial block, or odd scale rows
#pragma unroll
                        for (int r = 0; r < RT; ++r)
                            if (next0 + kL <= quick) load_scales(r, next0 / kL, next[r]);
#pragma unroll
                        for (int ln = 0; ln < kL; ++ln) {
                            u32x4 q0[RT], q1[RT];
                            take(ln, q0, q1);
                            if (line0 + ln < full) {
                                SpanScale<KIND> s[RT];
#pragma unroll
                                for (int r = 0; r < RT; ++r) s[r] = load_span_scale(unit0, r, line0 + ln, 0);
                                use(q0, s, line0 + ln, 0, false, &xr[DIRECT ? 2 * ln : 0]);
#pragma unroll
                                for (int r = 0; r < RT; ++r) s[r] = load_span_scale(unit0, r, line0 + ln, 1);
                                use(q1, s, line0 + ln, 1, false, &xr[DIRECT ? 2 * ln + 1 : 0]);
                            }
                            refill_x(ln);
                            __builtin_amdgcn_sched_barrier(0);
                        }
                    }
                }
                // columns behind the last whole line: the team's first wave,
                // with zeros in the lanes past the end
                if (tail && kq == 0) {
#pragma unroll 1
                    for (int v = 0; v < 2; ++v) {
                        u32x4 q[RT];
                        SpanScale<KIND> s[RT];
#pragma unroll
                        for (int r = 0; r < RT; ++r) {
                            const int u = min(unit0 + (kGate ? 0 : 16 * r) + n, a.units - 1);
                            const int64_t row = expert_row + (kGate && r == 1 ? a.units : 0) + u;
                            const int byte = full * 128 + 16 * (2 * c + v);
                            q[r] = u32x4{0, 0, 0, 0};
                            if (byte < row_bytes)
                                q[r] = *reinterpret_cast<const u32x4*>(a.w.data + row * row_bytes + byte);
                            s[r] = load_span_scale(unit0, r, full, v);
                            if (KIND == kMxfp4 && byte >= row_bytes) s[r].s[0] = 1.f;
                        }
                        use(q, s, full, v, true, nullptr);
                    }
                }
            }

            // ---- the waves' shares of a sum, added in wave order
            if (kw > 1) {
                f32x4* const mine_red = red + (step & 1) * kWaves * RT * TT * kWave;
                if (kq > 0)
#pragma unroll
                    for (int r = 0; r < RT; ++r)
#pragma unroll
                        for (int t = 0; t < TT; ++t)
                            mine_red[((wave * RT + r) * TT + t) * kWave + lane] = acc[r][t];
                lds_barrier();
                if (kq == 0)
                    for (int q = 1; q < kw; ++q)
#pragma unroll
                        for (int r = 0; r < RT; ++r)
#pragma unroll
                            for (int t = 0; t < TT; ++t)
                                acc[r][t] = add_sums<KIND>(acc[r][t], mine_red[(((wave + q) * RT + r) * TT + t) * kWave + lane]);
            }

            // ---- store: this lane has output n of rows 4c .. 4c+3 of each tile
            if (kq == 0 && here) {
                if constexpr (KIND == kInt8) {
#pragma unroll
                    for (int r = 0; r < RT; ++r)
#pragma unroll
                        for (int t = 0; t < TT; ++t)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                acc[r][t][i] = (float)__builtin_bit_cast(i32x4, acc[r][t])[i] * xs[t][i] * ws[r];
                }
#pragma unroll
                for (int t = 0; t < TT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int m = 16 * t + 4 * c + i;
                        if (m >= rows) continue;
                        const int64_t yr = list[first_row + m];
                        if constexpr (kGate) {
                            const int u = unit0 + n;
                            if (u >= a.units) continue;
                            const float ga = acc[0][t][i];
                            if constexpr (EPI == kSwigluBf16)
                                reinterpret_cast<uint16_t*>(a.y)[yr * a.ldy + u] = to_bf16(swiglu(ga, acc[1][t][i]));
                            else
                                store_split(a, yr, u, ga, acc[1][t][i]);
                        } else {
#pragma unroll
                            for (int r = 0; r < RT; ++r) {
                                const int u = unit0 + 16 * r + n;
                                if (u >= a.units) continue;
                                const int64_t to = yr * a.ldy + u;
                                if constexpr (EPI == kStoreBf16)
                                    reinterpret_cast<uint16_t*>(a.y)[to] = to_bf16(acc[r][t][i]);
                                else
                                    reinterpret_cast<float*>(a.y)[to] = acc[r][t][i];
                            }
                        }
                    }
            }
        }
        at = batch_stop;
        if (at < stop) lds_barrier();      // x and the list are read; the next batch's follow
    }
}

// ---- the down projection of a handful of tokens, with the sum over their experts ---
//
// Up to 16 tokens and 32 (or 8) pairs whose activations fit LDS.  A block owns 16
// outputs of every token.  Row m of the A operand is token m's activation for
// the expert whose weights are in B, so a token's experts add up in the same
// accumulators and nothing has to be combined afterwards.  Tokens that the
// expert is not for get any row; their sums are not kept (so that an infinity
// or NaN in a weight stays with the tokens that chose it).  The 16 waves take
// the (expert, block of columns) units in turn, one unit of weights ahead.
// Latency bound: a block has few bytes (196 KB for one token, bf16, 2048 x
// 768, top-8) and what counts is that they are asked for early.  One token
// (GPU time of the layer): 27.7 us with the general kernel and k_layer_reduce,
// 24.9 us with this one; MXFP4 20.6 and 16.8 us.
// The lane's pair: its group's key, expert + kMaxExperts * (how often the
// token listed it before), so that a group has each token once; -1: none.
__device__ __forceinline__ int few_key(const ProductArgs& a, int e)
{
    const int lane = threadIdx.x & (kWave - 1);
    const int first = lane / a.K * a.K;
    int key = e;
    for (int j = 1; j < a.K; ++j) {
        const int before = __shfl_up(e, j);
        if (e >= 0 && lane - j >= first && before == e) key += kMaxExperts;
    }
    return key;
}

// Token n's pair among `pairs`; -1: none.
__device__ __forceinline__ int pair_of_token(const ProductArgs& a, uint64_t pairs, int n)
{
    const uint64_t of = n * a.K < kWave ? pairs >> (n * a.K) & ((1ull << a.K) - 1) : 0ull;
    return of != 0 ? n * a.K + (int)__builtin_ctzll(of) : -1;
}

// Codes and scales of a line (both spans) of one tile's rows, past the row's
// end zeros.  row0: the tile's first row in the stack, have: its rows.
template <int KIND>
struct Line {
    u32x4 q[2];
    SpanScale<KIND> s[2];
};

template <int KIND>
__device__ __forceinline__ void load_line(const WeightArgs& w, int64_t row0, int have, int line, Line<KIND>& o)
{
    using F = Format<KIND>;
    const int lane = threadIdx.x & (kWave - 1), n = lane & 15, c = lane >> 4;
    const int byte = line * 128 + 16 * (lane >> 3);
    const int row_groups = (int)w.row_groups;
    const int64_t base = (row0 + min(n, have - 1)) * row_groups;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        o.q[v] = u32x4{0, 0, 0, 0};
        if (byte < w.row_bytes)
            o.q[v] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(
                w.data + (row0 + min(8 * v + (lane & 7), have - 1)) * w.row_bytes + byte));
        if constexpr (KIND == kMxfp4) {
            const int gi = min(line * 8 + 2 * c + v, row_groups - 1);
            o.s[v].s[0] = __uint_as_float((uint32_t)w.scales[base + gi] << 23);
        } else if constexpr (F::kInt4) {
#pragma unroll
            for (int q = 0; q < SpanScale<KIND>::kGroups; ++q) {
                const int want = line * (256 / F::kGroup) + group_in_line<KIND>(v, q);
                const int gi = min(want, row_groups - 1);
                const uint32_t sc = reinterpret_cast<const uint16_t*>(w.scales)[base + gi];
                o.s[v].s[q] = want == gi ? __uint_as_float(sc << 16) : 0.f;
                o.s[v].off[q] = w.zeros ? offset_of(w.zeros[base + gi]) : kOffset8;
            }
        }
    }
}

template <int KIND>
__global__ __launch_bounds__(kFewWaves* kWave, 4) void k_down_few(ProductArgs a)
{
    using F = Format<KIND>;
    constexpr int kL = KIND == kBf16 ? 2 : 1;        // lines of a unit
    extern __shared__ __align__(16) unsigned char smem[];   // the pairs' rows; later the sums
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int n = lane & 15, c = lane >> 4;
    const int row_bytes = (int)a.w.row_bytes;
    const int cols_up = (a.w.cols + F::kLine - 1) / F::kLine * F::kLine;
    const int stride = (int)x_stride(KIND, a.w.cols);
    const int lo_bytes = a.P * stride;

    int e = lane < a.P ? a.topk[lane] : -1;
    if ((uint32_t)e >= (uint32_t)a.E) e = -1;        // flagged by the up projection
    const int key = few_key(a, e);
    const uint64_t firsts = first_pairs(key, a.P);
    const int per = (row_bytes + 128 * kL - 1) / (128 * kL);     // units of an expert
    const int units = __popcll(firsts) * per;
    const int tile0 = blockIdx.x * 16;

    struct Unit {
        Line<KIND> w[kL];
        int line;
        uint64_t pairs;
    };
    const int have = min(16, a.units - tile0);
    auto load = [&](int u, Unit& o) {
        const int group = u / per;
        int k;
        find_few(key, firsts, group, &k, &o.pairs);
        o.line = (u - group * per) * kL;
#pragma unroll
        for (int l = 0; l < kL; ++l)
            load_line<KIND>(a.w, (int64_t)(k % kMaxExperts) * a.w.rows + tile0, have, o.line + l, o.w[l]);
    };
    Unit cur, next;
    if (wave < units) load(wave, cur);

    // ---- activations to LDS
    const int vecs = cols_up / 8;
    for (int m = wave; m < a.P; m += kFewWaves) {
        if (__builtin_amdgcn_readlane(e, m) < 0) continue;      // never read
        for (int v = lane; v < vecs; v += kWave)
#pragma unroll
            for (int pl = 0; pl < 2; ++pl) {
                u32x4 d = {0, 0, 0, 0};
                if (v * 8 < a.w.cols)
                    d = *reinterpret_cast<const u32x4*>((pl ? a.x_lo : a.x) + (int64_t)m * a.ldx + v * 8);
                if constexpr (F::kInt4) d = pair_columns(d);
                *reinterpret_cast<u32x4*>(smem + pl * lo_bytes + m * stride + 16 * v) = d;
            }
    }
    lds_barrier();

    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    for (int u = wave; u < units; u += kFewWaves) {
        if (u + kFewWaves < units) load(u + kFewWaves, next);
        // token n's pair of this group; none: any
        const int mine = pair_of_token(a, cur.pairs, n);
        const int m = mine >= 0 ? mine : (int)__builtin_ctzll(cur.pairs);
        f32x4 part = {0.f, 0.f, 0.f, 0.f};
        const unsigned char* xa = smem + m * stride + c * F::kLaneBytes;
#pragma unroll
        for (int ln = 0; ln < kL; ++ln) {
            if (ln > 0 && (cur.line + ln) * 128 >= row_bytes) break;
            u32x4 q[2];
            trade_halves(cur.w[ln].q[0], cur.w[ln].q[1], q[0], q[1]);
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                u32x4 b[F::kParts], x[2 * F::kParts];
                const unsigned char* p = xa + (cur.line + ln) * F::kLineBytes + v * F::kSpanBytes;
#pragma unroll
                for (int j = 0; j < F::kParts; ++j) {
                    x[j] = *reinterpret_cast<const u32x4*>(p + j * F::kPartBytes);
                    x[F::kParts + j] = *reinterpret_cast<const u32x4*>(p + lo_bytes + j * F::kPartBytes);
                }
                expand<KIND>(q[v], cur.w[ln].s[v], b);
                multiply<KIND, true>(b, cur.w[ln].s[v], x, part);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = pair_of_token(a, cur.pairs, 4 * c + i) >= 0 ? acc[i] + part[i] : acc[i];
        cur = next;
    }

    // ---- the waves' shares, added in wave order
    lds_barrier();
    f32x4* const red = reinterpret_cast<f32x4*>(smem);
    red[wave * kWave + lane] = acc;
    lds_barrier();
    if (wave != 0) return;
    f32x4 sum = red[lane];
    for (int w = 1; w < kFewWaves; ++w) sum += red[w * kWave + lane];
    const int tokens = a.P / a.K;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (4 * c + i < tokens && tile0 + n < a.units)
            reinterpret_cast<uint16_t*>(a.y)[(int64_t)(4 * c + i) * a.ldy + tile0 + n] = to_bf16(sum[i]);
}

// The down projection and the sum over experts in one kernel, if the batch is
// a handful (*done); the caller takes the general path otherwise.
template <int KIND>
hipError_t launch_down_few(const ProductArgs& a, bool* done, hipStream_t s)
{
    static_assert(few_pairs(KIND) <= kWave, "a pair a lane");
    *done = few_fits(KIND, a.P / a.K, a.P, a.w.cols);
    if (!*done) return hipSuccess;
    const int64_t lds = few_bytes(KIND, a.P, a.w.cols);
    if (lds > 32768)
        (void)hipFuncSetAttribute(reinterpret_cast<const void*>(k_down_few<KIND>),
                                  hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    hipLaunchKernelGGL(k_down_few<KIND>, dim3((a.units + 15) / 16), dim3(kFewWaves * kWave), (size_t)lds, s, a);
    return hipGetLastError();
}

// ---- launch -------------------------------------------------------------

inline int num_cus()
{
    static const int n = [] {
        int dev = 0, v = 0;
        if (hipGetDevice(&dev) != hipSuccess ||
            hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || v < 1)
            v = 256;
        return v;
    }();
    return n;
}

template <int KIND, int EPI, int TT, bool DIRECT, int U, int kWaves>
hipError_t launch_shape(ProductArgs a, const Shape& c, int64_t max_rows, hipStream_t s)
{
    constexpr int kPlanes = EPI == kStoreF32 ? 2 : 1;
    a.kw = c.kw;
    a.pass_rows = (int)c.rows;
    a.pass_magic = div_magic((uint32_t)c.rows);
    a.dense_passes = (int)((a.num_rows + c.rows - 1) / c.rows);
    const int64_t stride = x_stride(KIND, a.w.cols), sums = sums_bytes(kWaves, c.kw, TT);
    // rows of several passes go to LDS together, as many as there is room for
    int64_t x_rows = DIRECT ? kListRows : (c.room - sums) / (kPlanes * stride);
    x_rows = x_rows < max_rows ? x_rows : max_rows;
    a.x_rows = (int)(x_rows < kListRows ? x_rows : kListRows);
    a.x_bytes = DIRECT ? 0 : (int)(a.x_rows * kPlanes * stride);
    const int64_t lds = a.x_bytes + sums;
    if (lds > kLdsRoom) return hipErrorInvalidValue;
    const int64_t most = kWaves == 4 && TT == 1 ? 1 << 30 : (int64_t)num_cus();
    const int64_t need = (c.tiles + kWaves / c.kw - 1) / (kWaves / c.kw);
    const dim3 grid((unsigned)(need < most ? need : most));
    if (lds > 32768)
        (void)hipFuncSetAttribute(reinterpret_cast<const void*>(k_product<KIND, EPI, TT, DIRECT, U, kWaves>),
                                  hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    hipLaunchKernelGGL((k_product<KIND, EPI, TT, DIRECT, U, kWaves>), grid, dim3(kWaves * kWave), (size_t)lds, s, a);
    return hipGetLastError();
}

// One kernel for the whole product.
template <int KIND, int EPI>
hipError_t launch_kind(const ProductArgs& a, hipStream_t s)
{
    constexpr bool kPairs = EPI == kSwigluSplit || EPI == kStoreF32;
    constexpr bool kGate = EPI == kSwigluBf16 || EPI == kSwigluSplit;
    const bool grouped = kPairs || a.count != nullptr;
    const int64_t rows = grouped ? a.P : a.num_rows;
    const Shape c = choose_shape(KIND, kGate, EPI == kStoreF32 ? 2 : 1, a.w.cols, a.units, grouped ? a.E : 1, rows);
    switch (c.path) {
        case kPathNone: return hipSuccess;
        case kPathSmall: return launch_shape<KIND, EPI, 1, false, kSpansSmall, 4>(a, c, rows, s);
        case kPathOneTile: return launch_shape<KIND, EPI, 1, false, spans_ahead(KIND, false), 8>(a, c, rows, s);
        case kPathMemory: return launch_shape<KIND, EPI, 1, true, spans_ahead(KIND, true), 8>(a, c, rows, s);
        default:
            // (int8 rows above 8 an expert go to the tiled kernels)
            if constexpr (KIND == kInt8) return hipErrorInvalidValue;
            else return launch_shape<KIND, EPI, 2, false, spans_ahead(KIND, false), two_tile_waves(KIND)>(a, c, rows, s);
    }
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
