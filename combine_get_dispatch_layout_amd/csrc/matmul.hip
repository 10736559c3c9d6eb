// Products of many int8 rows with int8 weights on gfx950: a tiled kernel on the
// matrix cores.
//
// What is computed, for a tile of BM rows of one expert and BN of its weight
// rows: sum[m][n] = sum over k of W[n][k] x[m][k], exact in 32-bit integers, by
// v_mfma_i32_16x16x64_i8 with the weight rows as A and the rows of x as B, so
// that a lane's sums are four neighbouring outputs of one row of x; then scales,
// activation, one rounding.
//
// Both operands go from memory straight to LDS (buffer loads with an LDS
// destination), S stages of 128 columns in a ring, and from there to registers.
//  - 128 columns: a row's share of a load is a whole cache line.  With 64 columns
//    and twice the stages, the same bytes take twice the requests: 4096 rows,
//    7168 -> 4096, 118 us, with 128 columns 108 us.
//  - A load puts lane l's 16 bytes at 16 l, so the order of a row's eight pieces
//    in LDS is chosen by which piece a lane asks for: piece j of row r lies at
//    j ^ (r % 8), and the eight lanes that LDS serves at a time (eight rows, one
//    piece) find eight different places.  No bank conflicts are counted.
//  - Lanes whose row or columns are past the end ask for an address outside the
//    buffer: they get zeros and cost no traffic.
// Blocks stay: each takes tile after tile, and the loads run S - 1 stages ahead
// of the arithmetic across tile borders, so a new tile starts with its columns
// there.  Scales of a tile's rows and outputs ride along with its first stage.
//
// An expert's rows are spread evenly over its tiles, in 16s, and a tile's
// arithmetic skips groups of 16 rows behind the last.  Tiles are numbered so that
// the blocks of an XCD (blockIdx % 8), which share an L2, work side by side: a
// contiguous share of all tiles each, four tiles of rows by the tiles of outputs.
//
// Sums of integers may be taken in any order, so tiles of experts, or of one matrix
// and few rows, begin at a step of their own and go round: blocks that start
// together would ask for the same columns of rows a power of two apart, which lie
// in the same few channels of the memory.  Where an expert has one tile of rows
// nothing is shared, and the tiles of its outputs spread over all columns; with
// more, over four steps, so that they still find each other's columns in L2.  128 experts of 45 rows, 4096 -> 1408:
// 144 us, all from column 0 154 to 160; 64 of 768, 1536 -> 4096: 368 and 382;
// 128 of 256, 2048 -> 2 x 768: 168 and 171; 7168 columns: equal to 1 % slower.
//
// Where tiles are fewer than CUs, their columns are split over blocks if the caller
// has room for the sums, which a second kernel joins (choose_splits).
//
// What bounds it.  One matrix: power, and behind that the way through LDS; 4096
// rows, 7168 -> 4096, 96 to 101 us, 2.4 to 2.5 POP/s (the library's plain products:
// 2.1 to 2.2), launches without a pause 113 at 2.1 GHz of 2.4.  Experts: the way of
// their columns from L2 to LDS (128 experts of 256 rows, 2048 -> 2 x 768: 3840 tiles
// of 16 stages of 32 KB, 2.0 GB in 165 us), and of the outputs to memory, which all
// CUs write at once: 64 experts of 768 rows, 1536 -> 4096, 375 us, without the stores
// 305, loads alone 257.
#include "experts.hpp"
#include "matmul_shape.hpp"

namespace epk {

hipError_t launch_product_int8(const ProductArgs& a, int epilogue, hipStream_t s);

namespace mm {
namespace {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
// Vectors at any address of their elements, so that rows of odd length are stored
// as others are: 3324 rows, 1024 -> 2335, 18.6 us, element by element 25.6.
typedef u32x4 Any16 __attribute__((aligned(2)));
typedef u32x2 Any8 __attribute__((aligned(2)));
typedef i32x4 AnySums __attribute__((aligned(4)));

struct Args {
    const uint8_t* w;           // [E, rows, cols]
    const float* w_scales;      // [E, rows]
    int rows, cols, units;
    const uint8_t* x;           // [.., cols]
    const float* x_scales;
    int64_t num_rows;
    int E;
    const int32_t* psum;        // of received rows, else null
    const int32_t* count;
    int cap;
    uint16_t* y;                // [.., units]
    int splits;                 // of the columns, and their sums [splits, num_rows, rows]
    int32_t* part;
    uint32_t* flags;
};

typedef __amdgpu_buffer_rsrc_t Buffer;

__device__ __forceinline__ Buffer make_buffer(const void* base, int64_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00020000);
}

// 16 bytes a lane from memory straight to LDS, lane after lane.
__device__ __forceinline__ void load_to_lds(Buffer b, unsigned char* to, uint32_t lane_off, uint32_t off)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (__attribute__((address_space(3))) void*)to, 16, lane_off, off, 0, 0);
}

// 4 bytes a lane.
__device__ __forceinline__ void load_word_to_lds(Buffer b, unsigned char* to, uint32_t lane_off)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (__attribute__((address_space(3))) void*)to, 4, lane_off, 0, 0, 0);
}

__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b)
{
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}

// BM rows of x and BN weight rows, shared by WM x WN waves.
template <int BM, int BN, int WM, int WN, int S, bool GATE>
struct Tile {
    static constexpr int kWaves = WM * WN, kThreads = kWave * kWaves;
    static constexpr int kLoadRows = 1024 / kStep;              // of a load
    static constexpr int kXLoads = BM / kLoadRows / kWaves, kWLoads = BN / kLoadRows / kWaves;
    static constexpr int kLoads = kXLoads + kWLoads;            // of a wave a stage
    static constexpr int MT = BM / 16 / WM, NT = BN / 16 / WN;  // groups of 16 of a wave
    static constexpr int kStageBytes = (BM + BN) * kStep;
    static constexpr int kUnits = GATE ? BN / 2 : BN;
    static constexpr int kScaleBytes = (BM + BN) * 4, kScaleLoads = (BM + BN) / 64;
    // Tiles whose scales are held: a tile's are loaded when the last columns of the
    // one before it have been, S - 1 steps ahead of the arithmetic.
    static constexpr int kScales = scale_buffers(S);
    static constexpr int kLds = S * kStageBytes + kScales * kScaleBytes;
    // blocks of a CU: 160 KB of LDS, 5 KB of which are static
    static constexpr int kBlocks = 163840 / (kLds + 5632);
    static_assert(BM % (kLoadRows * kWaves) == 0 && BN % (kLoadRows * kWaves) == 0, "whole loads");
    static_assert(BM % (16 * WM) == 0 && BN % (16 * WN) == 0 && BM % 64 == 0 && BN % 64 == 0, "whole groups");
    // gate and up groups alternate; a wave's loads are of one kind
    static_assert(!GATE || (NT % 2 == 0 && kWaves * kLoadRows % 32 == 0), "pairs of groups");
};

// A tile of one expert.
struct Where {
    int expert, rows;
    int64_t row0;
    int unit0;
    int m, side;                // its place among the tiles of rows beside each other
    int split, first, steps;    // its steps
};

// ---- which tiles there are ------------------------------------------------------

// Tiles of rows before each expert.
struct Tiles {
    int before[kMaxExperts + 1];
    int wave_sum[16];
};

// Rows of expert e, of which row0 is the first.
__device__ __forceinline__ int64_t rows_of(const Args& a, int e, int64_t* row0, bool flag)
{
    if (a.count == nullptr) {
        *row0 = 0;
        return a.num_rows;
    }
    int64_t r = a.count[e];
    *row0 = a.psum[e];
    if (a.cap > 0 && r > a.cap) r = a.cap;
    if (*row0 + r > a.num_rows) {
        r = *row0 < a.num_rows ? a.num_rows - *row0 : 0;
        if (flag && blockIdx.x == 0) atomicOr(a.flags, kFlagCapacity);
    }
    return r;
}

// The tiles of BM rows that all experts have together, by WAVES waves.
template <int BM, int WAVES>
__device__ __forceinline__ int count_tiles(const Args& a, Tiles& o)
{
    if (a.count == nullptr) return (int)((a.num_rows + BM - 1) / BM);
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    int all = 0;
    for (int e0 = 0; e0 < a.E; e0 += WAVES * kWave) {
        const int e = e0 + tid;
        int64_t row0;
        const int t = e < a.E ? (int)((rows_of(a, e, &row0, true) + BM - 1) / BM) : 0;
        int upto = t;
#pragma unroll
        for (int d = 1; d < kWave; d *= 2) {
            const int v = __shfl_up(upto, d);
            if (lane >= d) upto += v;
        }
        if (lane == kWave - 1) o.wave_sum[wave] = upto;
        __syncthreads();
        int before = all;
        for (int w = 0; w < WAVES; ++w) {
            if (w < wave) before += o.wave_sum[w];
            all += o.wave_sum[w];
        }
        if (e < a.E) o.before[e] = before + upto - t;
        __syncthreads();
    }
    if (tid == 0) o.before[a.E] = all;
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(all);
}

// Tile t: of `tiles_m` tiles of rows by tiles_n of UNITS outputs, an expert's
// tiles of rows SIDE at a time beside each other for each tile of outputs.  Its
// rows are spread evenly over its tiles, in 16s.
template <int UNITS, int SIDE>
__device__ __forceinline__ void locate(const Args& a, const Tiles& tiles, int tiles_m, uint32_t tiles_n, uint32_t t,
                                       Where& o)
{
    const int lane = threadIdx.x & (kWave - 1);
    int e = 0, first = 0, mt = tiles_m;
    if (a.count != nullptr) {
        // the last expert whose tiles start at or before t, in two probes
        const int per = (a.E + kWave - 1) / kWave;
        auto starts = [&](int i) { return i < a.E && (uint32_t)tiles.before[min(i, a.E)] * tiles_n <= t; };
        const int g = (63 - (int)__builtin_clzll(__ballot(starts(lane * per)))) * per;
        e = g + 63 - (int)__builtin_clzll(__ballot(lane < per && starts(g + lane)));
        e = __builtin_amdgcn_readfirstlane(e);
        first = __builtin_amdgcn_readfirstlane(tiles.before[e]);
        mt = __builtin_amdgcn_readfirstlane(tiles.before[e + 1]) - first;
    }
    const uint32_t i = t - (uint32_t)first * tiles_n;
    const uint32_t band = i / (SIDE * tiles_n), r = i - band * SIDE * tiles_n;
    const uint32_t side = min((uint32_t)SIDE, (uint32_t)mt - band * SIDE);
    o.m = (int)(r % side);
    o.side = (int)side;
    const uint32_t m = band * SIDE + (uint32_t)o.m;
    int64_t row0;
    const int64_t rows = rows_of(a, e, &row0, false), each = ((rows + 15) / 16 + mt - 1) / mt * 16;
    const int64_t from = row0 + m * each, left = rows - m * each;
    o.expert = e;
    o.unit0 = (int)(r / side) * UNITS;
    o.rows = __builtin_amdgcn_readfirstlane((int)(left < each ? left : each));
    o.row0 = (int64_t)__builtin_amdgcn_readfirstlane((int)(from >> 32)) << 32 |
             (uint32_t)__builtin_amdgcn_readfirstlane((int)from);
}

// ---- the tiled kernel -----------------------------------------------------------

template <int BM, int BN, int WM, int WN, int S, bool GATE, bool SPLIT>
__global__ __launch_bounds__(64 * WM * WN, (WM * WN / 4 * Tile<BM, BN, WM, WN, S, GATE>::kBlocks)) void k_matmul(Args a)
{
    using T = Tile<BM, BN, WM, WN, S, GATE>;
    constexpr int MT = T::MT, NT = T::NT;
    extern __shared__ __align__(1024) unsigned char smem[];     // stages, scales of kScales tiles
    __shared__ Tiles tiles;
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int wm = wave % WM, wn = wave / WM;
    const int n = lane & 15, c = lane >> 4;
    const int tiles_m = count_tiles<BM, T::kWaves>(a, tiles);
    const uint32_t tiles_n = (uint32_t)((a.units + T::kUnits - 1) / T::kUnits);
    const uint32_t whole = (uint32_t)tiles_m * tiles_n;         // below 2^32: rows * outputs are below 2^35
    const uint32_t total = SPLIT ? whole * (uint32_t)a.splits : whole;
    const uint32_t xcd = blockIdx.x % 8, stride = gridDim.x / 8;
    const uint32_t share = total / 8, more = total % 8;
    uint32_t at = xcd * share + min(xcd, more);
    const uint32_t stop = at + share + (xcd < more ? 1u : 0u);
    at += blockIdx.x / 8;
    if (at >= stop) return;

    const int steps = (a.cols + kStep - 1) / kStep;
    // a tile; SPLIT: and its share of the steps
    auto find = [&](uint32_t t, Where& o) {
        if constexpr (SPLIT) {
            o.split = (int)(t / whole);
            o.first = o.split * steps / a.splits;
            o.steps = (o.split + 1) * steps / a.splits - o.first;
            t %= whole;
        }
        locate<T::kUnits, 4>(a, tiles, tiles_m, tiles_n, t, o);
    };

    // ---- loads, S - 1 stages ahead of the arithmetic
    const int l_row = lane / 8, l_piece = lane % 8 ^ l_row;
    const bool l_up = GATE && wave * T::kLoadRows / 16 % 2;     // this wave loads up rows
    const int last_cols = a.cols - (steps - 1) * kStep;         // of the last step
    uint32_t xo[T::kXLoads], wo[T::kWLoads];
    Buffer xb, wb;
    int l_step = 0, l_k = 0, l_first = 0, l_steps = 0, l_scales = 0;
    uint32_t l_tile = at;
    unsigned char* const scales = smem + S * T::kStageBytes;
    auto aim = [&] {
        Where p;
        find(l_tile, p);
        xb = make_buffer(a.x + p.row0 * a.cols, (int64_t)p.rows * a.cols);
#pragma unroll
        for (int j = 0; j < T::kXLoads; ++j) {
            const int r = (j * T::kWaves + wave) * T::kLoadRows + l_row;
            xo[j] = r < p.rows ? (uint32_t)r * (uint32_t)a.cols + 16u * l_piece : kNowhere;
        }
        const int have = min(T::kUnits, a.units - p.unit0);
        const int64_t w0 = (int64_t)p.expert * a.rows + (l_up ? a.units : 0) + p.unit0;
        wb = make_buffer(a.w + w0 * a.cols, (int64_t)have * a.cols);
#pragma unroll
        for (int j = 0; j < T::kWLoads; ++j) {
            const int r = (j * T::kWaves + wave) * T::kLoadRows + l_row;
            const int u = GATE ? r / 32 * 16 + r % 16 : r;
            wo[j] = u < have ? (uint32_t)u * (uint32_t)a.cols + 16u * l_piece : kNowhere;
        }
        if constexpr (!SPLIT) {
            // scales of its rows, then of its outputs in the order of the groups
            const Buffer xs = make_buffer(a.x_scales + p.row0, 4 * (int64_t)p.rows);
            const Buffer ws = make_buffer(a.w_scales + (int64_t)p.expert * a.rows, 4 * (int64_t)a.rows);
            for (int q = wave; q < T::kScaleLoads; q += T::kWaves) {
                unsigned char* const to = scales + l_scales * T::kScaleBytes + q * 256;
                if (q < BM / 64) {
                    load_word_to_lds(xs, to, (uint32_t)(q * 64 + lane) * 4);
                } else {
                    const int r = (q - BM / 64) * 64 + lane;
                    const int u = p.unit0 + (GATE ? r / 32 * 16 + r % 16 : r);
                    load_word_to_lds(ws, to, u < a.units ? (uint32_t)(u + (GATE && r / 16 % 2 ? a.units : 0)) * 4 : kNowhere);
                }
            }
            l_scales = l_scales == T::kScales - 1 ? 0 : l_scales + 1;
        }
        // Where a tile's columns begin.  (One matrix of many rows: at 0, where blocks
        // side by side share what they read; 4096 rows, 7168 -> 4096 102 us, turned
        // 105.  Of few rows: 64 rows, 4096 -> 65536 turned 51 us, all from 0 63.)
        if constexpr (SPLIT) {
            l_first = l_k = p.first;
            l_steps = p.steps;
        }
        if (a.count != nullptr || tiles_m == 1) {
            const int turn = 3 * (p.unit0 / T::kUnits) + 2 * p.m;
            if constexpr (SPLIT) l_k = l_first + turn % l_steps;
            else l_k = turn % (p.side == 1 ? steps : min(4, steps));
        }
    };
    auto load_stage = [&](int buf) {
        if (l_tile >= stop) return;
        unsigned char* const to = smem + buf * T::kStageBytes + wave * 1024;
        const uint32_t k0 = (uint32_t)l_k * kStep;
        const bool past = l_k == steps - 1 && 16 * l_piece >= last_cols;
#pragma unroll
        for (int j = 0; j < T::kXLoads; ++j)
            load_to_lds(xb, to + j * T::kWaves * 1024, past ? kNowhere : xo[j], k0);
#pragma unroll
        for (int j = 0; j < T::kWLoads; ++j)
            load_to_lds(wb, to + BM * kStep + j * T::kWaves * 1024, past ? kNowhere : wo[j], k0);
        if constexpr (SPLIT) l_k = l_k == l_first + l_steps - 1 ? l_first : l_k + 1;
        else l_k = l_k == steps - 1 ? 0 : l_k + 1;
        if (++l_step == (SPLIT ? l_steps : steps)) {
            l_step = 0;
            l_tile += stride;
            if (l_tile < stop) aim();
        }
    };

    // operands of half h of a step: 16 rows, the lane's 16 of 64 columns
    const int frag = n * kStep, piece = c ^ (n & 7);
    auto operand = [&](int buf, int row, int h) {
        return *reinterpret_cast<const i32x4*>(smem + buf * T::kStageBytes + row * kStep + frag + (piece ^ 4 * h) * 16);
    };

    aim();
#pragma unroll 1
    for (int s = 0; s < S - 1; ++s) load_stage(s);
    Where p;
    find(at, p);
    int live = (p.rows + 15) / 16, scale_buf = 0;   // groups of rows; scales
    i32x4 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    int step = 0, buf = 0;
    for (;;) {
        // this step's columns have arrived, and at the barrier for every wave;
        // the stage that is loaded next has been read.  (Behind the last load
        // nothing newer is on its way.)
        if (l_tile < stop) asm volatile("s_waitcnt vmcnt(%0)" ::"n"((S - 2) * T::kLoads) : "memory");
        else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        load_stage(buf == 0 ? S - 1 : buf - 1);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            i32x4 xf[MT], wf[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) wf[j] = operand(buf, BM + (wn * NT + j) * 16, h);
#pragma unroll
            for (int i = 0; i < MT; ++i) xf[i] = operand(buf, (i * WM + wm) * 16, h);
#pragma unroll
            for (int i = 0; i < MT; ++i)
                if (__builtin_expect(i * WM + wm < live, 1)) {
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[j], xf[i], acc[i][j], 0, 0, 0);
                }
        }
        buf = buf == S - 1 ? 0 : buf + 1;
        if (++step < (SPLIT ? p.steps : steps)) continue;
        step = 0;

        if constexpr (SPLIT) {
            // the sums as they are, in the order of the weight rows
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int m = (i * WM + wm) * 16 + n;
                if (m >= p.rows) continue;
                int32_t* const to = a.part + ((int64_t)p.split * a.num_rows + p.row0 + m) * a.rows;
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const int g = wn * NT + j;
                    const int u = p.unit0 + (GATE ? g / 2 : g) * 16 + 4 * c;
                    int32_t* const at4 = to + u + (GATE && g % 2 ? a.units : 0);
                    if (u + 4 <= a.units) {
                        *reinterpret_cast<AnySums*>(at4) = acc[i][j];
                    } else {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            if (u + q < a.units) at4[q] = acc[i][j][q];
                    }
                }
            }
        } else {
            // ---- store: this lane has outputs 4c .. 4c+3 of row n of each group
            constexpr int NO = GATE ? NT / 2 : NT;      // groups of outputs
            const float* const xs = reinterpret_cast<const float*>(scales + scale_buf * T::kScaleBytes) + n;
            const f32x4* const ws =
                reinterpret_cast<const f32x4*>(scales + scale_buf * T::kScaleBytes + 4 * BM) + wn * NT * 4 + c;
            f32x4 w4[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) w4[j] = ws[j * 4];
            const int u0 = p.unit0 + wn * NO * 16;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int m = (i * WM + wm) * 16 + n;
                if ((i * WM + wm) * 16 >= p.rows) continue;
                const float x1 = xs[(i * WM + wm) * 16];
                uint32_t lo[NO], hi[NO];
#pragma unroll
                for (int o = 0; o < NO; ++o) {
                    float v[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        v[q] = (float)acc[i][GATE ? 2 * o : o][q] * x1 * w4[GATE ? 2 * o : o][q];
                        // (the exponential is good to 2^-24 of its argument)
                        if constexpr (GATE)
                            v[q] = v[q] / (1.f + __expf(-v[q])) * ((float)acc[i][2 * o + 1][q] * x1 * w4[2 * o + 1][q]);
                    }
                    const u32x2 d = __builtin_bit_cast(u32x2, __builtin_convertvector(f32x4{v[0], v[1], v[2], v[3]}, bf16x4));
                    lo[o] = d[0];
                    hi[o] = d[1];
                }
                uint16_t* const to = a.y + (p.row0 + m) * a.units;
                // two groups: their lanes trade, 8 outputs of one group each
#pragma unroll
                for (int o = 0; o + 1 < NO; o += 2) {
                    swap16(lo[o], lo[o + 1]);
                    swap16(hi[o], hi[o + 1]);
                    const int u = u0 + (o + c % 2) * 16 + c / 2 * 8;
                    const u32x4 d = {lo[o], hi[o], lo[o + 1], hi[o + 1]};
                    if (m < p.rows && u + 8 <= a.units) {
                        *reinterpret_cast<Any16*>(to + u) = d;
                    } else if (m < p.rows) {
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            if (u + q < a.units) to[u + q] = (uint16_t)(d[q / 2] >> (q % 2 * 16));
                    }
                }
                if constexpr (NO % 2 != 0) {
                    const int u = u0 + (NO - 1) * 16 + 4 * c;
                    const u32x2 d = {lo[NO - 1], hi[NO - 1]};
                    if (m < p.rows && u + 4 <= a.units) {
                        *reinterpret_cast<Any8*>(to + u) = d;
                    } else if (m < p.rows) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            if (u + q < a.units) to[u + q] = (uint16_t)(d[q / 2] >> (q % 2 * 16));
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
        at += stride;
        if (at >= stop) return;
        scale_buf = scale_buf == T::kScales - 1 ? 0 : scale_buf + 1;
        find(at, p);
        live = (p.rows + 15) / 16;
    }
}

// ---- few rows and outputs of one matrix --------------------------------------------
//
// A block has G groups of 16 outputs (or 16 gate and 16 up rows) of up to 16 rows;
// its waves take the lines of 128 columns in turn, U of them in flight each,
// straight from memory to registers, and add their sums in LDS (exact, so in any
// order).  What bounds it is latency: the 29 MB of 7168 -> 4096 are 115 KB for each
// CU, and what counts is that all of them are asked for at once.  One row 8.3 us
// (15 us with the few-row kernel, whose 32-output tiles leave half of the CUs
// idle), 16 rows 10.4 (14.6).  Each block begins at lines of its own, as the tiles
// above do: one row, 16384 -> 4096 14.4 us, all from line 0 18.2.
//
// A load of weights takes 8 rows x 128 bytes (whole cache lines); of two, lanes
// 0-7 and 8-15 of each row of 16 lanes trade one, which makes two operands: lane
// (n, c) has bytes 32 c + 16 v of row n in operand v.
__device__ __forceinline__ void trade_halves(const u32x4& a, const u32x4& b, i32x4& q0, i32x4& q1)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // row_ror:8, written in lanes 8-15 (banks 2, 3) or 0-7 (banks 0, 1)
        q0[i] = __builtin_amdgcn_update_dpp((int)a[i], (int)b[i], 0x128, 0xF, 0xC, false);
        q1[i] = __builtin_amdgcn_update_dpp((int)b[i], (int)a[i], 0x128, 0xF, 0x3, false);
    }
}

__device__ __forceinline__ u32x4 load_line(Buffer b, uint32_t lane_off, uint32_t off)
{
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, lane_off, off, 0));
}

template <int U, int G, bool GATE>
__global__ __launch_bounds__(kThinWaves* kWave) void k_matmul_thin(Args a)
{
    static_assert(!GATE || G == 2, "a gate and an up group");
    constexpr int NO = GATE ? 1 : G;        // groups of outputs
    __shared__ i32x4 sums[kThinWaves][G][kWave];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int n = lane & 15, c = lane >> 4;
    const int unit0 = blockIdx.x * 16 * NO;
    const int64_t row0 = (int64_t)blockIdx.y * 16;
    const int rows = (int)min((int64_t)16, a.num_rows - row0);
    Buffer wb[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const ThinGroup at = thin_group(unit0, GATE ? 0 : g, a.units);
        wb[g] = make_buffer(a.w + ((GATE ? (int64_t)g * a.units : 0) + at.first) * a.cols, (int64_t)at.have * a.cols);
    }
    const Buffer xb = make_buffer(a.x + row0 * a.cols, (int64_t)rows * a.cols);
    const uint32_t xo = (uint32_t)n * (uint32_t)a.cols + 32u * c;

    i32x4 acc[G];
#pragma unroll
    for (int g = 0; g < G; ++g) acc[g] = i32x4{0, 0, 0, 0};
    const int lines = (a.cols + 127) / 128, turn = (int)(blockIdx.x * 3u % (uint32_t)lines);
    for (int l0 = wave; l0 < lines; l0 += kThinWaves * U) {
        u32x4 w[U][G][2], x[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = l0 + u * kThinWaves, line = at + turn < lines ? at + turn : at + turn - lines;
            const int left = at < lines ? a.cols - line * 128 : 0;              // columns from it on
            const uint32_t off = left > 0 ? (uint32_t)line * 128u : 0u;
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int v = 0; v < 2; ++v)     // (past the last row: past the buffer)
                    w[u][g][v] = load_line(wb[g], thin_offset(lane, v, a.cols, left), off);
#pragma unroll
            for (int v = 0; v < 2; ++v)
                x[u][v] = load_line(xb, n < rows && 32 * c + 16 * v < left ? xo + 16u * v : kNowhere, off);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int g = 0; g < G; ++g) {
                i32x4 q[2];
                trade_halves(w[u][g][0], w[u][g][1], q[0], q[1]);
#pragma unroll
                for (int v = 0; v < 2; ++v)
                    acc[g] = __builtin_amdgcn_mfma_i32_16x16x64_i8(q[v], __builtin_bit_cast(i32x4, x[u][v]), acc[g], 0, 0, 0);
            }
    }
#pragma unroll
    for (int g = 0; g < G; ++g) sums[wave][g][lane] = acc[g];
    __syncthreads();
    // a lane of the first waves has outputs 4c to 4c + 3 of row n, a group a wave
    const int u = unit0 + 16 * wave + 4 * c;
    if (wave >= NO || n >= rows || u >= a.units) return;
    i32x4 sum[GATE ? 2 : 1];
#pragma unroll
    for (int g = 0; g < (GATE ? 2 : 1); ++g) {
        sum[g] = i32x4{0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < kThinWaves; ++w) sum[g] += sums[w][GATE ? g : wave][lane];
    }
    const float x1 = a.x_scales[row0 + n];
    uint16_t* const to = a.y + (row0 + n) * a.units + u;
#pragma unroll
    for (int q = 0; q < 4; ++q)
        if (u + q < a.units) {
            float v = (float)sum[0][q] * x1 * a.w_scales[u + q];
            if constexpr (GATE) v = v / (1.f + __expf(-v)) * ((float)sum[1][q] * x1 * a.w_scales[a.units + u + q]);
            to[q] = __builtin_bit_cast(uint16_t, (__bf16)v);
        }
}

// Joins the sums of tiles whose columns were split over blocks: four outputs of a
// row a thread, in small blocks, since all that counts is that the loads of all
// are under way at once.
template <bool GATE>
__global__ __launch_bounds__(64) void k_matmul_join(Args a)
{
    const uint32_t quads = (uint32_t)(a.units + 3) / 4;
    const uint32_t i = blockIdx.x * 64 + threadIdx.x;
    const int64_t row = i / quads;
    if (row >= a.num_rows) return;
    const int u = (int)(i % quads) * 4;
    constexpr int G = GATE ? 2 : 1;
    i32x4 sum[G];
#pragma unroll
    for (int g = 0; g < G; ++g) sum[g] = i32x4{0, 0, 0, 0};
#pragma unroll 8
    for (int s = 0; s < a.splits; ++s) {
        const int32_t* const from = a.part + (s * a.num_rows + row) * a.rows + u;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            if (u + 4 <= a.units) {
                sum[g] += *reinterpret_cast<const AnySums*>(from + g * a.units);
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (u + q < a.units) sum[g][q] += from[g * a.units + q];
            }
        }
    }
    const float x1 = a.x_scales[row];
    uint16_t* const to = a.y + row * a.units + u;
#pragma unroll
    for (int q = 0; q < 4; ++q)
        if (u + q < a.units) {
            float v = (float)sum[0][q] * x1 * a.w_scales[u + q];
            if constexpr (GATE) v = v / (1.f + __expf(-v)) * ((float)sum[G - 1][q] * x1 * a.w_scales[a.units + u + q]);
            to[q] = __builtin_bit_cast(uint16_t, (__bf16)v);
        }
}

int num_cus()
{
    static const int n = [] {
        int dev = 0, v = 0;
        if (hipGetDevice(&dev) != hipSuccess ||
            hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || v < 8)
            v = 256;
        return v;
    }();
    return n;
}

// Tiles of BM rows that there can be: every expert may end in one of its own, and
// each has a row.
int64_t most_tiles(const Args& a, int64_t rows, int64_t bm)
{
    const int64_t n = (rows + bm - 1) / bm + (a.count ? a.E - 1 : 0);
    return n < rows ? n : rows;
}

template <int BM, int BN, int WM, int WN, int S, bool GATE, bool SPLIT = false>
hipError_t launch_tile(const Args& a, int64_t rows, hipStream_t s)
{
    using T = Tile<BM, BN, WM, WN, S, GATE>;
    const int64_t tiles = most_tiles(a, rows, BM) * ((a.units + T::kUnits - 1) / T::kUnits) * (SPLIT ? a.splits : 1);
    const int64_t most = (int64_t)num_cus() / 8 * T::kBlocks, need = (tiles + 7) / 8;
    const dim3 grid((unsigned)(8 * (need < most ? need : most)));
    (void)hipFuncSetAttribute(reinterpret_cast<const void*>(k_matmul<BM, BN, WM, WN, S, GATE, SPLIT>),
                              hipFuncAttributeMaxDynamicSharedMemorySize, T::kLds);
    hipLaunchKernelGGL((k_matmul<BM, BN, WM, WN, S, GATE, SPLIT>), grid, dim3(T::kThreads), (size_t)T::kLds, s, a);
    return hipGetLastError();
}

template <bool GATE>
hipError_t launch_split(const Args& a, int64_t rows, hipStream_t s)
{
    const hipError_t e = launch_tile<64, 64, 2, 2, stages(kPathTile64x64), GATE, true>(a, rows, s);
    if (e != hipSuccess) return e;
    const int64_t quads = rows * ((a.units + 3) / 4);      // at most 2^20 sums a split
    hipLaunchKernelGGL((k_matmul_join<GATE>), dim3((unsigned)((quads + 63) / 64)), dim3(64), 0, s, a);
    return hipGetLastError();
}

template <int U, int G, bool GATE>
hipError_t launch_thin(const Args& a, int64_t rows, hipStream_t s)
{
    const int outputs = GATE ? 16 : 16 * G;
    const dim3 grid((unsigned)((a.units + outputs - 1) / outputs), (unsigned)((rows + 15) / 16));
    hipLaunchKernelGGL((k_matmul_thin<U, G, GATE>), grid, dim3(kThinWaves * kWave), 0, s, a);
    return hipGetLastError();
}

template <bool GATE>
hipError_t launch_path(Path path, const Args& a, int64_t rows, hipStream_t s)
{
    switch (path) {
        case kPathThin:
            // two lines a wave at once if that is all there are: 2048 columns 4.4 us
            // (4.7 with four), 7168 columns 8.5 (7.9).  Two groups of outputs a block,
            // for one reading of x, where that makes about a block a CU: 16 rows, 18432
            // -> 7168 (224 blocks) 30 us, one group 38; 4096 -> 8192 (256) 9.3 and 10.7;
            // 4096 -> 4096 (128) 8.5 and 7.2, 7168 -> 8704 (272) 23.7 and 23.0, one row
            // 20.3 and 17.3
            if constexpr (!GATE)
                if (const int64_t t = thin_tiles(false, a.units, rows); t >= 448 && t <= 512)
                    return a.cols <= 2 * kThinWaves * 128 ? launch_thin<2, 2, false>(a, rows, s)
                                                          : launch_thin<4, 2, false>(a, rows, s);
            return a.cols <= 2 * kThinWaves * 128 ? launch_thin<2, GATE ? 2 : 1, GATE>(a, rows, s)
                                                  : launch_thin<4, GATE ? 2 : 1, GATE>(a, rows, s);
        case kPathTile64x64: return launch_tile<64, 64, 2, 2, stages(kPathTile64x64), GATE>(a, rows, s);
        case kPathTile64x128: return launch_tile<64, 128, 1, 4, stages(kPathTile64x128), GATE>(a, rows, s);
        case kPathTile128: return launch_tile<128, 128, 2, 2, stages(kPathTile128), GATE>(a, rows, s);
        default: return launch_tile<256, 256, 2, 4, stages(kPathTile256), GATE>(a, rows, s);
    }
}

}  // namespace
}  // namespace mm

int64_t matmul_workspace(bool gate, int64_t cols, int64_t units, int64_t rows)
{
    const int n = mm::choose_splits(gate, cols, units, rows);
    return n > 1 ? 4 * n * rows * units * (gate ? 2 : 1) : 0;
}

hipError_t launch_matmul(const ProductArgs& p, bool gate, int32_t* part, hipStream_t s)
{
    const int64_t rows = p.count ? p.P : p.num_rows, cols = 2 * (int64_t)p.w.cols;
    const mm::Path path = mm::choose_path(gate, cols, p.units, p.count ? p.E : 0, rows);
    if (path == mm::kPathNone) return hipSuccess;
    const int splits = part && !p.count ? mm::choose_splits(gate, cols, p.units, rows) : 1;
    if (path == mm::kPathFew) return launch_product_int8(p, gate ? kSwigluBf16 : kStoreBf16, s);
    mm::Args a = {};
    a.w = p.w.data;
    a.w_scales = reinterpret_cast<const float*>(p.w.scales);
    a.rows = p.w.rows;
    a.cols = (int)cols;
    a.units = p.units;
    a.x = reinterpret_cast<const uint8_t*>(p.x);
    a.x_scales = p.x_scales;
    a.num_rows = p.num_rows;
    a.E = p.E;
    a.psum = p.psum;
    a.count = p.count;
    a.cap = p.cap;
    a.y = static_cast<uint16_t*>(p.y);
    a.flags = p.flags;
    if (splits > 1) {
        a.splits = splits;
        a.part = part;
        return gate ? mm::launch_split<true>(a, rows, s) : mm::launch_split<false>(a, rows, s);
    }
    return gate ? mm::launch_path<true>(path, a, rows, s) : mm::launch_path<false>(path, a, rows, s);
}

}  // namespace epk
