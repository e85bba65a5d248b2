// Orthogonalisation of a list of matrices by a quintic Newton-Schulz iteration:
//
//     X = U / max(|U|_F, eps),  then per step (a, b, c)  X <- a X + (b A + c A A) X,  A = X X^T
//
// on the short side: a matrix with more rows than columns is worked on
// transposed, which its first load and last store do.
//
// What is rounded.  The iterate X and the two symmetric s x s matrices A and
// Q = a I + b A + c A A are held in fp16 between the products, each times a
// power of two that keeps typical entries far from fp16's small end (X: about
// sqrt(l), A and Q: 2^10); every sum is float32, |U|_F float64.  fp16 instead of
// bf16 because the iteration multiplies what is lost: on 1024 x 1024 matrices of
// noise plus a low-rank part the result is 1.1e-3 off (relative, Frobenius)
// with fp16 in these places and 1e-2 with bf16, at the same MFMA rate.  What
// decides where singular values fall is X's rounding after the early steps: what
// it leaves in a zero's place grows by a = 3.4 a step.  1024 x 1024, fp16 U: 2.3e-3
// for 1 / k, 7.5e-3 for 1 / k^2, 3.2e-2 for rank 16, where a model with X in two
// fp16 (three times the products of X, twice its memory) gives 3e-4.
//
// Products.  A step is three, X X^T, A A and Q X, in square tiles of T x T over
// a padded copy in the workspace, so no load is bounded and padding stays zero.
// X X^T and A A are symmetric: only tiles on and below the diagonal are formed,
// and stored twice.  T is 64, 128 or 256 for a whole list (step_cost); what a
// matrix becomes does not depend on it.  A product is one launch, the blocks
// that fit the CUs, which work off lists of tiles.
//
// What bounds it.  14 matrices of 405M elements (8 of 4096 x 4096, 6 of 4096 x
// 11008), us of a step: X X^T 1460, A A 978, Q X 2916, in tiles of 256; with 2 m n
// k for a product, half of it for the symmetric ones, 0.98 to 1.14e15 a second,
// where the loops between a tile's first loads and its stores run at 1.5e15,
// about what a large matrix product of a library reaches.  The MFMAs are busy 58
// to 69% of the time at 1.7 GHz, to which the power limit takes the clock from 2.4:
// more waves, deeper stages and the larger MFMA gain nothing, 32 x 32 x 16 loses 4%.
// HBM is not what bounds: Q X reads and writes 6.2 GB in 2.9 ms.  Small lists are
// bound by their 2 + 3 n_steps launches of 4 to 6 us, one after the other.
#include <hip/hip_runtime.h>

#include <cmath>
#include <type_traits>
#include <vector>

#include "orthogonalize.h"

namespace zero_shard {
namespace {

constexpr int kPanel = 32;                       // columns of a panel, and the inner elements of a stage

enum { kGram, kPoly, kApply };

// ---------------------------------------------------------------- load and norm

// Where element (r, c) of a matrix of `rows` rows is in the workspace: panels
// of 32 columns, each with its rows end to end.  A stage of either operand of
// any product is then made of runs of at least 1 KB.
__device__ __forceinline__ int64_t panel_at(int64_t r, int64_t c, int64_t rows) {
    return ((c / kPanel) * rows + r) * kPanel + c % kPanel;
}

// U is read in pieces of 64 rows and 256 columns (of the s x l matrix), whatever
// the tiles: the norm's sums, and so the results, do not depend on them.
constexpr int kPieceRows = 64, kPieceColumns = kChunkElements / kPieceRows;

template <int D>
__device__ __forceinline__ void load_piece(const ZS_CONSTANT MatrixItem& m, int r0, int c0, float x[8][8]) {
    load_box<kPieceRows, D>(m.udt, m.in, m.s, m.l, m.tall, r0, c0, x);
}

// One piece's sum of squares into its slot.  A read of U: 405M elements of bf16,
// 810 MB, take 129 us, 6.3 TB/s.
__global__ __launch_bounds__(kBlock) void ortho_squares(NsRef ref, int64_t first) {
    if (ref.skipped()) return;
    __shared__ double s_sq[kWaves];
    __shared__ uint32_t s_bad[kWaves];
    const ZS_CONSTANT TileRef& t = ref.tile(first + blockIdx.x);
    const ZS_CONSTANT MatrixItem& m = ref.item(t.item);
    const int r0 = t.i * kPieceRows, c0 = t.j * kPieceColumns;
    if (r0 >= m.s || c0 >= m.l) return;                      // padding alone
    float x[8][8];
    load_piece<kPieceRows>(m, r0, c0, x);
    double acc = 0.0;
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int k = 0; k < 8; ++k) acc = fma((double)x[n][k], (double)x[n][k], acc);
    uint32_t none = 0;
    block_reduce(acc, none, s_sq, s_bad);
    if (threadIdx.x == 0)
        reinterpret_cast<double*>(ref.ws + m.slots)[(int64_t)t.i * ((m.l + kPieceColumns - 1) / kPieceColumns) + t.j] = acc;
}

// max(|U|_F, eps), and NaN if U is not finite.
__device__ __forceinline__ double divisor(const ZS_CONSTANT MatrixItem& m, const char* ws, double eps, double* s_sq,
                                          uint32_t* s_bad) {
    const double* slots = reinterpret_cast<const double*>(ws + m.slots);
    double acc = 0.0;
    for (int k = threadIdx.x; k < m.n_slots; k += kBlock) acc += slots[k];
    uint32_t none = 0;
    block_reduce(acc, none, s_sq, s_bad);
    if (threadIdx.x == 0) s_sq[0] = acc;
    __syncthreads();
    const double norm = sqrt(s_sq[0]);
    return !(norm < INFINITY) ? NAN : norm > eps ? norm : eps;
}

// What is left of X's factor where the iterate is U times a power of two, in (1, 2].
__device__ __forceinline__ double* start_factor(const NsRef& ref, const ZS_CONSTANT MatrixItem& m) {
    return reinterpret_cast<double*>(ref.ws + m.slots) + m.n_slots;
}

// A piece of U times a power of two, 2^log2_scale / max(|U|, eps) to within 2,
// with its padding: a 16-bit U is not rounded by it (but for bf16 elements below
// 2^-14 of the typical one), and the first step's sums take the rest of the factor.
// With all of it here U would be rounded to fp16 once more, and what that leaves in
// a zero singular value's place grows by a in every step: 512 x 512, 1 / k^2, 2.0e-2
// instead of 7.3e-3 off.
// A read and a write: 405M elements take 336 to 358 us, 4.5 to 4.8 TB/s.  Each block
// forms the norm again from the slots, 2752 of them for 4096 x 11008, behind its
// loads; a launch of its own would take 4 us.  Bands of 8 rows at a time, so that a
// wave's stores fill whole rows of a panel.
__global__ __launch_bounds__(kBlock) void ortho_load(NsRef ref, int64_t first, double eps) {
    if (ref.skipped()) return;
    __shared__ double s_sq[kWaves];
    __shared__ uint32_t s_bad[kWaves];
    __shared__ __attribute__((aligned(16))) _Float16 block[kPieceRows][kPieceColumns + 8];
    const ZS_CONSTANT TileRef& t = ref.tile(first + blockIdx.x);
    const ZS_CONSTANT MatrixItem& m = ref.item(t.item);
    const int r0 = t.i * kPieceRows, c0 = t.j * kPieceColumns;
    float x[8][8];
    if (r0 < m.s && c0 < m.l) {
        load_piece<8>(m, r0, c0, x);
    } else {
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int k = 0; k < 8; ++k) x[n][k] = 0.0f;
    }
    const double by = divisor(m, ref.ws, eps, s_sq, s_bad);
    const float keep = by < INFINITY ? 1.0f : NAN;           // of a U that is not finite, all of X is NaN
    int up = 0;
    const double fraction = by > 0.0 && by < INFINITY ? frexp(by, &up) : 1.0;
    if (t.i == 0 && t.j == 0 && threadIdx.x == 0) *start_factor(ref, m) = 1.0 / fraction;
    const int e = m.log2_scale - up;
    _Float16* X = reinterpret_cast<_Float16*>(ref.ws + m.x0);
#pragma unroll
    for (int n = 0; n < 8; ++n) {
        const Vector8<kPieceRows, 8> v(m.s, m.l, m.tall, r0, c0, n);
        h8 h;
#pragma unroll
        for (int k = 0; k < 8; ++k) h[k] = k < v.valid ? (_Float16)(ldexpf(x[n][k], e) * keep) : (_Float16)0;
        if (m.tall) {
#pragma unroll
            for (int k = 0; k < 8; ++k) block[v.r + k][v.c] = h[k];
        } else if (c0 + v.c < m.lp) {
            *reinterpret_cast<h8*>(X + panel_at(r0 + v.r, c0 + v.c, m.sp)) = h;
        }
    }
    if (!m.tall) return;
    __syncthreads();
#pragma unroll
    for (int n = 0; n < 8; ++n) {
        const Vector8<kPieceRows, 8> v(m.s, m.l, 0, r0, c0, n);
        if (c0 + v.c < m.lp) *reinterpret_cast<h8*>(X + panel_at(r0 + v.r, c0 + v.c, m.sp)) = *reinterpret_cast<const h8*>(&block[v.r][v.c]);
    }
}

// ---------------------------------------------------------------- products

// 16 bytes per lane from base + offset straight into the LDS: lane l's at lds + 16 l.
// m0 is not in the list of what it clobbers, where the compiler would ignore it: each
// load sets its own, and a test of the generated code sees that nothing else uses it.
__device__ __forceinline__ void load_lds(const void* base, uint32_t offset, uint32_t lds) {
    __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                     :
                     : "s"(lds), "v"(offset), "s"(base)
                     : "memory");
}

// A wave's share of a T x T tile of a product, WM x WN waves.
//
// A stage is 32 inner elements of both operands, 64 bytes a row: 16 rows for
// each 1 KB that a wave loads at a time, straight into the LDS.  Four stages lie
// there; all but the one that is multiplied and the next are on their way, since
// a load that misses the L2 takes longer than a stage.  (T 256, products of X:
// 2.70 ms with four stages, 2.69 with five, 3.81 with three.)  One barrier a
// stage: behind it the next stage has landed for all waves, and the last one's
// place is free.  At T 64 a stage is four MFMAs a wave, less than its barrier:
// there one barrier serves two stages, of which six lie in the LDS, and three
// blocks fit a CU.  (One matrix of 512 x 512, of 1024 x 8192, four of 1024 x
// 1024: 87, 352 and 208 us; with five stages and a barrier each 92, 384 and 218,
// with five and a barrier for two 98 and more, with eight and two blocks a CU 89.)
//
// Operands in the LDS, as the 16 x 16 x 32 MFMA takes them (lane l: row or
// column l % 16, inner elements 8 (l / 16) .. + 7):
//  rows:     of a matrix whose inner dimension runs along the panel's columns.
//            The 16-byte pieces of row r lie in the order piece ^ row_order(r):
//            the 16 lanes that a 16-byte read serves at a time then meet all 64
//            banks (with piece ^ (r / 4) % 4 two and two of them meet).
//  columns:  the inner dimension runs down the panel's rows, read through the
//            transposing load: 16 lanes take 4 rows of 16 elements.  The 32-byte
//            halves of rows 8 to 15 of 16 are swapped, so that the two groups
//            of rows that a half wave reads meet all banks.
template <int T, int WM, int WN>
struct Product {
    static constexpr int kWaves = WM * WN;
    static constexpr int kUM = T / WM / 16, kUN = T / WN / 16;       // 16 x 16 results per wave
    static constexpr int kOperand = T * kPanel * 2;                  // bytes of a stage
    static constexpr int kLoads = kOperand / 1024 / kWaves;          // per wave and operand
    static constexpr bool kPairs = T == 64;                          // one barrier for two stages
    static constexpr int kStages = kPairs ? 6 : 4;
    static constexpr int kStage = 2 * kOperand;
    static constexpr int kMirrorRows = T == 64 ? 16 : 32;            // 16: three blocks fit a CU
    static constexpr int kMirror = kMirrorRows * (T / WN) * 2;       // of a wave: so many rows of its mirrored results
    static constexpr int kLds = kStages * kStage + kWaves * kMirror;
    static_assert(kLoads >= 1 && kLds <= 160 * 1024, "stages do not fit the LDS");

    // Where this lane reads its n-th piece of an operand of rows, from the first.
    __device__ static __forceinline__ uint32_t row_offset(int wave, int lane, int n) {
        const int r = (wave * kLoads + n) * 16 + lane / 4;
        return (uint32_t)(r * 64 + ((lane & 3) ^ row_order(r)) * 16);
    }
    // ... of an operand of columns, T / 32 panels of 32 rows, from the wave's first panel
    __device__ static __forceinline__ uint32_t column_offset(int wave, int lane, int n) {
        const int r = ((wave * kLoads + n) & 1) * 16 + lane / 4;
        return (uint32_t)(r * 64 + ((lane & 3) ^ ((r >> 2) & 2)) * 16);
    }
    // Where it finds its part of rows 0 .. 15, or of columns 0 .. 15, in the LDS.
    __device__ static __forceinline__ uint32_t row_read(int lane, int first) {
        const int r = first + (lane & 15);
        return (uint32_t)(r * 64 + ((lane >> 4) ^ row_order(r)) * 16);
    }
    __device__ static __forceinline__ uint32_t column_read(int lane, int first) {
        const int r = (lane >> 4) * 8 + ((lane & 15) >> 2), half = (first >> 4) & 1;
        return (uint32_t)((first / kPanel) * 2048 + r * 64 + (half ^ ((r >> 3) & 1)) * 32 + (lane & 3) * 8);
    }
};

// Stages of an inner dimension, an even number: behind them the padding is zero.
__device__ __host__ __forceinline__ int stages_of(int depth) { return (depth + 2 * kPanel - 1) / (2 * kPanel) * 2; }

struct NsStep {
    float a, b, c;
    int32_t odd;                                   // the iterate is in x1
    int32_t first, last;
};

// Four neighbours of a row of X into the caller's matrix.
template <int DT>
__device__ __forceinline__ void store_ortho(const ZS_CONSTANT MatrixItem& m, int64_t row, int64_t col, const float v[4]) {
    uint16_t* out = static_cast<uint16_t*>(m.out);
    if (!m.tall && col + 4 <= m.l) {
        st_any(pack4_16<DT>(v), out + row * m.l + col);
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (col + e >= m.l) break;
        global(out)[m.tall ? (col + e) * m.s + row : row * m.l + col + e] = (uint16_t)to16<DT>(v[e]);
    }
}

// Byte offset in a row of 32 mirrored results of the 16-byte piece that holds column c.
__device__ __forceinline__ int mirror_piece(int r, int c) { return (((c & 31) >> 3) ^ ((r >> 2) & 3)) << 4; }

// Waits until no more than N of this wave's loads are on their way, then for the other waves.
template <int N>
__device__ __forceinline__ void wait_stage() {
    __asm__ volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(N) : "memory");
}

// What a wave loads for a tile: where its operands begin, how far a stage moves
// them, and the stages.
struct Source {
    const char *m, *n;
    int64_t move_m, move_n;
    int stages;
};

template <int T, int WM, int WN, int MODE>
__device__ __forceinline__ Source source_of(const NsRef& ref, const TileRef tile, const NsStep& step, int wave) {
    using P = Product<T, WM, WN>;
    const ZS_CONSTANT MatrixItem& m = ref.item(tile.item);
    const char* X = ref.ws + (step.odd ? m.x1 : m.x0);
    const int64_t panel = (int64_t)m.sp * 64;
    if constexpr (MODE == kApply) {
        return Source{X + ((int64_t)tile.j * (T / kPanel) + ((wave * P::kLoads) >> 1)) * panel, ref.ws + m.b + tile.i * (T * 64),
                      kPanel * 64, panel, stages_of(m.s)};
    } else {
        const char* from = MODE == kGram ? X : ref.ws + m.a;
        return Source{from + tile.i * (T * 64), from + tile.j * (T * 64), panel, panel, stages_of(MODE == kGram ? m.l : m.s)};
    }
}

// The tiles of a product, block b taking tiles b, b + blocks, ... as far as there
// are any.  M runs over a tile's rows for kGram and kPoly and over its columns for kApply, so that a
// lane ends with four neighbours of a stored row: rows of X for kApply, of the
// transposed tile for the others.
//
// The loads run on from tile to tile: the next one's first stages land while
// this one's last are multiplied and its results leave.  (With a block per tile
// and one block a CU, all CUs loaded, multiplied and stored in step: 23 us a
// tile besides its stages at T 256, of 116 with 128 stages.)
template <int T, int WM, int WN, int MODE>
__global__ __launch_bounds__(64 * WM * WN) void ortho_product(NsRef ref, int64_t first, int64_t n_tiles, NsStep step) {
    using P = Product<T, WM, WN>;
    constexpr int UM = P::kUM, UN = P::kUN, L = P::kLoads, S = P::kStages, NL = 2 * L;
    if (ref.skipped()) return;
    __shared__ __attribute__((aligned(1024))) char smem[P::kLds];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int wm = wave / WN * (T / WM), wn = wave % WN * (T / WN);
    const auto tile_at = [&](int64_t i) {
        const ZS_CONSTANT TileRef& t = ref.tile(first + i);
        return TileRef{t.item, t.i, t.j};
    };
    uint32_t om[L], on[L];
#pragma unroll
    for (int q = 0; q < L; ++q) {
        on[q] = P::row_offset(wave, lane, q);
        om[q] = MODE == kApply ? P::column_offset(wave, lane, q) : on[q];
    }
    const uint32_t lds = lds_address(smem), mine = lds + wave * L * 1024;
    TileRef tile = tile_at(blockIdx.x);
    if (tile.item == kNoItem) return;
    Source now = source_of<T, WM, WN, MODE>(ref, tile, step, wave), then = now;
    int n = now.stages, left = n;
    uint32_t put = 0;
    const auto load = [&](int q) {                 // the q-th load of a stage
        if (q < L) load_lds(now.m, om[q], mine + put + q * 1024);
        else load_lds(now.n, on[q - L], mine + put + P::kOperand + (q - L) * 1024);
        if (q == NL - 1) {
            const bool over = --left == 0;
            now.m = over ? then.m : now.m + now.move_m;
            now.n = over ? then.n : now.n + now.move_n;
            now.move_m = over ? then.move_m : now.move_m;
            now.move_n = over ? then.move_n : now.move_n;
            left = over ? then.stages : left;
            put = put == (S - 1) * P::kStage ? 0 : put + P::kStage;
        }
    };

    f32x4 acc[UM][UN];
    h8 fm[UM], fn[2][UN];
    const uint32_t an = lds + P::kOperand + P::row_read(lane, wn);
    const uint32_t am = lds + (MODE == kApply ? 0u : P::row_read(lane, wm));
    // columns: 16 of a panel's 32 at a time; the two halves lie 32 bytes apart, either way round
    const uint32_t ac0 = lds + P::column_read(lane, wm), ac1 = lds + P::column_read(lane, wm + 16);
    const auto read_m = [&](uint32_t stage, int x) {
        if constexpr (MODE == kApply) {
            const uint32_t a = (x & 1 ? ac1 : ac0) + stage + (x >> 1) * 2048;
            return __builtin_shufflevector(lds_column(a), lds_column(a + 4 * 64), 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
            return lds_h8(am + stage + x * 1024);
        }
    };
    uint32_t next = 0;
    // One stage's products.  Between them, in this order, the loads of the stage
    // S - 1 ahead and the reads of the next one: a row of M is read as soon as
    // its products are issued, N into the other half of fn.
    const auto multiply = [&](auto half) {
        constexpr int p = decltype(half)::value;
        constexpr int kSlots = UM * UN;
#pragma unroll
        for (int x = 0; x < UM; ++x) {
#pragma unroll
            for (int y = 0; y < UN; ++y) {
                acc[x][y] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fm[x], fn[p][y], acc[x][y], 0, 0, 0);
                const int slot = x * UN + y;
                const int q = slot * NL / kSlots;
                if (q < (slot + 1) * NL / kSlots) load(q);
                const int k = slot * UN / kSlots;
                if (k < (slot + 1) * UN / kSlots) fn[1 - p][k] = lds_h8(an + next + k * 1024);
                if (y == UN - 1) fm[x] = read_m(next, x);
                if (slot & 1) __builtin_amdgcn_sched_barrier(0);
            }
        }
        next = next == (S - 1) * P::kStage ? 0 : next + P::kStage;
    };

    for (int k = 0; k < S - 1; ++k)                // every tile has more
#pragma unroll
        for (int q = 0; q < NL; ++q) load(q);
    wait_stage<(S - 2) * NL>();
#pragma unroll
    for (int y = 0; y < UN; ++y) fn[0][y] = lds_h8(an + y * 1024);
#pragma unroll
    for (int x = 0; x < UM; ++x) fm[x] = read_m(0, x);
    next = P::kStage;
    int landed = 0;                                // stages of this tile that need no wait
    for (int64_t index = blockIdx.x; tile.item != kNoItem; index += gridDim.x) {
        // behind the last tile one of its stages is read again, into places that nothing reads any more
        TileRef following{kNoItem, 0, 0};
        if (index + (int64_t)gridDim.x < n_tiles) following = tile_at(index + gridDim.x);
        if (following.item != kNoItem) {
            then = source_of<T, WM, WN, MODE>(ref, following, step, wave);
        } else {
            then = Source{now.m, now.n, 0, 0, INT32_MAX};
        }
        float rest = 1.0f;                         // read here: its latency passes behind the stages
        if (MODE != kPoly && step.first) rest = (float)*(const ZS_CONSTANT double*)start_factor(ref, ref.item(tile.item));
#pragma unroll
        for (int x = 0; x < UM; ++x)
#pragma unroll
            for (int y = 0; y < UN; ++y) acc[x][y] = f32x4{};
        for (int k = 0; k < n; k += 2) {
            if constexpr (P::kPairs) {
                // this wave's reads of stage k are done too: its place is filled behind this barrier
                __asm__ volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                if (k + 1 >= landed) wait_stage<(S - 4) * NL>();
                else __asm__ volatile("s_barrier" ::: "memory");
                multiply(std::integral_constant<int, 0>{});
                multiply(std::integral_constant<int, 1>{});
            } else {
                if (k >= landed) wait_stage<(S - 3) * NL>();
                else __asm__ volatile("s_barrier" ::: "memory");
                multiply(std::integral_constant<int, 0>{});
                if (k + 1 >= landed) wait_stage<(S - 3) * NL>();
                else __asm__ volatile("s_barrier" ::: "memory");
                multiply(std::integral_constant<int, 1>{});
            }
        }
        // What is on its way has had a stage's time: with it landed, the stores below
        // are the oldest that a later wait waits for.
        __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
        landed = S - 2;

        const ZS_CONSTANT MatrixItem& m = ref.item(tile.item);
        const int64_t sp = m.sp;
        const int ti = tile.i, tj = tile.j;
        // a lane holds four neighbours along M of one N
        const int im = wm + (lane >> 4) * 4, in = wn + (lane & 15);
        const int64_t at0 = MODE == kApply ? panel_at((int64_t)ti * T + in, (int64_t)tj * T + im, sp)
                                           : panel_at((int64_t)tj * T + in, (int64_t)ti * T + im, sp);
        const auto at = [&](int x, int y) { return at0 + (x >> 1) * sp * kPanel + (x & 1) * 16 + y * 16 * kPanel; };
        if constexpr (MODE == kApply) {
            const float scale = ldexpf(rest, step.last ? -kLog2A - m.log2_scale : -kLog2A);
            _Float16* out = reinterpret_cast<_Float16*>(ref.ws + (step.odd ? m.x0 : m.x1));
#pragma unroll
            for (int x = 0; x < UM; ++x)
#pragma unroll
                for (int y = 0; y < UN; ++y) {
                    float v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = as_float(acc[x][y][e] * scale);
                    if (!step.last) {
                        *reinterpret_cast<h4*>(out + at(x, y)) = h4{(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]};
                        continue;
                    }
                    const int64_t row = (int64_t)ti * T + in + y * 16, col = (int64_t)tj * T + im + x * 16;
                    if (row >= m.s) continue;
                    if (m.odt == ZERO_F16) store_ortho<ZERO_F16>(m, row, col, v);
                    else store_ortho<ZERO_BF16>(m, row, col, v);
                }
        } else {
            // (c, r .. r + 3) is what a lane holds of the symmetric result; its mirror
            // (r .. r + 3, c) goes through the LDS, 32 rows at a time, to leave in
            // whole rows of a panel
            const float scale = MODE == kGram ? ldexpf(rest * rest, kLog2A - 2 * m.log2_scale) : step.c * ldexpf(1.0f, -kLog2A);
            const float diagonal = step.a * (1 << kLog2A);
            const _Float16* old = reinterpret_cast<const _Float16*>(ref.ws + m.a);
            _Float16* out = reinterpret_cast<_Float16*>(ref.ws + (MODE == kGram ? m.a : m.b));
            char* mirror_at = smem + S * P::kStage + wave * P::kMirror;
#pragma unroll
            for (int x = 0; x < UM; x += P::kMirrorRows / 16) {
#pragma unroll
                for (int z = 0; z < P::kMirrorRows / 16; ++z)
#pragma unroll
                    for (int y = 0; y < UN; ++y) {
                        const int r = z * 16 + (lane >> 4) * 4, c = y * 16 + (lane & 15);
                        h4 h;
                        if constexpr (MODE == kGram) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) h[e] = to_half(acc[x + z][y][e] * scale);
                        } else {
                            const h4 a = *reinterpret_cast<const h4*>(old + at(x + z, y));
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float v = fmaf(step.b, (float)a[e], acc[x + z][y][e] * scale);
                                h[e] = to_half(ti == tj && im + (x + z) * 16 + e == in + y * 16 ? v + diagonal : v);
                            }
                        }
                        *reinterpret_cast<h4*>(out + at(x + z, y)) = h;
                        if (ti == tj) continue;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            *reinterpret_cast<_Float16*>(mirror_at + ((c / kPanel) * P::kMirrorRows + r + e) * 64 + mirror_piece(r, c) + (c & 7) * 2) = h[e];
                    }
                if (ti == tj) continue;
                __asm__ volatile("s_waitcnt lgkmcnt(0)" ::: "memory");     // a wave reads what it wrote
#pragma unroll
                for (int k = 0; k < P::kMirror / 1024; ++k) {
                    const int piece = k * 64 + lane, r = piece / 4 % P::kMirrorRows, c = piece / (4 * P::kMirrorRows) * kPanel + (piece & 3) * 8;
                    const h8 h = *reinterpret_cast<const h8*>(mirror_at + ((c / kPanel) * P::kMirrorRows + r) * 64 + mirror_piece(r, c));
                    *reinterpret_cast<h8*>(out + panel_at((int64_t)ti * T + wm + x * 16 + r, (int64_t)tj * T + wn + c, sp)) = h;
                }
                __asm__ volatile("s_waitcnt lgkmcnt(0)" ::: "memory");     // before the next 32 rows
            }
        }
        tile = following;
        n = then.stages;
    }
    wait_stage<0>();                               // nothing may land once the LDS is another workgroup's
}

// ---------------------------------------------------------------- host side

// What one step of the products is taken to cost with tiles of this size, in
// microseconds: per product the larger of one tile's chain of stages and of all
// tiles over the CUs.  A tile costs c0 besides its stages, and a chain of stages
// alone in its CU is slower than several (c1 against c1_full).  Measured with
// tiles of 64, 128 and 256 on 24 lists: one matrix of 512 x 512 takes 87, 142 and
// 273 us, 64 of 512 x 2048 1292, 1063 and 941, one of 4096 x 4096 2067, 1541 and
// 1434, 4 of 1024 x 1024 208, 224 and 428; the size that this picks is within 5%
// of the fastest on all of them.
double step_cost(const std::vector<OrthoMatrix>& matrices, int tile) {
    const double c0 = tile == 256 ? 12.0 : tile == 128 ? 2.4 : 0.55, first = tile == 256 ? 12.0 : tile == 128 ? 5.0 : 2.3;
    const double c1 = tile == 256 ? 0.68 : tile == 128 ? 0.23 : 0.17, c1_full = tile == 256 ? 0.68 : tile == 128 ? 0.28 : 0.098;
    double cost = 0.0;
    for (int product = 0; product < 3; ++product) {
        double tiles = 0.0, work = 0.0, deepest = 0.0;
        for (const OrthoMatrix& m : matrices) {
            const int64_t s = std::min(m.rows, m.cols), l = std::max(m.rows, m.cols);
            if (s <= kThin) continue;
            const double n = (double)((s + tile - 1) / tile), nl = (double)((l + tile - 1) / tile);
            const double k = product == kApply ? n * nl : n * (n + 1) / 2, depth = stages_of((int)(product == kGram ? l : s));
            tiles += k;
            work += k * depth;
            deepest = std::max(deepest, depth);
        }
        double full = (work * c1_full + tiles * c0) / 256;
        if (tile == 256) full *= std::ceil(tiles / 256) / (tiles / 256);       // one tile a CU
        cost += std::max(first + c1 * deepest, full);
    }
    return cost;
}

// A matrix's places in the workspace, from *at on.
void place_item(MatrixItem* it, int64_t* at) {
    const int64_t x = (int64_t)it->sp * it->lp * 2, a = (int64_t)it->sp * it->sp * 2;
    it->x0 = place(at, x);
    it->x1 = place(at, x);
    it->a = place(at, a);
    it->b = place(at, a);
    it->slots = place(at, (int64_t)(it->n_slots + 1) * 8);
}

constexpr int kXCDs = 8, kCUs = 256;
constexpr int64_t kMostTiles = 1 << 26;      // beyond any GPU's memory

// Blocks of a product: as many as the LDS lets the CUs hold.
int most_blocks(int tile) { return kCUs * (tile == 256 ? 1 : tile == 128 ? 2 : 3); }

// The tiles of the symmetric products (lower triangle), or of the iterate, of
// the items from `first` on, as rounds of one tile per block.  Blocks go to the
// eight XCDs in turn.  Of the tiles of one depth each XCD takes an equal run,
// within a matrix four tile rows at a time and column by column, so that its
// tiles share their operands in one L2; the deepest come first, and a tile goes
// to the block of its XCD that has the least to do (405M list: 1.35 ms for
// X X^T, 1.50 with every 256th tile to a block).
void add_tiles(OrthoPlan* plan, size_t first, int tile, bool symmetric, int32_t* blocks) {
    constexpr int kBand = 4;
    const double besides = tile == 256 ? 8.0 : 10.0;         // stages that a tile costs besides its own
    const auto depth = [&](uint32_t k) { return stages_of(symmetric ? plan->items[k].l : plan->items[k].s); };
    std::vector<uint32_t> order;
    for (size_t k = first; k < plan->items.size(); ++k) order.push_back((uint32_t)k);
    std::stable_sort(order.begin(), order.end(), [&](uint32_t a, uint32_t b) { return depth(a) > depth(b); });
    std::vector<std::pair<double, std::vector<TileRef>>> runs;       // of one depth
    int64_t all = 0;
    for (const uint32_t k : order) {
        const double cost = depth(k) + besides;
        if (runs.empty() || runs.back().first != cost) runs.push_back({cost, {}});
        std::vector<TileRef>& run = runs.back().second;
        const int n = plan->items[k].sp / tile, nl = symmetric ? n : plan->items[k].lp / tile;
        for (int i0 = 0; i0 < n; i0 += kBand)
            for (int j = 0; j < (symmetric ? std::min(i0 + kBand, n) : nl); ++j)
                for (int i = symmetric ? std::max(i0, j) : i0; i < std::min(i0 + kBand, n); ++i)
                    run.push_back({k, (uint16_t)i, (uint16_t)j});
        all += (int64_t)n * nl;
    }
    *blocks = (int32_t)std::min<int64_t>(most_blocks(tile), pad_to(all, kXCDs));
    struct Block {
        double load;
        int index;
        bool operator<(const Block& o) const { return load != o.load ? load > o.load : index > o.index; }     // for a heap with the least on top
    };
    std::vector<std::vector<Block>> heaps(kXCDs);
    for (int b = 0; b < *blocks; ++b) heaps[b % kXCDs].push_back({0.0, b});
    std::vector<std::vector<TileRef>> work(*blocks);
    size_t offset = 0;                                       // the XCD that the next run's odd tiles begin with
    for (const auto& [cost, run] : runs) {
        size_t next = 0;
        for (int x = 0; x < kXCDs; ++x) {
            const size_t xcd = (x + offset) % kXCDs, share = run.size() / kXCDs + ((size_t)x < run.size() % kXCDs);
            for (size_t k = 0; k < share; ++k) {
                std::vector<Block>& heap = heaps[xcd];
                std::pop_heap(heap.begin(), heap.end());
                work[heap.back().index].push_back(run[next++]);
                heap.back().load += cost;
                std::push_heap(heap.begin(), heap.end());
            }
        }
        offset += run.size();
    }
    size_t rounds = 0;
    for (const auto& w : work) rounds = std::max(rounds, w.size());
    for (size_t r = 0; r < rounds; ++r)
        for (const auto& w : work) plan->tiles.push_back(r < w.size() ? w[r] : TileRef{kNoItem, 0, 0});
}

template <int MODE>
int launch_product(const OrthoPass& p, const NsRef& ref, const NsStep& step, hipStream_t s) {
    const int64_t first = MODE == kApply ? p.x_first : p.sym_first, n = MODE == kApply ? p.n_x : p.n_sym;
    const dim3 grid((unsigned)(MODE == kApply ? p.x_blocks : p.sym_blocks));
    if (p.tile == 256)
        hipLaunchKernelGGL((ortho_product<256, 2, 4, MODE>), grid, dim3(512), 0, s, ref, first, n, step);
    else if (p.tile == 128)
        hipLaunchKernelGGL((ortho_product<128, 2, 2, MODE>), grid, dim3(256), 0, s, ref, first, n, step);
    else
        hipLaunchKernelGGL((ortho_product<64, 2, 2, MODE>), grid, dim3(256), 0, s, ref, first, n, step);
    return launch_status("ortho_product");
}

// The largest of what a step makes of singular values x in [0, top]: |x (a + b y +
// c y^2)| with y = x^2, |b y + c y^2| and |a + b y + c y^2|, from their values at the
// ends and where their derivatives vanish.
struct StepRange {
    double next, poly, factor;
};

StepRange step_range(double a, double b, double c, double top) {
    StepRange m{0.0, 0.0, std::fabs(a)};
    const double end = top * top;
    const auto at = [&](double y) {
        if (!(y > 0.0 && y <= end)) return;
        const double p = y * (b + c * y);
        m.poly = std::max(m.poly, std::fabs(p));
        m.factor = std::max(m.factor, std::fabs(a + p));
        m.next = std::max(m.next, std::sqrt(y) * std::fabs(a + p));
    };
    at(end);
    at(-0.5 * b / c);                            // b + 2 c y = 0
    const double d = 9.0 * b * b - 20.0 * a * c; // a + 3 b y + 5 c y^2 = 0
    if (d >= 0.0) {
        const double q = -0.5 * (3.0 * b + std::copysign(std::sqrt(d), b));
        at(q / (5.0 * c));
        at(a / q);
    }
    return m;
}

// The singular values start in [0, 1].  What each step makes of the largest
// interval they can be in has to stay within what fp16 holds of X, A and B at
// their scales, with room for single entries, and well above its small end.
int check_coefs(const double* coefs, int32_t n_steps, OrthoSteps* steps) {
    if (coefs == nullptr) return fail(ZERO_EINVAL, "coefs is NULL");
    if (n_steps < 1 || n_steps > ZERO_MAX_ORTHO_STEPS)
        return fail(ZERO_EINVAL, "n_steps must lie in [1, %d] (got %d)", ZERO_MAX_ORTHO_STEPS, n_steps);
    double top = 1.0, run = 1.0;
    *steps = OrthoSteps{};
    steps->n = n_steps;
    for (int k = 0; k < n_steps; ++k) {
        const double a = coefs[3 * k], b = coefs[3 * k + 1], c = coefs[3 * k + 2];
        if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c)) return fail(ZERO_EINVAL, "coefs must be finite");
        const StepRange m = step_range(a, b, c, top);
        const double poly = std::max(m.poly, m.factor);
        if (!(poly <= kMostPoly && m.next <= 4.0 && m.next >= 0.0625))
            return fail(ZERO_ERANGE, "step %d takes singular values of [0, 1] to %g (1/16 to 4), its polynomial to %g (at most 32)",
                        k, m.next, poly);
        top = m.next;
        if (run > kMostCarried || run * m.factor > kMostRun) {
            steps->begins |= 1u << k;
            run = 1.0;
        }
        run *= m.factor;
        steps->a[k] = (float)a;
        steps->b[k] = (float)b;
        steps->c[k] = (float)c;
    }
    return ZERO_OK;
}

}  // namespace

int plan_ortho(const std::vector<OrthoMatrix>& matrices, OrthoPlan* plan) {
    std::vector<MatrixItem> mine;
    int tile = 64;
    for (const int other : {128, 256})
        if (step_cost(matrices, other) < step_cost(matrices, tile)) tile = other;
    int64_t total = 0, n_all = 0;
    for (const OrthoMatrix& m : matrices) {
        if (std::min(m.rows, m.cols) <= kThin) continue;
        n_all += pad_to(m.rows, tile) / tile * (pad_to(m.cols, tile) / tile);
        if (n_all > kMostTiles) return fail(ZERO_ERANGE, "the list is too long");
        MatrixItem it{};
        it.in = m.in;
        it.out = m.out;
        it.tall = m.rows > m.cols;
        it.s = (int32_t)std::min(m.rows, m.cols);
        it.l = (int32_t)std::max(m.rows, m.cols);
        it.sp = (int32_t)pad_to(it.s, tile);
        it.lp = (int32_t)pad_to(it.l, tile);
        it.udt = m.udt;
        it.odt = m.odt;
        it.log2_scale = log2_scale(it.l);
        const int64_t n_slots = pad_to(it.s, kPieceRows) / kPieceRows * (pad_to(it.l, kPieceColumns) / kPieceColumns);
        it.n_slots = (int32_t)n_slots;
        place_item(&it, &total);
        mine.push_back(it);
    }
    // as many passes as the workspace takes, of about equal size; in each the deepest products first
    const int64_t share = total / ((total + kPassBytes - 1) / kPassBytes + !total) + 1;
    for (size_t done = 0; done < mine.size();) {
        OrthoPass pass{};
        pass.tile = tile;
        int64_t at = 0;
        size_t end = done;
        while (end < mine.size() && (end == done || at < share)) {
            int64_t after = at;
            place_item(&mine[end], &after);
            if (end > done && after > kPassBytes) break;
            at = after;
            ++end;
        }
        plan->workspace = std::max(plan->workspace, at);
        const size_t first_item = plan->items.size();
        plan->items.insert(plan->items.end(), mine.begin() + done, mine.begin() + end);
        pass.first_item = (int64_t)first_item;
        pass.n_items = (int32_t)(end - done);
        done = end;
        pass.sym_first = (int64_t)plan->tiles.size();
        add_tiles(plan, first_item, tile, true, &pass.sym_blocks);
        pass.n_sym = (int64_t)plan->tiles.size() - pass.sym_first;
        pass.x_first = (int64_t)plan->tiles.size();
        add_tiles(plan, first_item, tile, false, &pass.x_blocks);
        pass.n_x = (int64_t)plan->tiles.size() - pass.x_first;
        pass.piece_first = (int64_t)plan->tiles.size();
        for (size_t k = first_item; k < plan->items.size(); ++k)
            for (int i = 0; i < plan->items[k].sp / kPieceRows; ++i)
                for (int j = 0; j < (int)(pad_to(plan->items[k].lp, kPieceColumns) / kPieceColumns); ++j)
                    plan->tiles.push_back({(uint32_t)k, (uint16_t)i, (uint16_t)j});
        pass.n_pieces = (int64_t)plan->tiles.size() - pass.piece_first;
        plan->passes.push_back(pass);
    }
    return plan_thin(matrices, plan);
}

}  // namespace zero_shard

using namespace zero_shard;

extern "C" {

size_t zero_multi_orthogonalize_workspace_bytes(const void* table) {
    clear_error();
    MatrixHeader h;
    if (table == nullptr) return 0;
    std::memcpy(&h, table, sizeof(h));
    return h.magic == kMatrixMagic ? (size_t)h.workspace_bytes : 0;
}

int zero_multi_orthogonalize(const void* table, const void* d_table, const double* coefs, int32_t n_steps, double eps,
                             const int32_t* d_global_overflow, void* d_workspace, size_t workspace_bytes,
                             void* hip_stream) {
    clear_error();
    MatrixHeader h;
    int rc = read_matrix_table(table, d_table, kCanOrtho, "the orthogonalisation (update, ortho)", &h);
    OrthoSteps steps;
    if (rc == ZERO_OK) rc = check_coefs(coefs, n_steps, &steps);
    if (rc != ZERO_OK) return rc;
    if (!(eps >= 0.0) || !std::isfinite(eps)) return fail(ZERO_EINVAL, "eps must be finite and >= 0");
    // below the least norm that is not zero eps decides nothing, and 1 / eps might not be finite
    if (eps < 0x1p-149) eps = 0.0;
    if ((uintptr_t)d_global_overflow & 3u) return fail(ZERO_EALIGN, "d_global_overflow misaligned");
    if (h.n_entries == 0) return ZERO_OK;
    if (d_workspace == nullptr) return fail(ZERO_EINVAL, "d_workspace is NULL");
    if ((uintptr_t)d_workspace & 255u) return fail(ZERO_EALIGN, "d_workspace must be 256-byte aligned");
    if (workspace_bytes < (size_t)h.workspace_bytes)
        return fail(ZERO_ENOSPC, "workspace %zu bytes, need %lld", workspace_bytes, (long long)h.workspace_bytes);
    if (matrix_touched(table, h, d_workspace, h.workspace_bytes) ||
        overlaps(d_workspace, h.workspace_bytes, d_table, h.device_bytes) ||
        (d_global_overflow && overlaps(d_workspace, h.workspace_bytes, d_global_overflow, sizeof(int32_t))))
        return fail(ZERO_EINVAL, "the workspace overlaps a buffer of the list, the table or the flag");
    if (matrix_written(table, h, d_global_overflow, sizeof(int32_t)))
        return fail(ZERO_EINVAL, "the flag lies in a buffer the call writes");
    const hipStream_t s = static_cast<hipStream_t>(hip_stream);
    const NsRef ref{at<MatrixItem>(d_table, h.items_at), at<TileRef>(d_table, h.tiles_at), static_cast<char*>(d_workspace),
                    d_global_overflow};
    const OrthoPass* passes = at<OrthoPass>(table, h.passes_at);
    for (int p = 0; p < h.n_passes; ++p) {
        const OrthoPass& pass = passes[p];
        if (pass.tile <= 0) {
            rc = launch_thin(pass, ref, steps, eps, s);
            if (rc != ZERO_OK) return rc;
            continue;
        }
        hipLaunchKernelGGL(ortho_squares, dim3((unsigned)pass.n_pieces), dim3(kBlock), 0, s, ref, pass.piece_first);
        rc = launch_status("ortho_squares");
        if (rc != ZERO_OK) return rc;
        hipLaunchKernelGGL(ortho_load, dim3((unsigned)pass.n_pieces), dim3(kBlock), 0, s, ref, pass.piece_first, eps);
        rc = launch_status("ortho_load");
        for (int k = 0; k < n_steps && rc == ZERO_OK; ++k) {
            const NsStep step{steps.a[k], steps.b[k], steps.c[k], k & 1, k == 0, k + 1 == n_steps};
            rc = launch_product<kGram>(pass, ref, step, s);
            if (rc == ZERO_OK) rc = launch_product<kPoly>(pass, ref, step, s);
            if (rc == ZERO_OK) rc = launch_product<kApply>(pass, ref, step, s);
        }
        if (rc != ZERO_OK) return rc;
    }
    return ZERO_OK;
}

}  // extern "C"
