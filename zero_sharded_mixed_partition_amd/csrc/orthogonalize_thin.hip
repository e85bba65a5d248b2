// Orthogonalisation of matrices with a short side s of at most 128: low-rank
// adapters, single heads, small layers.
//
// Every step multiplies X from the left by a polynomial of A = X X^T, and A of
// the next step follows from A alone: with B = b A + c A A and Q = a I + B (all of
// them symmetric, and functions of the first A, so they commute)
//     X' = Q X,   A' = X' X'^T = Q Q A.
// So U is read once for its A, which is s x s; one workgroup per matrix carries A
// and P, the product of the steps' Q, through the steps; and U is read again,
// multiplied by P, and stored.  Three launches whatever the number of steps and 6
// to 8 bytes an element; the tiled products take 17 launches and 50 bytes, and
// multiply X five times as often.
//
// A run of steps ends where P could exceed 2^10, or Q Q .. of all but its last
// step 2^16: what rounding leaves of A's zero singular values, 1e-7 of the
// largest, positive or negative, would grow into something.  The next run starts
// from X, in fp16.  Five steps of (3.4445, -4.7750, 2.0315) are one run.
//
// What is rounded.  A small singular value's square is far below A's largest
// entries, and the steps multiply it by up to 11.8 each: A, Q A, B and P are held
// as two fp16 each (22 bits, times 2^10, P 2^4), and so is X where it is
// multiplied; products are three MFMAs of the four (the lower halves' own is
// below 2^-22), sums float32.  U enters A with 11 bits or what it has of them,
// float32 as two fp16.  fp16's range: each chunk of U is scaled by a power of two
// of its own, which follows it to the sum.  A run's result is 1e-6 to 2e-4 off, and
// up to 7e-4 where singular values fall as 1 / k^2: the float32 sums of A know it to
// 2^-24 of its largest entries, and small singular values by their squares.
//
// What bounds it.  64 matrices of 128 x 4096, bf16, 67 MB in and out: 31 us for A
// (2.2 TB/s; each block waits for its chunk, multiplies, and waits again), 46 for
// the steps (64 of 256 CUs; products through the LDS one after the other, each
// between barriers), 52 for P X, 2.6 TB/s (26 GF of 2 s s l three times over, which
// at the rate of a large product are 16 us, beside 21 us for its bytes, on two
// blocks a CU).  64 of 16 x 4096 and 64 of 4096 x 16, 17 MB: 20, 11 and 24 us.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>
#include <vector>

#include "orthogonalize.h"
#include "part_exponent.h"

namespace zero_shard {
namespace {

// The steps of one run.
struct ThinSteps {
    float a[ZERO_MAX_ORTHO_STEPS], b[ZERO_MAX_ORTHO_STEPS], c[ZERO_MAX_ORTHO_STEPS];
    int32_t n;
};

constexpr int kLog2P = 4;                        // a run's polynomial is held times 2^4: at most 2^14

template <int SP>
struct Thin {
    static constexpr int kR = SP / 16;                        // rows of 16 x 16 tiles
    static constexpr int kTiles = kR * (kR + 1) / 2;          // of the lower triangle
    static constexpr int kLC = kChunkElements / SP;           // columns of a chunk
    static constexpr int kWaves2 = SP == 128 ? 12 : SP == 64 ? 5 : 3;   // of the second kernel: tiles divide evenly
    static constexpr int kOwn = kTiles / kWaves2;
    static constexpr int kP = 2 * SP * SP;                    // halves of a run's polynomial
    // in the second kernel's LDS a place of its own for it, or A's
    static constexpr bool kOwnP = SP <= 64;
    static constexpr int kSquares = kOwnP ? 3 : 2;
    static constexpr int kStageLd = kLC + 4;                  // floats a row: four rows apart meet other banks
};

__device__ __forceinline__ int pair_index(int i, int j) { return i * (i + 1) / 2 + j; }

// ---------------------------------------------------------------- a chunk of U

template <int SP>
using ChunkVector = Vector8<SP, SP>;

// Of U, or of what a run of steps has left in the workspace.
struct ThinSource {
    const void* at;
    int dt;

    __device__ __forceinline__ ThinSource(const NsRef& ref, const ZS_CONSTANT ThinItem& m, bool again)
        : at(again ? ref.ws + m.x : static_cast<const char*>(m.in)), dt(again ? (int)ZERO_F16 : m.udt) {}
};

template <int SP>
__device__ __forceinline__ void load_chunk(const ZS_CONSTANT ThinItem& m, const ThinSource& from, int64_t first, float x[8][8]) {
    load_box<SP, SP>(from.dt, from.at, m.s, m.l, m.tall, 0, first, x);
}

// ---------------------------------------------------------------- first kernel: parts of U U^T

// The chunk in the LDS as halves.  Wide: [SP][kLC], the 16-byte pieces of row r
// in the order piece ^ r % 16.  Tall: [kLC][SP] for the transposing load, the
// 32-byte pieces of row r in an order by r, so that rows 0 .. 3 and 8 .. 11 of
// 16, which a half wave reads, meet all banks.
template <int SP>
__device__ __forceinline__ int tall_order(int r) {
    if (SP == 128) return (r & 3) | ((r >> 1) & 4);
    if (SP == 64) return ((r >> 1) & 1) | ((r >> 2) & 2);
    return (r >> 3) & 1;
}

template <int SP>
__device__ __forceinline__ h8 chunk_fragment(uint32_t lds, bool tall, int i, int kk, int lane) {
    if (tall) {
        const int r = kk * 32 + (lane >> 4) * 8 + ((lane & 15) >> 2);
        const uint32_t a = lds + r * (SP * 2) + (i ^ tall_order<SP>(r)) * 32 + (lane & 3) * 8;
        const int r4 = r + 4;
        const uint32_t b = lds + r4 * (SP * 2) + (i ^ tall_order<SP>(r4)) * 32 + (lane & 3) * 8;
        return __builtin_shufflevector(lds_column(a), lds_column(b), 0, 1, 2, 3, 4, 5, 6, 7);
    }
    const int r = i * 16 + (lane & 15);
    return lds_h8(lds + r * (Thin<SP>::kLC * 2) + (((kk * 4 + (lane >> 4)) ^ (r & 15)) << 4));
}

// The products of a chunk.  SP 128: a wave owns tile rows `wave` and 7 - wave,
// nine tiles.  Else: all tiles, on every fourth step of the inner dimension.
template <int SP, bool TWO>
__device__ __forceinline__ void chunk_products(f32x4* acc, uint32_t hi, uint32_t lo, bool tall, int wave, int lane) {
    using H = Thin<SP>;
    constexpr int R = H::kR;
    const auto product = [&](f32x4& into, const h8& ih, const h8& il, const h8& jh, const h8& jl) {
        into = __builtin_amdgcn_mfma_f32_16x16x32_f16(ih, jh, into, 0, 0, 0);
        if constexpr (TWO) {
            into = __builtin_amdgcn_mfma_f32_16x16x32_f16(ih, jl, into, 0, 0, 0);
            into = __builtin_amdgcn_mfma_f32_16x16x32_f16(il, jh, into, 0, 0, 0);
        }
    };
    const auto low = [&](int i, int kk) {
        if constexpr (TWO) return chunk_fragment<SP>(lo, tall, i, kk, lane);
        else return h8{};
    };
    if constexpr (SP == 128) {
#pragma unroll 1
        for (int kk = 0; kk < H::kLC / 32; ++kk) {
            const h8 ah = chunk_fragment<SP>(hi, tall, wave, kk, lane), al = low(wave, kk);
            const h8 bh = chunk_fragment<SP>(hi, tall, 7 - wave, kk, lane), bl = low(7 - wave, kk);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (j > 7 - wave) continue;
                const h8 jh = chunk_fragment<SP>(hi, tall, j, kk, lane), jl = low(j, kk);
                product(acc[4 + j], bh, bl, jh, jl);
                if (j < 4 && j <= wave) product(acc[j], ah, al, jh, jl);
            }
        }
    } else {
#pragma unroll 1
        for (int kk = wave; kk < H::kLC / 32; kk += kThreads / 64) {
            h8 fh[R], fl[R];
#pragma unroll
            for (int i = 0; i < R; ++i) {
                fh[i] = chunk_fragment<SP>(hi, tall, i, kk, lane);
                fl[i] = low(i, kk);
            }
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int j = 0; j <= i; ++j) product(acc[i * (i + 1) / 2 + j], fh[i], fl[i], fh[j], fl[j]);
        }
    }
}

// One part of an item: chunks_per_part chunks, summed in order; the next chunk's
// loads are on their way during a chunk's products.
template <int SP>
__global__ __launch_bounds__(kThreads, 2) void thin_gram(NsRef ref, int64_t first, bool again) {
    using H = Thin<SP>;
    if (ref.skipped()) return;
    __shared__ __attribute__((aligned(1024))) char smem[2 * kChunkElements * 2];
    __shared__ uint32_t s_top[kThreads / 64];
    const ZS_CONSTANT TileRef& t = ref.tile(first + blockIdx.x);
    const ZS_CONSTANT ThinItem& m = ((const ZS_CONSTANT ThinItem*)ref.items)[t.item];
    const int part = t.i, lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t hi = lds_address(smem), lo = hi + kChunkElements * 2;
    const ThinSource from(ref, m, again);
    const bool two = from.dt == ZERO_F32, tall = m.tall != 0;
    constexpr int kOwn = SP == 128 ? 12 : H::kTiles;
    f32x4 acc[kOwn];
#pragma unroll
    for (int k = 0; k < kOwn; ++k) acc[k] = f32x4{};
    int run = kAllZero;                          // exponent that the sums are scaled by
    bool bad = false;
    const int64_t c_first = (int64_t)part * m.chunks_per_part;
    const int64_t c_end = c_first + m.chunks_per_part < m.n_chunks ? c_first + m.chunks_per_part : m.n_chunks;
    float x[8][8];
    load_chunk<SP>(m, from, c_first * H::kLC, x);
    for (int64_t chunk = c_first; chunk < c_end; ++chunk) {
        uint32_t top = 0;
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t b = __float_as_uint(x[n][k]) & 0x7FFFFFFFu;
                top = b > top ? b : top;
            }
        for (int off = 32; off > 0; off >>= 1) {
            const uint32_t other = (uint32_t)__shfl_xor((int)top, off, 64);
            top = other > top ? other : top;
        }
        if (lane == 0) s_top[wave] = top;
        __syncthreads();                         // also: the last chunk's fragments have been read
        for (int w = 0; w < kThreads / 64; ++w) top = s_top[w] > top ? s_top[w] : top;
        top = (uint32_t)__builtin_amdgcn_readfirstlane((int)top);
        if (top >= 0x7F800000u) bad = true;
        if (top != 0 && !bad) {
            // the largest element lands in [2^14, 2^15)
            const int e = (int)ilogbf(__uint_as_float(top)) - 14;
            if (e > run) {
                const int down = part_shift(run, e);
#pragma unroll
                for (int k = 0; k < kOwn; ++k)
#pragma unroll
                    for (int q = 0; q < 4; ++q) acc[k][q] = ldexpf(acc[k][q], down);
                run = e;
            }
        }
        const int shift = has_exponent(run) ? -run : 0;
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            h8 h, g;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float y = ldexpf(x[n][k], shift);
                h[k] = (_Float16)y;
                g[k] = (_Float16)(y - (float)h[k]);
            }
            const ChunkVector<SP> v(m.s, m.l, m.tall, 0, 0, n);
            const uint32_t at = tall ? v.c * (SP * 2) + (((v.r >> 4) ^ tall_order<SP>(v.c)) << 5) + (v.r & 8) * 2
                                     : v.r * (H::kLC * 2) + (((v.c >> 3) ^ (v.r & 15)) << 4);
            *reinterpret_cast<h8*>(smem + at) = h;
            if (two) *reinterpret_cast<h8*>(smem + kChunkElements * 2 + at) = g;
        }
        if (chunk + 1 < c_end) load_chunk<SP>(m, from, (chunk + 1) * H::kLC, x);      // on its way during the products
        __syncthreads();
        if (two) chunk_products<SP, true>(acc, hi, lo, tall, wave, lane);
        else chunk_products<SP, false>(acc, hi, lo, tall, wave, lane);
    }
    float* out = reinterpret_cast<float*>(ref.ws + m.parts) + (int64_t)part * H::kTiles * 256;
    if constexpr (SP == 128) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (j <= 7 - wave) reinterpret_cast<f32x4*>(out + pair_index(7 - wave, j) * 256)[lane] = acc[4 + j];
            if (j < 4 && j <= wave) reinterpret_cast<f32x4*>(out + pair_index(wave, j) * 256)[lane] = acc[j];
        }
    } else {
        // the four waves' sums, added in their order
        __syncthreads();
        f32x4* all = reinterpret_cast<f32x4*>(smem);
#pragma unroll
        for (int k = 0; k < H::kTiles; ++k) all[(wave * H::kTiles + k) * 64 + lane] = acc[k];
        __syncthreads();
        for (int k = threadIdx.x; k < H::kTiles * 64; k += kThreads) {
            f32x4 sum = all[k];
            for (int w = 1; w < kThreads / 64; ++w) sum += all[w * H::kTiles * 64 + k];
            reinterpret_cast<f32x4*>(out)[k] = sum;
        }
    }
    if (threadIdx.x == 0) reinterpret_cast<int32_t*>(ref.ws + m.exponents)[part] = bad ? kNotFinite : run;
}

// ---------------------------------------------------------------- second kernel: the steps' polynomials

// [SP][SP] halves, the 16-byte pieces of row r in an order by r: 16 lanes that
// read one piece of 16 rows meet all banks.
template <int SP>
__device__ __forceinline__ uint32_t square_piece(int r, int piece) {
    const int order = SP == 128 ? r & 15 : SP == 64 ? (r >> 1) & 7 : row_order(r);
    return r * (SP * 2) + ((piece ^ order) << 4);
}

// Of four lanes in a row, lane t gets element t of each: a tile's mirror image
// then leaves in 8-byte pieces (2 bytes at a time the steps of 64 x 128 x 4096
// take 49.9 us, so 46.4).
__device__ __forceinline__ h4 quad_transpose(h4 v, int lane) {
    typedef int i2 __attribute__((ext_vector_type(2)));
    const i2 w = __builtin_bit_cast(i2, v);
    const bool upper = lane & 2;
    const auto from = [&](auto quad) {               // all four lanes' copy of one lane's pair that holds element t
        constexpr int kQuad = decltype(quad)::value;
        const int a = __builtin_amdgcn_update_dpp(0, w[0], kQuad, 0xF, 0xF, true);
        const int b = __builtin_amdgcn_update_dpp(0, w[1], kQuad, 0xF, 0xF, true);
        return upper ? b : a;
    };
    const int u0 = from(std::integral_constant<int, 0x00>{}), u1 = from(std::integral_constant<int, 0x55>{});
    const int u2 = from(std::integral_constant<int, 0xAA>{}), u3 = from(std::integral_constant<int, 0xFF>{});
    const uint32_t halves = lane & 1 ? 0x07060302u : 0x05040100u;
    const i2 out = {(int)__builtin_amdgcn_perm((uint32_t)u1, (uint32_t)u0, halves), (int)__builtin_amdgcn_perm((uint32_t)u3, (uint32_t)u2, halves)};
    return __builtin_bit_cast(h4, out);
}

// A tile's values (rows 16 i + 4 g + e, column 16 j + c) into a symmetric
// matrix of two fp16: hi at `at`, lo behind it.  Of a tile on the diagonal only
// the values below it are taken: a matrix carried through the steps has to stay
// symmetric to the last bit, since what it lacks grows by up to 11.8 a step.
// (With both halves kept as they are summed, 16 x 16 matrices are 4e-4 off after
// five steps, 5e-2 after seven, and not finite after twelve.)
template <int SP>
__device__ __forceinline__ void put_square(char* at, int i, int j, int lane, const f32x4& v) {
    constexpr int kLo = SP * SP * 2;
    const int g = lane >> 4, c = lane & 15;
    h4 h, l;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        h[e] = (_Float16)v[e];
        l[e] = (_Float16)(v[e] - (float)h[e]);
    }
    char* row = at + square_piece<SP>(16 * j + c, 2 * i + (g >> 1)) + (g & 1) * 8;
    if (i != j) {
        *reinterpret_cast<h4*>(row) = h;
        *reinterpret_cast<h4*>(row + kLo) = l;
        char* mirror = at + square_piece<SP>(16 * i + 4 * g + (c & 3), 2 * j + (c >> 3)) + (c & 4) * 2;
        *reinterpret_cast<h4*>(mirror) = quad_transpose(h, lane);
        *reinterpret_cast<h4*>(mirror + kLo) = quad_transpose(l, lane);
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (4 * g + e < c) continue;
        char* to = at + square_piece<SP>(16 * i + 4 * g + e, 2 * j + (c >> 3)) + (c & 7) * 2;
        *reinterpret_cast<_Float16*>(to) = h[e];
        *reinterpret_cast<_Float16*>(to + kLo) = l[e];
        *reinterpret_cast<_Float16*>(row + 2 * e) = h[e];
        *reinterpret_cast<_Float16*>(row + kLo + 2 * e) = l[e];
    }
}

// A wave's tiles (ti, tj) of the product of two symmetric matrices that commute.
// They follow each other along the rows of the triangle, so that all but the
// first always share their row, whose pieces are read once; alike: the first too.
template <int SP, int N, bool ALIKE>
__device__ __forceinline__ void square_products(uint32_t a, uint32_t b, const int* ti, const int* tj, int lane, f32x4* sum) {
    constexpr int kLo = SP * SP * 2;
#pragma unroll
    for (int n = 0; n < N; ++n) sum[n] = f32x4{};
#pragma unroll
    for (int kk = 0; kk < SP / 32; ++kk) {
        const auto piece = [&](uint32_t from, int i) { return from + square_piece<SP>(16 * i + (lane & 15), kk * 4 + (lane >> 4)); };
        const uint32_t last = piece(a, ti[N - 1]);
        const h8 h = lds_h8(last), l = lds_h8(last + kLo);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            h8 ah = h, al = l;
            if (!ALIKE && n == 0) {
                const uint32_t own = piece(a, ti[0]);
                ah = lds_h8(own);
                al = lds_h8(own + kLo);
            }
            const uint32_t pb = piece(b, tj[n]);
            const h8 bh = lds_h8(pb), bl = lds_h8(pb + kLo);
            sum[n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ah, bh, sum[n], 0, 0, 0);
            sum[n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ah, bl, sum[n], 0, 0, 0);
            sum[n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(al, bh, sum[n], 0, 0, 0);
        }
    }
}

// A tile of a run's polynomial for the third kernel, as its fragments:
// [i][k / 32][lane][8] halves with the inner elements of a lane in the order
// 4 g .. + 3 of two tiles of 16.
template <int SP>
__device__ __forceinline__ void put_fragments(_Float16* to, int i, int j, int lane, const f32x4& v) {
    const int g = lane >> 4, c = lane & 15;
    h4 h, l;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        h[e] = (_Float16)v[e];
        l[e] = (_Float16)(v[e] - (float)h[e]);
    }
    _Float16* at = to + (((j * (SP / 32) + i / 2) * 64 + g * 16 + c) * 8 + (i & 1) * 4);
    _Float16* mirror = to + (((i * (SP / 32) + j / 2) * 64 + (c >> 2) * 16 + 4 * g) * 8 + (j & 1) * 4);
    if (i != j) {
        *reinterpret_cast<h4*>(at) = h;
        *reinterpret_cast<h4*>(at + SP * SP) = l;
        mirror += (c & 3) * 8;
        *reinterpret_cast<h4*>(mirror) = quad_transpose(h, lane);
        *reinterpret_cast<h4*>(mirror + SP * SP) = quad_transpose(l, lane);
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (4 * g + e < c) continue;
        mirror[8 * e + (c & 3)] = h[e];
        mirror[8 * e + (c & 3) + SP * SP] = l[e];
        at[e] = h[e];
        at[SP * SP + e] = l[e];
    }
}

template <int SP>
__global__ __launch_bounds__(64 * Thin<SP>::kWaves2) void thin_steps(NsRef ref, int64_t first_item, ThinSteps steps, double eps, bool again) {
    using H = Thin<SP>;
    constexpr int kOwn = H::kOwn;
    if (ref.skipped()) return;
    __shared__ __attribute__((aligned(1024))) char smem[H::kSquares * 2 * SP * SP * 2];     // A, B and P, two fp16 each
    __shared__ double s_diag[SP];
    const ZS_CONSTANT ThinItem& m = ((const ZS_CONSTANT ThinItem*)ref.items)[first_item + blockIdx.x];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int32_t* exponents = reinterpret_cast<const int32_t*>(ref.ws + m.exponents);
    int top = kAllZero;
    for (int p = 0; p < m.n_parts; ++p) top = exponents[p] > top ? exponents[p] : top;
    const bool bad = top == kNotFinite;
    int ti[kOwn], tj[kOwn];
    f32x4 A[kOwn];
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
        const int tile = wave * kOwn + k;
        int i = 0;
        while ((i + 1) * (i + 2) / 2 <= tile) ++i;
        ti[k] = i;
        tj[k] = tile - i * (i + 1) / 2;
        A[k] = f32x4{};
    }
#pragma unroll 8
    for (int p = 0; p < m.n_parts; ++p) {
        const f32x4* part = reinterpret_cast<const f32x4*>(ref.ws + m.parts) + (int64_t)p * H::kTiles * 64;
        const int down = bad ? 0 : part_shift(exponents[p], top);
#pragma unroll
        for (int k = 0; k < kOwn; ++k) {
            const f32x4 v = part[(wave * kOwn + k) * 64 + lane];
#pragma unroll
            for (int e = 0; e < 4; ++e) A[k][e] += ldexpf(v[e], down);
        }
    }
    // |U|^2 = the trace
#pragma unroll
    for (int k = 0; k < kOwn; ++k)
        if (ti[k] == tj[k] && (lane & 15) >> 2 == lane >> 4) {
            const int e = lane & 3;
            s_diag[16 * ti[k] + (lane & 15)] = (double)(e == 0 ? A[k][0] : e == 1 ? A[k][1] : e == 2 ? A[k][2] : A[k][3]);
        }
    __syncthreads();
    double trace = s_diag[lane % SP] + (SP == 128 ? s_diag[lane + 64] : 0.0);
    for (int off = (SP < 64 ? SP : 64) / 2; off > 0; off >>= 1) trace += __shfl_xor(trace, off, 64);
    const int up = !has_exponent(top) || bad ? 0 : top;
    const double norm = ldexp(sqrt(trace), up);
    // what a run has left is X times a power of two
    const double by = again ? ldexp(1.0, m.log2_scale) : norm > eps ? norm : eps;
    const double factor = bad ? NAN : by > 0.0 ? 1.0 / by : 0.0;
    if (threadIdx.x == 0) *reinterpret_cast<double*>(ref.ws + m.factor) = factor;
    const double unit = by > 0.0 ? ldexp(1.0, up) / by : 0.0;
    const float f = (float)ldexp(unit * unit, kLog2A);
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
#pragma unroll
        for (int e = 0; e < 4; ++e) A[k][e] *= f;
        put_square<SP>(smem, ti[k], tj[k], lane, A[k]);
    }
    __syncthreads();
    const uint32_t a = lds_address(smem), b = a + 2 * SP * SP * 2, p = H::kOwnP ? b + 2 * SP * SP * 2 : a;
    char* const b_at = smem + (b - a);
    char* const p_at = smem + (p - a);
    constexpr float kDown = 1.0f / (1 << kLog2A);
    const auto products = [&](uint32_t of, uint32_t by, f32x4* sum) {
        if (ti[0] == ti[kOwn - 1]) square_products<SP, kOwn, true>(of, by, ti, tj, lane, sum);
        else square_products<SP, kOwn, false>(of, by, ti, tj, lane, sum);
    };
    f32x4 P[kOwn];
    for (int step = 0; step < steps.n; ++step) {
        const bool last = step + 1 == steps.n;
        const float sa = steps.a[step];
        f32x4 w[kOwn];
        products(a, a, w);
#pragma unroll
        for (int k = 0; k < kOwn; ++k) {
            f32x4 B;
#pragma unroll
            for (int e = 0; e < 4; ++e) B[e] = fmaf(steps.b[step], A[k][e], steps.c[step] * (w[k][e] * kDown));
            if (step > 0 || !last) put_square<SP>(b_at, ti[k], tj[k], lane, B);
            if (step == 0) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    P[k][e] = (float)(1 << kLog2P) * (B[e] * kDown + (ti[k] == tj[k] && 4 * (lane >> 4) + e == (lane & 15) ? sa : 0.0f));
            } else if (H::kOwnP) {
                put_square<SP>(p_at, ti[k], tj[k], lane, P[k]);
            }
        }
        const auto times_b = [&](f32x4* v, uint32_t by) {         // v <- a v + B v, of which `by` is the LDS's copy
            products(b, by, w);
#pragma unroll
            for (int k = 0; k < kOwn; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) v[k][e] = fmaf(sa, v[k][e], w[k][e] * kDown);
        };
        const auto put = [&](char* to, const f32x4* v) {
#pragma unroll
            for (int k = 0; k < kOwn; ++k) put_square<SP>(to, ti[k], tj[k], lane, v[k]);
        };
        __syncthreads();
        if (!last) times_b(A, a);
        if (step > 0) {
            if (!H::kOwnP) {
                __syncthreads();
                put(p_at, P);
                __syncthreads();
            }
            times_b(P, p);
        }
        if (last) break;
        __syncthreads();
        put(smem, A);
        __syncthreads();
        times_b(A, a);
        __syncthreads();
        put(smem, A);
        __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < kOwn; ++k) put_fragments<SP>(reinterpret_cast<_Float16*>(ref.ws + m.p), ti[k], tj[k], lane, P[k]);
}

// ---------------------------------------------------------------- third kernel: P X

template <int SP, int ODT>
__device__ __forceinline__ void store_chunk(const ZS_CONSTANT ThinItem& m, void* to, int64_t first, const float* stage, float back) {
    using H = Thin<SP>;
    uint16_t* out = static_cast<uint16_t*>(to);
#pragma unroll
    for (int n = 0; n < 8; ++n) {
        const ChunkVector<SP> v(m.s, m.l, m.tall, 0, first, n);
        if (v.valid == 0) continue;
        const float* from = stage + v.r * H::kStageLd + v.c;
        const int step = m.tall ? H::kStageLd : 1;
        if (v.valid == 8) {
            float a[4], b[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                a[k] = from[k * step] * back;
                b[k] = from[(k + 4) * step] * back;
            }
            st_any(pack4_16<ODT>(a), out + v.at);
            st_any(pack4_16<ODT>(b), out + v.at + 4);
        } else {
            for (int k = 0; k < v.valid; ++k) global(out)[v.at + k] = (uint16_t)to16<ODT>(from[k * step] * back);
        }
    }
}

// One chunk of columns.  A lane holds X as the MFMA leaves it, rows 16 i + 4 g
// .. + 3 of a column, which is how the next product takes it: with the inner
// elements in the order of put_fragments nothing moves between lanes.
template <int SP>
__global__ __launch_bounds__(kThreads, 2) void thin_apply(NsRef ref, int64_t first, bool again, bool last) {
    using H = Thin<SP>;
    constexpr int R = H::kR, kStrips = H::kLC / 64, kP = H::kP, kLoads = kP / 8 / kThreads;
    if (ref.skipped()) return;
    __shared__ __attribute__((aligned(1024))) char smem[SP * H::kStageLd * 4];
    static_assert(kP * 2 <= SP * H::kStageLd * 4 && kLoads * 8 * kThreads == kP, "a polynomial takes the stage's place");
    const ZS_CONSTANT TileRef& t = ref.tile(first + blockIdx.x);
    const ZS_CONSTANT ThinItem& m = ((const ZS_CONSTANT ThinItem*)ref.items)[t.item];
    const int64_t column = (int64_t)t.i * H::kLC;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    float* stage = reinterpret_cast<float*>(smem);
    {
        float x[8][8];
        load_chunk<SP>(m, ThinSource(ref, m, again), column, x);
        // x * factor as x * 2^e * f, f in [0.5, 1): neither the factor nor a product leaves float32
        int e;
        const float f = (float)frexp(*reinterpret_cast<const double*>(ref.ws + m.factor), &e);
        e += m.log2_scale;
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            const ChunkVector<SP> v(m.s, m.l, m.tall, 0, column, n);
            float* to = stage + v.r * H::kStageLd + v.c;
            if (m.tall) {
#pragma unroll
                for (int k = 0; k < 8; ++k) to[k * H::kStageLd] = scaled(x[n][k], f, e);
            } else {
#pragma unroll
                for (int k = 0; k < 8; k += 4)
                    *reinterpret_cast<f32x4*>(to + k) = f32x4{scaled(x[n][k], f, e), scaled(x[n][k + 1], f, e),
                                                              scaled(x[n][k + 2], f, e), scaled(x[n][k + 3], f, e)};
            }
        }
    }
    const u32x4* q = reinterpret_cast<const u32x4*>(ref.ws + m.p);
    u32x4 ahead[kLoads];
#pragma unroll
    for (int k = 0; k < kLoads; ++k) ahead[k] = q[k * kThreads + threadIdx.x];
    __syncthreads();
    const int own = wave * (H::kLC / 4) + (lane & 15), row = (lane >> 4) * 4;
    f32x4 X[kStrips][R];
#pragma unroll
    for (int y = 0; y < kStrips; ++y)
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) X[y][i][e] = stage[(i * 16 + row + e) * H::kStageLd + own + y * 16];
    const uint32_t p = lds_address(smem) + lane * 16;
    __syncthreads();                                          // the stage has been read
#pragma unroll
    for (int k = 0; k < kLoads; ++k) reinterpret_cast<u32x4*>(smem)[k * kThreads + threadIdx.x] = ahead[k];
    __syncthreads();
    h8 xh[kStrips][R / 2], xl[kStrips][R / 2];
#pragma unroll
    for (int y = 0; y < kStrips; ++y)
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const _Float16 h = (_Float16)X[y][i][e];
                xh[y][i / 2][(i & 1) * 4 + e] = h;
                xl[y][i / 2][(i & 1) * 4 + e] = (_Float16)(X[y][i][e] - (float)h);
            }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        f32x4 sum[kStrips];
#pragma unroll
        for (int y = 0; y < kStrips; ++y) sum[y] = f32x4{};
#pragma unroll
        for (int k = 0; k < R / 2; ++k) {
            const h8 ph = lds_h8(p + (i * (SP / 32) + k) * 1024), pl = lds_h8(p + SP * SP * 2 + (i * (SP / 32) + k) * 1024);
#pragma unroll
            for (int y = 0; y < kStrips; ++y) {
                sum[y] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ph, xh[y][k], sum[y], 0, 0, 0);
                sum[y] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ph, xl[y][k], sum[y], 0, 0, 0);
                sum[y] = __builtin_amdgcn_mfma_f32_16x16x32_f16(pl, xh[y][k], sum[y], 0, 0, 0);
            }
        }
#pragma unroll
        for (int y = 0; y < kStrips; ++y)
#pragma unroll
            for (int e = 0; e < 4; ++e) X[y][i][e] = sum[y][e] * (1.0f / (1 << kLog2P));
    }
    __syncthreads();
#pragma unroll
    for (int y = 0; y < kStrips; ++y)
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) stage[(i * 16 + row + e) * H::kStageLd + own + y * 16] = X[y][i][e];
    __syncthreads();
    const float back = last ? ldexpf(1.0f, -m.log2_scale) : 1.0f;
    if (!last) store_chunk<SP, ZERO_F16>(m, ref.ws + m.x, column, stage, back);
    else if (m.odt == ZERO_F16) store_chunk<SP, ZERO_F16>(m, m.out, column, stage, back);
    else store_chunk<SP, ZERO_BF16>(m, m.out, column, stage, back);
}

// ---------------------------------------------------------------- host side

int padded(int64_t s) { return s <= 32 ? 32 : s <= 64 ? 64 : 128; }

// One run of steps; again: not the first, last: the last.
template <int SP>
int launch_run(const OrthoPass& p, const NsRef& ref, const ThinSteps& steps, double eps, bool again, bool last, hipStream_t s) {
    hipLaunchKernelGGL(thin_gram<SP>, dim3((unsigned)p.n_sym), dim3(kThreads), 0, s, ref, p.sym_first, again);
    int rc = launch_status("thin_gram");
    if (rc != ZERO_OK) return rc;
    hipLaunchKernelGGL(thin_steps<SP>, dim3((unsigned)p.n_items), dim3(64 * Thin<SP>::kWaves2), 0, s, ref, p.first_item, steps, eps, again);
    rc = launch_status("thin_steps");
    if (rc != ZERO_OK) return rc;
    hipLaunchKernelGGL(thin_apply<SP>, dim3((unsigned)p.n_x), dim3(kThreads), 0, s, ref, p.x_first, again, last);
    return launch_status("thin_apply");
}

}  // namespace

int launch_thin(const OrthoPass& pass, const NsRef& ref, const OrthoSteps& steps, double eps, hipStream_t stream) {
    int rc = ZERO_OK;
    for (int k = 0; k < steps.n && rc == ZERO_OK;) {
        ThinSteps run{};
        const int begin = k;
        do {
            run.a[run.n] = steps.a[k];
            run.b[run.n] = steps.b[k];
            run.c[run.n] = steps.c[k];
            ++run.n;
            ++k;
        } while (k < steps.n && !(steps.begins >> k & 1));
        const bool again = begin > 0, last = k == steps.n;
        rc = pass.tile == -128  ? launch_run<128>(pass, ref, run, eps, again, last, stream)
             : pass.tile == -64 ? launch_run<64>(pass, ref, run, eps, again, last, stream)
                                : launch_run<32>(pass, ref, run, eps, again, last, stream);
    }
    return rc;
}

int plan_thin(const std::vector<OrthoMatrix>& matrices, OrthoPlan* plan) {
    for (const int sp : {128, 64, 32}) {
        const int tiles = sp / 16 * (sp / 16 + 1) / 2;
        const int64_t p_bytes = 2 * 2 * sp * sp;
        OrthoPass pass{};
        int64_t at = 0;
        size_t first = plan->items.size();
        const auto finish = [&]() {
            if (plan->items.size() == first) return;
            std::vector<ThinItem> items(plan->items.size() - first);
            std::memcpy(items.data(), plan->items.data() + first, items.size() * sizeof(ThinItem));
            pass.tile = -sp;
            pass.first_item = (int64_t)first;
            pass.n_items = (int32_t)(plan->items.size() - first);
            pass.sym_first = (int64_t)plan->tiles.size();
            for (size_t k = first; k < plan->items.size(); ++k)
                for (int p = 0; p < items[k - first].n_parts; ++p) plan->tiles.push_back({(uint32_t)k, (uint16_t)p, 0});
            pass.n_sym = (int64_t)plan->tiles.size() - pass.sym_first;
            pass.x_first = (int64_t)plan->tiles.size();
            for (size_t k = first; k < plan->items.size(); ++k)
                for (int c = 0; c < items[k - first].n_chunks; ++c) plan->tiles.push_back({(uint32_t)k, (uint16_t)c, 0});
            pass.n_x = (int64_t)plan->tiles.size() - pass.x_first;
            plan->passes.push_back(pass);
            plan->workspace = std::max(plan->workspace, at);
            first = plan->items.size();
            at = 0;
        };
        for (const OrthoMatrix& m : matrices) {
            const int64_t s = std::min(m.rows, m.cols), l = std::max(m.rows, m.cols);
            if (s > kThin || padded(s) != sp) continue;
            ThinItem it{};
            it.in = m.in;
            it.out = m.out;
            it.tall = m.rows > m.cols;
            it.s = (int32_t)s;
            it.l = (int32_t)l;
            it.sp = sp;
            it.udt = m.udt;
            it.odt = m.odt;
            it.log2_scale = log2_scale(l);
            it.n_chunks = (int32_t)((l + kChunkElements / sp - 1) / (kChunkElements / sp));
            // at least sp / 32 chunks a part, and no more than 2 MB of parts: one
            // workgroup sums them
            const int64_t most = (int64_t(2) << 20) / (tiles * 1024);
            it.chunks_per_part = (int32_t)std::max<int64_t>(sp / 32, (it.n_chunks + most - 1) / most);
            it.n_parts = (int32_t)((it.n_chunks + it.chunks_per_part - 1) / it.chunks_per_part);
            const int64_t x_bytes = s * l * 2;
            const int64_t need = pad_to((int64_t)it.n_parts * tiles * 1024, 256) + pad_to((int64_t)it.n_parts * 4, 256) +
                                 p_bytes + 256 + pad_to(x_bytes, 256);
            if ((at > 0 && at + need > kPassBytes) || plan->items.size() - first >= 1 << 20) finish();
            it.parts = place(&at, (int64_t)it.n_parts * tiles * 1024);
            it.exponents = place(&at, (int64_t)it.n_parts * 4);
            it.p = place(&at, p_bytes);
            it.factor = place(&at, sizeof(double));
            it.x = place(&at, x_bytes);
            MatrixItem slot;
            std::memcpy(&slot, &it, sizeof(it));
            plan->items.push_back(slot);
        }
        finish();
    }
    return ZERO_OK;
}

}  // namespace zero_shard
