// What the two paths of the orthogonalisation share: products in tiles
// (orthogonalize.hip) and matrices with a short side of at most 128
// (orthogonalize_thin.hip).
#pragma once
#include "matrix_table.h"

namespace zero_shard {

// n_steps steps on the matrices of a pass with a short side of at most kThin
// (orthogonalize_thin.hip).
struct NsRef;
struct OrthoSteps {
    float a[ZERO_MAX_ORTHO_STEPS], b[ZERO_MAX_ORTHO_STEPS], c[ZERO_MAX_ORTHO_STEPS];
    int32_t n;
    uint32_t begins;                             // bit k: a run of thin matrices' steps begins with step k (the first has none)
};
constexpr double kMostPoly = 32.0;               // of a step's polynomials, on the singular values that reach it
constexpr double kMostRun = 1024.0;              // of the product of a run's
constexpr double kMostCarried = 256.0;           // ... without its last
int launch_thin(const OrthoPass& pass, const NsRef& ref, const OrthoSteps& steps, double eps, hipStream_t stream);
// The passes, work lists and workspace of those matrices, appended to plan.
int plan_thin(const std::vector<OrthoMatrix>& matrices, OrthoPlan* plan);

constexpr int kThin = 128;
constexpr int64_t kPassBytes = int64_t(4) << 30; // workspace of a pass, if it holds more than one matrix

struct NsRef {
    const MatrixItem* items;
    const TileRef* tiles;
    char* ws;
    const int32_t* d_ovf;

    __device__ __forceinline__ const ZS_CONSTANT TileRef& tile(int64_t i) const {
        return ((const ZS_CONSTANT TileRef*)tiles)[i];
    }
    __device__ __forceinline__ const ZS_CONSTANT MatrixItem& item(uint32_t i) const {
        return ((const ZS_CONSTANT MatrixItem*)items)[i];
    }
    __device__ __forceinline__ bool skipped() const { return d_ovf != nullptr && *d_ovf != 0; }
};

namespace {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef short s4 __attribute__((ext_vector_type(4)));

constexpr int kLog2A = 10;                       // X X^T and the polynomial are held times 2^10

typedef __attribute__((address_space(3))) char lds_char;

__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return (uint32_t)(uintptr_t)(lds_char*)(char*)p;
}

__device__ __forceinline__ h8 lds_h8(uint32_t a) { return *(__attribute__((address_space(3))) h8*)(uintptr_t)a; }

// The order of the four 16-byte pieces of 64-byte rows for reads of 16 bytes of
// which lane l takes row l % 16, piece l / 16.  The hardware serves lanes 0-3,
// 12-15 and 20-27 at once, then 4-11, 16-19 and 28-31, and the upper half alike:
// rows 4 q .. 4 q + 3 of one piece with others of the next.  0, 2, 3, 1 by q
// keeps them apart in both.
__device__ __forceinline__ int row_order(int r) { return (((r >> 2) ^ (r >> 3)) & 1) * 2 + ((r >> 3) & 1); }

// Four values down a column of 4 x 16 blocks (a lane of 16 gives the address of a fourth of a row).
__device__ __forceinline__ h4 lds_column(uint32_t a) {
    return __builtin_bit_cast(h4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4*)(uintptr_t)a));
}

// The value as float32 has it.  Opaque to the compiler, which otherwise may or may
// not round the operation before it straight to 16 bits, and so make results depend
// on the tile size.
__device__ __forceinline__ float as_float(float x) {
    __asm__("" : "+v"(x));
    return x;
}

__device__ __forceinline__ _Float16 to_half(float x) { return (_Float16)as_float(x); }

// ---------------------------------------------------------------- boxes of U

constexpr int kThreads = 256;
constexpr int kChunkElements = 16384;            // of a box: 64 a thread, as eight vectors of eight

// Eight consecutive elements, the first `valid` of them; whole: eight may be read;
// full: all are valid.
template <int DT>
__device__ __forceinline__ void ld8(const void* U, int64_t e, int valid, bool whole, bool full, float v[8]) {
    if (whole) {
        if constexpr (DT == ZERO_F32) {
            const f32x4 a = ld_any(static_cast<const float*>(U) + e), b = ld_any(static_cast<const float*>(U) + e + 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[k] = a[k];
                v[k + 4] = b[k];
            }
        } else {
            const u32x4 w = ld16_any(static_cast<const uint16_t*>(U) + e);
#pragma unroll
            for (int k = 0; k < 4; ++k) unpack2<DT>(w[k], v[2 * k], v[2 * k + 1]);
        }
        if (full) return;
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = k < valid ? v[k] : 0.0f;
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = k < valid ? ld_grad1<DT>(U, e + k) : 0.0f;
    }
}

// A thread's n-th vector of a box of ROWS x 16384 / ROWS elements at (r0, c0) of
// the s x l matrix, which the caller holds transposed if it is tall: along the
// columns of a wide matrix, along the rows of a tall one.  BAND rows of a wide
// one come before the next columns.
template <int ROWS, int BAND>
struct Vector8 {
    int r, c;                                    // in the box
    int64_t at;                                  // of the first element, in the caller's matrix
    int valid;

    __device__ __forceinline__ Vector8(int s, int l, int tall, int r0, int64_t c0, int n) {
        constexpr int kAcross = kChunkElements / ROWS / 8;                     // vectors along a row
        constexpr int kBandAcross = kAcross * BAND / ROWS;                     // ... of a band of 256 / BAND vectors
        const int v = n * kThreads + threadIdx.x;
        if (tall) {
            r = v % (ROWS / 8) * 8;
            c = v / (ROWS / 8);
            at = (c0 + c) * s + r0 + r;
            valid = c0 + c < l ? s - r0 - r : 0;
        } else {
            if constexpr (BAND == ROWS) {
                r = v / kAcross;
                c = v % kAcross * 8;
            } else {
                r = v / kBandAcross % ROWS;
                c = (v / (kBandAcross * ROWS) * kBandAcross + v % kBandAcross) * 8;
            }
            at = (int64_t)(r0 + r) * l + c0 + c;
            const int64_t left = l - c0 - c;
            valid = r0 + r < s ? (int)(left < 8 ? left : 8) : 0;
        }
        valid = valid < 0 ? 0 : valid > 8 ? 8 : valid;
    }
};

template <int ROWS, int BAND, int DT>
__device__ __forceinline__ void load_box(const void* U, int s, int l, int tall, int r0, int64_t c0, float x[8][8]) {
    constexpr int kColumns = kChunkElements / ROWS;
    const int64_t all = (int64_t)s * l;
    // a vector may run over its row's end into the next row, but not over the matrix's
    const int64_t r_last = (r0 + ROWS < s ? r0 + ROWS : s) - 1, c_last = (c0 + kColumns < l ? c0 + kColumns : l) - 1;
    const int64_t last = tall ? c_last * s + r_last : r_last * (int64_t)l + c_last;
    if (r0 + ROWS <= s && c0 + kColumns <= l) {
#pragma unroll
        for (int n = 0; n < 8; ++n) ld8<DT>(U, Vector8<ROWS, BAND>(s, l, tall, r0, c0, n).at, 8, true, true, x[n]);
    } else if (last + 8 <= all) {
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            const Vector8<ROWS, BAND> v(s, l, tall, r0, c0, n);
            ld8<DT>(U, v.valid ? v.at : 0, v.valid, true, false, x[n]);
        }
    } else {
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            const Vector8<ROWS, BAND> v(s, l, tall, r0, c0, n);
            ld8<DT>(U, v.valid ? v.at : 0, v.valid, v.valid > 0 && v.at + 8 <= all, false, x[n]);
        }
    }
}

template <int ROWS, int BAND>
__device__ __forceinline__ void load_box(int dt, const void* U, int s, int l, int tall, int r0, int64_t c0, float x[8][8]) {
    if (dt == ZERO_F16) load_box<ROWS, BAND, ZERO_F16>(U, s, l, tall, r0, c0, x);
    else if (dt == ZERO_BF16) load_box<ROWS, BAND, ZERO_BF16>(U, s, l, tall, r0, c0, x);
    else load_box<ROWS, BAND, ZERO_F32>(U, s, l, tall, r0, c0, x);
}

// x * f * 2^e: with f in [0.5, 1) no product leaves float32 that the result does not.
__device__ __forceinline__ float scaled(float x, float f, int e) { return ldexpf(x, e) * f; }

// ---------------------------------------------------------------- host side

inline int64_t pad_to(int64_t x, int64_t t) { return (x + t - 1) / t * t; }

inline int64_t place(int64_t* at, int64_t bytes) {
    const int64_t here = *at;
    *at += pad_to(bytes, 256);
    return here;
}

// The iterate is held times 2^this: typical entries of an orthogonal matrix, about 1 / sqrt(l), become 1.
inline int32_t log2_scale(int64_t l) {
    int32_t k = 0;
    while (k < 12 && (int64_t(4) << (2 * k)) <= l) ++k;
    return k;
}

}  // namespace
}  // namespace zero_shard
