// What the two paths of the orthogonalisation share: products in tiles
// (orthogonalize.hip) and matrices with a short side of at most 128
// (orthogonalize_thin.hip).
#pragma once
#include "matrix_table.h"

namespace zero_shard {

// n_steps steps on the matrices of a pass with a short side of at most kThin
// (orthogonalize_thin.hip).
struct NsRef;
struct ThinSteps {
    float a[ZERO_MAX_ORTHO_STEPS], b[ZERO_MAX_ORTHO_STEPS], c[ZERO_MAX_ORTHO_STEPS];
    int32_t n;
};
int launch_thin(const OrthoPass& pass, const NsRef& ref, const ThinSteps& steps, double eps, hipStream_t stream);
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

// Four values down a column of 4 x 16 blocks (a lane of 16 gives the address of a fourth of a row).
__device__ __forceinline__ h4 lds_column(uint32_t a) {
    return __builtin_bit_cast(h4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4*)(uintptr_t)a));
}

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
