// The table of a list of matrices (zero_matrix_table_build), shared by the
// momentum pass and the update (matrix_step.hip) and the orthogonalisation
// (orthogonalize.hip).
//
// Its device image holds a descriptor per entry that has elements, the maps
// from units of elementwise work to entries, and for the orthogonalisation the
// single matrices (an entry may be a batch of them) with their places in the
// workspace, and the tiles of their products.  The host part holds the passes
// in which the orthogonalisation works the list off, and the address ranges.
#pragma once
#include <cstring>
#include <vector>

#include "list_table.h"
#include "moments8.h"

namespace zero_shard {

constexpr uint32_t kMatrixMagic = 0x5A534D58u;

struct MatrixDesc {
    float* master;
    float* momentum;
    const void* grad;
    void* update;
    void* ortho;
    void* param_out;
    double scale;
    int64_t numel;                      // > 0, over the whole batch
    int32_t gdt, udt, odt, pdt;         // pdt 0: no copy
    int32_t group;
    int32_t momentum_shift, master_shift;   // tasks start this many elements before multiples of kTask
    int32_t reserved;
};

// One matrix of the orthogonalisation, as its tiled products see it: s rows of l >= s elements (transposed if
// the caller's has more rows than columns), padded to sp x lp in the workspace.
struct MatrixItem {
    const void* in;
    void* out;
    int64_t x0, x1;                     // workspace: the iterate and the next one, half [sp][lp]
    int64_t a, b;                       // workspace: X X^T and the polynomial, half [sp][sp]
    int64_t slots;                      // workspace: partial sums of squares, double [n_slots], and start_factor
    int32_t n_slots;
    int32_t s, l, sp, lp;
    int32_t udt, odt;
    int32_t tall;                       // the caller's matrix has l rows
    int32_t log2_scale;                 // the iterate is held times this power of two
    int32_t reserved;
};

// The same memory for a thin matrix (s <= 128), padded to sp rows.
struct ThinItem {
    const void* in;
    void* out;
    int64_t parts;                      // workspace: partial X X^T, float [n_parts][tiles of the lower triangle][256]
    int64_t exponents;                  // workspace: each part's exponent, int32 [n_parts]
    int64_t p;                          // workspace: the polynomial of a run of steps, half, two of [sp][sp]
    int64_t factor;                     // workspace: 1 / max(|U|, eps), double
    int64_t x;                          // workspace: what a run that is not the last leaves, half, laid out as U
    int32_t n_parts;
    int32_t s, l, sp, n_chunks;
    int32_t udt, odt;
    int32_t tall;
    int32_t log2_scale;
    int32_t chunks_per_part;
};
static_assert(sizeof(ThinItem) == sizeof(MatrixItem), "one array holds both");

constexpr uint32_t kNoItem = UINT32_MAX;

struct TileRef {
    uint32_t item;                      // kNoItem: a block's round without a tile
    uint16_t i, j;                      // tile row (along s) and tile column
};

// A run of items of one tile size that the workspace holds at once.
// Thin ones (tile = minus the padded short side) have parts of X X^T in place of
// the first list, and chunks of columns in place of the second.
struct OrthoPass {
    int32_t tile;
    int32_t n_items;
    int64_t first_item;
    int64_t sym_first, n_sym;           // tiles of the symmetric products, lower triangle: rounds of sym_blocks
    int64_t x_first, n_x;               // tiles of the iterate: rounds of x_blocks
    int32_t sym_blocks, x_blocks;
    int64_t piece_first, n_pieces;      // pieces in which U is read (not of thin ones)
};

enum { kCanMomentum = 1, kCanOrtho = 2, kCanUpdate = 4 };

struct MatrixHeader {
    uint32_t magic;
    int32_t can, n_groups;
    int32_t n_user, n_entries;
    int32_t momentum_log2, master_log2;       // tasks per unit
    int32_t n_passes;
    int64_t n_momentum, n_master;             // units
    int64_t desc_at, momentum_at, master_at, items_at, tiles_at, device_bytes;
    int64_t workspace_bytes;
    int64_t passes_at, ranges_at, n_ranges, reads_at, n_reads, bytes;
};

// What the orthogonalisation of a list works on (orthogonalize.hip).
struct OrthoMatrix {
    const void* in;
    void* out;
    int64_t rows, cols;                 // > 0
    int32_t udt, odt;
};

// The matrices' tile sizes and places in the workspace, and the passes.
struct OrthoPlan {
    std::vector<MatrixItem> items;
    std::vector<TileRef> tiles;
    std::vector<OrthoPass> passes;
    int64_t workspace = 0;
};

int plan_ortho(const std::vector<OrthoMatrix>& matrices, OrthoPlan* plan);

namespace {

inline int read_matrix_table(const void* table, const void* d_table, int32_t need, const char* what, MatrixHeader* h) {
    if (table == nullptr) return fail(ZERO_EINVAL, "table is NULL");
    if ((uintptr_t)table & 7u) return fail(ZERO_EALIGN, "table must be 8-byte aligned");
    std::memcpy(h, table, sizeof(*h));
    if (h->magic != kMatrixMagic) return fail(ZERO_EINVAL, "not a table of zero_matrix_table_build");
    if (h->n_entries > 0) {
        if (d_table == nullptr) return fail(ZERO_EINVAL, "d_table is NULL");
        if (!aligned16(d_table)) return fail(ZERO_EALIGN, "d_table must be 16-byte aligned");
        if ((h->can & need) != need) return fail(ZERO_EINVAL, "the table's matrices lack the buffers of %s", what);
        if (meets(at<AddressRange>(table, h->ranges_at), h->n_ranges, d_table, h->device_bytes))
            return fail(ZERO_EINVAL, "the table lies in a buffer that its calls write");
    }
    return ZERO_OK;
}

// Whether [p, p + bytes) meets a buffer of the list that a call may write.
inline bool matrix_written(const void* table, const MatrixHeader& h, const void* p, int64_t bytes) {
    return meets(at<AddressRange>(table, h.ranges_at), h.n_ranges, p, bytes);
}

// ... any buffer of the list
inline bool matrix_touched(const void* table, const MatrixHeader& h, const void* p, int64_t bytes) {
    return matrix_written(table, h, p, bytes) || meets(at<AddressRange>(table, h.reads_at), h.n_reads, p, bytes);
}

}  // namespace
}  // namespace zero_shard
