// What the tables of lists share (multi_step.hip, matrix_step.hip): the maps
// from units of work to a list's members, and the host's sorted address ranges.
#pragma once
#include <algorithm>
#include <cstdint>
#include <vector>

namespace zero_shard {
namespace {

// A unit of the update is 2^k consecutive tasks of one tensor, k <= kMaxUnit;
// a tensor's last unit leaves workgroups idle.  The table takes the largest k
// whose workgroups exceed the tasks by no more than a tenth: 3,000 tensors of
// 500 elements take 2 tasks a unit and 9.7 us, with 32 a unit 108 us (8 bits:
// 10.6 and 82); 39 tensors of 1.07B elements keep 32 a unit and a map of 1 MB.
constexpr int kMaxUnit = 5;
// A list's fp32 tensors may start anywhere.  The update's tasks are laid out so
// that the master's runs start at multiples of 256 bytes: otherwise two waves,
// on different XCDs, share the cache line between their runs and each writes
// part of it.  Tensors cut end to end from flat buffers have the same phase in
// every stream.  57 tensors of 11.2M elements in all, end to end, none aligned:
// 50.4 us with it, 62.4 without (6.22 and 5.03 TB/s).  8-bit moments keep their
// blocks, which start with the tensor.
constexpr int64_t kPhase = 64;                            // elements

struct PieceRef {
    uint32_t tensor, piece;   // index of the descriptor, and which chunk or unit of that tensor
};

struct AddressRange {
    uintptr_t lo, hi;
};

template <typename T>
const T* at(const void* table, int64_t offset) {
    return reinterpret_cast<const T*>(static_cast<const char*>(table) + offset);
}

inline int64_t pad16(int64_t x) { return (x + 15) & ~(int64_t)15; }

// Whether [p, p + bytes) meets one of n sorted, disjoint address ranges.
inline bool meets(const AddressRange* r, int64_t n, const void* p, int64_t bytes) {
    if (p == nullptr || bytes == 0) return false;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p), hi = lo + (uintptr_t)bytes;
    const AddressRange* f = std::upper_bound(r, r + n, lo, [](uintptr_t x, const AddressRange& a) { return x < a.hi; });
    return f != r + n && f->lo < hi;
}

struct Region {
    uintptr_t lo, hi;
    bool write;
    int32_t tensor;
};

// Sorts the ranges of a list's buffers and merges those that are written and
// those that are only read.  No written range may meet another one; buffers
// that are only read may be shared.  The member at fault, or -1.
inline int32_t merge_regions(std::vector<Region>& regions, std::vector<AddressRange>* ranges,
                             std::vector<AddressRange>* reads) {
    std::sort(regions.begin(), regions.end(), [](const Region& a, const Region& b) { return a.lo < b.lo; });
    uintptr_t any_hi = 0, write_hi = 0;
    for (const Region& r : regions) {
        if (r.lo < (r.write ? any_hi : write_hi)) return r.tensor;
        any_hi = std::max(any_hi, r.hi);
        if (!r.write) {
            if (!reads->empty() && reads->back().hi >= r.lo) reads->back().hi = std::max(reads->back().hi, r.hi);
            else reads->push_back({r.lo, r.hi});
            continue;
        }
        write_hi = std::max(write_hi, r.hi);
        if (!ranges->empty() && ranges->back().hi == r.lo) ranges->back().hi = r.hi;
        else ranges->push_back({r.lo, r.hi});
    }
    return -1;
}

}  // namespace
}  // namespace zero_shard
