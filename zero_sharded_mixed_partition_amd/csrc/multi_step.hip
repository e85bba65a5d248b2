// The optimizer step over a list of tensors: the norm pass over their
// gradients and one AdamW launch over all of them, with 32- or 8-bit moments.
//
// The list is described once, in a table (zero_multi_table_build): one
// descriptor per tensor (its pointers, element types and hyperparameter group)
// and two maps, from the norm pass's chunks and from the update's units of work
// to their tensors.  A workgroup finds its work with two dependent scalar
// loads, whatever the number and the sizes of the tensors.  Each map costs 8
// bytes per 8192 elements, the second one more where tensors are small.
//
//  multi_sqnorm + multi_norm_finish: each block sums the exact fp64 squares
//          of its chunks and leaves one partial per tensor it meets, in a slot
//          that no other block writes: no atomics, nothing to clear.  The
//          second kernel adds the slots in a fixed order: all of them for the
//          total, a tensor's for its own sum.
//  multi_adam: one wave64 per 256 elements, the lane layout and the arithmetic
//          of the shard's update; the tensor's types and coefficients are
//          uniform over the wave.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <type_traits>
#include <vector>

#include "list_table.h"
#include "moments8.h"

namespace zero_shard {
namespace {

constexpr int64_t kChunk = 8192;                          // elements per entry of the norm pass's map
// LDS reserved per one-wave workgroup and never used, to cap residency (as for
// the shards' updates).  Measured on MI355X, 1.07B elements in 39 tensors with
// bf16 gradients and copies: 32 bits 6.62 TB/s at 15 KiB (10 resident per CU),
// 6.55 at 14, 6.44 at 12.5, 5.86 without; 8 bits 6.41 at 7 KiB (21 resident),
// 6.40 at 6, 6.18 at 8.5, 6.32 without.  Two tasks per wave: 6.13 (16 KiB) and
// 6.32 TB/s (10 KiB).
constexpr size_t kLds32 = 15 * 1024, kLds8 = 7 * 1024;
constexpr int64_t kMultiMaxGrid = (int64_t(1) << 26) - 1;
// Blocks of the norm pass: 512 (2 per CU, as the shard's pass) for long runs of
// chunks, twice as many where a block would meet several tensors or only a few
// chunks.  1.07B elements in 39 tensors: 306 us with 512, 311 with 1024; 67M in
// 4: 24.5 and 25.6; 17M in 4: 10.0 and 9.4; 3,000 tensors of 500: 13.8 and
// 11.0; 10,000 of 64: 26.2 and 18.3.
constexpr int kMultiNormBlocks = 512;
constexpr uint32_t kTableMagic = 0x5A53544Du;

// ---------------------------------------------------------------- the table

struct TensorDesc {
    float* master;
    void* exp_avg;            // 8 bits: the codes
    void* exp_avg_sq;         // 8 bits: the scales
    const void* grad;
    void* param_out;
    int64_t numel;            // > 0
    int32_t gdt, pdt;         // pdt 0: no copy
    int32_t group;
    uint32_t user;            // index in the caller's list
    uint32_t first_chunk, n_chunks;
    int32_t shift;            // the update's tasks start this many elements before multiples of kTask
    int32_t reserved;
};

// At the start of the table.  The device image is [0, device_bytes): this
// header, the descriptors of the tensors that hold elements, the two maps and
// the caller's indices of the empty ones.  The host part behind it holds the
// address ranges that the update writes and those of the gradients, each merged
// and sorted, so that a call checks a pointer against the whole list at once.
struct TableHeader {
    uint32_t magic;
    int32_t state_bits, n_groups;
    int32_t n_user, n_tensors, n_empty;
    int64_t n_chunks, n_units;
    int64_t unit_log2;
    int64_t desc_at, chunks_at, units_at, empty_at, device_bytes;
    int64_t ranges_at, n_ranges;
    int64_t grads_at, n_grads, bytes;
};

// What the kernels need of a table, by value.
struct TableRef {
    const TensorDesc* desc;
    const PieceRef* chunks;
    const PieceRef* units;
    const uint32_t* empty;
    int64_t n_chunks, n_units;
    int32_t unit_log2;
    int32_t n_tensors, n_empty;

    // the table does not change while a kernel runs: scalar reads
    __device__ __forceinline__ const ZS_CONSTANT PieceRef& chunk(int64_t i) const {
        return ((const ZS_CONSTANT PieceRef*)chunks)[i];
    }
    __device__ __forceinline__ const ZS_CONSTANT PieceRef& unit(int64_t i) const {
        return ((const ZS_CONSTANT PieceRef*)units)[i];
    }
    __device__ __forceinline__ const ZS_CONSTANT TensorDesc& tensor(int64_t i) const {
        return ((const ZS_CONSTANT TensorDesc*)desc)[i];
    }
};

// ---------------------------------------------------------------- norm pass

// The squares of chunks first .. stop of one tensor, by one block.
template <int DT>
__device__ __forceinline__ void tensor_squares(const void* G, int64_t n, uint32_t first, uint32_t stop, double& acc,
                                               uint32_t& bad) {
    constexpr int kPer = GradFmt<DT>::per_vec, kSize = 16 / kPer;
    constexpr int kLoads = (int)(kChunk / (kBlock * kPer));
    const char* g = static_cast<const char*>(G) + threadIdx.x * 16;
    const uint32_t whole = (uint32_t)(n / kChunk);
    uint32_t c = first;
    for (; c < stop && c < whole; ++c) {
        const char* at = g + (int64_t)c * (kChunk * kSize);
        u32x4 q[kLoads];
#pragma unroll
        for (int u = 0; u < kLoads; ++u) q[u] = ld16_any(at + u * (kBlock * 16));
#pragma unroll
        for (int u = 0; u < kLoads; ++u) accumulate_vec<DT>(q[u], acc, bad);
    }
    if (c == stop) return;
    // the tensor's last, partial chunk
    for (int64_t i = (int64_t)c * kChunk + threadIdx.x * kPer; i < n; i += kBlock * kPer) {
        if (i + kPer <= n) {
            accumulate_vec<DT>(ld16_any(static_cast<const char*>(G) + i * kSize), acc, bad);
        } else {
            for (int64_t k = i; k < n; ++k) {
                uint32_t w;
                if constexpr (DT == ZERO_F32) w = global(static_cast<const uint32_t*>(G))[k];
                else w = global(static_cast<const uint16_t*>(G))[k];
                bad |= (w & GradFmt<DT>::mask) + GradFmt<DT>::carry;
                const double a = (double)ld_grad1<DT>(G, k);
                acc = fma(a, a, acc);
            }
        }
    }
}

__device__ __forceinline__ int64_t block_begin(int64_t b, int64_t nb, int64_t n_chunks) { return b * n_chunks / nb; }

// Block b sums an equal run of consecutive chunks, tensor by tensor, and
// leaves one partial per tensor it meets.  Along the chunks block and tensor
// both rise, by at most one at a time, so block + tensor is a slot of its own:
// blocks + tensors - 1 slots hold every partial.  (With chunks dealt out in
// turn every block meets every large tensor and pays the reduction for each:
// 5.4 against 7.0 TB/s on 1.07B bf16 elements in 39 tensors.)  Block 0 also
// leaves the factor (1/scale)^2 behind the slots: the second kernel's decision
// may change the scale while its other blocks still need it.
__global__ __launch_bounds__(kBlock) void multi_sqnorm(TableRef t, double inv2, const double* __restrict__ d_scale,
                                                       double* __restrict__ slots, uint32_t* __restrict__ flags) {
    __shared__ double s_sq[kWaves];
    __shared__ uint32_t s_bad[kWaves];
    const int64_t end = block_begin((int64_t)blockIdx.x + 1, gridDim.x, t.n_chunks);
    uint32_t all_bad = 0;
    for (int64_t c = block_begin(blockIdx.x, gridDim.x, t.n_chunks); c < end;) {
        const ZS_CONSTANT PieceRef& ref = t.chunk(c);
        const ZS_CONSTANT TensorDesc& d = t.tensor(ref.tensor);
        const uint32_t first = ref.piece, left = d.n_chunks - first;
        const uint32_t stop = first + (left < end - c ? left : (uint32_t)(end - c));
        double acc = 0.0;
        uint32_t bad = 0;
        if (d.gdt == ZERO_F16) tensor_squares<ZERO_F16>(d.grad, d.numel, first, stop, acc, bad);
        else if (d.gdt == ZERO_BF16) tensor_squares<ZERO_BF16>(d.grad, d.numel, first, stop, acc, bad);
        else tensor_squares<ZERO_F32>(d.grad, d.numel, first, stop, acc, bad);
        block_reduce(acc, bad, s_sq, s_bad);
        c += stop - first;
        if (threadIdx.x == 0) {
            slots[blockIdx.x + ref.tensor] = acc;
            all_bad |= bad & kNonfiniteBits;
            // a run that ends with its tensor leaves out the slot before the next block's first
            if (c == end && c < t.n_chunks && stop == d.n_chunks) slots[blockIdx.x + ref.tensor + 1] = 0.0;
        }
        __syncthreads();                                   // s_sq is written again
    }
    if (threadIdx.x == 0) {
        flags[blockIdx.x] = all_bad;
        if (blockIdx.x == 0) {
            if (d_scale != nullptr) {
                const double inv = 1.0 / *d_scale;
                inv2 = inv * inv;
            }
            slots[gridDim.x + t.n_tensors] = inv2;
        }
    }
}

struct HyperSet {
    HyperArgs h[ZERO_MAX_GROUPS];
    int32_t n;
    int32_t unscaled;
};

// The sum of x[0 .. n) over one wave or block of kThreads threads, each adding
// every kThreads-th value in order; eight loads are in flight at a time.
template <int kThreads>
__device__ __forceinline__ double strided_sum(const double* __restrict__ x, int64_t n, int thread) {
    double acc = 0.0;
    int64_t i = thread;
    for (; i + 7 * kThreads < n; i += 8 * kThreads) {
        double v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = x[i + k * kThreads];
#pragma unroll
        for (int k = 0; k < 8; ++k) acc += v[k];
    }
    for (; i < n; i += kThreads) acc += x[i];
    return acc;
}

constexpr int kFinishThreads = 1024;
constexpr int kFinishWaves = kFinishThreads / 64;

// Block 0: the total, the flag and, with st given, the step's decision: a
// thread per group forms its coefficient block, then one advances the state.
// The other blocks: a wave per tensor sums that tensor's slots.
__global__ __launch_bounds__(kFinishThreads) void multi_norm_finish(
    TableRef t, int nb, const double* __restrict__ slots, const uint32_t* __restrict__ flags, double* __restrict__ d_sq,
    int32_t* __restrict__ d_ovf, double* __restrict__ d_tensor_sq, zero_step_state* __restrict__ st, HyperSet hs,
    StepCoef* __restrict__ coefs) {
    __shared__ double s_sq[kFinishWaves];
    __shared__ uint32_t s_bad[kFinishWaves];
    const double inv2 = slots[nb + t.n_tensors];
    // uniform over the wave
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    if (blockIdx.x > 0) {
        const int64_t i = (int64_t)(blockIdx.x - 1) * kFinishWaves + wave;
        if (i < t.n_tensors) {
            const ZS_CONSTANT TensorDesc& d = t.tensor(i);
            // the block that holds chunk c: the last one that begins at or before it
            const int64_t first = (((int64_t)d.first_chunk + 1) * nb - 1) / t.n_chunks;
            const int64_t last = (((int64_t)d.first_chunk + d.n_chunks) * nb - 1) / t.n_chunks;
            double acc = strided_sum<64>(slots + first + i, last - first + 1, lane);
            for (int off = 32; off > 0; off >>= 1) acc += __shfl_xor(acc, off, 64);
            if (lane == 0) d_tensor_sq[d.user] = acc * inv2;
        } else if (i < t.n_tensors + t.n_empty && lane == 0) {
            d_tensor_sq[t.empty[i - t.n_tensors]] = 0.0;
        }
        return;
    }
    double acc = strided_sum<kFinishThreads>(slots, t.n_tensors > 0 ? nb + t.n_tensors - 1 : 0, threadIdx.x);
    uint32_t bad = 0;
    for (int i = threadIdx.x; i < nb; i += kFinishThreads) bad |= flags[i];
    for (int off = 32; off > 0; off >>= 1) {
        acc += __shfl_xor(acc, off, 64);
        bad |= __shfl_xor(bad, off, 64);
    }
    if (lane == 0) {
        s_sq[wave] = acc;
        s_bad[wave] = bad;
    }
    if (st != nullptr && (int)threadIdx.x < hs.n) decide_coef(st, hs.h[threadIdx.x], hs.unscaled, coefs + threadIdx.x);
    __syncthreads();                                      // the blocks are formed before the state moves on
    if (threadIdx.x == 0) {
        for (int w = 1; w < kFinishWaves; ++w) {
            acc += s_sq[w];
            bad |= s_bad[w];
        }
        *d_sq = acc * inv2;
        *d_ovf = bad ? 1 : 0;
        if (st != nullptr) decide_advance(st, bad ? 1 : 0);
    }
}

__global__ __launch_bounds__(64) void multi_decide(zero_step_state* __restrict__ st, const int32_t* __restrict__ d_ovf,
                                                   HyperSet hs, StepCoef* __restrict__ coefs) {
    if ((int)threadIdx.x < hs.n) decide_coef(st, hs.h[threadIdx.x], hs.unscaled, coefs + threadIdx.x);
    __syncthreads();
    if (threadIdx.x == 0) decide_advance(st, *d_ovf != 0 ? 1 : 0);
}

// ---------------------------------------------------------------- AdamW

// Elements [base, base + 256) of one tensor, as far as they exist, by one wave;
// lane l owns four consecutive elements.
template <int GDT, int PDT>
__device__ __forceinline__ void adam32_task(float* P, float* M, float* V, const void* G, uint16_t* Pout, int64_t n,
                                            int64_t base, const StepCoef& c, const double* d_sq) {
    if (base >= 0 && base + kTask <= n) {
        const int64_t e = base + 4 * threadIdx.x;
        f32x4 p = ld_any(P + e), m = ld_any(M + e), v = ld_any(V + e);
        Grad4<GDT> gq;
        gq.load(G, e);
        const float gscale = clipped_scale(c, d_sq);          // while the loads are on their way
        float g[4], out[4];
        gq.values(g);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float pj = p[j], mj = m[j], vj = v[j];
            adam_elem(c, gscale, g[j], pj, mj, vj);
            p[j] = out[j] = pj;
            m[j] = mj;
            v[j] = vj;
        }
        st_any(p, P + e);
        st_any(m, M + e);
        st_any(v, V + e);
        if constexpr (PDT != 0) st_any(pack4_16<PDT>(out), Pout + e);
        return;
    }
    // a tensor's begin or end: one element per lane at a time
    const float gscale = clipped_scale(c, d_sq);
    const int64_t end = base + kTask < n ? base + kTask : n;
    for (int64_t e = base + threadIdx.x; e < end; e += kTaskThreads) {
        if (e < 0) continue;
        float pe = global(P)[e], me = global(M)[e], ve = global(V)[e];
        adam_elem(c, gscale, ld_grad1<GDT>(G, e), pe, me, ve);
        global(P)[e] = pe;
        global(M)[e] = me;
        global(V)[e] = ve;
        if constexpr (PDT != 0) global(Pout)[e] = (uint16_t)to16<PDT>(pe);
    }
}

template <int BITS, int GDT, int PDT>
__device__ __forceinline__ void list_task(const ZS_CONSTANT TensorDesc& d, int64_t base, const StepCoef& c, const double* d_sq,
                                          uint32_t key) {
    uint16_t* out = static_cast<uint16_t*>(d.param_out);
    if constexpr (BITS == 8)
        adam8_task<GDT, PDT>(d.master, static_cast<u32x2*>(d.exp_avg), static_cast<uint16_t*>(d.exp_avg_sq), d.grad,
                             out, d.numel, base, c, d_sq, dither_tensor(key, d.user, base));
    else
        adam32_task<GDT, PDT>(d.master, static_cast<float*>(d.exp_avg), static_cast<float*>(d.exp_avg_sq), d.grad, out,
                              d.numel, base, c, d_sq);
}

template <int BITS, int GDT>
__device__ __forceinline__ void list_task_p(const ZS_CONSTANT TensorDesc& d, int64_t base, const StepCoef& c, const double* d_sq,
                                            uint32_t key) {
    if (d.pdt == ZERO_F16) list_task<BITS, GDT, ZERO_F16>(d, base, c, d_sq, key);
    else if (d.pdt == ZERO_BF16) list_task<BITS, GDT, ZERO_BF16>(d, base, c, d_sq, key);
    else list_task<BITS, GDT, 0>(d, base, c, d_sq, key);
}

// The groups' coefficients and the keys of their steps' random bits, by value.
struct CoefSet {
    StepCoef c[ZERO_MAX_GROUPS];
    uint32_t key[ZERO_MAX_GROUPS];
};

template <int BITS>
__device__ __forceinline__ void list_wave(const TableRef& t, int64_t w, const StepCoef* coefs, const uint32_t* keys,
                                          uint32_t key, const double* d_sq) {
    const ZS_CONSTANT PieceRef& ref = t.unit(w >> t.unit_log2);
    const ZS_CONSTANT TensorDesc& d = t.tensor(ref.tensor);
    const int64_t task = ((int64_t)ref.piece << t.unit_log2) + (w & ((1 << t.unit_log2) - 1));
    const int64_t base = task * kTask - (BITS == 32 ? d.shift : 0);
    if (base >= d.numel) return;
    const StepCoef c = coefs[d.group];
    if (keys != nullptr) key = keys[d.group];
    if (d.gdt == ZERO_F16) list_task_p<BITS, ZERO_F16>(d, base, c, d_sq, key);
    else if (d.gdt == ZERO_BF16) list_task_p<BITS, ZERO_BF16>(d, base, c, d_sq, key);
    else list_task_p<BITS, ZERO_F32>(d, base, c, d_sq, key);
}

template <int BITS>
__global__ __launch_bounds__(kTaskThreads) void multi_adam(CoefSet cs, TableRef t, const double* __restrict__ d_sq,
                                                           const int32_t* __restrict__ d_ovf) {
    if (d_ovf != nullptr && *d_ovf != 0) return;          // skipped step: nothing is written
    for (int64_t w = blockIdx.x; w < t.n_units << t.unit_log2; w += gridDim.x)
        list_wave<BITS>(t, w, cs.c, cs.key, 0, d_sq);
}

template <int BITS>
__global__ __launch_bounds__(kTaskThreads) void multi_adam_devcoef(const StepCoef* __restrict__ coefs, uint64_t seed,
                                                                   const int64_t* __restrict__ d_step, TableRef t,
                                                                   const double* __restrict__ d_sq,
                                                                   const int32_t* __restrict__ d_ovf) {
    if (d_ovf != nullptr && *d_ovf != 0) return;
    const uint32_t key = BITS == 8 ? dither_key(seed, (uint64_t)*d_step) : 0;
    for (int64_t w = blockIdx.x; w < t.n_units << t.unit_log2; w += gridDim.x)
        list_wave<BITS>(t, w, coefs, nullptr, key, d_sq);
}

// ---------------------------------------------------------------- host side

// At least one block: it also leaves the factor for the second kernel.
int norm_grid(const TableHeader& h) {
    const bool short_runs = h.n_chunks <= 8 * kMultiNormBlocks || h.n_chunks < 8 * (int64_t)h.n_tensors;
    const int64_t most = short_runs ? 2 * kMultiNormBlocks : kMultiNormBlocks;
    return (int)(h.n_chunks < 1 ? 1 : h.n_chunks < most ? h.n_chunks : most);
}

size_t norm_workspace(const TableHeader& h) {
    const size_t nb = (size_t)norm_grid(h);
    return (((nb + (size_t)h.n_tensors + 1) * sizeof(double) + nb * sizeof(uint32_t)) + 255) & ~(size_t)255;
}

int read_table(const void* table, const void* d_table, TableHeader* h) {
    if (table == nullptr) return fail(ZERO_EINVAL, "table is NULL");
    if ((uintptr_t)table & 7u) return fail(ZERO_EALIGN, "table must be 8-byte aligned");
    std::memcpy(h, table, sizeof(*h));
    if (h->magic != kTableMagic) return fail(ZERO_EINVAL, "not a table of zero_multi_table_build");
    if (h->n_user > 0) {
        if (d_table == nullptr) return fail(ZERO_EINVAL, "d_table is NULL");
        if (!aligned16(d_table)) return fail(ZERO_EALIGN, "d_table must be 16-byte aligned");
    }
    return ZERO_OK;
}

TableRef table_ref(const TableHeader& h, const void* d_table) {
    return TableRef{at<TensorDesc>(d_table, h.desc_at), at<PieceRef>(d_table, h.chunks_at),
                    at<PieceRef>(d_table, h.units_at), at<uint32_t>(d_table, h.empty_at), h.n_chunks, h.n_units,
                    (int32_t)h.unit_log2, h.n_tensors, h.n_empty};
}

// ... one that the update writes
bool written(const void* table, const TableHeader& h, const void* p, int64_t bytes) {
    return meets(at<AddressRange>(table, h.ranges_at), h.n_ranges, p, bytes);
}

int check_groups(const TableHeader& h, int32_t n_groups) {
    if (n_groups < 1 || n_groups > ZERO_MAX_GROUPS)
        return fail(ZERO_EINVAL, "n_groups must lie in [1, %d] (got %d)", ZERO_MAX_GROUPS, n_groups);
    if (h.n_groups > n_groups)
        return fail(ZERO_EINVAL, "the table names group %d, n_groups is %d", h.n_groups - 1, n_groups);
    return ZERO_OK;
}

int hyper_set(const zero_adam_hyper* hp, int32_t n_groups, int32_t unscaled, HyperSet* out) {
    if (hp == nullptr) return fail(ZERO_EINVAL, "hp is NULL");
    if (n_groups < 1 || n_groups > ZERO_MAX_GROUPS)
        return fail(ZERO_EINVAL, "n_groups must lie in [1, %d] (got %d)", ZERO_MAX_GROUPS, n_groups);
    *out = HyperSet{};
    out->n = n_groups;
    out->unscaled = unscaled ? 1 : 0;
    for (int g = 0; g < n_groups; ++g) {
        const int st = check_hyper(hp[g].lr, hp[g].beta1, hp[g].beta2, hp[g].eps, hp[g].weight_decay, hp[g].max_grad_norm);
        if (st != ZERO_OK) return st;
        out->h[g] = HyperArgs{hp[g].lr, hp[g].beta1, hp[g].beta2, hp[g].eps, hp[g].weight_decay, hp[g].max_grad_norm};
    }
    return ZERO_OK;
}

int check_device_state(const zero_step_state* d_state, const void* d_coefs, bool coefs) {
    if (d_state == nullptr) return fail(ZERO_EINVAL, "d_state is NULL");
    if ((uintptr_t)d_state & 7u) return fail(ZERO_EALIGN, "d_state must be 8-byte aligned");
    if (coefs && (d_coefs == nullptr || ((uintptr_t)d_coefs & 7u)))
        return fail(ZERO_EINVAL, "d_coefs NULL or not 8-byte aligned");
    return ZERO_OK;
}

int multi_norm(const void* table, const void* d_table, double inv2, const double* d_scale, double* d_sqnorm,
               int32_t* d_overflow, double* d_tensor_sqnorm, void* d_workspace, size_t workspace_bytes, hipStream_t s,
               zero_step_state* st, const HyperSet& hs, StepCoef* coefs) {
    TableHeader h;
    int rc = read_table(table, d_table, &h);
    if (rc != ZERO_OK) return rc;
    if (d_sqnorm == nullptr || d_overflow == nullptr || d_workspace == nullptr)
        return fail(ZERO_EINVAL, "NULL output or workspace pointer");
    if (((uintptr_t)d_sqnorm & 7u) || ((uintptr_t)d_overflow & 3u) || ((uintptr_t)d_tensor_sqnorm & 7u) ||
        !aligned16(d_workspace))
        return fail(ZERO_EALIGN, "norm outputs or workspace misaligned");
    const size_t need = norm_workspace(h);
    if (workspace_bytes < need) return fail(ZERO_ENOSPC, "workspace %zu bytes, need %zu", workspace_bytes, need);
    struct {
        const void* p;
        int64_t bytes;
    } out[] = {{d_workspace, (int64_t)need},
               {d_sqnorm, sizeof(double)},
               {d_overflow, sizeof(int32_t)},
               {d_tensor_sqnorm, d_tensor_sqnorm ? (int64_t)h.n_user * (int64_t)sizeof(double) : 0},
               {coefs, st ? (int64_t)hs.n * (int64_t)sizeof(StepCoef) : 0},
               {st, st ? (int64_t)sizeof(zero_step_state) : 0},
               {d_scale, st || !d_scale ? 0 : (int64_t)sizeof(double)},
               {h.n_user ? d_table : nullptr, h.n_user ? h.device_bytes : 0}};
    const int n_out = (int)(sizeof(out) / sizeof(out[0]));
    for (int i = 0; i < n_out; ++i)
        for (int j = 0; j < i; ++j)
            if (out[i].bytes && out[j].bytes && overlaps(out[i].p, out[i].bytes, out[j].p, out[j].bytes))
                return fail(ZERO_EINVAL, "the norm pass's outputs, workspace and table must not overlap");
    for (int j = 0; j < 6; ++j)
        if (meets(at<AddressRange>(table, h.grads_at), h.n_grads, out[j].p, out[j].bytes))
            return fail(ZERO_EINVAL, "an output of the norm pass lies in a gradient");
    const int nb = norm_grid(h);
    double* slots = static_cast<double*>(d_workspace);
    uint32_t* flags = reinterpret_cast<uint32_t*>(slots + nb + h.n_tensors + 1);
    const TableRef t = table_ref(h, d_table);
    hipLaunchKernelGGL(multi_sqnorm, dim3(nb), dim3(kBlock), 0, s, t, inv2, d_scale, slots, flags);
    rc = launch_status("multi_sqnorm");
    if (rc != ZERO_OK) return rc;
    const int per_tensor = d_tensor_sqnorm ? (h.n_user + kFinishWaves - 1) / kFinishWaves : 0;
    hipLaunchKernelGGL(multi_norm_finish, dim3(1 + per_tensor), dim3(kFinishThreads), 0, s, t, nb, slots, flags, d_sqnorm,
                       d_overflow, d_tensor_sqnorm, st, hs, coefs);
    return launch_status("multi_norm_finish");
}

// Checks shared by the two forms of the update; sets *h.
int check_update(const void* table, const void* d_table, int32_t n_groups, const double* d_sq, const int32_t* d_ovf,
                 TableHeader* h) {
    const int rc = read_table(table, d_table, h);
    if (rc != ZERO_OK) return rc;
    if (h->state_bits != 32 && h->state_bits != 8) return fail(ZERO_EINVAL, "the table describes gradients only");
    if ((uintptr_t)d_sq & 7u) return fail(ZERO_EALIGN, "d_global_sqnorm misaligned");
    if ((uintptr_t)d_ovf & 3u) return fail(ZERO_EALIGN, "d_global_overflow misaligned");
    if (written(table, *h, d_sq, sizeof(double)) || written(table, *h, d_ovf, sizeof(int32_t)) ||
        (h->n_user && written(table, *h, d_table, h->device_bytes)))
        return fail(ZERO_EINVAL, "the norm, the flag or the table lies in a buffer the update writes");
    return check_groups(*h, n_groups);
}

dim3 update_grid(const TableHeader& h) {
    const int64_t w = h.n_units << h.unit_log2;
    return dim3((unsigned)(w < kMultiMaxGrid ? w : kMultiMaxGrid));
}

// Elements that the first task of a tensor starts before it.
int32_t phase_of(const zero_tensor& t, int32_t state_bits) {
    return state_bits == 32 ? (int32_t)(reinterpret_cast<uintptr_t>(t.master) / sizeof(float) % kPhase) : 0;
}

int64_t chunks_of(const zero_tensor& t) { return (t.numel + kChunk - 1) / kChunk; }

// Tasks of the update that a tensor takes (0 for an empty one).
int64_t tasks_of(const zero_tensor& t, int32_t state_bits) {
    return t.numel ? (t.numel + phase_of(t, state_bits) + kTask - 1) / kTask : 0;
}

int64_t units_of(const zero_tensor& t, int32_t state_bits, int unit_log2) {
    return (tasks_of(t, state_bits) + (1 << unit_log2) - 1) >> unit_log2;
}

int build_table(const zero_tensor* tensors, int32_t n_tensors, int32_t state_bits, void* table, size_t capacity,
                size_t* bytes, size_t* device_bytes) {
    if (bytes == nullptr || device_bytes == nullptr) return fail(ZERO_EINVAL, "bytes and device_bytes are required");
    *bytes = *device_bytes = 0;
    if (n_tensors < 0) return fail(ZERO_EINVAL, "n_tensors < 0");
    if (n_tensors > 0 && tensors == nullptr) return fail(ZERO_EINVAL, "tensors is NULL");
    if (state_bits != 0 && state_bits != 8 && state_bits != 32)
        return fail(ZERO_EINVAL, "state_bits must be 32, 8 or 0 (got %d)", state_bits);
    std::vector<Region> regions;
    regions.reserve((size_t)n_tensors * (state_bits ? 5 : 1));
    TableHeader h{};
    h.magic = kTableMagic;
    h.state_bits = state_bits;
    h.n_user = n_tensors;
    for (int32_t i = 0; i < n_tensors; ++i) {
        const zero_tensor& t = tensors[i];
        if (t.numel < 0) return fail(ZERO_EINVAL, "tensor %d: numel < 0", i);
        if (t.numel > INT64_MAX / 8) return fail(ZERO_ERANGE, "tensor %d: numel too large", i);
        if (t.grad_dtype != ZERO_F16 && t.grad_dtype != ZERO_BF16 && t.grad_dtype != ZERO_F32)
            return fail(ZERO_EINVAL, "tensor %d: unknown grad_dtype %d", i, t.grad_dtype);
        if (state_bits) {
            if (t.group < 0 || t.group >= ZERO_MAX_GROUPS)
                return fail(ZERO_EINVAL, "tensor %d: group %d outside [0, %d)", i, t.group, ZERO_MAX_GROUPS);
            if (t.param_out && t.param_dtype != ZERO_F16 && t.param_dtype != ZERO_BF16)
                return fail(ZERO_EINVAL, "tensor %d: unknown param_dtype %d", i, t.param_dtype);
            h.n_groups = std::max(h.n_groups, t.group + 1);
        }
        if (t.numel == 0) {
            ++h.n_empty;
            continue;
        }
        h.n_chunks += chunks_of(t);
        if (h.n_chunks > (int64_t)UINT32_MAX) return fail(ZERO_ERANGE, "the list is too long");
        ++h.n_tensors;
        if (t.grad == nullptr) return fail(ZERO_EINVAL, "tensor %d: grad is NULL", i);
        const int gb = grad_bytes(t.grad_dtype);
        if ((uintptr_t)t.grad & (unsigned)(gb - 1)) return fail(ZERO_EALIGN, "tensor %d: grad misaligned", i);
        const auto add = [&](const void* p, int64_t nbytes, bool write) {
            regions.push_back({reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + (uintptr_t)nbytes, write, i});
        };
        add(t.grad, t.numel * gb, false);
        if (!state_bits) continue;
        if (!t.master || !t.exp_avg || !t.exp_avg_sq) return fail(ZERO_EINVAL, "tensor %d: NULL state pointer", i);
        const unsigned first = state_bits == 8 ? 7u : 3u, second = state_bits == 8 ? 1u : 3u;
        if (((uintptr_t)t.master & 3u) || ((uintptr_t)t.exp_avg & first) || ((uintptr_t)t.exp_avg_sq & second) ||
            ((uintptr_t)t.param_out & 1u))
            return fail(ZERO_EALIGN, "tensor %d: a pointer is not aligned to its elements (8-bit codes: 8 bytes)", i);
        add(t.master, t.numel * 4, true);
        add(t.exp_avg, state_bits == 8 ? (int64_t)zero_moments8_bytes(t.numel) : t.numel * 4, true);
        add(t.exp_avg_sq, state_bits == 8 ? (int64_t)zero_scales8_bytes(t.numel) : t.numel * 4, true);
        if (t.param_out) add(t.param_out, t.numel * 2, true);
    }
    std::vector<AddressRange> ranges, grads;
    const int32_t clash = merge_regions(regions, &ranges, &grads);
    if (clash >= 0)
        return fail(ZERO_EINVAL, "tensor %d: a buffer the update writes overlaps another of the list", clash);
    if (state_bits) {
        int64_t tasks = 0;
        for (int32_t i = 0; i < n_tensors; ++i) tasks += tasks_of(tensors[i], state_bits);
        for (h.unit_log2 = kMaxUnit;; --h.unit_log2) {
            h.n_units = 0;
            for (int32_t i = 0; i < n_tensors; ++i) h.n_units += units_of(tensors[i], state_bits, (int)h.unit_log2);
            if (h.unit_log2 == 0 || (h.n_units << h.unit_log2) <= tasks + tasks / 10) break;
        }
        if (h.n_units > (int64_t)UINT32_MAX) return fail(ZERO_ERANGE, "the list is too long");
    }
    h.desc_at = pad16((int64_t)sizeof(TableHeader));
    h.chunks_at = pad16(h.desc_at + h.n_tensors * (int64_t)sizeof(TensorDesc));
    h.units_at = pad16(h.chunks_at + h.n_chunks * (int64_t)sizeof(PieceRef));
    h.empty_at = pad16(h.units_at + h.n_units * (int64_t)sizeof(PieceRef));
    h.device_bytes = pad16(h.empty_at + h.n_empty * (int64_t)sizeof(uint32_t));
    h.ranges_at = h.device_bytes;
    h.n_ranges = (int64_t)ranges.size();
    h.grads_at = pad16(h.ranges_at + h.n_ranges * (int64_t)sizeof(AddressRange));
    h.n_grads = (int64_t)grads.size();
    h.bytes = pad16(h.grads_at + h.n_grads * (int64_t)sizeof(AddressRange));
    *bytes = (size_t)h.bytes;
    *device_bytes = (size_t)h.device_bytes;
    if ((uintptr_t)table & 7u) return fail(ZERO_EALIGN, "table must be 8-byte aligned");
    if (table == nullptr || capacity < *bytes) return fail(ZERO_ENOSPC, "table %zu bytes, need %zu", capacity, *bytes);
    char* out = static_cast<char*>(table);
    std::memset(out, 0, (size_t)h.bytes);
    std::memcpy(out, &h, sizeof(h));
    PieceRef* chunks = reinterpret_cast<PieceRef*>(out + h.chunks_at);
    PieceRef* units = reinterpret_cast<PieceRef*>(out + h.units_at);
    uint32_t chunk = 0, tensor = 0, empty = 0;
    for (int32_t i = 0; i < n_tensors; ++i) {
        const zero_tensor& t = tensors[i];
        if (t.numel == 0) {
            const uint32_t u = (uint32_t)i;
            std::memcpy(out + h.empty_at + empty++ * sizeof(u), &u, sizeof(u));
            continue;
        }
        TensorDesc d{};
        d.grad = t.grad;
        d.numel = t.numel;
        d.gdt = t.grad_dtype;
        d.user = (uint32_t)i;
        d.first_chunk = chunk;
        d.n_chunks = (uint32_t)chunks_of(t);
        d.shift = phase_of(t, state_bits);
        if (state_bits) {
            d.master = t.master;
            d.exp_avg = t.exp_avg;
            d.exp_avg_sq = t.exp_avg_sq;
            d.param_out = t.param_out;
            d.pdt = t.param_out ? t.param_dtype : 0;
            d.group = t.group;
        }
        std::memcpy(out + h.desc_at + tensor * sizeof(d), &d, sizeof(d));
        for (uint32_t c = 0; c < d.n_chunks; ++c) *chunks++ = PieceRef{tensor, c};
        chunk += d.n_chunks;
        const uint32_t n_units = state_bits ? (uint32_t)units_of(t, state_bits, (int)h.unit_log2) : 0;
        for (uint32_t u = 0; u < n_units; ++u) *units++ = PieceRef{tensor, u};
        ++tensor;
    }
    if (!ranges.empty()) std::memcpy(out + h.ranges_at, ranges.data(), ranges.size() * sizeof(AddressRange));
    if (!grads.empty()) std::memcpy(out + h.grads_at, grads.data(), grads.size() * sizeof(AddressRange));
    return ZERO_OK;
}

}  // namespace
}  // namespace zero_shard

using namespace zero_shard;

extern "C" {

int zero_multi_table_build(const zero_tensor* tensors, int32_t n_tensors, int32_t state_bits, void* table,
                           size_t capacity, size_t* bytes, size_t* device_bytes) {
    clear_error();
    try {
        return build_table(tensors, n_tensors, state_bits, table, capacity, bytes, device_bytes);
    } catch (...) {
        return fail(ZERO_ENOSPC, "out of host memory");
    }
}

size_t zero_multi_norm_workspace_bytes(const void* table) {
    clear_error();
    TableHeader h;
    if (table == nullptr) return 0;
    std::memcpy(&h, table, sizeof(h));
    return h.magic == kTableMagic ? norm_workspace(h) : 0;
}

int zero_multi_unscale_norm_overflow(const void* table, const void* d_table, double inv_loss_scale, double* d_sqnorm,
                                     int32_t* d_overflow, double* d_tensor_sqnorm, void* d_workspace,
                                     size_t workspace_bytes, void* hip_stream) {
    clear_error();
    if (!(inv_loss_scale > 0.0) || !std::isfinite(inv_loss_scale))
        return fail(ZERO_EINVAL, "inv_loss_scale must be finite and > 0");
    return multi_norm(table, d_table, inv_loss_scale * inv_loss_scale, nullptr, d_sqnorm, d_overflow, d_tensor_sqnorm,
                      d_workspace, workspace_bytes, static_cast<hipStream_t>(hip_stream), nullptr, HyperSet{}, nullptr);
}

int zero_multi_unscale_norm_overflow_dev(const void* table, const void* d_table, int32_t unscaled,
                                         const zero_step_state* d_state, double* d_sqnorm, int32_t* d_overflow,
                                         double* d_tensor_sqnorm, void* d_workspace, size_t workspace_bytes,
                                         void* hip_stream) {
    clear_error();
    const int rc = check_device_state(d_state, nullptr, false);
    if (rc != ZERO_OK) return rc;
    return multi_norm(table, d_table, 1.0, unscaled ? nullptr : &d_state->scaler.scale, d_sqnorm, d_overflow,
                      d_tensor_sqnorm, d_workspace, workspace_bytes, static_cast<hipStream_t>(hip_stream), nullptr,
                      HyperSet{}, nullptr);
}

int zero_multi_norm_decide_dev(const void* table, const void* d_table, int32_t unscaled, const zero_adam_hyper* hp,
                               int32_t n_groups, zero_step_state* d_state, double* d_sqnorm, int32_t* d_overflow,
                               double* d_tensor_sqnorm, void* d_coefs, void* d_workspace, size_t workspace_bytes,
                               void* hip_stream) {
    clear_error();
    HyperSet hs;
    int rc = hyper_set(hp, n_groups, unscaled, &hs);
    if (rc != ZERO_OK) return rc;
    rc = check_device_state(d_state, d_coefs, true);
    if (rc != ZERO_OK) return rc;
    return multi_norm(table, d_table, 1.0, unscaled ? nullptr : &d_state->scaler.scale, d_sqnorm, d_overflow,
                      d_tensor_sqnorm, d_workspace, workspace_bytes, static_cast<hipStream_t>(hip_stream), d_state, hs,
                      static_cast<StepCoef*>(d_coefs));
}

int zero_multi_decide_dev(const zero_adam_hyper* hp, int32_t n_groups, int32_t unscaled, zero_step_state* d_state,
                          const int32_t* d_global_overflow, void* d_coefs, void* hip_stream) {
    clear_error();
    HyperSet hs;
    int rc = hyper_set(hp, n_groups, unscaled, &hs);
    if (rc != ZERO_OK) return rc;
    rc = check_device_state(d_state, d_coefs, true);
    if (rc != ZERO_OK) return rc;
    if (d_global_overflow == nullptr || ((uintptr_t)d_global_overflow & 3u))
        return fail(ZERO_EINVAL, "d_global_overflow NULL or misaligned");
    if (overlaps(d_state, sizeof(zero_step_state), d_coefs, (int64_t)n_groups * (int64_t)sizeof(StepCoef)) ||
        overlaps(d_global_overflow, sizeof(int32_t), d_coefs, (int64_t)n_groups * (int64_t)sizeof(StepCoef)))
        return fail(ZERO_EINVAL, "d_coefs overlaps the state or the flag");
    hipLaunchKernelGGL(multi_decide, dim3(1), dim3(64), 0, static_cast<hipStream_t>(hip_stream), d_state,
                       d_global_overflow, hs, static_cast<StepCoef*>(d_coefs));
    return launch_status("multi_decide");
}

int zero_multi_adam_step(const void* table, const void* d_table, const zero_adam_params* hp, int32_t n_groups,
                         uint64_t seed, const double* d_global_sqnorm, const int32_t* d_global_overflow,
                         void* hip_stream) {
    clear_error();
    if (hp == nullptr) return fail(ZERO_EINVAL, "hp is NULL");
    TableHeader h;
    int rc = check_update(table, d_table, n_groups, d_global_sqnorm, d_global_overflow, &h);
    if (rc != ZERO_OK) return rc;
    CoefSet cs{};
    for (int g = 0; g < n_groups; ++g) {
        rc = prepare_adam(hp + g, &cs.c[g]);
        if (rc != ZERO_OK) return rc;
        if (cs.c[g].clip && d_global_sqnorm == nullptr) return fail(ZERO_EINVAL, "clipping needs d_global_sqnorm");
        cs.key[g] = dither_key(seed, (uint64_t)hp[g].step);
    }
    if (h.n_units == 0) return ZERO_OK;
    const hipStream_t s = static_cast<hipStream_t>(hip_stream);
    const TableRef t = table_ref(h, d_table);
    if (h.state_bits == 8)
        hipLaunchKernelGGL(multi_adam<8>, update_grid(h), dim3(kTaskThreads), kLds8, s, cs, t, d_global_sqnorm,
                           d_global_overflow);
    else
        hipLaunchKernelGGL(multi_adam<32>, update_grid(h), dim3(kTaskThreads), kLds32, s, cs, t, d_global_sqnorm,
                           d_global_overflow);
    return launch_status("multi_adam");
}

int zero_multi_adam_step_coef(const void* table, const void* d_table, const void* d_coefs, int32_t n_groups,
                              uint64_t seed, const int64_t* d_step, const double* d_global_sqnorm,
                              const int32_t* d_global_overflow, void* hip_stream) {
    clear_error();
    if (d_coefs == nullptr || d_global_sqnorm == nullptr)
        return fail(ZERO_EINVAL, "d_coefs and d_global_sqnorm are required");
    if (((uintptr_t)d_coefs | (uintptr_t)d_step) & 7u)
        return fail(ZERO_EALIGN, "d_coefs and d_step must be 8-byte aligned");
    TableHeader h;
    const int rc = check_update(table, d_table, n_groups, d_global_sqnorm, d_global_overflow, &h);
    if (rc != ZERO_OK) return rc;
    if (h.state_bits == 8 && d_step == nullptr) return fail(ZERO_EINVAL, "8-bit moments need d_step");
    if (written(table, h, d_coefs, (int64_t)n_groups * (int64_t)sizeof(StepCoef)) ||
        written(table, h, d_step, sizeof(int64_t)))
        return fail(ZERO_EINVAL, "d_coefs or d_step lies in a buffer the update writes");
    if (h.n_units == 0) return ZERO_OK;
    const hipStream_t s = static_cast<hipStream_t>(hip_stream);
    const TableRef t = table_ref(h, d_table);
    const StepCoef* c = static_cast<const StepCoef*>(d_coefs);
    if (h.state_bits == 8)
        hipLaunchKernelGGL(multi_adam_devcoef<8>, update_grid(h), dim3(kTaskThreads), kLds8, s, c, seed, d_step, t,
                           d_global_sqnorm, d_global_overflow);
    else
        hipLaunchKernelGGL(multi_adam_devcoef<32>, update_grid(h), dim3(kTaskThreads), kLds32, s, c, seed, d_step, t,
                           d_global_sqnorm, d_global_overflow);
    return launch_status("multi_adam_devcoef");
}

}  // extern "C"
