// A step by orthogonalised momentum over a list of matrices: the table, the
// momentum pass in front of the orthogonalisation and the update behind it.
//
// Both passes are streams over the list, one wave64 per 256 elements, as the
// list's AdamW (multi_step.hip): the momentum pass reads the gradient and the
// momentum and writes the momentum and the update to orthogonalise, the update
// reads master and orthogonal matrix and writes master and 16-bit copy.  HBM
// bounds them: 405M elements with 16-bit gradients, updates and copies take 727
// and 737 us, 6.7 and 6.6 TB/s of 12 bytes an element (a large copy reaches 6.4).
// Unlike that update's six and eight streams, these gain nothing from fewer
// waves at a time: with 7, 10 and 16 KiB of LDS reserved a wave the momentum
// pass takes 750, 840 and 1092 us.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstring>
#include <new>
#include <vector>

#include "matrix_table.h"

namespace zero_shard {
namespace {

// What a table describes fits any GPU's memory: its maps stay small too.
constexpr int64_t kMostElements = int64_t(1) << 40, kMostMatrices = 1 << 24;
constexpr int64_t kMaxGrid = (int64_t(1) << 26) - 1;

struct MatrixRef {
    const MatrixDesc* desc;
    const PieceRef* units;
    int64_t n_units;
    int32_t unit_log2;

    // the table does not change while a kernel runs: scalar reads
    __device__ __forceinline__ const ZS_CONSTANT PieceRef& unit(int64_t i) const {
        return ((const ZS_CONSTANT PieceRef*)units)[i];
    }
    __device__ __forceinline__ const ZS_CONSTANT MatrixDesc& entry(int64_t i) const {
        return ((const ZS_CONSTANT MatrixDesc*)desc)[i];
    }
};

struct MuonCoef {
    double lr;
    float mu, omu;                      // momentum, 1 - momentum
    float keep;                         // 1 - lr * weight_decay
    int32_t nesterov;
};

struct MuonSet {
    MuonCoef c[ZERO_MAX_GROUPS];
};

// ---------------------------------------------------------------- momentum

// g = grad * gscale, m = mu m + (1 - mu) g and the update u, in float32.
__device__ __forceinline__ float momentum_elem(const MuonCoef& c, float gscale, float graw, float& m) {
    const float g = c.omu * (graw * gscale);
    m = fmaf(c.mu, m, g);
    return c.nesterov ? fmaf(c.mu, m, g) : m;
}

template <int DT>
__device__ __forceinline__ void st4(const float u[4], void* U, int64_t e) {
    if constexpr (DT == ZERO_F32) st_any(f32x4{u[0], u[1], u[2], u[3]}, static_cast<float*>(U) + e);
    else st_any(pack4_16<DT>(u), static_cast<uint16_t*>(U) + e);
}

template <int DT>
__device__ __forceinline__ void st1(float u, void* U, int64_t e) {
    if constexpr (DT == ZERO_F32) global(static_cast<float*>(U))[e] = u;
    else global(static_cast<uint16_t*>(U))[e] = (uint16_t)to16<DT>(u);
}

// Elements [base, base + 256) of one entry, as far as they exist, by one wave.
template <int GDT, int UDT>
__device__ __forceinline__ void momentum_task(float* M, const void* G, void* U, int64_t n, int64_t base, const MuonCoef& c,
                                              const StepCoef& step, const double* d_sq) {
    if (base >= 0 && base + kTask <= n) {
        const int64_t e = base + 4 * threadIdx.x;
        f32x4 m = ld_any(M + e);
        Grad4<GDT> gq;
        gq.load(G, e);
        const float gscale = clipped_scale(step, d_sq);       // while the loads are on their way
        float g[4], u[4];
        gq.values(g);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float mj = m[j];
            u[j] = momentum_elem(c, gscale, g[j], mj);
            m[j] = mj;
        }
        st_any(m, M + e);
        st4<UDT>(u, U, e);
        return;
    }
    // an entry's begin or end: one element per lane at a time
    const float gscale = clipped_scale(step, d_sq);
    const int64_t end = base + kTask < n ? base + kTask : n;
    for (int64_t e = base + threadIdx.x; e < end; e += kTaskThreads) {
        if (e < 0) continue;
        float m = global(M)[e];
        const float u = momentum_elem(c, gscale, ld_grad1<GDT>(G, e), m);
        global(M)[e] = m;
        st1<UDT>(u, U, e);
    }
}

template <int GDT>
__device__ __forceinline__ void momentum_task_u(const ZS_CONSTANT MatrixDesc& d, int64_t base, const MuonCoef& c,
                                                const StepCoef& step, const double* d_sq) {
    if (d.udt == ZERO_F16) momentum_task<GDT, ZERO_F16>(d.momentum, d.grad, d.update, d.numel, base, c, step, d_sq);
    else if (d.udt == ZERO_BF16) momentum_task<GDT, ZERO_BF16>(d.momentum, d.grad, d.update, d.numel, base, c, step, d_sq);
    else momentum_task<GDT, ZERO_F32>(d.momentum, d.grad, d.update, d.numel, base, c, step, d_sq);
}

// The gradients' factor comes by value, or from d_step (a coefficient block
// formed on the device).
template <bool DEVICE>
__global__ __launch_bounds__(kTaskThreads) void matrix_momentum(MuonSet set, StepCoef by_value, const StepCoef* __restrict__ d_step,
                                                                MatrixRef t, const double* __restrict__ d_sq,
                                                                const int32_t* __restrict__ d_ovf) {
    if (d_ovf != nullptr && *d_ovf != 0) return;          // skipped step: nothing is written
    for (int64_t w = blockIdx.x; w < t.n_units << t.unit_log2; w += gridDim.x) {
        const ZS_CONSTANT PieceRef& ref = t.unit(w >> t.unit_log2);
        const ZS_CONSTANT MatrixDesc& d = t.entry(ref.tensor);
        const int64_t task = ((int64_t)ref.piece << t.unit_log2) + (w & ((1 << t.unit_log2) - 1));
        const int64_t base = task * kTask - d.momentum_shift;
        if (base >= d.numel) continue;
        const MuonCoef c = set.c[d.group];
        StepCoef step;
        if constexpr (DEVICE) step = *d_step;
        else step = by_value;
        if (d.gdt == ZERO_F16) momentum_task_u<ZERO_F16>(d, base, c, step, d_sq);
        else if (d.gdt == ZERO_BF16) momentum_task_u<ZERO_BF16>(d, base, c, step, d_sq);
        else momentum_task_u<ZERO_F32>(d, base, c, step, d_sq);
    }
}

// ---------------------------------------------------------------- update

// p = keep p - (lr scale) o; the copy rounds the stored p.
template <int ODT, int PDT>
__device__ __forceinline__ void update_task(float* P, const void* O, uint16_t* Pout, int64_t n, int64_t base, float keep,
                                            float step) {
    if (base >= 0 && base + kTask <= n) {
        const int64_t e = base + 4 * threadIdx.x;
        f32x4 p = ld_any(P + e);
        Grad4<ODT> oq;
        oq.load(O, e);
        float o[4], out[4];
        oq.values(o);
#pragma unroll
        for (int j = 0; j < 4; ++j) p[j] = out[j] = fmaf(p[j], keep, -(step * o[j]));
        st_any(p, P + e);
        if constexpr (PDT != 0) st_any(pack4_16<PDT>(out), Pout + e);
        return;
    }
    const int64_t end = base + kTask < n ? base + kTask : n;
    for (int64_t e = base + threadIdx.x; e < end; e += kTaskThreads) {
        if (e < 0) continue;
        const float p = fmaf(global(P)[e], keep, -(step * ld_grad1<ODT>(O, e)));
        global(P)[e] = p;
        if constexpr (PDT != 0) global(Pout)[e] = (uint16_t)to16<PDT>(p);
    }
}

template <int ODT>
__device__ __forceinline__ void update_task_p(const ZS_CONSTANT MatrixDesc& d, int64_t base, float keep, float step) {
    uint16_t* out = static_cast<uint16_t*>(d.param_out);
    if (d.pdt == ZERO_F16) update_task<ODT, ZERO_F16>(d.master, d.ortho, out, d.numel, base, keep, step);
    else if (d.pdt == ZERO_BF16) update_task<ODT, ZERO_BF16>(d.master, d.ortho, out, d.numel, base, keep, step);
    else update_task<ODT, 0>(d.master, d.ortho, out, d.numel, base, keep, step);
}

__global__ __launch_bounds__(kTaskThreads) void matrix_update(MuonSet set, MatrixRef t, const int32_t* __restrict__ d_ovf) {
    if (d_ovf != nullptr && *d_ovf != 0) return;
    for (int64_t w = blockIdx.x; w < t.n_units << t.unit_log2; w += gridDim.x) {
        const ZS_CONSTANT PieceRef& ref = t.unit(w >> t.unit_log2);
        const ZS_CONSTANT MatrixDesc& d = t.entry(ref.tensor);
        const int64_t task = ((int64_t)ref.piece << t.unit_log2) + (w & ((1 << t.unit_log2) - 1));
        const int64_t base = task * kTask - d.master_shift;
        if (base >= d.numel) continue;
        const float keep = set.c[d.group].keep, step = (float)(set.c[d.group].lr * d.scale);
        if (d.odt == ZERO_F16) update_task_p<ZERO_F16>(d, base, keep, step);
        else update_task_p<ZERO_BF16>(d, base, keep, step);
    }
}

// ---------------------------------------------------------------- host side

bool float_dtype(int32_t dt) { return dt == ZERO_F16 || dt == ZERO_BF16 || dt == ZERO_F32; }
bool half_dtype(int32_t dt) { return dt == ZERO_F16 || dt == ZERO_BF16; }

int32_t phase_of(const void* fp32) { return (int32_t)(reinterpret_cast<uintptr_t>(fp32) / sizeof(float) % kPhase); }

int64_t tasks_of(int64_t numel, int32_t shift) { return (numel + shift + kTask - 1) / kTask; }

// The units of a map over entries with these tasks: the largest 2^k tasks a
// unit whose last units leave no more than a tenth of the workgroups idle.
int64_t unit_size(const std::vector<int64_t>& tasks, int32_t* log2) {
    int64_t all = 0, units = 0;
    for (const int64_t k : tasks) all += k;
    for (*log2 = kMaxUnit;; --*log2) {
        units = 0;
        for (const int64_t k : tasks) units += (k + (1 << *log2) - 1) >> *log2;
        if (*log2 == 0 || (units << *log2) <= all + all / 10) break;
    }
    return units;
}

int check_matrix(const zero_matrix& m, int32_t i, int64_t* numel) {
    if (m.rows < 0 || m.cols < 0 || m.batch < 0) return fail(ZERO_EINVAL, "matrix %d: negative size", i);
    if (m.rows > ZERO_MAX_MATRIX_SIDE || m.cols > ZERO_MAX_MATRIX_SIDE)
        return fail(ZERO_ERANGE, "matrix %d: a side above %d", i, ZERO_MAX_MATRIX_SIDE);
    if (__builtin_mul_overflow(m.rows * m.cols, m.batch, numel) || *numel > kMostElements)
        return fail(ZERO_ERANGE, "matrix %d: numel too large", i);
    if (m.group < 0 || m.group >= ZERO_MAX_GROUPS)
        return fail(ZERO_EINVAL, "matrix %d: group %d outside [0, %d)", i, m.group, ZERO_MAX_GROUPS);
    if (m.grad && !float_dtype(m.grad_dtype)) return fail(ZERO_EINVAL, "matrix %d: unknown grad_dtype %d", i, m.grad_dtype);
    if (m.update && !float_dtype(m.update_dtype))
        return fail(ZERO_EINVAL, "matrix %d: unknown update_dtype %d", i, m.update_dtype);
    if (m.ortho && !half_dtype(m.ortho_dtype))
        return fail(ZERO_EINVAL, "matrix %d: ortho_dtype must be a 16-bit type (got %d)", i, m.ortho_dtype);
    if (m.param_out && !half_dtype(m.param_dtype))
        return fail(ZERO_EINVAL, "matrix %d: unknown param_dtype %d", i, m.param_dtype);
    if (m.ortho && m.ortho == m.update && m.ortho_dtype != m.update_dtype)
        return fail(ZERO_EINVAL, "matrix %d: ortho in the update's place needs its type", i);
    if (!std::isfinite(m.scale)) return fail(ZERO_EINVAL, "matrix %d: scale must be finite", i);
    const uintptr_t f32 = (uintptr_t)m.master | (uintptr_t)m.momentum |
                          (m.grad && m.grad_dtype == ZERO_F32 ? (uintptr_t)m.grad : 0) |
                          (m.update && m.update_dtype == ZERO_F32 ? (uintptr_t)m.update : 0);
    const uintptr_t f16 = (uintptr_t)m.grad | (uintptr_t)m.update | (uintptr_t)m.ortho | (uintptr_t)m.param_out;
    if ((f32 & 3u) || (f16 & 1u)) return fail(ZERO_EALIGN, "matrix %d: a pointer is not aligned to its elements", i);
    return ZERO_OK;
}

int build_matrix_table(const zero_matrix* matrices, int32_t n, void* table, size_t capacity, size_t* bytes,
                       size_t* device_bytes) {
    if (bytes == nullptr || device_bytes == nullptr) return fail(ZERO_EINVAL, "bytes and device_bytes are required");
    *bytes = *device_bytes = 0;
    if (n < 0) return fail(ZERO_EINVAL, "n_matrices < 0");
    if (n > 0 && matrices == nullptr) return fail(ZERO_EINVAL, "matrices is NULL");
    MatrixHeader h{};
    h.magic = kMatrixMagic;
    h.n_user = n;
    h.can = kCanMomentum | kCanOrtho | kCanUpdate;
    std::vector<Region> regions;
    std::vector<MatrixDesc> desc;
    std::vector<OrthoMatrix> singles;
    std::vector<int64_t> momentum_tasks, master_tasks;
    int64_t n_singles = 0, n_elements = 0;
    for (int32_t i = 0; i < n; ++i) {
        const zero_matrix& m = matrices[i];
        int64_t numel = 0;
        const int rc = check_matrix(m, i, &numel);
        if (rc != ZERO_OK) return rc;
        h.n_groups = std::max(h.n_groups, m.group + 1);
        if (numel == 0) continue;
        if (!m.momentum || !m.grad || !m.update) h.can &= ~kCanMomentum;
        if (!m.update || !m.ortho) h.can &= ~kCanOrtho;
        if (!m.master || !m.ortho) h.can &= ~kCanUpdate;
        const auto add = [&](const void* p, int64_t nbytes, bool write) {
            if (p == nullptr) return;
            regions.push_back({reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + (uintptr_t)nbytes, write, i});
        };
        add(m.grad, numel * grad_bytes(m.grad_dtype), false);
        add(m.master, numel * 4, true);
        add(m.momentum, numel * 4, true);
        add(m.update, numel * grad_bytes(m.update_dtype), true);
        if (m.ortho != m.update) add(m.ortho, numel * 2, true);
        add(m.param_out, numel * 2, true);
        MatrixDesc d{};
        d.master = m.master;
        d.momentum = m.momentum;
        d.grad = m.grad;
        d.update = m.update;
        d.ortho = m.ortho;
        d.param_out = m.param_out;
        d.scale = m.scale;
        d.numel = numel;
        d.gdt = m.grad_dtype;
        d.udt = m.update_dtype;
        d.odt = m.ortho_dtype;
        d.pdt = m.param_out ? m.param_dtype : 0;
        d.group = m.group;
        d.momentum_shift = phase_of(m.momentum);
        d.master_shift = phase_of(m.master);
        desc.push_back(d);
        momentum_tasks.push_back(tasks_of(numel, d.momentum_shift));
        master_tasks.push_back(tasks_of(numel, d.master_shift));
        n_elements += numel;
        n_singles += m.batch;
        if (n_singles > kMostMatrices || n_elements > kMostElements) return fail(ZERO_ERANGE, "the list is too long");
    }
    h.n_entries = (int32_t)desc.size();
    std::vector<AddressRange> ranges, reads;
    const int32_t clash = merge_regions(regions, &ranges, &reads);
    if (clash >= 0) return fail(ZERO_EINVAL, "matrix %d: a buffer that is written overlaps another of the list", clash);
    if (h.can & kCanMomentum) h.n_momentum = unit_size(momentum_tasks, &h.momentum_log2);
    if (h.can & kCanUpdate) h.n_master = unit_size(master_tasks, &h.master_log2);
    if (std::max(h.n_momentum, h.n_master) > (int64_t)UINT32_MAX) return fail(ZERO_ERANGE, "the list is too long");
    OrthoPlan plan;
    if (h.can & kCanOrtho) {
        singles.reserve((size_t)n_singles);
        for (int32_t i = 0; i < n; ++i) {
            const zero_matrix& m = matrices[i];
            if (m.rows == 0 || m.cols == 0) continue;
            for (int64_t b = 0; b < m.batch; ++b)
                singles.push_back({static_cast<const char*>(m.update) + b * m.rows * m.cols * grad_bytes(m.update_dtype),
                                   static_cast<char*>(m.ortho) + b * m.rows * m.cols * 2, m.rows, m.cols, m.update_dtype,
                                   m.ortho_dtype});
        }
        const int rc = plan_ortho(singles, &plan);
        if (rc != ZERO_OK) return rc;
    }
    h.n_passes = (int32_t)plan.passes.size();
    h.workspace_bytes = plan.workspace;
    const auto size = [](const auto& v) { return (int64_t)(v.size() * sizeof(v[0])); };
    h.desc_at = pad16((int64_t)sizeof(MatrixHeader));
    h.momentum_at = pad16(h.desc_at + size(desc));
    h.master_at = pad16(h.momentum_at + h.n_momentum * (int64_t)sizeof(PieceRef));
    h.items_at = pad16(h.master_at + h.n_master * (int64_t)sizeof(PieceRef));
    h.tiles_at = pad16(h.items_at + size(plan.items));
    h.device_bytes = pad16(h.tiles_at + size(plan.tiles));
    h.passes_at = h.device_bytes;
    h.ranges_at = pad16(h.passes_at + size(plan.passes));
    h.n_ranges = (int64_t)ranges.size();
    h.reads_at = pad16(h.ranges_at + size(ranges));
    h.n_reads = (int64_t)reads.size();
    h.bytes = pad16(h.reads_at + size(reads));
    *bytes = (size_t)h.bytes;
    *device_bytes = (size_t)h.device_bytes;
    if ((uintptr_t)table & 7u) return fail(ZERO_EALIGN, "table must be 8-byte aligned");
    if (table == nullptr || capacity < *bytes) return fail(ZERO_ENOSPC, "table %zu bytes, need %zu", capacity, *bytes);
    char* out = static_cast<char*>(table);
    std::memset(out, 0, (size_t)h.bytes);
    std::memcpy(out, &h, sizeof(h));
    const auto put = [&](int64_t where, const auto& v) {
        if (!v.empty()) std::memcpy(out + where, v.data(), v.size() * sizeof(v[0]));
    };
    put(h.desc_at, desc);
    put(h.items_at, plan.items);
    put(h.tiles_at, plan.tiles);
    put(h.passes_at, plan.passes);
    put(h.ranges_at, ranges);
    put(h.reads_at, reads);
    const auto map = [&](int64_t where, const std::vector<int64_t>& tasks, int32_t log2) {
        PieceRef* units = reinterpret_cast<PieceRef*>(out + where);
        for (uint32_t e = 0; e < tasks.size(); ++e)
            for (uint32_t u = 0; u < (uint32_t)((tasks[e] + (1 << log2) - 1) >> log2); ++u) *units++ = PieceRef{e, u};
    };
    if (h.can & kCanMomentum) map(h.momentum_at, momentum_tasks, h.momentum_log2);
    if (h.can & kCanUpdate) map(h.master_at, master_tasks, h.master_log2);
    return ZERO_OK;
}

int muon_set(const zero_muon_params* hp, int32_t n_groups, const MatrixHeader& h, MuonSet* out) {
    if (hp == nullptr) return fail(ZERO_EINVAL, "hp is NULL");
    if (n_groups < 1 || n_groups > ZERO_MAX_GROUPS)
        return fail(ZERO_EINVAL, "n_groups must lie in [1, %d] (got %d)", ZERO_MAX_GROUPS, n_groups);
    if (h.n_groups > n_groups)
        return fail(ZERO_EINVAL, "the table names group %d, n_groups is %d", h.n_groups - 1, n_groups);
    *out = MuonSet{};
    for (int g = 0; g < n_groups; ++g) {
        const zero_muon_params& p = hp[g];
        if (!(p.lr >= 0.0) || !std::isfinite(p.lr)) return fail(ZERO_EINVAL, "lr must be finite and >= 0");
        if (!(p.momentum >= 0.0 && p.momentum < 1.0)) return fail(ZERO_EINVAL, "momentum must lie in [0, 1)");
        if (!(p.weight_decay >= 0.0) || !std::isfinite(p.weight_decay))
            return fail(ZERO_EINVAL, "weight_decay must be finite and >= 0");
        out->c[g] = MuonCoef{p.lr, (float)p.momentum, (float)(1.0 - p.momentum), (float)(1.0 - p.lr * p.weight_decay),
                             p.nesterov ? 1 : 0};
    }
    return ZERO_OK;
}

// The scalars that a call reads: aligned, and not in a buffer that it writes.
int check_scalars(const void* table, const MatrixHeader& h, const double* d_sq, const int32_t* d_ovf, const void* d_coef) {
    if (((uintptr_t)d_sq & 7u) || ((uintptr_t)d_coef & 7u))
        return fail(ZERO_EALIGN, "d_global_sqnorm or d_coef misaligned");
    if ((uintptr_t)d_ovf & 3u) return fail(ZERO_EALIGN, "d_global_overflow misaligned");
    if (matrix_written(table, h, d_sq, sizeof(double)) || matrix_written(table, h, d_ovf, sizeof(int32_t)) ||
        matrix_written(table, h, d_coef, sizeof(StepCoef)))
        return fail(ZERO_EINVAL, "the norm, the flag or the coefficients lie in a buffer the call writes");
    return ZERO_OK;
}

dim3 task_grid(int64_t units, int32_t log2) { return dim3((unsigned)std::min(units << log2, kMaxGrid)); }

int momentum_step(const void* table, const void* d_table, const zero_muon_params* hp, int32_t n_groups, const StepCoef& c,
                  const void* d_coef, const double* d_sq, const int32_t* d_ovf, void* hip_stream) {
    MatrixHeader h;
    int rc = read_matrix_table(table, d_table, kCanMomentum, "the momentum pass (momentum, grad, update)", &h);
    MuonSet set;
    if (rc == ZERO_OK) rc = muon_set(hp, n_groups, h, &set);
    if (rc == ZERO_OK) rc = check_scalars(table, h, d_sq, d_ovf, d_coef);
    if (rc != ZERO_OK || h.n_entries == 0) return rc;
    const MatrixRef t{at<MatrixDesc>(d_table, h.desc_at), at<PieceRef>(d_table, h.momentum_at), h.n_momentum,
                      h.momentum_log2};
    const dim3 grid = task_grid(h.n_momentum, h.momentum_log2);
    const hipStream_t s = static_cast<hipStream_t>(hip_stream);
    const StepCoef* d_step = static_cast<const StepCoef*>(d_coef);
    if (d_step != nullptr)
        hipLaunchKernelGGL(matrix_momentum<true>, grid, dim3(kTaskThreads), 0, s, set, c, d_step, t, d_sq, d_ovf);
    else
        hipLaunchKernelGGL(matrix_momentum<false>, grid, dim3(kTaskThreads), 0, s, set, c, d_step, t, d_sq, d_ovf);
    return launch_status("matrix_momentum");
}

}  // namespace
}  // namespace zero_shard

using namespace zero_shard;

extern "C" {

int zero_matrix_table_build(const zero_matrix* matrices, int32_t n_matrices, void* table, size_t capacity, size_t* bytes,
                            size_t* device_bytes) {
    clear_error();
    try {
        return build_matrix_table(matrices, n_matrices, table, capacity, bytes, device_bytes);
    } catch (...) {
        return fail(ZERO_ENOSPC, "out of host memory");
    }
}

int zero_multi_momentum_step(const void* table, const void* d_table, const zero_muon_params* hp, int32_t n_groups,
                             double inv_loss_scale, double max_grad_norm, const double* d_global_sqnorm,
                             const int32_t* d_global_overflow, void* hip_stream) {
    clear_error();
    if (!(inv_loss_scale > 0.0) || !std::isfinite(inv_loss_scale))
        return fail(ZERO_EINVAL, "inv_loss_scale must be finite and > 0");
    if (std::isnan(max_grad_norm) || (max_grad_norm > 0.0 && !std::isfinite(max_grad_norm)))
        return fail(ZERO_EINVAL, "max_grad_norm must be finite");
    StepCoef c{};
    c.clip = max_grad_norm > 0.0 ? 1 : 0;
    c.max_norm = c.clip ? max_grad_norm : 0.0;
    c.inv_scale = inv_loss_scale;
    c.gscale_fixed = (float)inv_loss_scale;
    if (c.clip && d_global_sqnorm == nullptr) return fail(ZERO_EINVAL, "clipping needs d_global_sqnorm");
    return momentum_step(table, d_table, hp, n_groups, c, nullptr, d_global_sqnorm, d_global_overflow, hip_stream);
}

int zero_multi_momentum_step_coef(const void* table, const void* d_table, const zero_muon_params* hp, int32_t n_groups,
                                  const void* d_coef, const double* d_global_sqnorm, const int32_t* d_global_overflow,
                                  void* hip_stream) {
    clear_error();
    if (d_coef == nullptr || d_global_sqnorm == nullptr)
        return fail(ZERO_EINVAL, "d_coef and d_global_sqnorm are required");
    return momentum_step(table, d_table, hp, n_groups, StepCoef{}, d_coef, d_global_sqnorm, d_global_overflow, hip_stream);
}

int zero_multi_muon_update(const void* table, const void* d_table, const zero_muon_params* hp, int32_t n_groups,
                           const int32_t* d_global_overflow, void* hip_stream) {
    clear_error();
    MatrixHeader h;
    int rc = read_matrix_table(table, d_table, kCanUpdate, "the update (master, ortho)", &h);
    MuonSet set;
    if (rc == ZERO_OK) rc = muon_set(hp, n_groups, h, &set);
    if (rc == ZERO_OK) rc = check_scalars(table, h, nullptr, d_global_overflow, nullptr);
    if (rc != ZERO_OK || h.n_entries == 0) return rc;
    const MatrixRef t{at<MatrixDesc>(d_table, h.desc_at), at<PieceRef>(d_table, h.master_at), h.n_master, h.master_log2};
    hipLaunchKernelGGL(matrix_update, task_grid(h.n_master, h.master_log2), dim3(kTaskThreads), 0,
                       static_cast<hipStream_t>(hip_stream), set, t, d_global_overflow);
    return launch_status("matrix_update");
}

}  // extern "C"
