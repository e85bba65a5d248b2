// One shard's AdamW step on 8-bit moments, and the conversion of moments
// between 32 and 8 bits (the format: moments8.h).
//
//  adam8_update: 16.125 B/element with a 16-bit gradient and copy (2 grad +
//          4 master + 2 codes + 2/32 scales read, 4 + 2 + 2/32 written back,
//          2 param written), against 28 with fp32 moments.
//  pack8 / unpack8: 10.06 B/element (8 B of fp32 moments, 2 B of codes).
// Both are elementwise streams in the lane layout of the fp32 update: one
// wave64 per workgroup, four consecutive elements per lane.
// Measured on MI355X at 251M elements, where a plain copy runs at 6.43 TB/s:
// the update 0.630 ms (6.42 TB/s; a skipped step 0.21 ms), pack8 0.365 ms (6.91)
// and unpack8 0.387 ms (6.51).  HBM counters: the update reads 5% more than its
// bytes, because the 128-byte lines of the scale bytes hold eight waves' scales
// and eight XCDs fetch each; giving an XCD 2, 4 or 8 consecutive tasks removes
// that and is slower all the same (0.631, 0.633 and 0.634 ms).
#include <hip/hip_runtime.h>

#include <cmath>
#include <type_traits>

#include "moments8.h"

namespace zero_shard {
namespace {

constexpr int64_t kMaxGrid = (int64_t(1) << 26) - 1;

// LDS that a workgroup reserves and never uses, to cap how many (one wave
// each) are resident on a CU of 160 KiB, as for the fp32 update: with fewer
// waves in competition HBM sustains more.  Measured on MI355X, 251M elements
// with fp16 gradient and copy: 7 KiB (21 resident) 6.44 TB/s, 6 KiB 6.39, none
// 6.32, 8.5 KiB 6.36, 10 KiB 6.13.  One task per wave: two reach 6.37 (at
// 10 KiB), four 6.32 (14 KiB).
constexpr size_t kLds8 = 7 * 1024;
// pack8: 6 KiB (25 resident) 6.78 TB/s, 7 KiB 6.71, none 6.35; unpack8: 6.48,
// 6.28 and 6.30 (251M elements).
constexpr size_t kLdsConvert = 6 * 1024;

dim3 task_grid(int64_t n) {
    const int64_t t = (n + kTask - 1) / kTask;
    return dim3((unsigned)(t < kMaxGrid ? t : kMaxGrid));
}

// DEV: coefficients and the step that keys the random bits read from device
// memory; else c and key by value.
template <int GDT, int PDT, bool DEV>
__global__ __launch_bounds__(kTaskThreads) void adam8_update(float* __restrict__ P, u32x2* __restrict__ C,
                                                             uint16_t* __restrict__ S, const void* __restrict__ G,
                                                             uint16_t* __restrict__ Pout, int64_t n, StepCoef c,
                                                             uint32_t key, uint64_t seed,
                                                             const StepCoef* __restrict__ pc,
                                                             const int64_t* __restrict__ d_step,
                                                             const double* __restrict__ d_sq,
                                                             const int32_t* __restrict__ d_ovf) {
    if (d_ovf != nullptr && *d_ovf != 0) return;          // skipped step: nothing is written
    if constexpr (DEV) {
        c = *pc;
        key = dither_key(seed, (uint64_t)*d_step);
    }
    const int64_t ntasks = (n + kTask - 1) / kTask;
    for (int64_t t = blockIdx.x; t < ntasks; t += gridDim.x)
        adam8_task<GDT, PDT>(P, C, S, G, Pout, n, t * kTask, c, d_sq, dither_tensor(key, 0, t * kTask));
}

__global__ __launch_bounds__(kTaskThreads) void pack8(u32x2* __restrict__ C, uint16_t* __restrict__ S,
                                                      const float* __restrict__ M, const float* __restrict__ V,
                                                      int64_t n) {
    const int64_t ntasks = (n + kTask - 1) / kTask;
    for (int64_t t = blockIdx.x; t < ntasks; t += gridDim.x) {
        const int64_t e0 = t * kTask + 4 * threadIdx.x;
        float m[4] = {}, s[4] = {};
        if (e0 + 4 <= n) {
            const f32x4 a = ld_any(M + e0), b = ld_any(V + e0);
            for (int j = 0; j < 4; ++j) {
                m[j] = a[j];
                s[j] = sqrtf(b[j]);
            }
        } else {
            for (int j = 0; j < 4; ++j) {
                if (e0 + j < n) {
                    m[j] = M[e0 + j];
                    s[j] = sqrtf(V[e0 + j]);
                }
            }
        }
        const uint32_t mb = scale_byte(top_of_block(m)), sb = scale_byte(top_of_block(s));
        const float smallest = __builtin_ldexpf(scale_of(sb), -9);
        for (int j = 0; j < 4; ++j) s[j] = floor_root(s[j], smallest);
        if (e0 < n) {
            u32x2 codes = {encode4_nearest(m, scale_of(mb)), encode4_nearest(s, scale_of(sb))};
            hold_to_float32(codes, mb, sb);
            st_stream(codes, C + (e0 >> 2));
            if ((threadIdx.x & 7) == 0) S[e0 >> 5] = (uint16_t)(mb | (sb << 8));
        }
    }
}

__global__ __launch_bounds__(kTaskThreads) void unpack8(float* __restrict__ M, float* __restrict__ V,
                                                        const u32x2* __restrict__ C, const uint16_t* __restrict__ S,
                                                        int64_t n) {
    const int64_t ntasks = (n + kTask - 1) / kTask;
    for (int64_t t = blockIdx.x; t < ntasks; t += gridDim.x) {
        const int64_t e0 = t * kTask + 4 * threadIdx.x;
        if (e0 >= n) continue;
        const u32x2 codes = ld_stream(C + (e0 >> 2));
        const uint32_t scales = S[e0 >> 5];
        float m[4], s[4];
        decode4(codes[0], scale_of(scales & 0xFFu), m);
        decode4(codes[1], scale_of(scales >> 8), s);
        if (e0 + 4 <= n) {
            f32x4 a, b;
            for (int j = 0; j < 4; ++j) {
                a[j] = m[j];
                b[j] = s[j] * s[j];
            }
            st_any(a, M + e0);
            st_any(b, V + e0);
        } else {
            for (int j = 0; j < 4; ++j) {
                if (e0 + j < n) {
                    M[e0 + j] = m[j];
                    V[e0 + j] = s[j] * s[j];
                }
            }
        }
    }
}

struct Range {
    const void* p;
    int64_t bytes;
};

int check8_args(float* master, void* moments8, void* scales8, const void* grad, int32_t grad_dtype, void* param_out,
                int32_t param_dtype, int64_t n, const Range* scalars, int n_scalars) {
    if (n < 0) return fail(ZERO_EINVAL, "n < 0");
    if (grad_dtype != ZERO_F16 && grad_dtype != ZERO_BF16 && grad_dtype != ZERO_F32)
        return fail(ZERO_EINVAL, "unknown grad_dtype %d", grad_dtype);
    if (param_out != nullptr && param_dtype != ZERO_F16 && param_dtype != ZERO_BF16)
        return fail(ZERO_EINVAL, "unknown param_dtype %d", param_dtype);
    if (n == 0) return ZERO_OK;
    if (n > INT64_MAX / 8) return fail(ZERO_ERANGE, "n too large");
    if (!master || !moments8 || !scales8 || !grad) return fail(ZERO_EINVAL, "NULL shard pointer");
    if (!aligned16(master) || !aligned16(moments8) || !aligned16(scales8) || !aligned16(grad) ||
        (param_out && !aligned16(param_out)))
        return fail(ZERO_EALIGN, "shard pointers must be 16-byte aligned");
    const Range w[] = {{master, n * 4},
                       {moments8, (int64_t)zero_moments8_bytes(n)},
                       {scales8, (int64_t)zero_scales8_bytes(n)},
                       {param_out, param_out ? n * 2 : 0}};
    for (int i = 0; i < 4; ++i) {
        if (w[i].p == nullptr) continue;
        if (overlaps(grad, n * grad_bytes(grad_dtype), w[i].p, w[i].bytes))
            return fail(ZERO_EINVAL, "grad aliases an output");
        for (int j = 0; j < i; ++j)
            if (overlaps(w[i].p, w[i].bytes, w[j].p, w[j].bytes)) return fail(ZERO_EINVAL, "state buffers overlap");
        // every workgroup reads the scalars while others write the shard
        for (int j = 0; j < n_scalars; ++j)
            if (scalars[j].p && overlaps(scalars[j].p, scalars[j].bytes, w[i].p, w[i].bytes))
                return fail(ZERO_EINVAL, "a scalar the update reads lies in a buffer it writes");
    }
    return ZERO_OK;
}

template <int GDT, int PDT>
void launch8(hipStream_t st, float* P, void* C, void* S, const void* G, void* Pout, int64_t n, const StepCoef& c,
             uint32_t key, uint64_t seed, const StepCoef* pc, const int64_t* d_step, const double* d_sq,
             const int32_t* d_ovf) {
    if (pc == nullptr)
        hipLaunchKernelGGL((adam8_update<GDT, PDT, false>), task_grid(n), dim3(kTaskThreads), kLds8, st, P,
                           static_cast<u32x2*>(C), static_cast<uint16_t*>(S), G, static_cast<uint16_t*>(Pout), n, c,
                           key, seed, pc, d_step, d_sq, d_ovf);
    else
        hipLaunchKernelGGL((adam8_update<GDT, PDT, true>), task_grid(n), dim3(kTaskThreads), kLds8, st, P,
                           static_cast<u32x2*>(C), static_cast<uint16_t*>(S), G, static_cast<uint16_t*>(Pout), n, c,
                           key, seed, pc, d_step, d_sq, d_ovf);
}

template <typename... A>
int launch8_any(int32_t gdt, int32_t pdt, A... a) {
    const auto by_param = [&](auto g) {
        constexpr int G = decltype(g)::value;
        if (pdt == ZERO_F16) launch8<G, ZERO_F16>(a...);
        else if (pdt == ZERO_BF16) launch8<G, ZERO_BF16>(a...);
        else launch8<G, 0>(a...);
    };
    if (gdt == ZERO_F16) by_param(std::integral_constant<int, ZERO_F16>{});
    else if (gdt == ZERO_BF16) by_param(std::integral_constant<int, ZERO_BF16>{});
    else by_param(std::integral_constant<int, ZERO_F32>{});
    return launch_status("adam8_update");
}

int check_convert(const void* exp_avg, const void* exp_avg_sq, const void* moments8, const void* scales8, int64_t n) {
    if (n < 0) return fail(ZERO_EINVAL, "n < 0");
    if (n == 0) return ZERO_OK;
    if (n > INT64_MAX / 8) return fail(ZERO_ERANGE, "n too large");
    if (!exp_avg || !exp_avg_sq || !moments8 || !scales8) return fail(ZERO_EINVAL, "NULL pointer");
    if ((((uintptr_t)exp_avg | (uintptr_t)exp_avg_sq) & 3u) || ((uintptr_t)moments8 & 7u) || ((uintptr_t)scales8 & 1u))
        return fail(ZERO_EALIGN, "fp32 moments must be 4-byte, moments8 8-byte and scales8 2-byte aligned");
    const Range r[] = {{exp_avg, n * 4},
                       {exp_avg_sq, n * 4},
                       {moments8, (int64_t)zero_moments8_bytes(n)},
                       {scales8, (int64_t)zero_scales8_bytes(n)}};
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < i; ++j)
            if (overlaps(r[i].p, r[i].bytes, r[j].p, r[j].bytes)) return fail(ZERO_EINVAL, "buffers overlap");
    return ZERO_OK;
}

}  // namespace
}  // namespace zero_shard

using namespace zero_shard;

extern "C" {

size_t zero_moments8_bytes(int64_t n) { return n < 0 ? 0 : ((size_t)n + 3) / 4 * 8; }

size_t zero_scales8_bytes(int64_t n) { return n < 0 ? 0 : ((size_t)n + kBlock8 - 1) / kBlock8 * 2; }

int zero_shard_adam8_step(float* master, void* moments8, void* scales8, const void* grad, int32_t grad_dtype,
                          void* param_out, int32_t param_dtype, int64_t n, const zero_adam_params* hp, uint64_t seed,
                          const double* d_global_sqnorm, const int32_t* d_global_overflow, void* hip_stream) {
    clear_error();
    StepCoef c;
    int st = prepare_adam(hp, &c);
    if (st != ZERO_OK) return st;
    if (c.clip && d_global_sqnorm == nullptr) return fail(ZERO_EINVAL, "clipping needs d_global_sqnorm");
    if ((uintptr_t)d_global_sqnorm & 7u) return fail(ZERO_EALIGN, "d_global_sqnorm misaligned");
    if ((uintptr_t)d_global_overflow & 3u) return fail(ZERO_EALIGN, "d_global_overflow misaligned");
    const Range scalars[] = {{d_global_sqnorm, sizeof(double)}, {d_global_overflow, sizeof(int32_t)}};
    st = check8_args(master, moments8, scales8, grad, grad_dtype, param_out, param_dtype, n, scalars, 2);
    if (st != ZERO_OK || n == 0) return st;
    return launch8_any(grad_dtype, param_out ? param_dtype : 0, static_cast<hipStream_t>(hip_stream), master, moments8,
                       scales8, grad, param_out, n, c, dither_key(seed, (uint64_t)hp->step), seed,
                       (const StepCoef*)nullptr, (const int64_t*)nullptr, d_global_sqnorm, d_global_overflow);
}

int zero_shard_adam8_step_coef(float* master, void* moments8, void* scales8, const void* grad, int32_t grad_dtype,
                               void* param_out, int32_t param_dtype, int64_t n, const void* d_coef, uint64_t seed,
                               const int64_t* d_step, const double* d_global_sqnorm, const int32_t* d_global_overflow,
                               void* hip_stream) {
    clear_error();
    if (d_coef == nullptr || d_step == nullptr || d_global_sqnorm == nullptr)
        return fail(ZERO_EINVAL, "d_coef, d_step and d_global_sqnorm are required");
    if (((uintptr_t)d_coef | (uintptr_t)d_step | (uintptr_t)d_global_sqnorm) & 7u)
        return fail(ZERO_EALIGN, "d_coef, d_step and d_global_sqnorm must be 8-byte aligned");
    if ((uintptr_t)d_global_overflow & 3u) return fail(ZERO_EALIGN, "d_global_overflow misaligned");
    const Range scalars[] = {{d_global_sqnorm, sizeof(double)},
                             {d_global_overflow, sizeof(int32_t)},
                             {d_coef, sizeof(StepCoef)},
                             {d_step, sizeof(int64_t)}};
    const int st = check8_args(master, moments8, scales8, grad, grad_dtype, param_out, param_dtype, n, scalars, 4);
    if (st != ZERO_OK || n == 0) return st;
    return launch8_any(grad_dtype, param_out ? param_dtype : 0, static_cast<hipStream_t>(hip_stream), master, moments8,
                       scales8, grad, param_out, n, StepCoef{}, 0u, seed, static_cast<const StepCoef*>(d_coef), d_step,
                       d_global_sqnorm, d_global_overflow);
}

int zero_moments8_pack(void* moments8, void* scales8, const float* exp_avg, const float* exp_avg_sq, int64_t n,
                       void* hip_stream) {
    clear_error();
    const int st = check_convert(exp_avg, exp_avg_sq, moments8, scales8, n);
    if (st != ZERO_OK || n == 0) return st;
    hipLaunchKernelGGL(pack8, task_grid(n), dim3(kTaskThreads), kLdsConvert, static_cast<hipStream_t>(hip_stream),
                       static_cast<u32x2*>(moments8), static_cast<uint16_t*>(scales8), exp_avg, exp_avg_sq, n);
    return launch_status("pack8");
}

int zero_moments8_unpack(float* exp_avg, float* exp_avg_sq, const void* moments8, const void* scales8, int64_t n,
                         void* hip_stream) {
    clear_error();
    const int st = check_convert(exp_avg, exp_avg_sq, moments8, scales8, n);
    if (st != ZERO_OK || n == 0) return st;
    hipLaunchKernelGGL(unpack8, task_grid(n), dim3(kTaskThreads), kLdsConvert, static_cast<hipStream_t>(hip_stream), exp_avg,
                       exp_avg_sq, static_cast<const u32x2*>(moments8), static_cast<const uint16_t*>(scales8), n);
    return launch_status("unpack8");
}

}  // extern "C"
