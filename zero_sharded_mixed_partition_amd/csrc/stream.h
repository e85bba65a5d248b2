// Device and launch helpers of the list and 8-bit sources: vector types and
// streaming accesses, the gradient formats, the block reduction, the step's
// decision and the AdamW element, and the host side's pointer checks.
// shard_step.hip has its own forms of these: the committed counter summaries
// of its kernels hold for its text (bench.py compares a hash), so what it is
// made of stays in it.  The two give the same bits, and are tested to.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "common.h"
#include "zero_shard.h"

namespace zero_shard {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kBlock = 256;              // four wave64s
constexpr int kWaves = kBlock / 64;

// ---------------------------------------------------------------- gradient formats

// Per gradient format: values per 16-byte vector, and the exponent-field test.
// For a 32-bit word w, (w & mask) + carry sets bit 15 (low 16-bit half) or
// bit 31 (high half, or the whole fp32 value) exactly when that value's
// exponent field is all ones, i.e. it is inf or NaN; no carry crosses into
// the neighbouring field.  OR-accumulating these words and testing
// kNonfiniteBits at the end is an exact inf/NaN test.
template <int DT>
struct GradFmt;
template <>
struct GradFmt<ZERO_F16> {
    static constexpr int per_vec = 8;
    static constexpr uint32_t mask = 0x7C007C00u, carry = 0x04000400u;
};
template <>
struct GradFmt<ZERO_BF16> {
    static constexpr int per_vec = 8;
    static constexpr uint32_t mask = 0x7F807F80u, carry = 0x00800080u;
};
template <>
struct GradFmt<ZERO_F32> {
    static constexpr int per_vec = 4;
    static constexpr uint32_t mask = 0x7F800000u, carry = 0x00800000u;
};
constexpr uint32_t kNonfiniteBits = 0x80008000u;

__device__ __forceinline__ float f16_to_f32(uint32_t h) {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)h);
}
__device__ __forceinline__ float bf16_to_f32(uint32_t h) { return __uint_as_float(h << 16); }

// low and high 16-bit halves of a 32-bit word as float
template <int DT>
__device__ __forceinline__ void unpack2(uint32_t w, float& lo, float& hi) {
    if constexpr (DT == ZERO_F16) {
        lo = f16_to_f32(w & 0xFFFFu);
        hi = f16_to_f32(w >> 16);
    } else {
        lo = __uint_as_float(w << 16);
        hi = __uint_as_float(w & 0xFFFF0000u);
    }
}

// round-to-nearest-even float -> 16-bit bits (hardware conversion under the
// default round-to-nearest-even mode: v_cvt_f16_f32 / v_cvt_pk_bf16_f32).
// x is the float32 master as stored.  The empty asm makes it an opaque
// register value, so the compiler cannot fuse the conversion into the
// arithmetic that produced it: a fused v_fma_mixlo_f16 rounds the unrounded
// result straight to fp16, which differs from rounding the stored float32
// master in the rare cases where the two roundings meet a tie.
template <int DT>
__device__ __forceinline__ uint32_t to16(float x) {
    __asm__("" : "+v"(x));
    if constexpr (DT == ZERO_F16) {
        return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)x);
    } else {
        return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x);
    }
}

template <typename T>
__device__ __forceinline__ T ld_stream(const T* p) { return __builtin_nontemporal_load(p); }
template <typename T>
__device__ __forceinline__ void st_stream(T v, T* p) { __builtin_nontemporal_store(v, p); }

// ---------------------------------------------------------------- block reduction

__device__ __forceinline__ void block_reduce(double& acc, uint32_t& bad, double* s_sq, uint32_t* s_bad) {
    for (int off = 32; off > 0; off >>= 1) {
        acc += __shfl_xor(acc, off, 64);
        bad |= __shfl_xor(bad, off, 64);
    }
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    if (lane == 0) {
        s_sq[wave] = acc;
        s_bad[wave] = bad;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        double t = s_sq[0];
        uint32_t b = s_bad[0];
        for (int w = 1; w < kWaves; ++w) {
            t += s_sq[w];
            b |= s_bad[w];
        }
        acc = t;
        bad = b;
    }
}

template <int DT>
__device__ __forceinline__ void accumulate_vec(u32x4 q, double& acc, uint32_t& bad) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        bad |= (q[k] & GradFmt<DT>::mask) + GradFmt<DT>::carry;
        if constexpr (DT == ZERO_F32) {
            const double a = (double)__uint_as_float(q[k]);   // exact; square exact in fp64
            acc = fma(a, a, acc);
        } else {
            float lo, hi;
            unpack2<DT>(q[k], lo, hi);
            const double a = (double)lo, b = (double)hi;
            acc = fma(a, a, acc);
            acc = fma(b, b, acc);
        }
    }
}

// ---------------------------------------------------------------- device-resident step state

struct HyperArgs {
    double lr, beta1, beta2, eps, weight_decay, max_grad_norm;
};

// After the (global) overflow flag is known: the coefficient block of step
// t = applied + 1 at the current loss scale, then the loss scale and the step
// counts advanced exactly as zero_loss_scaler_update does on the host.  The
// update kernel that follows reads the block and the flag.  One thread.
__device__ inline void decide_coef(const zero_step_state* __restrict__ st, const HyperArgs& h, int unscaled_grad,
                                   StepCoef* __restrict__ coef) {
    const double inv = unscaled_grad ? 1.0 : 1.0 / st->scaler.scale;
    StepCoef c;
    fill_step_coef(h.lr, h.beta1, h.beta2, h.eps, h.weight_decay, st->applied + 1, inv, h.max_grad_norm, &c);
    *coef = c;
}

__device__ inline void decide_advance(zero_step_state* __restrict__ st, int32_t ovf) {
    zero_loss_scaler s = st->scaler;
    if (ovf) {
        const double next = s.scale * s.backoff;
        s.scale = next > s.min_scale ? next : s.min_scale;
        s.good_steps = 0;
        st->skipped += 1;
    } else {
        st->applied += 1;
        s.good_steps += 1;
        if (s.good_steps >= s.growth_interval) {
            s.scale *= s.growth;
            s.good_steps = 0;
        }
    }
    st->scaler = s;
    st->last_overflow = ovf;
}

// ---------------------------------------------------------------- AdamW element

__device__ __forceinline__ void adam_elem(const StepCoef& c, float gscale, float graw, float& p, float& m,
                                          float& v) {
    const float g = graw * gscale;
    m = fmaf(c.beta1, m, c.omb1 * g);
    // (1 - beta2) g^2 as ((1 - beta2) g) g: the same three roundings as
    // (1 - beta2)(g g), but finite wherever the stored moment is, where g g
    // alone would overflow float32 once |g| passes 2^64
    v = fmaf(c.beta2, v, (c.omb2 * g) * g);
    const float denom = fmaf(sqrtf(v), c.rsqrt_bc2, c.eps);
    p = fmaf(p, c.decay, -(c.step_size * m) / denom);
}

// The factor on the raw gradient: 1/scale, times the clip coefficient
// min(1, max/(norm + 1e-6)) formed in fp64 from the global sum of squares.
__device__ __forceinline__ float clipped_scale(const StepCoef& c, const double* __restrict__ d_sq) {
    if (!c.clip) return c.gscale_fixed;
    double coef = c.max_norm / (sqrt(*d_sq) + 1e-6);
    if (!(coef < 1.0)) coef = 1.0;
    return (float)(c.inv_scale * coef);
}

// one wave64 per workgroup, four consecutive elements per lane
constexpr int kTaskThreads = 64;
constexpr int kTask = 4 * kTaskThreads;

// ---------------------------------------------------------------- host helpers

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool overlaps(const void* a, int64_t abytes, const void* b, int64_t bbytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + (uintptr_t)bbytes && y < x + (uintptr_t)abytes;
}

inline int launch_status(const char* what) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(ZERO_EHIP, "%s: %s", what, hipGetErrorString(e));
    return ZERO_OK;
}

inline int grad_bytes(int32_t dt) { return dt == ZERO_F32 ? 4 : 2; }

}  // namespace
}  // namespace zero_shard
