// AdamW moments held in 8 bits: the number format and the device code that
// reads and writes it (gfx950).
//
// A tensor's elements form blocks of 32.  exp_avg (m) and the square root of
// exp_avg_sq (s) are each stored as an OCP e4m3 code times a power of two per
// block, value = code * 2^k, with k = floor(log2(largest magnitude of the
// block)) - 7: the largest value lands in [128, 256), below e4m3's 448, so
// rounding up never leaves the codes, and the smallest code stands for 2^-16 to
// 2^-17 of it.  Only at float32's upper end would code 256 leave float32 (256 *
// 2^120, or the square of 256 * 2^56): there codes end at 240.  Power-of-two
// scales make decoding exact, and gfx950 converts two values with their scale
// in one instruction.  s instead of its square: the update needs s itself, and
// the format's range of 2^17 below the block's maximum then covers 2^34 of the
// second moment.  A positive s is stored as at least the smallest code, so that
// m / (s + eps) cannot grow without bound once s has become small beside its
// block.
//
// Rounding in the step is stochastic.  With beta2 = 0.999 the second moment
// moves by about 0.1% a step and e4m3 codes are 6-12% apart, so rounding to
// nearest would drop nearly every change (simulated on normal gradients over
// 4,000 steps: s then settles at 0.38 of its true value; with stochastic
// rounding at 1.01 of it, with a spread of 15% between elements).  The random
// bits are a function of (seed, step, tensor, element) alone, so a step is
// reproducible bit for bit.
//
// Layout: codes in quads of 8 bytes, four of m then four of s, and the two
// exponent bytes (k + 127) of a block side by side.  A lane that owns four
// consecutive elements reads and writes one 8-byte word of codes, and eight
// lanes share a block.
#pragma once
#include "stream.h"

namespace zero_shard {
namespace {

constexpr int kBlock8 = 32;                      // elements per scale
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef short s16x2 __attribute__((ext_vector_type(2)));

// Pointers read from a table are generic ones to the compiler; naming the
// address space keeps the accesses global (flat ones count against the LDS
// too), and the table's own reads scalar.
#define ZS_GLOBAL __attribute__((address_space(1)))
#define ZS_CONSTANT __attribute__((address_space(4)))

template <typename T>
__device__ __forceinline__ ZS_GLOBAL T* global(T* p) {
    return (ZS_GLOBAL T*)p;
}

// fp32 and 16-bit vectors at the alignment of their element: tensors of a list
// may start anywhere.  The hardware takes 8- and 16-byte accesses at any
// address, so an aligned tensor costs nothing extra.
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));

__device__ __forceinline__ f32x4 ld_any(const float* p) {
    return __builtin_nontemporal_load((const ZS_GLOBAL f32x4_any*)p);
}
__device__ __forceinline__ u32x2 ld_any(const uint16_t* p) {
    return __builtin_nontemporal_load((const ZS_GLOBAL u32x2_any*)p);
}
__device__ __forceinline__ u32x4 ld16_any(const void* p) {
    return __builtin_nontemporal_load((const ZS_GLOBAL u32x4_any*)p);
}
__device__ __forceinline__ u32x2 ld_codes(const u32x2* p) {
    return __builtin_nontemporal_load((const ZS_GLOBAL u32x2*)p);
}
__device__ __forceinline__ void st_any(f32x4 v, float* p) {
    __builtin_nontemporal_store(v, (ZS_GLOBAL f32x4_any*)p);
}
__device__ __forceinline__ void st_any(u32x2 v, uint16_t* p) {
    __builtin_nontemporal_store(v, (ZS_GLOBAL u32x2_any*)p);
}
__device__ __forceinline__ void st_codes(u32x2 v, u32x2* p) { __builtin_nontemporal_store(v, (ZS_GLOBAL u32x2*)p); }

// One gradient value, and four consecutive ones as loaded and as values.
template <int DT>
__device__ __forceinline__ float ld_grad1(const void* G, int64_t e) {
    if constexpr (DT == ZERO_F32) {
        return global(static_cast<const float*>(G))[e];
    } else {
        const uint32_t h = global(static_cast<const uint16_t*>(G))[e];
        return DT == ZERO_F16 ? f16_to_f32(h) : bf16_to_f32(h);
    }
}

template <int DT>
struct Grad4 {
    u32x2 w;
    __device__ __forceinline__ void load(const void* G, int64_t e) { w = ld_any(static_cast<const uint16_t*>(G) + e); }
    __device__ __forceinline__ void values(float g[4]) const {
        unpack2<DT>(w[0], g[0], g[1]);
        unpack2<DT>(w[1], g[2], g[3]);
    }
};
template <>
struct Grad4<ZERO_F32> {
    f32x4 w;
    __device__ __forceinline__ void load(const void* G, int64_t e) { w = ld_any(static_cast<const float*>(G) + e); }
    __device__ __forceinline__ void values(float g[4]) const {
        for (int j = 0; j < 4; ++j) g[j] = w[j];
    }
};

template <int DT>
__device__ __forceinline__ u32x2 pack4_16(const float p[4]) {
    u32x2 o;
    o[0] = to16<DT>(p[0]) | (to16<DT>(p[1]) << 16);
    o[1] = to16<DT>(p[2]) | (to16<DT>(p[3]) << 16);
    return o;
}

// ---------------------------------------------------------------- random bits

// 32-bit key of one step: the seed and the step mixed by multiplication and
// shifts, modulo 2^64.  Host and device form it alike.
ZS_HD inline uint32_t dither_key(uint64_t seed, uint64_t step) {
    uint64_t k = seed * 0x9E3779B97F4A7C15ull + step * 0xBB67AE8584CAA73Bull;
    k ^= k >> 32;
    k *= 0x6A09E667F3BCC909ull;
    return (uint32_t)(k ^ (k >> 32));
}

// the key of one tensor of a list (0 for a shard) and the upper half of the element index
__device__ __forceinline__ uint32_t dither_tensor(uint32_t key, uint32_t tensor, int64_t e) {
    return key + tensor * 0x3C6EF373u + (uint32_t)(e >> 32) * 0xA54FF53Bu;
}

// 32 random bits of the element whose index has the lower half e: two rounds
// of multiply and shift (every input bit flips every output bit with
// probability 0.5 +- 0.01).  m takes the upper 20 bits of them, s those of the
// word rotated by half.
__device__ __forceinline__ uint32_t dither_bits(uint32_t e, uint32_t key) {
    uint32_t x = e ^ key;
    x ^= x >> 16;
    x *= 0x9E3779B9u;
    x ^= x >> 13;
    x *= 0xBB67AE85u;
    return x ^ (x >> 16);
}

__device__ __forceinline__ uint32_t rotate16(uint32_t x) { return (x << 16) | (x >> 16); }

// ---------------------------------------------------------------- codes

// The largest of 8 lanes' values (the lanes of one block), in all of them.
__device__ __forceinline__ uint32_t max_of_block(uint32_t x) {
    const auto other = [](uint32_t v, auto ctrl) {
        return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, decltype(ctrl)::value, 0xF, 0xF, true);
    };
    uint32_t y = other(x, std::integral_constant<int, 0xB1>{});      // lane ^ 1
    x = x > y ? x : y;
    y = other(x, std::integral_constant<int, 0x4E>{});               // lane ^ 2
    x = x > y ? x : y;
    y = other(x, std::integral_constant<int, 0x141>{});              // 7 - lane, within each 8
    return x > y ? x : y;
}

// Exponent byte (k + 127) of a block whose largest magnitude has these bits.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top_bits) {
    const uint32_t e = top_bits >> 23;
    return (e > 8u ? e : 8u) - 7u;
}

__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// four codes to float32, times the scale (exact)
__device__ __forceinline__ void decode4(uint32_t codes, float scale, float x[4]) {
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((int)codes, scale, false);
    const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((int)codes, scale, true);
    x[0] = a[0];
    x[1] = a[1];
    x[2] = b[0];
    x[3] = b[1];
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// a positive root is at least the smallest code
__device__ __forceinline__ float floor_root(float s, float smallest) {
    return (s > 0.0f && s < smallest) ? smallest : s;
}

// Four values to codes.  The conversion with random bits adds the upper 20 of
// them below the last place of the code (of the smallest code's place for
// values below the normal range) and truncates: checked on every exponent
// against that definition.
__device__ __forceinline__ uint32_t encode4_random(const float x[4], float scale, const uint32_t r[4]) {
    uint32_t w = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(0, x[0], r[0], scale, 0);
    w = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(w, x[1], r[1], scale, 1);
    w = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(w, x[2], r[2], scale, 2);
    return __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(w, x[3], r[3], scale, 3);
}

__device__ __forceinline__ uint32_t encode4_nearest(const float x[4], float scale) {
    s16x2 w = {0, 0};
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, x[0], x[1], scale, false);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, x[2], x[3], scale, true);
    return __builtin_bit_cast(uint32_t, w);
}

// Codes of a block whose largest magnitude lies in float32's last binade, or
// whose largest root lies in the last one whose squares are float32 numbers.
constexpr uint32_t kLastMean = 127 + 120, kLastRoot = 127 + 56;

// There code 256 (0x78) would stand for 2^128, or for a root whose square is
// 2^128: values that round to it take the code below, 240 (0x77).  NaN stays.
__device__ __forceinline__ uint32_t below_256(uint32_t codes) {
    const uint32_t top = codes & (codes >> 1) & (codes >> 2) & (codes >> 3) & ~(codes << 3) & 0x08080808u;
    return codes - (top >> 3);
}

__device__ __forceinline__ void hold_to_float32(u32x2& codes, uint32_t m_byte, uint32_t s_byte) {
    if (!__any(m_byte == kLastMean || s_byte == kLastRoot)) return;
    if (m_byte == kLastMean) codes[0] = below_256(codes[0]);
    if (s_byte == kLastRoot) codes[1] = below_256(codes[1]);
}

// ---------------------------------------------------------------- one task of the step

// Root and quotient, correctly rounded as sqrtf and / give them, without their
// scaling and special cases.  root_normal: for every v in [2^-96, FLT_MAX] (all
// 1.9e9 of them compared).  quotient_normal: where no step under- or overflows;
// Newton's step for the reciprocal and Markstein's correction of the quotient
// by its residual.  y is the correctly rounded reciprocal (all 2^23 mantissas
// compared), so a * y is off by at most 1.5 units in the last place.  The
// residual is an integer of up to 1.5 * 2^24 of its smallest units; beyond 2^24
// it may be rounded, by one.  Before its rounding the last step is then off by
// at most 3 / (2D) units for y's error and 2.01 / (2D) for the residual's, D
// being d's mantissa as an integer, and it can misround only a quotient that
// lies this close to the middle between two floats: all those within 64 / (2D)
// units of one (3.7e8) were compared.
__device__ __forceinline__ float root_normal(float v) {
    const float y = __builtin_amdgcn_rsqf(v);
    const float s = v * y;
    return fmaf(fmaf(-s, s, v), 0.5f * y, s);
}

__device__ __forceinline__ float reciprocal_normal(float d) {
    const float y = __builtin_amdgcn_rcpf(d);
    return fmaf(fmaf(-d, y, 1.0f), y, y);
}

__device__ __forceinline__ float quotient_normal(float a, float d) {
    const float y = reciprocal_normal(d);
    const float q = a * y;
    return fmaf(fmaf(-d, q, a), y, q);
}

__device__ __forceinline__ uint32_t min_of4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    const uint32_t x = a < b ? a : b, y = c < d ? c : d;
    return x < y ? x : y;
}

__device__ __forceinline__ uint32_t max_of4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    const uint32_t x = a > b ? a : b, y = c > d ? c : d;
    return x > y ? x : y;
}

// The block's largest magnitude (its bits) from each lane's four values.
__device__ __forceinline__ uint32_t top_of_block(const float x[4]) {
    return max_of_block(max_of4(abs_bits(x[0]), abs_bits(x[1]), abs_bits(x[2]), abs_bits(x[3])));
}

// Whether the float with these bits (sign clear) lies in [2^LO, 2^HI).
template <int LO, int HI>
__device__ __forceinline__ bool in_powers(uint32_t bits) {
    return bits - ((uint32_t)(LO + 127) << 23) < (uint32_t)(HI - LO) << 23;
}

// Whether a step's coefficients allow root_normal and quotient_normal for
// values in the ranges that adam8_four asks of its moments: then
// d = s * RB + eps lies in [2^-48, 2^46], the numerator in [2^-74, 2^50] and
// the quotient in [2^-120, 2^98], and the residuals' smallest units (2^-122 and
// up, 2^-144 for the root's) are float32 numbers.
__device__ __forceinline__ bool usual_coefficients(const StepCoef& c) {
    return in_powers<-24, 10>(__float_as_uint(c.step_size)) && in_powers<0, 12>(__float_as_uint(c.rsqrt_bc2)) &&
           __float_as_uint(c.eps) < (127u + 20u) << 23;
}

// What a lane reads of its four consecutive elements.
template <int GDT>
struct Quad8 {
    f32x4 p;
    u32x2 codes;
    Grad4<GDT> g;
    uint32_t scales;
    __device__ __forceinline__ void load(const float* P, const u32x2* C, const uint16_t* S, const void* G, int64_t e) {
        p = ld_any(P + e);
        codes = ld_codes(C + (e >> 2));
        g.load(G, e);
        scales = global(S)[e >> 5];
    }
};

// The step of four elements from e on, of which `here` exist (4 everywhere but
// at the tensor's end; the block's lanes all take part in its maxima).  The
// arithmetic of adam_elem on a decoded root; the new root, which the
// denominator needs, is what is stored.  A correctly rounded root and quotient
// are about a third of the instructions, and with 16 bytes an element the
// kernel is bound by those as much as by memory: a wave whose moments all lie
// in the usual range takes the short forms of both (same results).  251M
// elements, fp16: 0.630 ms; 0.662 with a zero moment in every wave, on the
// general forms.
__device__ __forceinline__ void adam8_four(const StepCoef& c, bool usual, float gscale, uint32_t key, int64_t e, int here,
                                           const float g[4], float p[4], u32x2& codes, uint32_t& scales) {
    float m[4], s[4], v[4];
    decode4(codes[0], scale_of(scales & 0xFFu), m);
    decode4(codes[1], scale_of(scales >> 8), s);
    uint32_t mb[4], r[4], q[4];
    for (int j = 0; j < 4; ++j) {
        const float gj = g[j] * gscale;
        m[j] = fmaf(c.beta1, m[j], c.omb1 * gj);
        v[j] = fmaf(c.beta2, s[j] * s[j], (c.omb2 * gj) * gj);
        if (j >= here) m[j] = v[j] = 0.0f;
        mb[j] = abs_bits(m[j]);
        r[j] = dither_bits((uint32_t)(e + j), key);
        q[j] = rotate16(r[j]);
    }
    const uint32_t m_top = max_of4(mb[0], mb[1], mb[2], mb[3]);
    const uint32_t v0 = __float_as_uint(v[0]), v1 = __float_as_uint(v[1]), v2 = __float_as_uint(v[2]),
                   v3 = __float_as_uint(v[3]);
    // below the sign bit the order of the bits is the order of the values; a NaN is above them all
    usual = usual && in_powers<-50, 40>(min_of4(mb[0], mb[1], mb[2], mb[3])) && in_powers<-50, 40>(m_top) &&
            in_powers<-96, 64>(min_of4(v0, v1, v2, v3)) && in_powers<-96, 64>(max_of4(v0, v1, v2, v3));
    usual = __all(usual);
    if (usual) {
        for (int j = 0; j < 4; ++j) {
            s[j] = root_normal(v[j]);
            p[j] = fmaf(p[j], c.decay, quotient_normal(-(c.step_size * m[j]), fmaf(s[j], c.rsqrt_bc2, c.eps)));
        }
    } else {
        for (int j = 0; j < 4; ++j) {
            s[j] = sqrtf(v[j]);
            p[j] = fmaf(p[j], c.decay, -(c.step_size * m[j]) / fmaf(s[j], c.rsqrt_bc2, c.eps));
        }
    }
    const uint32_t m_byte = scale_byte(max_of_block(m_top));
    const uint32_t s_byte = scale_byte(top_of_block(s));
    const float smallest = __builtin_ldexpf(scale_of(s_byte), -9);
    for (int j = 0; j < 4; ++j) s[j] = floor_root(s[j], smallest);
    codes[0] = encode4_random(m, scale_of(m_byte), r);
    codes[1] = encode4_random(s, scale_of(s_byte), q);
    if (!usual) hold_to_float32(codes, m_byte, s_byte);   // the usual range ends below
    scales = m_byte | (s_byte << 8);
}

// Elements [base, base + 256) of one tensor, base a multiple of 256, by one
// wave; lane l owns four consecutive elements.  The clip coefficient's float64
// arithmetic (about 30 dependent instructions) runs while the loads are on
// their way.  key: dither_tensor.  PDT 0: no 16-bit copy.
template <int GDT, int PDT>
__device__ __forceinline__ void adam8_task(float* P, u32x2* C, uint16_t* S, const void* G, uint16_t* Pout, int64_t n,
                                           int64_t base, const StepCoef& c, const double* d_sq, uint32_t key) {
    const int lane = threadIdx.x;
    const int64_t e = base + 4 * lane;
    const bool usual = usual_coefficients(c);
    float p[4] = {}, g[4] = {};
    if (base + kTask <= n) {
        Quad8<GDT> quad;
        quad.load(P, C, S, G, e);
        const float gscale = clipped_scale(c, d_sq);
        quad.g.values(g);
        for (int j = 0; j < 4; ++j) p[j] = quad.p[j];
        adam8_four(c, usual, gscale, key, e, 4, g, p, quad.codes, quad.scales);
        const f32x4 v = {p[0], p[1], p[2], p[3]};
        st_any(v, P + e);
        st_codes(quad.codes, C + (e >> 2));
        if constexpr (PDT != 0) st_any(pack4_16<PDT>(p), Pout + e);
        if ((lane & 7) == 0) global(S)[e >> 5] = (uint16_t)quad.scales;
        return;
    }
    const int here = e >= n ? 0 : n - e < 4 ? (int)(n - e) : 4;
    u32x2 codes = {0, 0};
    uint32_t scales = 0;
    if (here > 0) {
        codes = ld_codes(C + (e >> 2));
        scales = global(S)[e >> 5];
    }
    for (int j = 0; j < 4; ++j) {
        if (j >= here) continue;
        p[j] = global(P)[e + j];
        g[j] = ld_grad1<GDT>(G, e + j);
    }
    adam8_four(c, usual, clipped_scale(c, d_sq), key, e, here, g, p, codes, scales);
    if (here > 0) {
        st_codes(codes, C + (e >> 2));
        if ((lane & 7) == 0) global(S)[e >> 5] = (uint16_t)scales;
    }
    for (int j = 0; j < 4; ++j) {
        if (j >= here) continue;
        global(P)[e + j] = p[j];
        if constexpr (PDT != 0) global(Pout)[e + j] = (uint16_t)to16<PDT>(p[j]);
    }
}

}  // namespace
}  // namespace zero_shard
