// Device helpers and internal entry points of the fused products with packed
// layers (fused.hip, fused_gemm.hip, fused_skinny.hip).
#pragma once

#include "common.h"

namespace gptq {

typedef __attribute__((ext_vector_type(4))) int i32x4;
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;
typedef __attribute__((ext_vector_type(2))) __bf16 fz_bf16x2;

__device__ __forceinline__ float fz_bf16(uint16_t b) { return __builtin_bit_cast(float, (unsigned)b << 16); }
__device__ __forceinline__ uint16_t fz_to_bf16(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }   // RNE
__device__ __forceinline__ float fz_ld(const void *p, int64_t i, int bf16) {
    return bf16 ? fz_bf16(((const uint16_t *)p)[i]) : ((const float *)p)[i];
}
__device__ __forceinline__ void fz_st(void *p, int64_t i, float v, int bf16) {
    if (bf16)
        ((uint16_t *)p)[i] = fz_to_bf16(v);
    else
        ((float *)p)[i] = v;
}
// four consecutive values of an operand whose element 0 is aligned to four
__device__ __forceinline__ f32x4 fz_ld4(const void *p, int64_t i, int bf16) {
    if (!bf16) return *(const f32x4 *)((const float *)p + i);
    const u32x2 u = *(const u32x2 *)((const uint16_t *)p + i);
    return f32x4{__builtin_bit_cast(float, u[0] << 16), __builtin_bit_cast(float, u[0] & 0xffff0000u),
                 __builtin_bit_cast(float, u[1] << 16), __builtin_bit_cast(float, u[1] & 0xffff0000u)};
}
// eight consecutive values, element 0 aligned to eight
__device__ __forceinline__ void fz_ld8(const void *p, int64_t i, int bf16, float (&v)[8]) {
    if (bf16) {
        const u32x4 u = *(const u32x4 *)((const uint16_t *)p + i);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = __builtin_bit_cast(float, u[e] << 16);
            v[2 * e + 1] = __builtin_bit_cast(float, u[e] & 0xffff0000u);
        }
    } else {
        const f32x4 a = *(const f32x4 *)((const float *)p + i), b = *(const f32x4 *)((const float *)p + i + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] = a[e];
            v[4 + e] = b[e];
        }
    }
}
// k / g for k < 2^24, with inv = 1.f / g
__device__ __forceinline__ int fz_div(int k, int g, float inv) {
    int q = (int)((float)k * inv);
    q -= q * g > k;
    return q + ((q + 1) * g <= k);
}
__device__ __forceinline__ unsigned fz_pack_bf16(float a, float b) {
    const fz_bf16x2 p = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(unsigned, p);
}
__device__ __forceinline__ void fz_st4(void *p, int64_t i, f32x4 v, int bf16) {
    if (bf16)
        *(u32x2 *)((uint16_t *)p + i) = u32x2{fz_pack_bf16(v[0], v[1]), fz_pack_bf16(v[2], v[3])};
    else
        *(f32x4 *)((float *)p + i) = v;
}

// eight values to an aligned place
__device__ __forceinline__ void fz_st8(void *x, int64_t o, int bf16, const float (&v)[8]) {
    if (bf16) {
        *(u32x4 *)((uint16_t *)x + o) = u32x4{fz_pack_bf16(v[0], v[1]), fz_pack_bf16(v[2], v[3]),
                                              fz_pack_bf16(v[4], v[5]), fz_pack_bf16(v[6], v[7])};
    } else {
        fz_st4(x, o, f32x4{v[0], v[1], v[2], v[3]}, 0);
        fz_st4(x, o + 4, f32x4{v[4], v[5], v[6], v[7]}, 0);
    }
}
// eight values from column n of a row (offset o) on, `width` at a time, those
// inside n_all (as n itself is)
__device__ __forceinline__ void fz_ld_row8(const void *x, int64_t o, int64_t n, int64_t n_all, int bf16, int width,
                                           float (&v)[8]) {
    if (width == 8) {
        fz_ld8(x, o, bf16, v);
    } else if (width == 4) {
        const bool more = n + 4 < n_all;
        const f32x4 a = fz_ld4(x, o, bf16), b = fz_ld4(x, more ? o + 4 : o, bf16);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] = a[e];
            v[4 + e] = b[e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = fz_ld(x, n + e < n_all ? o + e : o, bf16);
    }
}
__device__ __forceinline__ void fz_st_row8(void *x, int64_t o, int64_t n, int64_t n_all, int bf16, int width,
                                           const float (&v)[8]) {
    if (width == 8) {
        fz_st8(x, o, bf16, v);
    } else if (width == 4) {
        fz_st4(x, o, f32x4{v[0], v[1], v[2], v[3]}, bf16);
        if (n + 4 < n_all) fz_st4(x, o + 4, f32x4{v[4], v[5], v[6], v[7]}, bf16);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (n + e < n_all) fz_st(x, o + e, v[e], bf16);
    }
}

// The factor 2^t that brings v, positive and finite, to [2^14, 2^15) (f16's
// range), and the exponent -t that undoes it; 1 and 0 for 0.  A sum of scaled
// products returns by ldexpf with both operands' exponents added: the sums are
// of order 2^32, the exponents up to 126 each, and one factor at a time would
// overflow (or vanish) on the way to results that fp32 holds.
__device__ __forceinline__ void fz_pow2_scale(float v, float &mul, int &undo) {
    int e = (int)((__builtin_bit_cast(unsigned, v) >> 23) & 255u) - 127;   // (subnormals: -127)
    if (v == 0.f) e = 14;
    undo = max(-126, min(126, e - 14));
    mul = __builtin_bit_cast(float, (unsigned)(127 - undo) << 23);
}
__device__ __forceinline__ float fz_ldexp(float v, int e) { return __builtin_amdgcn_ldexpf(v, e); }

// ---------------------------------------------------------------------------
// activations and their slopes (fp32)
// ---------------------------------------------------------------------------
constexpr float FZ_SQRT_HALF = 0.70710678118654752f, FZ_INV_SQRT_2PI = 0.39894228040143268f;
constexpr float FZ_TWO_SQRT_2_PI = 1.5957691216057308f;   // 2 sqrt(2 / pi)

// p = sigmoid(x) and q = sigmoid(-x) from one exponential of -|x|: no
// cancellation on either side, a few fp32 steps of error for moderate x (the
// exponent's product is rounded: |x| 2^-24 relative).  The library's expf and
// divide took the gated pair's dZ pass (45 M elements) 180 us.
__device__ __forceinline__ void fz_sigmoids(float x, float &p, float &q) {
    const float e = __builtin_amdgcn_exp2f(-1.44269504088896341f * fabsf(x));
    const float r = __builtin_amdgcn_rcpf(1.f + e), s = e * r;
    p = x < 0.f ? s : r;   // (NaN: both NaN)
    q = x < 0.f ? r : s;
}

template <int ACT>
__device__ __forceinline__ float fz_act(float z) {
    float p, q;
    if constexpr (ACT == 1) return z < 0.f ? 0.f : z;   // NaN stays NaN
    if constexpr (ACT == 2) return 0.5f * z * erfcf(-z * FZ_SQRT_HALF);
    if constexpr (ACT == 3) {
        fz_sigmoids(FZ_TWO_SQRT_2_PI * (z + 0.044715f * z * z * z), p, q);
        return z * p;
    }
    if constexpr (ACT == 4) {
        fz_sigmoids(z, p, q);
        return z * p;
    }
    return z;
}

// (beyond |z| = 128 every slope is 0 or 1 in fp32, silu's, the slowest to
// vanish, from -108 on: clamped there, so that no product of a vanishing and an
// overflowing factor arises; NaN stays NaN)
template <int ACT>
__device__ __forceinline__ float fz_slope(float z) {
    float p, q;
    z = z > 128.f ? 128.f : (z < -128.f ? -128.f : z);
    if constexpr (ACT == 1) return z > 0.f ? 1.f : 0.f;
    if constexpr (ACT == 2)
        return 0.5f * erfcf(-z * FZ_SQRT_HALF) +
               z * FZ_INV_SQRT_2PI * __builtin_amdgcn_exp2f(-0.72134752044448170f * z * z);
    if constexpr (ACT == 3) {
        fz_sigmoids(FZ_TWO_SQRT_2_PI * (z + 0.044715f * z * z * z), p, q);
        return p + z * p * q * FZ_TWO_SQRT_2_PI * (1.f + 3.f * 0.044715f * z * z);
    }
    if constexpr (ACT == 4) {
        fz_sigmoids(z, p, q);
        return p + z * p * q;
    }
    return 1.f;
}

// A gate's gradient d u act'(z): the slope first, which is below 1.13, as d u
// can overflow where the slope brings it back (or is 0)
template <int ACT>
__device__ __forceinline__ float fz_gate_grad(float d, float u, float z) {
    return d * fz_slope<ACT>(z) * u;
}

// f(std::integral_constant<int, act>) for a run-time activation
template <class F>
__host__ __device__ __forceinline__ void fz_with_act(int act, F f) {
    switch (act) {
        case 1: f(std::integral_constant<int, 1>{}); break;
        case 2: f(std::integral_constant<int, 2>{}); break;
        case 3: f(std::integral_constant<int, 3>{}); break;
        case 4: f(std::integral_constant<int, 4>{}); break;
        default: f(std::integral_constant<int, 0>{}); break;
    }
}

// The eight codes k0 .. k0 + 7 (k0 % 8 == 0) of a row lie in the word (bits
// k0) / 32 and, for 3 and 8 bits, the next one, from bit (bits k0) % 32 of the
// first on.  fz_codes8 moves them to bit 0 of one word (two for 8 bits).
template <int BITS>
constexpr bool fz_two_words() { return BITS == 3 || BITS == 8; }
template <int BITS>
struct Codes8 {
    unsigned w[BITS == 8 ? 2 : 1];
    // code e as fp32
    __device__ __forceinline__ float at(int e) const {
        if constexpr (BITS == 8) return (float)((w[e >> 2] >> (8 * (e & 3))) & 255u);
        // two shared shifts and masks, then byte conversions
        if constexpr (BITS == 4) {
            const unsigned half = (e & 1) ? (w[0] >> 4) & 0x0f0f0f0fu : w[0] & 0x0f0f0f0fu;
            return (float)((half >> (8 * (e >> 1))) & 255u);
        }
        return (float)__builtin_amdgcn_ubfe(w[0], BITS * e, BITS);
    }
};
template <int BITS>
__device__ __forceinline__ Codes8<BITS> fz_codes8(unsigned lo, unsigned hi, int sh) {
    Codes8<BITS> c;
    if constexpr (BITS == 8) {
        c.w[0] = lo;
        c.w[BITS == 8 ? 1 : 0] = hi;
    } else if constexpr (BITS == 3) {
        c.w[0] = __builtin_amdgcn_alignbit(hi, lo, sh);
    } else {
        c.w[0] = BITS == 4 ? lo : lo >> sh;
    }
    return c;
}

// ---------------------------------------------------------------------------
// LDS stages filled by buffer loads
// ---------------------------------------------------------------------------
typedef __attribute__((address_space(3))) void gm_lds_void;

template <int N>
__device__ __forceinline__ void gm_wait() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory"); }
// barrier without the fence of __syncthreads(), which would wait for every
// stage in flight; this wave's LDS reads are drained first
__device__ __forceinline__ void gm_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}
// buffer resource over [p, p + bytes), base and size in scalar registers
__device__ __forceinline__ __amdgpu_buffer_rsrc_t gm_rsrc(const void *p, int64_t bytes) {
    const uint64_t b = reinterpret_cast<uint64_t>(p);
    const uint64_t bu = ((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((unsigned)(b >> 32)) << 32) |
                        (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((unsigned)b);
    const int n = __builtin_amdgcn_readfirstlane((int)std::min<int64_t>(std::max<int64_t>(bytes, 0), (int64_t)0x7fffffff));
    return __builtin_amdgcn_make_buffer_rsrc((void *)bu, (short)0, n, 0x00020000);
}

// ---------------------------------------------------------------------------
// dense form (fused_gemm.hip)
// ---------------------------------------------------------------------------
size_t dense_forward_ws(const FusedShape &s);
size_t dense_backward_ws(const FusedShape &s);
hipError_t dense_forward_launch(const FusedForward &a, hipStream_t st);
hipError_t dense_backward_launch(const FusedBackward &a, hipStream_t st);

// ---------------------------------------------------------------------------
// packed form (fused_skinny.hip)
// ---------------------------------------------------------------------------
bool skinny_forward_takes(const FusedShape &s);
size_t skinny_forward_ws(const FusedShape &s);
hipError_t skinny_forward_launch(const FusedForward &a, hipStream_t st);
bool skinny_backward_takes(const FusedShape &s);
size_t skinny_backward_ws(const FusedShape &s);
hipError_t skinny_backward_launch(const FusedBackward &a, hipStream_t st);

}  // namespace gptq
