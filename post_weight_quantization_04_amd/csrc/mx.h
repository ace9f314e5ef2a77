// Device helpers of the MX formats: rounding to their grids, and the epilogue
// of the products with MX weights.
#pragma once

#include "fused.h"

namespace gptq {

// The value in fp32 with its last bit set where the conversion drops
// something (round to odd): rounding it again to a few bits gives what rounding
// the 64-bit value once would.  Values beyond fp32's range become infinite.
__device__ __forceinline__ float mx_odd(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    // 20 mantissa bits stay, any bit below them goes into the last: exact in fp32
    const uint64_t hi = (b >> 32) | ((uint32_t)b != 0u);
    return (float)__builtin_bit_cast(double, hi << 32);
}

// The scale byte of a block from the bits of its largest magnitude: the
// exponent floor(log2 max) - emax, at least -127, biased by 127; 255 where a
// value is not finite.
template <int FMT>
__device__ __forceinline__ unsigned mx_scale_byte(unsigned max_bits) {
    const int field = (int)(max_bits >> 23) - (FMT == MX_FP4 ? 2 : 8);
    return max_bits >= 0x7f800000u ? 255u : (unsigned)max(field, 0);
}
// Eight values of a block of that scale as codes: one word of e2m1, two of
// e4m3; rounded to nearest even, saturated at 6 and 448.  v 2^-E is exact in
// fp32 but where it is far below the smallest code.  The conversion to e2m1
// saturates by itself, the one to e4m3 does not.
template <int FMT>
__device__ __forceinline__ u32x2 mx_codes8(const float (&v)[8], unsigned byte) {
    u32x2 c = {0u, 0u};
    if (byte == 255u) return c;
    const float f = __builtin_bit_cast(float, (254u - byte) << 23);   // 2^(127 - byte)
    if constexpr (FMT == MX_FP4) {
        c[0] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c[0], v[0] * f, v[1] * f, 1.f, 0);
        c[0] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c[0], v[2] * f, v[3] * f, 1.f, 1);
        c[0] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c[0], v[4] * f, v[5] * f, 1.f, 2);
        c[0] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c[0], v[6] * f, v[7] * f, 1.f, 3);
    } else {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = __builtin_amdgcn_fmed3f(v[e] * f, -448.f, 448.f);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            int w = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * h], x[4 * h + 1], 0, false);
            c[h] = (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(x[4 * h + 2], x[4 * h + 3], w, true);
        }
    }
    return c;
}
// A lane's eight values (columns 8 piece ..) quantized with the other lanes of
// its block (four neighbours, all active) and stored.
template <int FMT>
__device__ __forceinline__ void mx_put8(const float (&v)[8], int64_t rows, int64_t row, int64_t piece,
                                        int64_t row_bytes, uint8_t *codes, uint8_t *scales) {
    unsigned top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __builtin_bit_cast(unsigned, v[e]) & 0x7fffffffu);
    top = max(top, (unsigned)__shfl_xor((int)top, 1));
    top = max(top, (unsigned)__shfl_xor((int)top, 2));
    const unsigned byte = mx_scale_byte<FMT>(top);
    const u32x2 c = mx_codes8<FMT>(v, byte);
    uint8_t *out = codes + row * row_bytes + piece * (FMT == MX_FP4 ? 4 : 8);
    if constexpr (FMT == MX_FP4)
        *(unsigned *)out = c[0];
    else
        *(u32x2 *)out = c;
    if ((piece & 3) == 0) scales[((piece >> 4) * rows + row) * 4 + ((piece >> 2) & 3)] = (uint8_t)byte;
}

// eight values of a row from column k on, zeros past its end
__device__ __forceinline__ void mx_ld8(const void *x, int64_t row, int64_t d, int64_t k, int bf16, int vec,
                                       float (&v)[8]) {
    if (k >= d) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.f;
    } else if (vec) {
        fz_ld8(x, row * d + k, bf16, v);
    } else {   // (clamped and selected: a branch around each load would wait for each)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = fz_ld(x, row * d + std::min(k + e, d - 1), bf16);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = k + e < d ? v[e] : 0.f;
    }
}

// The epilogue of the products: bias, the pre-activation kept, activation,
// residual.
struct MxEpilogue {
    int64_t n;                  // outputs per row
    const void *bias;
    int bias_bf16, act;
    const void *residual;
    void *Y, *pre;
    int out_bf16;
    int width;                  // consecutive outputs that load and store together: 8, 4 or 1
};
// R rows (those below m) of eight outputs from column n, inside the row, on:
// their sums z become the outputs.  Loads first, so that they overlap.
template <int R>
__device__ __forceinline__ void mx_epilogue(const MxEpilogue &p, int64_t m, const int64_t (&row)[R], int64_t n,
                                            const float (&bias)[8], float (&z)[R][8]) {
    float res[R][8];
    if (p.residual) {
#pragma unroll
        for (int r = 0; r < R; ++r)
            fz_ld_row8(p.residual, std::min(row[r], m - 1) * p.n + n, n, p.n, p.out_bf16, p.width, res[r]);
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int e = 0; e < 8; ++e) z[r][e] += bias[e];
    if (p.pre) {
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (row[r] < m) fz_st_row8(p.pre, row[r] * p.n + n, n, p.n, p.out_bf16, p.width, z[r]);
    }
    fz_with_act(p.act, [&](auto act) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int e = 0; e < 8; ++e) z[r][e] = fz_act<decltype(act)::value>(z[r][e]);
    });
    if (p.residual) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int e = 0; e < 8; ++e) z[r][e] += res[r][e];
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (row[r] < m) fz_st_row8(p.Y, row[r] * p.n + n, n, p.n, p.out_bf16, p.width, z[r]);
}
__device__ __forceinline__ void mx_bias8(const MxEpilogue &p, int64_t n, float (&b)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) b[e] = 0.f;
    if (p.bias) fz_ld_row8(p.bias, n, n, p.n, p.bias_bf16, p.width, b);
}

// the products' forms
MxEpilogue mx_epilogue_of(const MxLinear &a);
bool mx_skinny_takes(int64_t m, int64_t d_out, int64_t d_in, int kind);
hipError_t mx_skinny_launch(const MxLinear &a, hipStream_t st);
bool mx_skinny_backward_takes(const FusedShape &s, int act);
size_t mx_skinny_backward_ws(const FusedShape &s);
hipError_t mx_skinny_backward_launch(const FusedBackward &a, hipStream_t st);
size_t mx_gemm_ws(int64_t m, int64_t d_out, int64_t d_in);
hipError_t mx_gemm_launch(const MxLinear &a, hipStream_t st);

}  // namespace gptq
