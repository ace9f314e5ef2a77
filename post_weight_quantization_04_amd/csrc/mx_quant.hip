// MX formats (OCP Microscaling Formats, version 1.0): matrices in blocks of 32
// columns that share a power of two,
//   x ~ 2^E c,  E = clamp(floor(log2 max |x|) - emax, -127, 127),
// with elements c in e2m1 (emax 2) or e4m3 (emax 8), rounded to nearest even
// and saturated.  "Optimization Gptq", "Configuracoes de quantizacao" (low-bit
// weights in groups): the group's range as a power of two instead of an fp32
// scale and zero point, which the matrix cores apply by themselves.
//
// Both directions are bound by memory.  A lane takes eight columns, four lanes
// a block, a wave four pieces of 512 columns of one row, so that four loads of
// each lane are in flight; of rows up to 256 columns wide, several at a time.
#include "mx.h"

#include <algorithm>

namespace gptq {

namespace {

constexpr int QC = 4, QCOLS = QC * 512;   // pieces, and columns, of a wave

// The units of work of the waves: QC pieces of a row, or of 64 >> shift rows
// with 1 << shift lanes each
struct Units {
    int64_t chunks, units;      // a row's waves, all waves
    int shift;                  // 4 or 5: narrow rows; 0: not
    __device__ __forceinline__ void at(int64_t u, int c, int64_t &row, int64_t &k) const {
        const int lane = threadIdx.x & 63;
        if (shift) {
            row = ((u * QC + c) << (6 - shift)) + (lane >> shift);
            k = 8 * (lane & ((1 << shift) - 1));
        } else {
            row = u / chunks;
            k = (u - row * chunks) * QCOLS + 512 * c + 8 * lane;
        }
    }
};
Units units_of(int64_t rows, int64_t d) {
    Units u{};
    const int64_t steps = mx_steps(d);
    u.shift = steps == 1 ? 4 : (steps == 2 ? 5 : 0);
    u.chunks = cdiv(steps * MX_PAD, QCOLS);
    u.units = u.shift ? cdiv(rows, (int64_t)QC << (6 - u.shift)) : rows * u.chunks;
    return u;
}

struct QuantMx {
    const void *X;
    int bf16, vec;
    int64_t rows, d, steps, row_bytes;
    uint8_t *codes, *scales;
    Units w;
};

template <int FMT, bool VEC>
__global__ __launch_bounds__(256) void mx_quantize_kernel(QuantMx p) {
    p.vec = VEC;   // (known here: the other way of loading costs registers)
    for (int64_t u = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); u < p.w.units; u += (int64_t)gridDim.x * 4) {
        int64_t row[QC], k[QC];
        float v[QC][8];
#pragma unroll
        for (int c = 0; c < QC; ++c) {
            p.w.at(u, c, row[c], k[c]);
            mx_ld8(p.X, row[c], p.d, row[c] < p.rows ? k[c] : p.d, p.bf16, p.vec, v[c]);
        }
#pragma unroll
        for (int c = 0; c < QC; ++c)
            // (a block's four lanes are inside or outside together)
            if (row[c] < p.rows && k[c] < p.steps * MX_PAD)
                mx_put8<FMT>(v[c], p.rows, row[c], k[c] >> 3, p.row_bytes, p.codes, p.scales);
    }
}

struct DequantMx {
    MxMatrix x;
    int64_t rows, d, row_bytes;
    void *Y;
    int bf16, vec;
    Units w;
};

template <int FMT>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(DequantMx p) {
    for (int64_t u = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); u < p.w.units; u += (int64_t)gridDim.x * 4) {
        int64_t at[QC], k[QC];
        u32x2 w[QC];
        unsigned byte[QC];
#pragma unroll
        for (int c = 0; c < QC; ++c) {
            p.w.at(u, c, at[c], k[c]);
            const int64_t row = at[c], piece = k[c] >> 3;
            w[c] = u32x2{0u, 0u};
            byte[c] = 0;
            if (row < p.rows && k[c] < p.d) {
                const uint8_t *in = p.x.codes + row * p.row_bytes + piece * (FMT == MX_FP4 ? 4 : 8);
                if constexpr (FMT == MX_FP4)
                    w[c][0] = *(const unsigned *)in;
                else
                    w[c] = *(const u32x2 *)in;
                byte[c] = p.x.scales[((piece >> 4) * p.rows + row) * 4 + ((piece >> 2) & 3)];
            }
        }
#pragma unroll
        for (int c = 0; c < QC; ++c) {
            if (at[c] >= p.rows || k[c] >= p.d) continue;
            float v[8];
            if constexpr (FMT == MX_FP4) {
                // (the conversion reads the scale's exponent bits: 0 is 2^-127, 255 NaN)
                const float s = __builtin_bit_cast(float, byte[c] << 23);
                typedef __attribute__((ext_vector_type(2))) float f32x2;
                f32x2 x[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[c][0], s, 0),
                              __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[c][0], s, 1),
                              __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[c][0], s, 2),
                              __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[c][0], s, 3)};
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = x[e >> 1][e & 1];
            } else {
                const int e2 = byte[c] == 255u ? 0 : (int)byte[c] - 127;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    v[4 * h] = __builtin_amdgcn_cvt_f32_fp8((int)w[c][h], 0);
                    v[4 * h + 1] = __builtin_amdgcn_cvt_f32_fp8((int)w[c][h], 1);
                    v[4 * h + 2] = __builtin_amdgcn_cvt_f32_fp8((int)w[c][h], 2);
                    v[4 * h + 3] = __builtin_amdgcn_cvt_f32_fp8((int)w[c][h], 3);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = byte[c] == 255u ? __builtin_nanf("") : fz_ldexp(v[e], e2);
            }
            const int64_t o = at[c] * p.d + k[c];
            if (p.vec) {
                fz_st8(p.Y, o, p.bf16, v);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (k[c] + e < p.d) fz_st(p.Y, o + e, v[e], p.bf16);
            }
        }
    }
}

bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
unsigned wave_blocks(int64_t units) { return (unsigned)std::min<int64_t>(cdiv(units, 4), (int64_t)1 << 22); }

}  // namespace

hipError_t mx_quantize_launch(const void *X, int x_bf16, int64_t rows, int64_t d, int fmt, uint8_t *codes,
                              uint8_t *scales, hipStream_t st) {
    QuantMx p{};
    p.X = X;
    p.bf16 = x_bf16;
    p.vec = d % 8 == 0 && aligned16(X);
    p.rows = rows;
    p.d = d;
    p.steps = mx_steps(d);
    p.row_bytes = mx_row_bytes(d, fmt);
    p.codes = codes;
    p.scales = scales;
    p.w = units_of(rows, d);
    const unsigned blocks = wave_blocks(p.w.units);
    if (fmt == MX_FP4 && p.vec)
        mx_quantize_kernel<MX_FP4, true><<<blocks, 256, 0, st>>>(p);
    else if (fmt == MX_FP4)
        mx_quantize_kernel<MX_FP4, false><<<blocks, 256, 0, st>>>(p);
    else if (p.vec)
        mx_quantize_kernel<MX_FP8, true><<<blocks, 256, 0, st>>>(p);
    else
        mx_quantize_kernel<MX_FP8, false><<<blocks, 256, 0, st>>>(p);
    return hipGetLastError();
}

hipError_t mx_dequantize_launch(const MxMatrix &x, int64_t rows, int64_t d, void *Y, int y_bf16, hipStream_t st) {
    DequantMx p{};
    p.x = x;
    p.rows = rows;
    p.d = d;
    p.row_bytes = mx_row_bytes(d, x.fmt);
    p.Y = Y;
    p.bf16 = y_bf16;
    p.vec = d % 8 == 0 && aligned16(Y);
    p.w = units_of(rows, d);
    if (x.fmt == MX_FP4)
        mx_dequantize_kernel<MX_FP4><<<wave_blocks(p.w.units), 256, 0, st>>>(p);
    else
        mx_dequantize_kernel<MX_FP8><<<wave_blocks(p.w.units), 256, 0, st>>>(p);
    return hipGetLastError();
}

}  // namespace gptq
