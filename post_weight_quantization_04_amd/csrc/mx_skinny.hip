// Products with MX weights in 4 bits, few activation rows (decoding): bound by
// reading the weights once.
//
// A work group takes 16 outputs, its eight waves share the contraction in steps
// of 128 columns, and each step is one 16-byte load of a lane: block g = lane / 16
// of weight row lane % 16, which is how the matrix cores take an e2m1 operand.
//   fp8 / fp4 activations   one scaled MFMA (16 x 16 x 128) per 16 rows and
//                           step, on the codes and scale bytes as they lie
//   bf16 / fp32             the codes become bf16, exactly, with their scale in
//                           one conversion; four bf16 MFMAs (16 x 16 x 32), the
//                           i-th on the i-th word of every lane's block (both
//                           operands take the contraction in that order).  fp32
//                           activations are cut into three bf16 terms (8 bits
//                           each, together all 24): three times the MFMAs.
//   fp8, F32 results        activations and weights both as bf16, exactly: the
//                           scaled MFMA adds the products of e4m3 operands with
//                           about 14 bits below the largest (see mx_gemm.hip)
// The waves' sums meet in LDS and are added in their order.
#include "mx.h"

namespace gptq {

namespace {

constexpr int SK_WAVES = 8, SK_UNROLL = 4;

struct SkinnyArgs {
    int64_t m, d_out, d_in;
    int steps;
    const void *A;
    MxMatrix a, w;
    int64_t w_bytes, a_bytes;   // code bytes of a row
    int vec;                    // A: whole aligned pieces of eight
    MxEpilogue out;
};

typedef __attribute__((ext_vector_type(8))) int i32x8;

// eight values of activation row `row`, columns k .., as they lie in memory
// (BYTES 2 or 4 each); zeros past the end
template <int BYTES>
__device__ __forceinline__ void act_raw(const SkinnyArgs &p, int64_t row, int64_t k, u32x4 *out) {
    const char *a = (const char *)p.A + row * p.d_in * BYTES;
    if (p.vec) {
        const bool in = k < p.d_in;
#pragma unroll
        for (int i = 0; i < BYTES / 2; ++i) {
            const u32x4 u = *(const u32x4 *)(a + (in ? k : 0) * BYTES + 16 * i);
            out[i] = in ? u : u32x4{0u, 0u, 0u, 0u};
        }
    } else {   // (clamped and selected: a branch around each load would wait for each)
        unsigned v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int64_t at = std::min(k + e, p.d_in - 1);
            if constexpr (BYTES == 2)
                v[e] = ((const uint16_t *)a)[at];
            else
                v[e] = ((const unsigned *)a)[at];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = k + e < p.d_in ? v[e] : 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (BYTES == 2) {
                out[0][i] = v[2 * i] | v[2 * i + 1] << 16;
            } else {
                out[0][i] = v[i];
                out[BYTES / 2 - 1][i] = v[4 + i];
            }
        }
    }
}
// fp32 values as N bf16 terms, each the leading bits of what is left (truncated,
// so that no term overflows; the last of two rounded to nearest); infinities
// and NaN in the first alone
template <int N>
__device__ __forceinline__ void bf16_terms(const float (&v)[8], bf16x8 (&t)[N]) {
    u32x4 u[N] = {};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const unsigned b = __builtin_bit_cast(unsigned, v[e]), mag = b & 0x7fffffffu;
        const bool finite = mag < 0x7f800000u;
        const unsigned hi = (b & 0xffff0000u) | (mag > 0x7f800000u ? 0x400000u : 0u);
        const float r1 = finite ? v[e] - __builtin_bit_cast(float, hi) : 0.f;
        u[0][e >> 1] |= (e & 1) ? hi : hi >> 16;
        if constexpr (N == 2) u[1][e >> 1] |= (unsigned)fz_to_bf16(r1) << (16 * (e & 1));
        if constexpr (N == 3) {
            const unsigned mid = __builtin_bit_cast(unsigned, r1) & 0xffff0000u;
            const float r2 = r1 - __builtin_bit_cast(float, mid);
            const unsigned lo = __builtin_bit_cast(unsigned, r2);
            u[1][e >> 1] |= (e & 1) ? mid : mid >> 16;
            u[N - 1][e >> 1] |= (e & 1) ? lo & 0xffff0000u : lo >> 16;
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) t[i] = __builtin_bit_cast(bf16x8, u[i]);
}
// a word's eight codes times 2^(scale byte - 127)
__device__ __forceinline__ bf16x8 codes_bf16(unsigned w, float scale) {
    const unsigned u[4] = {__builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0)),
                           __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1)),
                           __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2)),
                           __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3))};
    return __builtin_bit_cast(bf16x8, u32x4{u[0], u[1], u[2], u[3]});
}

// eight e4m3 codes of a block times its scale
__device__ __forceinline__ bf16x8 codes8_bf16(u32x2 w, float scale) {
    const unsigned u[4] = {__builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[0], scale, false)),
                           __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[0], scale, true)),
                           __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[1], scale, false)),
                           __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[1], scale, true))};
    return __builtin_bit_cast(bf16x8, u32x4{u[0], u[1], u[2], u[3]});
}

// KIND: of the activations (MX_WIDE_FP8: fp8 as bf16); MT: their 16-row tiles
template <int KIND, int MT>
__global__ __launch_bounds__(64 * SK_WAVES) void mx_skinny_kernel(SkinnyArgs p) {
    __shared__ f32x4 lds[SK_WAVES][MT][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    // (rows past the ends: the last ones again, whose results are not stored)
    const int64_t wrow = std::min<int64_t>(n0 + r, p.d_out - 1);
    const uint8_t *wc = p.w.codes + wrow * p.w_bytes + 16 * g;
    const unsigned *wsc = (const unsigned *)p.w.scales + wrow;
    int64_t arow[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) arow[t] = std::min<int64_t>(16 * t + r, p.m - 1);
    f32x4 acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};

    // A step's work in units of whole operands: the activations of one are loaded
    // beside the products of the one before it.
    constexpr bool MX = KIND == MX_FP8 || KIND == MX_FP4, SCALED = MX || KIND == MX_WIDE_FP8;
    constexpr int UNITS = MX ? 1 : 2;
    constexpr int RAW = KIND == MX_ACT_F32 ? 4 : (KIND == MX_ACT_BF16 || KIND == MX_FP8 ? 2 : 1);
    struct Acts {
        u32x4 x[MT][RAW];
        unsigned sc[MT];
    };
    auto load = [&](int s, int unit, Acts &a) {
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            if constexpr (SCALED) {
                const uint8_t *c = p.a.codes + arow[t] * p.a_bytes;
                a.sc[t] = ((const unsigned *)p.a.scales)[s * p.m + arow[t]];
                if constexpr (KIND == MX_FP4) {
                    a.x[t][0] = *(const u32x4 *)(c + (int64_t)s * (MX_PAD / 2) + 16 * g);
                } else if constexpr (KIND == MX_FP8) {
                    // e4m3 operands: a lane holds columns 16 g .. and 64 + 16 g ..
                    a.x[t][0] = *(const u32x4 *)(c + (int64_t)s * MX_PAD + 16 * g);
                    a.x[t][RAW - 1] = *(const u32x4 *)(c + (int64_t)s * MX_PAD + 64 + 16 * g);
                } else {
                    a.x[t][0] = *(const u32x4 *)(c + (int64_t)s * MX_PAD + MX_BLOCK * g + 16 * unit);
                }
            } else {
                const int64_t k = (int64_t)s * MX_PAD + MX_BLOCK * g + 16 * unit;
                constexpr int BYTES = KIND == MX_ACT_BF16 ? 2 : 4;
                act_raw<BYTES>(p, arow[t], k, a.x[t]);
                act_raw<BYTES>(p, arow[t], k + 8, a.x[t] + RAW / 2);
            }
        }
    };
    auto products = [&](const u32x4 &w, unsigned sc, int unit, const Acts &a) {
        if constexpr (MX) {
            const i32x8 wb = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
            const int ws = (int)(sc >> (8 * g));
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const u32x4 a0 = a.x[t][0], a1 = KIND == MX_FP8 ? a.x[t][RAW - 1] : u32x4{0u, 0u, 0u, 0u};
                const i32x8 ab = {(int)a0[0], (int)a0[1], (int)a0[2], (int)a0[3],
                                  (int)a1[0], (int)a1[1], (int)a1[2], (int)a1[3]};
                const int as = (int)(a.sc[t] >> (8 * g));
                acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wb, ab, acc[t], 4, KIND == MX_FP4 ? 4 : 0, 0,
                                                                         ws, 0, as);
            }
        } else {
            const float scale = __builtin_bit_cast(float, ((sc >> (8 * g)) & 255u) << 23);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const bf16x8 wb = codes_bf16(unit ? w[2 + j] : w[j], scale);
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    if constexpr (KIND == MX_WIDE_FP8) {
                        const float as = __builtin_bit_cast(float, ((a.sc[t] >> (8 * g)) & 255u) << 23);
                        const u32x2 ac = {a.x[t][0][2 * j], a.x[t][0][2 * j + 1]};
                        acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb, codes8_bf16(ac, as), acc[t], 0, 0, 0);
                    } else if constexpr (KIND == MX_ACT_BF16) {
                        acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            wb, __builtin_bit_cast(bf16x8, a.x[t][j]), acc[t], 0, 0, 0);
                    } else {
                        float v[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const unsigned bits = a.x[t][(RAW / 2) * j + (e >> 2)][e & 3];
                            v[e] = __builtin_bit_cast(float, bits);
                        }
                        bf16x8 term[3];
                        bf16_terms<3>(v, term);
#pragma unroll
                        for (int i = 2; i >= 0; --i)
                            acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb, term[i], acc[t], 0, 0, 0);
                    }
                }
            }
        }
    };
    auto steps = [&](int s0, auto count) {
        constexpr int N = decltype(count)::value;
        u32x4 w[N];
        unsigned sc[N];
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const int s = s0 + u * SK_WAVES;
            w[u] = *(const u32x4 *)(wc + (int64_t)s * (MX_PAD / 2));
            sc[u] = wsc[(int64_t)s * p.d_out];
        }
        Acts a[2];
        load(s0, 0, a[0]);
#pragma unroll
        for (int i = 0; i < N * UNITS; ++i) {
            if (i + 1 < N * UNITS) load(s0 + (i + 1) / UNITS * SK_WAVES, (i + 1) % UNITS, a[(i + 1) & 1]);
            if (KIND != MX_ACT_F32) __builtin_amdgcn_sched_barrier(0);   // (fp32's terms fill the time themselves)
            products(w[i / UNITS], sc[i / UNITS], i % UNITS, a[i & 1]);
        }
    };
    int s = wave;
    for (; s + (SK_UNROLL - 1) * SK_WAVES < p.steps; s += SK_UNROLL * SK_WAVES)
        steps(s, std::integral_constant<int, SK_UNROLL>{});
    for (; s < p.steps; s += SK_WAVES) steps(s, std::integral_constant<int, 1>{});

#pragma unroll
    for (int t = 0; t < MT; ++t) lds[wave][t][lane] = acc[t];
    __syncthreads();
    // lane, element e of tile t <-> activation row 16 t + lane % 16, output n0 + 4 (lane / 16) + e;
    // half a wave forms the outputs of a tile, eight per lane
    if (wave >= MT || g >= 2) return;
    f32x4 z0 = lds[0][wave][32 * g + r], z1 = lds[0][wave][32 * g + 16 + r];
#pragma unroll
    for (int w = 1; w < SK_WAVES; ++w) {
        z0 += lds[w][wave][32 * g + r];
        z1 += lds[w][wave][32 * g + 16 + r];
    }
    const int64_t row[1] = {16 * wave + r}, n = n0 + 8 * g;
    if (row[0] >= p.m || n >= p.d_out) return;
    float bias[8], z[1][8] = {{z0[0], z0[1], z0[2], z0[3], z1[0], z1[1], z1[2], z1[3]}};
    mx_bias8(p.out, n, bias);
    mx_epilogue(p.out, p.m, row, n, bias, z);
}

template <int KIND>
hipError_t launch(const SkinnyArgs &p, hipStream_t st) {
    const unsigned blocks = (unsigned)cdiv(p.d_out, 16);
    constexpr int MOST = KIND == MX_ACT_F32 ? 2 : 4;   // tiles of mx_skinny_takes' rows
    switch (cdiv(p.m, 16)) {
        case 1: mx_skinny_kernel<KIND, 1><<<blocks, 64 * SK_WAVES, 0, st>>>(p); break;
        case 2: mx_skinny_kernel<KIND, 2><<<blocks, 64 * SK_WAVES, 0, st>>>(p); break;
        default: mx_skinny_kernel<KIND, MOST><<<blocks, 64 * SK_WAVES, 0, st>>>(p); break;
    }
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// backward: dA = dZ W, few rows
// ---------------------------------------------------------------------------
// A work group takes 128 columns (a step of the weights' rows) and a range of
// outputs r; a wave 32 outputs at a time: lane (g, l) loads 8 codes (columns 8 l ..)
// of the 8 rows 8 g .., which it turns around in registers into the operands of
// eight bf16 MFMAs (16 x 16 x 32), the c-th for columns 8 l + c.  The weights are
// exact in bf16; dZ, formed from dY and the saved Z on the way, enters in three bf16
// terms (24 bits) for an F32 result, one where it is bf16 itself, and two (16) for a
// BF16 result: what they leave, 2^-15 of dZ at most, is a 128th of that result's own
// rounding, and a third term would be half as many MFMAs again.  The waves' sums meet
// in LDS, the ranges' in memory, both added in their order.  Bias gradients: the
// groups of the first 128 columns add their dZ over the rows.
struct SkinnyBack {
    const void *dY, *pre;
    int in_bf16, act, vec;      // vec: whole aligned pieces of eight
    int64_t m, d_out, d_in;
    MxMatrix w;
    int64_t w_bytes;
    float *dbias;               // NULL: not formed
    void *dA;
    int out_bf16;
    float *part;                // [nsplit][m][np]
    int64_t np;                 // d_in padded to whole steps
    int nsplit;
};

// dZ of activation row `row`, outputs r .. r + 7; zeros past the ends
__device__ __forceinline__ void back_dz(const SkinnyBack &p, int64_t row, int64_t r, float (&v)[8]) {
    const bool in = row < p.m;
    mx_ld8(p.dY, in ? row : 0, p.d_out, in ? r : p.d_out, p.in_bf16, p.vec, v);
    if (p.act) {
        float z[8];
        mx_ld8(p.pre, in ? row : 0, p.d_out, in ? r : p.d_out, p.in_bf16, p.vec, z);
        fz_with_act(p.act, [&](auto act) {
            constexpr int ACT = decltype(act)::value;
            if constexpr (ACT) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = v[e] * fz_slope<ACT>(z[e]);
            }
        });
    }
}

// TERMS bf16 terms of dZ; MT: 16-row tiles
template <int TERMS, int MT>
__global__ __launch_bounds__(64 * SK_WAVES) void mx_skinny_backward_kernel(SkinnyBack p) {
    __shared__ float lds[SK_WAVES / 2][16][MX_PAD + 4];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l = lane & 15, g = lane >> 4;
    const int64_t tile = blockIdx.x;
    const int split = blockIdx.y;
    const int64_t pieces = (p.d_out + 31) / 32;           // of 32 outputs
    const int64_t q0 = pieces * split / p.nsplit, q1 = pieces * (split + 1) / p.nsplit;
    const unsigned *sc = (const unsigned *)p.w.scales + tile * p.d_out;
    const uint8_t *wc = p.w.codes + tile * (MX_PAD / 2) + 4 * l;
    f32x4 acc[8][MT];
#pragma unroll
    for (int c = 0; c < 8; ++c)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[c][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int64_t q = q0 + wave; q < q1; q += SK_WAVES) {
        const int64_t r0 = 32 * q + 8 * g;
        unsigned code[8], scale[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {                     // (rows past the end: the last one, against dZ = 0 ...)
            const int64_t r = std::min(r0 + e, p.d_out - 1);
            code[e] = *(const unsigned *)(wc + r * p.w_bytes);
            scale[e] = sc[r];
        }
        bf16x8 dz[MT][TERMS];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            float v[8];
            back_dz(p, 16 * t + l, r0, v);
            if (p.dbias && tile == 0) {
                // the tile's 16 rows are the lanes of a group
                float sum[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    sum[e] = v[e];
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1) sum[e] += __shfl_xor(sum[e], o);
                }
                if (l == 0)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (r0 + e < p.d_out) p.dbias[r0 + e] = t ? p.dbias[r0 + e] + sum[e] : sum[e];
            }
            bf16_terms<TERMS>(v, dz[t]);
        }
        u32x4 wt[8];                                      // operand c: eight rows of column 8 l + c
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            unsigned lo[2], hi[2];
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                unsigned x[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    // (... and weights 0, also where they stand for NaN)
                    const bool in = r0 + e + i < p.d_out;
                    const float s = __builtin_bit_cast(
                        float, in ? ((scale[e + i] >> (8 * (l >> 2))) & 255u) << 23 : 0u);
                    const unsigned w = in ? code[e + i] : 0u;
                    switch (h) {
                        case 0: x[i] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0)); break;
                        case 1: x[i] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1)); break;
                        case 2: x[i] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2)); break;
                        default: x[i] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3)); break;
                    }
                }
                wt[2 * h][e >> 1] = (x[0] & 0xffffu) | (x[1] << 16);
                wt[2 * h + 1][e >> 1] = (x[0] >> 16) | (x[1] & 0xffff0000u);
            }
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const bf16x8 w = __builtin_bit_cast(bf16x8, wt[c]);
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int i = TERMS - 1; i >= 0; --i)
                    acc[c][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, dz[t][i], acc[c][t], 0, 0, 0);
        }
    }
    // register e of lane (g, l), operand c <-> column 8 (4 g + e) + c, row l of the tile;
    // the waves' sums, the later four first to LDS, then added to the earlier four's
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        for (int half = 1; half >= 0; --half) {
            __syncthreads();
            if (wave / (SK_WAVES / 2) == half) {
                float (*out)[MX_PAD + 4] = lds[wave % (SK_WAVES / 2)];
#pragma unroll
                for (int c = 0; c < 8; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float &x = out[l][8 * (4 * g + e) + c];
                        x = half ? acc[c][t][e] : x + acc[c][t][e];
                    }
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 16 * MX_PAD / 4; i += 64 * SK_WAVES) {
            const int row = i / (MX_PAD / 4), col = 4 * (i % (MX_PAD / 4));
            if (16 * t + row >= p.m) continue;
            f32x4 z = *(const f32x4 *)&lds[0][row][col];
#pragma unroll
            for (int w = 1; w < SK_WAVES / 2; ++w) z += *(const f32x4 *)&lds[w][row][col];
            *(f32x4 *)(p.part + ((int64_t)split * p.m + 16 * t + row) * p.np + tile * MX_PAD + col) = z;
        }
    }
}

// the ranges' sums, four columns per thread
__global__ __launch_bounds__(256) void mx_skinny_join_kernel(SkinnyBack p) {
    const int64_t per = p.np / 4, t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (t >= p.m * per) return;
    const int64_t i = t / per, k = 4 * (t - i * per);
    f32x4 z = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int s = 0; s < p.nsplit; ++s) z += *(const f32x4 *)(p.part + ((int64_t)s * p.m + i) * p.np + k);
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (k + e < p.d_in) fz_st(p.dA, i * p.d_in + k + e, z[e], p.out_bf16);
}

// ranges of outputs: two work groups a CU, at least 32 outputs to a wave
int back_splits(int64_t d_out, int64_t d_in) {
    return (int)std::max<int64_t>(1, std::min<int64_t>({512 / mx_steps(d_in), cdiv(d_out, 32 * SK_WAVES), 64}));
}

template <int TERMS>
hipError_t launch_backward(const SkinnyBack &p, hipStream_t st) {
    const dim3 grid((unsigned)mx_steps(p.d_in), (unsigned)p.nsplit);
    switch (cdiv(p.m, 16)) {
        case 1: mx_skinny_backward_kernel<TERMS, 1><<<grid, 64 * SK_WAVES, 0, st>>>(p); break;
        case 2: mx_skinny_backward_kernel<TERMS, 2><<<grid, 64 * SK_WAVES, 0, st>>>(p); break;
        default: mx_skinny_backward_kernel<TERMS, 4><<<grid, 64 * SK_WAVES, 0, st>>>(p); break;
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    mx_skinny_join_kernel<<<(unsigned)cdiv(p.m * (p.np / 4), 256), 256, 0, st>>>(p);
    return hipGetLastError();
}

}  // namespace

// Few rows: where this form takes less time than the tiled ones.  Its time goes
// with the row tiles times a work group's steps times the rounds of groups; us a
// call, few / many: fp8 4096 x 4096, 64 rows (128 of them) 10.8 / 13.9, 4096 x
// 11008, 32 rows (172) 15.3 / 15.2; fp4 1024 x 8192, 64 rows (256) 12.0 / 13.6, 4096
// x 11008, 64 rows (344) 15.6 / 14.8.  The dense form of the other kinds writes the
// whole layer first: bf16 4096 x 4096, 64 rows 22 / 30, 11008 x 4096 56 / 54, 2048 x
// 2048 10.5 / 22, 1024 x 8192 (few work groups) 32 / 28; fp8 with an F32 result, whose
// rows are half as long, 64 rows of the same four 11.5 / 30, 32 / 55, 8.3 / 22, 20 / 28,
// 28672 x 8192 137 / 265; fp32 4096 x 4096, 32 rows 27 / 34, 4096 x 11008 62 / 61, 64
// rows 122 / 63.
bool mx_skinny_takes(int64_t m, int64_t d_out, int64_t d_in, int kind) {
    const int64_t cost = cdiv(m, 16) * mx_steps(d_in) * cdiv(cdiv(d_out, 16), 256);
    switch (kind) {
        case MX_FP8: return m <= 16 || (m <= 64 && cost <= 160);
        case MX_FP4: return m <= 16 || (m <= 64 && cost <= 300);
        case MX_WIDE_FP8: return m <= 64;
        case MX_ACT_F32: return m <= 32;
        default: return m <= 32 || (m <= 64 && d_out >= 2048);
    }
}

hipError_t mx_skinny_launch(const MxLinear &a, hipStream_t st) {
    SkinnyArgs p{};
    p.m = a.m;
    p.d_out = a.d_out;
    p.d_in = a.d_in;
    p.steps = (int)mx_steps(a.d_in);
    p.A = a.A;
    p.a = a.a;
    p.w = a.w;
    p.w_bytes = mx_row_bytes(a.d_in, MX_FP4);
    p.a_bytes = a.A ? 0 : mx_row_bytes(a.d_in, a.a.fmt);
    p.vec = a.d_in % 8 == 0 && reinterpret_cast<uintptr_t>(a.A) % 16 == 0;
    p.out = mx_epilogue_of(a);
    switch (mx_kind(a)) {
        case MX_FP8: return launch<MX_FP8>(p, st);
        case MX_FP4: return launch<MX_FP4>(p, st);
        case MX_WIDE_FP8: return launch<MX_WIDE_FP8>(p, st);
        case MX_ACT_BF16: return launch<MX_ACT_BF16>(p, st);
        default: return launch<MX_ACT_F32>(p, st);
    }
}

// Few rows, us a call, this form / the dense one, with SiLU: bf16 32 rows 4096 x 4096
// 22 / 31, 4096 x 11008 39 / 55; 64 rows 2048 x 2048 17 / 24, 8192 x 1024 21 / 34, but
// 4096 x 4096 33 / 30 and 4096 x 11008 66 / 57: every group of columns forms dZ again,
// which costs most there and little without an activation (bf16 25 / 30, 39 / 56).  f32
// with bias gradients: 32 rows 25 / 39, 48 / 76; 64 rows 2048 x 2048 22 / 32, 8192 x 1024
// 26 / 46, 4096 x 4096 42 / 39; with few outputs there are few ranges and so few groups:
// 333 x 1000 bf16 22 / 18, 1000 x 1000 16 / 19.
bool mx_skinny_backward_takes(const FusedShape &s, int act) {
    if (s.m <= 32) return true;
    return s.m <= 64 && ((s.d_out >= 768 && s.d_out * s.d_in <= (1 << 23)) || (!act && s.in_bf16));
}
size_t mx_skinny_backward_ws(const FusedShape &s) {
    return align256((size_t)back_splits(s.d_out, s.d_in) * s.m * mx_steps(s.d_in) * MX_PAD * sizeof(float));
}
hipError_t mx_skinny_backward_launch(const FusedBackward &a, hipStream_t st) {
    SkinnyBack p{};
    p.dY = a.dY;
    p.pre = a.pre[0];
    p.in_bf16 = a.s.in_bf16;
    p.act = a.act;
    p.vec = a.s.d_out % 8 == 0 && reinterpret_cast<uintptr_t>(a.dY) % 16 == 0 &&
            (!a.act || reinterpret_cast<uintptr_t>(a.pre[0]) % 16 == 0);
    p.m = a.s.m;
    p.d_out = a.s.d_out;
    p.d_in = a.s.d_in;
    p.w = a.mx;
    p.w_bytes = mx_row_bytes(a.s.d_in, MX_FP4);
    p.dbias = a.dbias[0];
    p.dA = a.dA;
    p.out_bf16 = a.s.out_bf16;
    p.part = (float *)a.ws;
    p.np = mx_steps(a.s.d_in) * MX_PAD;
    p.nsplit = back_splits(a.s.d_out, a.s.d_in);
    if (a.s.in_bf16 && !a.act) return launch_backward<1>(p, st);
    return a.s.out_bf16 ? launch_backward<2>(p, st) : launch_backward<3>(p, st);
}

}  // namespace gptq
