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

// eight bf16 of activation row `row`, columns k ..; zeros past the end
__device__ __forceinline__ bf16x8 act_bf16(const SkinnyArgs &p, int64_t row, int64_t k) {
    const uint16_t *a = (const uint16_t *)p.A + row * p.d_in;
    if (p.vec) {
        const bool in = k < p.d_in;
        const u32x4 u = *(const u32x4 *)(a + (in ? k : 0));
        return __builtin_bit_cast(bf16x8, in ? u : u32x4{0u, 0u, 0u, 0u});
    }
    u32x4 u = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (k + e < p.d_in) u[e >> 1] |= (unsigned)a[k + e] << (16 * (e & 1));
    return __builtin_bit_cast(bf16x8, u);
}
// fp32 activations as three bf16 terms, each the leading bits of what is left
// (truncated, so that no term overflows); infinities and NaN in the first alone
__device__ __forceinline__ void act_terms(const SkinnyArgs &p, int64_t row, int64_t k, bf16x8 (&t)[3]) {
    float v[8];
    mx_ld8(p.A, row, p.d_in, k, 0, p.vec, v);
    u32x4 u[3] = {};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const unsigned b = __builtin_bit_cast(unsigned, v[e]), mag = b & 0x7fffffffu;
        const bool finite = mag < 0x7f800000u;
        const unsigned hi = (b & 0xffff0000u) | (mag > 0x7f800000u ? 0x400000u : 0u);
        const float r1 = finite ? v[e] - __builtin_bit_cast(float, hi) : 0.f;
        const unsigned mid = __builtin_bit_cast(unsigned, r1) & 0xffff0000u;
        const float r2 = r1 - __builtin_bit_cast(float, mid);
        const unsigned lo = __builtin_bit_cast(unsigned, r2);
        u[0][e >> 1] |= (e & 1) ? hi : hi >> 16;
        u[1][e >> 1] |= (e & 1) ? mid : mid >> 16;
        u[2][e >> 1] |= (e & 1) ? lo & 0xffff0000u : lo >> 16;
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) t[i] = __builtin_bit_cast(bf16x8, u[i]);
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

// KIND: MX_FP8, MX_FP4, MX_ACT_F32, MX_ACT_BF16, or WIDE_FP8 (fp8 as bf16);
// MT: 16-row tiles of activations
constexpr int WIDE_FP8 = 4;
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
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const int s = s0 + u * SK_WAVES;
            if constexpr (KIND == MX_FP8 || KIND == MX_FP4) {
                const i32x8 wb = {(int)w[u][0], (int)w[u][1], (int)w[u][2], (int)w[u][3], 0, 0, 0, 0};
                const int ws = (int)(sc[u] >> (8 * g));
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    const uint8_t *a = p.a.codes + arow[t] * p.a_bytes + 16 * g;
                    const int as = (int)(((const unsigned *)p.a.scales)[s * p.m + arow[t]] >> (8 * g));
                    if constexpr (KIND == MX_FP8) {
                        // e4m3 operands: a lane holds columns 16 g .. and 64 + 16 g ..
                        const i32x4 a0 = *(const i32x4 *)(a + (int64_t)s * MX_PAD);
                        const i32x4 a1 = *(const i32x4 *)(a + (int64_t)s * MX_PAD + 64);
                        const i32x8 ab = {a0[0], a0[1], a0[2], a0[3], a1[0], a1[1], a1[2], a1[3]};
                        acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wb, ab, acc[t], 4, 0, 0, ws, 0, as);
                    } else {
                        const i32x4 a0 = *(const i32x4 *)(a + (int64_t)s * (MX_PAD / 2));
                        const i32x8 ab = {a0[0], a0[1], a0[2], a0[3], 0, 0, 0, 0};
                        acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wb, ab, acc[t], 4, 4, 0, ws, 0, as);
                    }
                }
            } else {
                const float scale = __builtin_bit_cast(float, ((sc[u] >> (8 * g)) & 255u) << 23);
                const int64_t k = (int64_t)s * MX_PAD + MX_BLOCK * g;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bf16x8 wb = codes_bf16(w[u][j], scale);
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        if constexpr (KIND == WIDE_FP8) {
                            const unsigned as = ((const unsigned *)p.a.scales)[s * p.m + arow[t]];
                            const u32x2 ac = *(const u32x2 *)(p.a.codes + arow[t] * p.a_bytes + k + 8 * j);
                            acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                wb, codes8_bf16(ac, __builtin_bit_cast(float, ((as >> (8 * g)) & 255u) << 23)), acc[t],
                                0, 0, 0);
                        } else if constexpr (KIND == MX_ACT_BF16) {
                            acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb, act_bf16(p, arow[t], k + 8 * j),
                                                                            acc[t], 0, 0, 0);
                        } else {
                            bf16x8 a[3];
                            act_terms(p, arow[t], k + 8 * j, a);
#pragma unroll
                            for (int i = 2; i >= 0; --i)
                                acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb, a[i], acc[t], 0, 0, 0);
                        }
                    }
                }
            }
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
    switch (cdiv(p.m, 16)) {
        case 1: mx_skinny_kernel<KIND, 1><<<blocks, 64 * SK_WAVES, 0, st>>>(p); break;
        case 2: mx_skinny_kernel<KIND, 2><<<blocks, 64 * SK_WAVES, 0, st>>>(p); break;
        default: mx_skinny_kernel<KIND, 4><<<blocks, 64 * SK_WAVES, 0, st>>>(p); break;
    }
    return hipGetLastError();
}

}  // namespace

bool mx_skinny_takes(int64_t m, int64_t, int64_t, int) { return m <= 64; }

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
    if (!a.A && a.a.fmt == MX_FP8) return a.out_bf16 ? launch<MX_FP8>(p, st) : launch<WIDE_FP8>(p, st);
    if (!a.A) return launch<MX_FP4>(p, st);
    return a.a_bf16 ? launch<MX_ACT_BF16>(p, st) : launch<MX_ACT_F32>(p, st);
}

}  // namespace gptq
