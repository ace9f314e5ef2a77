// Packed form of the fused products (few activation rows): one pass over the
// packed words, dequantized in registers and multiplied on the matrix cores.
#include "fused.h"

#include <algorithm>

namespace gptq {

namespace {

// Work groups go round the 8 XCDs in turn; consecutive tiles share 128-byte
// lines of the packed words, so each XCD takes a contiguous run of tiles.
__device__ __forceinline__ int xcd_run(int b, int total) {
    const int q = total / 8, r = total % 8, x = b % 8;
    return x * q + min(x, r) + b / 8;
}

// ---------------------------------------------------------------------------
// Forward, few rows (up to 64 per work group): Z = A_p (q - z)^T per group on 16 x 16 x 32 bf16 MFMAs.
// q - z is an integer in [-255, 255], exact in bf16, and a chunk's products
// sum in fp32 before the group's scale: the same arithmetic for every output
// type.  The integers carry a factor 2^-(bits + 7), which the sums of a chunk
// of 128 codes at most cannot grow out of again (without it, activations above
// 1e35 overflowed there although the scaled sums did not); it leaves with the
// waves' sums.
// fp32 activations enter as three bf16 terms of eight bits each, one MFMA per
// term.  The terms are cut, not rounded: the largest finite values would round
// to bf16's infinity, and a mask is cheaper than a conversion (11008 x 4096, 3
// bits, one row: 25 us a call, 29 with conversions).
//
// A work group (8 waves) owns 16 V adjacent outputs of the layer (of both
// layers of a gated pair, so that the product act(G) U is local) and the whole
// contraction, each wave a contiguous run of 32-code units; the waves' sums
// meet in LDS in wave order, and no group waits for another.  The bound is the
// read of the packed words and the conversion of their codes: every lane loads
// the words of V adjacent outputs for its eight codes of a unit (a quarter
// wave's 16 V outputs are 64 V contiguous bytes), PF units ahead.  The loop
// has no branch around a load: rows past m and outputs past the end re-read
// the last ones, units past a wave's run its last unit.  Measured: 1 row, 4096
// x 4096, 4 bits 5.8 us (9.0 with a group's end looked for at every unit; the
// loop has 45 instructions a unit and one MFMA); pair 11008 x 4096, 3 bits,
// groups of 32, 1 row 31 us, 1.8 TB/s of words, scales and zero points (50
// instructions for eight codes of a lane).
// ---------------------------------------------------------------------------
constexpr int SK_NW = 8;
constexpr int SK_MAX_M = 128;   // bf16 rows, in blocks of up to 64

struct SkinnyForward {
    FusedForward f;
    const void *A;          // the rows in processing order, 16-byte aligned
    int64_t lda;            // elements of a row: whole units, zeros past d_in
    int nunits, gs;         // units of 32 codes; 16-code halves per group
    int tail;               // words of the last unit
    int tiles;
};

template <int V>
__device__ __forceinline__ void load_rows(const char *base, unsigned off, unsigned (&out)[V]) {
    if constexpr (V == 2) {
        const u32x2 v = *(const u32x2 *)(base + off);
        out[0] = v[0];
        out[1] = v[1];
    } else {
        out[0] = *(const unsigned *)(base + off);
    }
}

// eight codes as bf16 values (q - z) 2^-int_shift, zs: the zero point with that
// factor (both products are exact: one rounding, of the difference, as without)
template <int BITS>
constexpr int int_shift() { return BITS + 7; }
template <int BITS>
constexpr float int_factor() { return 1.f / (float)(1 << int_shift<BITS>()); }
template <int BITS>
__device__ __forceinline__ bf16x8 int_weights(const Codes8<BITS> &c, float zs) {
    u32x4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        w[e] = fz_pack_bf16(fmaf(c.at(2 * e), int_factor<BITS>(), -zs), fmaf(c.at(2 * e + 1), int_factor<BITS>(), -zs));
    return __builtin_bit_cast(bf16x8, w);
}

// CH: units of a chunk (1 or 4) that lies in one group; 0: chunks of one unit
// whose halves may belong to two groups (g not a multiple of 32)
template <int BITS, int V, int MT, int NL, bool A32, int CH>
__global__ __launch_bounds__(64 * SK_NW) void skinny_forward_kernel(SkinnyForward p) {
    constexpr bool HALF = CH == 0;
    constexpr int C = HALF ? 1 : CH;                            // units of a chunk
    constexpr int ROWS = 16 * V, NWD = fz_two_words<BITS>() ? 2 : 1;
    constexpr int AP = A32 ? 3 : 1, AL = A32 ? 2 : 1, ES = A32 ? 4 : 2;   // bf16 terms, loads and bytes of activations
    // chunks in flight
    constexpr int PF = C == 4 ? (MT > 1 || NL * V * NWD > 2 || A32 ? 1 : 3) : (MT > 1 ? 2 : (V * NL == 1 ? 8 : 4));
    __shared__ float red[SK_NW * NL * 16 * ROWS];
    const FusedShape &s = p.f.s;
    const int tid = threadIdx.x, lane = tid & 63, li = lane & 15, kg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t r0 = (int64_t)xcd_run(blockIdx.x, p.tiles) * ROWS;
    const int m0 = MT > 1 ? 16 * MT * (int)blockIdx.y : 0;      // first activation row
    const int nch = p.nunits / C;                               // (whole chunks: see the launch)
    const int c0 = __builtin_amdgcn_readfirstlane((int)((int64_t)nch * wave / SK_NW));
    const int c1 = __builtin_amdgcn_readfirstlane((int)((int64_t)nch * (wave + 1) / SK_NW));

    struct Slot {
        unsigned w[C][NL][NWD][V], z[NL][V], s0[NL][V], s1[NL][HALF ? V : 1];   // (s1: the second half's scale)
        u32x4 a[C][MT][AL];
    };

    // Chunks are fetched in order: scalar pointers move along, the lanes'
    // offsets stay.
    const unsigned stride = (unsigned)s.d_out * 4;   // bytes of a word row, of a group's scales
    const unsigned ro = (unsigned)std::min<int64_t>(r0 + V * li, s.d_out - V) * 4;
    const int wd = (BITS * 8 * kg) >> 5;             // the lane's first word of a unit
    unsigned qo[NWD], qlast[NWD], ao[MT];
#pragma unroll
    for (int d = 0; d < NWD; ++d) {
        qo[d] = (unsigned)std::min(wd + d, BITS - 1) * stride + ro;
        qlast[d] = (unsigned)std::min(wd + d, p.tail - 1) * stride + ro;
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
        ao[t] = (unsigned)((std::min(m0 + 16 * t + li, (int)s.m - 1) * (int)p.lda + 8 * kg) * ES);
    int at = std::min(c0, nch - 1);                  // the next chunk to fetch
    const char *ap = (const char *)p.A + (int64_t)at * C * 32 * ES;
    const char *qp[NL], *zp[NL], *sp[NL];
    // the chunk's group (its first half's, and that half's place in it), or
    // the chunks left in it
    int g = 0, place = 0;
    if constexpr (HALF) {
        g = __builtin_amdgcn_readfirstlane(2 * at / p.gs);
        place = __builtin_amdgcn_readfirstlane(2 * at - g * p.gs);
    } else {
        const int per = p.gs / (2 * C);              // chunks of a group
        g = __builtin_amdgcn_readfirstlane(at / per);
        place = per - __builtin_amdgcn_readfirstlane(at - g * per);
    }
#pragma unroll
    for (int l = 0; l < NL; ++l) {
        qp[l] = (const char *)p.f.w[l].Q + (int64_t)at * C * BITS * stride;
        zp[l] = (const char *)p.f.w[l].zeros + (int64_t)g * stride;
        sp[l] = (const char *)p.f.w[l].scales + (int64_t)g * stride;
    }
    auto fetch = [&](Slot &sl) {
        const bool last = at == nch - 1;
        // (past the end the last group's parameters stand in)
        const bool between = HALF && place + 1 >= p.gs && g + 1 < s.ngroups;
        const unsigned second = between ? stride : 0u;
#pragma unroll
        for (int l = 0; l < NL; ++l) {
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int d = 0; d < NWD; ++d)
                    load_rows<V>(qp[l] + c * BITS * stride, last && c == C - 1 ? qlast[d] : qo[d], sl.w[c][l][d]);
            load_rows<V>(zp[l], ro + (HALF && kg >= 2 ? second : 0u), sl.z[l]);
            load_rows<V>(sp[l], ro, sl.s0[l]);
            if constexpr (HALF) load_rows<V>(sp[l], ro + second, sl.s1[l]);
        }
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int h = 0; h < AL; ++h) sl.a[c][t][h] = *(const u32x4 *)(ap + ao[t] + 32 * ES * c + 16 * h);
        if (at + 1 < c1) {
            ++at;
            ap += C * 32 * ES;
            int on;   // groups to move on
            if constexpr (HALF) {
                place += 2;
                on = place >= p.gs;
                place -= on ? p.gs : 0;
                const int again = place >= p.gs;   // (two groups a unit for g of 16)
                place -= again ? p.gs : 0;
                on = std::min(on + again, s.ngroups - 1 - g);
                g += on;
            } else {
                on = --place == 0;
                place += on ? p.gs / (2 * C) : 0;
            }
#pragma unroll
            for (int l = 0; l < NL; ++l) {
                qp[l] += C * BITS * stride;
                zp[l] += on * stride;
                sp[l] += on * stride;
            }
        }
    };

    f32x4 acc[NL][V][MT];
#pragma unroll
    for (int l = 0; l < NL; ++l)
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int t = 0; t < MT; ++t) acc[l][j][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    // a chunk's products in fp32, then its scale
    auto use = [&](const Slot &sl) {
        const int sh = (BITS * 8 * kg) & 31;   // (a unit starts on a word)
        bf16x8 a[C][MT][AP];
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                if constexpr (A32) {
                    u32x4 term[3];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float x[2];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const unsigned bits = sl.a[c][t][e >> 1 & (AL - 1)][2 * (e & 1) + h];
                            x[h] = __builtin_bit_cast(float, bits);
                        }
#pragma unroll
                        for (int q = 0; q < 3; ++q) {
                            const unsigned b0 = __builtin_bit_cast(unsigned, x[0]), b1 = __builtin_bit_cast(unsigned, x[1]);
                            term[q][e] = __builtin_amdgcn_perm(b1, b0, 0x07060302u);   // both upper halves
                            // (an infinity only in the first term; NaN in all, also where its
                            // payload was cut off)
                            x[0] = q == 0 && fabsf(x[0]) == __builtin_inff()
                                       ? 0.f : x[0] - __builtin_bit_cast(float, b0 & 0xffff0000u);
                            x[1] = q == 0 && fabsf(x[1]) == __builtin_inff()
                                       ? 0.f : x[1] - __builtin_bit_cast(float, b1 & 0xffff0000u);
                        }
                    }
#pragma unroll
                    for (int q = 0; q < AP; ++q) a[c][t][q] = __builtin_bit_cast(bf16x8, term[q]);
                } else {
                    a[c][t][0] = __builtin_bit_cast(bf16x8, sl.a[c][t][0]);
                }
            }
#pragma unroll
        for (int l = 0; l < NL; ++l)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float zs = __builtin_bit_cast(float, sl.z[l][j]) * int_factor<BITS>();
                const unsigned s0 = sl.s0[l][j], s1 = sl.s1[l][HALF ? j : 0];
                f32x4 dg[MT], dh[MT];
#pragma unroll
                for (int t = 0; t < MT; ++t) dg[t] = dh[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const bf16x8 w = int_weights<BITS>(fz_codes8<BITS>(sl.w[c][l][0][j], sl.w[c][l][NWD - 1][j], sh), zs);
                    const bf16x8 w0 = HALF && kg >= 2 ? bf16x8{} : w, w1 = kg < 2 ? bf16x8{} : w;
#pragma unroll
                    for (int t = 0; t < MT; ++t)
#pragma unroll
                        for (int q = AP - 1; q >= 0; --q) {
                            if constexpr (HALF) {   // (lanes of the other half: no activations either, see inf)
                                const bf16x8 x0 = kg >= 2 ? bf16x8{} : a[c][t][q], x1 = kg < 2 ? bf16x8{} : a[c][t][q];
                                dg[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x0, w0, dg[t], 0, 0, 0);
                                dh[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x1, w1, dh[t], 0, 0, 0);
                            } else {
                                dg[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[c][t][q], w, dg[t], 0, 0, 0);
                            }
                        }
                }
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        acc[l][j][t][e] = fmaf(__builtin_bit_cast(float, s0), dg[t][e], acc[l][j][t][e]);
                        if (HALF) acc[l][j][t][e] = fmaf(__builtin_bit_cast(float, s1), dh[t][e], acc[l][j][t][e]);
                    }
            }
    };

    Slot sl[PF];
#pragma unroll
    for (int q = 0; q < PF; ++q) fetch(sl[q]);
    for (int c = c0; c < c1; c += PF) {
#pragma unroll
        for (int q = 0; q < PF; ++q) {
            if (c + q < c1) use(sl[q]);
            if (c + q + PF < c1) fetch(sl[q]);
        }
    }

    // lane, register e of (j, t) <-> row m0 + 16 t + 4 kg + e of A, output r0 + V li + j
    const void *bias0 = p.f.bias[0], *bias1 = p.f.bias[1];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        if (t > 0) __syncthreads();
        if (m0 + 16 * t >= s.m) break;
#pragma unroll
        for (int l = 0; l < NL; ++l)
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    red[((wave * NL + l) * 16 + 4 * kg + e) * ROWS + V * li + j] = acc[l][j][t][e];
        __syncthreads();
        for (int x = tid; x < 16 * ROWS; x += 64 * SK_NW) {
            const int64_t i = m0 + 16 * t + x / ROWS, n = r0 + x % ROWS;
            if (i >= s.m || n >= s.d_out) continue;
            float z[NL];
#pragma unroll
            for (int l = 0; l < NL; ++l) {
                z[l] = 0.f;
#pragma unroll
                for (int w = 0; w < SK_NW; ++w) z[l] += red[(w * NL + l) * 16 * ROWS + x];
                z[l] = fz_ldexp(z[l], int_shift<BITS>());
            }
            const int64_t o = i * s.d_out + n;
            if (bias0) z[0] += fz_ld(bias0, n, p.f.bias_bf16);
            if (p.f.pre[0]) fz_st(p.f.pre[0], o, z[0], s.out_bf16);
            float y = 0.f;
            fz_with_act(p.f.act, [&](auto act) { y = fz_act<decltype(act)::value>(z[0]); });
            if constexpr (NL == 2) {
                if (bias1) z[1] += fz_ld(bias1, n, p.f.bias_bf16);
                if (p.f.pre[1]) fz_st(p.f.pre[1], o, z[1], s.out_bf16);
                y *= z[1];
            }
            if (p.f.residual) y += fz_ld(p.f.residual, o, s.out_bf16);
            fz_st(p.f.Y, o, y, s.out_bf16);
        }
    }
}

// rows of A in processing order, padded to whole units with zeros
template <class T>
__global__ __launch_bounds__(256) void gather_rows_kernel(const T *A, const int32_t *perm, T *out, int64_t d_in,
                                                          int64_t lda) {
    const int64_t i = blockIdx.y, k = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (k < lda) out[i * lda + k] = k < d_in ? A[i * d_in + (perm ? (int64_t)perm[k] : k)] : (T)0;
}

// ---------------------------------------------------------------------------
// Backward, m <= 16: dA = dZ W on 16 x 16 x 32 f16 MFMAs.  The contraction
// runs over the outputs r, whose scales differ, so the scale is folded into
// the weight: w = s (q - z) rounded to 11 bits; dZ is rounded to 11 bits too.
// An F32 result takes both in two parts and three products (hi hi + hi lo +
// lo hi).  Power-of-two factors bring a group's weights and a row's dZ into
// f16's range; they are taken over the work group's own outputs and undone
// before its sums leave.
//
// A work group (4 waves) owns 128 columns and a range of outputs of one
// layer.  A lane's words of eight outputs hold an 8 x 8 block of codes: eight
// MFMA operands (columns 8 li + j, j = 0..7) without any exchange.  dZ of the
// range enters LDS once per group (formed from dY and the saved
// pre-activations by a kernel before, where there is an activation).  The groups' sums are added in range order by a second
// kernel, which also moves the columns back to their original order.
// Measured: 7 rows, 4096 x 4096, 4 bits 13 us + 3-4 us for the sums;
// 62% of the wave cycles wait (the loads before the first product, the
// exchanges for the ranges, the barriers), the rest is the conversion.
// ---------------------------------------------------------------------------
constexpr int BK_COLS = 128, BK_RANGE = 512;   // columns, and outputs at most, of a work group
constexpr int BK_MAX_M = 16;

struct SkinnyBackward {
    FusedBackward f;
    const void *dz[2];      // dZ of each layer [m][d_out]: dY itself, or formed in the workspace
    int dz_bf16;
    float *dzw;             // room for it: [layers][m][d_out] fp32
    float *part;            // [layers * splits][m][d_in]; NULL: one range, straight to dA
    int splits, range;      // ranges per layer, outputs per range (a multiple of 32)
    int64_t nwords;
    int wvec;               // four outputs' words, scales and zero points load together
};

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
    return v;
}
__device__ __forceinline__ float finite_abs(float v) {
    const float a = fabsf(v);
    return a < __builtin_inff() ? a : 0.f;
}

// dZ of every layer in fp32, and the bias gradients: 64 outputs per work
// group, a wave every fourth row
__global__ __launch_bounds__(256) void skinny_dz_kernel(SkinnyBackward p, int write) {
    __shared__ float red[2][4][64];
    const FusedShape &s = p.f.s;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t r = (int64_t)blockIdx.x * 64 + lane, rc = std::min(r, s.d_out - 1);
    float sum[2] = {0.f, 0.f};
    for (int ib = wave; ib < s.m; ib += 16) {
        float dy[4], z[4], u[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int64_t o = std::min<int64_t>(ib + 4 * b, s.m - 1) * s.d_out + rc;
            dy[b] = fz_ld(p.f.dY, o, s.in_bf16);
            z[b] = p.f.pre[0] ? fz_ld(p.f.pre[0], o, s.in_bf16) : 0.f;
            u[b] = s.layers == 2 ? fz_ld(p.f.pre[1], o, s.in_bf16) : 1.f;
        }
        fz_with_act(p.f.act, [&](auto act) {
            constexpr int ACT = decltype(act)::value;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const float d0 = fz_gate_grad<ACT>(dy[b], u[b], z[b]), d1 = dy[b] * fz_act<ACT>(z[b]);
                const int64_t i = ib + 4 * b;
                if (i >= s.m) break;
                sum[0] += d0;
                sum[1] += d1;
                if (write && r < s.d_out) {
                    p.dzw[i * s.d_out + r] = d0;
                    if (s.layers == 2) p.dzw[(s.m + i) * s.d_out + r] = d1;
                }
            }
        });
    }
    red[0][wave][lane] = sum[0];
    red[1][wave][lane] = sum[1];
    __syncthreads();
    float *db = wave < s.layers ? p.f.dbias[wave & 1] : nullptr;
    if (db && r < s.d_out) db[r] = red[wave & 1][0][lane] + red[wave & 1][1][lane] + red[wave & 1][2][lane] + red[wave & 1][3][lane];
}

template <int BITS, bool HI>
__global__ __launch_bounds__(256) void skinny_backward_kernel(SkinnyBackward p) {
    constexpr int AP = HI ? 2 : 1, LD = BK_RANGE + 8, PER = BK_RANGE / 64;
    __shared__ __attribute__((aligned(16))) _Float16 dz[AP][16][LD];
    __shared__ float red[4 * 16 * BK_COLS];
    __shared__ float gmax[8];
    __shared__ int rowexp[16];
    const FusedShape &s = p.f.s;
    const int tid = threadIdx.x, lane = tid & 63, li = lane & 15, kg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l = (int)blockIdx.y / p.splits;
    const int64_t rb = (int64_t)((int)blockIdx.y % p.splits) * p.range;
    const int64_t rend = std::min<int64_t>(s.d_out, rb + p.range);
    const int64_t c0 = (int64_t)blockIdx.x * BK_COLS;
    const PackedLayer w = p.f.w[l];
    const int steps = (int)((rend - rb + 31) / 32);

    // this lane's columns k0 .. k0 + 7, their group and words
    const int g0 = (int)(c0 / s.group), g1 = (int)((std::min<int64_t>(c0 + BK_COLS, s.d_in) - 1) / s.group);
    const int64_t k0 = c0 + 8 * li;
    const int gi = std::min((int)(k0 / s.group), g1);
    const int64_t j0 = std::min((BITS * k0) >> 5, p.nwords - 1), j1 = std::min(j0 + 1, p.nwords - 1);
    const int sh = (int)((BITS * k0) & 31);
    const unsigned *ql = w.Q + j0 * s.d_out + rb + 8 * kg, *qh = w.Q + j1 * s.d_out + rb + 8 * kg;
    const float *sp = w.scales + (int64_t)gi * s.d_out + rb + 8 * kg, *zp = w.zeros + (int64_t)gi * s.d_out + rb + 8 * kg;
    struct Slot {
        u32x4 lo[2], hi[fz_two_words<BITS>() ? 2 : 1];
        f32x4 s[2], z[2];
    };
    auto fetch = [&](int step, Slot &sl) {
        const int at = 32 * step;
        if (p.wvec && rb + at + 32 <= s.d_out) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                sl.lo[h] = *(const u32x4 *)(ql + at + 4 * h);
                if constexpr (fz_two_words<BITS>()) sl.hi[h] = *(const u32x4 *)(qh + at + 4 * h);
                sl.s[h] = *(const f32x4 *)(sp + at + 4 * h);
                sl.z[h] = *(const f32x4 *)(zp + at + 4 * h);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {   // (outputs past the end: dZ is 0)
                const int o = (int)(std::min<int64_t>(rb + at + 8 * kg + e, s.d_out - 1) - rb) - 8 * kg;
                sl.lo[e >> 2][e & 3] = ql[o];
                if constexpr (fz_two_words<BITS>()) sl.hi[e >> 2][e & 3] = qh[o];
                sl.s[e >> 2][e & 3] = sp[o];
                sl.z[e >> 2][e & 3] = zp[o];
            }
        }
    };
    // the first steps' words travel while dZ is formed
    Slot sl[2];
    fetch(std::min(wave, steps - 1), sl[0]);
    fetch(std::min(wave + 4, steps - 1), sl[1]);

    // dZ of the range in f16 (wave w takes rows w, w + 4, ...), and the largest
    // scale of each of the columns' groups over the range: all loads in flight
    // together, the maxima's exchanges side by side
    {
        float v[4][PER], sc[PER], mx[5] = {0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < PER; ++c) {
            const int64_t r = std::min<int64_t>(rb + 64 * c + lane, rend - 1);
#pragma unroll
            for (int b = 0; b < 4; ++b)
                v[b][c] = fz_ld(p.dz[l], std::min<int64_t>(wave + 4 * b, s.m - 1) * s.d_out + r, p.dz_bf16);
            sc[c] = w.scales[(int64_t)std::min(g0 + wave, g1) * s.d_out + r];
        }
#pragma unroll
        for (int c = 0; c < PER; ++c) {
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                if (rb + 64 * c + lane >= rend) v[b][c] = 0.f;
                mx[b] = fmaxf(mx[b], finite_abs(v[b][c]));
            }
            mx[4] = fmaxf(mx[4], finite_abs(sc[c]));
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
            float t[5];
#pragma unroll
            for (int b = 0; b < 5; ++b) t[b] = __shfl_xor(mx[b], o);
#pragma unroll
            for (int b = 0; b < 5; ++b) mx[b] = fmaxf(mx[b], t[b]);
        }
        if (lane == 0 && g0 + wave <= g1) gmax[wave] = mx[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int i = wave + 4 * b;
            if (i < s.m) {
                float mul;
                int undo;
                fz_pow2_scale(mx[b], mul, undo);
                if (lane == 0) rowexp[i] = undo;
#pragma unroll
                for (int c = 0; c < PER; ++c) {
                    float x = v[b][c] * mul;
                    asm("" : "+v"(x));   // (rounded to f16 from this value alone, both times)
                    const bool finite = fabsf(x) < __builtin_inff();   // (others only in the last part: see put_planes)
                    const _Float16 h = (_Float16)(finite || !HI ? x : 0.f);
                    dz[0][i][64 * c + lane] = h;
                    if (HI) dz[AP - 1][i][64 * c + lane] = (_Float16)(finite ? x - (float)h : x);
                }
            }
        }
        for (int gq = g0 + wave + 4; gq <= g1; gq += 4) {
            float m2 = 0.f;
#pragma unroll
            for (int c = 0; c < PER; ++c)
                m2 = fmaxf(m2, finite_abs(w.scales[(int64_t)gq * s.d_out +
                                                   std::min<int64_t>(rb + 64 * c + lane, rend - 1)]));
            m2 = wave_max(m2);
            if (lane == 0) gmax[gq - g0] = m2;
        }
    }
    __syncthreads();
    float mul;
    int undo;
    fz_pow2_scale(gmax[gi - g0] * (float)((1 << BITS) - 1), mul, undo);

    f32x4 acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto use = [&](int step, const Slot &sl) {
        const f16x8 a0 = *(const f16x8 *)&dz[0][li][32 * step + 8 * kg];
        const f16x8 a1 = *(const f16x8 *)&dz[AP - 1][li][32 * step + 8 * kg];
        Codes8<BITS> c[8];
        float sc[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            constexpr int H = fz_two_words<BITS>() ? 1 : 0;
            c[e] = fz_codes8<BITS>(sl.lo[e >> 2][e & 3], H ? sl.hi[(e >> 2) & H][e & 3] : 0u, sh);
            sc[e] = sl.s[e >> 2][e & 3] * mul;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            f16x8 h, r;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float x = (c[e].at(j) - sl.z[e >> 2][e & 3]) * sc[e];
                if (HI) asm("" : "+v"(x));
                h[e] = (_Float16)x;
                if (HI) r[e] = (_Float16)(x - (float)h[e]);
            }
            if (HI) {
                acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a1, h, acc[j], 0, 0, 0);
                acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a0, r, acc[j], 0, 0, 0);
            }
            acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a0, h, acc[j], 0, 0, 0);
        }
    };
    for (int step = wave; step < steps; step += 8) {
        use(step, sl[0]);
        if (step + 8 < steps) fetch(step + 8, sl[0]);
        if (step + 4 < steps) {
            use(step + 4, sl[1]);
            if (step + 12 < steps) fetch(step + 12, sl[1]);
        }
    }
    // lane, register e of j <-> row 4 kg + e, column k0 + j
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int i = 4 * kg + e;
        const int both = (i < s.m ? rowexp[i] : 0) + undo;
#pragma unroll
        for (int j = 0; j < 8; ++j) red[(wave * 16 + i) * BK_COLS + 8 * li + j] = fz_ldexp(acc[j][e], both);
    }
    __syncthreads();
    for (int x = tid; x < (int)s.m * BK_COLS; x += 256) {
        const int64_t i = x / BK_COLS, k = c0 + x % BK_COLS;
        if (k >= s.d_in) continue;
        const float v = red[x] + red[16 * BK_COLS + x] + red[2 * 16 * BK_COLS + x] + red[3 * 16 * BK_COLS + x];
        if (p.part)
            p.part[(blockIdx.y * s.m + i) * s.d_in + k] = v;
        else
            fz_st(p.f.dA, i * s.d_in + (p.f.perm ? (int64_t)p.f.perm[k] : k), v, s.out_bf16);
    }
}

__global__ __launch_bounds__(256) void skinny_backward_reduce_kernel(SkinnyBackward p) {
    const FusedShape &s = p.f.s;
    const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x, i = blockIdx.y;
    if (k >= s.d_in) return;
    const int n = p.splits * s.layers;
    float v = 0.f;
    for (int q0 = 0; q0 < n; q0 += 8) {   // in range order, eight loads in flight
        float t[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) t[q] = q0 + q < n ? p.part[((q0 + q) * s.m + i) * s.d_in + k] : 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q) v += t[q];
    }
    fz_st(p.f.dA, i * s.d_in + (p.f.perm ? (int64_t)p.f.perm[k] : k), v, s.out_bf16);
}

// ranges: about 512 work groups in all, of at least 128 outputs (one step a wave)
void backward_ranges(const FusedShape &s, int &splits, int &range) {
    const int64_t blocks = cdiv(s.d_in, BK_COLS) * s.layers;
    const int64_t want = std::max<int64_t>(1, 512 / blocks);
    range = (int)std::min<int64_t>(BK_RANGE, std::max<int64_t>(128, cdiv(cdiv(s.d_out, want), 32) * 32));
    splits = (int)cdiv(s.d_out, range);
}

bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

template <int BITS, int V, int NL, int CH>
void launch_forward_k(const SkinnyForward &p, hipStream_t st) {
    const dim3 grid((unsigned)p.tiles, p.f.s.m > 16 ? (unsigned)cdiv(p.f.s.m, 64) : 1u), block(64 * SK_NW);
    if (p.f.s.m > 16) {
        if constexpr (V * NL <= 2) skinny_forward_kernel<BITS, V, 4, NL, false, CH><<<grid, block, 0, st>>>(p);
    } else if (p.f.s.in_bf16) {
        skinny_forward_kernel<BITS, V, 1, NL, false, CH><<<grid, block, 0, st>>>(p);
    } else {
        if constexpr (V == 1) skinny_forward_kernel<BITS, V, 1, NL, true, CH><<<grid, block, 0, st>>>(p);
    }
}

template <int BITS, int NL>
hipError_t launch_forward(const SkinnyForward &p, int v, hipStream_t st) {
    // whole chunks of four units, each in one group
    const bool four = p.gs % 8 == 0 && p.nunits % 4 == 0;
    if (p.gs % 2 == 1)
        launch_forward_k<BITS, 1, NL, 0>(p, st);
    else if (v == 2)
        four ? launch_forward_k<BITS, 2, NL, 4>(p, st) : launch_forward_k<BITS, 2, NL, 1>(p, st);
    else
        four ? launch_forward_k<BITS, 1, NL, 4>(p, st) : launch_forward_k<BITS, 1, NL, 1>(p, st);
    return hipGetLastError();
}
template <int BITS>
hipError_t launch_forward(const SkinnyForward &p, int v, hipStream_t st) {
    return p.f.s.layers == 2 ? launch_forward<BITS, 2>(p, v, st) : launch_forward<BITS, 1>(p, v, st);
}

template <int BITS>
void launch_backward(const SkinnyBackward &p, hipStream_t st) {
    const dim3 grid((unsigned)cdiv(p.f.s.d_in, BK_COLS), (unsigned)(p.splits * p.f.s.layers));
    if (p.f.s.out_bf16)
        skinny_backward_kernel<BITS, false><<<grid, 256, 0, st>>>(p);
    else
        skinny_backward_kernel<BITS, true><<<grid, 256, 0, st>>>(p);
}

}  // namespace

bool skinny_forward_takes(const FusedShape &s) { return s.m <= (s.in_bf16 ? SK_MAX_M : 16); }

size_t skinny_forward_ws(const FusedShape &s) {
    return align256((size_t)(s.m * cdiv(s.d_in, 32) * 32) * (s.in_bf16 ? 2 : 4));   // gathered rows
}

hipError_t skinny_forward_launch(const FusedForward &a, hipStream_t st) {
    const FusedShape &s = a.s;
    SkinnyForward p{};
    p.f = a;
    p.A = a.A;
    p.lda = s.d_in;
    p.nunits = (int)cdiv(s.d_in, 32);
    p.gs = s.ngroups == 1 ? 1 << 30 : s.group / 16;
    p.tail = (int)(cdiv(s.bits * s.d_in, 32) - (int64_t)s.bits * (p.nunits - 1));
    if (a.perm || s.d_in % 32 != 0 || !aligned(a.A, 16)) {
        p.A = a.ws;
        p.lda = (int64_t)p.nunits * 32;
        const dim3 grid((unsigned)cdiv(p.lda, 256), (unsigned)s.m);
        if (s.in_bf16)
            gather_rows_kernel<<<grid, 256, 0, st>>>((const uint16_t *)a.A, a.perm, (uint16_t *)a.ws, s.d_in, p.lda);
        else
            gather_rows_kernel<<<grid, 256, 0, st>>>((const float *)a.A, a.perm, (float *)a.ws, s.d_in, p.lda);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    // Adjacent outputs per lane: two where that still fills the CUs and pairs
    // load together (not for groups that end inside a unit, for fp32
    // activations, or for a pair of layers with four row tiles, whose
    // registers it would double).
    bool pairs = s.d_out % 2 == 0 && cdiv(s.d_out, 32) >= 256 && p.gs % 2 == 0 && s.in_bf16 &&
                 !(s.layers == 2 && s.m > 16);
    for (int l = 0; l < s.layers; ++l)
        pairs = pairs && aligned(a.w[l].Q, 8) && aligned(a.w[l].scales, 8) && aligned(a.w[l].zeros, 8);
    const int v = pairs ? 2 : 1;
    p.tiles = (int)cdiv(s.d_out, 16 * v);
    switch (s.bits) {
        case 2: return launch_forward<2>(p, v, st);
        case 3: return launch_forward<3>(p, v, st);
        case 4: return launch_forward<4>(p, v, st);
        case 8: return launch_forward<8>(p, v, st);
    }
    return hipErrorInvalidValue;
}

// One tile of 16 rows.  With more tiles of it (an earlier version of this
// kernel; packed / dense at 4096 x 4096): linear 17 rows 33 / 35 us, 32 rows
// 39 / 35, 64 rows 64 / 35; pair 17 rows 55 / 50; 11008 x 4096, 3 bits, 17 rows
// 76 / 61.  Only fp32 outputs gained, up to 32 rows (42 / 48, pair 69 / 80).
bool skinny_backward_takes(const FusedShape &s) { return s.m <= BK_MAX_M; }

struct SkinnyBackwardWs {
    size_t part, bytes;   // offset of the ranges' sums behind dZ
};
SkinnyBackwardWs skinny_backward_layout(const FusedShape &s) {
    int splits, range;
    backward_ranges(s, splits, range);
    SkinnyBackwardWs w;
    w.part = align256((size_t)(s.layers * s.m * s.d_out) * sizeof(float));
    w.bytes = w.part + (splits * s.layers > 1 ? align256((size_t)(splits * s.layers) * s.m * s.d_in * sizeof(float)) : 0);
    return w;
}
size_t skinny_backward_ws(const FusedShape &s) { return skinny_backward_layout(s).bytes; }

hipError_t skinny_backward_launch(const FusedBackward &a, hipStream_t st) {
    const FusedShape &s = a.s;
    const SkinnyBackwardWs wl = skinny_backward_layout(s);
    SkinnyBackward p{};
    p.f = a;
    const bool form = s.layers == 2 || a.act != 0;
    if (!form) p.f.pre[0] = nullptr;
    p.dzw = (float *)a.ws;
    p.dz[0] = form ? (const void *)p.dzw : a.dY;
    p.dz[1] = p.dzw + s.m * s.d_out;
    p.dz_bf16 = !form && s.in_bf16;
    backward_ranges(s, p.splits, p.range);
    p.part = p.splits * s.layers > 1 ? (float *)(a.ws + wl.part) : nullptr;
    p.nwords = cdiv(s.bits * s.d_in, 32);
    p.wvec = s.d_out % 4 == 0;
    for (int l = 0; l < s.layers; ++l)
        p.wvec = p.wvec && aligned(a.w[l].Q, 16) && aligned(a.w[l].scales, 16) && aligned(a.w[l].zeros, 16);
    hipError_t e = hipSuccess;
    if (form || a.dbias[0] || a.dbias[1]) {
        skinny_dz_kernel<<<(unsigned)cdiv(s.d_out, 64), 256, 0, st>>>(p, form);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    switch (s.bits) {
        case 2: launch_backward<2>(p, st); break;
        case 3: launch_backward<3>(p, st); break;
        case 4: launch_backward<4>(p, st); break;
        case 8: launch_backward<8>(p, st); break;
    }
    e = hipGetLastError();
    if (e != hipSuccess || !p.part) return e;
    skinny_backward_reduce_kernel<<<dim3((unsigned)cdiv(s.d_in, 256), (unsigned)s.m), 256, 0, st>>>(p);
    return hipGetLastError();
}

}  // namespace gptq
