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
// Forward, m <= 64: Z = A_p (q - z)^T per group on 16 x 16 x 32 bf16 MFMAs.
// q - z is an integer in [-255, 255], exact in bf16, and a group's products
// sum in fp32 before its scale: the same arithmetic for every output type.
// fp32 activations enter as three bf16 terms (24 bits), one MFMA each.
//
// A work group (8 waves) owns 16 V adjacent outputs of the layer (of both
// layers of a gated pair, so that the product act(G) U is local) and the whole
// contraction, each wave a contiguous run of 32-code units; the waves' sums
// meet in LDS in wave order, and no group waits for another.  The bound is the
// read of the packed words and the conversion of their codes: every lane loads
// the words of V adjacent outputs for its eight codes of a unit (a quarter
// wave's 16 V outputs are 64 V contiguous bytes), PF units ahead.  The loop
// has no branch around a load: rows past m and outputs past the end re-read
// the last ones, units past a wave's run its last unit.
// ---------------------------------------------------------------------------
constexpr int SK_NW = 8;

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

// eight codes as bf16 integers q - z
template <int BITS>
__device__ __forceinline__ bf16x8 int_weights(const Codes8<BITS> &c, float z) {
    bf16x8 w;
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = (__bf16)(c.at(e) - z);
    return w;
}

// HALF: groups may end between the halves of a unit (g not a multiple of 32)
template <int BITS, int V, int MT, int NL, bool A32, bool HALF>
__global__ __launch_bounds__(64 * SK_NW) void skinny_forward_kernel(SkinnyForward p) {
    constexpr int ROWS = 16 * V, NWD = fz_two_words<BITS>() ? 2 : 1;
    constexpr int PF = MT > 1 ? 2 : (V * NL == 1 ? 8 : 4);      // units in flight
    constexpr int AP = A32 ? 3 : 1, AL = A32 ? 2 : 1, ES = A32 ? 4 : 2;   // bf16 terms, loads and bytes of activations
    __shared__ float red[SK_NW * NL * 16 * ROWS];
    const FusedShape &s = p.f.s;
    const int tid = threadIdx.x, lane = tid & 63, li = lane & 15, kg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t r0 = (int64_t)xcd_run(blockIdx.x, p.tiles) * ROWS;
    const int u0 = __builtin_amdgcn_readfirstlane((int)((int64_t)p.nunits * wave / SK_NW));
    const int u1 = __builtin_amdgcn_readfirstlane((int)((int64_t)p.nunits * (wave + 1) / SK_NW));

    struct Slot {
        unsigned w[NL][NWD][V], z[NL][V], s0[NL][V], s1[NL][HALF ? V : 1];   // (s1: the second half's scale)
        u32x4 a[MT][AL];
    };
    // group of a unit's first half, and that half's place in the group
    struct Place {
        int g, at;
        __device__ __forceinline__ void next(int gs) {
            at += 2;
            g += at >= gs;
            at -= at >= gs ? gs : 0;
            if (HALF) {   // (two groups a unit for g of 16)
                g += at >= gs;
                at -= at >= gs ? gs : 0;
            }
        }
    };
    Place ahead, here;
    ahead.g = here.g = __builtin_amdgcn_readfirstlane(2 * u0 / p.gs);
    ahead.at = here.at = __builtin_amdgcn_readfirstlane(2 * u0 - here.g * p.gs);

    // Units are fetched in order: scalar pointers move along, the lanes'
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
        ao[t] = (unsigned)((std::min(16 * t + li, (int)s.m - 1) * (int)p.lda + 8 * kg) * ES);
    int at = std::min(u0, p.nunits - 1);             // the next unit to fetch
    const char *qp[NL], *ap = (const char *)p.A + (int64_t)at * 32 * ES;
#pragma unroll
    for (int l = 0; l < NL; ++l) qp[l] = (const char *)p.f.w[l].Q + (int64_t)at * BITS * stride;
    auto fetch = [&](Slot &sl) {
        const bool last = at == p.nunits - 1;
        const int64_t go = (int64_t)std::min(ahead.g, s.ngroups - 1) * stride;
        const bool between = HALF && ahead.at + 1 >= p.gs && ahead.g + 1 < s.ngroups;
        const unsigned second = between ? stride : 0u;
#pragma unroll
        for (int l = 0; l < NL; ++l) {
#pragma unroll
            for (int d = 0; d < NWD; ++d) load_rows<V>(qp[l], last ? qlast[d] : qo[d], sl.w[l][d]);
            load_rows<V>((const char *)p.f.w[l].zeros + go, ro + (HALF && kg >= 2 ? second : 0u), sl.z[l]);
            load_rows<V>((const char *)p.f.w[l].scales + go, ro, sl.s0[l]);
            if constexpr (HALF) load_rows<V>((const char *)p.f.w[l].scales + go, ro + second, sl.s1[l]);
        }
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int h = 0; h < AL; ++h) sl.a[t][h] = *(const u32x4 *)(ap + ao[t] + 16 * h);
        const bool more = at + 1 < u1;
        ap += more ? 32 * ES : 0;
#pragma unroll
        for (int l = 0; l < NL; ++l) qp[l] += more ? BITS * stride : 0u;
        at += more;
        if (more) ahead.next(p.gs);
    };

    f32x4 acc[NL][V][MT], dg[NL][V][MT];
#pragma unroll
    for (int l = 0; l < NL; ++l)
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int t = 0; t < MT; ++t) acc[l][j][t] = dg[l][j][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    float scale[NL][V];   // of the group that dg belongs to
    auto fold = [&] {
#pragma unroll
        for (int l = 0; l < NL; ++l)
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int t = 0; t < MT; ++t) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[l][j][t][e] = fmaf(scale[l][j], dg[l][j][t][e], acc[l][j][t][e]);
                    dg[l][j][t] = f32x4{0.f, 0.f, 0.f, 0.f};
                }
    };
    auto use = [&](const Slot &sl) {
        const int sh = (BITS * 8 * kg) & 31;   // (a unit starts on a word)
        bf16x8 w[NL][V], a[MT][AP];
#pragma unroll
        for (int l = 0; l < NL; ++l)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const unsigned zb = sl.z[l][j], sb = sl.s0[l][j];
                w[l][j] = int_weights<BITS>(fz_codes8<BITS>(sl.w[l][0][j], sl.w[l][NWD - 1][j], sh),
                                            __builtin_bit_cast(float, zb));
                scale[l][j] = __builtin_bit_cast(float, sb);
            }
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            if constexpr (A32) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const unsigned bits = sl.a[t][e >> 2 & (AL - 1)][e & 3];
                    const float x = __builtin_bit_cast(float, bits);
                    const bool finite = fabsf(x) < __builtin_inff();   // (others only in the first term)
                    const __bf16 b0 = (__bf16)x;
                    const float x1 = finite ? x - (float)b0 : 0.f;
                    const __bf16 b1 = (__bf16)x1;
                    a[t][0][e] = b0;
                    a[t][AP > 1 ? 1 : 0][e] = AP > 1 ? b1 : b0;
                    a[t][AP - 1][e] = AP > 1 ? (__bf16)(x1 - (float)b1) : b0;
                }
            } else {
                a[t][0] = __builtin_bit_cast(bf16x8, sl.a[t][0]);
            }
        }
        auto multiply = [&](bool keep) {   // keep: this lane's codes take part
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int q = AP - 1; q >= 0; --q) {
                    const bf16x8 x = keep ? a[t][q] : bf16x8{};
#pragma unroll
                    for (int l = 0; l < NL; ++l)
#pragma unroll
                        for (int j = 0; j < V; ++j)
                            dg[l][j][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, w[l][j], dg[l][j][t], 0, 0, 0);
                }
        };
        if (!HALF || here.at + 1 < p.gs) {   // both halves in one group
            multiply(true);
            if (here.at + 2 == p.gs) fold();
        } else {                             // a group ends between them
            multiply(kg < 2);
            fold();
#pragma unroll
            for (int l = 0; l < NL; ++l)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const unsigned sb = sl.s1[l][HALF ? j : 0];
                    scale[l][j] = __builtin_bit_cast(float, sb);
                }
            multiply(kg >= 2);
            if (p.gs == 1) fold();
        }
        here.next(p.gs);
    };

    Slot sl[PF];
#pragma unroll
    for (int q = 0; q < PF; ++q) fetch(sl[q]);
    for (int u = u0; u < u1; u += PF) {
#pragma unroll
        for (int q = 0; q < PF; ++q) {
            if (u + q < u1) use(sl[q]);
            fetch(sl[q]);
        }
    }
    if (u1 > u0) fold();

    // lane, register e of (j, t) <-> token 16 t + 4 kg + e, output row + j
    const void *bias0 = p.f.bias[0], *bias1 = p.f.bias[1];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        if (t > 0) __syncthreads();
        if (16 * t >= s.m) break;
#pragma unroll
        for (int l = 0; l < NL; ++l)
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    red[((wave * NL + l) * 16 + 4 * kg + e) * ROWS + V * li + j] = acc[l][j][t][e];
        __syncthreads();
        for (int x = tid; x < 16 * ROWS; x += 64 * SK_NW) {
            const int64_t i = 16 * t + x / ROWS, n = r0 + x % ROWS;
            if (i >= s.m || n >= s.d_out) continue;
            float z[NL];
#pragma unroll
            for (int l = 0; l < NL; ++l) {
                z[l] = 0.f;
#pragma unroll
                for (int w = 0; w < SK_NW; ++w) z[l] += red[(w * NL + l) * 16 * ROWS + x];
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
// A work group (4 waves) owns 128 columns and up to BK_RANGE outputs of one
// layer.  A lane's words of eight outputs hold an 8 x 8 block of codes: eight
// MFMA operands (columns 8 li + j, j = 0..7) without any exchange.  dZ of the
// range is formed once per group in LDS, from dY and the saved
// pre-activations.  The groups' sums are added in range order by a second
// kernel, which also moves the columns back to their original order.
// ---------------------------------------------------------------------------
constexpr int BK_RANGE = 512, BK_COLS = 128, BK_ROWS = 16;

struct SkinnyBackward {
    FusedBackward f;
    float *part;            // [layers * splits][m][d_in]; NULL: one range, straight to dA
    int splits, range;      // ranges per layer, outputs per range (a multiple of 32)
    int64_t nwords;
    int wvec;               // four outputs' words, scales and zero points load together
};

// 2^t that brings v (> 0) to [2^14, 2^15), and 2^-t; 1 for 0
__device__ __forceinline__ void f16_scale(float v, float &mul, float &inv) {
    const int e = v == 0.f ? 14 : (int)((__builtin_bit_cast(unsigned, v) >> 23) & 255u) - 127;
    const int t = max(-126, min(126, 14 - e));
    mul = __builtin_bit_cast(float, (unsigned)(127 + t) << 23);
    inv = __builtin_bit_cast(float, (unsigned)(127 - t) << 23);
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
    return v;
}
__device__ __forceinline__ float finite_abs(float v) {
    const float a = fabsf(v);
    return a < __builtin_inff() ? a : 0.f;
}

template <int BITS, bool HI>
__global__ __launch_bounds__(256) void skinny_backward_kernel(SkinnyBackward p) {
    constexpr int AP = HI ? 2 : 1, LD = BK_RANGE + 8;
    __shared__ __attribute__((aligned(16))) _Float16 dz[AP][BK_ROWS][LD];
    __shared__ float red[4 * BK_ROWS * BK_COLS];   // also the bias sums' [4][BK_RANGE]
    __shared__ float rowinv[BK_ROWS], gmax[8];
    const FusedShape &s = p.f.s;
    const int tid = threadIdx.x, lane = tid & 63, li = lane & 15, kg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l = (int)blockIdx.y / p.splits;
    const int64_t rb = (int64_t)((int)blockIdx.y % p.splits) * p.range;
    const int64_t rend = std::min<int64_t>(s.d_out, rb + p.range);
    const int64_t c0 = (int64_t)blockIdx.x * BK_COLS;
    const PackedLayer w = p.f.w[l];
    const int steps = (int)((rend - rb + 31) / 32);

    // dZ of the range: wave w forms rows w, w + 4, ...
    float bsum[BK_RANGE / 64] = {};
    for (int i = wave; i < s.m; i += 4) {
        float v[BK_RANGE / 64];
        float mx = 0.f;
#pragma unroll
        for (int c = 0; c < BK_RANGE / 64; ++c) {
            const int64_t r = rb + 64 * c + lane, o = i * s.d_out + r;
            v[c] = 0.f;
            if (r < rend) {
                const float dy = fz_ld(p.f.dY, o, s.in_bf16);
                const float z = p.f.pre[0] ? fz_ld(p.f.pre[0], o, s.in_bf16) : 0.f;
                const float u = s.layers == 2 && l == 0 ? fz_ld(p.f.pre[1], o, s.in_bf16) : 1.f;
                fz_with_act(p.f.act, [&](auto act) {
                    constexpr int ACT = decltype(act)::value;
                    v[c] = dy * u * (l == 1 ? fz_act<ACT>(z) : fz_slope<ACT>(z));
                });
            }
            mx = fmaxf(mx, finite_abs(v[c]));
            bsum[c] += v[c];
        }
        float mul, inv;
        f16_scale(wave_max(mx), mul, inv);
        if (lane == 0) rowinv[i] = inv;
#pragma unroll
        for (int c = 0; c < BK_RANGE / 64; ++c) {
            float x = v[c] * mul;
            asm("" : "+v"(x));   // (rounded to f16 from this value alone, both times)
            const bool finite = fabsf(x) < __builtin_inff();   // (others only in the last part: see put_planes)
            const _Float16 h = (_Float16)(finite || !HI ? x : 0.f);
            dz[0][i][64 * c + lane] = h;
            if (HI) dz[AP - 1][i][64 * c + lane] = (_Float16)(finite ? x - (float)h : x);
        }
    }
    const bool bias = blockIdx.x == 0 && p.f.dbias[l];
    if (bias) {
#pragma unroll
        for (int c = 0; c < BK_RANGE / 64; ++c) red[wave * BK_RANGE + 64 * c + lane] = bsum[c];
    }
    // the largest scale of each of the columns' groups, over the range
    const int g0 = (int)(c0 / s.group), g1 = (int)(std::min<int64_t>(c0 + BK_COLS, s.d_in) - 1) / s.group;
    for (int gi = g0 + wave; gi <= g1; gi += 4) {
        float mx = 0.f;
        for (int64_t r = rb + lane; r < rend; r += 64)
            mx = fmaxf(mx, finite_abs(w.scales[(int64_t)gi * s.d_out + r]));
        mx = wave_max(mx);
        if (lane == 0) gmax[gi - g0] = mx;
    }
    __syncthreads();
    if (bias) {
        for (int x = tid; rb + x < rend; x += 256)
            p.f.dbias[l][rb + x] = red[x] + red[BK_RANGE + x] + red[2 * BK_RANGE + x] + red[3 * BK_RANGE + x];
    }
    const int64_t k0 = c0 + 8 * li;
    const int gi = std::min<int>((int)(k0 / s.group), g1);
    float mul, inv;
    f16_scale(gmax[gi - g0] * (float)((1 << BITS) - 1), mul, inv);
    const int64_t j0 = std::min((BITS * k0) >> 5, p.nwords - 1), j1 = std::min(j0 + 1, p.nwords - 1);
    const int sh = (int)((BITS * k0) & 31);

    struct Slot {
        unsigned lo[8], hi[8];
        float s[8], z[8];
    };
    auto fetch = [&](int step, Slot &sl) {
        const int64_t r = rb + 32 * step + 8 * kg;
        if (p.wvec && r + 8 <= s.d_out) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t at = r + 4 * h;
                const u32x4 a = *(const u32x4 *)(w.Q + j0 * s.d_out + at);
                const u32x4 b = fz_two_words<BITS>() ? *(const u32x4 *)(w.Q + j1 * s.d_out + at) : u32x4{0u, 0u, 0u, 0u};
                const f32x4 sc = *(const f32x4 *)(w.scales + (int64_t)gi * s.d_out + at);
                const f32x4 zp = *(const f32x4 *)(w.zeros + (int64_t)gi * s.d_out + at);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    sl.lo[4 * h + e] = a[e];
                    sl.hi[4 * h + e] = b[e];
                    sl.s[4 * h + e] = sc[e];
                    sl.z[4 * h + e] = zp[e];
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {   // (outputs past the end: dZ is 0)
                const int64_t at = std::min<int64_t>(r + e, s.d_out - 1);
                sl.lo[e] = w.Q[j0 * s.d_out + at];
                sl.hi[e] = fz_two_words<BITS>() ? w.Q[j1 * s.d_out + at] : 0u;
                sl.s[e] = w.scales[(int64_t)gi * s.d_out + at];
                sl.z[e] = w.zeros[(int64_t)gi * s.d_out + at];
            }
        }
    };
    f32x4 acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto use = [&](int step, const Slot &sl) {
        const f16x8 a0 = *(const f16x8 *)&dz[0][li][32 * step + 8 * kg];
        f16x8 a1 = a0;
        if (HI) a1 = *(const f16x8 *)&dz[AP - 1][li][32 * step + 8 * kg];
        Codes8<BITS> c[8];
        float sc[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            c[e] = fz_codes8<BITS>(sl.lo[e], sl.hi[e], sh);
            sc[e] = sl.s[e] * mul;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            f16x8 h, r;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float x = (c[e].at(j) - sl.z[e]) * sc[e];
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
    Slot sl[2];
    if (wave < steps) fetch(wave, sl[0]);
    if (wave + 4 < steps) fetch(wave + 4, sl[1]);
    for (int step = wave; step < steps; step += 8) {
        use(step, sl[0]);
        if (step + 8 < steps) fetch(step + 8, sl[0]);
        if (step + 4 < steps) {
            use(step + 4, sl[1]);
            if (step + 12 < steps) fetch(step + 12, sl[1]);
        }
    }
    __syncthreads();   // (the bias sums have been read)
    // lane, register e of j <-> row 4 kg + e, column k0 + j
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int i = 4 * kg + e;
        if (i < s.m) {
            const float f = rowinv[i];
#pragma unroll
            for (int j = 0; j < 8; ++j) red[(wave * BK_ROWS + i) * BK_COLS + 8 * li + j] = acc[j][e] * f * inv;
        }
    }
    __syncthreads();
    for (int x = tid; x < (int)s.m * BK_COLS; x += 256) {
        const int64_t i = x / BK_COLS, k = c0 + x % BK_COLS;
        if (k >= s.d_in) continue;
        const float v = red[x] + red[BK_ROWS * BK_COLS + x] + red[2 * BK_ROWS * BK_COLS + x] +
                        red[3 * BK_ROWS * BK_COLS + x];
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

template <int BITS, int V, int NL, bool HALF>
void launch_forward_k(const SkinnyForward &p, hipStream_t st) {
    const dim3 grid((unsigned)p.tiles), block(64 * SK_NW);
    if (p.f.s.m > 16) {
        if constexpr (V * NL <= 2) skinny_forward_kernel<BITS, V, 4, NL, false, HALF><<<grid, block, 0, st>>>(p);
    } else if (p.f.s.in_bf16) {
        skinny_forward_kernel<BITS, V, 1, NL, false, HALF><<<grid, block, 0, st>>>(p);
    } else {
        if constexpr (V == 1) skinny_forward_kernel<BITS, V, 1, NL, true, HALF><<<grid, block, 0, st>>>(p);
    }
}

template <int BITS, int NL>
hipError_t launch_forward(const SkinnyForward &p, int v, hipStream_t st) {
    if (p.gs % 2 == 1)
        launch_forward_k<BITS, 1, NL, true>(p, st);
    else if (v == 2)
        launch_forward_k<BITS, 2, NL, false>(p, st);
    else
        launch_forward_k<BITS, 1, NL, false>(p, st);
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

bool skinny_forward_takes(const FusedShape &s) { return s.m <= (s.in_bf16 ? 64 : 16); }

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

bool skinny_backward_takes(const FusedShape &s) { return s.m <= BK_ROWS; }

size_t skinny_backward_ws(const FusedShape &s) {
    int splits, range;
    backward_ranges(s, splits, range);
    return splits * s.layers > 1 ? align256((size_t)(splits * s.layers) * s.m * s.d_in * sizeof(float)) : 0;
}

hipError_t skinny_backward_launch(const FusedBackward &a, hipStream_t st) {
    const FusedShape &s = a.s;
    SkinnyBackward p{};
    p.f = a;
    if (s.layers == 1 && a.act == 0) p.f.pre[0] = nullptr;
    backward_ranges(s, p.splits, p.range);
    p.part = p.splits * s.layers > 1 ? (float *)a.ws : nullptr;
    p.nwords = cdiv(s.bits * s.d_in, 32);
    p.wvec = s.d_out % 4 == 0;
    for (int l = 0; l < s.layers; ++l)
        p.wvec = p.wvec && aligned(a.w[l].Q, 16) && aligned(a.w[l].scales, 16) && aligned(a.w[l].zeros, 16);
    switch (s.bits) {
        case 2: launch_backward<2>(p, st); break;
        case 3: launch_backward<3>(p, st); break;
        case 4: launch_backward<4>(p, st); break;
        case 8: launch_backward<8>(p, st); break;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !p.part) return e;
    skinny_backward_reduce_kernel<<<dim3((unsigned)cdiv(s.d_in, 256), (unsigned)s.m), 256, 0, st>>>(p);
    return hipGetLastError();
}

}  // namespace gptq
