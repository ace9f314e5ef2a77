// Dense form of the fused products with packed layers (many activation rows).
//
// The packed weights of the call are written once, dequantized, as 11-bit
// (f16) values into the workspace, contraction index contiguous, and the
// product runs as a plain NT matrix product on the f16 matrix cores with the
// bias, activation, residual or gate product in its epilogue:
//   forward   Z[i][n]  = sum_k A16[i][k] W16[n][k]   n: output, k: input column
//   backward  dA[i][n] = sum_k D16[i][k] W16[n][k]   n: input column, k: output
//             (the gated pair: k runs over the gate's outputs, then the up's)
// A layer's dequantization costs d_out d_in elements of traffic, the product
// m times as many multiplications: from about a hundred rows on the products
// dominate, and the inner loop then carries neither code extraction nor group
// scales.  Measured: the product 1.22 PFLOP/s for the pair 28672 x 8192 with
// 2048 rows (1.58 ms), 1.25 for K = 22016 and 4096 x 4096 outputs (0.59 ms), 1.05
// where the last tiles leave CUs idle (pair 11008 x 4096, 4096 rows: 0.70 ms);
// matrix cores busy 62-63% of cycles at a clock of 1.4-1.7 GHz, no LDS conflicts.
// A large library product reaches 1.31-1.42 on the same card.
// The dequantized weights are written at 2.6-4.0 TB/s (pair 28672 x 8192: 940
// MB in 287 us).
//
// f16 operands.  Every row of A16 / D16 is scaled by a power of two that
// brings its largest finite magnitude M to [2^14, 2^15), every row n of W16 by
// one that does the same for its weights; the epilogue undoes both exactly.
// bf16 activations are then exact in f16 (down to 2^-31 M), weights, computed
// gradients and fp32 activations are rounded once to 11 bits, an eighth of a
// bf16 result's own rounding (down to 2^-28 M; f16's smallest step leaves
// 2^-39 M below).  For an F32 result the operands are split in two f16 planes,
// x = hi + lo: 22 bits down to 2^-17 M, where lo meets f16's smallest step, and
// 2^-39 M below.  The product is then three passes over K, hi hi + hi lo + lo
// hi (two when the activations are exact), which the matrix cores' fp32
// accumulators add in one run.
#include "fused.h"

#include <algorithm>

namespace gptq {

namespace {

constexpr int GK = 32;                    // contraction elements per stage
constexpr int64_t DENSE_ROWS = 16384;     // activation rows per pass (bounds the workspace)
constexpr int DZ_ROWS = 16, DZ_ROWS_MANY = 64;   // rows of dZ formed (and summed) by one work group

__device__ __forceinline__ float finite_abs(float v) {
    const float a = fabsf(v);
    return a < __builtin_inff() ? a : 0.f;   // NaN and infinities do not count
}

// largest of v over the work group's NW waves
template <int NW = 4>
__device__ __forceinline__ float block_max(float v) {
    __shared__ float red[NW];
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NW; ++w) v = fmaxf(v, red[w]);
    return v;
}

// Operand layout: tiles of 256 rows, inside a tile stages of GK contraction
// elements, a stage's 256 rows of 64 bytes side by side with their 16-byte
// pieces permuted as the product's LDS reads want them.  A stage of a tile is
// then 16 contiguous kilobytes, moved into LDS as it is.
constexpr int64_t TILE_STAGE = 256 * GK;   // elements of a stage of a tile
__host__ __device__ __forceinline__ int64_t pad_tile(int64_t rows) { return (rows + 255) / 256 * 256; }
__host__ __device__ __forceinline__ int swz(int row) { return ((row >> 1) & 3) ^ ((row >> 3) & 1); }
// element k (a multiple of 8) of row `row`, ktot contraction elements per row
__device__ __forceinline__ int64_t operand_at(int64_t row, int64_t k, int64_t ktot) {
    return ((row >> 8) * (ktot / GK) + k / GK) * TILE_STAGE + (row & 255) * GK +
           8 * ((int)((k >> 3) & 3) ^ swz((int)row));
}

// Eight values as f16 planes at out and, when there are two, out + plane.
// One plane: the rounded values.  Two: hi, and lo = x - hi; of activations
// that are exact in f16 (EXACT), x itself again.  Values that are not finite
// appear in the second plane only, which meets the weights' high plane alone:
// an infinity must not meet the low one, whose signs are arbitrary.
// The value is pinned to its register first: otherwise the compiler may round
// the product behind it to f16 twice, once from its exact value and once from
// its fp32 one, and the two parts no longer belong together.
__device__ __forceinline__ void put_planes(uint16_t *out, int64_t plane, int planes, int exact, const float (&v)[8]) {
    f16x8 hi, lo;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float x = v[e];
        asm("" : "+v"(x));
        const bool finite = fabsf(x) < __builtin_inff();
        hi[e] = (_Float16)(finite || planes == 1 ? x : 0.f);
        lo[e] = (_Float16)(finite && !exact ? x - (float)hi[e] : x);
    }
    *(f16x8 *)out = hi;
    if (planes > 1) *(f16x8 *)(out + plane) = lo;
}

// ---------------------------------------------------------------------------
// forward operands: rows of A (gathered into processing order), weights [n][k]
// ---------------------------------------------------------------------------
struct ForwardPrep {
    const void *A;              // NULL: fp8 activations in amx, all_rows of them, from row0 on
    MxMatrix amx;
    int64_t all_rows, row0;
    int a_bf16, vec;            // vec: whole aligned 16-byte pieces
    const int32_t *perm;
    int64_t m, d_in, kp;        // kp: d_in padded to whole stages
    uint16_t *A16;              // rows [m], contraction [planes_a][kp]
    int planes_a;
    int *ea;                    // [m] exponents that undo the rows' factors
    int pairs;                  // gather from two bf16 rows staged in the launch's LDS
    PackedLayer w[2];
    MxMatrix mx;
    int64_t d_out, nwords;
    int g, ngroups, layers;
    uint16_t *W16;              // per layer: rows [d_out], contraction [planes_w][kp]
    int planes_w;
    int *ew;                    // [layers][d_out] exponents
    int64_t row_blocks;         // work groups of the activation rows, then those of the weights
    int kchunks;
};

// Two rows i, i + 1 (which share 128-byte lines of the operand).
__device__ void prep_rows(const ForwardPrep &p, int64_t i, char *lds) {
    const int tid = threadIdx.x, rows = i + 1 < p.m ? 2 : 1;
    const int d = (int)p.d_in, kp = (int)p.kp, es = p.a_bf16 ? 2 : 4;
    const int64_t ktot = (int64_t)p.planes_a * p.kp;
    const char *row[2] = {(const char *)p.A + i * d * es, (const char *)p.A + (i + rows - 1) * d * es};
    float mx[2] = {0.f, 0.f}, mul[2];
    if (p.vec) {
        for (int k = 8 * tid; k < d; k += 8 * 256) {
            float v[2][8];
#pragma unroll
            for (int r = 0; r < 2; ++r) fz_ld8(row[r], k, p.a_bf16, v[r]);
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int e = 0; e < 8; ++e) mx[r] = fmaxf(mx[r], finite_abs(v[r][e]));
            if (p.pairs) {   // both rows' bf16 values of a column in one word
                u32x4 w[2];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    w[e >> 2][e & 3] = (__builtin_bit_cast(unsigned, +v[0][e]) >> 16) |
                                       (__builtin_bit_cast(unsigned, +v[1][e]) & 0xffff0000u);
                *(u32x4 *)(lds + 4 * k) = w[0];
                *(u32x4 *)(lds + 4 * k + 16) = w[1];
            }
        }
    } else {
        for (int k = tid; k < d; k += 256)
#pragma unroll
            for (int r = 0; r < 2; ++r) mx[r] = fmaxf(mx[r], finite_abs(fz_ld(row[r], k, p.a_bf16)));
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        int undo;
        fz_pow2_scale(block_max(mx[r]), mul[r], undo);   // (its barriers also cover the staged rows)
        if (tid == 0 && r < rows) p.ea[i + r] = undo;
    }
    for (int k0 = 8 * tid; k0 < kp; k0 += 8 * 256) {
        float v[2][8];
        if (p.pairs && k0 < d) {
            int c[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) c[e] = p.perm[k0 + e];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const unsigned w = *(const unsigned *)(lds + 4 * c[e]);
                v[0][e] = fz_bf16((uint16_t)w);
                v[1][e] = fz_bf16((uint16_t)(w >> 16));
            }
        } else if (p.vec && !p.perm && k0 < d) {
#pragma unroll
            for (int r = 0; r < 2; ++r) fz_ld8(row[r], k0, p.a_bf16, v[r]);   // (from the cache)
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int k = k0 + e, c = k < d ? (p.perm ? p.perm[k] : k) : -1;
#pragma unroll
                for (int r = 0; r < 2; ++r) v[r][e] = c < 0 ? 0.f : fz_ld(row[r], c, p.a_bf16);
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            if (r >= rows) break;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[r][e] *= mul[r];
            put_planes(p.A16 + operand_at(i + r, k0, ktot), p.kp * 256, p.planes_a, p.a_bf16, v[r]);
        }
    }
}

// One work group: 32 rows of the layer(s) and FW_K of their columns.  A wave
// takes 8 rows by 64 columns at a time, so that it reads words of eight rows
// side by side and writes 512 contiguous bytes.  Bound by the write of W16;
// 1024 columns measured best (4096 x 11008: 35 us; 512: 39, 2048: 46).
constexpr int FW_ROWS = 32, FW_K = 1024;
template <int BITS>
__device__ void prep_weights(const ForwardPrep &p, unsigned b, float *lds) {
    const int tid = threadIdx.x, d_out = (int)p.d_out, d_in = (int)p.d_in;
    const unsigned tiles = (unsigned)((d_out + FW_ROWS - 1) / FW_ROWS), t = b / (unsigned)p.kchunks;
    const int kc = (int)(b - t * (unsigned)p.kchunks), l = t >= tiles;
    const int r0 = (int)(t - l * tiles) * FW_ROWS;
    const PackedLayer w = p.w[l];
    // the rows' largest scales, over all groups
    float mx = 0.f;
    {
        const float *sc = w.scales + std::min(r0 + (tid & 31), d_out - 1);
        for (int gi = tid >> 5; gi < p.ngroups; gi += 8) mx = fmaxf(mx, finite_abs(sc[(int64_t)gi * d_out]));
        lds[tid] = mx;
    }
    __syncthreads();
    const int wave = tid >> 6, lane = tid & 63;
    const int rl = 8 * wave + (lane & 7);       // row within the tile
    const int r = std::min(r0 + rl, d_out - 1);
    mx = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) mx = fmaxf(mx, lds[32 * e + rl]);
    float mul;
    int undo;
    fz_pow2_scale(mx * (float)((1 << BITS) - 1), mul, undo);
    if (kc == 0 && lane < 8 && r0 + rl < d_out) p.ew[l * d_out + r] = undo;
    if (r0 + rl >= d_out) return;
    const float ginv = 1.f / (float)p.g;
    uint16_t *out = p.W16 + (int64_t)l * pad_tile(d_out) * p.planes_w * p.kp;
    const int kend = std::min((int)p.kp, (kc + 1) * FW_K);
    struct Block {
        unsigned lo, hi;
        float s, z;
    };
    auto load = [&](int k0) {   // (past d_in: the last words again, not used)
        k0 = std::min(k0, (d_in - 1) & ~7);
        const int64_t j = (BITS * k0) >> 5;
        const int64_t gi = fz_div(k0, p.g, ginv);
        Block x;
        x.lo = w.Q[j * d_out + r];
        x.hi = fz_two_words<BITS>() ? w.Q[std::min(j + 1, p.nwords - 1) * d_out + r] : 0u;
        x.s = w.scales[gi * d_out + r] * mul;
        x.z = w.zeros[gi * d_out + r];
        return x;
    };
    // two blocks ahead of the one that is written
    const int first = kc * FW_K + 8 * (lane >> 3);
    Block x0 = load(first), x1 = load(first + 64);
    for (int k0 = first; k0 < kend; k0 += 64) {
        const Block x2 = load(k0 + 128);
        float v[8];
        const Codes8<BITS> c = fz_codes8<BITS>(x0.lo, x0.hi, (BITS * k0) & 31);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = k0 + e < d_in ? (c.at(e) - x0.z) * x0.s : 0.f;
        put_planes(out + operand_at(r, k0, p.planes_w * p.kp), p.kp * 256, p.planes_w, 0, v);
        x0 = x1;
        x1 = x2;
    }
}

// MX weights as f16: a row's factor brings 6 times its largest scale to [2^14,
// 2^15); two significant bits leave them exact in f16 down to 2^-37 of that,
// one plane therefore serves F32 results too.  (Weights below lose bits, 2^-39 of the
// row's largest at most: beside the largest one's product that is beneath an fp32
// sum's own rounding, 2^-24, unless the activations' sizes undo 2^15 of it.)
typedef __attribute__((ext_vector_type(2))) _Float16 mx_f16x2;
// the factor of a block of scale byte `byte` in a row (or a column) whose
// largest is `top`, as the fp32 scale that the conversion takes (it reads the
// exponent bits; NaN for 255, 0 far below)
__device__ __forceinline__ float mx_f16_scale(int byte, int top) {
    return __builtin_bit_cast(float, (unsigned)(byte == 255 ? 255 : max(0, byte - top + 12 + 127)) << 23);
}
__device__ __forceinline__ int mx_undo(int top) { return top - 127 - 12; }   // the exponent that undoes it
__device__ __forceinline__ int mx_top(unsigned scales) {   // largest of four scale bytes, NaN aside
    int t = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const int s = (int)((scales >> (8 * b)) & 255u);
        t = max(t, s == 255 ? 0 : s);
    }
    return t;
}
// rows and columns as in prep_weights: a lane takes eight codes of a row
__device__ void prep_mx_weights(const ForwardPrep &p, unsigned b, int *lds) {
    const int tid = threadIdx.x, d_out = (int)p.d_out;
    const int tile = (int)(b / (unsigned)p.kchunks), kc = (int)b - tile * p.kchunks, r0 = tile * FW_ROWS;
    const int steps = (int)mx_steps(p.d_in);
    const unsigned *sc = (const unsigned *)p.mx.scales;
    int top = 0;
    for (int s = tid >> 5; s < steps; s += 8)
        top = max(top, mx_top(sc[(int64_t)s * d_out + std::min(r0 + (tid & 31), d_out - 1)]));
    lds[tid] = top;
    __syncthreads();
    const int wave = tid >> 6, lane = tid & 63, rl = 8 * wave + (lane & 7), r = r0 + rl;
    top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, lds[32 * e + rl]);
    if (r >= d_out) return;
    if (kc == 0 && lane < 8) p.ew[r] = mx_undo(top);
    const unsigned *codes = (const unsigned *)(p.mx.codes + r * mx_row_bytes(p.d_in, MX_FP4));
    const int kend = std::min((int)p.kp, (kc + 1) * FW_K);
#pragma unroll 4
    for (int k0 = kc * FW_K + 8 * (lane >> 3); k0 < kend; k0 += 64) {
        const unsigned w = codes[k0 >> 3];
        const float s = mx_f16_scale((int)((sc[(int64_t)(k0 >> 7) * d_out + r] >> (8 * ((k0 >> 5) & 3))) & 255u), top);
        const mx_f16x2 x0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 0);
        const mx_f16x2 x1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 1);
        const mx_f16x2 x2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 2);
        const mx_f16x2 x3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 3);
        *(f16x8 *)(p.W16 + operand_at(r, k0, p.kp)) = f16x8{x0[0], x0[1], x1[0], x1[1], x2[0], x2[1], x3[0], x3[1]};
    }
}

// Two rows of fp8 activations as f16: a row's factor brings 448 times its
// largest scale to [2^14, 2^15), four significant bits leave the values exact
// down to 2^-35 of that
__device__ void prep_mx_rows(const ForwardPrep &p, int64_t i0) {
    const int64_t row_bytes = mx_row_bytes(p.d_in, MX_FP8);
    for (int64_t i = i0; i < std::min(i0 + 2, p.m); ++i) {
        const unsigned *sc = (const unsigned *)p.amx.scales + p.row0 + i;
        int top = 0;
        for (int64_t s = threadIdx.x; s < mx_steps(p.d_in); s += 256) top = max(top, mx_top(sc[s * p.all_rows]));
        top = (int)block_max((float)top);
        if (threadIdx.x == 0) p.ea[i] = top - 127 - 6;
        const uint8_t *codes = p.amx.codes + (p.row0 + i) * row_bytes;
        for (int64_t k = 8 * threadIdx.x; k < p.kp; k += 8 * 256) {
            const u32x2 w = *(const u32x2 *)(codes + k);
            const int byte = (int)((sc[(k >> 7) * p.all_rows] >> (8 * ((k >> 5) & 3))) & 255u);
            const float s = __builtin_bit_cast(float, (unsigned)(byte == 255 ? 255 : max(0, byte - top + 6 + 127)) << 23);
            f16x8 v;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const mx_f16x2 x0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[h], s, false);
                const mx_f16x2 x1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[h], s, true);
                v[4 * h] = x0[0];
                v[4 * h + 1] = x0[1];
                v[4 * h + 2] = x1[0];
                v[4 * h + 3] = x1[1];
            }
            *(f16x8 *)(p.A16 + operand_at(i, k, p.kp)) = v;
        }
    }
}

// (BITS 0: an MX layer)
template <int BITS>
__global__ __launch_bounds__(256) void forward_prep_kernel(ForwardPrep p) {
    extern __shared__ __attribute__((aligned(16))) char dyn[];
    if ((int64_t)blockIdx.x < p.row_blocks) {
        if (BITS == 0 && !p.A)
            prep_mx_rows(p, 2 * (int64_t)blockIdx.x);
        else
            prep_rows(p, 2 * (int64_t)blockIdx.x, dyn);
    } else if constexpr (BITS == 0)
        prep_mx_weights(p, (unsigned)((int64_t)blockIdx.x - p.row_blocks), (int *)dyn);
    else
        prep_weights<BITS>(p, (unsigned)((int64_t)blockIdx.x - p.row_blocks), (float *)dyn);
}

// ---------------------------------------------------------------------------
// backward operands: dZ rows, weights [input column][output]
// ---------------------------------------------------------------------------
struct BackwardPrep {
    const void *dY;
    const void *pre[2];
    int act;
    int bf16, vec;              // vec: rows of whole aligned 8-element pieces
    int64_t m, d_out, kp;       // kp: d_out padded to whole stages
    int layers;
    uint16_t *D16;              // rows [m], contraction [planes_a][layers][kp]
    int planes_a;
    float *fa;                  // [m] row factors
    int *ea;                    // [m] exponents that undo them
    float *bias_part;           // [row blocks][layers][d_out], or NULL: no bias gradients
    PackedLayer w[2];
    MxMatrix mx;
    const int32_t *perm;
    int64_t d_in, nwords;
    int g, ngroups, wvec;       // wvec: four rows' words load together
    float *fg;                  // [ngroups] largest scales
    uint16_t *W16;              // rows [d_in], contraction [planes_w][layers][kp]
    int planes_w;
    int *ew;                    // [d_in] exponents that undo the weights' factors, original order
    int dz_rows;                // rows of a dZ tile (bias gradients)
    int64_t dz_blocks, dz_cols; // dZ tiles, then weight tiles
};

// The factors of a row from a bound on its |dZ| (|act'| and |act(z) / z| are
// below 1.13 and 1): its largest finite |dY|, |G| and |U|
__device__ __forceinline__ void bound_scale(const BackwardPrep &p, float md, float mg, float mu, float &mul,
                                            int &undo) {
    const float f = p.layers == 2 ? fmaxf(mg, 1.13f * mu) : (p.pre[0] ? 1.13f : 1.f);
    // (an overflowing bound: the largest finite one)
    fz_pow2_scale(fminf(md * f, 3.0e38f), mul, undo);
}
__device__ __forceinline__ void row_scale(const BackwardPrep &p, int64_t i, float &mul, int &undo) {
    const int64_t o = i * p.d_out;
    float md = 0.f, mg = 0.f, mu = 0.f;
    if (p.vec) {
        for (int r = 8 * threadIdx.x; r < p.d_out; r += 8 * 256) {
            float d[8], g[8], u[8];
            fz_ld8(p.dY, o + r, p.bf16, d);
            if (p.layers == 2) {
                fz_ld8(p.pre[0], o + r, p.bf16, g);
                fz_ld8(p.pre[1], o + r, p.bf16, u);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                md = fmaxf(md, finite_abs(d[e]));
                if (p.layers == 2) {
                    mg = fmaxf(mg, finite_abs(g[e]));
                    mu = fmaxf(mu, finite_abs(u[e]));
                }
            }
        }
    } else {
        for (int r = threadIdx.x; r < p.d_out; r += 256) {
            md = fmaxf(md, finite_abs(fz_ld(p.dY, o + r, p.bf16)));
            if (p.layers == 2) {
                mg = fmaxf(mg, finite_abs(fz_ld(p.pre[0], o + r, p.bf16)));
                mu = fmaxf(mu, finite_abs(fz_ld(p.pre[1], o + r, p.bf16)));
            }
        }
    }
    md = block_max(md);
    if (p.layers == 2) {
        mg = block_max(mg);
        mu = block_max(mu);
    }
    bound_scale(p, md, mg, mu, mul, undo);
}

// eight values of a row's inputs, zeros past the end
__device__ __forceinline__ void load_row8(const BackwardPrep &p, const void *x, int64_t i, int64_t r0, float (&v)[8]) {
    const int64_t o = i * p.d_out + r0;
    if (p.vec && r0 < p.d_out) {
        fz_ld8(x, o, p.bf16, v);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = r0 + e < p.d_out ? fz_ld(x, o + e, p.bf16) : 0.f;
    }
}

// outputs r0 .. r0 + 7 of row i of dZ (of dG and dU) from dY and what was
// saved, as operand planes; the values themselves in d0 (and d1)
__device__ __forceinline__ void put_dz8(const BackwardPrep &p, int64_t i, int64_t r0, float mul, const float (&d)[8],
                                        const float (&z)[8], const float (&u)[8], float (&d0)[8], float (&d1)[8]) {
    const int64_t ktot = (int64_t)p.planes_a * p.layers * p.kp;
    auto put = [&](int l, const float (&x)[8]) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = r0 + e < p.d_out ? x[e] * mul : 0.f;
        put_planes(p.D16 + operand_at(i, l * p.kp + r0, ktot), p.layers * p.kp * 256, p.planes_a, 0, v);
    };
    fz_with_act(p.act, [&](auto act) {
        constexpr int ACT = decltype(act)::value;
        if (p.layers == 2) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                d0[e] = fz_gate_grad<ACT>(d[e], u[e], z[e]);
                d1[e] = d[e] * fz_act<ACT>(z[e]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) d0[e] = ACT ? d[e] * fz_slope<ACT>(z[e]) : d[e];
        }
    });
    put(0, d0);
    if (p.layers == 2) put(1, d1);
}
__device__ __forceinline__ void form_dz8(const BackwardPrep &p, int64_t i, int64_t r0, float mul, float (&d0)[8],
                                         float (&d1)[8]) {
    float d[8], z[8], u[8];
    load_row8(p, p.dY, i, r0, d);
    if (p.pre[0]) load_row8(p, p.pre[0], i, r0, z);
    if (p.layers == 2) load_row8(p, p.pre[1], i, r0, u);
    put_dz8(p, i, r0, mul, d, z, u, d0, d1);
}

// a group's largest scale, over all outputs (and both layers)
template <int NW>
__device__ __forceinline__ void group_range(const BackwardPrep &p, int gi) {
    float mx = 0.f;
    if (p.mx.codes) {   // an MX layer: the largest scale bytes of block gi's columns
        for (int64_t r = threadIdx.x; r < p.d_out; r += 64 * NW) {
            const uint8_t s = p.mx.scales[((int64_t)(gi >> 2) * p.d_out + r) * 4 + (gi & 3)];
            mx = fmaxf(mx, s == 255 ? 0.f : (float)s);
        }
        mx = block_max<NW>(mx);
        if (threadIdx.x == 0) p.fg[gi] = mx;
        return;
    }
    for (int l = 0; l < p.layers; ++l)
        for (int64_t r = threadIdx.x; r < p.d_out; r += 64 * NW)
            mx = fmaxf(mx, finite_abs(p.w[l].scales[(int64_t)gi * p.d_out + r]));
    mx = block_max<NW>(mx);
    if (threadIdx.x == 0) p.fg[gi] = mx;
}

// First pass, rows of bf16 that fit NC eight-element pieces per thread (512
// threads), no bias gradients: a row is read once into registers, its factor
// found, and dZ written.  (Gated pair of 11008, 4096 rows: read twice, which
// the L2 does not hold, the pass moved 750 MB in 180 us.)
// NS: dY alone, with Z, or with G and U
constexpr int ROW_NW = 8, ROW_PIECES = 4;
template <int NC, int NS>
__global__ __launch_bounds__(64 * ROW_NW, 4) void backward_row_kernel(BackwardPrep p) {
    if ((int64_t)blockIdx.x >= p.m) {
        group_range<ROW_NW>(p, (int)((int64_t)blockIdx.x - p.m));
        return;
    }
    constexpr int STEP = 8 * 64 * ROW_NW;
    const int64_t i = blockIdx.x, o = i * p.d_out;
    const int r0 = 8 * threadIdx.x;
    const uint16_t *src[3] = {(const uint16_t *)p.dY + o, (const uint16_t *)p.pre[0] + o, (const uint16_t *)p.pre[1] + o};
    u32x4 raw[NS][NC];
#pragma unroll
    for (int a = 0; a < NS; ++a)
#pragma unroll
        for (int c = 0; c < NC; ++c)
            raw[a][c] = r0 + c * STEP < p.d_out ? *(const u32x4 *)(src[a] + r0 + c * STEP) : u32x4{0u, 0u, 0u, 0u};
    auto unpack = [](const u32x4 &w, float (&v)[8]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = __builtin_bit_cast(float, w[e] << 16);
            v[2 * e + 1] = __builtin_bit_cast(float, w[e] & 0xffff0000u);
        }
    };
    float mx[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int a = 0; a < NS; ++a) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            float v[8];
            unpack(raw[a][c], v);
#pragma unroll
            for (int e = 0; e < 8; ++e) mx[a] = fmaxf(mx[a], finite_abs(v[e]));
        }
        mx[a] = block_max<ROW_NW>(mx[a]);
    }
    float mul;
    int undo;
    bound_scale(p, mx[0], mx[1], mx[2], mul, undo);
    if (threadIdx.x == 0) {
        p.fa[i] = mul;
        p.ea[i] = undo;
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int r = r0 + c * STEP;
        if (r < p.kp) {
            float d[8], z[8], u[8], d0[8], d1[8];
            unpack(raw[0][c], d);
            unpack(raw[NS > 1 ? 1 : 0][c], z);
            unpack(raw[NS > 2 ? 2 : 0][c], u);
            put_dz8(p, i, r, mul, d, z, u, d0, d1);
        }
    }
}

// First pass otherwise: whole rows of dZ in two sweeps, or, where the second
// pass also sums columns for bias gradients, the rows' factors alone
__global__ __launch_bounds__(256) void backward_rows_kernel(BackwardPrep p) {
    if ((int64_t)blockIdx.x >= p.m) {
        group_range<4>(p, (int)((int64_t)blockIdx.x - p.m));
        return;
    }
    const int64_t i = blockIdx.x;
    float mul;
    int undo;
    row_scale(p, i, mul, undo);
    if (threadIdx.x == 0) {
        p.fa[i] = mul;
        p.ea[i] = undo;
    }
    if (p.bias_part) return;
    float d0[8], d1[8];
    for (int64_t r0 = 8 * threadIdx.x; r0 < p.kp; r0 += 8 * 256) form_dz8(p, i, r0, mul, d0, d1);
}

// dz_rows rows by 256 columns of dZ (of dG and dU) with their columns' sums
__device__ void prep_dz(const BackwardPrep &p, unsigned b, float *lds) {
    const int tid = threadIdx.x;
    const unsigned rbu = b / (unsigned)p.dz_cols;
    const int64_t rb = rbu, cb = b - rbu * (unsigned)p.dz_cols;
    const int64_t r0 = cb * 256 + 8 * (tid & 31);
    const int64_t ilast = std::min<int64_t>(p.m, (rb + 1) * p.dz_rows);
    float sum[2][8] = {};
    if (r0 < p.kp)
        for (int64_t i = rb * p.dz_rows + (tid >> 5); i < ilast; i += 8) {
            float d0[8], d1[8] = {};
            form_dz8(p, i, r0, p.fa[i], d0, d1);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                sum[0][e] += d0[e];
                sum[1][e] += d1[e];
            }
        }
    // the eight row lanes of a column, added in their order
    for (int l = 0; l < p.layers; ++l) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) lds[(tid >> 5) * 256 + 8 * (tid & 31) + e] = l ? sum[1][e] : sum[0][e];
        __syncthreads();
        float v = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) v += lds[256 * e + tid];
        if (cb * 256 + tid < p.d_out) p.bias_part[(rb * p.layers + l) * p.d_out + cb * 256 + tid] = v;
    }
}

// 128 outputs by 128 processing columns: a thread turns a block of 8 outputs
// by 8 columns around in registers.  A wave's lanes take 32 outputs (a
// stage's 64 bytes of a W16 row) of 16 column blocks: words are read as whole
// 128-byte lines, and eight consecutive columns are 512 contiguous bytes.
constexpr int BW_ROWS = 128, BW_COLS = 128;
template <int BITS>
__device__ void prep_weights_t(const BackwardPrep &p, unsigned b) {
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const unsigned rtiles = (unsigned)((p.kp + BW_ROWS - 1) / BW_ROWS);
    const unsigned ctiles = (unsigned)((p.d_in + BW_COLS - 1) / BW_COLS);
    const unsigned tc = b / rtiles;
    const int l = tc >= ctiles;
    const int64_t r0 = (int64_t)(b - tc * rtiles) * BW_ROWS + 32 * wave + 8 * (lane & 3);
    const int64_t k0 = (int64_t)(tc - l * ctiles) * BW_COLS + 8 * (lane >> 2);
    if (r0 >= p.kp || k0 >= p.d_in) return;
    const PackedLayer w = p.w[l];
    const int64_t gi = fz_div((int)k0, p.g, 1.f / (float)p.g);
    float mul;
    int undo;
    fz_pow2_scale(p.fg[gi] * (float)((1 << BITS) - 1), mul, undo);
    const int64_t pos = BITS * k0, j = pos >> 5, j1 = std::min<int64_t>(j + 1, p.nwords - 1);
    const int sh = (int)(pos & 31);
    float s[8], z[8];
    unsigned lo[8], hi[8];
    const bool whole = p.wvec && r0 + 8 <= p.d_out;
    if (whole) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const f32x4 sv = *(const f32x4 *)(w.scales + gi * p.d_out + r0 + 4 * h);
            const f32x4 zv = *(const f32x4 *)(w.zeros + gi * p.d_out + r0 + 4 * h);
            const u32x4 lv = *(const u32x4 *)(w.Q + j * p.d_out + r0 + 4 * h);
            const u32x4 hv = fz_two_words<BITS>() ? *(const u32x4 *)(w.Q + j1 * p.d_out + r0 + 4 * h)
                                                  : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[4 * h + e] = sv[e] * mul;
                z[4 * h + e] = zv[e];
                lo[4 * h + e] = lv[e];
                hi[4 * h + e] = hv[e];
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int64_t r = r0 + e;
            const bool in = r < p.d_out;
            s[e] = in ? w.scales[gi * p.d_out + r] * mul : 0.f;
            z[e] = in ? w.zeros[gi * p.d_out + r] : 0.f;
            lo[e] = in ? w.Q[j * p.d_out + r] : 0u;
            hi[e] = in && fz_two_words<BITS>() ? w.Q[j1 * p.d_out + r] : 0u;
        }
    }
    Codes8<BITS> c[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = fz_codes8<BITS>(lo[e], hi[e], sh);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        if (k0 + k >= p.d_in) break;
        const int64_t col = p.perm ? (int64_t)p.perm[k0 + k] : k0 + k;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = (c[e].at(k) - z[e]) * s[e];
        put_planes(p.W16 + operand_at(col, l * p.kp + r0, p.planes_w * p.layers * p.kp), p.layers * p.kp * 256,
                   p.planes_w, 0, v);
        if (l == 0 && r0 == 0) p.ew[col] = undo;
    }
}

// the same for an MX layer: the eight rows' scales, of one block, relative to
// the largest of the block's columns
__device__ void prep_mx_weights_t(const BackwardPrep &p, unsigned b) {
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const unsigned rtiles = (unsigned)((p.kp + BW_ROWS - 1) / BW_ROWS), tc = b / rtiles;
    const int64_t r0 = (int64_t)(b - tc * rtiles) * BW_ROWS + 32 * wave + 8 * (lane & 3);
    const int64_t k0 = (int64_t)tc * BW_COLS + 8 * (lane >> 2);
    if (r0 >= p.kp || k0 >= p.d_in) return;
    const int top = (int)p.fg[k0 >> 5];
    const int64_t row_bytes = mx_row_bytes(p.d_in, MX_FP4);
    unsigned code[8], sc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {   // (rows past the end: the last one again, as zeros)
        const int64_t r = std::min(r0 + e, p.d_out - 1);
        code[e] = *(const unsigned *)(p.mx.codes + r * row_bytes + (k0 >> 1));
        sc[e] = ((const unsigned *)p.mx.scales)[(k0 >> 7) * p.d_out + r];
    }
    mx_f16x2 h[8][4];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const bool in = r0 + e < p.d_out;
        const unsigned w = in ? code[e] : 0u;
        const float s = mx_f16_scale(in ? (int)((sc[e] >> (8 * ((k0 >> 5) & 3))) & 255u) : 0, top);
        h[e][0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 0);
        h[e][1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 1);
        h[e][2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 2);
        h[e][3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 3);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        if (k0 + k >= p.d_in) break;
        f16x8 v;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = h[e][k >> 1][k & 1];
        *(f16x8 *)(p.W16 + operand_at(k0 + k, r0, p.kp)) = v;
        if (r0 == 0) p.ew[k0 + k] = mx_undo(top);
    }
}

template <int BITS>
__global__ __launch_bounds__(256) void backward_prep_kernel(BackwardPrep p) {
    __shared__ float lds[2048];
    if ((int64_t)blockIdx.x < p.dz_blocks)
        prep_dz(p, blockIdx.x, lds);
    else if constexpr (BITS == 0)
        prep_mx_weights_t(p, (unsigned)((int64_t)blockIdx.x - p.dz_blocks));
    else
        prep_weights_t<BITS>(p, (unsigned)((int64_t)blockIdx.x - p.dz_blocks));
}

// a bias gradient from its row blocks' sums, in their order; more: added to
// what earlier passes left
__global__ __launch_bounds__(256) void bias_reduce_kernel(const float *part, int64_t blocks, int layers,
                                                          int64_t d_out, float *db0, float *db1, int more) {
    const int64_t r = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int l = blockIdx.y;
    float *db = l ? db1 : db0;
    if (r >= d_out || !db) return;
    float v = more ? db[r] : 0.f;
#pragma unroll 8
    for (int64_t b = 0; b < blocks; ++b) v += part[(b * layers + l) * d_out + r];
    db[r] = v;
}

// ---------------------------------------------------------------------------
// the product
// ---------------------------------------------------------------------------
struct Gemm {
    const uint16_t *A, *B;      // f16 operands of m rows, and of n rows for each layer
    int64_t lda, ldb;           // contraction elements of a row, all planes
    int64_t kp;                 // elements of one pass over the contraction (whole stages)
    int passes;                 // pass 1 reads B's second plane (b_plane further on; 0: B has one)
    int a_pass;                 // the pass that reads A's second plane
    int64_t a_plane, b_plane;   // elements between the planes of a row
    int64_t m, n;
    int layers;                 // 2: the gated pair's forward product
    const int *ea, *ew;         // exponents that undo the operands' factors [m], [layers * n]
    const void *bias[2];
    int bias_bf16, act;
    const void *residual;
    void *Y;
    void *pre[2];
    int out_bf16, vec;          // vec: four consecutive outputs load and store together (n % 4 == 0)
    int width;                  // how many do: 8, 4 or 1
    float *part;                // [nsplit][layers][m][np] when nsplit > 1
    int64_t np;                 // n padded to whole quads
    int nsplit;
    int mt, nt;                 // tiles
};

// The epilogue of W (four, where p.vec allows; else one) consecutive columns,
// of both layers when gated: what depends on the columns alone ...
template <bool GATED, int W>
struct Columns {
    i32x4 ew[GATED ? 2 : 1];
    f32x4 bias[GATED ? 2 : 1];
    __device__ __forceinline__ static f32x4 load(const void *x, int64_t at, int bf16) {
        if constexpr (W == 4) return fz_ld4(x, at, bf16);
        return f32x4{fz_ld(x, at, bf16), 0.f, 0.f, 0.f};
    }
    __device__ __forceinline__ Columns(const Gemm &p, int64_t n) {
#pragma unroll
        for (int l = 0; l < (GATED ? 2 : 1); ++l) {
            if constexpr (W == 4)
                ew[l] = *(const i32x4 *)(p.ew + l * p.n + n);
            else
                ew[l] = i32x4{p.ew[l * p.n + n], 0, 0, 0};
            bias[l] = p.bias[l] ? load(p.bias[l], n, p.bias_bf16) : f32x4{0.f, 0.f, 0.f, 0.f};
        }
    }
};
// ... and row i's outputs at columns n .. from their sums
template <bool GATED, int W>
__device__ __forceinline__ void epilogue(const Gemm &p, const Columns<GATED, W> &col, int64_t i, int64_t n, int ea,
                                         f32x4 z, f32x4 u) {
    const int64_t o = i * p.n + n;
    auto store = [&](void *x, f32x4 v) {
        if constexpr (W == 4)
            fz_st4(x, o, v, p.out_bf16);
        else
            fz_st(x, o, v[0], p.out_bf16);
    };
#pragma unroll
    for (int e = 0; e < W; ++e) z[e] = fz_ldexp(z[e], ea + col.ew[0][e]) + col.bias[0][e];
    if (p.pre[0]) store(p.pre[0], z);
    f32x4 y = z;
    fz_with_act(p.act, [&](auto act) {
#pragma unroll
        for (int e = 0; e < W; ++e) y[e] = fz_act<decltype(act)::value>(z[e]);
    });
    if constexpr (GATED) {
#pragma unroll
        for (int e = 0; e < W; ++e) u[e] = fz_ldexp(u[e], ea + col.ew[GATED][e]) + col.bias[GATED][e];
        if (p.pre[1]) store(p.pre[1], u);
        y *= u;
    }
    if (p.residual) y += col.load(p.residual, o, p.out_bf16);
    store(p.Y, y);
}

// The same for eight consecutive columns, and R rows (those below m) together:
// loads first, so that they overlap
template <bool GATED>
struct Columns8 {
    int ew[GATED ? 2 : 1][8];
    float bias[GATED ? 2 : 1][8];
    __device__ __forceinline__ Columns8(const Gemm &p, int64_t n) {
#pragma unroll
        for (int l = 0; l < (GATED ? 2 : 1); ++l) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                ew[l][e] = n + e < p.n ? p.ew[l * p.n + n + e] : 0;
                bias[l][e] = 0.f;
            }
            if (p.bias[l] && n < p.n) fz_ld_row8(p.bias[l], n, n, p.n, p.bias_bf16, p.width, bias[l]);
        }
    }
};
template <bool GATED, int R>
__device__ __forceinline__ void epilogue8(const Gemm &p, const Columns8<GATED> &col, const int64_t (&row)[R],
                                          const int (&ea)[R], int64_t n, float (&z)[GATED ? 2 : 1][R][8]) {
    float res[R][8];
    if (p.residual) {
#pragma unroll
        for (int r = 0; r < R; ++r)
            fz_ld_row8(p.residual, std::min(row[r], p.m - 1) * p.n + n, n, p.n, p.out_bf16, p.width, res[r]);
    }
#pragma unroll
    for (int l = 0; l < (GATED ? 2 : 1); ++l) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int e = 0; e < 8; ++e) z[l][r][e] = fz_ldexp(z[l][r][e], ea[r] + col.ew[l][e]) + col.bias[l][e];
        if (p.pre[l]) {
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (row[r] < p.m) fz_st_row8(p.pre[l], row[r] * p.n + n, n, p.n, p.out_bf16, p.width, z[l][r]);
        }
    }
    fz_with_act(p.act, [&](auto act) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int e = 0; e < 8; ++e) z[0][r][e] = fz_act<decltype(act)::value>(z[0][r][e]);
    });
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if constexpr (GATED) z[0][r][e] *= z[1][r][e];
            if (p.residual) z[0][r][e] += res[r][e];
        }
        if (row[r] < p.m) fz_st_row8(p.Y, row[r] * p.n + n, n, p.n, p.out_bf16, p.width, z[0][r]);
    }
}

// C tile of 64 NJ columns n by 64 MI rows, four waves of 32 NJ by 32 MI as
// 32 x 32 MFMA tiles.  The weights are the MFMA's first operand, so that a lane holds
// four consecutive columns of one activation row.  Both operands move by
// 16-byte buffer loads straight into a ring of four LDS stages of 32 k (each
// load a contiguous kilobyte: read from rows a stage apart in K-major
// matrices, 64 bytes each, the same loop took 1.86 ms against 1.65 for the pair
// 28672 x 8192 with 2048 rows);
// the permuted 16-byte pieces put the operand reads of a wave on distinct
// banks.  Each half stage's MFMAs run
// between the reads of the next half's operands and half of a refill; the
// wait for a stage counts loads, so two later stages stay in flight across
// the one barrier per stage.
template <int MI, int NJ, bool GATED>
__global__ __launch_bounds__(256, MI * NJ == 16 ? 1 : 2) void fused_gemm_kernel(Gemm p) {
    constexpr int BM = 64 * MI, BN = 64 * NJ, NBUF = 4;
    constexpr int NSIDE = BN * GK * 2, STAGE = NSIDE + BM * GK * 2;   // bytes
    constexpr int NDMA = NJ, MDMA = MI;                               // loads per wave and stage
    constexpr int PER_STAGE = NDMA + MDMA;
    constexpr int COLS = GATED ? BN / 2 : BN;                         // columns n of one layer
    constexpr int EROW = 32 * NJ + 4;                                 // floats of an epilogue row (padded)
    __shared__ __attribute__((aligned(16))) char lds[std::max(NBUF * STAGE, (4 * 64 * EROW + BM) * 4)];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wn = wave >> 1, wm = wave & 1;
    const int h = lane >> 5, li = lane & 31;

    // Work groups go round the 8 XCDs in turn; each XCD takes a contiguous
    // run of tiles, ordered in strips of four tiles n by all tiles m, so that
    // the tiles it works on at once share their operands in its L2.
    const int total = p.mt * p.nt * p.nsplit;
    const int q8 = total / 8, r8 = total % 8;
    const int x = (int)blockIdx.x % 8, y = (int)blockIdx.x / 8;
    int id = x * q8 + min(x, r8) + y;
    const int split = id / (p.mt * p.nt);
    id -= split * p.mt * p.nt;
    const int strip = id / (4 * p.mt), in = id - strip * 4 * p.mt;
    const int width = min(4, p.nt - 4 * strip);
    const int64_t m0 = (int64_t)(in / width) * BM, n0 = (int64_t)(4 * strip + in % width) * COLS;

    const int spp = (int)(p.kp / GK);                 // stages per pass
    const int all = spp * p.passes;
    const int st0 = (int)((int64_t)all * split / p.nsplit);
    const int nst = (int)((int64_t)all * (split + 1) / p.nsplit) - st0;   // >= 1

    // (rows past the end are room of the operands' last tiles: whatever they
    // hold only reaches results that are never stored)
    const uint16_t *abase = p.A + (m0 >> 8) * (p.lda / GK) * TILE_STAGE + (m0 & 255) * GK;
    // the gated pair: waves 2 and 3 move the up layer's rows
    const int64_t bskip = GATED ? (wave >> 1) * pad_tile(p.n) * p.ldb - (wave >> 1) * (BN / 2) * GK : 0;
    const uint16_t *bbase = p.B + (n0 >> 8) * (p.ldb / GK) * TILE_STAGE + (n0 & 255) * GK + bskip;
    const __amdgpu_buffer_rsrc_t arsrc = gm_rsrc(abase, p.lda / GK * TILE_STAGE * 2);
    const __amdgpu_buffer_rsrc_t brsrc = gm_rsrc(bbase, p.ldb / GK * TILE_STAGE * 2);
    // Stages are issued in order, each in two parts (part 0, then 1) of this
    // wave's loads: offsets of the one in turn into both operands, and the
    // stages left of its pass; past the end the last stage again, unused.
    int turn = 0;                                     // the next stage's ring slot is turn % NBUF
    const int pass0 = st0 / spp;
    int pass = __builtin_amdgcn_readfirstlane(pass0);
    int left = __builtin_amdgcn_readfirstlane(spp - (st0 - pass0 * spp));
    constexpr int BYTES = (int)TILE_STAGE * 2;
    const int bsecond = (int)(p.b_plane / GK) * BYTES, asecond = (int)(p.a_plane / GK) * BYTES;
    const int apass = p.a_pass;
    int bk = (st0 - pass0 * spp) * BYTES + (pass0 == 1 ? bsecond : 0);
    int ak = (st0 - pass0 * spp) * BYTES + (pass0 == apass ? asecond : 0);
    auto issue = [&](int part) {
        char *buf = lds + (turn % NBUF) * STAGE;
#pragma unroll
        for (int q = NDMA / 2 * part; q < NDMA / 2 * (part + 1); ++q)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(brsrc, (gm_lds_void *)(buf + (NDMA * wave + q) * 1024), 16,
                                                     (NDMA * wave + q) * 1024 + lane * 16, bk, 0, 0);
#pragma unroll
        for (int q = MDMA / 2 * part; q < MDMA / 2 * (part + 1); ++q)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(arsrc, (gm_lds_void *)(buf + NSIDE + (MDMA * wave + q) * 1024),
                                                     16, (MDMA * wave + q) * 1024 + lane * 16, ak, 0, 0);
    };
    // on to the next stage (after both parts; selects only, so that the
    // products around it stay one scheduling region)
    auto advance = [&] {
        ++turn;
        const bool more = turn < nst, wrap = left == 1;
        pass += more && wrap;
        left = more ? (wrap ? spp : left - 1) : left;
        bk = more ? (wrap ? (pass == 1 ? bsecond : 0) : bk + BYTES) : bk;
        ak = more ? (wrap ? (pass == apass ? asecond : 0) : ak + BYTES) : ak;
    };

    // operand reads: lane l supplies row l % 32 of a 32-row tile, k 8 (l / 32) .. +7
    const int sw = swz(li);
    int brow[4];
#pragma unroll
    for (int j = 0; j < NJ; ++j)
        brow[j] = (GATED ? j / (NJ / 2) * (BN / 2) + wn * (BN / 4) + j % (NJ / 2) * 32 : wn * (BN / 2) + 32 * j) + li;
    const int arow = wm * 32 * MI + li;
    auto frags = [&](int st, int ks, f16x8 (&fb)[NJ], f16x8 (&fa)[MI]) {
        const char *buf = lds + (st % NBUF) * STAGE;
        const int piece = 16 * ((2 * ks + h) ^ sw);
#pragma unroll
        for (int j = 0; j < NJ; ++j) fb[j] = *(const f16x8 *)(buf + brow[j] * GK * 2 + piece);
#pragma unroll
        for (int i = 0; i < MI; ++i) fa[i] = *(const f16x8 *)(buf + NSIDE + (arow + 32 * i) * GK * 2 + piece);
    };
    f32x16 acc[NJ][MI];
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < MI; ++i) acc[j][i] = f32x16{};
    auto products = [&](const f16x8 (&fb)[NJ], const f16x8 (&fa)[MI]) {
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int i = 0; i < MI; ++i)
                acc[j][i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fb[j], fa[i], acc[j][i], 0, 0, 0);
    };
    // the half stage's instruction order: operand reads one behind each MFMA
    // (the first MFMA waits for every read before it), then its loads, spread
    // over the rest
    auto spread = [] {
        constexpr int MFMA = 0x008, VMEM = 0x010, DSR = 0x100;
#pragma unroll
        for (int i = 0; i < NJ + MI; ++i) {
            __builtin_amdgcn_sched_group_barrier(MFMA, 1, 0);
            __builtin_amdgcn_sched_group_barrier(DSR, 1, 0);
        }
#pragma unroll
        for (int i = 0; i < PER_STAGE / 2; ++i) {
            __builtin_amdgcn_sched_group_barrier(VMEM, 1, 0);
            __builtin_amdgcn_sched_group_barrier(MFMA, MI * NJ == 16 ? 2 : 1, 0);
        }
    };
    f16x8 fb0[NJ], fa0[MI], fb1[NJ], fa1[MI];
    for (int st = 0; st < NBUF - 1; ++st) {
        issue(0);
        issue(1);
        advance();
    }
    gm_wait<(NBUF - 2) * PER_STAGE>();     // stage 0 landed
    gm_barrier();
    issue(0);
    frags(0, 0, fb0, fa0);
    for (int st = 0; st < nst - 1; ++st) {
        frags(st, 1, fb1, fa1);
        issue(1);
        products(fb0, fa0);
        spread();
        __builtin_amdgcn_sched_barrier(0);
        advance();
        gm_wait<(NBUF - 2) * PER_STAGE>(); // stage st + 1 landed
        gm_barrier();                      // every wave has read stage st: its buffer is free
        __builtin_amdgcn_sched_barrier(0);
        frags(st + 1, 0, fb0, fa0);
        issue(0);
        products(fb1, fa1);
        spread();
        __builtin_amdgcn_sched_barrier(0);
    }
    frags(nst - 1, 1, fb1, fa1);
    products(fb0, fa0);
    products(fb1, fa1);
    gm_wait<0>();   // the loads past the end must land before the ring is reused
    gm_barrier();

    // lane (h, li), register 4 q + e of tile (j, i) <-> column 8 q + 4 h + e, row li.
    // Each wave turns 64 rows at a time around through its own part of LDS, so
    // that it reads and writes whole row segments, eight columns a lane, R rows
    // in flight together (through buffers of the work group, one row at a time,
    // the sums of a 256 x 256 tile took as long as the products of K = 1200).
    constexpr int WCOLS = GATED ? 16 * NJ : 32 * NJ;   // columns n of a wave
    constexpr int LPR = WCOLS / 8, RPP = 64 / LPR, R = GATED ? 2 : 4;
    const int tid = threadIdx.x, lc = 8 * (lane % LPR), lr = lane / LPR;
    const int64_t n = n0 + wn * WCOLS + lc;
    float *out = (float *)lds + wave * 64 * EROW;
    int *eas = (int *)lds + 4 * 64 * EROW;
    for (int r = tid; r < BM; r += 256) eas[r] = m0 + r < p.m ? p.ea[m0 + r] : 0;
    gm_barrier();   // (the tile's row exponents are there)
    const Columns8<GATED> col(p, n);
#pragma unroll
    for (int i0 = 0; i0 < MI; i0 += 2) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    *(f32x4 *)(out + (32 * i + li) * EROW + 32 * j + 8 * q + 4 * h) =
                        f32x4{acc[j][i0 + i][4 * q], acc[j][i0 + i][4 * q + 1], acc[j][i0 + i][4 * q + 2],
                              acc[j][i0 + i][4 * q + 3]};
        // (other lanes of the wave read what this one wrote)
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (p.nsplit > 1) {   // the sums as they are, a quad a lane
            constexpr int QPR = WCOLS / 4, QROWS = 64 / QPR;
            const int qc = 4 * (lane % QPR);
            const int64_t nq = n0 + wn * WCOLS + qc;
            if (nq < p.np)
#pragma unroll 8
                for (int at = lane / QPR; at < 64; at += QROWS) {
                    const int64_t row = m0 + wm * 32 * MI + 32 * i0 + at;
                    if (row >= p.m) continue;
                    float *part = p.part + (((int64_t)split * p.layers * p.m) + row) * p.np + nq;
#pragma unroll
                    for (int l = 0; l < (GATED ? 2 : 1); ++l)
                        *(f32x4 *)(part + l * p.m * p.np) = *(const f32x4 *)(out + at * EROW + l * WCOLS + qc);
                }
        } else if (n < p.n) {
#pragma unroll 1
            for (int c0 = 0; c0 < 64 / RPP; c0 += R) {
                int64_t row[R];
                int ea[R];
                float z[GATED ? 2 : 1][R][8];
#pragma unroll
                for (int c = 0; c < R; ++c) {
                    const int at = (c0 + c) * RPP + lr, r = wm * 32 * MI + 32 * i0 + at;
                    row[c] = m0 + r;
                    ea[c] = eas[r];
#pragma unroll
                    for (int l = 0; l < (GATED ? 2 : 1); ++l) {
                        const float *in = out + at * EROW + l * WCOLS + lc;
                        const f32x4 z0 = *(const f32x4 *)in, z1 = *(const f32x4 *)(in + 4);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            z[l][c][e] = z0[e];
                            z[l][c][4 + e] = z1[e];
                        }
                    }
                }
                epilogue8<GATED, R>(p, col, row, ea, n, z);
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // (read before the next rows overwrite them)
    }
}

// the splits' sums in split order, and the epilogue: W columns per thread
template <bool GATED, int W>
__global__ __launch_bounds__(256) void split_reduce_kernel(Gemm p) {
    const int64_t per = (p.n + W - 1) / W;
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (t >= p.m * per) return;
    const int64_t i = t / per, n = W * (t - i * per);
    f32x4 z = {0.f, 0.f, 0.f, 0.f}, u = z;
    for (int s = 0; s < p.nsplit; ++s) {
        const float *z0 = p.part + ((int64_t)s * p.layers * p.m + i) * p.np + n;
        const float *u0 = z0 + p.m * p.np;
        if constexpr (W == 4) {
            z += *(const f32x4 *)z0;
            if (GATED) u += *(const f32x4 *)u0;
        } else {
            z[0] += z0[0];
            if (GATED) u[0] += u0[0];
        }
    }
    epilogue<GATED, W>(p, Columns<GATED, W>(p, n), i, n, p.ea[i], z, u);
}

int64_t pad_stage(int64_t k) { return cdiv(k, GK) * GK; }
int64_t pad_quad(int64_t n) { return cdiv(n, 4) * 4; }
bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Tiles of 256 x 256 where at least 32 of them, with their k splits, fill half
// the CUs; otherwise of 128 x 128 (509 x 251 fp32: 23 us a call against 31;
// 2048 x 4096 of 11008, 128 large tiles with two splits: 263 us against 294
// with small ones).  k splits for grids that leave CUs idle, each of at least
// eight stages.
struct Plan {
    int mi, nj, mt, nt, nsplit;   // tile of 64 mi rows by 64 nj columns
};
Plan plan_gemm(int64_t m, int64_t n, int layers, int stages) {
    Plan p;
    for (int size = 4; size >= 2; size -= 2) {
        p.mi = p.nj = size;
        p.mt = (int)cdiv(m, 64 * p.mi);
        p.nt = (int)cdiv(n, (layers == 2 ? 32 : 64) * p.nj);
        const int64_t tiles = (int64_t)p.mt * p.nt;
        p.nsplit = (int)std::max<int64_t>(1, std::min<int64_t>({256 / tiles, (int64_t)stages / 8, (int64_t)16}));
        if (tiles >= 32 && tiles * p.nsplit >= 128) break;
    }
    return p;
}

struct Layout {
    size_t bytes = 0;
    char *base;
    explicit Layout(char *b) : base(b) {}
    template <class T>
    T *take(int64_t count) {
        char *p = base + bytes;   // (a size query only reads `bytes`)
        bytes += align256((size_t)count * sizeof(T));
        return base ? (T *)p : nullptr;
    }
};

struct ForwardWs {
    int *ew, *ea;
    float *part;
    uint16_t *W16, *A16;
    size_t bytes;
    int planes_a, planes_w, passes;
    int64_t kp, rows;
    Plan plan;
};
ForwardWs forward_layout(const FusedShape &s, char *base) {
    ForwardWs w{};
    w.planes_a = w.planes_w = s.out_bf16 ? 1 : 2;
    w.passes = s.out_bf16 ? 1 : (s.in_bf16 ? 2 : 3);
    if (s.bits == 0) {   // MX weights are exact in one plane; bf16 activations too
        w.planes_a = w.passes = s.out_bf16 || s.in_bf16 ? 1 : 2;
        w.planes_w = 1;
    }
    w.kp = pad_stage(s.d_in);
    w.rows = std::min(s.m, DENSE_ROWS);
    w.plan = plan_gemm(w.rows, s.d_out, s.layers, (int)(w.kp / GK) * w.passes);
    Layout l(base);
    w.ew = l.take<int>(s.layers * s.d_out);
    w.ea = l.take<int>(w.rows);
    w.W16 = l.take<uint16_t>(s.layers * pad_tile(s.d_out) * w.planes_w * w.kp);
    w.A16 = l.take<uint16_t>(pad_tile(w.rows) * w.planes_a * w.kp);
    w.part = l.take<float>(w.plan.nsplit > 1 ? w.plan.nsplit * s.layers * w.rows * pad_quad(s.d_out) : 0);
    w.bytes = l.bytes;
    return w;
}

// Few rows: enough work groups; many rows: fewer partial sums per column
int dz_rows(int64_t m) { return m > 1024 ? DZ_ROWS_MANY : DZ_ROWS; }

struct BackwardWs {
    int *ew, *ea;
    float *fg, *fa, *part, *bias;
    uint16_t *W16, *D16;
    size_t bytes;
    int planes_a, planes_w, passes;
    int64_t kp, rows;
    Plan plan;
};
BackwardWs backward_layout(const FusedShape &s, char *base) {
    BackwardWs w{};
    w.planes_a = w.planes_w = s.out_bf16 ? 1 : 2;
    w.passes = s.out_bf16 ? 1 : 3;
    if (s.bits == 0) {
        w.passes = w.planes_a;
        w.planes_w = 1;
    }
    w.kp = pad_stage(s.d_out);
    w.rows = std::min(s.m, DENSE_ROWS);
    w.plan = plan_gemm(w.rows, s.d_in, 1, (int)(w.kp / GK) * s.layers * w.passes);
    Layout l(base);
    w.ew = l.take<int>(s.d_in);
    w.fg = l.take<float>(s.ngroups);
    w.fa = l.take<float>(w.rows);
    w.ea = l.take<int>(w.rows);
    w.W16 = l.take<uint16_t>(pad_tile(s.d_in) * w.planes_w * s.layers * w.kp);
    w.D16 = l.take<uint16_t>(pad_tile(w.rows) * w.planes_a * s.layers * w.kp);
    w.bias = l.take<float>(cdiv(w.rows, dz_rows(w.rows)) * s.layers * s.d_out);
    w.part = l.take<float>(w.plan.nsplit > 1 ? w.plan.nsplit * w.rows * pad_quad(s.d_in) : 0);
    w.bytes = l.bytes;
    return w;
}

template <int MI, int NJ, bool GATED>
hipError_t launch_gemm_k(Gemm g, hipStream_t st) {
    g.width = !g.vec ? 1 : (g.n % 8 ? 4 : 8);
    fused_gemm_kernel<MI, NJ, GATED><<<(unsigned)(g.mt * g.nt * g.nsplit), 256, 0, st>>>(g);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || g.nsplit == 1) return e;
    if (g.vec)
        split_reduce_kernel<GATED, 4><<<(unsigned)cdiv(g.m * cdiv(g.n, 4), 256), 256, 0, st>>>(g);
    else
        split_reduce_kernel<GATED, 1><<<(unsigned)cdiv(g.m * g.n, 256), 256, 0, st>>>(g);
    return hipGetLastError();
}

template <bool GATED>
hipError_t launch_gemm(const Gemm &g, const Plan &p, hipStream_t st) {
    return p.mi == 4 ? launch_gemm_k<4, 4, GATED>(g, st) : launch_gemm_k<2, 2, GATED>(g, st);
}
hipError_t launch_gemm(const Gemm &g, const Plan &p, hipStream_t st) {
    return g.layers == 2 ? launch_gemm<true>(g, p, st) : launch_gemm<false>(g, p, st);
}

constexpr size_t PREP_LDS_MAX = 128 * 1024;   // bytes of two activation rows staged for their gather

template <int BITS>
hipError_t launch_forward_prep(ForwardPrep p, int64_t blocks, hipStream_t st) {
    // The rows' staging would take LDS from the weights' groups too (fewer of
    // them per CU): beyond 16 KB they go in a launch of their own.
    size_t lds = 1024;
    if (p.pairs) {
        const size_t rows = (size_t)p.d_in * 4;
        if (rows > 16 * 1024) {
            if (rows > 64 * 1024) {   // above the default limit a launch needs the kernel's attribute
                const hipError_t e = hipFuncSetAttribute((const void *)forward_prep_kernel<BITS>,
                                                         hipFuncAttributeMaxDynamicSharedMemorySize,
                                                         (int)PREP_LDS_MAX);
                if (e != hipSuccess) return e;
            }
            forward_prep_kernel<BITS><<<(unsigned)p.row_blocks, 256, rows, st>>>(p);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess || blocks == p.row_blocks) return e;
            blocks -= p.row_blocks;
            p.row_blocks = 0;
        } else {
            lds = std::max(lds, rows);
        }
    }
    forward_prep_kernel<BITS><<<(unsigned)blocks, 256, lds, st>>>(p);
    return hipGetLastError();
}

void launch_row(const BackwardPrep &p, int npre, unsigned blocks, hipStream_t st) {
    switch (npre) {
        case 0: backward_row_kernel<ROW_PIECES, 1><<<blocks, 64 * ROW_NW, 0, st>>>(p); break;
        case 1: backward_row_kernel<ROW_PIECES, 2><<<blocks, 64 * ROW_NW, 0, st>>>(p); break;
        default: backward_row_kernel<ROW_PIECES, 3><<<blocks, 64 * ROW_NW, 0, st>>>(p); break;
    }
}

const char *at(const void *p, int64_t elements, int bf16) { return (const char *)p + elements * (bf16 ? 2 : 4); }

}  // namespace

size_t dense_forward_ws(const FusedShape &s) { return forward_layout(s, nullptr).bytes; }
size_t dense_backward_ws(const FusedShape &s) { return backward_layout(s, nullptr).bytes; }

hipError_t dense_forward_launch(const FusedForward &a, hipStream_t st) {
    const FusedShape &s = a.s;
    const ForwardWs w = forward_layout(s, a.ws);
    for (int64_t i0 = 0; i0 < s.m; i0 += DENSE_ROWS) {
        const int64_t m = std::min(DENSE_ROWS, s.m - i0);
        ForwardPrep p{};
        p.A = a.A ? at(a.A, i0 * s.d_in, s.in_bf16) : nullptr;
        p.amx = a.amx;
        p.all_rows = s.m;
        p.row0 = i0;
        p.a_bf16 = s.in_bf16;
        p.vec = s.d_in % 8 == 0 && aligned(a.A, 16);
        p.perm = a.perm;
        p.m = m;
        p.d_in = s.d_in;
        p.kp = w.kp;
        p.A16 = w.A16;
        p.planes_a = w.planes_a;
        p.ea = w.ea;
        p.pairs = p.perm && p.vec && s.in_bf16 && (size_t)s.d_in * 4 <= PREP_LDS_MAX;
        for (int l = 0; l < s.layers; ++l) p.w[l] = a.w[l];
        p.mx = a.mx;
        p.d_out = s.d_out;
        p.nwords = cdiv(s.bits * s.d_in, 32);
        p.g = s.group;
        p.ngroups = s.ngroups;
        p.layers = s.layers;
        p.W16 = w.W16;
        p.planes_w = w.planes_w;
        p.ew = w.ew;
        p.row_blocks = cdiv(m, 2);
        p.kchunks = (int)cdiv(w.kp, FW_K);
        // the weights once, with the first rows
        const int64_t blocks = p.row_blocks + (i0 == 0 ? s.layers * cdiv(s.d_out, FW_ROWS) * p.kchunks : 0);
        hipError_t e = hipErrorInvalidValue;
        switch (s.bits) {
            case 0: e = launch_forward_prep<0>(p, blocks, st); break;
            case 2: e = launch_forward_prep<2>(p, blocks, st); break;
            case 3: e = launch_forward_prep<3>(p, blocks, st); break;
            case 4: e = launch_forward_prep<4>(p, blocks, st); break;
            case 8: e = launch_forward_prep<8>(p, blocks, st); break;
        }
        if (e != hipSuccess) return e;
        Gemm g{};
        g.A = w.A16;
        g.B = w.W16;
        g.lda = w.planes_a * w.kp;
        g.ldb = w.planes_w * w.kp;
        g.kp = g.a_plane = w.kp;
        g.b_plane = w.planes_w > 1 ? w.kp : 0;
        g.passes = w.passes;
        // (activations that are exact meet the weights' high plane as their second, in pass 0)
        g.a_pass = s.bits == 0 ? 1 : (w.passes == 2 ? 0 : 2);
        g.m = m;
        g.n = s.d_out;
        g.layers = s.layers;
        g.ea = w.ea;
        g.ew = w.ew;
        g.bias_bf16 = a.bias_bf16;
        g.act = a.act;
        const int64_t o = i0 * s.d_out;
        g.vec = s.d_out % 4 == 0 && aligned(a.Y, 16) && (!a.residual || aligned(a.residual, 16));
        for (int l = 0; l < s.layers; ++l) {
            g.bias[l] = a.bias[l];
            g.pre[l] = a.pre[l] ? (void *)at(a.pre[l], o, s.out_bf16) : nullptr;
            g.vec = g.vec && (!a.bias[l] || aligned(a.bias[l], 16)) && (!a.pre[l] || aligned(a.pre[l], 16));
        }
        g.residual = a.residual ? at(a.residual, o, s.out_bf16) : nullptr;
        g.Y = (void *)at(a.Y, o, s.out_bf16);
        g.out_bf16 = s.out_bf16;
        g.part = w.part;
        g.np = pad_quad(g.n);
        g.nsplit = w.plan.nsplit;
        g.mt = (int)cdiv(m, 64 * w.plan.mi);   // (the last rows may be fewer)
        g.nt = w.plan.nt;
        e = launch_gemm(g, w.plan, st);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t dense_backward_launch(const FusedBackward &a, hipStream_t st) {
    const FusedShape &s = a.s;
    const BackwardWs w = backward_layout(s, a.ws);
    const bool bias = a.dbias[0] || a.dbias[1];
    for (int64_t i0 = 0; i0 < s.m; i0 += DENSE_ROWS) {
        const int64_t m = std::min(DENSE_ROWS, s.m - i0), o = i0 * s.d_out;
        BackwardPrep p{};
        p.dY = at(a.dY, o, s.in_bf16);
        p.bf16 = s.in_bf16;
        p.vec = s.d_out % 8 == 0 && aligned(a.dY, 16);
        const int npre = s.layers == 2 ? 2 : (a.act ? 1 : 0);
        for (int l = 0; l < npre; ++l) {
            p.pre[l] = at(a.pre[l], o, s.in_bf16);
            p.vec = p.vec && aligned(a.pre[l], 16);
        }
        p.act = a.act;
        p.m = m;
        p.d_out = s.d_out;
        p.kp = w.kp;
        p.layers = s.layers;
        p.D16 = w.D16;
        p.planes_a = w.planes_a;
        p.fa = w.fa;
        p.ea = w.ea;
        p.bias_part = bias ? w.bias : nullptr;
        p.mx = a.mx;
        p.perm = a.perm;
        p.d_in = s.d_in;
        p.nwords = cdiv(s.bits * s.d_in, 32);
        p.g = s.group;
        p.ngroups = s.ngroups;
        p.wvec = s.d_out % 4 == 0;
        for (int l = 0; l < s.layers; ++l) {
            p.w[l] = a.w[l];
            p.wvec = p.wvec && aligned(a.w[l].Q, 16) && aligned(a.w[l].scales, 16) && aligned(a.w[l].zeros, 16);
        }
        p.fg = w.fg;
        p.W16 = w.W16;
        p.planes_w = w.planes_w;
        p.ew = w.ew;
        p.dz_cols = cdiv(w.kp, 256);
        p.dz_rows = dz_rows(m);
        const int64_t row_blocks = cdiv(m, p.dz_rows);
        p.dz_blocks = bias ? p.dz_cols * row_blocks : 0;
        // the groups' ranges and the weights once, with the first rows
        const unsigned firsts = (unsigned)(m + (i0 == 0 ? s.ngroups : 0));
        const int64_t pieces = cdiv(w.kp, 8 * 64 * ROW_NW);
        if (p.vec && p.bf16 && !bias && pieces <= ROW_PIECES)
            launch_row(p, npre, firsts, st);
        else
            backward_rows_kernel<<<firsts, 256, 0, st>>>(p);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        const int64_t blocks =
            p.dz_blocks + (i0 == 0 ? s.layers * cdiv(w.kp, BW_ROWS) * cdiv(s.d_in, BW_COLS) : 0);
        if (blocks > 0) {
            switch (s.bits) {
                case 0: backward_prep_kernel<0><<<(unsigned)blocks, 256, 0, st>>>(p); break;
                case 2: backward_prep_kernel<2><<<(unsigned)blocks, 256, 0, st>>>(p); break;
                case 3: backward_prep_kernel<3><<<(unsigned)blocks, 256, 0, st>>>(p); break;
                case 4: backward_prep_kernel<4><<<(unsigned)blocks, 256, 0, st>>>(p); break;
                case 8: backward_prep_kernel<8><<<(unsigned)blocks, 256, 0, st>>>(p); break;
            }
            e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        if (bias) {
            bias_reduce_kernel<<<dim3((unsigned)cdiv(s.d_out, 256), (unsigned)s.layers), 256, 0, st>>>(
                w.bias, row_blocks, s.layers, s.d_out, a.dbias[0], a.dbias[1], i0 > 0);
            e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        Gemm g{};
        g.A = w.D16;
        g.B = w.W16;
        g.kp = s.layers * w.kp;
        g.lda = w.planes_a * g.kp;
        g.ldb = w.planes_w * g.kp;
        g.a_plane = g.kp;
        g.b_plane = w.planes_w > 1 ? g.kp : 0;
        g.passes = w.passes;
        g.a_pass = s.bits == 0 ? 1 : 2;
        g.m = m;
        g.n = s.d_in;
        g.layers = 1;
        g.ea = w.ea;
        g.ew = w.ew;
        g.Y = (void *)at(a.dA, i0 * s.d_in, s.out_bf16);
        g.out_bf16 = s.out_bf16;
        g.vec = s.d_in % 4 == 0 && aligned(a.dA, 16);
        g.part = w.part;
        g.np = pad_quad(g.n);
        g.nsplit = w.plan.nsplit;
        g.mt = (int)cdiv(m, 64 * w.plan.mi);
        g.nt = w.plan.nt;
        e = launch_gemm(g, w.plan, st);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace gptq
