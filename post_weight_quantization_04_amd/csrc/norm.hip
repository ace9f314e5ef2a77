// Root-mean-square norm of the residual stream in front of a projection, with
// the residual's addition and an output that may be quantized to an MX format
// on the way, and its backward pass.
//
//   S = X + residual, rounded to its type;  r = (mean_j S_j^2 + eps)^(-1/2)
//   Y_j = S_j r w_j
//   c = mean_j dY_j w_j S_j;  dX_j = r (w_j dY_j - (S_j r) (r c)) + dS_j
//   dw_j = sum over rows of dY_j S_j r
//
// S is the stream as it is stored, so that the backward pass, and a norm of
// the stored stream, see the values that this one did.  (The addition in fp32
// and its rounding to bf16 round as once: fp32 holds 24 bits, more than twice
// bf16's 8 and two.)
#include "mx.h"

#include <algorithm>

namespace gptq {

namespace {

// Sums over the LANES threads of a row (256 / LANES rows of a block up to a
// wave each).  Fixed order: lanes by halves, then waves in turn.
template <int LANES, class T>
__device__ __forceinline__ T row_sum(T v, T *lds) {
#pragma unroll
    for (int o = std::min(LANES, 64) / 2; o > 0; o >>= 1) v += __shfl_xor(v, o);
    if constexpr (LANES > 64) {
        const int wave = threadIdx.x >> 6;
        __syncthreads();   // (the sums of the row before have been read)
        if ((threadIdx.x & 63) == 0) lds[wave] = v;
        __syncthreads();
        v = lds[0];
#pragma unroll
        for (int w = 1; w < LANES / 64; ++w) v += lds[w];
    }
    return v;
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
struct NormArgs {
    RmsNorm a;
    int vec;                    // whole aligned pieces of eight
    int64_t padded, row_bytes;  // columns that are written (MX: whole 128), code bytes of a row
    int64_t row0;               // the launch's first row
};

__device__ __forceinline__ void norm_load(const NormArgs &p, int64_t row, int64_t k, float (&v)[8]) {
    mx_ld8(p.a.X, row, p.a.d, k, p.a.bf16, p.vec, v);
    if (p.a.residual) {
        float r[8];
        mx_ld8(p.a.residual, row, p.a.d, k, p.a.bf16, p.vec, r);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[e] += r[e];
            if (p.a.bf16) v[e] = fz_bf16(fz_to_bf16(v[e]));
        }
    }
}
__device__ __forceinline__ void put8(void *x, int64_t row, int64_t d, int64_t k, int bf16, int vec,
                                     const float (&v)[8]) {
    const int64_t o = row * d + k;
    if (vec && k < d) {
        fz_st8(x, o, bf16, v);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (k + e < d) fz_st(x, o + e, v[e], bf16);
    }
}
// a / q with r = 1 / q: the product's last bits mended by what it leaves of a, so
// that exact quotients come out as they are (S = 49 in a row of 49s: 49 r is 1 -
// 2^-53, which on a grid of 8 or 4 bits is another value than 1).  Zeros, infinities
// and NaN leave nothing to mend by.
__device__ __forceinline__ double norm_quotient(double a, double q, double r) {
    constexpr int FINITE = 0x198;   // normal and subnormal, either sign
    const double y = a * r, rest = fma(-y, q, a);
    return __builtin_amdgcn_class(rest, FINITE) ? fma(rest, r, y) : y;
}
// Y = S w / q, q = 1 / r, in 64 bits (S w is exact there), rounded once to its type
// or its grid: a value on or next to a border of a grid of 8 or 4 bits falls on the
// side the definition says.  The 64-bit operations hide behind the memory, but for
// the quotient's (us with an fp8 output and a residual, S w r / so: 2048 x 8192 26.6 /
// 28.5, 64000 x 128 13.0 / 14.3).
template <bool MX>
__device__ __forceinline__ void norm_store(const NormArgs &p, int64_t row, int64_t k, double q, double r,
                                           const float (&v)[8]) {
    float w[8], y[8];
    mx_ld8(p.a.weight, 0, p.a.d, k, p.a.bf16, p.vec, w);
    if constexpr (!MX) {   // (one 64-bit step off or not, a value rounds to the nearest of its type)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const double z = (double)v[e] * (double)w[e] * r;
            y[e] = p.a.bf16 ? mx_odd(z) : (float)z;
        }
        put8(p.a.Y, row, p.a.d, k, p.a.bf16, p.vec, y);
    } else {
        if (k >= p.a.d) r = 0.0;   // (padding, 0 whatever the row's factor is)
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = mx_odd(norm_quotient((double)v[e] * (double)w[e], q, r));
        if (p.a.fmt == MX_FP8)
            mx_put8<MX_FP8>(y, p.a.m, row, k >> 3, p.row_bytes, p.a.codes, p.a.scales);
        else
            mx_put8<MX_FP4>(y, p.a.m, row, k >> 3, p.row_bytes, p.a.codes, p.a.scales);
    }
}

// LANES threads per row, each NC pieces of eight columns held in registers
// between the two sweeps; columns beyond them are formed again from the inputs
template <int LANES, int NC, bool VEC, bool MX>
__global__ __launch_bounds__(std::max(LANES, 256)) void rms_norm_kernel(NormArgs p) {
    p.vec = VEC;   // (known here: the other way of loading costs registers)
    constexpr int STEP = 8 * LANES, ROWS = std::max(1, 256 / LANES);
    __shared__ double lds[std::max(1, LANES / 64)];
    const int64_t row = p.row0 + (int64_t)blockIdx.x * ROWS + threadIdx.x / LANES;
    if (row >= p.a.m) return;   // (all lanes of a row together)
    const int64_t k0 = 8 * (threadIdx.x % LANES);
    float v[NC][8];
#pragma unroll
    for (int c = 0; c < NC; ++c) norm_load(p, row, k0 + c * STEP, v[c]);
    double sum = 0.0;
    auto take = [&](int64_t k, const float (&x)[8]) {
        if (p.a.S && k < p.a.d) put8(p.a.S, row, p.a.d, k, p.a.bf16, p.vec, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += (double)x[e] * (double)x[e];
    };
#pragma unroll
    for (int c = 0; c < NC; ++c) take(k0 + c * STEP, v[c]);
    for (int64_t k = k0 + NC * STEP; k < p.a.d; k += STEP) {
        float x[8];
        norm_load(p, row, k, x);
        take(k, x);
    }
    const double q = sqrt(row_sum<LANES>(sum, lds) / (double)p.a.d + p.a.eps), r = 1.0 / q;
#pragma unroll
    for (int c = 0; c < NC; ++c)
        if (k0 + c * STEP < p.padded) norm_store<MX>(p, row, k0 + c * STEP, q, r, v[c]);
    for (int64_t k = k0 + NC * STEP; k < p.padded; k += STEP) {
        float x[8];
        if (p.a.S)   // (the inputs may be S itself, which holds the sums by now)
            mx_ld8(p.a.S, row, p.a.d, k, p.a.bf16, p.vec, x);
        else
            norm_load(p, row, k, x);
        norm_store<MX>(p, row, k, q, r, x);
    }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
struct NormBackArgs {
    RmsNormBackward a;
    int vec;
    double inv_d;
    float *part;                // [groups][d] the groups' sums of dw, or NULL
    double *stats;              // [m][2] r and r c of wide rows
    int64_t row0;               // the first row whose factors a launch finds
    int64_t groups;
};

// eight values as they lie in memory, zeros past the row's end
template <bool BF16>
struct Raw8 {
    u32x4 q[BF16 ? 1 : 2];
    __device__ __forceinline__ void load(const void *x, int64_t row, int64_t d, int64_t k, int vec) {
        if (vec) {
            const bool in = k < d;
            const u32x4 *src = (const u32x4 *)((const char *)x + (in ? row * d + k : 0) * (BF16 ? 2 : 4));
#pragma unroll
            for (int i = 0; i < (BF16 ? 1 : 2); ++i) q[i] = in ? src[i] : u32x4{0u, 0u, 0u, 0u};
        } else {   // (clamped and selected: a branch around each load would wait for each)
            unsigned v[8];
            const char *base = (const char *)x + row * d * (BF16 ? 2 : 4);   // (and 32-bit offsets: eight
#pragma unroll                                                              //  addresses cost 16 registers)
            for (int e = 0; e < 8; ++e) {
                const unsigned o = std::min((unsigned)k + e, (unsigned)d - 1u);
                if constexpr (BF16)
                    v[e] = ((const uint16_t *)base)[o];
                else
                    v[e] = ((const unsigned *)base)[o];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = k + e < d ? v[e] : 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (BF16) {
                    q[0][i] = v[2 * i] | v[2 * i + 1] << 16;
                } else {
                    q[0][i] = v[i];
                    q[BF16 ? 0 : 1][i] = v[4 + i];
                }
            }
        }
    }
    __device__ __forceinline__ void opaque() {   // nothing computed from it is kept from before
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); ++i) asm volatile("" : "+v"(q[i]));
    }
    __device__ __forceinline__ float at(int e) const {
        if constexpr (BF16)
            return __builtin_bit_cast(float, (e & 1) ? q[0][e >> 1] & 0xffff0000u : q[0][e >> 1] << 16);
        return __builtin_bit_cast(float, +q[BF16 ? 0 : e >> 2][e & 3]);   // (of a value: of an element in place it takes the first)
    }
};

// a row's contribution to sum S^2 and sum dY w S, in 64 bits: squares of large
// values stay finite, and c keeps its digits where its terms cancel
template <bool BF16>
__device__ __forceinline__ void norm_sums(const Raw8<BF16> &s, const Raw8<BF16> &g, const Raw8<BF16> &w, double &sq,
                                          double &dot) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const double v = (double)s.at(e);
        sq += v * v;
        dot += v * ((double)g.at(e) * (double)w.at(e));
    }
}
// Eight columns of a row: dX = r (w dY - (S r) (r c)) + dS, and dw's terms.  In 64
// bits but for dS's addition: of rows of very large or small values r, r^2 c or w dY
// leave fp32's range where dX does not.  (us a call, in fp32 throughout / so: bf16 4096 x
// 4096 30.0 / 30.6, 64000 x 128 36 / 43; f32 2048 x 8192 51 / 54, 4096 x 4099 159 / 186.)
template <bool BF16>
__device__ __forceinline__ void norm_leave(const NormBackArgs &p, int64_t row, int64_t k, double r, double rc,
                                           const Raw8<BF16> &s, const Raw8<BF16> &g, const Raw8<BF16> &w,
                                           const Raw8<BF16> &t, double (&dw)[8]) {
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const double n = (double)s.at(e) * r;
        x[e] = (float)(r * ((double)g.at(e) * (double)w.at(e) - n * rc)) + t.at(e);
        dw[e] += (double)g.at(e) * n;   // (in fp32 a long chain of rows would lose its small terms)
    }
    put8(p.a.dX, row, p.a.d, k, BF16, p.vec, x);
}
__device__ __forceinline__ void norm_factors(const NormBackArgs &p, double sq, double dot, double &r, double &rc) {
    r = 1.0 / sqrt(sq * p.inv_d + p.a.eps);
    rc = r * (dot * p.inv_d);
}
__device__ __forceinline__ void norm_put_sums(const NormBackArgs &p, int64_t group, int64_t k, const double (&dw)[8]) {
    if (!p.part || k >= p.a.d) return;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (float)dw[e];
    put8(p.part, group, p.a.d, k, 0, p.a.d % 4 == 0 && k + 8 <= p.a.d, v);
}

// Rows that fit a group of WPR waves, eight columns a thread: read once.  A
// group takes every groups-th row, the next one's loads in flight behind the
// present one's sums; the weights and its sums of dw stay in registers.
template <int WPR, bool BF16, bool VEC>
__global__ __launch_bounds__(WPR < 4 ? 256 : 64 * WPR) void rms_norm_backward_kernel(NormBackArgs p) {
    p.vec = VEC;
    constexpr int PER = WPR < 4 ? 4 / WPR : 1;   // groups of a block
    __shared__ double lds[2][PER][2][WPR];
    const int sub = threadIdx.x / (64 * WPR), tid = threadIdx.x % (64 * WPR);
    const int64_t group = (int64_t)blockIdx.x * PER + (PER > 1 ? sub : 0), d = p.a.d, k = 8 * tid;
    Raw8<BF16> w, s, g, t, s1, g1, t1;
    w.load(p.a.weight, 0, d, k, p.vec);
    auto load = [&](int64_t row) {
        row = std::min(row, p.a.m - 1);
        s1.load(p.a.S, row, d, k, p.vec);
        g1.load(p.a.dY, row, d, k, p.vec);
        if (p.a.dS) t1.load(p.a.dS, row, d, k, p.vec);
    };
#pragma unroll
    for (int i = 0; i < (BF16 ? 1 : 2); ++i) t1.q[i] = u32x4{0u, 0u, 0u, 0u};
    double dw[8] = {};
    load(group);
    int turn = 0;
    // (every group of a block makes the same number of turns: they meet at the barriers)
    for (int64_t first = (int64_t)blockIdx.x * PER; first < p.a.m; first += p.groups, turn ^= 1) {
        const int64_t row = first + (PER > 1 ? sub : 0);
        s = s1;
        g = g1;
        t = t1;
        w.opaque();   // (its 64-bit values, kept over the loop, would cost a third of the registers)
        load(row + p.groups);
        double sq = 0.0, dot = 0.0;
        norm_sums(s, g, w, sq, dot);
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
            sq += __shfl_xor(sq, o);
            dot += __shfl_xor(dot, o);
        }
        if constexpr (WPR > 1) {   // (two buffers in turn: one barrier a row)
            if ((tid & 63) == 0) {
                lds[turn][sub][0][tid >> 6] = sq;
                lds[turn][sub][1][tid >> 6] = dot;
            }
            __syncthreads();
            sq = lds[turn][sub][0][0];
            dot = lds[turn][sub][1][0];
#pragma unroll
            for (int i = 1; i < WPR; ++i) {
                sq += lds[turn][sub][0][i];
                dot += lds[turn][sub][1][i];
            }
        }
        double r, rc;
        norm_factors(p, sq, dot, r, rc);
        if (row < p.a.m && k < d) norm_leave(p, row, k, r, rc, s, g, w, t, dw);
    }
    if (group < p.groups) norm_put_sums(p, group, k, dw);
}

// Wider rows: their factors first ...
template <bool BF16, bool VEC>
__global__ __launch_bounds__(1024) void norm_factors_kernel(NormBackArgs p) {
    p.vec = VEC;
    __shared__ double lds[2][16];
    const int64_t row = p.row0 + blockIdx.x, d = p.a.d;
    double sq = 0.0, dot = 0.0;
    for (int64_t k = 8 * threadIdx.x; k < d; k += 8 * 1024) {
        Raw8<BF16> s, g, w;
        s.load(p.a.S, row, d, k, p.vec);
        g.load(p.a.dY, row, d, k, p.vec);
        w.load(p.a.weight, 0, d, k, p.vec);
        norm_sums(s, g, w, sq, dot);
    }
    sq = row_sum<1024>(sq, lds[0]);
    dot = row_sum<1024>(dot, lds[1]);
    if (threadIdx.x == 0) norm_factors(p, sq, dot, p.stats[2 * row], p.stats[2 * row + 1]);
}
// ... then 2048 columns of every groups-th row to a block
template <bool BF16, bool VEC>
__global__ __launch_bounds__(256) void norm_columns_kernel(NormBackArgs p) {
    p.vec = VEC;
    const int64_t k = (int64_t)blockIdx.x * 2048 + 8 * threadIdx.x, group = blockIdx.y, d = p.a.d;
    if (k >= d) return;
    Raw8<BF16> w;
    w.load(p.a.weight, 0, d, k, p.vec);
    double dw[8] = {};
#pragma unroll 2
    for (int64_t row = group; row < p.a.m; row += p.groups) {
        Raw8<BF16> s, g, t;
        s.load(p.a.S, row, d, k, p.vec);
        g.load(p.a.dY, row, d, k, p.vec);
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); ++i) t.q[i] = u32x4{0u, 0u, 0u, 0u};
        if (p.a.dS) t.load(p.a.dS, row, d, k, p.vec);
        norm_leave(p, row, k, p.stats[2 * row], p.stats[2 * row + 1], s, g, w, t, dw);
    }
    norm_put_sums(p, group, k, dw);
}

// Few rows of whole pieces of eight: one launch.  A block takes 512 columns and
// finds every row's factors by itself, a wave per row; the waves' terms of dw
// meet in LDS.  us a call from Python, this / two launches: bf16 1 x 4096 8.3 /
// 11.8, 16 x 4096 10.7 / 11.6; beyond, the blocks' repeated reads cost more: fp32 46 x
// 1408 14.8 / 12, rows that are not whole pieces (16 x 1407) 47 / 12.
constexpr int SMALL_ROWS = 16, SMALL_COLS = 4096;
template <bool BF16>
__global__ __launch_bounds__(64 * SMALL_ROWS) void norm_backward_small_kernel(NormBackArgs p) {
    __shared__ float sums[SMALL_ROWS][512];
    const int lane = threadIdx.x & 63, row = threadIdx.x >> 6;
    const int64_t d = p.a.d, k0 = (int64_t)blockIdx.x * 512 + 8 * lane;
    double dw[8] = {};
    if (row < p.a.m) {
        Raw8<BF16> s, g, w, t;
        double sq = 0.0, dot = 0.0;
        for (int64_t k = 8 * lane; k < d; k += 512) {
            s.load(p.a.S, row, d, k, p.vec);
            g.load(p.a.dY, row, d, k, p.vec);
            w.load(p.a.weight, 0, d, k, p.vec);
            norm_sums(s, g, w, sq, dot);
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
            sq += __shfl_xor(sq, o);
            dot += __shfl_xor(dot, o);
        }
        double r, rc;
        norm_factors(p, sq, dot, r, rc);
        s.load(p.a.S, row, d, k0, p.vec);
        g.load(p.a.dY, row, d, k0, p.vec);
        w.load(p.a.weight, 0, d, k0, p.vec);
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); ++i) t.q[i] = u32x4{0u, 0u, 0u, 0u};
        if (p.a.dS) t.load(p.a.dS, row, d, k0, p.vec);
        if (k0 < d) norm_leave(p, row, k0, r, rc, s, g, w, t, dw);
    }
    if (!p.a.dweight) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[row][8 * lane + e] = (float)dw[e];
    __syncthreads();
    const int64_t k = (int64_t)blockIdx.x * 512 + threadIdx.x;
    if (threadIdx.x >= 512 || k >= d) return;
    double sum = 0.0;
    for (int i = 0; i < p.a.m; ++i) sum += (double)sums[i][threadIdx.x];
    p.a.dweight[k] = (float)sum;
}

// dw from the groups' sums: 32 columns of a block, 32 threads a column, each
// every 32nd group in turn, added in their order in 64 bits
__global__ __launch_bounds__(1024) void norm_weight_reduce_kernel(const float *part, int64_t groups, int64_t d,
                                                                  float *dw) {
    __shared__ double lds[1024];
    const int64_t k = (int64_t)blockIdx.x * 32 + (threadIdx.x & 31);
    double sum = 0.0;
    if (k < d)
#pragma unroll 8
        for (int64_t g = threadIdx.x >> 5; g < groups; g += 32) sum += (double)part[g * d + k];
    lds[threadIdx.x] = sum;
    __syncthreads();
    if (threadIdx.x >= 32 || k >= d) return;
    for (int i = 1; i < 32; ++i) sum += lds[32 * i + threadIdx.x];
    dw[k] = (float)sum;
}

bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Threads per row and pieces per thread.  Few rows: many threads (a row's latency
// counts); many: as many as hold it in a few pieces, so that a CU holds several
// rows.  us with a residual: 4096 x 4096 fp32 512 threads 45, 256 53, bf16 26, 27,
// and 1024 48; 64000 x 128 bf16 16 threads 13, 64 44.
struct RowPlan {
    int lanes, nc;
};
RowPlan row_plan(int64_t m, int64_t d) {
    if (d <= 128 && m >= 256) return {16, 1};
    if (d <= 2048 && m >= 256) return {64, d <= 512 ? 1 : d <= 1024 ? 2 : 4};
    if (d <= 8192 && m >= 256) return {512, d <= 4096 ? 1 : 2};
    return {1024, d <= 8192 ? 1 : d <= 16384 ? 2 : 4};
}
constexpr int64_t MAX_BLOCKS = 1 << 20;   // of a launch (which has less than 2^32 threads)
template <int LANES, int NC>
hipError_t launch_norm(NormArgs p, hipStream_t st) {
    constexpr int ROWS = std::max(1, 256 / LANES), THREADS = std::max(LANES, 256);
    for (p.row0 = 0; p.row0 < p.a.m; p.row0 += MAX_BLOCKS * ROWS) {
        const unsigned blocks = (unsigned)std::min(cdiv(p.a.m - p.row0, ROWS), MAX_BLOCKS);
        if (p.a.Y && p.vec)
            rms_norm_kernel<LANES, NC, true, false><<<blocks, THREADS, 0, st>>>(p);
        else if (p.a.Y)
            rms_norm_kernel<LANES, NC, false, false><<<blocks, THREADS, 0, st>>>(p);
        else if (p.vec)
            rms_norm_kernel<LANES, NC, true, true><<<blocks, THREADS, 0, st>>>(p);
        else
            rms_norm_kernel<LANES, NC, false, true><<<blocks, THREADS, 0, st>>>(p);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// The backward pass: waves of a group (0: rows wider than one group reads; -1:
// few rows), and the groups of rows that sum dw at once, multiples of a block's.
struct BackPlan {
    int wpr;
    int64_t groups;
};
constexpr int64_t NORM_WAVES = 4096;
BackPlan back_plan(int64_t m, int64_t d) {
    BackPlan p{1, 0};
    if (m <= SMALL_ROWS && d <= SMALL_COLS && d % 8 == 0) return {-1, 0};
    if (d > 8192) {
        p.wpr = 0;
        p.groups = std::min(m, std::max<int64_t>(1, 1024 / cdiv(d, 2048)));
        return p;
    }
    while (512 * p.wpr < d) p.wpr *= 2;
    const int64_t per = p.wpr < 4 ? 4 / p.wpr : 1;
    p.groups = std::min(cdiv(m, per) * per, NORM_WAVES / p.wpr);
    return p;
}
template <bool BF16, bool VEC>
hipError_t launch_backward(NormBackArgs p, int wpr, hipStream_t st) {
    const unsigned blocks = (unsigned)p.groups;
    switch (wpr) {
        case 1: rms_norm_backward_kernel<1, BF16, VEC><<<blocks / 4, 256, 0, st>>>(p); break;
        case 2: rms_norm_backward_kernel<2, BF16, VEC><<<blocks / 2, 256, 0, st>>>(p); break;
        case 4: rms_norm_backward_kernel<4, BF16, VEC><<<blocks, 256, 0, st>>>(p); break;
        case 8: rms_norm_backward_kernel<8, BF16, VEC><<<blocks, 512, 0, st>>>(p); break;
        case 16: rms_norm_backward_kernel<16, BF16, VEC><<<blocks, 1024, 0, st>>>(p); break;
        default: {
            for (p.row0 = 0; p.row0 < p.a.m; p.row0 += MAX_BLOCKS) {
                const unsigned rows = (unsigned)std::min(p.a.m - p.row0, MAX_BLOCKS);
                norm_factors_kernel<BF16, VEC><<<rows, 1024, 0, st>>>(p);
                const hipError_t e = hipGetLastError();
                if (e != hipSuccess) return e;
            }
            norm_columns_kernel<BF16, VEC><<<dim3((unsigned)cdiv(p.a.d, 2048), blocks), 256, 0, st>>>(p);
        }
    }
    return hipGetLastError();
}

}  // namespace

hipError_t rms_norm_launch(const RmsNorm &a, hipStream_t st) {
    NormArgs p{};
    p.a = a;
    p.vec = a.d % 8 == 0 && aligned16(a.X) && aligned16(a.weight) && (!a.residual || aligned16(a.residual)) &&
            (!a.S || aligned16(a.S)) && (!a.Y || aligned16(a.Y));
    p.padded = a.Y ? a.d : mx_steps(a.d) * MX_PAD;
    p.row_bytes = a.Y ? 0 : mx_row_bytes(a.d, a.fmt);
    const RowPlan plan = row_plan(a.m, a.d);
    switch (plan.lanes * 8 + plan.nc) {
        case 16 * 8 + 1: return launch_norm<16, 1>(p, st);
        case 64 * 8 + 1: return launch_norm<64, 1>(p, st);
        case 64 * 8 + 2: return launch_norm<64, 2>(p, st);
        case 64 * 8 + 4: return launch_norm<64, 4>(p, st);
        case 512 * 8 + 1: return launch_norm<512, 1>(p, st);
        case 512 * 8 + 2: return launch_norm<512, 2>(p, st);
        case 1024 * 8 + 1: return launch_norm<1024, 1>(p, st);
        case 1024 * 8 + 2: return launch_norm<1024, 2>(p, st);
        default: return launch_norm<1024, 4>(p, st);
    }
}

size_t rms_norm_backward_ws(int64_t m, int64_t d) {
    if (m == 0) return 0;
    const BackPlan p = back_plan(m, d);
    if (p.wpr < 0) return 0;
    return align256((size_t)p.groups * d * sizeof(float)) + (p.wpr ? 0 : align256((size_t)m * 2 * sizeof(double)));
}

hipError_t rms_norm_backward_launch(const RmsNormBackward &a, hipStream_t st) {
    NormBackArgs p{};
    p.a = a;
    p.vec = a.d % 8 == 0 && aligned16(a.dY) && aligned16(a.S) && aligned16(a.weight) && (!a.dS || aligned16(a.dS)) &&
            aligned16(a.dX);
    p.inv_d = 1.0 / (double)a.d;
    if (a.m > 0) {
        const BackPlan plan = back_plan(a.m, a.d);
        if (plan.wpr < 0) {
            const unsigned blocks = (unsigned)cdiv(a.d, 512);
            if (a.bf16)
                norm_backward_small_kernel<true><<<blocks, 64 * SMALL_ROWS, 0, st>>>(p);
            else
                norm_backward_small_kernel<false><<<blocks, 64 * SMALL_ROWS, 0, st>>>(p);
            return hipGetLastError();
        }
        p.groups = plan.groups;
        p.part = a.dweight ? (float *)a.ws : nullptr;
        p.stats = (double *)(a.ws + align256((size_t)p.groups * a.d * sizeof(float)));
        hipError_t e;
        if (p.vec)
            e = a.bf16 ? launch_backward<true, true>(p, plan.wpr, st) : launch_backward<false, true>(p, plan.wpr, st);
        else
            e = a.bf16 ? launch_backward<true, false>(p, plan.wpr, st) : launch_backward<false, false>(p, plan.wpr, st);
        if (e != hipSuccess) return e;
    }
    if (!a.dweight) return hipSuccess;
    norm_weight_reduce_kernel<<<(unsigned)cdiv(a.d, 32), 1024, 0, st>>>(p.part, p.groups, a.d, a.dweight);
    return hipGetLastError();
}

}  // namespace gptq
