// Root-mean-square norm of the residual stream in front of a projection, with
// the residual's addition and an output that may be quantized to an MX format
// on the way, and its backward pass.
//
//   S = X + residual, rounded to its type;  r = (mean_j S_j^2 + eps)^(-1/2)
//   Y_j = S_j r w_j
//   c = mean_j dY_j w_j S_j;  dX_j = r (w_j dY_j - S_j r^2 c) + dS_j
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

// Sums over the threads of a row: WPR waves (4 / WPR rows of a block where
// WPR is 1).  Fixed order: lanes by halves, then waves in turn.
template <int WPR, class T>
__device__ __forceinline__ T row_sum(T v, T *lds) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    if constexpr (WPR > 1) {
        const int wave = threadIdx.x >> 6;
        __syncthreads();   // (the sums of the row before have been read)
        if ((threadIdx.x & 63) == 0) lds[wave] = v;
        __syncthreads();
        v = lds[0];
#pragma unroll
        for (int w = 1; w < WPR; ++w) v += lds[w];
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
    double inv_d;
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
        fz_st4(x, o, f32x4{v[0], v[1], v[2], v[3]}, bf16);
        fz_st4(x, o + 4, f32x4{v[4], v[5], v[6], v[7]}, bf16);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (k + e < d) fz_st(x, o + e, v[e], bf16);
    }
}
// Y = S w r in 64 bits (S w is exact there), rounded once to its type or its
// grid: a value next to a border of a grid of 8 or 4 bits falls on the side
// the definition says.  The 64-bit operations hide behind the memory.
__device__ __forceinline__ void norm_store(const NormArgs &p, int64_t row, int64_t k, double r, const float (&v)[8]) {
    float w[8], y[8];
    mx_ld8(p.a.weight, 0, p.a.d, k, p.a.bf16, p.vec, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = mx_odd((double)v[e] * (double)w[e] * r);
    if (p.a.Y) {
        if (!p.a.bf16) {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = (float)((double)v[e] * (double)w[e] * r);
        }
        put8(p.a.Y, row, p.a.d, k, p.a.bf16, p.vec, y);
    } else if (p.a.fmt == MX_FP8) {
        mx_put8<MX_FP8>(y, p.a.m, row, k >> 3, p.row_bytes, p.a.codes, p.a.scales);
    } else {
        mx_put8<MX_FP4>(y, p.a.m, row, k >> 3, p.row_bytes, p.a.codes, p.a.scales);
    }
}

// WPR waves per row, each thread NC pieces of eight columns held in registers
// between the two sweeps; columns beyond them are formed again from the inputs
template <int WPR, int NC>
__global__ __launch_bounds__(WPR == 1 ? 256 : 64 * WPR) void rms_norm_kernel(NormArgs p) {
    constexpr int STEP = 512 * WPR;
    __shared__ double lds[WPR];
    const int64_t row = WPR == 1 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : (int64_t)blockIdx.x;
    if (row >= p.a.m) return;   // (whole waves, and whole blocks where they meet at barriers)
    const int64_t k0 = 8 * (WPR == 1 ? threadIdx.x & 63 : threadIdx.x);
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
    const double r = 1.0 / sqrt(row_sum<WPR>(sum, lds) * p.inv_d + p.a.eps);
#pragma unroll
    for (int c = 0; c < NC; ++c)
        if (k0 + c * STEP < p.padded) norm_store(p, row, k0 + c * STEP, r, v[c]);
    for (int64_t k = k0 + NC * STEP; k < p.padded; k += STEP) {
        float x[8];
        if (p.a.S)   // (the inputs may be S itself, which holds the sums by now)
            mx_ld8(p.a.S, row, p.a.d, k, p.a.bf16, p.vec, x);
        else
            norm_load(p, row, k, x);
        norm_store(p, row, k, r, x);
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
    int64_t groups;
};

// A group (WPR waves) takes every groups-th row.  The weights and the group's
// sums of dw stay in registers, NC pieces of eight columns a thread; columns
// beyond them go through memory (their sums in the group's own row of `part`).
template <int WPR, int NC>
__global__ __launch_bounds__(WPR == 1 ? 256 : 64 * WPR) void rms_norm_backward_kernel(NormBackArgs p) {
    constexpr int STEP = 512 * WPR;
    __shared__ double lds[2 * WPR];
    const int64_t group = WPR == 1 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : (int64_t)blockIdx.x;
    if (group >= p.groups) return;
    const int64_t k0 = 8 * (WPR == 1 ? threadIdx.x & 63 : threadIdx.x), d = p.a.d;
    const int bf16 = p.a.bf16;
    float w[NC][8], dw[NC][8] = {};
#pragma unroll
    for (int c = 0; c < NC; ++c) mx_ld8(p.a.weight, 0, d, k0 + c * STEP, bf16, p.vec, w[c]);
    for (int64_t row = group; row < p.a.m; row += p.groups) {
        float s[NC][8], g[NC][8];
        double dot = 0.0, sq = 0.0;   // (64 bits: squares of large values stay finite)
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            mx_ld8(p.a.S, row, d, k0 + c * STEP, bf16, p.vec, s[c]);
            mx_ld8(p.a.dY, row, d, k0 + c * STEP, bf16, p.vec, g[c]);
        }
        auto take = [&](const float (&s)[8], const float (&g)[8], const float (&w)[8]) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                sq += (double)s[e] * (double)s[e];
                dot += (double)s[e] * (double)g[e] * (double)w[e];
            }
        };
#pragma unroll
        for (int c = 0; c < NC; ++c) take(s[c], g[c], w[c]);
        for (int64_t k = k0 + NC * STEP; k < d; k += STEP) {
            float s1[8], g1[8], w1[8];
            mx_ld8(p.a.S, row, d, k, bf16, p.vec, s1);
            mx_ld8(p.a.dY, row, d, k, bf16, p.vec, g1);
            mx_ld8(p.a.weight, 0, d, k, bf16, p.vec, w1);
            take(s1, g1, w1);
        }
        sq = row_sum<WPR>(sq, lds);
        dot = row_sum<WPR>(dot, lds + (WPR > 1 ? WPR : 0));
        const double rd = 1.0 / sqrt(sq * p.inv_d + p.a.eps);
        const float r = (float)rd, f = (float)(rd * rd * (dot * p.inv_d));
        auto leave = [&](int64_t k, const float (&s)[8], const float (&g)[8], const float (&w)[8], float (&dw)[8]) {
            float x[8], t[8] = {};
            if (p.a.dS) mx_ld8(p.a.dS, row, d, k, bf16, p.vec, t);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[e] = r * (g[e] * w[e] - s[e] * f) + t[e];
                dw[e] += g[e] * (s[e] * r);
            }
            put8(p.a.dX, row, d, k, bf16, p.vec, x);
        };
#pragma unroll
        for (int c = 0; c < NC; ++c)
            if (k0 + c * STEP < d) leave(k0 + c * STEP, s[c], g[c], w[c], dw[c]);
        for (int64_t k = k0 + NC * STEP; k < d; k += STEP) {
            float s1[8], g1[8], w1[8], dw1[8] = {};
            mx_ld8(p.a.S, row, d, k, bf16, p.vec, s1);
            mx_ld8(p.a.dY, row, d, k, bf16, p.vec, g1);
            mx_ld8(p.a.weight, 0, d, k, bf16, p.vec, w1);
            if (p.part && row != group) mx_ld8(p.part, group, d, k, 0, 0, dw1);
            leave(k, s1, g1, w1, dw1);
            if (p.part) put8(p.part, group, d, k, 0, 0, dw1);
        }
    }
    if (p.part)
#pragma unroll
        for (int c = 0; c < NC; ++c)
            if (k0 + c * STEP < d) put8(p.part, group, d, k0 + c * STEP, 0, d % 4 == 0 && k0 + c * STEP + 8 <= d, dw[c]);
}

// dw from the groups' sums: 32 columns of a block, eight threads a column, each
// every eighth group in turn, added in their order in 64 bits
__global__ __launch_bounds__(256) void norm_weight_reduce_kernel(const float *part, int64_t groups, int64_t d,
                                                                 float *dw) {
    __shared__ double lds[256];
    const int64_t k = (int64_t)blockIdx.x * 32 + (threadIdx.x & 31);
    double sum = 0.0;
    if (k < d)
#pragma unroll 8
        for (int64_t g = threadIdx.x >> 5; g < groups; g += 8) sum += (double)part[g * d + k];
    lds[threadIdx.x] = sum;
    __syncthreads();
    if (threadIdx.x >= 32 || k >= d) return;
    for (int i = 1; i < 8; ++i) sum += lds[32 * i + threadIdx.x];
    dw[k] = (float)sum;
}

bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Pieces per thread and waves per row.  Few rows: many waves (a row's latency
// counts); many: one or four, so that a CU holds several rows.
struct RowPlan {
    int wpr, nc;
};
RowPlan row_plan(int64_t m, int64_t d) {
    if (d <= 2048 && m >= 256) return {1, d <= 512 ? 1 : d <= 1024 ? 2 : 4};
    if (d <= 8192 && m >= 256) return {4, d <= 2048 ? 1 : d <= 4096 ? 2 : 4};
    return {16, d <= 8192 ? 1 : d <= 16384 ? 2 : 4};
}
template <class F>
hipError_t with_plan(const RowPlan &p, F f) {
    using std::integral_constant;
    auto waves = [&](auto w) {
        switch (p.nc) {
            case 1: f(w, integral_constant<int, 1>{}); break;
            case 2: f(w, integral_constant<int, 2>{}); break;
            default: f(w, integral_constant<int, 4>{}); break;
        }
    };
    switch (p.wpr) {
        case 1: waves(integral_constant<int, 1>{}); break;
        case 4: waves(integral_constant<int, 4>{}); break;
        default: waves(integral_constant<int, 16>{}); break;
    }
    return hipGetLastError();
}

constexpr int64_t NORM_GROUPS = 512;   // groups of rows that sum dw at once
int64_t norm_groups(int64_t m, const RowPlan &p) {
    return std::min<int64_t>(m, p.wpr == 1 ? 4 * NORM_GROUPS : NORM_GROUPS);
}

}  // namespace

hipError_t rms_norm_launch(const RmsNorm &a, hipStream_t st) {
    NormArgs p{};
    p.a = a;
    p.vec = a.d % 8 == 0 && aligned16(a.X) && aligned16(a.weight) && (!a.residual || aligned16(a.residual)) &&
            (!a.S || aligned16(a.S)) && (!a.Y || aligned16(a.Y));
    p.padded = a.Y ? a.d : mx_steps(a.d) * MX_PAD;
    p.row_bytes = a.Y ? 0 : mx_row_bytes(a.d, a.fmt);
    p.inv_d = 1.0 / (double)a.d;
    const RowPlan plan = row_plan(a.m, a.d);
    return with_plan(plan, [&](auto w, auto n) {
        constexpr int W = decltype(w)::value, N = decltype(n)::value;
        const unsigned blocks = (unsigned)(W == 1 ? cdiv(a.m, 4) : a.m);
        rms_norm_kernel<W, N><<<blocks, W == 1 ? 256 : 64 * W, 0, st>>>(p);
    });
}

size_t rms_norm_backward_ws(int64_t m, int64_t d) {
    return m == 0 ? 0 : align256((size_t)norm_groups(m, row_plan(m, d)) * d * sizeof(float));
}

hipError_t rms_norm_backward_launch(const RmsNormBackward &a, hipStream_t st) {
    NormBackArgs p{};
    p.a = a;
    p.vec = a.d % 8 == 0 && aligned16(a.dY) && aligned16(a.S) && aligned16(a.weight) && (!a.dS || aligned16(a.dS)) &&
            aligned16(a.dX);
    p.inv_d = 1.0 / (double)a.d;
    p.part = a.dweight ? (float *)a.ws : nullptr;
    const RowPlan plan = row_plan(a.m, a.d);
    p.groups = norm_groups(a.m, plan);
    if (a.m > 0) {
        const hipError_t e = with_plan(plan, [&](auto w, auto n) {
            constexpr int W = decltype(w)::value, N = decltype(n)::value;
            const unsigned blocks = (unsigned)(W == 1 ? cdiv(p.groups, 4) : p.groups);
            rms_norm_backward_kernel<W, N><<<blocks, W == 1 ? 256 : 64 * W, 0, st>>>(p);
        });
        if (e != hipSuccess || !a.dweight) return e;
    }
    if (!a.dweight) return hipSuccess;
    norm_weight_reduce_kernel<<<(unsigned)cdiv(a.d, 32), 256, 0, st>>>(p.part, a.m > 0 ? p.groups : 0, a.d, a.dweight);
    return hipGetLastError();
}

}  // namespace gptq
