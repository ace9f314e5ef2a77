// Fused products with packed layers: Y = act(A W_hat^T + bias) + residual,
// the gated pair H = act(A W_gate^T + b_gate) (A W_up^T + b_up), and the
// gradients of both with respect to the activations and the biases.
// "Optimization Gptq", "Backends de kernel" (kernels that run the quantized
// model on its packed weights); storage as in dequant.hip:
//   W_hat[r][perm[k]] = s[k/g][r] (q[r][k] - z[k/g][r]).
//
// First form: one lane per output column, eight activation rows per lane,
// fp32 sums over the whole contraction.
#include "common.h"

#include <algorithm>

namespace gptq {

namespace {

constexpr int ROWS = 8;   // activation rows per thread

__device__ __forceinline__ float ld(const void *p, int64_t i, int bf16) {
    if (bf16) return __builtin_bit_cast(float, (unsigned)((const uint16_t *)p)[i] << 16);
    return ((const float *)p)[i];
}
__device__ __forceinline__ void st(void *p, int64_t i, float v, int bf16) {
    if (bf16)
        ((__bf16 *)p)[i] = (__bf16)v;   // round to nearest even
    else
        ((float *)p)[i] = v;
}

__device__ __forceinline__ float sigmoidf(float x) { return 1.f / (1.f + expf(-x)); }

constexpr float SQRT_HALF = 0.70710678118654752f, INV_SQRT_2PI = 0.39894228040143268f;
constexpr float TWO_SQRT_2_PI = 1.5957691216057308f;   // 2 sqrt(2 / pi)

__device__ __forceinline__ float act_value(int act, float z) {
    switch (act) {
        case 1: return z < 0.f ? 0.f : z;
        case 2: return 0.5f * z * erfcf(-z * SQRT_HALF);
        case 3: return z * sigmoidf(TWO_SQRT_2_PI * (z + 0.044715f * z * z * z));
        case 4: return z * sigmoidf(z);
    }
    return z;
}

// (beyond |z| = 64 every slope is 0 or 1 in fp32: clamped there, so that no
// product of a vanishing and an overflowing factor arises; NaN stays NaN)
__device__ __forceinline__ float act_slope(int act, float z) {
    z = z > 64.f ? 64.f : (z < -64.f ? -64.f : z);
    switch (act) {
        case 1: return z > 0.f ? 1.f : 0.f;
        case 2: return 0.5f * erfcf(-z * SQRT_HALF) + z * INV_SQRT_2PI * expf(-0.5f * z * z);
        case 3: {
            const float u = TWO_SQRT_2_PI * (z + 0.044715f * z * z * z);
            const float p = sigmoidf(u);
            return p + z * p * sigmoidf(-u) * TWO_SQRT_2_PI * (1.f + 3.f * 0.044715f * z * z);
        }
        case 4: {
            const float p = sigmoidf(z);
            return p + z * p * sigmoidf(-z);
        }
    }
    return 1.f;
}

__device__ __forceinline__ float weight(const PackedLayer &w, int64_t d_out, int bits, int g, int64_t k, int64_t r) {
    const int64_t pos = bits * k, j = pos >> 5;
    const int sh = (int)(pos & 31);
    uint64_t v = w.Q[j * d_out + r];
    if (sh + bits > 32) v |= (uint64_t)w.Q[(j + 1) * d_out + r] << 32;
    const float q = (float)(unsigned)((v >> sh) & ((1u << bits) - 1u));
    return w.scales[k / g * d_out + r] * (q - w.zeros[k / g * d_out + r]);
}

__global__ __launch_bounds__(256) void fused_forward_kernel(FusedForward a) {
    const FusedShape &s = a.s;
    const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (n >= s.d_out) return;
    for (int64_t i0 = (int64_t)blockIdx.y * ROWS; i0 < s.m; i0 += (int64_t)gridDim.y * ROWS) {
        float z[2][ROWS] = {};
        for (int64_t k = 0; k < s.d_in; ++k) {
            const int64_t c = a.perm ? a.perm[k] : k;
            float w[2] = {0.f, 0.f};
            for (int l = 0; l < s.layers; ++l) w[l] = weight(a.w[l], s.d_out, s.bits, s.group, k, n);
            for (int e = 0; e < ROWS; ++e) {
                const float x = i0 + e < s.m ? ld(a.A, (i0 + e) * s.d_in + c, s.in_bf16) : 0.f;
                z[0][e] = fmaf(x, w[0], z[0][e]);
                z[1][e] = fmaf(x, w[1], z[1][e]);
            }
        }
        for (int e = 0; e < ROWS && i0 + e < s.m; ++e) {
            const int64_t o = (i0 + e) * s.d_out + n;
            for (int l = 0; l < s.layers; ++l) {
                if (a.bias[l]) z[l][e] += ld(a.bias[l], n, a.bias_bf16);
                if (a.pre[l]) st(a.pre[l], o, z[l][e], s.out_bf16);
            }
            float y = act_value(a.act, z[0][e]);
            if (s.layers == 2) y *= z[1][e];
            if (a.residual) y += ld(a.residual, o, s.out_bf16);
            st(a.Y, o, y, s.out_bf16);
        }
    }
}

// dZ of layer l at element o
__device__ __forceinline__ float grad(const FusedBackward &a, int l, int64_t o) {
    const float dy = ld(a.dY, o, a.s.in_bf16);
    if (a.s.layers == 1) return a.act ? dy * act_slope(a.act, ld(a.pre[0], o, a.s.in_bf16)) : dy;
    const float zg = ld(a.pre[0], o, a.s.in_bf16);
    return l ? dy * act_value(a.act, zg) : dy * ld(a.pre[1], o, a.s.in_bf16) * act_slope(a.act, zg);
}

__global__ __launch_bounds__(256) void fused_backward_kernel(FusedBackward a) {
    const FusedShape &s = a.s;
    const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (k >= s.d_in) return;
    for (int64_t i0 = (int64_t)blockIdx.y * ROWS; i0 < s.m; i0 += (int64_t)gridDim.y * ROWS) {
        float d[ROWS] = {};
        for (int l = 0; l < s.layers; ++l)
            for (int64_t r = 0; r < s.d_out; ++r) {
                const float w = weight(a.w[l], s.d_out, s.bits, s.group, k, r);
                for (int e = 0; e < ROWS; ++e)
                    d[e] = fmaf(i0 + e < s.m ? grad(a, l, (i0 + e) * s.d_out + r) : 0.f, w, d[e]);
            }
        const int64_t c = a.perm ? a.perm[k] : k;
        for (int e = 0; e < ROWS && i0 + e < s.m; ++e) st(a.dA, (i0 + e) * s.d_in + c, d[e], s.out_bf16);
    }
}

__global__ __launch_bounds__(256) void fused_bias_grad_kernel(FusedBackward a) {
    const int64_t r = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int l = blockIdx.y;
    if (r >= a.s.d_out || !a.dbias[l]) return;
    float v = 0.f;
    for (int64_t i = 0; i < a.s.m; ++i) v += grad(a, l, i * a.s.d_out + r);
    a.dbias[l][r] = v;
}

unsigned row_blocks(int64_t m) { return (unsigned)std::min<int64_t>(cdiv(m, ROWS), 65535); }

}  // namespace

size_t fused_forward_ws(const FusedShape &s) { return 0; }
size_t fused_backward_ws(const FusedShape &s) { return 0; }

hipError_t fused_forward_launch(const FusedForward &a, hipStream_t st) {
    fused_forward_kernel<<<dim3((unsigned)cdiv(a.s.d_out, 256), row_blocks(a.s.m)), 256, 0, st>>>(a);
    return hipGetLastError();
}

hipError_t fused_backward_launch(const FusedBackward &a, hipStream_t st) {
    if (a.s.m > 0) {
        fused_backward_kernel<<<dim3((unsigned)cdiv(a.s.d_in, 256), row_blocks(a.s.m)), 256, 0, st>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (!a.dbias[0] && !a.dbias[1]) return hipSuccess;
    fused_bias_grad_kernel<<<dim3((unsigned)cdiv(a.s.d_out, 256), (unsigned)a.s.layers), 256, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace gptq
