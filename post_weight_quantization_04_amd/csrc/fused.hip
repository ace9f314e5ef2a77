// Fused products with packed layers: Y = act(A W_hat^T + bias) + residual,
// the gated pair H = act(A W_gate^T + b_gate) (A W_up^T + b_up), and the
// gradients of both with respect to the activations and the biases.
// "Optimization Gptq", "Backends de kernel" (kernels that run the quantized
// model on its packed weights); storage as in dequant.hip:
//   W_hat[r][perm[k]] = s[k/g][r] (q[r][k] - z[k/g][r]).
//
// Two forms.  Few activation rows (fused_skinny.hip): one pass over the packed
// words, bound by reading and converting them.  Many rows (fused_gemm.hip):
// the weights dequantized once into the workspace, bound by the matrix cores.
// Where they meet, per call from Python, packed / dense, at 4096 x 4096, 4 bits,
// groups of 128: forward 64 rows 18 / 32 us, 128 rows 32 / 33, 129 rows 36 / 35,
// 192 rows 46 / 36 (11008 x 4096, 3 bits: 128 rows 63 / 73, 192 rows 105 / 78);
// fp32 activations 16 rows 12.6 / 42; backward 16 rows 19 / 31, fp32 20 / 45.
#include "fused.h"

#include <algorithm>

namespace gptq {

namespace {

__global__ __launch_bounds__(256) void zero_kernel(float *a, float *b, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n && a) a[i] = 0.f;
    if (i < n && b) b[i] = 0.f;
}

}  // namespace

size_t fused_forward_ws(const FusedShape &s) {
    if (s.m == 0) return 0;
    return skinny_forward_takes(s) ? skinny_forward_ws(s) : dense_forward_ws(s);
}
size_t fused_backward_ws(const FusedShape &s) {
    if (s.m == 0) return 0;
    return skinny_backward_takes(s) ? skinny_backward_ws(s) : dense_backward_ws(s);
}

hipError_t fused_forward_launch(const FusedForward &a, hipStream_t st) {
    return skinny_forward_takes(a.s) ? skinny_forward_launch(a, st) : dense_forward_launch(a, st);
}

hipError_t fused_backward_launch(const FusedBackward &a, hipStream_t st) {
    if (a.s.m == 0) {
        if (!a.dbias[0] && !a.dbias[1]) return hipSuccess;
        zero_kernel<<<(unsigned)cdiv(a.s.d_out, 256), 256, 0, st>>>(a.dbias[0], a.dbias[1], a.s.d_out);
        return hipGetLastError();
    }
    return skinny_backward_takes(a.s) ? skinny_backward_launch(a, st) : dense_backward_launch(a, st);
}

}  // namespace gptq
