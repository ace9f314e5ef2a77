// Products of MX activations (8 or 4 bits) with MX weights in 4 bits, many
// rows, on the scaled matrix cores: codes and scale bytes enter the MFMAs as
// they lie in memory, no value is ever converted.
//
// The 32 x 32 x 64 scaled MFMA takes two blocks of the contraction, one scale
// byte each: lane l supplies row l % 32, an e2m1 operand block l / 32 whole, an
// e4m3 operand bytes 16 (l / 32) .. of both blocks; the scale of block b comes
// from the lanes of half b.  A stage of 128 columns holds four blocks; the
// s-th of its two MFMAs takes blocks s and 2 + s, so that a lane's two scale
// bytes lie side by side and the MFMA selects one by its immediate.
//
// Measured, us a call without an activation: fp8 2048 rows by 28672 outputs of K =
// 8192 360 (2.67 PFLOP/s; 4096 rows 2.90), a large library product of two fp8
// operands 2.73; the matrix cores busy 59% of the cycles at 1.8 GHz, the clock under
// that load.  fp4 4096 rows by 11008 outputs: K = 16384 365 (4.05 PFLOP/s), K = 4096
// 113-116 (3.2; 142 with silu and a second output, which the epilogues write).
//
// Precision.  Products of two e2m1 operands add exactly into fp32.  With an e4m3
// operand the MFMA aligns a group's products to the largest and keeps about 14
// bits below it (measured: 2^-15 to 2^-14 of the sum of magnitudes, for any
// length).  A BF16 result, which rounds at 2^-9, is as far from the 64-bit one as
// with fp32 sums (1.7e-3 of its norm both; 2-3e-4 apart, as a few values in a hundred
// cross a rounding border), for twice the 16-bit rate and no conversion.  An F32
// result of fp8 activations is formed on the 16-bit matrix cores instead (the dense
// form of the fused products, mx_skinny.hip), where both operands are exact.
#include "mx.h"

#include <algorithm>

namespace gptq {

namespace {

typedef __attribute__((ext_vector_type(8))) int i32x8;

struct MxGemm {
    MxMatrix a, w;
    int64_t m, n;
    int64_t a_bytes, w_bytes;   // code bytes of a row
    int steps;                  // stages of the contraction
    MxEpilogue out;
    float *part;                // [nsplit][m][np] when nsplit > 1
    int64_t np;                 // n padded to whole eights
    int nsplit;
    int mt, nt;                 // tiles
};

// The 16-byte piece of a 64-byte (e2m1) or 128-byte (e4m3) row at which piece 0
// lies: the 16 lanes that a b128 read serves together (0-3, 12-15, 20-23, 24-27 and
// their complements) then meet 16 different pieces of 256 bytes.  (row & 7 for
// e4m3: a third of the LDS cycles were conflicts, in the same time, which the
// clock under load sets.)
__device__ __forceinline__ int swz4(int row) { return ((row >> 1) & 3) ^ ((row >> 3) & 1); }
__device__ __forceinline__ int swz8(int row) { return ((row >> 1) & 1) | (((row >> 3) & 3) << 1); }

// C tile of 64 NJ outputs by 64 MI rows, four waves of 32 NJ by 32 MI.  Both
// operands' codes and scales move by buffer loads straight into a ring of LDS
// stages of 128 columns; the wait for a stage counts loads, so the later stages
// stay in flight across the one barrier per stage.  Each MFMA group runs beside
// the operand reads of the next and half of a refill.
template <int FA, int MI, int NJ, int NBUF>
__global__ __launch_bounds__(256, MI * NJ == 16 ? 1 : 2) void mx_gemm_kernel(MxGemm p) {
    constexpr int BM = 64 * MI, BN = 64 * NJ;
    constexpr int AROW = FA == MX_FP4 ? 64 : 128, AQ = AROW / 64;     // bytes of a row's stage, reads of a fragment
    constexpr int WSIDE = BN * 64, ASIDE = BM * AROW, SSIDE = (BM + BN) * 4;
    constexpr int STAGE = WSIDE + ASIDE + SSIDE;
    constexpr int WDMA = NJ, ADMA = AQ * MI, SDMA = (MI + NJ) / 4;    // loads per wave and stage
    constexpr int PER_STAGE = WDMA + ADMA + SDMA;
    constexpr int EROW = 32 * NJ + 4;                                 // floats of an epilogue row (padded)
    __shared__ __attribute__((aligned(16))) char lds[std::max(NBUF * STAGE, 4 * 64 * EROW * 4)];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wn = wave >> 1, wm = wave & 1;
    const int h = lane >> 5, li = lane & 31;

    // each XCD takes a contiguous run of tiles, ordered in strips of four tiles
    // n by all tiles m
    const int total = p.mt * p.nt * p.nsplit;
    const int q8 = total / 8, r8 = total % 8;
    const int x = (int)blockIdx.x % 8, y = (int)blockIdx.x / 8;
    int id = x * q8 + min(x, r8) + y;
    const int split = id / (p.mt * p.nt);
    id -= split * p.mt * p.nt;
    const int strip = id / (4 * p.mt), in = id - strip * 4 * p.mt;
    const int width = min(4, p.nt - 4 * strip);
    const int64_t m0 = (int64_t)(in / width) * BM, n0 = (int64_t)(4 * strip + in % width) * BN;
    const int st0 = (int)((int64_t)p.steps * split / p.nsplit);
    const int nst = (int)((int64_t)p.steps * (split + 1) / p.nsplit) - st0;   // >= 1

    // (rows past the end load zeros, and only reach results that are never stored)
    const __amdgpu_buffer_rsrc_t wrsrc =
        gm_rsrc(p.w.codes + n0 * p.w_bytes, std::min<int64_t>(p.n - n0, BN) * p.w_bytes);
    const __amdgpu_buffer_rsrc_t arsrc =
        gm_rsrc(p.a.codes + m0 * p.a_bytes, std::min<int64_t>(p.m - m0, BM) * p.a_bytes);
    // a wave moves the scales of 64 SDMA rows of one side
    const bool sw_side = wave * SDMA < NJ;
    const int srow = 64 * (sw_side ? wave * SDMA : wave * SDMA - NJ);
    const int64_t srows = sw_side ? p.n : p.m, sfirst = (sw_side ? n0 : m0) + srow;
    const uint8_t *sbase = (sw_side ? p.w.scales : p.a.scales) + sfirst * 4;
    const int64_t sbytes = std::max<int64_t>(0, std::min<int64_t>(srows - sfirst, 64 * SDMA)) * 4;

    int turn = 0, slot = 0;                           // the next stage to load, its ring slot
    const int wrow = 16 * WDMA * wave + (lane >> 2);  // load q: 16 rows further
    const int wv = (int)(wrow * p.w_bytes) + 16 * ((lane & 3) ^ swz4(wrow));
    const int arow = (16 / AQ) * ADMA * wave + (FA == MX_FP4 ? lane >> 2 : lane >> 3);
    int av[8];                                        // ADMA of them (rows 16 apart share their swizzle, 8 apart not)
#pragma unroll
    for (int q = 0; q < ADMA; ++q) {
        const int row = arow + q * (16 / AQ);
        av[q] = (int)(row * p.a_bytes) + 16 * (FA == MX_FP4 ? (lane & 3) ^ swz4(row) : (lane & 7) ^ swz8(row));
    }
    // (a row's offset is in the lane's part, which the bounds check sees)
    const int wstep = 16 * (int)p.w_bytes;
    auto issue = [&](int part) {
        char *buf = lds + slot * STAGE;
        const int st = st0 + min(turn, nst - 1);      // (past the end the last stage again, unused)
#pragma unroll
        for (int q = part * WDMA / 2; q < (part + 1) * WDMA / 2; ++q)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(wrsrc, (gm_lds_void *)(buf + (WDMA * wave + q) * 1024), 16,
                                                     wv + q * wstep, st * 64, 0, 0);
#pragma unroll
        for (int q = part * ADMA / 2; q < (part + 1) * ADMA / 2; ++q)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(arsrc, (gm_lds_void *)(buf + WSIDE + (ADMA * wave + q) * 1024),
                                                     16, av[q], st * AROW, 0, 0);
        if (part) {
            const __amdgpu_buffer_rsrc_t srsrc = gm_rsrc(sbase + (int64_t)st * srows * 4, sbytes);
#pragma unroll
            for (int q = 0; q < SDMA; ++q)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    srsrc, (gm_lds_void *)(buf + WSIDE + ASIDE + (SDMA * wave + q) * 256), 4, lane * 4 + q * 256, 0, 0, 0);
        }
    };
    auto advance = [&] {
        ++turn;
        slot = slot == NBUF - 1 ? 0 : slot + 1;
    };

    const int wfirst = wn * 32 * NJ + li, afirst = wm * 32 * MI + li;
    auto frags = [&](const char *buf, int s, i32x4 (&fw)[NJ], i32x4 (&fa)[MI][AQ]) {
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            fw[j] = *(const i32x4 *)(buf + (wfirst + 32 * j) * 64 + 16 * ((2 * h + s) ^ swz4(li)));
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            if constexpr (FA == MX_FP4) {
                fa[i][0] = *(const i32x4 *)(buf + WSIDE + (afirst + 32 * i) * 64 + 16 * ((2 * h + s) ^ swz4(li)));
            } else {
                const char *row = buf + WSIDE + (afirst + 32 * i) * 128;
                fa[i][0] = *(const i32x4 *)(row + 16 * ((2 * s + h) ^ swz8(li)));
                fa[i][AQ - 1] = *(const i32x4 *)(row + 16 * ((4 + 2 * s + h) ^ swz8(li)));
            }
        }
    };
    auto scales = [&](const char *buf, int (&sw)[NJ], int (&sa)[MI]) {
        const char *s = buf + WSIDE + ASIDE + 2 * h;
#pragma unroll
        for (int j = 0; j < NJ; ++j) sw[j] = *(const uint16_t *)(s + (wfirst + 32 * j) * 4);
#pragma unroll
        for (int i = 0; i < MI; ++i) sa[i] = *(const uint16_t *)(s + (BN + afirst + 32 * i) * 4);
    };
    f32x16 acc[NJ][MI];
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < MI; ++i) acc[j][i] = f32x16{};
    auto products = [&](auto sub, const i32x4 (&fw)[NJ], const i32x4 (&fa)[MI][AQ], const int (&sw)[NJ],
                        const int (&sa)[MI]) {
        constexpr int S = decltype(sub)::value;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const i32x8 wb = {fw[j][0], fw[j][1], fw[j][2], fw[j][3], 0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                const i32x4 a0 = fa[i][0], a1 = fa[i][AQ - 1];
                if constexpr (FA == MX_FP4)
                    acc[j][i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                        wb, i32x8{a0[0], a0[1], a0[2], a0[3], 0, 0, 0, 0}, acc[j][i], 4, 4, S, sw[j], S, sa[i]);
                else
                    acc[j][i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                        wb, i32x8{a0[0], a0[1], a0[2], a0[3], a1[0], a1[1], a1[2], a1[3]}, acc[j][i], 4, 0, S, sw[j],
                        S, sa[i]);
            }
        }
    };
    auto spread = [](auto part) {   // operand reads one behind each MFMA, then the loads over the rest
        constexpr int MFMA = 0x008, VMEM = 0x010, DSR = 0x100, P = decltype(part)::value;
        constexpr int READS = NJ + AQ * MI + P * (NJ + MI), LOADS = (WDMA + ADMA) / 2 + (1 - P) * SDMA;
        constexpr int PER = (READS + LOADS + MI * NJ - 1) / (MI * NJ);
#pragma unroll
        for (int i = 0; i < (READS + PER - 1) / PER; ++i) {
            __builtin_amdgcn_sched_group_barrier(MFMA, 1, 0);
            __builtin_amdgcn_sched_group_barrier(DSR, PER, 0);
        }
#pragma unroll
        for (int i = 0; i < (LOADS + PER - 1) / PER; ++i) {
            __builtin_amdgcn_sched_group_barrier(MFMA, 1, 0);
            __builtin_amdgcn_sched_group_barrier(VMEM, PER, 0);
        }
    };
    using Zero = std::integral_constant<int, 0>;
    using One = std::integral_constant<int, 1>;
    i32x4 fw0[NJ], fa0[MI][AQ], fw1[NJ], fa1[MI][AQ];
    int sw0[NJ], sa0[MI], sw1[NJ], sa1[MI];
    for (int st = 0; st < NBUF - 1; ++st) {
        issue(0);
        issue(1);
        advance();
    }
    gm_wait<(NBUF - 2) * PER_STAGE>();     // stage 0 landed
    gm_barrier();
    issue(0);
    const char *buf = lds;
    int at = 0;
    frags(buf, 0, fw0, fa0);
    scales(buf, sw0, sa0);
    for (int st = 0; st < nst - 1; ++st) {
        frags(buf, 1, fw1, fa1);
        issue(1);
        products(Zero{}, fw0, fa0, sw0, sa0);
        spread(Zero{});
        __builtin_amdgcn_sched_barrier(0);
        advance();
        gm_wait<(NBUF - 2) * PER_STAGE>(); // stage st + 1 landed
        gm_barrier();                      // every wave has read stage st: its buffer is free
        __builtin_amdgcn_sched_barrier(0);
        at = at == NBUF - 1 ? 0 : at + 1;
        buf = lds + at * STAGE;
        frags(buf, 0, fw0, fa0);
        scales(buf, sw1, sa1);
        issue(0);
        products(One{}, fw1, fa1, sw0, sa0);
        spread(One{});
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < NJ; ++j) sw0[j] = sw1[j];
#pragma unroll
        for (int i = 0; i < MI; ++i) sa0[i] = sa1[i];
    }
    frags(buf, 1, fw1, fa1);
    products(Zero{}, fw0, fa0, sw0, sa0);
    products(One{}, fw1, fa1, sw0, sa0);
    gm_wait<0>();   // the loads past the end must land before the ring is reused
    gm_barrier();

    // lane (h, li), register 4 q + e of tile (j, i) <-> output 8 q + 4 h + e, row li.
    // Each wave turns 64 rows at a time around through its own part of LDS, so
    // that it reads and writes whole row segments, 16 bytes a lane, several rows
    // in flight together.  (Four outputs a lane and one row at a time took 23 us
    // per tile of 256 x 256, as long as the products of K = 4096.)
    constexpr int COLS = 32 * NJ, LPR = COLS / 8, RPP = 64 / LPR, R = 4;   // lanes per row, rows per pass
    const int lc = 8 * (lane % LPR), lr = lane / LPR;
    const int64_t n = n0 + wn * COLS + lc;
    float *out = (float *)lds + wave * 64 * EROW;
    float bias[8] = {};
    if (p.nsplit == 1 && n < p.n) mx_bias8(p.out, n, bias);
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
            constexpr int QPR = COLS / 4, QROWS = 64 / QPR;
            const int qc = 4 * (lane % QPR);
            const int64_t nq = n0 + wn * COLS + qc;
            if (nq < p.np)
#pragma unroll 8
                for (int at = lane / QPR; at < 64; at += QROWS) {
                    const int64_t row = m0 + wm * 32 * MI + 32 * i0 + at;
                    if (row < p.m)
                        *(f32x4 *)(p.part + ((int64_t)split * p.m + row) * p.np + nq) =
                            *(const f32x4 *)(out + at * EROW + qc);
                }
        } else if (n < p.n) {
#pragma unroll 1
            for (int c0 = 0; c0 < 64 / RPP; c0 += R) {
                int64_t row[R];
                float z[R][8];
#pragma unroll
                for (int c = 0; c < R; ++c) {
                    const int at = (c0 + c) * RPP + lr;
                    const f32x4 z0 = *(const f32x4 *)(out + at * EROW + lc), z1 = *(const f32x4 *)(out + at * EROW + lc + 4);
                    row[c] = m0 + wm * 32 * MI + 32 * i0 + at;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        z[c][e] = z0[e];
                        z[c][4 + e] = z1[e];
                    }
                }
                mx_epilogue(p.out, p.m, row, n, bias, z);
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // (read before the next rows overwrite them)
    }
}

// the splits' sums in split order, and the epilogue: eight outputs per thread
__global__ __launch_bounds__(256) void mx_split_reduce_kernel(MxGemm p) {
    const int64_t per = p.np / 8;
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (t >= p.m * per) return;
    const int64_t row[1] = {t / per}, n = 8 * (t - row[0] * per);
    float z[1][8] = {};
    for (int s = 0; s < p.nsplit; ++s) {
        const float *z0 = p.part + ((int64_t)s * p.m + row[0]) * p.np + n;
        const f32x4 a = *(const f32x4 *)z0, b = *(const f32x4 *)(z0 + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            z[0][e] += a[e];
            z[0][4 + e] += b[e];
        }
    }
    float bias[8];
    mx_bias8(p.out, n, bias);
    mx_epilogue(p.out, p.m, row, n, bias, z);
}

// Tiles of 256 x 256 where they fill half the CUs at once and K is long; otherwise
// of 128 x 128, two groups to a CU, so that one's epilogue runs beside the
// other's products.  Large / small, us a call: fp4 4096 x 11008 outputs K = 1024
// 60 / 50, 4096 116 / 126, 16384 365 / 483; fp8 2048 x 28672 outputs K = 1024 87 /
// 65, 4096 199 / 206, 8192 360 / 393; 1000 x 4096 outputs (64 large tiles) K = 11008
// fp4 64 / 32, fp8 95 / 41.
// k splits for grids that leave CUs idle, each of at least four stages.
struct Plan {
    int size, mt, nt, nsplit;   // tile of 64 size rows and outputs
};
Plan plan_mx(int64_t m, int64_t n, int steps) {
    Plan p;
    p.size = cdiv(m, 256) * cdiv(n, 256) >= 128 && steps >= 32 ? 4 : 2;
    p.mt = (int)cdiv(m, 64 * p.size);
    p.nt = (int)cdiv(n, 64 * p.size);
    const int64_t tiles = (int64_t)p.mt * p.nt;
    p.nsplit = p.size == 4 ? 1 : (int)std::max<int64_t>(1, std::min<int64_t>({256 / tiles, (int64_t)steps / 4, 16}));
    return p;
}

bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

template <int FA>
void launch_tiles(const MxGemm &g, int size, hipStream_t st) {
    const unsigned blocks = (unsigned)(g.mt * g.nt * g.nsplit);
    if (size == 4)
        mx_gemm_kernel<FA, 4, 4, FA == MX_FP4 ? 4 : 3><<<blocks, 256, 0, st>>>(g);
    else
        mx_gemm_kernel<FA, 2, 2, FA == MX_FP4 ? 4 : 3><<<blocks, 256, 0, st>>>(g);
}

}  // namespace

MxEpilogue mx_epilogue_of(const MxLinear &a) {
    MxEpilogue e{};
    e.n = a.d_out;
    e.bias = a.bias;
    e.bias_bf16 = a.bias_bf16;
    e.act = a.act;
    e.residual = a.residual;
    e.Y = a.Y;
    e.pre = a.pre;
    e.out_bf16 = a.out_bf16;
    const bool whole = aligned(a.Y, 16) && (!a.residual || aligned(a.residual, 16)) && (!a.bias || aligned(a.bias, 16)) &&
                       (!a.pre || aligned(a.pre, 16));
    e.width = !whole || a.d_out % 4 ? 1 : (a.d_out % 8 ? 4 : 8);
    return e;
}

size_t mx_gemm_ws(int64_t m, int64_t d_out, int64_t d_in) {
    const Plan p = plan_mx(m, d_out, (int)mx_steps(d_in));
    return p.nsplit > 1 ? align256((size_t)p.nsplit * m * (cdiv(d_out, 8) * 8) * sizeof(float)) : 0;
}

hipError_t mx_gemm_launch(const MxLinear &a, hipStream_t st) {
    MxGemm g{};
    g.a = a.a;
    g.w = a.w;
    g.m = a.m;
    g.n = a.d_out;
    g.a_bytes = mx_row_bytes(a.d_in, a.a.fmt);
    g.w_bytes = mx_row_bytes(a.d_in, MX_FP4);
    g.steps = (int)mx_steps(a.d_in);
    g.out = mx_epilogue_of(a);
    g.part = (float *)a.ws;
    g.np = cdiv(g.n, 8) * 8;
    const Plan p = plan_mx(g.m, g.n, g.steps);
    g.mt = p.mt;
    g.nt = p.nt;
    g.nsplit = p.nsplit;
    if (a.a.fmt == MX_FP4)
        launch_tiles<MX_FP4>(g, p.size, st);
    else
        launch_tiles<MX_FP8>(g, p.size, st);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || g.nsplit == 1) return e;
    mx_split_reduce_kernel<<<(unsigned)cdiv(g.m * (g.np / 8), 256), 256, 0, st>>>(g);
    return hipGetLastError();
}

size_t mx_linear_ws(int64_t m, int64_t d_out, int64_t d_in, int kind, int out_bf16) {
    if (m == 0 || mx_skinny_takes(m, d_out, d_in, kind)) return 0;
    if (kind == MX_FP4 || kind == MX_FP8) return mx_gemm_ws(m, d_out, d_in);
    FusedShape s{};
    s.m = m;
    s.d_out = d_out;
    s.d_in = d_in;
    s.layers = 1;
    s.in_bf16 = kind != MX_ACT_F32;   // (fp8 activations are exact in f16 too)
    s.out_bf16 = out_bf16;
    return dense_forward_ws(s);
}

hipError_t mx_linear_launch(const MxLinear &a, hipStream_t st) {
    const int kind = mx_kind(a);
    if (mx_skinny_takes(a.m, a.d_out, a.d_in, kind)) return mx_skinny_launch(a, st);
    if (kind == MX_FP4 || kind == MX_FP8) return mx_gemm_launch(a, st);
    FusedForward f{};
    f.s.m = a.m;
    f.s.d_out = a.d_out;
    f.s.d_in = a.d_in;
    f.s.layers = 1;
    f.s.in_bf16 = kind != MX_ACT_F32;
    f.s.out_bf16 = a.out_bf16;
    f.A = a.A;
    f.amx = a.a;
    f.mx = a.w;
    f.bias[0] = a.bias;
    f.bias_bf16 = a.bias_bf16;
    f.act = a.act;
    f.residual = a.residual;
    f.Y = a.Y;
    f.pre[0] = a.pre;
    f.ws = a.ws;
    return dense_forward_launch(f, st);
}

size_t mx_linear_backward_ws(const FusedShape &s) {
    if (s.m == 0) return 0;
    // (the size is asked for without the activation, on which the form may depend)
    const bool with = mx_skinny_backward_takes(s, 1), without = mx_skinny_backward_takes(s, 0);
    return std::max(with || without ? mx_skinny_backward_ws(s) : 0, with && without ? 0 : dense_backward_ws(s));
}

hipError_t mx_linear_backward_launch(const FusedBackward &a, hipStream_t st) {
    if (a.s.m == 0) return fused_backward_launch(a, st);   // (zero bias gradients)
    return mx_skinny_backward_takes(a.s, a.act) ? mx_skinny_backward_launch(a, st) : dense_backward_launch(a, st);
}

}  // namespace gptq
