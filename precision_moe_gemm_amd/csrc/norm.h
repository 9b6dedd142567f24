// norm.h -- the residual's addition, the root-mean-square norm and the MXFP8
// encode of its result in one pass (the activation operand of the W4A8
// products, page "DeepSeek-V4.1-Flash-NVFP4", section 二: activations in
// 8 bits with power-of-two block scales).
//
//   r = bf16(x + residual)                    (or x)
//   i = fp32(1 / sqrt(mean(r^2) + eps))       (the sum in 64 bits)
//   y = bf16((r * i) * w)                     (fp32 steps)
//   codes, scales = mxfp8_quantize(y)
//
// r^2 of a bf16 value is exact, and a row's sum in fp64 is off by at most
// cols 2^-53 of itself in any order (2^-37 at 65536 columns): i is the fp32
// value of the exact sum but where that lies so close to a border of fp32's
// rounding.  The order of the sum is set by cols alone, so a row gives the same
// bytes in every call.
#pragma once
#include "common.h"
#include "mx8.h"

namespace nvfp4 {

struct NormArgs {
    const u32x4* x;
    const u32x4* residual;  // may be null
    const u32x4* weight;    // may be null (all ones)
    u32x4* sum;             // r; may be null, may be x or residual
    u32x4* y;               // may be null
    u32x2* fp8;             // may be null (with e8m0)
    uint8_t* e8m0;
    int64_t rows;
    int64_t ld_x, ld_res, ld_sum, ld_y;  // row strides in 16-byte chunks
    int chunks;                          // cols / 8
    double cols;
    double eps;
};

// 1 / sqrt(v) rounded to fp32: the hardware estimate and two Newton steps in
// fp64 (1e-7, 1e-14, then the rounding of fp64), far cheaper than fp64's
// square root and division.  v is mean + eps, rescaled by an even power of
// two so that the estimate's fp32 argument is never subnormal.
NVFP4_DEV float inv_sqrt_f64(double v)
{
    if (!(v > 0.0))
        return v == 0.0 ? __builtin_inff() : __builtin_nanf("");
    if (v == __builtin_inf())  // (frexp and the steps below give NaN)
        return 0.0f;
    int e = 0;
    const double m = __builtin_frexp(v, &e);  // m in [0.5, 1)
    const int half = e >> 1;                  // v = (m * 2^(e & 1)) * 2^(2 half)
    const double a = (e & 1) ? m * 2.0 : m;
    double y = (double)__builtin_amdgcn_rsqf((float)a);
    y = y * (1.5 - 0.5 * a * y * y);
    y = y * (1.5 - 0.5 * a * y * y);
    return (float)__builtin_ldexp(y, -half);
}

// Chunk c of row `row`: r, stored if wanted.
NVFP4_DEV u32x4 norm_add(const NormArgs& a, int64_t row, int c)
{
    u32x4 v = a.x[row * a.ld_x + c];
    if (a.residual) {
        const u32x4 q = a.residual[row * a.ld_res + c];
#pragma unroll
        for (int i = 0; i < 4; i++)
            v[i] = pack_bf16x2(bf16_lo(v[i]) + bf16_lo(q[i]), bf16_hi(v[i]) + bf16_hi(q[i]));
    }
    if (a.sum)
        a.sum[row * a.ld_sum + c] = v;
    return v;
}

NVFP4_DEV double norm_squares(u32x4 r, double ss)
{
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const double lo = bf16_lo(r[i]), hi = bf16_hi(r[i]);
        ss = __builtin_fma(lo, lo, ss);
        ss = __builtin_fma(hi, hi, ss);
    }
    return ss;
}

// y and its MXFP8 encode; four consecutive lanes hold one 32-element block
// (all 64 lanes execute it, `in`: the chunk exists).
NVFP4_DEV void norm_store(const NormArgs& a, int64_t row, int c, bool in, u32x4 r, float inv)
{
    u32x4 w = (u32x4){0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
    if (a.weight && in)
        w = a.weight[c];
    u32x4 y;
#pragma unroll
    for (int i = 0; i < 4; i++)
        y[i] = pack_bf16x2((bf16_lo(r[i]) * inv) * bf16_lo(w[i]), (bf16_hi(r[i]) * inv) * bf16_hi(w[i]));
    if (a.y && in)
        a.y[row * a.ld_y + c] = y;
    if (a.fp8) {
        uint32_t am = absmax_bits8(y);
        am = umax_u32(am, swz_xor<1>(am));
        am = umax_u32(am, swz_xor<2>(am));
        const int e = mx8_exponent(am);
        if (in) {
            const int64_t o = row * a.chunks + c;
            a.fp8[o] = mx8_encode8(y, e);
            if ((c & 3) == 0)
                a.e8m0[o >> 2] = (uint8_t)(e + 127);
        }
    }
}

// One row per workgroup trip; thread t holds chunks t + u * blockDim of 8
// elements (a 16-byte load).  HBM-bound: what counts is how many rows are on
// their way while others wait at their two barriers.  512 threads (four
// workgroups per CU) took 159 us for 16384 x 7168 with a residual (5.2 TB/s, a
// copy's rate), 1024 threads 188, 256 threads 168; 64 rows 4.7, 5.0 and 6.3 us.
constexpr int kNormThreads = 512;

template <int U>
__global__ void __launch_bounds__(kNormThreads)
add_rmsnorm_kernel(NormArgs a)
{
    __shared__ double red[kNormThreads / 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        u32x4 r[U];
        double ss = 0.0;
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int c = u * blockDim.x + threadIdx.x;
            r[u] = (u32x4){0, 0, 0, 0};
            if (c < a.chunks)
                r[u] = norm_add(a, row, c);
            ss = norm_squares(r[u], ss);
        }
#pragma unroll
        for (int off = 32; off > 0; off >>= 1)
            ss += __shfl_xor(ss, off, 64);
        __syncthreads();  // the last trip's reads of red are done
        if (lane == 0)
            red[wave] = ss;
        __syncthreads();
        ss = 0.0;
        for (int i = 0; i < waves; i++)
            ss += red[i];
        const float inv = inv_sqrt_f64(ss / a.cols + a.eps);
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int c = u * blockDim.x + threadIdx.x;
            norm_store(a, row, c, c < a.chunks, r[u], inv);
        }
    }
}

// Rows of at most 8 L elements (heads): L lanes per row, 64 / L rows per wave,
// no barrier.  20000 rows of 128 took 5.9 us, 11.8 with a workgroup per row.
template <int L>
__global__ void __launch_bounds__(256)
add_rmsnorm_narrow_kernel(NormArgs a)
{
    const int c = threadIdx.x % L;
    for (int64_t row0 = (int64_t)blockIdx.x * (256 / L); row0 < a.rows; row0 += (int64_t)gridDim.x * (256 / L)) {
        const int64_t row = row0 + threadIdx.x / L;
        const bool in = row < a.rows && c < a.chunks;
        u32x4 r = (u32x4){0, 0, 0, 0};
        if (in)
            r = norm_add(a, row, c);
        double ss = norm_squares(r, 0.0);
#pragma unroll
        for (int off = L / 2; off > 0; off >>= 1)
            ss += __shfl_xor(ss, off, 64);
        norm_store(a, row, c, in, r, inv_sqrt_f64(ss / a.cols + a.eps));
    }
}

}  // namespace nvfp4
