// wa_f64.cuh — the float64 arithmetic of the re-runs: dot products, reductions, rounding to bf16.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace wa {

namespace {

constexpr int kRerunThreads = 256;

__device__ __forceinline__ double bf16_bits_to_f64(uint16_t b) {
    return static_cast<double>(__uint_as_float(static_cast<uint32_t>(b) << 16));
}

// Round a float64 value to bf16, nearest-even, in one step; an underflow keeps its sign.
__device__ uint16_t f64_to_bf16_rn(double x) {
    const uint16_t sign = (__double_as_longlong(x) < 0) ? 0x8000u : 0u;
    if (isnan(x)) return sign | 0x7FC0u;
    const double ax = fabs(x);
    if (isinf(ax)) return sign | 0x7F80u;
    if (ax < 0x1p-126) {   // subnormal range: quantum 2^-133
        return sign | static_cast<uint16_t>(rint(ax * 0x1p133));
    }
    int e;
    const double m = frexp(ax, &e);      // ax = m * 2^e, m in [0.5, 1)
    double sig = rint(ldexp(m, 8));      // 8 significant bits
    if (sig >= 256.0) {
        sig = 128.0;
        e += 1;
    }
    const int biased = e - 1 + 127;
    if (biased >= 255) return sign | 0x7F80u;
    return sign | static_cast<uint16_t>((biased << 7) | (static_cast<int>(sig) - 128));
}

__device__ __forceinline__ double block_reduce(double x, bool is_max, double* red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        const double y = __shfl_xor_sync(0xFFFFFFFFu, x, off);
        x = is_max ? ((isnan(x) || isnan(y)) ? (x + y) : fmax(x, y)) : (x + y);
    }
    if (lane == 0) red[warp] = x;
    __syncthreads();
    double r = red[0];
    for (int w = 1; w < kRerunThreads / 32; ++w) {
        const double y = red[w];
        r = is_max ? ((isnan(r) || isnan(y)) ? (r + y) : fmax(r, y)) : (r + y);
    }
    __syncthreads();
    return r;
}

// d bf16 values of a row as float64 (16-byte loads; the row is 16-byte aligned).
__device__ __forceinline__ double dot_f64(const double* qd, const uint16_t* kr, int d) {
    double s = 0.0;
    for (int e = 0; e < d; e += 8) {
        const uint4 u = *reinterpret_cast<const uint4*>(kr + e);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s = s + qd[e + 2 * i] * static_cast<double>(__uint_as_float(w[i] << 16));
            s = s + qd[e + 2 * i + 1] * static_cast<double>(__uint_as_float(w[i] & 0xFFFF0000u));
        }
    }
    return s;
}

// The same dot product in fp32: every product of two bf16 values is exact in fp32 unless it
// overflows or underflows, so a finite float64 score can only come out non-finite here through
// overflow, and a float64 NaN or infinity always shows as non-finite.
__device__ __forceinline__ float dot_f32(const float* qf, const uint16_t* kr, int d) {
    float s = 0.f;
    for (int e = 0; e < d; e += 8) {
        const uint4 u = *reinterpret_cast<const uint4*>(kr + e);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s = fmaf(qf[e + 2 * i], __uint_as_float(w[i] << 16), s);
            s = fmaf(qf[e + 2 * i + 1], __uint_as_float(w[i] & 0xFFFF0000u), s);
        }
    }
    return s;
}

}  // namespace

}  // namespace wa
