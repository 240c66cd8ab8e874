// wa_paged.cu — decode over a cache in pages: one new token a sequence.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "wa_f64.cuh"
#include "wa_internal.h"

namespace wa {

namespace {

__device__ __forceinline__ float e4m3_to_f32(uint8_t b) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(b, __NV_E4M3);
    return __half2float(__half(h));
}

// A stored value as fp32 (exact).
__device__ __forceinline__ float stored(const void* base, int64_t at, int e4m3) {
    return e4m3 ? e4m3_to_f32(static_cast<const uint8_t*>(base)[at])
                : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(base)[at]) << 16);
}

// A row's last position as every kernel uses it.
__device__ __forceinline__ int paged_pos(int raw, int most, int page_log) {
    return raw < -1 ? -1 : (raw >> page_log) >= most ? (most << page_log) - 1 : raw;
}

// The float64 value of one (row, head) a block: the maximum score, then weights and their sums in key order, 256 keys at
// a time; a NaN or +inf score settles the output before that.
__global__ void __launch_bounds__(kRerunThreads) paged_f64_kernel(const __grid_constant__ PagedArgs a) {
    __shared__ double qd[256], wb[kRerunThreads], red[kRerunThreads / 32];
    __shared__ int64_t vat[kRerunThreads];
    const int t = threadIdx.x, d = a.d, G = a.hq / a.hkv;
    const int units = a.rows * a.hq;
    for (int f = blockIdx.x; f < units; f += gridDim.x) {
        const int row = f / a.hq, h = f % a.hq, g = h / G;
        const int raw = a.pos[row], p = paged_pos(raw, a.most, a.page_log);
        uint16_t* orow = static_cast<uint16_t*>(a.out) + row * a.o_row + static_cast<int64_t>(h) * d;
        if (raw != p && t == 0) atomicOr(&a.hdr->status, WA_STATUS_BAD_POS);
        if (p < 0) {
            if (t < d) orow[t] = 0;
            continue;
        }
        const int lo = a.win > 0 ? max(0, p - a.win + 1) : 0;
        if (t < d) qd[t] = bf16_bits_to_f64(static_cast<const uint16_t*>(a.q)[row * a.q_row + static_cast<int64_t>(h) * d + t]);
        __syncthreads();
        const double scale = static_cast<double>(a.scale) * (a.kv[0].scale ? static_cast<double>(a.kv[0].scale[g]) : 1.0);
        // where key j's head starts in k or v; -1 in a page that is none
        auto at = [&](const PageSide& side, int j) -> int64_t {
            const int page = a.table[row * a.table_row + (j >> a.page_log)];
            if (page < 0 || page >= a.pages) {
                atomicOr(&a.hdr->status, WA_STATUS_BAD_PAGE);
                return -1;
            }
            return page * side.page + (j & ((1 << a.page_log) - 1)) * side.slot + g * side.head;
        };
        auto score = [&](int j) {
            const int64_t k = at(a.kv[0], j);
            double s = 0.0;
            for (int e = 0; e < d; ++e) s = s + qd[e] * (k < 0 ? 0.0 : static_cast<double>(stored(a.kv[0].base, k + e, a.e4m3)));
            return s * scale;
        };
        double mloc = -INFINITY;
        for (int j = lo + t; j <= p; j += kRerunThreads) {
            const double s = score(j);
            mloc = (isnan(s) || isnan(mloc)) ? (s + mloc) : fmax(mloc, s);
        }
        const double M = block_reduce(mloc, true, red);
        double lloc = 0.0, acc = 0.0;
        for (int base = lo; base <= p; base += kRerunThreads) {
            const int j = base + t;
            double w = 0.0;
            if (j <= p) {
                w = exp(score(j) - M);
                lloc = lloc + w;
                vat[t] = at(a.kv[1], j);
            }
            wb[t] = w;
            __syncthreads();
            if (t < d) {
                const int cnt = min(kRerunThreads, p - base + 1);
                for (int jj = 0; jj < cnt; ++jj)
                    acc = acc + wb[jj] * (vat[jj] < 0 ? 0.0 : static_cast<double>(stored(a.kv[1].base, vat[jj] + t, a.e4m3)));
            }
            __syncthreads();
        }
        const double l = block_reduce(lloc, false, red);
        if (t < d) orow[t] = f64_to_bf16_rn(acc / l * (a.kv[1].scale ? static_cast<double>(a.kv[1].scale[g]) : 1.0));
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_paged_decode(const PagedArgs& a, cudaStream_t s) {
    cudaError_t e = cudaMemsetAsync(a.hdr, 0, kHeaderBytes, s);
    if (e != cudaSuccess) return e;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return cudaErrorInvalidValue;
    const int64_t units = static_cast<int64_t>(a.rows) * a.hq;
    paged_f64_kernel<<<static_cast<int>(units < 4LL * sms ? units : 4LL * sms), kRerunThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace wa
