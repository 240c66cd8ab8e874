// wa_paged_append.cu — rotary positions, alone or on the way into a cache in pages.
//
// Pair (a, b) of token t turns by pos[t] * inv_freq[j]:
//   y_a = f (x_a cos - x_b sin),  y_b = f (x_b cos + x_a sin).
// One kernel serves both calls: wa_rope is an append of query heads alone.
//
// Angles.  fl32(pos * inv_freq) is off by up to 2^-24 of the angle, 0.06 rad at
// position 10^6, and a float64 product runs at a fiftieth of the fp32 rate here.
// So inv_freq / (2 pi) becomes a 64-bit fixed-point fraction of a turn, by a 24 x
// 96-bit integer product, and times pos, modulo 2^64, that is the angle's
// fraction of a turn to 2^-33 for every int32 position.  Its upper 32 bits, rounded to fp32 (by 2^-26 of a turn at most), go to
// sincospif.
//
// HBM-bound: a head is served by L = d / 16 lanes of two 16-byte pieces each, so
// that both halves of a pair sit in one lane for either layout, a warp takes P =
// 32 / L heads a pass and PASSES passes of one token, all loads issued before the
// angles are worked out, two or four a lane, which the others fetch by shuffles.  (8,185 tokens of 32 + 2 x 8 heads of 128 into bf16
// pages 32.3 us for 29.7 at the rate of a copy, into 8-bit pages 39.2 for 27.2, a division a value; rope of 8,192 x 40 heads of
// 128 26.0 for 24.7, its inverse over 64 of 256 dims of 5,003 x 24 heads 20.2 for 18.1.  Times of replayed graphs.)
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "wa.h"
#include "wa_internal.h"

namespace wa {

namespace {

constexpr int kAppendWarps = 4;       // (of 8, blocks end unevenly: rope of 8,192 x 40 heads of 128 29.7 us, with 4 26.0)
// Up to this many tokens one more block checks them all and writes the status word, which spares a launch; beyond, a kernel
// before this one clears it and the warps that look up the places of keys and values report what is wrong with them.  (The
// block, and two launches: 600 tokens of 8 + 2 x 1 heads of 128 3.2 us each, 3.5 and 4.6 eager; 1,024 4.9 and 4.1, of 32 + 2 x 8
// heads 6.5 each.)
constexpr int kStatusBlockTokens = 1024;

struct AppendParams {
    PagedAppendArgs a;
    int cleared;      // the status word is clear: the warps report
};

// Two products, and two fused multiply-adds, an instruction.
__device__ __forceinline__ void mul2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b0, float b1, float c0, float c1) {
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}

__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ void unpack(const uint4& u, float* x) {
    x[0] = low(u.x); x[1] = high(u.x); x[2] = low(u.y); x[3] = high(u.y);
    x[4] = low(u.z); x[5] = high(u.z); x[6] = low(u.w); x[7] = high(u.w);
}

__device__ __forceinline__ uint32_t pair_bf16(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint4 pack(const float* x) {
    return make_uint4(pair_bf16(x[0], x[1]), pair_bf16(x[2], x[3]), pair_bf16(x[4], x[5]), pair_bf16(x[6], x[7]));
}

__device__ __forceinline__ uint32_t quad_e4m3(const float* x, float scale) {
    const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(x[0] / scale, x[1] / scale), __NV_SATFINITE, __NV_E4M3);
    const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(x[2] / scale, x[3] / scale), __NV_SATFINITE, __NV_E4M3);
    return a | (b << 16);
}

// |w| / (2 pi) modulo 1 as a 64-bit fraction, for |w| < 16: w = m 2^(e - 150), times 2^96 / (2 pi) to the nearest
// integer, shifted down to units of 2^-64.  Cut off, so off by less than 2^-64 + 2^-73.
__device__ __forceinline__ uint64_t turn_fraction(float w) {
    const uint32_t b = __float_as_uint(w), e = (b >> 23) & 255u, exp = e ? e : 1u;
    const uint64_t m = (b & 0x7FFFFFu) | (e ? 0x800000u : 0u);
    const uint64_t p0 = m * 0x7F09D5F4u, p1 = m * 0x9391054Au + (p0 >> 32), p2 = m * 0x28BE60DBu + (p1 >> 32);
    const uint64_t lo = (p1 << 32) | (p0 & 0xFFFFFFFFu), hi = p2;
    const uint32_t s = 182u - exp;
    const uint64_t f = s < 64u ? (hi << (64u - s)) | (lo >> s) : s < 128u ? hi >> (s - 64u) : 0ull;
    return (b >> 31) ? 0ull - f : f;
}

// The bad bits of token t's place, and where it is: page < 0 for none.
__device__ __forceinline__ int place(const PagedAppendArgs& a, int t, int pos, int& page) {
    page = -1;
    if (pos < 0) return pos < -1 ? WA_STATUS_BAD_POS : 0;
    if ((pos >> a.page_log) >= a.most) return WA_STATUS_BAD_POS;
    const int row = a.row ? a.row[t] : t;
    if (row < 0 || row >= a.rows) return WA_STATUS_BAD_PAGE;
    page = a.table[row * a.table_row + (pos >> a.page_log)];
    if (page >= 0 && page < a.pages) return 0;
    page = -1;
    return WA_STATUS_BAD_PAGE;
}

// Checks every token's place and writes the status word, by a block of THREADS; kAtOnce tokens a thread at a time.
constexpr int kAtOnce = 4;
template <int THREADS>
__device__ void append_status(const PagedAppendArgs& a) {
    int bad = 0;
    for (int t0 = threadIdx.x; t0 < a.n; t0 += kAtOnce * THREADS) {
        int pos[kAtOnce], page;
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) pos[i] = t0 + i * THREADS < a.n ? a.pos[t0 + i * THREADS] : -1;
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) bad |= place(a, t0 + i * THREADS, pos[i], page);
    }
    const int where = __syncthreads_or(bad & WA_STATUS_BAD_POS), which = __syncthreads_or(bad & WA_STATUS_BAD_PAGE);
    if (threadIdx.x == 0) a.hdr->status = (where ? WA_STATUS_BAD_POS : 0) | (which ? WA_STATUS_BAD_PAGE : 0);
}

// Clears the status word; the next kernel sets itself up meanwhile and waits for this one's end.
__global__ void append_clear_kernel(int* status) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    *status = 0;
}

template <int D, bool CACHE, bool FP8, int PASSES>
__global__ void __launch_bounds__(kAppendWarps * 32) append_kernel(const __grid_constant__ AppendParams p) {
    const PagedAppendArgs& a = p.a;
    constexpr int L = D / 16;              // lanes a head
    constexpr int P = 32 / L;              // heads a pass
    constexpr int HPW = P * PASSES;        // heads a warp
    constexpr int NA = D / 64;             // pairs whose angle a lane works out
    // Launched while the kernel before still runs, waits for its end here.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if constexpr (CACHE) {
        if (!p.cleared && blockIdx.x == gridDim.x - 1) {
            if (blockIdx.y == 0) append_status<kAppendWarps * 32>(a);
            return;
        }
    }
    const int t = static_cast<int>(blockIdx.x) * kAppendWarps + (static_cast<int>(threadIdx.x) >> 5), first = static_cast<int>(blockIdx.y) * HPW;
    if (t >= a.n) return;                  // warp-uniform
    const int lane = threadIdx.x & 31, li = lane % L, hp = lane / L;
    const int nqk = a.hq + a.hkv, heads = nqk + a.hkv;
    const int pos = a.pos[t];
    const bool turns = li < a.dims / 16;
    // a lane's two pieces of a head that turns: of dims (j, j + dims / 2), or 16 neighbours; of any other, 16 neighbours
    const int one = turns && a.layout == WA_ROTARY_HALF ? 8 * li : 16 * li;
    const int two = turns && a.layout == WA_ROTARY_HALF ? a.dims / 2 + 8 * li : 16 * li + 8;
    const uint16_t* src = static_cast<const uint16_t*>(a.src) + t * a.src_tok;
    uint4 raw[PASSES][2];
    float scale[PASSES];
#pragma unroll
    for (int u = 0; u < PASSES; ++u) {
        const int h = first + u * P + hp;
        scale[u] = 1.f;
        if (CACHE && FP8 && h >= a.hq && h < heads) {
            const float* of = a.kv[h < nqk ? 0 : 1].scale;
            if (of) scale[u] = of[h - (h < nqk ? a.hq : nqk)];
        }
        if (h < heads) {
            const uint16_t* x = src + static_cast<int64_t>(h) * D;
            raw[u][0] = *reinterpret_cast<const uint4*>(x + (h < nqk ? one : 16 * li));
            raw[u][1] = *reinterpret_cast<const uint4*>(x + (h < nqk ? two : 16 * li + 8));
        }
    }
    int page = -1;
    if constexpr (CACHE) {
        if (first + HPW > a.hq) {                                          // a warp with keys or values
            const int bad = place(a, t, pos, page);
            if (p.cleared && bad && blockIdx.y == gridDim.y - 1 && lane == 0) atomicOr(&a.hdr->status, bad);
        }
        if (pos < 0 || (pos >> a.page_log) >= a.most) return;
    }
    // Angles: a lane works out NA pairs of the token, and takes the eight of its dims from where they are.
    float c[8], s[8];
    if (a.dims > 0 && first < nqk) {
        float mc[NA], ms[NA];
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            const int j = NA * lane + i;
            const float w = 2 * j < a.dims ? a.inv_freq[j] : 0.f;
            const uint64_t turn = turn_fraction(w) * static_cast<uint64_t>(static_cast<int64_t>(pos));
            sincospif(static_cast<float>(static_cast<int>(turn >> 32)) * 0x1p-31f, &ms[i], &mc[i]);
            const float f = fabsf(w) < 16.f ? a.factor : NAN;
            mc[i] *= f;
            ms[i] *= a.inverse ? -f : f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int from = li * (8 / NA) + e / NA;
            c[e] = __shfl_sync(0xFFFFFFFFu, mc[e % NA], from);
            s[e] = __shfl_sync(0xFFFFFFFFu, ms[e % NA], from);
        }
    }
    const int64_t slot = CACHE ? pos & ((1 << a.page_log) - 1) : 0;
#pragma unroll
    for (int u = 0; u < PASSES; ++u) {
        const int h = first + u * P + hp;
        if (h >= heads) continue;
        float x[16];
        unpack(raw[u][0], x);
        unpack(raw[u][1], x + 8);
        if (turns && h < nqk) {
            if (a.layout == WA_ROTARY_HALF) {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    float u0, u1, v0, v1;
                    mul2(u0, u1, x[8 + e], x[9 + e], -s[e], -s[e + 1]);
                    mul2(v0, v1, x[e], x[e + 1], s[e], s[e + 1]);
                    fma2(x[e], x[e + 1], x[e], x[e + 1], c[e], c[e + 1], u0, u1);
                    fma2(x[8 + e], x[9 + e], x[8 + e], x[9 + e], c[e], c[e + 1], v0, v1);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float u0, u1;
                    mul2(u0, u1, x[2 * e + 1], x[2 * e], -s[e], s[e]);
                    fma2(x[2 * e], x[2 * e + 1], x[2 * e], x[2 * e + 1], c[e], c[e], u0, u1);
                }
            }
        }
        const int o1 = h < nqk ? one : 16 * li, o2 = h < nqk ? two : 16 * li + 8;
        if (!CACHE || h < a.hq) {
            uint16_t* out = static_cast<uint16_t*>(a.q_out) + t * a.q_tok + static_cast<int64_t>(h) * D;
            *reinterpret_cast<uint4*>(out + o1) = pack(x);
            *reinterpret_cast<uint4*>(out + o2) = pack(x + 8);
        } else if (page >= 0) {
            const PageSide& side = a.kv[h < nqk ? 0 : 1];
            const int g = h - (h < nqk ? a.hq : nqk);
            const int64_t at = page * side.page + slot * side.slot + g * side.head;
            if constexpr (FP8) {
                uint8_t* out = static_cast<uint8_t*>(side.base) + at;
                *reinterpret_cast<uint2*>(out + o1) = make_uint2(quad_e4m3(x, scale[u]), quad_e4m3(x + 4, scale[u]));
                *reinterpret_cast<uint2*>(out + o2) = make_uint2(quad_e4m3(x + 8, scale[u]), quad_e4m3(x + 12, scale[u]));
            } else {
                uint16_t* out = static_cast<uint16_t*>(side.base) + at;
                *reinterpret_cast<uint4*>(out + o1) = pack(x);
                *reinterpret_cast<uint4*>(out + o2) = pack(x + 8);
            }
        }
    }
}

}  // namespace

namespace {

template <int PASSES>
cudaError_t launch_append(const AppendParams& p, cudaLaunchConfig_t& cfg) {
    const PagedAppendArgs& a = p.a;
    const int hpw = 32 / (a.d / 16) * PASSES;
    cfg.gridDim = dim3((a.n - 1) / kAppendWarps + 1 + (a.hkv > 0 && !p.cleared), (a.hq + 2 * a.hkv + hpw - 1) / hpw);
    cfg.blockDim = dim3(kAppendWarps * 32);
    auto run = [&](auto kernel) { return cudaLaunchKernelEx(&cfg, kernel, p); };
    if (a.d == 256) {
        if (a.hkv == 0) return run(append_kernel<256, false, false, PASSES>);
        return a.e4m3 ? run(append_kernel<256, true, true, PASSES>) : run(append_kernel<256, true, false, PASSES>);
    }
    if (a.hkv == 0) return run(append_kernel<128, false, false, PASSES>);
    return a.e4m3 ? run(append_kernel<128, true, true, PASSES>) : run(append_kernel<128, true, false, PASSES>);
}

// Few tokens: one pass a warp, for more warps at once (64 tokens of 48 heads of 128 to 8-bit pages: 2.5 us, with four passes
// 4.7); many: four, for fewer angles and more bytes in flight (rope of 8,192 x 40 heads of 128: 26.0 us, with two 26.9, with one
// 32.5; 8,185 tokens of 48 heads appended to bf16 pages 32.3, 33.9 and 42.0, to 8-bit ones 39.2, 37.0 and 45.1).
constexpr int64_t kFewValues = 1 << 20;

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t s) {
    AppendParams p{};
    p.a = a;
    p.cleared = a.hkv > 0 && a.n > kStatusBlockTokens;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (p.cleared) {
        cfg.gridDim = dim3(1);
        cfg.blockDim = dim3(1);
        const cudaError_t e = cudaLaunchKernelEx(&cfg, append_clear_kernel, &a.hdr->status);
        if (e != cudaSuccess) return e;
    }
    const bool few = static_cast<int64_t>(a.n) * (a.hq + 2 * a.hkv) * a.d <= kFewValues;
    const cudaError_t e = few ? launch_append<1>(p, cfg) : launch_append<4>(p, cfg);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace wa
