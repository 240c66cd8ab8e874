// wa_tree.cu — attention of trees of drafted tokens over ring caches.
//
// Node i of row r, at position P = pos[r] + 1 + depth(i), sees the ring's keys
// [max(0, P - win + 1), pos[r]] and those of its tree's nodes that are its
// ancestors or itself and less than win positions back:
//   o = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale q.k_j - m).
//
// One warp per (node, query head): lanes share the head's dims, keys one by one
// with a running maximum, sum and output in fp32.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "wa_internal.h"

namespace wa {

namespace {

constexpr int kTreeWarps = 4;

template <int D>
__global__ void __launch_bounds__(kTreeWarps * 32) tree_warp_kernel(const TreeArgs a) {
    constexpr int DPL = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kTreeWarps + (threadIdx.x >> 5);
    if (unit >= static_cast<int64_t>(a.rows) * a.nodes * a.hq) return;
    const int h = static_cast<int>(unit % a.hq), node = static_cast<int>(unit / a.hq % a.nodes);
    const int r = static_cast<int>(unit / a.hq / a.nodes);
    const int g = h / (a.hq / a.hkv);
    int n = a.n ? a.n[r] : a.nodes;
    int p = a.pos[r];
    if (lane == 0 && h == 0 && node == 0) {
        if (n < 0 || n > a.nodes) atomicOr(&a.hdr->status, WA_STATUS_BAD_TREE);
        if (p < -1 || (a.win == 0 && p >= a.ring)) atomicOr(&a.hdr->status, WA_STATUS_BAD_POS);
    }
    n = min(max(n, 0), a.nodes);
    p = max(p, -1);
    if (a.win == 0) p = min(p, a.ring - 1);
    if (node >= n) return;
    const int32_t* par = a.parent + static_cast<int64_t>(r) * a.nodes;
    if (lane == 0 && h == 0 && tree_parent(par[node], node) != par[node]) atomicOr(&a.hdr->status, WA_STATUS_BAD_TREE);
    int depth = 0;
    for (int x = node; (x = tree_parent(par[x], x)) >= 0;) ++depth;

    float q[DPL], o[DPL];
    const uint16_t* qr = static_cast<const uint16_t*>(a.q) + r * a.q_row + node * a.q_tok + static_cast<int64_t>(h) * D;
    for (int e = 0; e < DPL; ++e) {
        q[e] = __uint_as_float(static_cast<uint32_t>(qr[lane * DPL + e]) << 16);
        o[e] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    auto fold = [&](const uint16_t* k, const uint16_t* v) {
        float s = 0.f;
        for (int e = 0; e < DPL; ++e) s = fmaf(q[e], __uint_as_float(static_cast<uint32_t>(k[lane * DPL + e]) << 16), s);
        for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
        s *= a.scale;
        const float mn = fmaxf(m, s);
        const float al = mn == m ? 1.f : expf(m - mn);
        const float w = expf(s - mn);
        l = l * al + w;
        for (int e = 0; e < DPL; ++e)
            o[e] = fmaf(w, __uint_as_float(static_cast<uint32_t>(v[lane * DPL + e]) << 16), o[e] * al);
        m = mn;
    };
    const int64_t kst = static_cast<int64_t>(a.hkv) * D;
    const uint16_t* kr = static_cast<const uint16_t*>(a.k) + r * a.ring * kst + static_cast<int64_t>(g) * D;
    const uint16_t* vr = static_cast<const uint16_t*>(a.v) + r * a.ring * kst + static_cast<int64_t>(g) * D;
    for (int j = a.win > 0 ? max(0, p + 1 + depth - a.win + 1) : 0; j <= p; ++j) fold(kr + j % a.ring * kst, vr + j % a.ring * kst);
    const uint16_t* kt = static_cast<const uint16_t*>(a.kt) + r * a.kt_row + static_cast<int64_t>(g) * D;
    const uint16_t* vt = static_cast<const uint16_t*>(a.vt) + r * a.vt_row + static_cast<int64_t>(g) * D;
    for (int x = node, back = 0; x >= 0 && (a.win == 0 || back < a.win); x = tree_parent(par[x], x), ++back)
        fold(kt + x * a.kt_tok, vt + x * a.vt_tok);

    uint16_t* orow = static_cast<uint16_t*>(a.out) + r * a.o_row + node * a.o_tok + static_cast<int64_t>(h) * D;
    bool bad = false;
    for (int e = 0; e < DPL; ++e) {
        const float x = __fdiv_rn(o[e], l);
        bad |= !isfinite(x);
        orow[lane * DPL + e] = __bfloat16_as_ushort(__float2bfloat16_rn(x));
    }
    if (__any_sync(0xFFFFFFFFu, bad) && lane == 0)
        a.flags[atomicAdd(&a.hdr->nflag, 1)] = static_cast<int>(unit);
}

}  // namespace

cudaError_t launch_tree(const TreeArgs& a, cudaStream_t s) {
    const int64_t units = static_cast<int64_t>(a.rows) * a.nodes * a.hq;
    const unsigned grid = static_cast<unsigned>((units + kTreeWarps - 1) / kTreeWarps);
    if (a.d == 256) tree_warp_kernel<256><<<grid, kTreeWarps * 32, 0, s>>>(a);
    else tree_warp_kernel<128><<<grid, kTreeWarps * 32, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace wa
