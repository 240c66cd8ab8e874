// wa_tree_verify.cu — verification of drafted tokens against the target's probabilities.
//
// Walk from node 0: at node v with W = p = target[v], s = 1, child c with token x is
// kept when u_c q(x) s < W(x); otherwise W = max(W - s q, 0), s = sum of W.  Since a
// weight that reached 0 stays there,
//   W_k(x) = max(p(x) - S_k q(x), 0),  S_k = s_0 + .. + s_{k-1}:
// the state of a node is the one scalar S, and a test needs p and q at one token.
// Children without draft probabilities take their own token out instead (q = 1 there).
//
// One block per row, everything in float64.
#include <cuda_runtime.h>

#include "wa_internal.h"

namespace wa {

namespace {

constexpr int kVerThreads = 256;

__device__ __forceinline__ double prob(float x) { return x > 0.f ? static_cast<double>(fminf(x, 1.f)) : 0.0; }

__device__ double block_sum(double x, double* red) {
    for (int off = 16; off >= 1; off >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, off);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    double s = 0.0;
    for (int w = 0; w < kVerThreads / 32; ++w) s += red[w];
    __syncthreads();
    return s;
}

__global__ void __launch_bounds__(kVerThreads) verify_kernel(const VerifyArgs a) {
    __shared__ double red[kVerThreads / 32];
    __shared__ int gone[WA_TREE_MAX_NODES];   // tokens taken out of W (no draft probabilities)
    __shared__ int found;
    const int r = blockIdx.x, t = threadIdx.x, lane = t & 31, warp = t >> 5;
    int n = a.n ? a.n[r] : a.nodes;
    if (t == 0 && (n < 0 || n > a.nodes)) atomicOr(&a.hdr->status, WA_STATUS_BAD_TREE);
    n = min(max(n, 0), a.nodes);
    const int32_t* par = a.parent + static_cast<int64_t>(r) * a.nodes;
    const int32_t* tok = a.tokens + static_cast<int64_t>(r) * a.nodes;
    const float* u = a.u + static_cast<int64_t>(r) * a.nodes;
    int32_t* path = a.path + static_cast<int64_t>(r) * a.nodes;
    for (int i = t; i < n; i += kVerThreads)
        if (tree_parent(par[i], i) != par[i] || (i > 0 && (tok[i] < 0 || tok[i] >= a.vocab)))
            atomicOr(&a.hdr->status, WA_STATUS_BAD_TREE);
    int len = 0, node = 0, ngone = 0;
    double S = 0.0, s = 1.0;
    const float *p = nullptr, *q = nullptr;
    auto weight = [&](int x) -> double {
        if (q) return fmax(prob(p[x]) - S * prob(q[x]), 0.0);
        for (int k = 0; k < ngone; ++k)
            if (gone[k] == x) return 0.0;
        return prob(p[x]);
    };
    auto mass = [&]() {
        double y = 0.0;
        for (int x = t; x < a.vocab; x += kVerThreads) y += weight(x);
        return block_sum(y, red);
    };
    if (n == 0) {
        for (int i = t; i < a.nodes; i += kVerThreads) path[i] = -1;
        if (t == 0) {
            a.length[r] = 0;
            a.token[r] = -1;
        }
        return;
    }
    if (t == 0) path[0] = 0;
    for (bool moved = true; moved;) {
        moved = false;
        ++len;
        p = a.target + r * a.t_row + node * a.t_node;
        q = a.draft ? a.draft + r * a.d_row + node * a.d_node : nullptr;
        S = 0.0;
        s = 1.0;
        ngone = 0;
        for (int c = node + 1; c < n; ++c) {
            if (tree_parent(par[c], c) != node || tok[c] < 0 || tok[c] >= a.vocab) continue;
            const double qx = q ? prob(q[tok[c]]) : 1.0;
            if (static_cast<double>(u[c]) * qx * s < weight(tok[c])) {
                node = c;
                if (t == 0) path[len] = c;
                moved = true;
                break;
            }
            const double S0 = S;
            __syncthreads();
            if (q) S += s;
            else if (t == 0) gone[ngone] = tok[c];
            ++ngone;
            __syncthreads();
            const double left = mass();
            if (left > 0.0) {
                s = left;
            } else {
                S = S0;
                --ngone;
            }
        }
        __syncthreads();
    }
    // the last node's token: the first x whose running sum passes u[0] * mass
    const double want = static_cast<double>(u[0]) * mass();
    if (t == 0) found = -1;
    __syncthreads();
    double before = 0.0;
    int last = -1;      // the last x with weight, for a running sum that rounds to below `want`
    for (int base = 0; base < a.vocab; base += kVerThreads) {
        const int x = base + t;
        const double w = x < a.vocab ? weight(x) : 0.0;
        double y = w;
        for (int off = 1; off < 32; off <<= 1) {
            const double z = __shfl_up_sync(0xFFFFFFFFu, y, off);
            if (lane >= off) y += z;
        }
        if (lane == 31) red[warp] = y;
        __syncthreads();
        double at = before + y;
        for (int k = 0; k < warp; ++k) at += red[k];
        const bool hit = w > 0.0 && at > want;
        if (hit) atomicMin(reinterpret_cast<unsigned*>(&found), static_cast<unsigned>(x));
        if (w > 0.0) last = x;
        for (int k = 0; k < kVerThreads / 32; ++k) before += red[k];
        __syncthreads();
        if (found >= 0) break;
    }
    if (found < 0) {
        __shared__ int hi;
        if (t == 0) hi = -1;
        __syncthreads();
        atomicMax(&hi, last);
        __syncthreads();
        if (t == 0) found = hi;
        __syncthreads();
    }
    for (int i = len + t; i < a.nodes; i += kVerThreads) path[i] = -1;
    if (t == 0) {
        a.length[r] = len;
        a.token[r] = found;
        if (found < 0) atomicOr(&a.hdr->status, WA_STATUS_NO_MASS);
    }
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t s) {
    verify_kernel<<<a.rows, kVerThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace wa
