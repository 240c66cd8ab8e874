// wa_tree_verify.cu — verification of drafted tokens against the target's probabilities.
//
// Walk from node 0: at node v with W = p = target[v], s = 1, child c with token x is
// kept when u_c q(x) s < W(x); otherwise W = max(W - s q, 0), s = sum of W.  Since a
// weight that reached 0 stays there,
//   W_k(x) = max(p(x) - S_k q(x), 0),  S_k = s_0 + .. + s_{k-1}:
// the state of a node is the one scalar S, and a test needs p and q at one token.
// Children without draft probabilities take their own token out instead (q = 1 there).
// The vocabulary's rows are read only where a child was dropped (for the sum of W) and
// where the walk ends (for the token's place in the running sum of W).
//
// What bounds it: a chain of dependent passes over one node's rows, each of vocab / 8
// tokens a CTA, and at many rows the reads of those rows.  So
//   - a cluster of 8 CTAs serves a row, each a slice of the vocabulary, each warp a
//     stretch of the slice; totals meet in the cluster's shared memory;
//   - the tests' probabilities of all nodes are fetched at once at the start;
//   - a pass leaves the sums of every stretch, so the search for the token reads one
//     stretch again and not the rows.
//
// Sums carry hi + lo fp32 pairs (about 46 bits: the fp64 pipe of this GPU would take ten
// times as long), so that a border of the running sum that 64 bits would place on one
// side of a random number stays on that side but for numbers within about 2^-40 of it.
// Their order is fixed by vocab alone.
#include <cuda_runtime.h>

#include "wa_internal.h"

namespace wa {

namespace {

constexpr int kCluster = 8;
constexpr int kVerWarps = 16;
constexpr int kVerThreads = kVerWarps * 32;

__device__ __forceinline__ float prob(float x) { return x > 0.f ? fminf(x, 1.f) : 0.f; }

// An unevaluated sum hi + lo of two fp32 values.
struct Pair {
    float hi, lo;
};

// s + (d + e), |e| far below |d|: Knuth's exact sum of hi parts, the errors gathered in lo.
__device__ __forceinline__ void pair_add(Pair& s, float d, float e) {
    const float t = __fadd_rn(s.hi, d);
    const float b = __fsub_rn(t, s.hi);
    s.lo = __fadd_rn(s.lo, __fadd_rn(__fadd_rn(__fsub_rn(s.hi, __fsub_rn(t, b)), __fsub_rn(d, b)), e));
    s.hi = t;
}

// max(p - S q, 0) with S = sh + sl: the product's and the difference's rounding errors are kept.
__device__ __forceinline__ Pair weight_pair(float p, float q, float sh, float sl) {
    const float m = __fmul_rn(sh, q);
    const float me = __fmaf_rn(sl, q, __fmaf_rn(sh, q, -m));
    const float d = __fsub_rn(p, m);
    const float b = __fsub_rn(d, p);
    const float e = __fsub_rn(__fsub_rn(__fsub_rn(p, __fsub_rn(d, b)), __fadd_rn(m, b)), me);
    return __fadd_rn(d, e) > 0.f ? Pair{d, e} : Pair{0.f, 0.f};
}

__device__ __forceinline__ double pair_f64(const Pair& s) { return static_cast<double>(s.hi) + static_cast<double>(s.lo); }

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Store to the same shared-memory variable of CTA `rank` of the cluster.
__device__ __forceinline__ void st_cluster_f64(double* p, uint32_t rank, double x) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
    asm volatile("st.shared::cluster.f64 [%0], %1;" :: "r"(a), "d"(x) : "memory");
}

__device__ __forceinline__ double warp_scan_f64(double x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// The first of the warp's parts whose running sum (`before` + the inclusive scan) passes `want`, else the
// last part with any weight (rounding can leave the sum just below); -1 if there is none.  `before`
// becomes the sum before that part.
__device__ __forceinline__ int pick(double part, double want, double& before, int lane) {
    const double run = before + warp_scan_f64(part, lane);
    const uint32_t some = __ballot_sync(0xFFFFFFFFu, part > 0.0);
    const uint32_t hit = some & __ballot_sync(0xFFFFFFFFu, run > want);
    if (some == 0u) return -1;
    const int at = hit ? __ffs(hit) - 1 : 31 - __clz(some);
    const double prev = __shfl_sync(0xFFFFFFFFu, run, max(at - 1, 0));
    if (at > 0) before = prev;
    return at;
}

struct VerifyShared {
    double seg[kVerWarps];              // sums of this CTA's stretches
    double tot[2][kCluster];            // the CTAs' sums, by pass parity
    double sub[kVerWarps];
    double mass, want, before;
    float pp[WA_TREE_MAX_NODES], qq[WA_TREE_MAX_NODES];   // a node's token at its parent: target, draft
    float u[WA_TREE_MAX_NODES];
    int par[WA_TREE_MAX_NODES], tok[WA_TREE_MAX_NODES];
    uint32_t kids[WA_TREE_MAX_NODES][4];
    int gone[WA_TREE_MAX_NODES];        // tokens out of W (no draft probabilities)
    int ngone, node, len, cmd, stretch;
    float sh, sl;                       // S
};

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kVerThreads, 2) verify_kernel(const VerifyArgs a) {
    __shared__ VerifyShared sm;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int rank = static_cast<int>(cluster_rank());
    const int r = blockIdx.x / kCluster;
    const int raw_n = a.n ? a.n[r] : a.nodes;
    const int n = min(max(raw_n, 0), a.nodes);
    const bool draft = a.draft != nullptr;
    // shared memory of another CTA may be written once that CTA runs: the wait is before the walk
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    const float* trow = a.target + r * a.t_row;
    const float* drow = draft ? a.draft + r * a.d_row : nullptr;
    int32_t* path = a.path + static_cast<int64_t>(r) * a.nodes;

    // the tree, and every test's probabilities
    if (t < WA_TREE_MAX_NODES) {
#pragma unroll
        for (int w = 0; w < 4; ++w) sm.kids[t][w] = 0u;
    }
    if (t == 0) sm.ngone = 0;
    __syncthreads();
    if (t < n) {
        const int64_t at = static_cast<int64_t>(r) * a.nodes + t;
        const int raw = a.parent[at], par = tree_parent(raw, t);
        const int tok = t > 0 ? a.tokens[at] : 0;
        const bool in = tok >= 0 && tok < a.vocab;
        if (rank == 0 && (raw != par || !in)) atomicOr(&a.hdr->status, WA_STATUS_BAD_TREE);
        sm.par[t] = par;
        sm.tok[t] = tok;
        sm.u[t] = a.u[at];
        if (par >= 0 && in) {
            sm.pp[t] = prob(trow[par * a.t_node + tok]);
            sm.qq[t] = draft ? prob(drow[par * a.d_node + tok]) : 1.f;
            atomicOr(&sm.kids[par][t >> 5], 1u << (t & 31));
        }
    }
    if (t == 0 && rank == 0 && raw_n != n) atomicOr(&a.hdr->status, WA_STATUS_BAD_TREE);
    __syncthreads();

    // this warp's stretch of the vocabulary
    const int slice = (a.vocab + kCluster - 1) / kCluster;
    const int len_w = ((slice + kVerWarps - 1) / kVerWarps + 31) / 32 * 32;
    const int c0 = min(a.vocab, rank * slice), c1 = min(a.vocab, c0 + slice);
    const int x0 = min(c1, c0 + warp * len_w), x1 = min(c1, x0 + len_w);

    // the weight of token x at the current node
    auto weight_at = [&](const float* p, const float* q, int x, float sh, float sl, int ngone) -> Pair {
        if (draft) return weight_pair(prob(p[x]), prob(q[x]), sh, sl);
        for (int k = 0; k < ngone; ++k)
            if (sm.gone[k] == x) return Pair{0.f, 0.f};
        return Pair{prob(p[x]), 0.f};
    };
    // The sum of W over [b0, b1) by one warp, in lane 0.
    auto stretch_sum = [&](const float* p, const float* q, int b0, int b1, float sh, float sl) -> double {
        int ngone = 0;
        if (!draft) {       // only the stretches that hold a token taken out look for it
            bool here = false;
            for (int k = lane; k < sm.ngone; k += 32) here |= sm.gone[k] >= b0 && sm.gone[k] < b1;
            ngone = __any_sync(0xFFFFFFFFu, here) ? sm.ngone : 0;
        }
        Pair s{0.f, 0.f};
        int x = b0 + lane;
        if (draft) {
            for (; x + 7 * 32 < b1; x += 8 * 32) {
                float pv[8], qv[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    pv[e] = __ldg(p + x + e * 32);
                    qv[e] = __ldg(q + x + e * 32);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const Pair w = weight_pair(prob(pv[e]), prob(qv[e]), sh, sl);
                    pair_add(s, w.hi, w.lo);
                }
            }
        } else if (ngone == 0) {
            for (; x + 7 * 32 < b1; x += 8 * 32) {
                float pv[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) pv[e] = __ldg(p + x + e * 32);
#pragma unroll
                for (int e = 0; e < 8; ++e) pair_add(s, prob(pv[e]), 0.f);
            }
        }
        for (; x < b1; x += 32) {
            const Pair w = weight_at(p, q, x, sh, sl, ngone);
            pair_add(s, w.hi, w.lo);
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
            const float hi = __shfl_xor_sync(0xFFFFFFFFu, s.hi, o), lo = __shfl_xor_sync(0xFFFFFFFFu, s.lo, o);
            pair_add(s, hi, lo);
        }
        return pair_f64(s);
    };

    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    // Warp 0 of every CTA walks alike; the whole cluster sums W when it asks for it.
    int pass = 0;
    int len = 0, node = 0;
    double S = 0.0, s = 1.0;
    uint32_t kids[4] = {0u, 0u, 0u, 0u};
    bool summed = false;      // the stretches' sums are those of the current W
    double S_prev = 0.0;
    bool asked = false;       // a child was dropped and the sum is awaited
    if (warp == 0 && n > 0) {
        len = 1;
        if (rank == 0 && lane == 0) path[0] = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) kids[w] = sm.kids[0][w];
    }
    while (n > 0) {
        if (warp == 0) {
            bool pass_wanted = false;
            if (asked) {
                asked = false;
                const double left = sm.mass;
                if (left > 0.0) {
                    s = left;
                    summed = true;
                } else {               // nothing left: W stays as it was
                    S = S_prev;
                    if (!draft && lane == 0) --sm.ngone;
                    summed = false;
                }
                __syncwarp();
            }
            for (;;) {
                int c = -1;
#pragma unroll
                for (int w = 3; w >= 0; --w)
                    if (kids[w]) c = 32 * w + __ffs(kids[w]) - 1;
                if (c < 0) break;
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    if (w == (c >> 5)) kids[w] &= kids[w] - 1u;
                const double pp = sm.pp[c], qq = sm.qq[c];
                double W = pp - S * qq;
                if (!draft) {
                    W = pp;
                    for (int k = 0; k < sm.ngone; ++k)
                        if (sm.gone[k] == sm.tok[c]) W = 0.0;
                }
                if (static_cast<double>(sm.u[c]) * qq * s < fmax(W, 0.0)) {
                    node = c;
                    if (rank == 0 && lane == 0) path[len] = c;
                    ++len;
                    S = 0.0;
                    s = 1.0;
                    summed = false;
                    __syncwarp();
                    if (lane == 0) sm.ngone = 0;
                    __syncwarp();
#pragma unroll
                    for (int w = 0; w < 4; ++w) kids[w] = sm.kids[c][w];
                    continue;
                }
                S_prev = S;
                if (draft) S += s;
                __syncwarp();
                if (!draft && lane == 0) sm.gone[sm.ngone++] = sm.tok[c];
                __syncwarp();
                asked = pass_wanted = true;
                break;
            }
            if (lane == 0) {
                sm.cmd = pass_wanted ? 1 : summed ? 0 : 2;     // 0: sample; 1: sum and go on; 2: sum, then sample
                sm.node = node;
                sm.sh = static_cast<float>(S);
                sm.sl = static_cast<float>(S - static_cast<double>(static_cast<float>(S)));
            }
        }
        __syncthreads();
        const int cmd = sm.cmd;
        const float sh = sm.sh, sl = sm.sl;
        const float* p = trow + sm.node * a.t_node;
        const float* q = draft ? drow + sm.node * a.d_node : nullptr;
        if (cmd != 0) {
            const double x = stretch_sum(p, q, x0, x1, sh, sl);
            if (lane == 0) sm.seg[warp] = x;
            __syncthreads();
            double* tot = sm.tot[pass & 1];
            if (warp == 0) {
                const double run = warp_scan_f64(lane < kVerWarps ? sm.seg[lane] : 0.0, lane);
                const double all = __shfl_sync(0xFFFFFFFFu, run, 31);
                if (lane < kCluster) st_cluster_f64(&tot[rank], lane, all);
            }
            cluster_sync_all();
            if (warp == 0) {
                const double run = warp_scan_f64(lane < kCluster ? tot[lane] : 0.0, lane);
                if (lane == 31) sm.mass = run;
            }
            ++pass;
            __syncthreads();
        }
        if (cmd == 1) continue;

        // the token: the CTA, its stretch, a sixteenth of the stretch, the place
        if (warp == 0) {
            const double want = static_cast<double>(sm.u[0]) * sm.mass;
            double before = 0.0;
            const int at = pick(lane < kCluster ? sm.tot[(pass - 1) & 1][lane] : 0.0, want, before, lane);
            int st = -1;
            if (at == rank) st = pick(lane < kVerWarps ? sm.seg[lane] : 0.0, want, before, lane);
            if (at < 0 && rank == 0 && lane == 0) {
                a.token[r] = -1;
                atomicOr(&a.hdr->status, WA_STATUS_NO_MASS);
            }
            if (lane == 0) {
                sm.stretch = st;
                sm.want = want;
                sm.before = before;
            }
        }
        __syncthreads();
        if (sm.stretch < 0) break;
        const int b0 = min(c1, c0 + sm.stretch * len_w), b1 = min(c1, b0 + len_w);
        const int part = ((b1 - b0 + kVerWarps - 1) / kVerWarps + 31) / 32 * 32;
        const int y0 = min(b1, b0 + warp * part), y1 = min(b1, y0 + part);
        const double x = stretch_sum(p, q, y0, y1, sh, sl);
        if (lane == 0) sm.sub[warp] = x;
        __syncthreads();
        if (warp == 0) {
            const double want = sm.want;
            double before = sm.before;
            const int k = max(pick(lane < kVerWarps ? sm.sub[lane] : 0.0, want, before, lane), 0);
            const int z0 = min(b1, b0 + k * part), z1 = min(b1, z0 + part);
            int found = -1, last = -1;
            for (int z = z0; z < z1 && found < 0; z += 32) {
                const double w = z + lane < z1 ? pair_f64(weight_at(p, q, z + lane, sh, sl, sm.ngone)) : 0.0;
                const double run = before + warp_scan_f64(w, lane);
                const uint32_t some = __ballot_sync(0xFFFFFFFFu, w > 0.0);
                const uint32_t hit = some & __ballot_sync(0xFFFFFFFFu, run > want);
                if (hit) found = z + __ffs(hit) - 1;
                if (some) last = z + 31 - __clz(some);
                before = __shfl_sync(0xFFFFFFFFu, run, 31);
            }
            if (lane == 0) a.token[r] = found >= 0 ? found : last;
        }
        break;
    }
    if (warp == 0 && rank == 0) {
        for (int i = len + lane; i < a.nodes; i += 32) path[i] = -1;
        if (lane == 0) {
            a.length[r] = len;
            if (n == 0) a.token[r] = -1;
        }
    }
    // no CTA leaves while another one may still write to its shared memory: every such write is
    // followed by a cluster barrier that both pass
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t s) {
    verify_kernel<<<a.rows * kCluster, kVerThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace wa
