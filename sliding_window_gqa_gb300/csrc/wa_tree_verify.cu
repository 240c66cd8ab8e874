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
// What bounds it: a chain of dependent passes over one node's rows, each a trip to memory
// and a meeting of the CTAs, and at many rows the reads of those rows (one row of 8 nodes,
// 32,768 tokens: 7.6 us; 64 rows of 16 nodes, 131,072 tokens: 44.9 us, where the rows that the
// walks need take 10 us at the copy rate; 24 rows of 26 nodes without draft probabilities,
// 100,003 tokens: 19.9 us; as graph replays, and 8.7, 46.7 and 21.7 us called from Python one
// after another).  So
//   - the vocabulary is cut into 8 slices of 16 stretches; a cluster of 8, 4, 2 or 1 CTAs
//     serves a row (fewer for many rows), each with its share
//     of the slices, each warp one stretch of a slice; the slices' sums meet in the cluster's
//     shared memory;
//   - the tests' probabilities of all nodes are fetched at once at the start;
//   - a pass leaves the sums of every stretch, so the search for the token reads one
//     stretch again and not the rows, and a token taken out (no draft probabilities) only
//     changes its own stretch.
//
// All arithmetic is in hi + lo fp32 pairs (about 46 bits), two tokens an instruction where it
// counts: the fp64 pipe of this GPU has a fiftieth of the fp32 rate.  A weight is off by at most 2^-45 p(x) and by q(x)
// times S's error, 2^-47 a dropped child; a weight that is not 0 enters the sums as hi > 0 with |lo| <= 2^-24 hi, so that
// hi alone says whether a sum, however small, has any weight.  So the token differs from the one that 64 bits would
// choose only where a random number's place in the running sum is within about 2^-42 of a border: that is of
// probability 1, not of what the drafts have left of it.  The order of the sums is fixed by vocab alone, whatever the
// cluster.
#include <cuda_runtime.h>

#include "wa_internal.h"
#include "wa_ptx.cuh"

namespace wa {

namespace {

constexpr int kSlices = 8;
constexpr int kVerWarps = 16;
constexpr int kVerThreads = kVerWarps * 32;

// x in [0, 1]; NaN is 0.
__device__ __forceinline__ float prob(float x) { return __saturatef(x); }

// An unevaluated sum hi + lo of two fp32 values.
struct __align__(8) Pair {
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
    const float h = __fadd_rn(d, e);
    return h > 0.f ? Pair{h, __fsub_rn(e, __fsub_rn(h, d))} : Pair{0.f, 0.f};
}

// Two tokens at a time: packed fp32 operations (one instruction each, rounded as the plain ones).
struct Two {
    float a, b;
};
__device__ __forceinline__ Two mul2(const Two& x, const Two& y) {
    Two r;
    asm("{\n\t.reg .b64 p, q, r;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\tmul.rn.f32x2 r, p, q;\n\tmov.b64 {%0, %1}, r;\n\t}"
        : "=f"(r.a), "=f"(r.b) : "f"(x.a), "f"(x.b), "f"(y.a), "f"(y.b));
    return r;
}
__device__ __forceinline__ Two add2(const Two& x, const Two& y) {
    Two r;
    asm("{\n\t.reg .b64 p, q, r;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\tadd.rn.f32x2 r, p, q;\n\tmov.b64 {%0, %1}, r;\n\t}"
        : "=f"(r.a), "=f"(r.b) : "f"(x.a), "f"(x.b), "f"(y.a), "f"(y.b));
    return r;
}
__device__ __forceinline__ Two fma2(const Two& x, const Two& y, const Two& z) {
    Two r;
    asm("{\n\t.reg .b64 p, q, c, r;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 r, p, q, c;\n\tmov.b64 {%0, %1}, r;\n\t}"
        : "=f"(r.a), "=f"(r.b) : "f"(x.a), "f"(x.b), "f"(y.a), "f"(y.b), "f"(z.a), "f"(z.b));
    return r;
}
__device__ __forceinline__ Two sub2(const Two& x, const Two& y) { return fma2(y, Two{-1.f, -1.f}, x); }

// pair_add of two sums side by side.
__device__ __forceinline__ void pair_add2(Two& hi, Two& lo, const Two& d, const Two& e) {
    const Two t = add2(hi, d), b = sub2(t, hi);
    lo = add2(lo, add2(add2(sub2(hi, sub2(t, b)), sub2(d, b)), e));
    hi = t;
}

// weight_pair of two tokens; ns* = -S.
__device__ __forceinline__ void weight_pair2(const Two& p, const Two& q, const Two& sh, const Two& nsh, const Two& nsl, Two& d, Two& e) {
    const Two m = mul2(sh, q);
    const Two nme = fma2(nsl, q, fma2(nsh, q, m));                 // m - S q
    d = sub2(p, m);
    const Two b = sub2(d, p);
    e = add2(sub2(sub2(p, sub2(d, b)), add2(m, b)), nme);
    const Two h = add2(d, e);
    e = sub2(e, sub2(h, d));
    d = h;
    if (!(h.a > 0.f)) d.a = e.a = 0.f;
    if (!(h.b > 0.f)) d.b = e.b = 0.f;
}

// Whether a < b: equal hi parts are told apart by lo.
__device__ __forceinline__ bool pair_less(const Pair& a, const Pair& b) {
    return __fadd_rn(__fsub_rn(a.hi, b.hi), __fsub_rn(a.lo, b.lo)) < 0.f;
}

// x * s
__device__ __forceinline__ Pair pair_scale(float x, const Pair& s) {
    const float h = __fmul_rn(x, s.hi);
    return Pair{h, __fmaf_rn(x, s.lo, __fmaf_rn(x, s.hi, -h))};
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// Store to the same shared-memory variable of CTA `rank` of the cluster, counted on that CTA's mbarrier.
__device__ __forceinline__ void st_cluster_pair(Pair* p, uint64_t* bar, uint32_t rank, const Pair& x) {
    uint32_t a, b;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(smem_u32(bar)), "r"(rank));
    const uint64_t v = static_cast<uint64_t>(__float_as_uint(x.hi)) | static_cast<uint64_t>(__float_as_uint(x.lo)) << 32;
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" :: "r"(a), "l"(v), "r"(b) : "memory");
}

__device__ __forceinline__ Pair warp_scan(Pair x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float hi = __shfl_up_sync(0xFFFFFFFFu, x.hi, o), lo = __shfl_up_sync(0xFFFFFFFFu, x.lo, o);
        if (lane >= o) pair_add(x, hi, lo);
    }
    return x;
}

__device__ __forceinline__ Pair warp_get(const Pair& x, int lane) {
    return Pair{__shfl_sync(0xFFFFFFFFu, x.hi, lane), __shfl_sync(0xFFFFFFFFu, x.lo, lane)};
}

// The first of the warp's parts whose running sum (`before` + the inclusive scan) passes `want`, else the
// last part with any weight (rounding can leave the sum just below); -1 if there is none.  `before`
// becomes the sum before that part.
__device__ __forceinline__ int pick(const Pair& part, const Pair& want, Pair& before, int lane) {
    Pair run = warp_scan(part, lane);
    pair_add(run, before.hi, before.lo);
    const uint32_t some = __ballot_sync(0xFFFFFFFFu, part.hi > 0.f);
    const uint32_t hit = some & __ballot_sync(0xFFFFFFFFu, pair_less(want, run));
    if (some == 0u) return -1;
    const int at = hit ? __ffs(hit) - 1 : 31 - __clz(some);
    const Pair prev = warp_get(run, max(at - 1, 0));
    if (at > 0) before = prev;
    return at;
}

struct VerifyShared {
    uint64_t bar[2];                    // the slices' sums of a pass have arrived, by pass parity
    Pair seg[kSlices][kVerWarps];       // sums of the stretches of this CTA's slices
    Pair tot[2][kSlices];               // the slices' sums, by pass parity
    Pair sub[kVerWarps];
    Pair mass, want, before;
    float pp[WA_TREE_MAX_NODES], qq[WA_TREE_MAX_NODES];   // a node's token at its parent: target, draft
    float u[WA_TREE_MAX_NODES];
    int par[WA_TREE_MAX_NODES], tok[WA_TREE_MAX_NODES];
    uint2 kids[WA_TREE_MAX_NODES][2];   // a node's children as bits
    int gone[WA_TREE_MAX_NODES];        // tokens out of W (no draft probabilities)
    // the walk, as warp 0 left it
    Pair s, S_prev;
    unsigned long long kids_lo, kids_hi;      // the current node's children that are still to test
    int summed;                               // the stretches' sums are those of the current W
    int asked;                                // a child was dropped and the sum is awaited
    int ngone, node, len, cmd, slice, stretch;
    int late;                           // a sum of another CTA did not arrive in time
    int changed;                        // no draft: the one token that left W since the sums, or -1
    Pair S;
};

// The status word before the rows' kernel, which is launched while this one runs.
__global__ void clear_kernel(WsHeader* hdr) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    hdr->status = 0;
}

template <int CL, bool DRAFT>
__global__ void __cluster_dims__(CL, 1, 1) __launch_bounds__(kVerThreads, 2) verify_kernel(const __grid_constant__ VerifyArgs a) {
    constexpr int PER = kSlices / CL;           // slices of a CTA
    __shared__ VerifyShared sm;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int rank = static_cast<int>(cluster_rank());
    const int r = blockIdx.x / CL;
    const int raw_n = a.n ? a.n[r] : a.nodes;
    const int n = min(max(raw_n, 0), a.nodes);
    const float* trow = a.target + r * a.t_row;
    const float* drow = DRAFT ? a.draft + r * a.d_row : nullptr;
    int32_t* path = a.path + static_cast<int64_t>(r) * a.nodes;

    // the tree, and every test's probabilities
    if (t < WA_TREE_MAX_NODES) {
        sm.kids[t][0] = sm.kids[t][1] = make_uint2(0u, 0u);
    }
    if (t == 0) {
        if (a.rows == 1 && rank == 0) a.hdr->status = 0;     // seen by the others after the barriers below
        sm.ngone = 0;
        mbar_init(smem_u32(&sm.bar[0]), 1);
        mbar_init(smem_u32(&sm.bar[1]), 1);
        fence_mbar_init();
    }
    __syncthreads();
    // another CTA's shared memory may be written once that CTA has come here: the wait is before the walk
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    int bad = 0;
    if (t < n) {
        const int64_t at = static_cast<int64_t>(r) * a.nodes + t;
        const int raw = a.parent[at], par = tree_parent(raw, t);
        const int tok = t > 0 ? a.tokens[at] : 0;
        const bool in = tok >= 0 && tok < a.vocab;
        if (raw != par || !in) bad = WA_STATUS_BAD_TREE;
        sm.par[t] = par;
        sm.tok[t] = tok;
        sm.u[t] = a.u[at];
        if (par >= 0 && in) {
            sm.pp[t] = prob(trow[par * a.t_node + tok]);
            sm.qq[t] = DRAFT ? prob(drow[par * a.d_node + tok]) : 1.f;
            atomicOr(reinterpret_cast<uint32_t*>(&sm.kids[par][0]) + (t >> 5), 1u << (t & 31));
        }
    }
    if (raw_n != n) bad = WA_STATUS_BAD_TREE;
    __syncthreads();

    // stretch `st` of slice `sl` is [stretch_at(sl, st), stretch_at(sl, st + 1))
    const int slice = ((a.vocab + kSlices - 1) / kSlices + 3) / 4 * 4;
    const int len_w = ((slice + kVerWarps - 1) / kVerWarps + 127) / 128 * 128;
    auto stretch_at = [&](int sl, int st) { return min(a.vocab, min((sl + 1) * slice, sl * slice + st * len_w)); };   // multiples of 4, or vocab

    // a token's weight at the current node, given its probabilities
    auto weight = [&](float px, float qx, int x, const Pair& S, int ngone) -> Pair {
        if (DRAFT) return weight_pair(prob(px), prob(qx), S.hi, S.lo);
        for (int k = 0; k < ngone; ++k)
            if (sm.gone[k] == x) return Pair{0.f, 0.f};
        return Pair{prob(px), 0.f};
    };
    // The sum of W over [b0, b1), b0 a multiple of 4, by one warp, the same in every lane.  A lane takes four
    // tokens in a row, 16 bytes where the rows lie on such borders (the order of the sum is the same where
    // they do not), and kLoads such groups at a time.
    constexpr int kLoads = DRAFT ? 4 : 8;
    auto stretch_sum = [&](const float* p, const float* q, int b0, int b1, const Pair& S) -> Pair {
        int ngone = 0;
        if (!DRAFT) {       // only the stretches that hold a token taken out look for it
            bool here = false;
            for (int k = lane; k < sm.ngone; k += 32) here |= sm.gone[k] >= b0 && sm.gone[k] < b1;
            ngone = __any_sync(0xFFFFFFFFu, here) ? sm.ngone : 0;
        }
        const bool vec_p = (reinterpret_cast<uintptr_t>(p) & 15u) == 0, vec_q = (reinterpret_cast<uintptr_t>(q) & 15u) == 0;
        auto load = [&](const float* row, int x, bool vec) -> float4 {
            if (vec && x + 4 <= b1) return __ldg(reinterpret_cast<const float4*>(row + x));
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (x < b1) v.x = __ldg(row + x);
            if (x + 1 < b1) v.y = __ldg(row + x + 1);
            if (x + 2 < b1) v.z = __ldg(row + x + 2);
            if (x + 3 < b1) v.w = __ldg(row + x + 3);
            return v;
        };
        Two hi{0.f, 0.f}, lo{0.f, 0.f};
        const Two sh{S.hi, S.hi}, nsh{-S.hi, -S.hi}, nsl{-S.lo, -S.lo};
        for (int x = b0 + 4 * lane; x - 4 * lane < b1; x += kLoads * 128) {
            float4 pv[kLoads], qv[kLoads];
#pragma unroll
            for (int e = 0; e < kLoads; ++e) {
                pv[e] = load(p, x + e * 128, vec_p);
                if (DRAFT) qv[e] = load(q, x + e * 128, vec_q);
            }
#pragma unroll
            for (int e = 0; e < kLoads; ++e) {
                Two p0{prob(pv[e].x), prob(pv[e].y)}, p1{prob(pv[e].z), prob(pv[e].w)};
                if (DRAFT) {
                    const Two q0{prob(qv[e].x), prob(qv[e].y)}, q1{prob(qv[e].z), prob(qv[e].w)};
                    Two d, err;
                    weight_pair2(p0, q0, sh, nsh, nsl, d, err);
                    pair_add2(hi, lo, d, err);
                    weight_pair2(p1, q1, sh, nsh, nsl, d, err);
                    pair_add2(hi, lo, d, err);
                } else {
                    for (int k = 0; k < ngone; ++k) {
                        const int at = sm.gone[k] - (x + e * 128);
                        if (at == 0) p0.a = 0.f;
                        if (at == 1) p0.b = 0.f;
                        if (at == 2) p1.a = 0.f;
                        if (at == 3) p1.b = 0.f;
                    }
                    pair_add2(hi, lo, p0, Two{0.f, 0.f});
                    pair_add2(hi, lo, p1, Two{0.f, 0.f});
                }
            }
        }
        Pair s{hi.a, lo.a};
        pair_add(s, hi.b, lo.b);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
            const float hi = __shfl_xor_sync(0xFFFFFFFFu, s.hi, o), lo = __shfl_xor_sync(0xFFFFFFFFu, s.lo, o);
            pair_add(s, hi, lo);
        }
        return s;
    };

    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");      // the status word is clear
    if (bad != 0 && rank == 0) atomicOr(&a.hdr->status, bad);
    // Warp 0 of every CTA walks alike; the whole cluster sums W when it asks for it.  Between two passes the
    // walk's state lies in shared memory (as registers it was spilled).
    int pass = 0;
    if (t == 0) {
        sm.kids_lo = sm.kids[0][0].x | static_cast<unsigned long long>(sm.kids[0][0].y) << 32;
        sm.kids_hi = sm.kids[0][1].x | static_cast<unsigned long long>(sm.kids[0][1].y) << 32;
        sm.S = sm.S_prev = Pair{0.f, 0.f};
        sm.s = Pair{1.f, 0.f};
        sm.summed = sm.asked = sm.late = 0;
        sm.node = 0;
        sm.len = n > 0;
        if (rank == 0 && n > 0) path[0] = 0;
    }
    while (n > 0) {
        if (warp == 0) {
            __syncwarp();
            Pair S = sm.S, s = sm.s, S_prev = sm.S_prev;
            unsigned long long kids_lo = sm.kids_lo, kids_hi = sm.kids_hi;
            int node = sm.node, len = sm.len, ngone = sm.ngone;
            bool summed = sm.summed != 0, asked = false;
            int changed = -1;         // the only token whose weight has changed since the last sums, or -1
            if (sm.asked) {
                const Pair left = sm.mass;
                summed = left.hi > 0.f;
                if (summed) {
                    s = left;
                } else {               // nothing left: W stays as it was
                    S = S_prev;
                    if (!DRAFT) --ngone;
                }
            }
            while (kids_lo | kids_hi) {
                int c;
                if (kids_lo) {
                    c = __ffsll(kids_lo) - 1;
                    kids_lo &= kids_lo - 1;
                } else {
                    c = 63 + __ffsll(kids_hi);
                    kids_hi &= kids_hi - 1;
                }
                const float pp = sm.pp[c], qq = sm.qq[c], uc = sm.u[c], uq = __fmul_rn(uc, qq);
                const int x = sm.tok[c];
                Pair W{pp, 0.f};
                if (DRAFT) {
                    W = weight_pair(pp, qq, S.hi, S.lo);
                } else {
                    for (int k = 0; k < ngone; ++k)
                        if (sm.gone[k] == x) W.hi = 0.f;
                }
                Pair bar = pair_scale(uq, s);                 // u q s, with u q's own rounding error
                bar.lo = __fmaf_rn(__fmaf_rn(uc, qq, -uq), s.hi, bar.lo);
                if (pair_less(bar, W)) {
                    node = c;
                    if (rank == 0 && lane == 0) path[len] = c;
                    ++len;
                    S = Pair{0.f, 0.f};
                    s = Pair{1.f, 0.f};
                    summed = false;
                    ngone = 0;
                    kids_lo = sm.kids[c][0].x | static_cast<unsigned long long>(sm.kids[c][0].y) << 32;
                    kids_hi = sm.kids[c][1].x | static_cast<unsigned long long>(sm.kids[c][1].y) << 32;
                    continue;
                }
                S_prev = S;
                if (DRAFT) {
                    pair_add(S, s.hi, s.lo);
                } else {
                    changed = summed ? x : -1;
                    if (lane == 0) sm.gone[ngone] = x;
                    ++ngone;
                }
                asked = true;
                break;
            }
            if (lane == 0) {
                sm.S = S;
                sm.s = s;
                sm.S_prev = S_prev;
                sm.kids_lo = kids_lo;
                sm.kids_hi = kids_hi;
                sm.node = node;
                sm.len = len;
                sm.ngone = ngone;
                sm.summed = summed;
                sm.asked = asked;
                sm.changed = asked ? changed : -1;
                // 0: sample; 1: sum and go on; 2: sum, then sample; 3: stop, nothing more is sent
                sm.cmd = sm.late ? 3 : asked ? 1 : summed ? 0 : 2;
            }
        }
        __syncthreads();
        const int cmd = sm.cmd;
        if (cmd == 3) break;
        const Pair Sn = sm.S;
        const float* p = trow + sm.node * a.t_node;
        const float* q = DRAFT ? drow + sm.node * a.d_node : nullptr;
        if (cmd != 0) {
            const int only = sm.changed;
#pragma unroll 1
            for (int k = 0; k < PER; ++k) {
                const int sl_ = rank * PER + k, b0 = stretch_at(sl_, warp), b1 = stretch_at(sl_, warp + 1);
                if (only >= 0 && (only < b0 || only >= b1)) continue;
                const Pair x = stretch_sum(p, q, b0, b1, Sn);
                if (lane == 0) sm.seg[k][warp] = x;
            }
            __syncthreads();
            Pair* tot = sm.tot[pass & 1];
            uint64_t* bar = &sm.bar[pass & 1];
            if (warp < PER) {
                const Pair all = warp_get(warp_scan(lane < kVerWarps ? sm.seg[warp][lane] : Pair{0.f, 0.f}, lane), 31);
                if (lane < CL) st_cluster_pair(&tot[rank * PER + warp], bar, lane, all);
            }
            // Only warp 0 waits for the other CTAs' sums (a cluster barrier of all warps lets the last one go
            // 4,000 cycles after the first).  A pass's barrier and buffer are used again two passes on, when
            // every CTA has sent, and so has read this pass's.
            if (warp == 0) {
                if (lane == 0) mbar_arrive_expect_tx(smem_u32(bar), kSlices * sizeof(Pair));
                const bool ok = warp_wait(smem_u32(bar), (pass >> 1) & 1, &a.hdr->status);
                const Pair run = warp_scan(ok && lane < kSlices ? tot[lane] : Pair{0.f, 0.f}, lane);
                if (lane == 31) {
                    sm.mass = run;
                    sm.late = !ok;
                }
                __syncwarp();
            }
            ++pass;
        }
        if (cmd == 1) continue;

        // the token: the CTA, its stretch, a sixteenth of the stretch, the place
        if (warp == 0) {
            const Pair want = pair_scale(sm.u[0], sm.mass);
            Pair before{0.f, 0.f};
            const bool sums = lane < kSlices && !sm.late;
            const int at = pick(sums ? sm.tot[(pass - 1) & 1][lane] : Pair{0.f, 0.f}, want, before, lane);
            int st = -1;
            if (at >= 0 && at / PER == rank) st = pick(lane < kVerWarps ? sm.seg[at % PER][lane] : Pair{0.f, 0.f}, want, before, lane);
            if (at < 0 && rank == 0 && lane == 0) {
                a.token[r] = -1;
                atomicOr(&a.hdr->status, WA_STATUS_NO_MASS);
            }
            if (lane == 0) {
                sm.slice = at;
                sm.stretch = st;
                sm.want = want;
                sm.before = before;
            }
        }
        __syncthreads();
        if (sm.stretch < 0) break;
        const int b0 = stretch_at(sm.slice, sm.stretch), b1 = stretch_at(sm.slice, sm.stretch + 1);
        const int part = ((b1 - b0 + kVerWarps - 1) / kVerWarps + 31) / 32 * 32;   // a multiple of 4
        const int y0 = min(b1, b0 + warp * part), y1 = min(b1, y0 + part);
        const Pair x = stretch_sum(p, q, y0, y1, Sn);
        if (lane == 0) sm.sub[warp] = x;
        __syncthreads();
        if (warp == 0) {
            const Pair want = sm.want;
            Pair before = sm.before;
            const int k = max(pick(lane < kVerWarps ? sm.sub[lane] : Pair{0.f, 0.f}, want, before, lane), 0);
            const int z0 = min(b1, b0 + k * part), z1 = min(b1, z0 + part);
            int found = -1, last = -1;
            for (int z = z0; z < z1 && found < 0; z += 32) {
                const bool in = z + lane < z1;
                const Pair w = in ? weight(p[z + lane], DRAFT ? q[z + lane] : 0.f, z + lane, Sn, sm.ngone) : Pair{0.f, 0.f};
                Pair run = warp_scan(w, lane);
                pair_add(run, before.hi, before.lo);
                const uint32_t some = __ballot_sync(0xFFFFFFFFu, w.hi > 0.f);
                const uint32_t hit = some & __ballot_sync(0xFFFFFFFFu, pair_less(want, run));
                if (hit) found = z + __ffs(hit) - 1;
                if (some) last = z + 31 - __clz(some);
                before = warp_get(run, 31);
            }
            if (lane == 0) a.token[r] = found >= 0 ? found : last;
        }
        break;
    }
    if (warp == 0 && rank == 0) {
        __syncwarp();
        for (int i = sm.len + lane; i < a.nodes; i += 32) path[i] = -1;
        if (lane == 0) {
            a.length[r] = sm.len;
            if (n == 0) a.token[r] = -1;
        }
    }
    // No CTA leaves while another one may still write to its shared memory.  One that had all sums of every pass gets no
    // more, since all make the same passes; it arrives at the cluster's barrier and leaves.  One that gave up on a pass
    // stays until all have arrived, which is bounded, since every wait before it is: until then a CTA that did get
    // everything may send the next pass's sums.  Then it waits once more for the pass that it gave up on, since a slow CTA
    // may have sent its sums only just now; a later pass's have landed, for their sender has waited in vain since.  (With
    // every CTA waiting here a row of 32,768 tokens took 10.3 us a call from Python; now 8.6, as without a barrier.)
    if (n > 0) {
        __syncwarp();
        asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
        if (sm.late) {
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
            if (warp == 0) warp_wait(smem_u32(&sm.bar[(pass - 1) & 1]), ((pass - 1) >> 1) & 1, &a.hdr->status);
        }
    }
}

template <int CL>
cudaError_t launch_cl(const VerifyArgs& a, cudaStream_t s) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(a.rows) * CL);
    cfg.blockDim = dim3(kVerThreads);
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = a.rows > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, a.draft ? verify_kernel<CL, true> : verify_kernel<CL, false>, a);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t s) {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return cudaErrorInvalidValue;
    // a single row's cluster clears the status itself: 7.6 us a graph replay, 10.5 with a memset before it
    if (a.rows > 1) {
        clear_kernel<<<1, 1, 0, s>>>(a.hdr);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    // As many CTAs a row as are up to two waves of two an SM, since rows end after one to five passes.  16 nodes, 131,072
    // tokens, with draft probabilities, clusters of 8, 4, 2 and 1: 32 rows 29, 30, 49 and 86 us; 64 rows 45, 52, 64 and
    // 113; 128 rows 77, 75, 83 and 130 (the rule's 4); 256 rows 125, 107, 115 and 144 (its 2).
    const int most = 4 * sms / a.rows;
    const cudaError_t e = most >= 8 ? launch_cl<8>(a, s) : most >= 4 ? launch_cl<4>(a, s) : most >= 2 ? launch_cl<2>(a, s) : launch_cl<1>(a, s);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace wa
