// wa_tree.cu — attention of trees of drafted tokens over ring caches, on the tensor cores.
//
// Node i of row r, at position P = pos[r] + 1 + depth(i), sees the ring's keys
// [max(0, P - win + 1), pos[r]] and those of its tree's nodes that are its
// ancestors or itself and less than win positions back:
//   o = sum_j w_j v_j / sum_j w_j,  w_j = 2^(c q.k_j - m),  c = scale log2(e).
//
// Split.  A key head's G query heads of 128 / G nodes make a tile of up to 128
// query rows (tensor-memory lane m = node m / G, head m % G), so K and V are read
// once for all of them.  A row's keys are cut into spans at multiples of
// tree_span() keys, which depends on the row's own key count and hkv; the tree's
// own keys are one more 128-key tile of the last span.  A unit of work is (row,
// key head, query tile, span); it leaves (m, l, O) in fp32 and tree_merge_kernel
// joins a row's spans in order.  Nothing in a unit depends on the other rows, so
// neither do the bits.
//
// tree_kernel<D>: a persistent grid, one CTA an SM, 384 threads, that streams the
// keys of its units without a break between units:
//   warp 0      TMA producer: K and V in half-tiles through a ring of slots, in the
//               order the tensor core reads them (K0, K1, V0, K2, V1, ...), on across
//               unit ends.  A tile that wraps around the end of a ring is loaded in
//               8-row boxes; the one 8-row piece that holds the wrap itself is
//               copied by the warp.
//   warp 1      allocates tensor memory; lane 0 issues S(t + 1) = Q K^T and
//               O += P(t) V (two bf16 parts of P), commits free the slots.
//   warp 2      zeroes V rows that no node of the row sees (stale ring slots, nodes
//               past n), so that they never meet a zero probability as 0 * inf.
//   warp 3      takes units from a counter, publishes them through a ring of unit
//               slots, and loads each unit's Q once the previous unit's last S is done.
//   warps 4..11 softmax, one query row a thread in two column halves: mask,
//               exponentials, P over S in tensor memory, a lazy rescale of O, and
//               the unit's partial result.
// Every wait is bounded (a status bit after kWaitLimitNs) and warp-uniform where a
// warp waits.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "wa_prompt_kernel.cuh"

namespace wa {

namespace {

constexpr int kTile = 128;         // keys a tile
constexpr int kUnits = 4;          // unit slots
constexpr int kAhead = 2;          // units published beyond the one whose Q is loaded next

// Keys a span: enough spans that hkv key heads of one row occupy the card, in powers of two.
__host__ __device__ inline int tree_span(int64_t keys, int hkv) {
    const int64_t want = keys * hkv / 128;
    int len = 512;
    while (len < 2048 && 2 * len <= want) len *= 2;
    return len;
}

// Spans of a row at (clamped) position p, given its first visible key: at least one, for the tree.
__host__ __device__ inline int tree_first(int p, int win) { return win > 0 && p + 2 - win > 0 ? p + 2 - win : 0; }
__host__ __device__ inline int64_t tree_keys(int p, int win) { return win > 0 ? win : static_cast<int64_t>(p) + 1; }
__host__ __device__ inline int tree_spans(int p, int win, int hkv) {
    const int lo = tree_first(p, win);
    if (lo > p) return 1;
    const int len = tree_span(tree_keys(p, win), hkv);
    return p / len - lo / len + 1;
}

struct TreeParams {
    CUtensorMap tq;            // [rows][nodes][hq][d], box 64 dims x G heads x 128 / G nodes
    CUtensorMap tk, tv;        // rings [rows][ring][hkv][d], boxes of 128 keys (K) and 64 keys (V)
    CUtensorMap tk8, tv8;      // the same in boxes of 8 keys
    CUtensorMap tkt, tvt;      // nodes' keys and values [rows][nodes][hkv][d], boxes of 128 and 64
    const uint16_t* k;
    const uint16_t* v;
    const int32_t* pos;
    const int32_t* parent;
    const int32_t* n;
    float* part_o;             // [unit][lanes][d]
    float4* part_ml;           // [unit][lanes]: m (log2 units), l of each column half
    int* status;
    int* next_unit;
    int rows, nodes, hq, hkv, gsz, npt, mtiles, spans, lanes, win, ring, units, shared_kv;
    float c;                   // |scale| * log2(e)
    int neg;
};

template <int D>
struct TreeCfg {
    static constexpr int KB = D / 64;
    static constexpr int Q_BLOCK = 128 * 128;                 // 64 dims of 128 rows
    static constexpr int Q_BYTES = KB * Q_BLOCK;
    static constexpr int SLOT = D * 128;                      // K: 128 keys x d / 2; V: 64 keys x d
    static constexpr int NSLOT = D == 256 ? 5 : 10;
    // Load barriers are per operand half and tile, tile mod NB: a parity wait is sound while the
    // load of tile t + NB cannot land before the one of tile t was waited for, which the slot
    // ring gives for 4 NB > NSLOT (four half-loads a tile).
    static constexpr int NB = D == 256 ? 2 : 4;
    static_assert(4 * NB > NSLOT, "load barrier phases");
    static constexpr int K_BLOCK = kTile * 128;
    static constexpr int V_BLOCK = (kTile / 2) * 128;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_RING = OFF_Q + Q_BYTES;
    static constexpr int OFF_X = OFF_RING + NSLOT * SLOT;     // row maxima [2 tiles][2 halves][128]
    static constexpr int B_KFULL = 0;                         // [half][NB]
    static constexpr int B_VFULL = B_KFULL + 2 * NB;
    static constexpr int B_VREADY = B_VFULL + 2 * NB;
    static constexpr int B_FREE = B_VREADY + 2 * NB;          // [NSLOT]
    static constexpr int B_SFULL = B_FREE + NSLOT;            // [tile & 1] from here
    static constexpr int B_PVDONE = B_SFULL + 2;
    static constexpr int B_XCHG = B_PVDONE + 2;
    static constexpr int B_PHALF = B_XCHG + 2;
    static constexpr int B_PFULL = B_PHALF + 2;
    static constexpr int B_QFULL = B_PFULL + 2;
    static constexpr int B_QFREE = B_QFULL + 1;
    static constexpr int B_UFULL = B_QFREE + 1;               // [kUnits]
    static constexpr int B_UFREE = B_UFULL + kUnits;
    static constexpr int B_DRAIN = B_UFREE + kUnits;
    static constexpr int NBAR = B_DRAIN + 1;
    static constexpr int OFF_BAR = OFF_X + 2 * 2 * 128 * 4;
    static constexpr int OFF_UNIT = (OFF_BAR + NBAR * 8 + 15) / 16 * 16;   // 8 ints and 128 parents a slot
    static constexpr int UNIT_BYTES = 32 + WA_TREE_MAX_NODES;
    static constexpr int OFF_MISC = OFF_UNIT + kUnits * UNIT_BYTES;
    static constexpr int SMEM = OFF_MISC + 16;
    static_assert(SMEM <= 232448, "shared memory budget");
    // tensor memory: O (D columns), two S buffers; P's two parts over S
    static constexpr int TMEM_COLS = 512;
    __host__ __device__ static constexpr int s_col(int b) { return D + b * kTile; }
    static_assert(s_col(1) + kTile <= TMEM_COLS, "tensor memory budget");
};

// The load order is K(0), then for each tile t: K(t + 1) if there is one, V(t).  Operand index of K(t)
// and V(t) in it (two half-loads each).
__device__ __forceinline__ int op_k(int t) { return t == 0 ? 0 : 2 * t - 1; }
__device__ __forceinline__ int op_v(int t, bool last_of_all) { return last_of_all ? 2 * t + 1 : 2 * t + 2; }

// A published unit.  nt = 0 marks the end.
struct TreeUnit {
    int r, g, node0, span, t0, nring, nt, p, n, lo;
};

template <int D>
__global__ void __launch_bounds__(384, 1) tree_kernel(const __grid_constant__ TreeParams p) {
    using C = TreeCfg<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    if (sbase & 1023u) {
        if (threadIdx.x == 0) atomicOr(p.status, WA_STATUS_LAYOUT);
        return;
    }
    const uint32_t bar0 = sbase + C::OFF_BAR;
    auto BAR = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
    auto SLOT = [&](int s) { return sbase + C::OFF_RING + static_cast<uint32_t>(s) * C::SLOT; };
    auto LOADBAR = [&](int base, int half, int t) { return BAR(base + half * C::NB + t % C::NB); };
    auto LOADPH = [&](int t) { return static_cast<uint32_t>(t / C::NB) & 1u; };
    uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
    float* xbuf = reinterpret_cast<float*>(smem + C::OFF_X);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::NBAR; ++i) {
            int count = 1;
            if (i >= C::B_XCHG && i < C::B_PFULL) count = 8;               // XCHG, PHALF: the softmax warps
            else if (i >= C::B_PFULL && i < C::B_QFULL) count = 4;         // PFULL: those of the second half
            else if (i >= C::B_UFREE && i < C::B_DRAIN) count = 11;        // producer, MMA, V, softmax warps
            mbar_init(BAR(i), count);
        }
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(misc), C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = misc[0];

    auto unit_ints = [&](int U) { return reinterpret_cast<volatile int*>(smem + C::OFF_UNIT + (U % kUnits) * C::UNIT_BYTES); };
    // Unit U as published; the caller arrives on its UFREE barrier when it has read what it needs.
    auto read_unit = [&](int U, TreeUnit& x) {
        volatile int* e = unit_ints(U);
        x.r = e[0]; x.g = e[1] & 0xFFFF; x.node0 = e[1] >> 16; x.span = e[2]; x.t0 = e[3];
        x.nring = e[4] & 0xFFFFFF; x.nt = x.nring + (e[4] >> 24); x.p = e[5]; x.n = e[6]; x.lo = e[7];
    };
    auto take_unit = [&](int U, TreeUnit& x, bool whole) -> bool {
        const uint32_t ph = static_cast<uint32_t>(U / kUnits) & 1u;
        const uint32_t full = BAR(C::B_UFULL + U % kUnits);
        if (!(whole ? warp_wait(full, ph, p.status) : mbar_wait(full, ph, p.status))) return false;
        read_unit(U, x);
        if (whole) __syncwarp();
        if (!whole || lane == 0) mbar_arrive(BAR(C::B_UFREE + U % kUnits));
        return true;
    };

    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        if (lane == 0) {
            prefetch_tensormap(&p.tk);
            prefetch_tensormap(&p.tv);
            prefetch_tensormap(&p.tkt);
            prefetch_tensormap(&p.tvt);
        }
        // K and V are read once, unless several query tiles of a row share them
        const uint64_t pol = p.shared_kv ? policy_evict_last() : policy_evict_first();
        const int64_t tok = static_cast<int64_t>(p.hkv) * D;
        int u = 0;                                // half-loads issued
        uint32_t lastbar[C::NSLOT], lastph[C::NSLOT];   // barrier and phase of the load in each slot
        // one half-operand: keys [key0, key0 + nkeys) of a ring or node buffer, dims from dim0
        auto load_half = [&](const TreeUnit& x, int idx, int t, bool is_v, int half) -> bool {
            const int s = u % C::NSLOT, use = u / C::NSLOT;
            if (use > 0 && !warp_wait(BAR(C::B_FREE + s), (use - 1) & 1, p.status)) return false;
            const uint32_t full = LOADBAR(is_v ? C::B_VFULL : C::B_KFULL, half, t);
            const uint32_t dst = SLOT(s);
            const int nblk = is_v ? C::KB : C::KB / 2, dim0 = is_v ? 0 : half * (D / 2);
            const int nkeys = is_v ? 64 : kTile, blk = nkeys * 128;
            if (idx >= x.nring) {                 // the nodes' own keys
                if (lane == 0) {
                    mbar_arrive_expect_tx(full, C::SLOT);
                    for (int b = 0; b < nblk; ++b)
                        tma_load_4d(dst + b * blk, is_v ? &p.tvt : &p.tkt, dim0 + b * 64, x.g, is_v ? half * 64 : 0, x.r, full,
                                    pol);
                }
            } else {
                const int key0 = (x.t0 + idx) * kTile + (is_v ? half * 64 : 0);
                const int slot0 = p.win > 0 ? key0 % p.ring : key0;
                if (p.win == 0 || slot0 + nkeys <= p.ring) {
                    if (lane == 0) {
                        mbar_arrive_expect_tx(full, C::SLOT);
                        for (int b = 0; b < nblk; ++b)
                            tma_load_4d(dst + b * blk, is_v ? &p.tv : &p.tk, dim0 + b * 64, x.g, slot0, x.r, full, pol);
                    }
                } else {
                    // pieces of 8 keys: by TMA, or by the warp where the piece itself wraps
                    const uint16_t* base = (is_v ? p.v : p.k) + static_cast<int64_t>(x.r) * p.ring * tok + static_cast<int64_t>(x.g) * D + dim0;
                    int whole = 0;
                    for (int a = 0; a < nkeys / 8; ++a) {
                        const int sl = (slot0 + 8 * a) % p.ring;
                        if (sl + 8 <= p.ring) {
                            ++whole;
                            continue;
                        }
                        for (int e = lane; e < 64 * nblk; e += 32) {
                            const int k = e / (8 * nblk), rem = e % (8 * nblk), b = rem / 8, cc = rem % 8;
                            const uint4 val = ld_global_nc_v4(base + (sl + k) % p.ring * tok + b * 64 + cc * 8);
                            st_shared_v4(dst + b * blk + (8 * a + k) * 128 + ((cc ^ k) * 16), val.x, val.y, val.z, val.w);
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive_expect_tx(full, whole * nblk * 1024);
                        for (int a = 0; a < nkeys / 8; ++a) {
                            const int sl = (slot0 + 8 * a) % p.ring;
                            if (sl + 8 > p.ring) continue;
                            for (int b = 0; b < nblk; ++b)
                                tma_load_4d(dst + b * blk + a * 1024, is_v ? &p.tv8 : &p.tk8, dim0 + b * 64, x.g, sl, x.r, full,
                                            pol);
                        }
                    }
                }
            }
            __syncwarp();
            lastbar[s] = full;
            lastph[s] = LOADPH(t);
            ++u;
            return true;
        };
        TreeUnit cur, nxt;
        int U = 0, t = 0, idx = 0;
        bool ok = take_unit(U++, cur, true);
        bool more = ok && cur.nt > 0;
        if (more) ok = load_half(cur, 0, 0, false, 0) && load_half(cur, 0, 0, false, 1);
        while (ok && more) {
            // the tile after (cur, idx)
            const bool same = idx + 1 < cur.nt;
            if (!same) {
                if (!(ok = take_unit(U++, nxt, true))) break;
                more = nxt.nt > 0;
            }
            if (same) ok = load_half(cur, idx + 1, t + 1, false, 0) && load_half(cur, idx + 1, t + 1, false, 1);
            else if (more) ok = load_half(nxt, 0, t + 1, false, 0) && load_half(nxt, 0, t + 1, false, 1);
            ok = ok && load_half(cur, idx, t, true, 0) && load_half(cur, idx, t, true, 1);
            if (same) {
                ++idx;
            } else {
                cur = nxt;
                idx = 0;
            }
            ++t;
        }
        // the copies in flight land before the block exits, whichever role stopped early
        if (lane == 0)
            for (int i = max(0, u - C::NSLOT); i < u; ++i) mbar_wait(lastbar[i % C::NSLOT], lastph[i % C::NSLOT], p.status);
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer (one thread)
        if (lane == 0) {
            const uint32_t idS = idesc_bf16_f32(128, kTile, 0, 0, p.neg ? 1u : 0u);
            constexpr uint32_t idO = idesc_bf16_f32(128, D, 0, 1);
            const uint64_t aq = sdesc_sw128(sbase + C::OFF_Q, 16, 1024);
            // slots in load order: K of tile t, then V of tile t - 1; V of the last tile has no K before it
            auto issue_s = [&](int t) -> bool {
#pragma unroll
                for (int kh = 0; kh < 2; ++kh) {
                    const int s = (2 * op_k(t) + kh) % C::NSLOT;
                    if (!mbar_wait(LOADBAR(C::B_KFULL, kh, t), LOADPH(t), p.status)) return false;
                    tc_fence_after();
                    const uint64_t bk = sdesc_sw128(SLOT(s), 16, 1024);
#pragma unroll
                    for (int k8 = 0; k8 < D / 32; ++k8) {
                        const int kk = (D / 32) * kh + k8;
                        mma_bf16_ss(tbase + C::s_col(t & 1), aq + (((kk >> 2) * C::Q_BLOCK + (kk & 3) * 32) >> 4),
                                    bk + (((k8 >> 2) * C::K_BLOCK + (k8 & 3) * 32) >> 4), idS, kk > 0 ? 1u : 0u);
                    }
                    mma_commit(BAR(C::B_FREE + s));
                }
                mma_commit(BAR(C::B_SFULL + (t & 1)));
                return true;
            };
            auto issue_pv = [&](int t, bool first, bool last_of_all) -> bool {
                const int b = t & 1;
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const int s = (2 * op_v(t, last_of_all) + hh) % C::NSLOT;
                    if (!mbar_wait(LOADBAR(C::B_VREADY, hh, t), LOADPH(t), p.status)) return false;
                    if (!mbar_wait(BAR((hh ? C::B_PFULL : C::B_PHALF) + b), (t >> 1) & 1, p.status)) return false;
                    tc_fence_after();
                    const uint64_t v0 = sdesc_sw128(SLOT(s), C::V_BLOCK, 1024);
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int k4 = 0; k4 < 4; ++k4)
                            mma_bf16_ts(tbase, tbase + C::s_col(b) + hh * 64 + part * 32 + k4 * 8, v0 + ((k4 * 16 * 128) >> 4),
                                        idO, (!first || hh > 0 || part > 0 || k4 > 0) ? 1u : 0u);
                    mma_commit(BAR(C::B_FREE + s));
                }
                mma_commit(BAR(C::B_PVDONE + b));
                return true;
            };
            int t = 0;
            bool ok = true, pending = false, pending_first = false;
            for (int U = 0; ok; ++U) {
                TreeUnit x;
                if (!(ok = take_unit(U, x, false))) break;
                // a unit's last P V goes before the next unit's S, which may still wait for its Q
                if (pending) ok = issue_pv(t - 1, pending_first, x.nt <= 0);
                pending = false;
                if (!ok || x.nt <= 0) break;
                ok = mbar_wait(BAR(C::B_QFULL), U & 1, p.status);
                for (int idx = 0; ok && idx < x.nt; ++idx, ++t) {
                    ok = issue_s(t);
                    if (ok && idx == x.nt - 1) mma_commit(BAR(C::B_QFREE));
                    if (ok && pending) ok = issue_pv(t - 1, pending_first, false);
                    pending = true;
                    pending_first = idx == 0;
                }
            }
            // every product issued has finished before tensor memory can be released
            mma_commit(BAR(C::B_DRAIN));
            mbar_wait(BAR(C::B_DRAIN), 0, p.status);
        }
        __syncwarp();
    } else if (warp == 2) {
        // ------------------------------------------------ V rows that no node sees -> 0
        int t = 0;
        TreeUnit x, nxt;
        bool ok = take_unit(0, x, true);
        for (int U = 1; ok && x.nt > 0; ++U) {
            bool have_next = false;
            for (int idx = 0; ok && idx < x.nt; ++idx, ++t) {
                // whether this is the very last tile decides where its V sits in the load order
                if (idx == x.nt - 1) {
                    if (!(ok = take_unit(U, nxt, true))) break;
                    have_next = true;
                }
                const bool last_of_all = have_next && nxt.nt <= 0;
                for (int hh = 0; hh < 2; ++hh) {
                    const int s = (2 * op_v(t, last_of_all) + hh) % C::NSLOT;
                    if (!(ok = warp_wait(LOADBAR(C::B_VFULL, hh, t), LOADPH(t), p.status))) break;
                    int z_lo, z_hi, z_end = 64;       // rows [0, z_lo) and [z_hi, z_end) are cleared
                    if (idx < x.nring) {
                        const int key0 = (x.t0 + idx) * kTile + hh * 64;
                        z_lo = min(64, max(0, x.lo - key0));
                        z_hi = max(0, min(64, x.p - key0 + 1));
                    } else {
                        z_lo = 0;
                        z_hi = max(0, min(64, x.n - hh * 64));
                        z_end = max(0, min(64, p.nodes - hh * 64));   // past the buffer's nodes TMA has filled zeros
                    }
                    z_hi = max(z_hi, z_lo);
                    const int nz = z_lo + max(0, z_end - z_hi);
                    if (nz > 0) {
                        const uint32_t vst = SLOT(s);
                        for (int e = lane; e < nz * C::KB * 8; e += 32) {
                            const int zr = e / (C::KB * 8), rem = e % (C::KB * 8);
                            const int row = zr < z_lo ? zr : z_hi + (zr - z_lo);
                            st_shared_v4(vst + (rem / 8) * C::V_BLOCK + row * 128 + (rem % 8) * 16, 0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async_smem();
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(LOADBAR(C::B_VREADY, hh, t));
                }
            }
            if (ok) x = nxt;
        }
    } else if (warp == 3) {
        // ------------------------------------------------ units; Q
        if (lane == 0) prefetch_tensormap(&p.tq);
        int k_cur = blockIdx.x, k_ans = 0, pub = 0, loaded = 0;
        bool asked = false, ended = false, ok = true;
        // the next unit with any work (nt = 0: none left); its number is asked for one unit ahead
        auto next_unit = [&](TreeUnit& x) {
            for (;;) {
                if (asked) k_cur = __shfl_sync(0xFFFFFFFFu, k_ans, 0) + static_cast<int>(gridDim.x);
                x.nt = 0;
                x.nring = 0;
                if (k_cur >= p.units) return;
                if (lane == 0) k_ans = atomicAdd(p.next_unit, 1);
                asked = true;
                int k = k_cur;
                const int mt = k % p.mtiles;
                k /= p.mtiles;
                x.span = k % p.spans;
                k /= p.spans;
                x.g = k % p.hkv;
                x.r = k / p.hkv;
                x.node0 = mt * p.npt;
                const int raw_p = p.pos[x.r], raw_n = p.n ? p.n[x.r] : p.nodes;
                x.n = min(max(raw_n, 0), p.nodes);
                x.p = tree_pos(raw_p, p.win, p.ring);
                if (x.g == 0 && mt == 0 && x.span == 0) {     // reported once a row
                    int bad = 0;
                    if (raw_n != x.n) bad |= WA_STATUS_BAD_TREE;
                    if (raw_p != x.p) bad |= WA_STATUS_BAD_POS;
                    for (int i = lane; i < x.n; i += 32) {
                        const int a = p.parent[static_cast<int64_t>(x.r) * p.nodes + i];
                        if (tree_parent(a, i) != a) bad |= WA_STATUS_BAD_TREE;
                    }
                    if (bad) atomicOr(p.status, bad);
                }
                if (x.node0 >= x.n) continue;
                x.lo = tree_first(x.p, p.win);
                if (x.lo > x.p) {                             // no key of the ring: the tree alone
                    if (x.span > 0) continue;
                    x.t0 = 0;
                    x.nt = 1;
                    return;
                }
                const int len = tree_span(tree_keys(x.p, p.win), p.hkv);
                const int sp = x.lo / len + x.span;
                if (sp > x.p / len) continue;
                const int kb = max(x.lo, sp * len), ke = min(x.p, sp * len + (len - 1));
                x.t0 = kb / kTile;
                x.nring = ke / kTile - x.t0 + 1;
                x.nt = x.nring + (sp == x.p / len ? 1 : 0);
                return;
            }
        };
        TreeUnit ahead[kAhead + 1];
        auto publish_next = [&](TreeUnit& x) -> bool {
            if (ended) return true;
            next_unit(x);
            ended = x.nt <= 0;
            if (pub >= kUnits && !warp_wait(BAR(C::B_UFREE + pub % kUnits), static_cast<uint32_t>(pub / kUnits - 1) & 1u, p.status))
                return false;
            volatile int* e = unit_ints(pub);
            if (!ended) {
                volatile uint8_t* par = reinterpret_cast<volatile uint8_t*>(e + 8);
                for (int i = lane; i < p.nodes; i += 32)
                    par[i] = static_cast<uint8_t>(tree_parent(p.parent[static_cast<int64_t>(x.r) * p.nodes + i], i));
            }
            if (lane == 0) {
                e[0] = x.r; e[1] = x.g | (x.node0 << 16); e[2] = x.span; e[3] = x.t0;
                e[4] = x.nring | ((x.nt - x.nring) << 24); e[5] = x.p; e[6] = x.n; e[7] = x.lo;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(C::B_UFULL + pub % kUnits));
            ++pub;
            return true;
        };
        for (int i = 0; ok && i <= kAhead; ++i) {
            ahead[i].nt = 0;
            ok = publish_next(ahead[i]);
        }
        for (int U = 0; ok; ++U) {
            const TreeUnit x = ahead[0];
            if (x.nt <= 0) break;
            // Q of unit U, once the last S of unit U - 1 has read the buffer
            if (U > 0 && !(ok = warp_wait(BAR(C::B_QFREE), (U - 1) & 1, p.status))) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(BAR(C::B_QFULL), C::KB * p.gsz * p.npt * 128);
                for (int b = 0; b < C::KB; ++b)
                    tma_load_4d(sbase + C::OFF_Q + b * C::Q_BLOCK, &p.tq, b * 64, x.g * p.gsz, x.node0, x.r, BAR(C::B_QFULL),
                                policy_evict_last());
            }
            loaded = U + 1;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < kAhead; ++i) ahead[i] = ahead[i + 1];
            ahead[kAhead].nt = 0;
            ok = publish_next(ahead[kAhead]);
        }
        if (lane == 0 && loaded > 0) mbar_wait(BAR(C::B_QFULL), (loaded - 1) & 1, p.status);
    } else {
        // ------------------------------------------------ softmax: query row r, column half wg
        const int wg = (warp - 4) >> 2;
        const int r = (warp & 3) * 32 + lane;
        const int rn = r / p.gsz;                             // the row's node within the tile
        const int col0 = wg * 64;
        const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const float c = p.c;
        int t = 0;
        bool ok = true;
        for (int U = 0; ok; ++U) {
            TreeUnit x;
            if (!(ok = warp_wait(BAR(C::B_UFULL + U % kUnits), static_cast<uint32_t>(U / kUnits) & 1u, p.status))) break;
            read_unit(U, x);
            const int node = x.node0 + rn;
            const bool live = x.nt > 0 && rn < p.npt && node < x.n;
            // the node's depth, and which of its ancestors (and itself) are in its window
            int row_lo = INT_MIN / 2;                         // rows without a node: nothing masked, nothing stored
            uint32_t m0 = 0xFFFFFFFFu, m1 = 0xFFFFFFFFu;      // tree columns [64 wg, 64 wg + 64)
            if (live) {
                const volatile uint8_t* par = reinterpret_cast<const volatile uint8_t*>(unit_ints(U) + 8);
                int back = 0;
                m0 = m1 = 0u;
                for (int a = node; a != 255; a = par[a], ++back) {
                    const int col = a - col0;
                    if (p.win == 0 || back < p.win) {
                        if (col >= 0 && col < 32) m0 |= 1u << col;
                        if (col >= 32 && col < 64) m1 |= 1u << (col - 32);
                    }
                }
                row_lo = p.win > 0 ? max(0, x.p + back - p.win + 1) : 0;   // back = depth + 1
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(C::B_UFREE + U % kUnits));
            if (x.nt <= 0) break;
            const bool idle = !__any_sync(0xFFFFFFFFu, live);     // a warp without rows only keeps the barriers going
            float m_run = -INFINITY, l_run = 0.f;
            for (int idx = 0; idx < x.nt; ++idx, ++t) {
                const int b = t & 1;
                const uint32_t ph = static_cast<uint32_t>(t >> 1) & 1u;
                if (!(ok = warp_wait(BAR(C::B_SFULL + b), ph, p.status))) break;
                if (idle) {
                    if (lane == 0) {
                        mbar_arrive(BAR(C::B_XCHG + b));
                        mbar_arrive(BAR(C::B_PHALF + b));
                        if (wg == 1) mbar_arrive(BAR(C::B_PFULL + b));
                    }
                    __syncwarp();
                    continue;
                }
                tc_fence_after();
                const uint32_t t_s = tbase + lane_addr + C::s_col(b) + col0;
                float sv[64];
                load_s<64>(t_s, sv);
                // visible columns of this half as bits
                uint32_t w0 = m0, w1 = m1;
                if (idx < x.nring) {
                    const int kbase = (x.t0 + idx) * kTile + col0;
                    const int vlo = live ? max(0, row_lo - kbase) : 0, vhi = live ? min(63, x.p - kbase) : 63;
                    const unsigned long long bits = vlo > vhi ? 0ull : (~0ull >> (63 - (vhi - vlo))) << vlo;
                    w0 = static_cast<uint32_t>(bits);
                    w1 = static_cast<uint32_t>(bits >> 32);
                }
                const bool masked = !__all_sync(0xFFFFFFFFu, (w0 & w1) == 0xFFFFFFFFu);
                float mx8[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) mx8[e] = -INFINITY;
                if (masked) {
#pragma unroll
                    for (int k = 0; k < 64; ++k)
                        mx8[k & 7] = fmaxf(mx8[k & 7], ((k < 32 ? w0 : w1) >> (k & 31)) & 1u ? sv[k] : -INFINITY);
                } else {
#pragma unroll
                    for (int k = 0; k < 64; k += 2) mx8[(k >> 1) & 7] = max3(mx8[(k >> 1) & 7], sv[k], sv[k + 1]);
                }
                const float mh = fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])),
                                       fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])));
                float* xs = xbuf + b * 256;
                xs[wg * 128 + r] = mh;
                __syncwarp();   // the warp's stores precede lane 0's (cumulative) release
                if (lane == 0) mbar_arrive(BAR(C::B_XCHG + b));
                float ls8[8];
                auto exponents = [&](float m_sub) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) ls8[e] = 0.f;
                    if (masked) {   // a masked column is 0 whatever its score
#pragma unroll
                        for (int k = 0; k < 64; ++k) {
                            const float pk = ((k < 32 ? w0 : w1) >> (k & 31)) & 1u ? ex2(fmaf(sv[k], c, -m_sub)) : 0.f;
                            sv[k] = pk;
                            ls8[2 * ((k >> 1) & 3) + (k & 1)] += pk;
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 64; k += 2) {
                            float x0, x1;
                            fma_x2(x0, x1, sv[k], sv[k + 1], c, c, -m_sub, -m_sub);
                            sv[k] = ex2(x0);
                            sv[k + 1] = ex2(x1);
                            add_x2(ls8[2 * ((k >> 1) & 3)], ls8[2 * ((k >> 1) & 3) + 1], sv[k], sv[k + 1]);
                        }
                    }
                };
                // The running max usually stays (lazy rule), so the exponentials start with it while
                // the other half's maximum is on its way, and are redone from S if it moved.
                const bool spec = __all_sync(0xFFFFFFFFu, !live || (m_run != -INFINITY && mh * c <= m_run + kLazy));
                if (spec) exponents(m_run);
                if (!(ok = warp_wait(BAR(C::B_XCHG + b), ph, p.status))) break;
                const float mt = fmaxf(xs[r], xs[128 + r]) * c;
                const float m_new = (mt > m_run + kLazy) ? mt : m_run;
                const float alpha = (m_new == m_run) ? 1.f : ex2(m_run - m_new);
                const float m_sub = (m_new == -INFINITY) ? 0.f : m_new;
                if (!spec || __any_sync(0xFFFFFFFFu, live && m_new != m_run)) {
                    if (spec) load_s<64>(t_s, sv);
                    exponents(m_sub);
                }
                // O's rescale, once the previous P V is done; a unit's first P V starts O afresh
                if (idx > 0 && __any_sync(0xFFFFFFFFu, live && alpha != 1.f)) {
                    if (!(ok = warp_wait(BAR(C::B_PVDONE + ((t - 1) & 1)), static_cast<uint32_t>((t - 1) >> 1) & 1u, p.status)))
                        break;
                    tc_fence_after();
#pragma unroll 1
                    for (int cc = 0; cc < D / 64; ++cc) {
                        uint32_t o[32];
                        const uint32_t ta = tbase + lane_addr + wg * (D / 2) + cc * 32;
                        tmem_ld32_wait(ta, o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        tmem_st32(ta, o);
                    }
                    tmem_wait_st();
                }
                if (wg == 1) {   // the second half's O columns are ready for this tile's first P V half
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(BAR(C::B_PHALF + b));
                }
                // P = bf16(p) + bf16(p - bf16(p)) over this half's own S columns: within 2^-17 of p, which
                // keeps the output to the decode form's accuracy (one bf16 part alone: 2^-9)
#pragma unroll
                for (int cc = 0; cc < 2; ++cc) {
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float a = sv[cc * 32 + 2 * e], bb = sv[cc * 32 + 2 * e + 1];
                        hi[e] = pack_bf16(a, bb);
                        lo[e] = pack_bf16(a - __uint_as_float(hi[e] << 16), bb - __uint_as_float(hi[e] & 0xFFFF0000u));
                    }
                    tmem_st16(t_s + cc * 16, hi);
                    tmem_st16(t_s + 32 + cc * 16, lo);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(BAR((wg == 0 ? C::B_PHALF : C::B_PFULL) + b));
                const float lsum = ((ls8[0] + ls8[1]) + (ls8[2] + ls8[3])) + ((ls8[4] + ls8[5]) + (ls8[6] + ls8[7]));
                l_run = (alpha == 1.f) ? (l_run + lsum) : fmaf(l_run, alpha, lsum);
                m_run = m_new;
            }
            if (!ok) break;
            if (idle) continue;
            // the unit's partial result; the next unit's first P V waits for this warp's next PHALF
            if (!(ok = warp_wait(BAR(C::B_PVDONE + ((t - 1) & 1)), static_cast<uint32_t>((t - 1) >> 1) & 1u, p.status))) break;
            tc_fence_after();
            const int64_t unit = ((static_cast<int64_t>(x.r) * p.hkv + x.g) * p.mtiles + x.node0 / p.npt) * p.spans + x.span;
            const int64_t rec = unit * p.lanes + r;
#pragma unroll 1
            for (int cc = 0; cc < D / 64; ++cc) {
                uint32_t o[32];
                tmem_ld32_wait(tbase + lane_addr + wg * (D / 2) + cc * 32, o);
                if (live) {
                    float4* dst = reinterpret_cast<float4*>(p.part_o + rec * D + wg * (D / 2) + cc * 32);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        dst[e] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                             __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
                }
            }
            if (live) {
                float* ml = reinterpret_cast<float*>(p.part_ml + rec);
                if (wg == 0) *reinterpret_cast<float2*>(ml) = make_float2(m_run, l_run);
                else ml[2] = l_run;
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tbase, C::TMEM_COLS);
}

// o = sum_s a_s O_s / sum_s a_s l_s over a row's spans in order, a_s = 2^(m_s - M); one warp a (node, query head).
template <int D>
__global__ void __launch_bounds__(256) tree_merge_kernel(const float* __restrict__ part_o, const float4* __restrict__ part_ml,
                                                         const TreeArgs a, int npt, int mtiles, int spans, int lanes) {
    constexpr int V4 = D / 128;      // float4 a lane
    const int lane = threadIdx.x & 31;
    const int unit = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (unit >= a.rows * a.nodes * a.hq) return;
    const int h = unit % a.hq, node = unit / a.hq % a.nodes, r = unit / a.hq / a.nodes;
    if (node >= min(a.n ? a.n[r] : a.nodes, a.nodes)) return;
    const int p = tree_pos(a.pos[r], a.win, a.ring);
    const int G = a.hq / a.hkv, g = h / G;
    const int count = tree_spans(p, a.win, a.hkv);
    const int64_t rec0 = ((static_cast<int64_t>(r) * a.hkv + g) * mtiles + node / npt) * spans * lanes + (node % npt) * G + h % G;
    float M = -INFINITY;
    for (int s = 0; s < count; ++s) M = fmaxf(M, part_ml[rec0 + static_cast<int64_t>(s) * lanes].x);
    float4 num[V4];
#pragma unroll
    for (int e = 0; e < V4; ++e) num[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    float den = 0.f;
    for (int s = 0; s < count; ++s) {
        const int64_t rec = rec0 + static_cast<int64_t>(s) * lanes;
        const float4 ml = part_ml[rec];
        const float w = exp2f(ml.x - M);
        den = fmaf(w, ml.y + ml.z, den);
        const float4* o = reinterpret_cast<const float4*>(part_o + rec * D);
#pragma unroll
        for (int e = 0; e < V4; ++e) {
            const float4 x = o[e * 32 + lane];
            num[e].x = fmaf(w, x.x, num[e].x);
            num[e].y = fmaf(w, x.y, num[e].y);
            num[e].z = fmaf(w, x.z, num[e].z);
            num[e].w = fmaf(w, x.w, num[e].w);
        }
    }
    uint2* orow = reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + r * a.o_row + node * a.o_tok + static_cast<int64_t>(h) * D);
    bool bad = false;
#pragma unroll
    for (int e = 0; e < V4; ++e) {
        const float x = __fdiv_rn(num[e].x, den), y = __fdiv_rn(num[e].y, den);
        const float z = __fdiv_rn(num[e].z, den), w = __fdiv_rn(num[e].w, den);
        bad |= !(isfinite(x) && isfinite(y) && isfinite(z) && isfinite(w));
        orow[e * 32 + lane] = make_uint2(pack_bf16(x, y), pack_bf16(z, w));
    }
    if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) a.flags[atomicAdd(&a.hdr->nflag, 1)] = unit;
}

// A [rows][toks][heads][d] bf16 tensor in boxes of 64 dims x box_heads x box_toks, 128-byte swizzle.
bool encode_4d(CUtensorMap* m, const void* base, int d, int heads, int toks, int rows, int64_t tok, int64_t row, int box_heads,
               int box_toks) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(toks),
                          static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[3] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(tok) * 2, static_cast<cuuint64_t>(row) * 2};
    cuuint32_t box[4] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_toks), 1};
    cuuint32_t es[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_tree_d(const TreeArgs& a, cudaStream_t s) {
    using C = TreeCfg<D>;
    const TreePlan pl = tree_plan(a.rows, a.nodes, a.hq, a.hkv, a.win, a.ring);
    TreeParams t{};
    const int G = a.hq / a.hkv;
    const int64_t ktok = static_cast<int64_t>(a.hkv) * D, krow = ktok * a.ring;
    if (!encode_4d(&t.tq, a.q, D, a.hq, a.nodes, a.rows, a.q_tok, a.q_row, G, pl.npt) ||
        !encode_4d(&t.tk, a.k, D, a.hkv, a.ring, a.rows, ktok, krow, 1, kTile) ||
        !encode_4d(&t.tv, a.v, D, a.hkv, a.ring, a.rows, ktok, krow, 1, kTile / 2) ||
        !encode_4d(&t.tk8, a.k, D, a.hkv, a.ring, a.rows, ktok, krow, 1, 8) ||
        !encode_4d(&t.tv8, a.v, D, a.hkv, a.ring, a.rows, ktok, krow, 1, 8) ||
        !encode_4d(&t.tkt, a.kt, D, a.hkv, a.nodes, a.rows, a.kt_tok, a.kt_row, 1, kTile) ||
        !encode_4d(&t.tvt, a.vt, D, a.hkv, a.nodes, a.rows, a.vt_tok, a.vt_row, 1, kTile / 2))
        return cudaErrorInvalidValue;
    t.k = static_cast<const uint16_t*>(a.k);
    t.v = static_cast<const uint16_t*>(a.v);
    t.pos = a.pos; t.parent = a.parent; t.n = a.n;
    t.part_ml = static_cast<float4*>(a.part);
    t.part_o = reinterpret_cast<float*>(t.part_ml + pl.units * pl.lanes);
    t.status = &a.hdr->status;
    t.next_unit = &a.hdr->next_unit;
    t.rows = a.rows; t.nodes = a.nodes; t.hq = a.hq; t.hkv = a.hkv; t.gsz = G; t.npt = pl.npt; t.mtiles = pl.mtiles;
    t.spans = pl.spans; t.lanes = pl.lanes; t.win = a.win; t.ring = a.ring; t.units = static_cast<int>(pl.units);
    t.shared_kv = pl.mtiles > 1;
    t.neg = a.scale < 0.f ? 1 : 0;
    t.c = (a.scale < 0.f ? -a.scale : a.scale) * 1.4426950408889634f;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return cudaErrorInvalidValue;
    const int grid = static_cast<int>(pl.units < sms ? pl.units : sms);
    tree_kernel<D><<<grid, 384, C::SMEM, s>>>(t);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int outs = a.rows * a.nodes * a.hq;
    tree_merge_kernel<D><<<(outs + 7) / 8, 256, 0, s>>>(t.part_o, t.part_ml, a, pl.npt, pl.mtiles, pl.spans, pl.lanes);
    return cudaGetLastError();
}

}  // namespace

TreePlan tree_plan(int rows, int nodes, int hq, int hkv, int win, int ring) {
    TreePlan pl{};
    const int G = hq / hkv;
    pl.npt = 128 / G;
    pl.mtiles = (nodes + pl.npt - 1) / pl.npt;
    pl.lanes = (nodes < pl.npt ? nodes : pl.npt) * G;
    pl.spans = 1;
    if (win > 0) {
        // win - 1 keys from any position touch at most this many spans
        const int len = tree_span(win, hkv);
        pl.spans = win > 1 ? (win - 2 + len - 1) / len + 1 : 1;
    } else {
        for (int len = 512; len <= 2048; len *= 2) {
            // the most keys with this span
            int64_t keys = len == 2048 ? ring : (256LL * len + hkv - 1) / hkv - 1;
            keys = keys < ring ? keys : ring;
            const int spans = static_cast<int>((keys + len - 1) / len);
            pl.spans = spans > pl.spans ? spans : pl.spans;
        }
    }
    pl.units = static_cast<int64_t>(rows) * hkv * pl.mtiles * pl.spans;
    return pl;
}

cudaError_t tree_prepare_device(int) {
    cudaError_t e = cudaFuncSetAttribute(tree_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, TreeCfg<128>::SMEM);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(tree_kernel<256>, cudaFuncAttributeMaxDynamicSharedMemorySize, TreeCfg<256>::SMEM);
}

cudaError_t launch_tree(const TreeArgs& a, cudaStream_t s) {
    return a.d == 256 ? launch_tree_d<256>(a, s) : launch_tree_d<128>(a, s);
}

}  // namespace wa
