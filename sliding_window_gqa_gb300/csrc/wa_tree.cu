// wa_tree.cu — attention of trees of drafted tokens over ring caches, on the tensor cores.
//
// Node i of row r, at position P = pos[r] + 1 + depth(i), sees the ring's keys
// [max(0, P - win + 1), pos[r]] and those of its tree's nodes that are its
// ancestors or itself and less than win positions back:
//   o = sum_j w_j v_j / sum_j w_j,  w_j = 2^(c q.k_j - m),  c = scale log2(e).
//
// Split.  A key head's G query heads of 128 / G nodes make a tile of up to 128
// query rows (tensor-memory lane m = node m / G, head m % G), so K and V are read
// once for all of them.  A row's keys are taken in tiles of 128 from its first
// visible one (a window of 1,024 keys from anywhere is then 8 tiles; cut at absolute
// multiples it was 9 mostly, and a batch over a window 7 % slower), its tree's own
// keys are one tile more, and the tiles are cut evenly into spans, whose number
// depends on the row's own position, the window and hq.  A unit of work is (row, key
// head, query tile, span); it leaves (m, l, O) in fp32 and tree_merge_kernel joins a
// row's spans in order.  Nothing in a unit depends on the other rows, so neither do
// the bits.
//
// What bounds it.  Up to 64 query rows a tile: the reads of K and V (a linear batch of
// 8 rows, 32/16 heads of 256, 9,000 to 32,700 keys: 441 us, 92 % of the measured copy
// rate over the whole call; 64 rows over a window of 1,024, 32/16 heads: 216 us, 75 %,
// the rest being the start and the join of the spans).  128 query rows at head dim 128:
// the softmax warps, whose chain S -> P of a tile takes 2,500 cycles where its products
// take 1,536 (32 rows of 64 nodes, 32/4 heads: 442 us; 268 us of products at the measured
// rate).  One sequence over a window (19 us): the start of three kernels, one CTA's loads
// (36 bytes a cycle) and that chain.  Times in this file are of calls replayed as CUDA
// graphs; called from Python one after another the four take 457, 218, 470 and 22 us.
//
// tree_plan_kernel: one block lists the (row, span) pairs, longest first, with all that a
// unit needs of its row (position, nodes, parents), checks the rows' numbers for the status
// word, and clears the header.
// tree_kernel<D>: a persistent grid, one CTA an SM, 640 threads, that streams the
// keys of its units without a break between units:
//   warp 0      TMA producer: K and V through a ring of 32 KiB slots (head dim 256: half a
//               tile's K or V each), in the order the tensor core reads them (K0, K1, V0,
//               K2, V1, ...), on across unit ends.  A tile that wraps around the end of a
//               ring goes through load_wrapped.
//   warp 1      allocates tensor memory; one lane issues S(t) = Q K^T and
//               O += P(t - NS + 1) V (two bf16 parts of P), commits free the slots.
//   warp 2      zeroes V rows that no node of the row sees (stale ring slots, nodes
//               past n), so that they never meet a zero probability as 0 * inf.
//   warp 3      takes units from the list by a counter (long ones first: taken as they came, the
//               last ones ended 10 % after the mean), publishes them through a ring of unit
//               slots, and loads each unit's Q once the previous unit's last S is done.
//   warps 4..19 softmax, one query row a thread in four column quarters: mask,
//               exponentials, P over S in tensor memory, a lazy rescale of O, and the
//               unit's partial result.  Four warps share a row group, so that the chain
//               S -> P of a tile is 32 columns long (with two warps of 64 columns it took
//               about 3,000 cycles at 16 query rows, more than the tile's reads).
// Every wait is bounded (a status bit after kWaitLimitNs) and warp-uniform where a
// warp waits.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "wa_f64.cuh"
#include "wa_prompt_kernel.cuh"

namespace wa {

namespace {

constexpr int kTile = 128;         // keys a tile
constexpr int kTreeThreads = 640;
constexpr int kUnits = 4;          // unit slots
constexpr int kAhead = 2;          // units published beyond the one whose Q is loaded next

// log2 units the running max may trail before O is rescaled.  P, l and O are floating point, so a stale
// maximum costs no accuracy; 2^32 leaves them 2^90 below overflow, and what does overflow is computed again.
constexpr float kTreeLazy = 32.0f;

// Keys a span, a power of two: keys * hq / 128 on a linear cache, win * hq / 64 on a window, 2,048 at most.  Short
// spans put a single row's keys on more SMs, long ones leave fewer partial results and fewer ends of the pipeline.
// Linear, with / 64, / 128 and / 256: one row of 32,000 keys, 16/8 heads, 52, 52 and 68 us; 32 rows of 64 nodes, 32/4
// heads, 431, 442 and 508; 8 rows of 32/16 heads 440, 441 and 448; at most 1,024 with / 128: 68, 490 and 471.  A window
// of 1,024 with / 32, / 64 and / 128: one row of 16/8 heads 23, 18.7 and 18.5; 64 rows of 32/16 heads 208, 216 and 238;
// 13 ragged rows of 24/8 heads, a window of 1,000: 26.4, 25 and 24.  The rule sees no number of rows, so that a row's
// bits do not either.
constexpr int kSpanMinWindow = 256, kSpanMinLinear = 512, kSpanMax = 2048, kSpanLinear = 128, kSpanWindow = 64;
__host__ __device__ inline int tree_span(int64_t keys, bool window, int hq) {
    const int64_t want = keys * hq / (window ? kSpanWindow : kSpanLinear);
    int len = window ? kSpanMinWindow : kSpanMinLinear;
    while (len < kSpanMax && 2 * len <= want) len *= 2;
    return len;
}

// A row at (clamped) position p has tiles of 128 keys from its first visible one, and one of its tree's; they are
// cut evenly into spans of at most a tile more than tree_span()'s keys, the longer ones last (the tree's tile is little
// to read: with the longer ones first a batch over a window took 226 us instead of 216).
__host__ __device__ inline int tree_first(int p, int win) { return win > 0 && p + 2 - win > 0 ? p + 2 - win : 0; }
__host__ __device__ inline int64_t tree_keys(int p, int win) { return win > 0 ? win : static_cast<int64_t>(p) + 1; }
__host__ __device__ inline int tree_tiles(int p, int win) { return (max(p - tree_first(p, win) + 1, 0) + kTile - 1) / kTile + 1; }
__host__ __device__ inline int tree_cut(int tiles, int64_t keys, int win, int hq) {
    const int most = tree_span(keys, win > 0, hq) / kTile + 1;
    return (tiles + most - 1) / most;
}
__host__ __device__ inline int tree_spans(int p, int win, int hq) { return tree_cut(tree_tiles(p, win), tree_keys(p, win), win, hq); }

// A listed pair: row, span, first key, ring tiles, tiles, position, nodes, first key, then the row's 128 parents
// as bytes (255: a root).
constexpr int kPair = 8 + WA_TREE_MAX_NODES / 4;
static_assert(kPair * 4 == kTreePairBytes, "workspace");

struct TreeParams {
    // five dimensions (64 dims, tokens, blocks of 64 dims, heads, rows) put a whole half-operand, in the
    // [block][token][64] order that the tensor core reads, into one copy
    CUtensorMap tq;            // q: 64 x G heads x qn nodes x D / 64 blocks or one
    CUtensorMap tk, tv;        // rings: 128 keys x 2 blocks (K), VKEYS keys x all blocks (V)
    CUtensorMap tkp, tvp;      // rings in pieces of kPiece keys x one block
    CUtensorMap tkt, tvt;      // nodes' keys and values, boxes as tk's and tv's
    const uint16_t* k;
    const uint16_t* v;
    float4* part_o;            // [unit][lanes / 32][d / 4][32]: a store of 32 lanes is 512 bytes in a row
    float4* part_l;            // [unit][lanes]: l of each column quarter
    float* part_m;             // [unit][lanes]: m (log2 units)
    int* status;
    int* next_unit;
    const int* list;           // kPair ints a (row, span) pair
    const int* pairs;          // how many
    int rows, nodes, hq, hkv, gsz, npt, qn, mtiles, spans, lanes, win, ring, shared_kv;
    float c;                   // |scale| * log2(e)
    int neg;
};

// QR: query rows that the Q buffer holds.  A tile of up to 64 rows leaves room for one more slot at head
// dim 256; the tensor core then reads rows past the buffer, which no output uses.
template <int D, int QR>
struct TreeCfg {
    static constexpr int KB = D / 64;
    static constexpr int Q_BLOCK = QR * 128;                  // 64 dims of QR rows
    static constexpr int Q_BYTES = KB * Q_BLOCK;
    static constexpr int HV = D / 128;                        // loads an operand and tile
    static constexpr int SLOT = 32768;                        // K: 128 keys x 128 dims; V: 128 / HV keys x D dims
    static constexpr int NSLOT = D == 256 && QR == 128 ? 5 : 6;
    // Load barriers are per operand part and tile, tile mod NB: a parity wait is sound while the
    // load of tile t + NB cannot land before the one of tile t was waited for, which the slot
    // ring gives for 2 HV NB > NSLOT + HV - 1 (2 HV loads a tile).
    static constexpr int NB = D == 256 ? 2 : 4;
    static_assert(2 * HV * NB > NSLOT + HV - 1, "load barrier phases");
    static constexpr int VKEYS = kTile / HV;                  // keys of a V load
    static constexpr int K_BLOCK = kTile * 128;
    static constexpr int V_BLOCK = VKEYS * 128;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_RING = OFF_Q + Q_BYTES;
    static constexpr int OFF_X = OFF_RING + NSLOT * SLOT;     // row maxima [3 tiles][128]
    static constexpr int B_KFULL = 0;                         // [HV][NB]
    static constexpr int B_VFULL = B_KFULL + HV * NB;
    static constexpr int B_VREADY = B_VFULL + HV * NB;
    static constexpr int B_FREE = B_VREADY + HV * NB;         // [NSLOT]
    // S buffers: S runs NS - 1 tiles ahead of P V, so with three (head dim 128 has the columns) the softmax
    // finds its next tile done while the tensor core works on P V of the last two.
    static constexpr int NS = D == 128 ? 3 : 2;
    static constexpr int B_SFULL = B_FREE + NSLOT;            // [tile mod NS] from here
    static constexpr int B_PVDONE = B_SFULL + NS;
    static constexpr int B_PHALF = B_PVDONE + NS;
    static constexpr int B_PFULL = B_PHALF + NS;
    static constexpr int B_XCHG = B_PFULL + NS;                // [lane quarter][tile & 1]
    static constexpr int B_QFULL = B_XCHG + 8;
    static constexpr int B_QFREE = B_QFULL + 1;
    static constexpr int B_UFULL = B_QFREE + 1;               // [kUnits]
    static constexpr int B_UFREE = B_UFULL + kUnits;
    static constexpr int B_DRAIN = B_UFREE + kUnits;
    static constexpr int NBAR = B_DRAIN + 1;
    static constexpr int OFF_BAR = OFF_X + 3 * 128 * 4;
    static constexpr int OFF_UNIT = (OFF_BAR + NBAR * 8 + 15) / 16 * 16;   // 8 ints and 128 parents a slot
    static constexpr int UNIT_BYTES = 32 + WA_TREE_MAX_NODES;
    static constexpr int OFF_MISC = OFF_UNIT + kUnits * UNIT_BYTES;
    static constexpr int SMEM = OFF_MISC + 16;
    static_assert(SMEM <= 232448, "shared memory budget");
    // tensor memory: O (D columns), NS buffers of S; P's two parts over S
    static constexpr int TMEM_COLS = 512;
    __host__ __device__ static constexpr int s_col(int b) { return D + b * kTile; }
    static_assert(s_col(NS - 1) + kTile <= TMEM_COLS, "tensor memory budget");
};

// The load order is K(0), then for each tile t: K(t + 1) if there is one, V(t).  Operand index of V(t) in
// it (HV loads each).
__device__ __forceinline__ int op_v(int t, bool last_of_all) { return last_of_all ? 2 * t + 1 : 2 * t + 2; }

// Its inverse: operand o is K or V of tile t, where K loads have begun for `tiles` tiles.
__device__ __forceinline__ void load_at(int o, int tiles, int& t, bool& is_v) {
    is_v = o > 0 && ((o & 1) == 0 || o == 2 * tiles - 1);
    t = o == 0 ? 0 : is_v ? (o == 2 * tiles - 1 ? tiles - 1 : o / 2 - 1) : (o + 1) / 2;
}

// One tcgen05.mma with its operands in the form the issue needs: descriptors as two 32-bit halves of which
// only the low one (the address) changes, and the accumulate flag as an immediate.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);      // stride 1024, version 1, 128-byte swizzle
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return ((saddr >> 4) & 0x3FFFu) | ((lbo >> 4) << 16); }
template <bool ACC>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tmov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
        "setp.ne.u32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}"
        :: "r"(d), "r"(a_lo), "r"(b_lo), "r"(idesc), "n"(ACC ? 1 : 0), "n"(kDescHi));
}
template <bool ACC>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tmov.b64 db, {%2, %5};\n\t"
        "setp.ne.u32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}"
        :: "r"(d), "r"(a), "r"(b_lo), "r"(idesc), "n"(ACC ? 1 : 0), "n"(kDescHi));
}
// One lane of a converged warp, always the same.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// fp32 values as integers of the same order (NaN aside), and -inf in that order.
__device__ __forceinline__ int ordered(float x) {
    const int b = __float_as_int(x);
    return b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float unordered(int b) { return __int_as_float(b ^ ((b >> 31) & 0x7FFFFFFF)); }
constexpr int kNoMax = static_cast<int>(0xFF800000u) ^ 0x7FFFFFFF;

// A published unit.  nt = 0 marks the end.
struct TreeUnit {
    int r, g, node0, span, k0, nring, nt, p, n, lo;
};

// One block, a warp a row at a time, and nothing reads keys before it is done: 5 to 8 us up to 64 rows, then 50 ns a row.
// Calls of many short rows feel it (4 nodes, 4/2 heads of 128, a window of 256): 13 of 50 us at 256 rows, 46 of 157 at
// 1,024, 201 of 625 at 4,096, 795 of 2,490 at 16,384.
__global__ void __launch_bounds__(1024) tree_plan_kernel(const int32_t* __restrict__ pos, const int32_t* __restrict__ parent,
                                                         const int32_t* __restrict__ n, int rows, int nodes, int hq, int win,
                                                         int ring, WsHeader* hdr, int* __restrict__ list) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ int count[32], at[32];          // pairs of so many tiles (at most 16 of a span and the tree's)
    static_assert(kSpanMax / kTile + 1 < 32, "tiles of a pair");
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    struct Row {
        int p, n, lo, spans, each, more;       // the last `more` spans have each + 1 tiles, the others each
    };
    auto row_at = [&](int r, int& bad) {
        Row x;
        const int raw_p = __ldg(pos + r), raw_n = n ? __ldg(n + r) : nodes;
        x.n = min(max(raw_n, 0), nodes);
        x.p = tree_pos(raw_p, win, ring);
        x.lo = tree_first(x.p, win);
        const int tiles = tree_tiles(x.p, win), spans = tree_cut(tiles, tree_keys(x.p, win), win, hq);
        x.spans = x.n > 0 ? spans : 0;
        x.each = tiles / spans;
        x.more = tiles - x.each * spans;
        bad |= (raw_n != x.n ? WA_STATUS_BAD_TREE : 0) | (raw_p != x.p ? WA_STATUS_BAD_POS : 0);
        return x;
    };
    // four parents a lane, as bytes
    auto parents = [&](int r) {
        int4 v;
        const int32_t* row = parent + static_cast<int64_t>(r) * nodes + 4 * lane;
        v.x = 4 * lane < nodes ? __ldg(row) : -1;
        v.y = 4 * lane + 1 < nodes ? __ldg(row + 1) : -1;
        v.z = 4 * lane + 2 < nodes ? __ldg(row + 2) : -1;
        v.w = 4 * lane + 3 < nodes ? __ldg(row + 3) : -1;
        return v;
    };
    int4 raw = warp < rows ? parents(warp) : make_int4(-1, -1, -1, -1);
    if (t < 32) count[t] = 0;
    __syncthreads();
    int bad = 0;
    for (int r = t; r < rows; r += 1024) {
        const Row x = row_at(r, bad);
        if (x.spans == 0) continue;
        atomicAdd(&count[x.each], x.spans - x.more);
        if (x.more > 0) atomicAdd(&count[x.each + 1], x.more);
    }
    __syncthreads();
    if (warp == 0) {       // longest first: a pair goes after all longer ones
        const int mine = count[31 - lane];
        int sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if (lane >= o) sum += y;
        }
        at[31 - lane] = sum - mine;
        if (lane == 31) {
            hdr->nflag = 0;
            hdr->next_unit = 0;
            hdr->pairs = sum;
        }
    }
    __syncthreads();
    for (int r = warp; r < rows; r += 32) {
        const Row x = row_at(r, bad);
        if (r != warp) raw = parents(r);
        const int v[4] = {raw.x, raw.y, raw.z, raw.w};
        uint32_t bytes = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = 4 * lane + e, a = tree_parent(v[e], i);
            if (i < x.n && a != v[e]) bad |= WA_STATUS_BAD_TREE;
            bytes |= (static_cast<uint32_t>(a) & 255u) << (8 * e);
        }
        for (int s0 = 0; s0 < x.spans; s0 += 32) {       // a span a lane
            const int s = s0 + lane, left = min(32, x.spans - s0);
            int slot = 0;
            if (lane < left) {
                const int extra = s - (x.spans - x.more), t0 = s * x.each + max(extra, 0), nt = x.each + (extra >= 0 ? 1 : 0);
                slot = atomicAdd(&at[nt], 1);
                int4* rec = reinterpret_cast<int4*>(list + static_cast<int64_t>(slot) * kPair);
                rec[0] = make_int4(r, s, x.lo + t0 * kTile, nt - (s == x.spans - 1 ? 1 : 0));
                rec[1] = make_int4(nt, x.p, x.n, x.lo);
            }
            for (int i = 0; i < left; ++i)
                list[static_cast<int64_t>(__shfl_sync(0xFFFFFFFFu, slot, i)) * kPair + 8 + lane] = static_cast<int>(bytes);
        }
    }
    const int tree = __syncthreads_or(bad & WA_STATUS_BAD_TREE), where = __syncthreads_or(bad & WA_STATUS_BAD_POS);
    if (t == 0) hdr->status = (tree ? WA_STATUS_BAD_TREE : 0) | (where ? WA_STATUS_BAD_POS : 0);
}

// 16 bytes to shared memory, without a register in between; over with cp.async.wait_all.
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(src) : "memory");
}

// Keys at ring slots sl0, sl0 + 1, ... (sl0 < ring) that pass the ring's end, into a slot of the shared-memory ring,
// by one warp: pieces of kPiece keys by TMA, a lane each, and the piece that itself wraps by asynchronous copies;
// nothing is waited for.  It takes the producer about 2,400 cycles: 150 for a copy of the warp, 70 for a box. The
// slots come into range by subtraction: `x %= ring` under an `if` was run always, division and all (a batch over a
// window 232 us, then 222).  Pieces of 8, 16 and 32 keys: 217.6, 216.5 and 220.8 us; one sequence over a window 19.1, 18.7
// and 19.9.  Out of line and not unrolled: few tiles come here, once or twice a call, from a cold instruction cache, and
// among the producer's code it cost the other roles 14 % at 128 query rows.
// `lg`: log2 of a key's 16-byte parts of the load; `base`: the first of them of ring slot 0; `map`: boxes of kPiece
// keys and 64 dims.
constexpr int kPiece = 16;
__device__ __noinline__ void load_wrapped(const CUtensorMap* map, const uint16_t* base, int64_t tok, int ring, int nkeys, int lg,
                                          int blk0, int g, int r, int sl0, uint32_t dst, uint32_t full, uint64_t pol) {
    const int lane = static_cast<int>(threadIdx.x) & 31, blk = nkeys * 128;
    // piece `lane`: its ring slot, and whether it wraps
    int mine = sl0 + kPiece * lane;
    while (mine >= ring) mine -= ring;               // more than once only where a ring is shorter than a tile
    const bool in = lane * kPiece < nkeys, whole = in && mine + kPiece <= ring;
    const uint32_t wholes = __ballot_sync(0xFFFFFFFFu, whole);
    uint32_t split = __ballot_sync(0xFFFFFFFFu, in && !whole);
    // the pieces that wrap, by asynchronous copies
    while (split != 0u) {
        const int a = __ffs(split) - 1, sl = __shfl_sync(0xFFFFFFFFu, mine, a);
        split &= split - 1;
#pragma unroll 1
        for (int e = lane; e < kPiece << lg; e += 32) {
            const int k = e >> lg, part = e & ((1 << lg) - 1);
            int slot = sl + k;
            while (slot >= ring) slot -= ring;
            cp_async_16(dst + (part >> 3) * blk + (kPiece * a + k) * 128 + (((part & 7) ^ (k & 7)) * 16), base + slot * tok + part * 8);
        }
    }
    // the others by TMA (which may land before the barrier is told how much to expect: its one arrival is still to
    // come, and one more for each lane, once its own copies have landed)
    if (whole) {
#pragma unroll 1
        for (int b = 0; b < 1 << (lg - 3); ++b)
            tma_load_5d(dst + b * blk + lane * kPiece * 128, map, 0, mine, blk0 + b, g, r, full, pol);
    }
    asm volatile("cp.async.mbarrier.arrive.shared::cta.b64 [%0];" :: "r"(full) : "memory");
    __syncwarp();
    if (lane == 0) mbar_arrive_expect_tx(full, (__popc(wholes) * kPiece * 16) << lg);
    __syncwarp();
}

template <int D, int QR>
__global__ void __launch_bounds__(kTreeThreads, 1) tree_kernel(const __grid_constant__ TreeParams p) {
    using C = TreeCfg<D, QR>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    if (sbase & 1023u) {
        asm volatile("griddepcontrol.wait;" ::: "memory");     // the plan writes the status word
        if (threadIdx.x == 0) atomicOr(p.status, WA_STATUS_LAYOUT);
        return;
    }
    const uint32_t bar0 = sbase + C::OFF_BAR;
    auto BAR = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
    auto SLOT = [&](int s) { return sbase + C::OFF_RING + static_cast<uint32_t>(s) * C::SLOT; };
    auto LOADBAR = [&](int base, int half, int t) { return BAR(base + half * C::NB + t % C::NB); };
    auto LOADPH = [&](int t) { return static_cast<uint32_t>(t / C::NB) & 1u; };
    uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
    int* xbuf = reinterpret_cast<int*>(smem + C::OFF_X);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // a barrier a thread: one thread takes 100 cycles each, 6,000 for all
    static_assert(C::NBAR <= 128, "warps 4..7 set up the barriers");
    if (threadIdx.x >= 128 && threadIdx.x < 128 + C::NBAR) {
        const int i = threadIdx.x - 128;
        int count = 1;
        if (i >= C::B_PHALF && i < C::B_PFULL) count = 16;             // the softmax warps
        else if (i >= C::B_PFULL && i < C::B_XCHG) count = 8;          // those of keys 64 and up
        else if (i >= C::B_XCHG && i < C::B_QFULL) count = 4;          // those of a lane quarter
        else if (i >= C::B_UFREE && i < C::B_DRAIN) count = 19;        // producer, MMA, V, softmax warps
        mbar_init(BAR(i), count);
        fence_mbar_init();
    }
    if (threadIdx.x >= 128 && threadIdx.x < 256) xbuf[threadIdx.x - 128] = kNoMax;    // the first tile's maxima
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
        x.r = e[0]; x.g = e[1] & 0xFFFF; x.node0 = e[1] >> 16; x.span = e[2]; x.k0 = e[3];
        x.nring = e[4] & 0xFFFFFF; x.nt = x.nring + (e[4] >> 24); x.p = e[5]; x.n = e[6]; x.lo = e[7];
    };
    auto take_unit = [&](int U, TreeUnit& x) -> bool {
        if (!warp_wait(BAR(C::B_UFULL + U % kUnits), static_cast<uint32_t>(U / kUnits) & 1u, p.status)) return false;
        read_unit(U, x);
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(C::B_UFREE + U % kUnits));
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
        int u = 0;                                // loads issued
        int tk = 0;                               // tiles whose K loads have begun
        // one load: K of 128 keys and 128 dims, or V of VKEYS keys and all dims; slot0: the ring slot of the
        // tile's first key, -1 for the nodes' own keys
        auto load_half = [&](const TreeUnit& x, int slot0, int t, bool is_v, int half) -> bool {
            const int s = u % C::NSLOT, use = u / C::NSLOT;
            if (use > 0 && !warp_wait(BAR(C::B_FREE + s), (use - 1) & 1, p.status)) return false;
            const uint32_t full = LOADBAR(is_v ? C::B_VFULL : C::B_KFULL, half, t);
            const uint32_t dst = SLOT(s);
            const int blk0 = is_v ? 0 : half * 2, key = is_v ? half * C::VKEYS : 0, nkeys = is_v ? C::VKEYS : kTile;
            int sl0 = slot0 + key;
            if (p.win > 0)
                while (sl0 >= p.ring) sl0 -= p.ring;       // more than once only where a ring is shorter than a tile
            if (slot0 < 0 || p.win == 0 || sl0 + nkeys <= p.ring) {
                if (lane == 0) {
                    mbar_arrive_expect_tx(full, C::SLOT);
                    if (slot0 < 0) tma_load_5d(dst, is_v ? &p.tvt : &p.tkt, 0, key, blk0, x.g, x.r, full, pol);
                    else tma_load_5d(dst, is_v ? &p.tv : &p.tk, 0, sl0, blk0, x.g, x.r, full, pol);
                }
            } else {
                const int64_t tok = static_cast<int64_t>(p.hkv) * D;
                load_wrapped(is_v ? &p.tvp : &p.tkp, (is_v ? p.v : p.k) + (static_cast<int64_t>(x.r) * p.ring * p.hkv + x.g) * D + blk0 * 64, tok, p.ring, nkeys,
                             is_v && D == 256 ? 5 : 4, blk0, x.g, x.r, sl0, dst, full, pol);
            }
            __syncwarp();
            ++u;
            return true;
        };
        auto load_k = [&](const TreeUnit& x, int slot0, int t) -> bool {
            tk = t + 1;
            bool ok = true;
#pragma unroll
            for (int h = 0; h < C::HV; ++h) ok = ok && load_half(x, slot0, t, false, h);
            return ok;
        };
        // the ring slot of a unit's first tile, and of the tile after one
        auto first_slot = [&](const TreeUnit& x) { return x.nring == 0 ? -1 : p.win > 0 ? x.k0 % p.ring : x.k0; };
        auto next_slot = [&](const TreeUnit& x, int idx, int slot0) {
            if (idx + 1 >= x.nring) return -1;
            int sl = slot0 + kTile;
            if (p.win > 0)
                while (sl >= p.ring) sl -= p.ring;
            return sl;
        };
        TreeUnit cur, nxt;
        int U = 0, t = 0, idx = 0, sc = -1;
        bool ok = take_unit(U++, cur);
        bool more = ok && cur.nt > 0;
        if (more) {
            sc = first_slot(cur);
            ok = load_k(cur, sc, 0);
        }
        while (ok && more) {
            // the tile after (cur, idx): its K goes first
            const bool same = idx + 1 < cur.nt;
            int sn = -1;
            if (same) {
                sn = next_slot(cur, idx, sc);
                ok = load_k(cur, sn, t + 1);
            } else {
                if (!(ok = take_unit(U++, nxt))) break;
                more = nxt.nt > 0;
                if (more) {
                    sn = first_slot(nxt);
                    ok = load_k(nxt, sn, t + 1);
                }
            }
            if (!ok) break;
#pragma unroll
            for (int h = 0; h < C::HV; ++h) ok = ok && load_half(cur, sc, t, true, h);
            if (same) {
                ++idx;
            } else {
                cur = nxt;
                idx = 0;
            }
            sc = sn;
            ++t;
        }
        // the copies in flight land before the block exits, whichever role stopped early (after a whole
        // run every one was consumed, and the waits return at once)
        if (lane == 0) {
            for (int i = max(0, u - C::NSLOT); i < u; ++i) {
                int tt;
                const int half = i % C::HV;
                bool v;
                load_at(i / C::HV, tk, tt, v);
                mbar_wait(LOADBAR(v ? C::B_VFULL : C::B_KFULL, half, tt), LOADPH(tt), p.status);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer: the warp together, one lane's instructions
        // The warp walks converged over values that the compiler can see to be the same in every lane, so that
        // addresses and descriptors live in uniform registers.  As one thread's code over 64-bit descriptors an
        // instruction took about 130 cycles to issue beside the softmax warps, twice its time on the tensor core.
        const uint32_t tb = __shfl_sync(0xFFFFFFFFu, tbase, 0);
        const bool leader = elect_one();
        const uint32_t idS = idesc_bf16_f32(128, kTile, 0, 0, p.neg ? 1u : 0u);
        constexpr uint32_t idO = idesc_bf16_f32(128, D, 0, 1);
        const uint32_t aq = desc_lo(sbase + C::OFF_Q, 16);
        // the slots of K(t) and V(t): K0, K1, V0, K2, V1, ... with HV loads each; the last tile's V has no K before it
        int ks = 0, vs = 2 * C::HV % C::NSLOT;
        auto wrap = [](int x) { return x >= C::NSLOT ? x - C::NSLOT : x; };
        auto issue_s = [&](int t) -> bool {
            const uint32_t d = tb + C::s_col(t % C::NS);
#pragma unroll
            for (int kh = 0; kh < C::HV; ++kh) {
                const int s = wrap(ks + kh);
                if (!warp_wait(LOADBAR(C::B_KFULL, kh, t), LOADPH(t), p.status)) return false;
                fence_proxy_async_smem();        // for load_wrapped's copies
                tc_fence_after();
                const uint32_t bk = desc_lo(SLOT(s), 16);
                if (leader) {
#pragma unroll
                    for (int k8 = 0; k8 < 8; ++k8) {
                        const int kk = 8 * kh + k8;
                        const uint32_t a = aq + (((kk >> 2) * C::Q_BLOCK + (kk & 3) * 32) >> 4);
                        const uint32_t b = bk + (((k8 >> 2) * C::K_BLOCK + (k8 & 3) * 32) >> 4);
                        if (kk == 0) mma_ss<false>(d, a, b, idS);
                        else mma_ss<true>(d, a, b, idS);
                    }
                    mma_commit(BAR(C::B_FREE + s));
                    if (kh == C::HV - 1) mma_commit(BAR(C::B_SFULL + t % C::NS));
                }
                __syncwarp();
            }
            ks = wrap(ks + (t == 0 ? C::HV : 2 * C::HV));
            return true;
        };
        // keys 0..63 of the tile, then 64..127, as their P arrives
        auto issue_pv = [&](int t, bool first, bool last_of_all) -> bool {
            const uint32_t pb = tb + C::s_col(t % C::NS);
            const int v = last_of_all ? wrap(vs + C::NSLOT - C::HV) : vs;
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const int part_v = hh * 64 / C::VKEYS;
                const int s = wrap(v + part_v);
                if (hh * 64 % C::VKEYS == 0 && !warp_wait(LOADBAR(C::B_VREADY, part_v, t), LOADPH(t), p.status)) return false;
                if (!warp_wait(BAR((hh ? C::B_PFULL : C::B_PHALF) + t % C::NS), (t / C::NS) & 1, p.status)) return false;
                tc_fence_after();
                const uint32_t v0 = desc_lo(SLOT(s) + (hh * 64 % C::VKEYS) * 128, C::V_BLOCK);
                if (leader) {
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int k4 = 0; k4 < 4; ++k4) {
                            const uint32_t a = pb + hh * 64 + (k4 >> 1) * 32 + part * 16 + (k4 & 1) * 8;
                            const uint32_t b = v0 + ((k4 * 16 * 128) >> 4);
                            if (hh == 0 && part == 0 && k4 == 0 && first) mma_ts<false>(tb, a, b, idO);
                            else mma_ts<true>(tb, a, b, idO);
                        }
                    if ((hh + 1) * 64 % C::VKEYS == 0) mma_commit(BAR(C::B_FREE + s));
                    if (hh == 1) mma_commit(BAR(C::B_PVDONE + t % C::NS));
                }
                __syncwarp();
            }
            vs = wrap(vs + 2 * C::HV);
            return true;
        };
        int t = 0;
        bool ok = true;
        int ntl = 0;                              // the last unit's tiles: P V of its last NS - 1 is still to issue
        for (int U = 0; ok; ++U) {
            TreeUnit x;
            if (!(ok = take_unit(U, x))) break;
            const int nt = __shfl_sync(0xFFFFFFFFu, x.nt, 0);
            // a unit's last P V go before the next unit's S, which may still wait for its Q
            for (int i = min(ntl, C::NS - 1); ok && i > 0; --i) ok = issue_pv(t - i, ntl == i, nt <= 0 && i == 1);
            if (!ok || nt <= 0) break;
            ok = warp_wait(BAR(C::B_QFULL), U & 1, p.status);
            for (int idx = 0; ok && idx < nt; ++idx, ++t) {
                ok = issue_s(t);
                if (ok && idx == nt - 1 && leader) mma_commit(BAR(C::B_QFREE));
                if (ok && idx >= C::NS - 1) ok = issue_pv(t - (C::NS - 1), idx == C::NS - 1, false);
            }
            ntl = nt;
        }
        // every product issued has finished before tensor memory can be released
        if (leader) {
            mma_commit(BAR(C::B_DRAIN));
            mbar_wait(BAR(C::B_DRAIN), 0, p.status);
        }
        __syncwarp();
    } else if (warp == 2) {
        // ------------------------------------------------ V rows that no node sees -> 0
        int t = 0;
        TreeUnit x, nxt;
        bool ok = take_unit(0, x);
        for (int U = 1; ok && x.nt > 0; ++U) {
            bool have_next = false;
            for (int idx = 0; ok && idx < x.nt; ++idx, ++t) {
                // whether this is the very last tile decides where its V sits in the load order
                if (idx == x.nt - 1) {
                    if (!(ok = take_unit(U, nxt))) break;
                    have_next = true;
                }
                const bool last_of_all = have_next && nxt.nt <= 0;
                for (int hh = 0; hh < C::HV; ++hh) {
                    const int s = (C::HV * op_v(t, last_of_all) + hh) % C::NSLOT;
                    if (!(ok = warp_wait(LOADBAR(C::B_VFULL, hh, t), LOADPH(t), p.status))) break;
                    int z_lo, z_hi, z_end = C::VKEYS;       // rows [0, z_lo) and [z_hi, z_end) are cleared
                    if (idx < x.nring) {
                        const int key0 = x.k0 + idx * kTile + hh * C::VKEYS;
                        z_lo = min(C::VKEYS, max(0, x.lo - key0));
                        z_hi = max(0, min(C::VKEYS, x.p - key0 + 1));
                    } else {
                        z_lo = 0;
                        z_hi = max(0, min(C::VKEYS, x.n - hh * C::VKEYS));
                        z_end = max(0, min(C::VKEYS, p.nodes - hh * C::VKEYS));   // past the buffer's nodes TMA has filled zeros
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
                    }
                    fence_proxy_async_smem();        // for these, and for load_wrapped's copies
                    __syncwarp();
                    if (lane == 0) mbar_arrive(LOADBAR(C::B_VREADY, hh, t));
                }
            }
            if (ok) x = nxt;
        }
    } else if (warp == 3) {
        // ------------------------------------------------ units; Q
        // this kernel starts while the plan still runs (and so does all that follows its first published unit)
        asm volatile("griddepcontrol.wait;" ::: "memory");
        const int per = p.hkv * p.mtiles, units = *p.pairs * per;
        int k_cur = blockIdx.x, k_ans = 0, pub = 0, loaded = 0;
        bool asked = false, ended = false, ok = true;
        int par = 0;              // four of the unit's parents a lane
        // the next unit with any work (nt = 0: none left); its number was asked for one unit ahead
        auto next_unit = [&](TreeUnit& x) {
            for (;;) {
                if (asked) k_cur = __shfl_sync(0xFFFFFFFFu, k_ans, 0) + static_cast<int>(gridDim.x);
                x.nt = 0;
                x.nring = 0;
                if (k_cur >= units) return;
                const int pair = k_cur / per, rem = k_cur % per;
                const int* rec = p.list + static_cast<int64_t>(pair) * kPair;
                const int field = rec[lane & 7];
                par = rec[8 + lane];
                if (lane == 0) k_ans = atomicAdd(p.next_unit, 1);
                asked = true;
                x.g = rem / p.mtiles;
                x.node0 = rem % p.mtiles * p.npt;
                x.r = __shfl_sync(0xFFFFFFFFu, field, 0);
                x.span = __shfl_sync(0xFFFFFFFFu, field, 1);
                x.k0 = __shfl_sync(0xFFFFFFFFu, field, 2);
                x.nring = __shfl_sync(0xFFFFFFFFu, field, 3);
                x.nt = __shfl_sync(0xFFFFFFFFu, field, 4);
                x.p = __shfl_sync(0xFFFFFFFFu, field, 5);
                x.n = __shfl_sync(0xFFFFFFFFu, field, 6);
                x.lo = __shfl_sync(0xFFFFFFFFu, field, 7);
                if (x.node0 < x.n) return;
            }
        };
        auto publish_next = [&](TreeUnit& x) -> bool {
            x.nt = 0;
            if (ended) return true;
            next_unit(x);
            ended = x.nt <= 0;
            if (pub >= kUnits && !warp_wait(BAR(C::B_UFREE + pub % kUnits), static_cast<uint32_t>(pub / kUnits - 1) & 1u, p.status))
                return false;
            volatile int* e = unit_ints(pub);
            if (!ended) e[8 + lane] = par;
            if (lane == 0) {
                e[0] = x.r; e[1] = x.g | (x.node0 << 16); e[2] = x.span; e[3] = x.k0;
                e[4] = x.nring | ((x.nt - x.nring) << 24); e[5] = x.p; e[6] = x.n; e[7] = x.lo;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(C::B_UFULL + pub % kUnits));
            ++pub;
            return true;
        };
        auto load_q = [&](const TreeUnit& x) {
            if (lane == 0) {
                mbar_arrive_expect_tx(BAR(C::B_QFULL), C::KB * p.gsz * p.qn * 128);
                if (p.gsz * p.qn == QR) {
                    tma_load_5d(sbase + C::OFF_Q, &p.tq, 0, x.g * p.gsz, x.node0, 0, x.r, BAR(C::B_QFULL), policy_evict_last());
                } else {        // a tile that does not fill a block: block by block
                    for (int b = 0; b < C::KB; ++b)
                        tma_load_5d(sbase + C::OFF_Q + b * C::Q_BLOCK, &p.tq, 0, x.g * p.gsz, x.node0, b, x.r, BAR(C::B_QFULL),
                                    policy_evict_last());
                }
            }
            __syncwarp();
            ++loaded;
        };
        TreeUnit u0, u1, u2;      // the unit whose Q is next, and kAhead = 2 more
        static_assert(kAhead == 2, "units held here");
        ok = publish_next(u0);
        if (ok && u0.nt > 0) load_q(u0);
        u1.nt = u2.nt = 0;
        ok = ok && publish_next(u1) && publish_next(u2);
        for (int U = 1; ok; ++U) {
            u0 = u1;
            u1 = u2;
            if (u0.nt <= 0 || !(ok = publish_next(u2))) break;
            // Q of unit U, once the last S of unit U - 1 has read the buffer
            if (!(ok = warp_wait(BAR(C::B_QFREE), (U - 1) & 1, p.status))) break;
            load_q(u0);
        }
        if (lane == 0 && loaded > 0) mbar_wait(BAR(C::B_QFULL), (loaded - 1) & 1, p.status);
    } else {
        // ------------------------------------------------ softmax: query row r, column quarter cq
        const int cq = (warp - 4) >> 2, quarter = warp & 3;
        const int r = quarter * 32 + lane;
        const int rn = r / p.gsz;                             // the row's node within the tile
        const int col0 = cq * 32;
        const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
        const float c = p.c;
        // a unit as this thread sees it
        int k0 = 0, nring = 0, nt = 0, row_lo = 0, row_hi = 0;
        uint32_t seen = 0;                                    // tree columns [col0, col0 + 32) that the row sees
        int first_full = 0, last_full = 0;                    // keys that every row of the warp sees
        bool live = false, idle = true;
        int64_t unit = 0;
        auto fetch = [&](int U) -> bool {
            if (!warp_wait(BAR(C::B_UFULL + U % kUnits), static_cast<uint32_t>(U / kUnits) & 1u, p.status)) return false;
            TreeUnit x;
            read_unit(U, x);
            k0 = x.k0;
            nring = x.nring;
            nt = x.nt;
            row_hi = x.p;
            const int node = x.node0 + rn;
            live = x.nt > 0 && rn < p.npt && node < x.n;
            row_lo = 0;
            seen = 0xFFFFFFFFu;                               // rows without a node: nothing masked
            if (live) {
                const uint32_t par = sbase + C::OFF_UNIT + (U % kUnits) * C::UNIT_BYTES + 32;
                uint32_t a = node;
                int back = 0;
                seen = 0u;
                do {
                    const uint32_t col = a - col0;
                    if (col < 32u && (p.win == 0 || back < p.win)) seen |= 1u << col;
                    ++back;
                    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(a) : "r"(par + a) : "memory");
                } while (a != 255u);
                row_lo = p.win > 0 ? max(0, x.p + back - p.win + 1) : 0;   // back = depth + 1
            }
            idle = !__any_sync(0xFFFFFFFFu, live);            // a warp without rows only keeps the barriers going
            first_full = __reduce_max_sync(0xFFFFFFFFu, row_lo);
            last_full = x.p;
            unit = ((static_cast<int64_t>(x.r) * p.hkv + x.g) * p.mtiles + x.node0 / p.npt) * p.spans + x.span;
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(C::B_UFREE + U % kUnits));
            return true;
        };
        int t = 0;
        bool ok = fetch(0);
        for (int U = 0; ok && nt > 0; ++U) {
            float m_run = -INFINITY, l_run = 0.f;
            for (int idx = 0; idx < nt; ++idx, ++t) {
                const int b = t % C::NS;
                const uint32_t ph = static_cast<uint32_t>(t >> 1) & 1u;
                const uint32_t xbar = BAR(C::B_XCHG + 2 * quarter + (t & 1));
                if (!(ok = warp_wait(BAR(C::B_SFULL + b), static_cast<uint32_t>(t / C::NS) & 1u, p.status))) break;
                const int xb = t % 3 * 128, xnext = (t + 1) % 3 * 128;
                if (cq == 0) xbuf[xnext + r] = kNoMax;        // free since every warp read tile t - 2's maxima
                if (idle) {
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(xbar);
                        mbar_arrive(BAR(C::B_PHALF + b));
                        if (cq >= 2) mbar_arrive(BAR(C::B_PFULL + b));
                    }
                    __syncwarp();
                    // the quarter's warps stay within a tile of each other, as the maxima's buffers need
                    if (!(ok = warp_wait(xbar, ph, p.status))) break;
                    continue;
                }
                tc_fence_after();
                const uint32_t t_s = tbase + lane_addr + C::s_col(b) + col0;
                // visible columns of this quarter as bits, unless every row sees them all
                const int kbase = k0 + idx * kTile + col0;
                const bool masked = idx >= nring || kbase < first_full || kbase + 31 > last_full;
                uint32_t vis = seen;
                if (masked && idx < nring) {
                    const int vlo = live ? max(0, row_lo - kbase) : 0, vhi = live ? min(31, row_hi - kbase) : 31;
                    vis = vlo > vhi ? 0u : (0xFFFFFFFFu >> (31 - (vhi - vlo))) << vlo;
                }
                float sv[32];
                auto load = [&]() {
                    load_s<32>(t_s, sv);
                    if (masked) {   // a masked score is -inf, whatever it was: weight 0
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (!((vis >> k) & 1u)) sv[k] = -INFINITY;
                    }
                };
                load();
                float mx4[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    mx4[e] = max3(max3(sv[e], sv[e + 4], sv[e + 8]), max3(sv[e + 12], sv[e + 16], sv[e + 20]),
                                  fmaxf(sv[e + 24], sv[e + 28]));
                const float mh = max3(fmaxf(mx4[0], mx4[1]), mx4[2], mx4[3]);
                if (mh > -INFINITY) atomicMax(&xbuf[xb + r], ordered(mh));   // (not for a NaN)
                __syncwarp();   // the warp's stores precede lane 0's (cumulative) release
                if (lane == 0) mbar_arrive(xbar);
                // The row's maximum over the four quarters; lazy rule: the running one stays unless the tile's
                // exceeds it by more than kTreeLazy.  So the exponentials below start with the running one while
                // the other quarters' maxima are on their way, and are done again, from S, where it moved.
                float m_old = m_run, alpha = 1.f;
                bool spec = __all_sync(0xFFFFFFFFu, !live || m_run != -INFINITY);
                float lsum;
                for (;;) {
                    if (!spec) {
                        if (!(ok = warp_wait(xbar, ph, p.status))) break;
                        const float mt = unordered(xbuf[xb + r]) * c;
                        m_run = (mt > m_old + kTreeLazy) ? mt : m_old;
                        alpha = (m_run == m_old) ? 1.f : ex2(m_old - m_run);
                    }
                    const float m_sub = (m_run == -INFINITY) ? 0.f : m_run;
                    float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        float x0, x1;
                        fma_x2(x0, x1, sv[k], sv[k + 1], c, c, -m_sub, -m_sub);
                        sv[k] = ex2(x0);
                        sv[k + 1] = ex2(x1);
                    }
                    if (c == 0.f && masked) {   // scale 0: -inf * 0 is no weight
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (!((vis >> k) & 1u)) sv[k] = 0.f;
                    }
#pragma unroll
                    for (int k = 0; k < 32; k += 4) {
                        add_x2(ls[0], ls[1], sv[k], sv[k + 1]);
                        add_x2(ls[2], ls[3], sv[k + 2], sv[k + 3]);
                    }
                    lsum = (ls[0] + ls[1]) + (ls[2] + ls[3]);
                    if (!spec) break;
                    if (!(ok = warp_wait(xbar, ph, p.status))) break;
                    const float mt = unordered(xbuf[xb + r]) * c;
                    if (!__any_sync(0xFFFFFFFFu, live && mt > m_old + kTreeLazy)) break;
                    spec = false;
                    load();
                }
                if (!ok) break;
                // O's rescale, once the previous P V is done; a unit's first P V starts O afresh, and a row
                // that has seen nothing yet has an O of zeros
                if (idx > 0 && __any_sync(0xFFFFFFFFu, live && alpha != 1.f && m_old != -INFINITY)) {
                    if (!(ok = warp_wait(BAR(C::B_PVDONE + (t - 1) % C::NS), static_cast<uint32_t>((t - 1) / C::NS) & 1u, p.status)))
                        break;
                    tc_fence_after();
#pragma unroll 1
                    for (int cc = 0; cc < D / 64; ++cc) {
                        uint32_t o[16];
                        const uint32_t ta = tbase + lane_addr + cq * (D / 4) + cc * 16;
                        tmem_ld16_wait(ta, o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        tmem_st16(ta, o);
                    }
                    tmem_wait_st();
                }
                if (cq >= 2) {   // this quarter's O columns are ready for the tile's first P V half
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(BAR(C::B_PHALF + b));
                }
                // P over this quarter's own columns of S: hi = bf16(p) in the first 16, lo = bf16(p - hi) in the others,
                // so their sum is within 2^-17 of p, as in the one-token decode (one part alone: 2^-8).  hi as p's upper
                // half, cut and not rounded, would leave twice the error.
                {
                    uint32_t w[32];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float a = sv[2 * e], bb = sv[2 * e + 1];
                        float ra, rb;                       // exact
                        w[e] = pack_bf16(a, bb);
                        fma_x2(ra, rb, __uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u), -1.f, -1.f, a, bb);
                        w[16 + e] = pack_bf16(ra, rb);
                    }
                    tmem_st32(t_s, w);
                }
                l_run = (alpha == 1.f) ? (l_run + lsum) : fmaf(l_run, alpha, lsum);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(BAR((cq < 2 ? C::B_PHALF : C::B_PFULL) + b));
            }
            if (!ok) break;
            // the next unit's rows are looked up while the last P V runs
            const bool was_idle = idle;
            const int64_t done = unit;
            if (!(ok = fetch(U + 1))) break;
            if (was_idle) continue;
            // the unit's partial result; the next unit's first P V waits for this warp's next PHALF
            if (!(ok = warp_wait(BAR(C::B_PVDONE + (t - 1) % C::NS), static_cast<uint32_t>((t - 1) / C::NS) & 1u, p.status))) break;
            tc_fence_after();
            float4* po = p.part_o + ((done * (p.lanes >> 5) + quarter) * (D / 4) + cq * (D / 16)) * 32 + lane;
#pragma unroll 1
            for (int cc = 0; cc < D / 128; ++cc) {
                uint32_t o[32];
                tmem_ld32_wait(tbase + lane_addr + cq * (D / 4) + cc * 32, o);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    po[(cc * 8 + e) * 32] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                                        __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
            }
            reinterpret_cast<float*>(p.part_l + done * p.lanes + r)[cq] = l_run;
            if (cq == 0) p.part_m[done * p.lanes + r] = m_run;
        }
    }

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tbase, C::TMEM_COLS);
}

// The float64 value of 64 of an output's dims (from col0), by the whole block: a node's keys are numbered
// lo .. p (the ring) and then p + 1 + t for node t of its tree, of which those in `anc` count.
struct TreeRerun {
    double qd[256];
    float qf[256];
    double wb[kRerunThreads], red[kRerunThreads / 32];
    unsigned char anc[WA_TREE_MAX_NODES], use[kRerunThreads];
};

__device__ void tree_rerun(const TreeArgs& a, TreeRerun& sm, int r, int node, int h, int col0) {
    const int t = threadIdx.x, d = a.d, g = h / (a.hq / a.hkv);
    const int32_t* par = a.parent + static_cast<int64_t>(r) * a.nodes;
    const int p = tree_pos(a.pos[r], a.win, a.ring);
    int depth = 0;
    for (int x = node; (x = tree_parent(par[x], x)) >= 0;) ++depth;
    for (int x = t; x < a.nodes; x += kRerunThreads) sm.anc[x] = 0;
    __syncthreads();
    if (t == 0)
        for (int x = node, back = 0; x >= 0 && (a.win == 0 || back < a.win); x = tree_parent(par[x], x), ++back) sm.anc[x] = 1;
    const int lo = min(a.win > 0 ? max(0, p + 1 + depth - a.win + 1) : 0, p + 1);
    const int last = p + 1 + node;           // an ancestor has a smaller index
    const uint16_t* qrow = static_cast<const uint16_t*>(a.q) + r * a.q_row + node * a.q_tok + static_cast<int64_t>(h) * d;
    const int64_t kst = static_cast<int64_t>(a.hkv) * d, base = r * a.ring * kst + static_cast<int64_t>(g) * d;
    const uint16_t* kb = static_cast<const uint16_t*>(a.k) + base;
    const uint16_t* vb = static_cast<const uint16_t*>(a.v) + base;
    const uint16_t* ktb = static_cast<const uint16_t*>(a.kt) + r * a.kt_row + static_cast<int64_t>(g) * d;
    const uint16_t* vtb = static_cast<const uint16_t*>(a.vt) + r * a.vt_row + static_cast<int64_t>(g) * d;
    uint16_t* orow = static_cast<uint16_t*>(a.out) + r * a.o_row + node * a.o_tok + static_cast<int64_t>(h) * d + col0;
    if (t < d) {
        const float x = __uint_as_float(static_cast<uint32_t>(qrow[t]) << 16);
        sm.qf[t] = x * a.scale;   // only the class of the fp32 score matters
        sm.qd[t] = static_cast<double>(x);
    }
    __syncthreads();
    auto visible = [&](int j) { return j <= last && (j <= p || sm.anc[j - p - 1] != 0); };
    auto key = [&](int j) { return j > p ? ktb + (j - p - 1) * a.kt_tok : kb + static_cast<int64_t>(j % a.ring) * kst; };
    auto val = [&](int j) { return j > p ? vtb + (j - p - 1) * a.vt_tok : vb + static_cast<int64_t>(j % a.ring) * kst; };
    auto score = [&](int j) { return dot_f64(sm.qd, key(j), d) * static_cast<double>(a.scale); };
    // a float64 score that is NaN or +inf makes the output NaN: settled without the passes below
    for (int b = lo; b <= last; b += kRerunThreads) {
        const int j = b + t;
        bool hit = false;
        if (visible(j) && !isfinite(dot_f32(sm.qf, key(j), d))) {
            const double s = score(j);
            hit = isnan(s) || (isinf(s) && s > 0.0);
        }
        if (__syncthreads_or(hit)) {
            if (t < 64) orow[t] = 0x7FC0u;
            return;
        }
    }
    double mloc = -INFINITY;
    for (int j = lo + t; j <= last; j += kRerunThreads) {
        if (!visible(j)) continue;
        const double s = score(j);
        mloc = (isnan(s) || isnan(mloc)) ? (s + mloc) : fmax(mloc, s);
    }
    const double M = block_reduce(mloc, true, sm.red);
    double lloc = 0.0, acc = 0.0;
    for (int b = lo; b <= last; b += kRerunThreads) {
        const int j = b + t;
        const bool use = visible(j);
        double w = 0.0;
        if (use) {
            w = exp(score(j) - M);
            lloc += w;
        }
        sm.wb[t] = w;
        sm.use[t] = use ? 1 : 0;
        __syncthreads();
        if (t < 64) {
            const int cnt = min(kRerunThreads, last - b + 1);
            for (int jj = 0; jj < cnt; ++jj)
                if (sm.use[jj]) acc = acc + sm.wb[jj] * bf16_bits_to_f64(val(b + jj)[col0 + t]);
        }
        __syncthreads();
    }
    const double l = block_reduce(lloc, false, sm.red);
    if (t < 64) orow[t] = f64_to_bf16_rn(acc / l);
}

constexpr int kMergeSpans = 2;

// o = sum_s a_s O_s / sum_s a_s l_s over a row's spans in order, a_s = 2^(m_s - M).  A block takes 32 query
// rows (lanes) and 64 dims (8 a warp) of a tile, reads the partial results in the order they were stored
// (512 bytes a warp and load, kMergeSpans spans in flight), and turns them round in shared memory for the output.
// A row with a value that is not finite is computed again in float64.  Issue bound it when each block worked out its
// place and each output its quotient by divisions (64 rows over a window, 32/16 heads, 222 us a call, then 217).  Four,
// five and six blocks an SM: that batch 216.9, 216.5 and 218.5 us, 32 rows of 64 nodes, 32/4 heads, 441, 442 and 450 (six
// spill); four is within the noise of five.
template <int D>
__global__ void __launch_bounds__(256, 5) tree_merge_kernel(const float4* part_o, const float4* part_l, const float* part_m,
                                                            const __grid_constant__ TreeArgs a, int npt, int mtiles, int spans,
                                                            int lanes, int G, int by_quarters, int by_group) {
    __shared__ __align__(16) uint8_t tile[32 * 144];
    __shared__ int bad[32];
    __shared__ TreeRerun again;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    // x / quarters and x / G by a factor, for x below 2^7 (a runtime division takes 30 instructions or more)
    const int quarters = lanes >> 5, r = blockIdx.x, g = blockIdx.y, z = blockIdx.z / (D / 64), db = blockIdx.z % (D / 64);
    const int mt = z * by_quarters >> 16, qd = z - mt * quarters, node0 = mt * npt;
    auto node_of = [&](int row) { return row * by_group >> 16; };
    const int64_t unit0 = ((static_cast<int64_t>(r) * a.hkv + g) * mtiles + mt) * spans;
    const int n = min(a.n ? __ldg(a.n + r) : a.nodes, a.nodes);
    const int count = tree_spans(tree_pos(__ldg(a.pos + r), a.win, a.ring), a.win, a.hq);
    const int first = node_of(qd * 32);                        // the block's first node
    if (t < 32) bad[t] = 0;
    // The partial results (plain pointers: they are written while this kernel is there already, so no load may go
    // the read-only way or before this line).  Blocks without work wait too: nothing behind the call starts early.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (first >= npt || node0 + first >= n) return;
    __syncthreads();
    const int64_t rec = unit0 * lanes + qd * 32 + lane;
    const float4* po = part_o + ((unit0 * quarters + qd) * (D / 4) + db * 16 + warp * 2) * 32 + lane;
    const int64_t ostep = static_cast<int64_t>(quarters) * (D / 4) * 32;
    float M = -INFINITY, den = 0.f, num[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) num[e] = 0.f;
    // kMergeSpans at a time, all their loads in flight together, folded in order
    for (int s0 = 0; s0 < count; s0 += kMergeSpans) {
        float m[kMergeSpans];
        float4 l[kMergeSpans], o[kMergeSpans][2];
#pragma unroll
        for (int i = 0; i < kMergeSpans; ++i) {
            if (s0 + i >= count) break;
            const int64_t at = rec + static_cast<int64_t>(s0 + i) * lanes;
            m[i] = part_m[at];
            l[i] = part_l[at];
            o[i][0] = po[(s0 + i) * ostep];
            o[i][1] = po[(s0 + i) * ostep + 32];
        }
        float top = M;
#pragma unroll
        for (int i = 0; i < kMergeSpans; ++i)
            if (s0 + i < count) top = fmaxf(top, m[i]);
        const float keep = (M == -INFINITY) ? 0.f : exp2f(M - top);
        M = top;
        den *= keep;
#pragma unroll
        for (int e = 0; e < 8; ++e) num[e] *= keep;
#pragma unroll
        for (int i = 0; i < kMergeSpans; ++i) {
            if (s0 + i >= count) break;
            const float w = exp2f(m[i] - M);
            den = fmaf(w, (l[i].x + l[i].y) + (l[i].z + l[i].w), den);
            num[0] = fmaf(w, o[i][0].x, num[0]);
            num[1] = fmaf(w, o[i][0].y, num[1]);
            num[2] = fmaf(w, o[i][0].z, num[2]);
            num[3] = fmaf(w, o[i][0].w, num[3]);
            num[4] = fmaf(w, o[i][1].x, num[4]);
            num[5] = fmaf(w, o[i][1].y, num[5]);
            num[6] = fmaf(w, o[i][1].z, num[6]);
            num[7] = fmaf(w, o[i][1].w, num[7]);
        }
    }
    const int row = qd * 32 + lane;
    const bool live = node_of(row) < npt && node0 + node_of(row) < n;
    bool nonfinite = false;
    const float inv = __frcp_rn(den);        // two roundings of 2^-24 each, beside the output's 2^-9
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        num[e] *= inv;
        nonfinite |= !isfinite(num[e]);
    }
    if (live && nonfinite) bad[lane] = 1;
    *reinterpret_cast<uint4*>(tile + lane * 144 + warp * 16) =
        make_uint4(pack_bf16(num[0], num[1]), pack_bf16(num[2], num[3]), pack_bf16(num[4], num[5]), pack_bf16(num[6], num[7]));
    const int any = __syncthreads_or(live && nonfinite);
    {   // eight threads a row
        const int m = qd * 32 + t / 8, rn = node_of(m);
        if (rn < npt && node0 + rn < n && !bad[t / 8]) {
            uint16_t* orow = static_cast<uint16_t*>(a.out) + r * a.o_row + (node0 + rn) * a.o_tok +
                             static_cast<int64_t>(g * G + m - rn * G) * D + db * 64;
            reinterpret_cast<uint4*>(orow)[t % 8] = *reinterpret_cast<const uint4*>(tile + t / 8 * 144 + t % 8 * 16);
        }
    }
    if (!any) return;
    for (int i = 0; i < 32; ++i) {
        if (!bad[i]) continue;
        const int m = qd * 32 + i, rn = node_of(m);
        tree_rerun(a, again, r, node0 + rn, g * G + m - rn * G, db * 64);
        __syncthreads();
    }
}

// A [rows][toks][heads][d] bf16 tensor as (64 dims, tokens or heads x tokens, blocks of 64 dims, ...), 128-byte
// swizzle.  `heads_first`: q, whose boxes take heads and tokens (64, heads, tokens, blocks, rows); otherwise
// k and v (64, tokens, blocks, heads, rows).
bool encode_5d(CUtensorMap* m, const void* base, int d, int heads, int toks, int rows, int64_t tok, int64_t row, bool heads_first,
               int box1, int box2, int box3) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t nd = static_cast<cuuint64_t>(d) / 64, nh = heads, nt = toks, nr = rows;
    const cuuint64_t sh = static_cast<cuuint64_t>(d) * 2, st = static_cast<cuuint64_t>(tok) * 2, sb = 128,
                     sr = static_cast<cuuint64_t>(row) * 2;
    cuuint64_t dims_q[5] = {64, nh, nt, nd, nr}, strides_q[4] = {sh, st, sb, sr};
    cuuint64_t dims_k[5] = {64, nt, nd, nh, nr}, strides_k[4] = {st, sb, sh, sr};
    cuuint32_t box[5] = {64, static_cast<cuuint32_t>(box1), static_cast<cuuint32_t>(box2), static_cast<cuuint32_t>(box3), 1};
    cuuint32_t es[5] = {1, 1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), heads_first ? dims_q : dims_k,
               heads_first ? strides_q : strides_k, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int QR>
cudaError_t launch_tree_d(const TreeArgs& a, cudaStream_t s) {
    using C = TreeCfg<D, QR>;
    const TreePlan pl = tree_plan(a.rows, a.nodes, a.hq, a.hkv, a.win, a.ring);
    TreeParams t{};
    const int G = a.hq / a.hkv;
    const int64_t ktok = static_cast<int64_t>(a.hkv) * D, krow = ktok * a.ring;
    constexpr int KB = C::KB;
    t.qn = a.nodes < pl.npt ? a.nodes : pl.npt;
    const bool whole = G * t.qn == QR;       // a tile's rows fill a block of the Q buffer: one copy for all blocks
    if (!encode_5d(&t.tq, a.q, D, a.hq, a.nodes, a.rows, a.q_tok, a.q_row, true, G, t.qn, whole ? KB : 1) ||
        !encode_5d(&t.tk, a.k, D, a.hkv, a.ring, a.rows, ktok, krow, false, kTile, 2, 1) ||
        !encode_5d(&t.tv, a.v, D, a.hkv, a.ring, a.rows, ktok, krow, false, C::VKEYS, KB, 1) ||
        !encode_5d(&t.tkp, a.k, D, a.hkv, a.ring, a.rows, ktok, krow, false, kPiece, 1, 1) ||
        !encode_5d(&t.tvp, a.v, D, a.hkv, a.ring, a.rows, ktok, krow, false, kPiece, 1, 1) ||
        !encode_5d(&t.tkt, a.kt, D, a.hkv, a.nodes, a.rows, a.kt_tok, a.kt_row, false, kTile, 2, 1) ||
        !encode_5d(&t.tvt, a.vt, D, a.hkv, a.nodes, a.rows, a.vt_tok, a.vt_row, false, C::VKEYS, KB, 1))
        return cudaErrorInvalidValue;
    t.k = static_cast<const uint16_t*>(a.k);
    t.v = static_cast<const uint16_t*>(a.v);
    t.part_l = static_cast<float4*>(a.part);
    t.part_o = t.part_l + pl.units * pl.lanes;
    t.part_m = reinterpret_cast<float*>(t.part_o + pl.units * pl.lanes * (D / 4));
    t.status = &a.hdr->status;
    t.next_unit = &a.hdr->next_unit;
    t.pairs = &a.hdr->pairs;
    int* list = reinterpret_cast<int*>(t.part_m + pl.units * pl.lanes);
    t.list = list;
    t.rows = a.rows; t.nodes = a.nodes; t.hq = a.hq; t.hkv = a.hkv; t.gsz = G; t.npt = pl.npt; t.mtiles = pl.mtiles;
    t.spans = pl.spans; t.lanes = pl.lanes; t.win = a.win; t.ring = a.ring;
    t.shared_kv = pl.mtiles > 1;
    t.neg = a.scale < 0.f ? 1 : 0;
    t.c = (a.scale < 0.f ? -a.scale : a.scale) * 1.4426950408889634f;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return cudaErrorInvalidValue;
    const int grid = static_cast<int>(pl.units < sms ? pl.units : sms);
    tree_plan_kernel<<<1, 1024, 0, s>>>(a.pos, a.parent, a.n, a.rows, a.nodes, a.hq, a.win, a.ring, a.hdr, list);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // each kernel is launched while the one before it runs, sets itself up and waits for it on the GPU
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kTreeThreads);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, tree_kernel<D, QR>, t);
    if (e != cudaSuccess) return e;
    const int quarters = pl.lanes / 32;
    cfg.gridDim = dim3(a.rows, a.hkv, pl.mtiles * quarters * (D / 64));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, tree_merge_kernel<D>, const_cast<const float4*>(t.part_o), const_cast<const float4*>(t.part_l),
                           const_cast<const float*>(t.part_m), a, pl.npt, pl.mtiles, pl.spans, pl.lanes, G,
                           (65536 + quarters - 1) / quarters, (65536 + G - 1) / G);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

template <int D, int QR>
cudaError_t tree_attr() {
    return cudaFuncSetAttribute(tree_kernel<D, QR>, cudaFuncAttributeMaxDynamicSharedMemorySize, TreeCfg<D, QR>::SMEM);
}

}  // namespace

TreePlan tree_plan(int rows, int nodes, int hq, int hkv, int win, int ring) {
    TreePlan pl{};
    const int G = hq / hkv;
    pl.npt = 128 / G;
    pl.mtiles = (nodes + pl.npt - 1) / pl.npt;
    pl.lanes = ((nodes < pl.npt ? nodes : pl.npt) * G + 31) / 32 * 32;
    pl.spans = 1;
    if (win > 0) {
        pl.spans = tree_spans(kTreeMaxPos, win, hq);       // any position with the whole window
    } else {
        for (int len = kSpanMinLinear; len <= kSpanMax; len *= 2) {
            // the most keys with this span
            int64_t keys = len == kSpanMax ? ring : (2LL * kSpanLinear * len + hq - 1) / hq - 1;
            keys = keys < ring ? keys : ring;
            const int spans = tree_cut(static_cast<int>((keys + kTile - 1) / kTile) + 1, keys, win, hq);
            pl.spans = spans > pl.spans ? spans : pl.spans;
        }
    }
    pl.units = static_cast<int64_t>(rows) * hkv * pl.mtiles * pl.spans;
    return pl;
}

cudaError_t tree_prepare_device(int) {
    cudaError_t e;
    if ((e = tree_attr<128, 128>()) != cudaSuccess) return e;
    if ((e = tree_attr<256, 64>()) != cudaSuccess) return e;
    return tree_attr<256, 128>();
}

cudaError_t launch_tree(const TreeArgs& a, cudaStream_t s) {
    if (a.d == 128) return launch_tree_d<128, 128>(a, s);
    return tree_plan(a.rows, a.nodes, a.hq, a.hkv, a.win, a.ring).lanes <= 64 ? launch_tree_d<256, 64>(a, s)
                                                                              : launch_tree_d<256, 128>(a, s);
}

}  // namespace wa
