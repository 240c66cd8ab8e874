// wa_paged.cu — decode over a cache in pages: one new token a sequence, on the tensor cores.
//
//   o = vs sum_j w_j v_j / sum_j w_j,  w_j = 2^(c q.k_j - m),  c = scale ks log2(e)
//
// over the row's visible keys, for the G query heads of a key head together, so K and V
// are read once.
//
// Turned round.  With one token a row there are at most 16 query heads a key head, and a product with the queries as the
// 128 rows of the tensor core would be 7/8 padding.  So the keys are the rows: S^T = K Q^T (128 keys x 16) and O^T = V^T P^T
// (128 dims x the parts of P).  Both A operands are then the cache's own tiles as the copies leave them, both B operands
// small; P's parts are columns of one product, so V is read from shared memory once for all of them.  A key is a lane of
// tensor memory, so a mask is one bit a thread, and the scores of a whole span (16 columns a tile) stay there: its keys come
// first, then its maximum is known, then its values.  Nothing is ever scaled again.  (With a running maximum every other
// tile of 8-bit pages moved some head's, since P has to fit its type: 309 us for the 8-bit batch below, then 199 without.)
//
// 8-bit pages.  A query, of 8 significant bits, is two 8-bit numbers, and S comes from exact products as with bf16.  Up to 8
// heads: 2^k q = hi + lo / 32, both e4m3 (4 significant bits), columns of their own, with the head's largest value at 128 to 256:
// exactly down to 2^-14 of that value and to 2^-22 of it below.  16 heads have no columns left for lo, so the two products add
// up and lo has to reach further down by itself: hi is e5m2 (3 bits, so what is left takes 4), lo e4m3, the largest at 2^11 to
// 2^12: exactly down to 2^-13 of it and to 2^-21 below.  (As e4m3 numbers hi + lo, exactly down to 2^-9 only: outputs 0.7 off
// where one value of a head is 4,096 times the others.  16 heads as three e5m2 numbers: 64 us for 61.)  P is three e4m3 numbers:
// 256 p = p1 + p2 / 32 + p3 / 1024 to 2^-14 of p (two: 2^-9, about what the output's own rounding loses), or to 2^-28 of the
// largest where that is more.
//
// Split.  A row's tiles of 128 keys, from its first visible one (rounded down to a copy's keys), are cut into even spans
// (row_cut).  A unit of work is (row, key head, span); it leaves (m, l, O) in fp32, and a kernel of its own joins a row's
// spans.  (Joined by the CTA that finished a row's last unit, one long row ended, then, in 60 us of one SM reading what the
// others had left.)  Nothing in a unit depends on the other rows, so neither do the bits.
//
// paged_kernel<D, F8, GP>: a persistent grid, one CTA an SM, 512 threads, that streams the keys of its units without a break
// between units:
//   warps 0, 3    TMA producers of K and of V, a ring of slots each, a copy a page (or piece of one) and 128 dims.  (One warp
//                 for both took 900 cycles a load, where one of 8-bit pages lands every 700: then 199 us, 182 with two.)
//   warps 1, 13   MMA issuers of S (a unit ahead of its P V, at most two) and of P V.  Before O += V^T P^T of a row's first
//                 and last tile the second zeroes V's slots without a visible key, so that what they hold never meets a
//                 zero probability as 0 * inf.  (One warp for both took 1,000 cycles a tile, where one of 8-bit pages lands
//                 every 1,400: then 186 us, 170 with two.)  Warp 1 allocates tensor memory.
//   warp 2        takes units, looks up their pages, publishes them
//   warps 12, 14  Q to shared memory, split in two for 8-bit pages, once for units of one (row, key head) in a row: every
//                 other one each; of 16 heads, they and warp 15 four heads each of all
//   warps 4..7    softmax of even units, a key a thread: the maximum, exponentials, P to shared memory, the unit's result;
//   and 8..11     of odd units.  One group's chain (a unit's ends, 2,500 cycles) runs beside the other's.
// Every wait is bounded (a status bit after kWaitLimitNs).
//
// Times here and beside the constants are of replayed graphs of calls on one workspace, from one run of the present code but
// where a comment says "then".  Bound by HBM for batches: 64 rows of 100 to 16,000 keys, 32/8 heads of 128 ("the batch"), 315 us for
// 311 at the rate of a copy; 48 rows, 32/16 heads of 256, window 1,024 ("the window"), 126 for 117; one row of 131,072 keys, 32/4
// heads of 128, 49 for 40 (start and join); 8-bit pages, 64 rows of 500 to 30,000 keys ("the 8-bit batch"), 163 for 148; 7 rows of 0 to
// 40,000, 24/2 heads of 256 ("the ragged one"), 37 for 21 (the softmax warps' chain, few units an SM).  One row of 700 keys, 16/8
// heads of 256: 9.1 (two kernels' trips to memory).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "wa_f64.cuh"
#include "wa_prompt_kernel.cuh"

namespace wa {

namespace {

constexpr int kPTile = 128;          // keys a tile
constexpr int kPThreads = 512;
// Tiles of a span at most: as many as have room for their scores twice, beside O.  (Of 4, 6 and 8: the 8-bit batch 172.5, 164.1
// and 163.0 us; one row of 131,072 keys 51.5, 50.4 and 49.2; one of 8,000, 32/8 heads, 14.9, 13.9 and 14.0.)
constexpr int kSpanTiles = 8;
// A span holds at least so many bytes of keys and values, and of 8-bit pages at least two tiles, for a unit has costs of its
// own, of which those of the softmax warps show most with 8-bit pages.  Large batches would like more, one row of a few thousand
// keys less.  (bf16 pages, 64 and 128 KiB, 32/8 heads of 128: 256 rows of 300 keys 66.6 and 65.1 us, 64 of 500 30.0 and 28.9, 4 of
// 2,000 13.6 and 13.7.  8-bit pages of 2, 3 and 4 tiles of 32 KiB, 32/4 heads of 128: one row of 2,000 keys 9.1, 9.5 and 10.3, 64 rows
// of 4,000 60.3, 54.5 and 48.9; of 1 and 2 tiles of 64 KiB, 24/2 heads of 256: 64 rows of 4,000 79.2 and 61.2.)
__host__ __device__ constexpr int fewest_bytes(int e4m3) { return e4m3 ? 98304 : 65536; }
__host__ __device__ constexpr int fewest_tiles(int d, int e4m3) {
    const int tiles = fewest_bytes(e4m3) / (2 * kPTile * d * (e4m3 ? 1 : 2)), least = e4m3 ? 2 : 1;
    return tiles > least ? tiles : least;
}
// A row is cut into this many units over its key heads, or twice as many, .., as spans of kSpanTiles allow: fewer than the
// SMs, for two thirds of them read as fast as all, and a unit has costs of its own.  Of 152, 100 and 76 the one that loses least
// where it is not the best: one row of 8,000 keys, 32/8 heads of 128, 13.7, 14.2 and 15.3 us; over 8-bit pages, 32/4 heads, 11.1, 10.4
// and 10.8; the window 130.2, 126.9 and 126.4; the ragged one 37.4, 37.3 and 37.2.
constexpr int kFill = 100;
constexpr int kPagedRows = 256;      // rows a launch, and the fewest that some kernels have room for
constexpr int kPagedFewest = 64;
constexpr int kPagedGrid = 256;      // CTAs of a launch at most
// Launches are joined together as long as their partial results are no more than this, and each by itself beyond, so that the
// workspace does not grow with the rows.  (Each by itself always: 4,096 rows of 41 keys, 8/1 heads of 128, 188 us, together
// 178; 512 rows of 300, 32/8 heads, 136 each.)
constexpr int64_t kHeldBytes = 64 << 20;
// Units go to the CTAs in turn up to kInTurn a CTA, beyond that by a counter, in jobs of about 256 KiB of units and kJobs a CTA
// at least.  (In turn up to 2 and 8 a CTA: 16 rows of 1,000 keys, 32/8 heads of 128, 20.0 and 19.2 us; always: the batch 324.5, not
// 314.5, 64 rows of 500 31.0, not 30.0.  8 jobs a CTA and 4: 64 rows of 500 32.7 and 30.0; jobs of 1 MiB: 256 rows of 300 70.6, not 66.6.)
constexpr int kInTurn = 8;
constexpr int kJobs = 4;

// How a row is cut: spans of `each` tiles, the first `more` of them of one more.  (Without runtime divisions: as two of 64
// bits and two of 32 this took 2,000 cycles, and each unit's publication waited for it.)
struct RowCut {
    int lo, k0, tiles, spans, each, more;      // lo: the first visible key; k0: the first tile's first key
};
__host__ __device__ inline int64_t row_waves(int64_t tiles, int hkv) { return (tiles * hkv + kFill * kSpanTiles - 1) / (kFill * kSpanTiles); }
// `align`: keys of a copy
__host__ __device__ inline RowCut row_cut(int p, int win, int align, int hkv, int fewest) {
    RowCut c{};
    c.lo = win > 0 && p - win + 1 > 0 ? p - win + 1 : 0;
    c.k0 = c.lo & ~(align - 1);
    if (p < 0) return c;
    c.tiles = (p - c.k0) / kPTile + 1;
    const int64_t all = static_cast<int64_t>(c.tiles) * hkv, units = kFill * row_waves(c.tiles, hkv);
    int most = 1;                              // tiles of a span at most: all / units, rounded up, or `fewest`
#pragma unroll
    for (int e = 1; e < kSpanTiles; ++e) most += e * units < all;
    most = most < fewest ? fewest : most;
    // tiles / most, rounded up: by 2^32 / most, rounded up, for up to 2^28 tiles
    constexpr uint32_t by[kSpanTiles + 1] = {0u, 0u, 0x80000000u, 0x55555556u, 0x40000000u, 0x33333334u, 0x2AAAAAABu, 0x24924925u, 0x20000000u};
    uint32_t m = 0u;
#pragma unroll
    for (int e = 2; e <= kSpanTiles; ++e) m = e == most ? by[e] : m;
    const uint64_t up = static_cast<uint64_t>(c.tiles + most - 1) * m;
    c.spans = most == 1 ? c.tiles : static_cast<int>(up >> 32);
    c.each = 0;
#pragma unroll
    for (int e = 1; e <= kSpanTiles; ++e) c.each += static_cast<int64_t>(e) * c.spans <= c.tiles;
    c.more = c.tiles - c.each * c.spans;
    return c;
}

// Keys of one copy: a page, of at most one tile.
__host__ __device__ inline int copy_keys(int page_log) { return page_log >= 7 ? kPTile : 1 << page_log; }

// A row's last position as every kernel uses it.
__device__ __forceinline__ int paged_pos(int raw, int most, int page_log) {
    return raw < -1 ? -1 : (raw >> page_log) >= most ? (most << page_log) - 1 : raw;
}

__device__ __forceinline__ float e4m3_to_f32(uint8_t b) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(b, __NV_E4M3);
    return __half2float(__half(h));
}

// A stored value as fp32 (exact).
__device__ __forceinline__ float stored(const void* base, int64_t at, int e4m3) {
    return e4m3 ? e4m3_to_f32(static_cast<const uint8_t*>(base)[at])
                : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(base)[at]) << 16);
}

// How a copy names the keys of a page: dimensions (128 bytes, 8 keys, blocks of 128 bytes, key groups, heads) where pages
// are apart by a whole number of 8 positions (`by_slots`), and otherwise (.., key groups of a page, heads of all pages).
struct PageCoord {
    int ratio, none, by_slots;     // none: a key group that is past the end (read as zeros)
};

struct PagedParams {
    CUtensorMap map[2];
    PageCoord at[2];
    PagedArgs a;
    int* next_unit;                // null: units go to the CTAs in turn
    int* said;                     // [CTA]: its WA_STATUS_* bits
    int* cut;                      // [row]: its spans, for the join
    float* m;                      // [unit of the rows from held0 on][G]
    float* l;                      // [unit][G][4]: of each quarter of a tile's keys
    float* part;                   // [unit][G][d]
    int row0, rows;                // the launch's rows
    int held0;                     // the first row whose partial results are held
    int spans;                     // most spans of a (row, key head)
    int align;                     // keys of a copy
    float c;                       // |scale| log2(e) (bf16 pages)
};

template <int D_, bool F8_, int GP_>
struct PagedCfg {
    static constexpr int D = D_, GP = GP_;               // GP: query heads a key head, rounded up to 4, 8 or 16
    static constexpr bool F8 = F8_;
    static constexpr int ESZ = F8 ? 1 : 2;
    static constexpr int HV = D / 128;                   // loads a tile and operand: 128 keys x 128 dims each,
    static constexpr int UNROLL = GP == 16 ? 1 : HV;     // (the most code: see the softmax's)
    static constexpr int KB = ESZ;                       // in blocks of 128 bytes of a key,
    static constexpr int SLOT = kPTile * KB * 128;       // as [16 groups of 8 keys][KB][8][128 bytes]
    // slots of K, and of V: as many as leave room for P.  (bf16 pages, 2 and 3: one row of 8,000 keys 15.4 and 14.0 us, the batch
    // 318.5 and 314.5.  8-bit pages, 3 and 6: the batch 164.7 and 163.0, the ragged one (of 5) 37.2 and 36.6, 64 rows of 4,000 and
    // one of 8,000 the same.)
    static constexpr int NSLOT = F8 ? (D == 256 && GP == 16 ? 5 : 6) : 3;
    // rows of Q: the heads; 8-bit: their hi parts, then from lo_row() on the lo parts, which a group of up to 8 heads has as
    // columns of its own (S = column h + column 8 + h / 32) and a larger one adds by a second product
    static constexpr int QN = F8 && GP == 16 ? 32 : 16;
    __host__ __device__ static constexpr int lo_row() { return QN / 2; }
    static constexpr int Q_WARPS = GP == 16 ? 3 : 1;     // that stage a (row, key head)'s queries
    static constexpr int Q_READERS = GP == 16 ? 3 : 2;   // that look at each unit for it
    static constexpr int Q_BYTES = QN * D * ESZ;         // [D * ESZ / 128][QN / 8][8][128 bytes]
    static constexpr int PARTS = F8 ? 3 : 2;
    static constexpr int PN = (PARTS * GP + 15) / 16 * 16;
    static constexpr int P_CHUNK = PN * 128;             // 128 bytes of keys: [PN / 8][8][128 bytes]
    static constexpr int P_BYTES = ESZ * P_CHUNK;
    static constexpr int NP = 2 * NSLOT * SLOT + 2 * Q_BYTES + 4 * P_BYTES <= 220 * 1024 ? 2 : 1;   // P buffers a group that fit
    static constexpr int KSTEP = 32 / ESZ;               // keys or dims a product
    static constexpr int TMEM_COLS = 512;                // tensor memory: a group's scores, [tile][16]; its O, [HV][PN]
    __host__ __device__ static constexpr int s_col(int group) { return group * kSpanTiles * 16; }
    __host__ __device__ static constexpr int o_col(int group) { return 2 * kSpanTiles * 16 + group * HV * PN; }
    static_assert(o_col(2) <= TMEM_COLS, "tensor memory budget");
    static constexpr int ROWS = D == 256 && !F8 && GP == 16 ? 64 : kPagedRows;   // rows a launch
    static_assert(ROWS >= kPagedFewest, "counters");
    static constexpr int UNITS = ROWS == kPagedRows ? 8 : 4;  // unit slots
    static constexpr int FEWEST = fewest_tiles(D, F8);
    static constexpr int JOB_TILES = 262144 / (2 * kPTile * D * ESZ);   // tiles of K and V in 256 KiB
    static constexpr int PAGES = kSpanTiles * kPTile / 16;   // copies of a unit at most
    static constexpr int OFF_RING = 0;
    static constexpr int OFF_Q = OFF_RING + 2 * NSLOT * SLOT;
    static constexpr int OFF_P = OFF_Q + 2 * Q_BYTES;        // [group][NP]
    static constexpr int OFF_UNIT = OFF_P + 2 * NP * P_BYTES;    // 8 ints a slot
    static constexpr int OFF_PAGES = OFF_UNIT + UNITS * 32;
    static constexpr int OFF_PRE = OFF_PAGES + UNITS * PAGES * 4;   // units of the rows before
    static constexpr int OFF_LAST = OFF_PRE + (ROWS + 4) * 4;        // last positions
    static constexpr int OFF_EACH = OFF_LAST + ROWS * 4;              // tiles of a row's spans, a byte each
    static constexpr int OFF_X = OFF_EACH + ROWS;                     // [group][4 warps][16] maxima
    static constexpr int OFF_C = OFF_X + 512;                // [n mod UNITS][16] c of each head (8-bit)
    static constexpr int OFF_BAR = OFF_C + (F8 ? UNITS * 64 : 0);
    static constexpr int B_FULL = 0;                         // [K, V][NSLOT]
    static constexpr int B_FREE = B_FULL + 2 * NSLOT;
    static constexpr int B_SFULL = B_FREE + 2 * NSLOT;           // [group]: all scores of the unit
    static constexpr int B_PFULL = B_SFULL + 2;              // [group][NP]
    static constexpr int B_PVDONE = B_PFULL + 2 * NP;
    static constexpr int B_SFREE = B_PVDONE + 2 * NP;        // [group]: the unit's scores have been read
    static constexpr int B_QFULL = B_SFREE + 2;              // [n & 1]
    static constexpr int B_QFREE = B_QFULL + 2;
    static constexpr int B_UFULL = B_QFREE + 2;              // [unit mod UNITS] from here
    static constexpr int B_UFREE = B_UFULL + UNITS;
    static constexpr int B_UTOOK = B_UFREE + UNITS;        // the producer has begun the unit
    static constexpr int B_UC = B_UTOOK + UNITS;           // [n mod UNITS]: c are there (8-bit)
    static constexpr int B_DRAIN = B_UC + UNITS;
    static constexpr int NBAR = B_DRAIN + 2;                 // [S, P V]
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;      // tensor-memory base
    static constexpr int SMEM = OFF_MISC + 16;
    static_assert(SMEM <= 232448, "shared memory budget");
    static_assert(NBAR <= 128, "warps 4..7 set up the barriers");
};

constexpr uint32_t desc_hi(uint32_t sbo) { return (sbo >> 4) | (1u << 14) | (2u << 29); }   // version 1, 128-byte swizzle
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return ((saddr >> 4) & 0x3FFFu) | ((lbo >> 4) << 16); }

// One tcgen05.mma, descriptors as two halves of which only the low one (the address) changes.
template <bool F8, uint32_t A_HI, uint32_t B_HI>
__device__ __forceinline__ void paged_mma(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool more) {
    if constexpr (F8)
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tmov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %6};\n\t"
            "setp.ne.u32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, p;\n\t}"
            :: "r"(d), "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(more ? 1u : 0u), "n"(A_HI), "n"(B_HI));
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tmov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %6};\n\t"
            "setp.ne.u32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}"
            :: "r"(d), "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(more ? 1u : 0u), "n"(A_HI), "n"(B_HI));
}

// Instruction descriptor: fp32 accumulator, bf16 or e4m3 operands, or B in e5m2; B K-major.
constexpr uint32_t paged_idesc(bool f8, uint32_t n, uint32_t a_mn, bool b_e5m2 = false) {
    return (1u << 4) | (f8 ? (b_e5m2 ? 1u << 10 : 0u) : (1u << 7) | (1u << 10)) | (a_mn << 15) | ((n >> 3) << 17) | ((128u >> 4) << 24);
}

__device__ __forceinline__ bool paged_elect() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// N consecutive columns of the thread's own lane.
template <int N>
__device__ __forceinline__ void tm_load(uint32_t taddr, uint32_t (&r)[N]) {
    static_assert(N == 4 || N == 8, "columns");
    if constexpr (N == 4)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(taddr));
    else
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(taddr));
}
// The wait, with the registers passed through it, so that no use of them is scheduled before the data has arrived.
template <int N>
__device__ __forceinline__ void tm_wait(uint32_t (&r)[N]) {
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < N; ++e) asm volatile("" : "+r"(r[e]));
}
__device__ __forceinline__ void st_shared_u8(uint32_t addr, uint32_t v) { asm volatile("st.shared.u8 [%0], %1;" :: "r"(addr), "r"(v) : "memory"); }
__device__ __forceinline__ void st_shared_u16(uint32_t addr, uint32_t v) {
    asm volatile("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tst.shared.b16 [%0], h;\n\t}" :: "r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_shared_u32(uint32_t addr, uint32_t v) { asm volatile("st.shared.u32 [%0], %1;" :: "r"(addr), "r"(v) : "memory"); }

__device__ __forceinline__ float4 ld_shared_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// A softmax group's barrier, alone and as a vote.
__device__ __forceinline__ void group_sync(int group) { named_bar_sync(1 + group, 128); }
__device__ __forceinline__ bool group_any(int group, bool x) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r) : "r"(x ? 1u : 0u), "r"(1 + group) : "memory");
    return r != 0;
}

// Each of N values over the warp's lanes, by halves: lane l keeps N / 2 of them and hands on the others, and so on (for
// 16 values 16 shuffles instead of 80).  Returns value l / (32 / N) in lane l.
template <int N, class F>
__device__ __forceinline__ float reduce_each(float (&x)[N], F op) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int n = N / 2, o = 16; n >= 1; n >>= 1, o >>= 1) {
        const bool upper = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float keep = upper ? x[n + i] : x[i], give = upper ? x[i] : x[n + i];
            x[i] = op(keep, __shfl_xor_sync(0xFFFFFFFFu, give, o));
        }
    }
#pragma unroll
    for (int o = 16 / N; o >= 1; o >>= 1) x[0] = op(x[0], __shfl_xor_sync(0xFFFFFFFFu, x[0], o));
    return x[0];
}

__device__ __forceinline__ uint32_t e4m3_pair(float a, float b) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 e4m3_pair_f32(uint32_t v) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v), __NV_E4M3);
    return __half22float2(__half2(h));
}

__device__ __forceinline__ uint32_t e5m2_pair(float a, float b) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E5M2);
}
__device__ __forceinline__ float2 e5m2_pair_f32(uint32_t v) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v), __NV_E5M2);
    return __half22float2(__half2(h));
}

// warp_wait in less code (see the softmax's).
__device__ __forceinline__ bool paged_wait(uint32_t bar, uint32_t parity, int* status) {
    bool ok = mbar_try(bar, parity);
    if (!__all_sync(0xFFFFFFFFu, ok)) {
        const uint64_t t0 = globaltimer();
#pragma unroll 1
        while (!(ok = mbar_try(bar, parity)) && globaltimer() - t0 <= kWaitLimitNs) {}
        if (!ok) atomicOr(status, WA_STATUS_TIMEOUT);
        ok = __all_sync(0xFFFFFFFFu, ok);
    }
    return ok;
}

// Clears what a call counts; the next kernel sets itself up meanwhile.
__global__ void __launch_bounds__(1024) paged_clear_kernel(int* taken, int n) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (static_cast<int>(threadIdx.x) < n) taken[threadIdx.x] = 0;
}
static_assert(65535 / kPagedFewest < 1024, "a counter a thread");

// A published unit.  nt = 0 marks the end; n counts the (row, key head)s so far, whose queries are staged one after another.
struct PUnit {
    int row, g, span, k0, nt, lo, p, n;
};

template <int D, bool F8, int GP>
__global__ void __launch_bounds__(kPThreads, 1) paged_kernel(const __grid_constant__ PagedParams p) {
    using C = PagedCfg<D, F8, GP>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    int* const status = p.said + blockIdx.x;
    if (sbase & 1023u) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (threadIdx.x == 0) *status = WA_STATUS_LAYOUT;
        return;
    }
    const uint32_t bar0 = sbase + C::OFF_BAR;
    auto BAR = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
    auto SLOT = [&](int s) { return sbase + C::OFF_RING + static_cast<uint32_t>(s) * C::SLOT; };      // V's after K's
    int* pre = reinterpret_cast<int*>(smem + C::OFF_PRE);
    int* lasts = reinterpret_cast<int*>(smem + C::OFF_LAST);
    volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC);
    const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
    const int G = p.a.hq / p.a.hkv;

    // ---- set-up: barriers, tensor memory, zeros of Q and P, the units of each row
    if (tid >= 128 && tid < 128 + C::NBAR) {
        const int i = tid - 128;
        int count = 1;
        if (i >= C::B_PFULL && i < C::B_PVDONE) count = 4;                    // a group's softmax warps
        else if (i >= C::B_SFREE && i < C::B_QFULL) count = 4;
        else if (i >= C::B_UFREE && i < C::B_UTOOK) count = 8 + C::Q_READERS;       // producers, MMA, Q, softmax warps
        else if (i >= C::B_QFULL && i < C::B_QFREE) count = C::Q_WARPS;
        else if (i >= C::B_UC && i < C::B_DRAIN) count = C::Q_WARPS;
        mbar_init(BAR(i), count);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(smem + C::OFF_MISC), C::TMEM_COLS);
        tmem_relinquish();
    }
    for (int e = tid; e < (2 * C::Q_BYTES + 2 * C::NP * C::P_BYTES) / 16; e += kPThreads)
        st_shared_v4(sbase + C::OFF_Q + 16 * e, 0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
    // nothing before this line reads or writes what a kernel before this one may be at
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");    // the join waits for this kernel's end by itself
    int bad = 0, tiles = 0;
    static_assert(C::ROWS <= kPThreads, "a row a thread");
    {
        int mine = 0;
        if (tid < p.rows) {
            const int raw = p.a.pos[p.row0 + tid], at = paged_pos(raw, p.a.most, p.a.page_log);
            bad = raw != at;
            const RowCut cut = row_cut(at, p.a.win, p.align, p.a.hkv, C::FEWEST);
            mine = cut.spans;
            tiles = min(cut.tiles, 1 << 20);
            if (blockIdx.x == 0) p.cut[p.row0 + tid] = cut.spans;
            lasts[tid] = at;
            smem[C::OFF_EACH + tid] = static_cast<uint8_t>(cut.each);
        }
        tiles = __reduce_add_sync(0xFFFFFFFFu, tiles);
        int sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if (lane >= o) sum += y;
        }
        int* tot = reinterpret_cast<int*>(smem + C::OFF_X);
        if (lane == 31) {
            tot[warp] = sum;
            tot[16 + warp] = tiles;
        }
        bad = __syncthreads_or(bad);
        if (tid == 0) *status = bad && blockIdx.x == 0 ? WA_STATUS_BAD_POS : 0;
        tiles = 0;
#pragma unroll
        for (int w = 0; w < C::ROWS / 32; ++w) {      // (the warps that have rows)
            if (w < warp) sum += tot[w];
            tiles += tot[16 + w];
        }
        if (tid < C::ROWS) pre[tid + 1] = sum;
        if (tid == 0) pre[0] = 0;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = misc[0];

    auto unit_ints = [&](int U) { return reinterpret_cast<volatile int*>(smem + C::OFF_UNIT + (U % C::UNITS) * 32); };
    auto unit_pages = [&](int U) { return reinterpret_cast<volatile int*>(smem + C::OFF_PAGES + (U % C::UNITS) * C::PAGES * 4); };
    auto uph = [](int U) { return static_cast<uint32_t>(U / C::UNITS) & 1u; };
    auto read_unit = [&](int U, PUnit& x) {
        volatile int* e = unit_ints(U);
        x.row = e[0]; x.g = e[1]; x.span = e[2]; x.k0 = e[3]; x.nt = e[4]; x.lo = e[5]; x.p = e[6]; x.n = e[7];
    };
    const int pieces = kPTile / p.align;          // copies a tile

    if (warp == 0 || warp == 3) {
        // ------------------------------------------------ TMA producers: K, V
        const int side = warp == 0 ? 0 : 1;
        const PageCoord at = p.at[side];
        const CUtensorMap* map = &p.map[side];
        if (lane == 0) prefetch_tensormap(map);
        const uint64_t pol = policy_evict_first();
        const int in_page = (1 << p.a.page_log) - 1;
        static_assert(C::PAGES <= 64, "two copies of a unit a lane");
        int c3[2], c4[2];                         // where the unit's copies `lane` and `lane` + 32 start
        bool want[2];
        auto look_up = [&](int U, const PUnit& x) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = lane + 32 * e, id = i < x.nt * pieces ? unit_pages(U)[i] : -2;
                const int group = ((x.k0 + i * p.align) & in_page) >> 3;
                want[e] = id != -2;
                c3[e] = id < 0 ? at.none : at.by_slots ? id * at.ratio + group : group;
                c4[e] = id < 0 || at.by_slots ? x.g : id * at.ratio + x.g;
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(BAR(C::B_UFREE + U % C::UNITS));
                if (side == 0) mbar_arrive(BAR(C::B_UTOOK + U % C::UNITS));
            }
        };
        int s = 0, use = 0, loads = 0;            // the next load's slot
        // tile idx of the unit: lane j copies its j-th piece, of each 128 dims
        auto load = [&](int idx) -> bool {
            const int first = idx * pieces, hi = first >> 5, from = (first & 31) + lane;
            const int x3 = __shfl_sync(0xFFFFFFFFu, hi ? c3[1] : c3[0], from), x4 = __shfl_sync(0xFFFFFFFFu, hi ? c4[1] : c4[0], from);
            const uint32_t wanted = (__ballot_sync(0xFFFFFFFFu, hi ? want[1] : want[0]) >> (first & 31)) & ((1u << pieces) - 1u);
            const uint32_t bytes = __popc(wanted) * p.align * C::KB * 128;
#pragma unroll(C::UNROLL)
            for (int half = 0; half < C::HV; ++half) {
                const int at_s = side * C::NSLOT + s;
                if (use > 0 && !paged_wait(BAR(C::B_FREE + at_s), (use - 1) & 1, status)) return false;
                // (a copy may land before the barrier is told how much to expect: its one arrival is still to come)
                if (lane == 0) mbar_arrive_expect_tx(BAR(C::B_FULL + at_s), bytes);
                if ((wanted >> lane) & 1u)
                    tma_load_5d(SLOT(at_s) + lane * p.align * C::KB * 128, map, 0, 0, half * C::KB, x3, x4, BAR(C::B_FULL + at_s), pol);
                __syncwarp();
                ++loads;
                if (++s == C::NSLOT) {
                    s = 0;
                    ++use;
                }
            }
            return true;
        };
        PUnit x;
#pragma unroll 1
        for (int U = 0;; ++U) {
            if (!paged_wait(BAR(C::B_UFULL + U % C::UNITS), uph(U), status)) break;
            read_unit(U, x);
            if (x.nt <= 0) break;
            look_up(U, x);
            bool ok = true;
#pragma unroll 1
            for (int i = 0; ok && i < x.nt; ++i) ok = load(i);
            if (!ok) break;
        }
        // the copies in flight land before the block exits, whichever role stopped early
#pragma unroll 1
        for (int i = max(0, loads - C::NSLOT); i < loads; ++i)
            if (!mbar_wait(BAR(C::B_FULL + side * C::NSLOT + i % C::NSLOT), static_cast<uint32_t>(i / C::NSLOT) & 1u, status)) break;
    } else if (warp == 1 || warp == 13) {
        // ------------------------------------------------ MMA issuers of S and of P V: the warp together, one lane's instructions
        const uint32_t tb = __shfl_sync(0xFFFFFFFFu, tbase, 0);
        const bool leader = paged_elect();
        constexpr uint32_t idS[2] = {paged_idesc(F8, 16, 0, GP == 16), paged_idesc(F8, 16, 0)}, idO = paged_idesc(F8, C::PN, 1);
        constexpr uint32_t kTileHi = desc_hi(C::KB * 1024), kSmallHi = desc_hi(1024);
        int s = warp == 1 ? 0 : C::NSLOT, use = 0;     // the next load's slot
        const int end = s + C::NSLOT;
        auto next_slot = [&]() {
            if (++s == end) {
                s -= C::NSLOT;
                ++use;
            }
        };
        PUnit x;
        auto take = [&](int U) -> bool {
            if (!paged_wait(BAR(C::B_UFULL + U % C::UNITS), uph(U), status)) return false;
            read_unit(U, x);
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(C::B_UFREE + U % C::UNITS));
            x.nt = __shfl_sync(0xFFFFFFFFu, x.nt, 0);
            x.n = __shfl_sync(0xFFFFFFFFu, x.n, 0);
            return x.nt > 0;
        };
        if (warp == 1) {
            // S^T = K Q^T
            bool ok = true;
            int n = 0;
            for (int U = 0; ok && take(U); ++U) {
                if (x.n != n) {                   // the queries before are done with
                    if (leader) mma_commit(BAR(C::B_QFREE + (n & 1)));
                    __syncwarp();
                    n = x.n;
                }
                // the group's last scores have been read, this unit's queries are there
                if (U >= 2 && !paged_wait(BAR(C::B_SFREE + (U & 1)), static_cast<uint32_t>((U >> 1) - 1) & 1u, status)) break;
                if (!paged_wait(BAR(C::B_QFULL + (n & 1)), static_cast<uint32_t>(n >> 1) & 1u, status)) break;
                tc_fence_after();
                const uint32_t q0 = desc_lo(sbase + C::OFF_Q + (n & 1) * C::Q_BYTES, 16);
#pragma unroll 1
                for (int idx = 0; ok && idx < x.nt; ++idx) {
                    const uint32_t d = tb + C::s_col(U & 1) + idx * 16;
#pragma unroll(C::UNROLL)
                    for (int half = 0; half < C::HV; ++half) {
                        if (!(ok = paged_wait(BAR(C::B_FULL + s), use & 1, status))) break;
                        if (leader) {
                            const uint32_t k = desc_lo(SLOT(s), 16), q = q0 + ((half * C::KB * C::QN * 128) >> 4);
#pragma unroll
                            for (int set = 0; set < C::QN / 16; ++set)
#pragma unroll
                                for (int i = 0; i < 128 / C::KSTEP; ++i) {
                                    const uint32_t a = k + (((i / 4) * 1024 + (i % 4) * 32) >> 4);
                                    const uint32_t b = q + (((i / 4) * C::QN * 128 + set * 2048 + (i % 4) * 32) >> 4);
                                    paged_mma<F8, kTileHi, kSmallHi>(d, a, b, idS[set], half > 0 || set > 0 || i > 0);
                                }
                            mma_commit(BAR(C::B_FREE + s));
                        }
                        __syncwarp();
                        next_slot();
                    }
                }
                if (ok && leader) mma_commit(BAR(C::B_SFULL + (U & 1)));
                __syncwarp();
            }
        } else {
            // O^T += V^T P^T
            bool ok = true;
            int tp[2] = {0, 0};                   // tiles of each group so far
            for (int U = 0; ok && take(U); ++U) {
                const int group = U & 1;
                int tg = group ? tp[1] : tp[0];
#pragma unroll 1
                for (int idx = 0; ok && idx < x.nt; ++idx, ++tg) {
                    const int buf = group * C::NP + tg % C::NP;
                    // keys from .. to - 1 of the tile are visible
                    const int key0 = x.k0 + idx * kPTile, from = max(0, x.lo - key0), to = min(kPTile, x.p - key0 + 1);
#pragma unroll(C::UNROLL)
                    for (int half = 0; half < C::HV; ++half) {
                        if (!(ok = paged_wait(BAR(C::B_FULL + s), use & 1, status))) break;
                        if (from > 0 || to < kPTile) {
                            const int nz = from + kPTile - to;
#pragma unroll 1
                            for (int e = lane; e < nz * C::KB * 8; e += 32) {
                                const int zr = e / (C::KB * 8), rem = e % (C::KB * 8), key = zr < from ? zr : to + (zr - from);
                                st_shared_v4(SLOT(s) + (key >> 3) * (C::KB * 1024) + (rem >> 3) * 1024 + (key & 7) * 128 + (rem & 7) * 16, 0u, 0u, 0u, 0u);
                            }
                            fence_proxy_async_smem();
                            __syncwarp();
                        }
                        if (half == 0) {
                            if (!(ok = paged_wait(BAR(C::B_PFULL + buf), static_cast<uint32_t>(tg / C::NP) & 1u, status))) break;
                            tc_fence_after();
                        }
                        if (leader) {
                            const uint32_t v = desc_lo(SLOT(s), F8 ? 16 : 1024), pp = desc_lo(sbase + C::OFF_P + buf * C::P_BYTES, 16);
                            const uint32_t d = tb + C::o_col(group) + half * C::PN;
#pragma unroll
                            for (int i = 0; i < kPTile / C::KSTEP; ++i) {
                                const uint32_t a = v + ((i * (C::KSTEP / 8) * C::KB * 1024) >> 4), b = pp + (((i / 4) * C::P_CHUNK + (i % 4) * 32) >> 4);
                                paged_mma<F8, kTileHi, kSmallHi>(d, a, b, idO, i > 0 || idx > 0);
                            }
                            mma_commit(BAR(C::B_FREE + s));
                            if (half == C::HV - 1) mma_commit(BAR(C::B_PVDONE + buf));
                        }
                        __syncwarp();
                        next_slot();
                    }
                }
                if (group) tp[1] = tg; else tp[0] = tg;
            }
        }
        // every product issued has finished before tensor memory can be released
        if (leader) {
            const int drain = C::B_DRAIN + (warp == 1 ? 0 : 1);
            mma_commit(BAR(drain));
            mbar_wait(BAR(drain), 0, status);
        }
        __syncwarp();
    } else if (warp == 2) {
        // ------------------------------------------------ units
        // In turn, or in jobs that a counter gives out.  A unit's pages are asked for once the producer has
        // begun the unit before: no earlier, so that the last units go to whoever is free.
        const int units = pre[p.rows] * p.a.hkv;
        const int ctas = static_cast<int>(gridDim.x);
        const bool in_turn = !p.next_unit || units <= kInTurn * ctas;
        int job = 1;
        if (!in_turn) {
            const float of_tiles = static_cast<float>(C::JOB_TILES) * static_cast<float>(pre[p.rows]) / static_cast<float>(max(tiles, 1));
            job = max(1, min(min(16, units / (kJobs * ctas)), static_cast<int>(of_tiles)));
        }
        // A row's units are numbered span by span of each key head where they come in jobs, so that a job's queries are often
        // those of the unit before and are not staged again (64 rows of 2,000 keys, 32/8 heads of 128, 88 us, then 85; of 4,000,
        // 24/2 heads of 256, 8-bit pages, 74, then 67), and otherwise key head by key head of each span.
        int k = 0, in_job = 0, row = -1, s = 0, g = 0;       // span s of the row, key head g
        int last = 0, lo = 0, k00 = 0, each = 0, more = 0, first = 0, spans = 0;
        bool moved = true;                                    // s and g are not those of k
        PUnit cur;
        int id[2];                                // the unit's pages `lane` and `lane` + 32
        static_assert(C::PAGES <= 64, "two pages a lane");
        auto look_up = [&]() {
            PUnit& x = cur;
            x.nt = 0;
            if (k >= units) return;
            if (static_cast<uint32_t>(k - first) >= static_cast<uint32_t>(spans * p.a.hkv)) {
                int a = row + 1, b = p.rows;          // pre[row] hkv <= k < pre[row + 1] hkv
                if (row < 0 || k < first || k >= pre[row + 2] * p.a.hkv) {
                    a = 0;
#pragma unroll 1
                    while (b - a > 1) {
                        const int m = (a + b) >> 1;
                        if (pre[m] * p.a.hkv <= k) a = m; else b = m;
                    }
                }
                row = a;
                first = pre[row] * p.a.hkv;
                spans = pre[row + 1] - pre[row];
                last = lasts[row];
                lo = p.a.win > 0 ? max(0, last - p.a.win + 1) : 0;
                k00 = lo & ~(p.align - 1);
                each = smem[C::OFF_EACH + row];
                more = (last - k00) / kPTile + 1 - each * spans;
                moved = true;
            }
            if (moved) {
                const uint32_t at = k - first;
                if (in_turn) {
                    s = at / static_cast<uint32_t>(p.a.hkv);
                    g = at - s * p.a.hkv;
                } else {
                    g = at / static_cast<uint32_t>(spans);
                    s = at - g * spans;
                }
                moved = false;
            }
            x.n += x.row != p.row0 + row || x.g != g;
            x.row = p.row0 + row;
            x.g = g;
            x.p = last;
            x.lo = lo;
            x.span = s;
            x.nt = each + (x.span < more ? 1 : 0);
            x.k0 = k00 + (x.span * each + min(x.span, more)) * kPTile;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = lane + 32 * e, key = x.k0 + i * p.align;
                id[e] = -2;                      // without a visible key: nothing is copied
                if (i < x.nt * pieces && key <= last && key + p.align > lo) id[e] = max(-1, p.a.table[x.row * p.a.table_row + (key >> p.a.page_log)]);
            }
        };
        auto step = [&]() {                       // the next unit's number
            if (in_turn) {
                k += ctas;
                moved = true;
            } else if (++in_job < job) {
                ++k;
                if (++s == spans) {
                    s = 0;
                    ++g;
                }
            } else {
                int asked = 0;
                if (lane == 0) asked = atomicAdd(p.next_unit, 1);
                k = (__shfl_sync(0xFFFFFFFFu, asked, 0) + ctas) * job;
                moved = true;
                in_job = 0;
            }
        };
        k = static_cast<int>(blockIdx.x) * (in_turn ? 1 : job);
        cur.row = cur.g = cur.n = -1;
        bool ended = false;
#pragma unroll 1
        for (int U = 0;; ++U) {
            look_up();
            // the slot's last unit has been read by everyone
            if (U >= C::UNITS && !paged_wait(BAR(C::B_UFREE + U % C::UNITS), uph(U - C::UNITS), status)) break;
            if (cur.nt > 0) {
                volatile int* ids = unit_pages(U);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (lane + 32 * e >= cur.nt * pieces) continue;
                    if (id[e] != -2 && (id[e] < 0 || id[e] >= p.a.pages)) {
                        id[e] = -1;
                        atomicOr(status, WA_STATUS_BAD_PAGE);
                    }
                    ids[lane + 32 * e] = id[e];
                }
            }
            if (lane == 0) {
                volatile int* x = unit_ints(U);
                x[0] = cur.row; x[1] = cur.g; x[2] = cur.span; x[3] = cur.k0; x[4] = cur.nt; x[5] = cur.lo; x[6] = cur.p; x[7] = cur.n;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(C::B_UFULL + U % C::UNITS));
            if (cur.nt == 0) {
                if (ended) break;                 // an end for each softmax group
                ended = true;
                continue;
            }
            if (!paged_wait(BAR(C::B_UTOOK + U % C::UNITS), uph(U), status)) break;
            step();
        }
    } else if (warp >= 12) {
        // ------------------------------------------------ Q: four heads at a time, in a loop, which a unit -1 of no heads
        // goes through first: its code comes in while nothing else is asked of the memory.  (All heads' code in a row, 16
        // heads split in two, came line by line behind the first keys: 6 us to the first product.)
        constexpr int EL = D / 32;                // values a lane and head
        // up to 8 heads: a warp every other (row, key head); 16: three warps all
        constexpr bool ALL = C::Q_WARPS > 1;
        const int turn = ALL && warp > 12 ? warp - 13 : 0;
        const int mine = warp == 12 ? 0 : 1;      // of what this warp stages, unless ALL
        PUnit x;
        x.row = x.g = 0;
        int n = -1;
        for (int U = -1; ALL || warp != 15; ++U) {
            int live = 0;                         // heads (the buffer's other rows: zeros)
            if (U >= 0) {
                if (!paged_wait(BAR(C::B_UFULL + U % C::UNITS), uph(U), status)) break;
                read_unit(U, x);
                if (x.nt <= 0) break;
                x.n = __shfl_sync(0xFFFFFFFFu, x.n, 0);
                if (x.n == n || (!ALL && (x.n & 1) != mine)) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(BAR(C::B_UFREE + U % C::UNITS));
                    continue;
                }
                n = x.n;
                live = G;
            }
            const int at_q = U < 0 ? mine : n;
            const uint16_t* q = static_cast<const uint16_t*>(p.a.q) + x.row * p.a.q_row + static_cast<int64_t>(x.g) * G * D + lane * EL;
            uint32_t raw[4][EL / 2];
            auto fetch = [&](int h0) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
#pragma unroll
                    for (int e = 0; e < EL / 2; ++e) raw[i][e] = 0u;
                    if (h0 + i < live) {
                        if constexpr (EL == 4) {
                            const uint2 v = *reinterpret_cast<const uint2*>(q + (h0 + i) * D);
                            raw[i][0] = v.x; raw[i][1] = v.y;
                        } else {
                            const uint4 v = *reinterpret_cast<const uint4*>(q + (h0 + i) * D);
                            raw[i][0] = v.x; raw[i][1] = v.y; raw[i][2] = v.z; raw[i][3] = v.w;
                        }
                    }
                }
            };
            fetch(4 * turn);
            float c = p.a.scale * 1.4426950408889634f;
            if constexpr (F8) c *= p.a.kv[0].scale ? p.a.kv[0].scale[x.g] : 1.f;
            const bool neg = c < 0.f;             // the sign goes into Q, exactly
            // the scores by the buffer's last queries have been worked out
            if (U >= 0 && n >= 2 && !paged_wait(BAR(C::B_QFREE + (n & 1)), static_cast<uint32_t>((n >> 1) - 1) & 1u, status)) break;
            const uint32_t dst = sbase + C::OFF_Q + (at_q & 1) * C::Q_BYTES;
#pragma unroll 1
            for (int h0 = 4 * turn; h0 < GP; h0 += 4 * C::Q_WARPS) {
                uint32_t now[4][EL / 2];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < EL / 2; ++e) now[i][e] = raw[i][e];
                if (h0 + 4 * C::Q_WARPS < GP) fetch(h0 + 4 * C::Q_WARPS);
                if constexpr (!F8) {
                    // dims lane * EL ..: block of 64 dims, 16-byte chunk, swizzled by the row
                    const int el = lane * EL, chunk = (el & 63) * 2;
                    const uint32_t flip = neg ? 0x80008000u : 0u;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int h = h0 + i;
                        const uint32_t at = dst + (el >> 6) * (C::QN * 128) + (h >> 3) * 1024 + (h & 7) * 128 + (chunk ^ ((h & 7) << 4));
#pragma unroll
                        for (int e = 0; e < EL / 2; ++e) st_shared_u32(at + 4 * e, now[i][e] ^ flip);
                    }
                } else {
                    // the largest value of each head (as bits: infinities and NaN are larger than any other)
                    float top[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t b = 0;
#pragma unroll
                        for (int e = 0; e < EL / 2; ++e) b = max(b, max((now[i][e] << 16) & 0x7FFFFFFFu, now[i][e] & 0x7FFF0000u));
                        top[i] = __uint_as_float(b);
                    }
                    const float most = reduce_each(top, [](float a, float b) {
                        return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b)));
                    });
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t bits = __float_as_uint(__shfl_sync(0xFFFFFFFFu, most, 8 * i));
                        // 2^k brings the largest value to [2^TOP, 2^(TOP + 1)) (k at most 120: what is smaller than 2^-113 loses bits)
                        constexpr int TOP = GP == 16 ? 11 : 7;
                        const int h = h0 + i, k = min(127 + TOP - static_cast<int>(bits >> 23), 120);
                        const float f = __int_as_float((k + 127) << 23) * (neg ? -1.f : 1.f);
                        const bool fine = bits < 0x7F800000u;
                        const int el = lane * EL, low = h + C::lo_row();
                        const uint32_t block = dst + (el >> 7) * (C::QN * 128);
                        const uint32_t ah = block + (h >> 3) * 1024 + (h & 7) * 128 + ((el & 127) ^ ((h & 7) << 4));
                        const uint32_t al = block + (low >> 3) * 1024 + (low & 7) * 128 + ((el & 127) ^ ((low & 7) << 4));
#pragma unroll
                        for (int w = 0; w < EL / 4; ++w) {
                            float v[4];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                v[2 * e] = __uint_as_float(now[i][2 * w + e] << 16) * f;
                                v[2 * e + 1] = __uint_as_float(now[i][2 * w + e] & 0xFFFF0000u) * f;
                            }
                            uint32_t a, b;
                            float2 fa, fb;
                            if constexpr (GP == 16) {
                                a = e5m2_pair(v[0], v[1]); b = e5m2_pair(v[2], v[3]);
                                fa = e5m2_pair_f32(a); fb = e5m2_pair_f32(b);
                            } else {
                                a = e4m3_pair(v[0], v[1]); b = e4m3_pair(v[2], v[3]);
                                fa = e4m3_pair_f32(a); fb = e4m3_pair_f32(b);
                            }
                            constexpr float UP = GP == 16 ? 1.f : 32.f;
                            const uint32_t rest = e4m3_pair((v[0] - fa.x) * UP, (v[1] - fa.y) * UP) |
                                                  (e4m3_pair((v[2] - fb.x) * UP, (v[3] - fb.y) * UP) << 16);
                            st_shared_u32(ah + 4 * w, fine ? a | (b << 16) : 0x7F7F7F7Fu);      // NaN: the head is computed again
                            st_shared_u32(al + 4 * w, fine ? rest : 0u);
                        }
                        if (lane == i)
                            reinterpret_cast<volatile float*>(smem + C::OFF_C)[(at_q & (C::UNITS - 1)) * 16 + h] = fabsf(c) * __int_as_float((127 - k) << 23);
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && U >= 0) {
                mbar_arrive(BAR(C::B_QFULL + (n & 1)));
                if constexpr (F8) mbar_arrive(BAR(C::B_UC + n % C::UNITS));
                mbar_arrive(BAR(C::B_UFREE + U % C::UNITS));
            }
            __syncwarp();
        }
    } else {
        // ------------------------------------------------ softmax: key `quarter` * 32 + lane of a tile
        const int quarter = warp & 3, group = (warp >> 2) - 1, gt = tid & 127;
        const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
        volatile float* xbuf = reinterpret_cast<volatile float*>(smem + C::OFF_X) + group * 64;
        const uint32_t x_addr = sbase + C::OFF_X + group * 256;
        constexpr float kShift = F8 ? 8.f : 0.f;         // P is 2^kShift times the weight, in l and O alike
        // Sixteen heads go through the code of eight twice, with their values exchanged in between: the warps' roles are more
        // code than the instruction cache holds, and waited for it (64 rows of 4,000 keys, 24/2 heads of 256, 8-bit pages, 66 us,
        // then 60; one such row 12.7, then 13.2).
        constexpr int H = GP == 16 ? 8 : GP, TURNS = GP / H;
        auto turn = [](float (&x)[GP]) {
#pragma unroll
            for (int h = 0; h < GP / 2; ++h) {
                if constexpr (TURNS == 2) {
                    const float y = x[h];
                    x[h] = x[h + H];
                    x[h + H] = y;
                }
            }
        };
        // A wait that runs out does not take a warp from the others' barriers: it carries on without waiting until the
        // next vote, at which the four warps leave together.
        bool dead = false;
        auto wait = [&](int bar, uint32_t ph) {
            if (!dead && !paged_wait(BAR(bar), ph, status)) dead = true;
        };
        const uint32_t pk = quarter * 32 + lane;         // this thread's key: its column of P
        const uint32_t s_addr = tbase + lane_addr + C::s_col(group);
        const uint32_t o_addr = tbase + lane_addr + C::o_col(group);
        int t = 0;                                       // the group's tiles
#pragma unroll 1
        for (int U = group;; U += 2) {
            PUnit x;
            wait(C::B_UFULL + U % C::UNITS, uph(U));
            read_unit(U, x);
            float c[GP];
            if constexpr (F8) {
                if (!dead && x.nt > 0) wait(C::B_UC + x.n % C::UNITS, uph(x.n));
#pragma unroll
                for (int h = 0; h < GP; ++h)
                    c[h] = h < G ? reinterpret_cast<volatile float*>(smem + C::OFF_C)[(x.n % C::UNITS) * 16 + h] : 0.f;
            } else {
                c[0] = p.c;                     // (of every head)
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(C::B_UFREE + U % C::UNITS));
            if (group_any(group, dead) || x.nt <= 0) break;
            wait(C::B_SFULL + group, static_cast<uint32_t>(U >> 1) & 1u);
            tc_fence_after();
            // a tile's products q.k of this thread's key and heads from h0 on
            auto scores = [&](int idx, int h0, float (&y)[H]) {
                if constexpr (F8 && GP < 16) {
                    uint32_t r[H], q[H];
                    tm_load(s_addr + idx * 16, r);
                    tm_load(s_addr + idx * 16 + C::lo_row(), q);
                    tm_wait(r);
                    tm_wait(q);
#pragma unroll
                    for (int h = 0; h < H; ++h) y[h] = fmaf(__uint_as_float(q[h]), 0.03125f, __uint_as_float(r[h]));
                } else {
                    uint32_t r[H];
                    tm_load(s_addr + idx * 16 + h0, r);
                    tm_wait(r);
#pragma unroll
                    for (int h = 0; h < H; ++h) y[h] = __uint_as_float(r[h]);
                }
            };
            auto visible = [&](int idx) {
                const int key = x.k0 + idx * kPTile + static_cast<int>(pk);
                return key >= x.lo && key <= x.p;
            };
            // ---- the largest product of each head over the unit (-inf where there is none: not finite then, worked out again).
            // It is taken from the others before they are multiplied by c, so that its own weight is 1 whatever its size: c q.k
            // less the rounded c of the largest would be up to half a step of those away from zero, and e4m3 holds no 2^9.
            float m[GP], l[GP];
#pragma unroll
            for (int h = 0; h < GP; ++h) l[h] = 0.f;
#pragma unroll 1
            for (int h0 = 0; h0 < GP; h0 += H) {
                float best[H];
#pragma unroll
                for (int h = 0; h < H; ++h) best[h] = -INFINITY;
#pragma unroll 1
                for (int idx = 0; idx < x.nt; ++idx) {
                    float y[H];
                    scores(idx, h0, y);
                    if (visible(idx)) {
#pragma unroll
                        for (int h = 0; h < H; ++h) best[h] = fmaxf(best[h], y[h]);
                    }
                }
                const float top = reduce_each(best, [](float a, float b) { return fmaxf(a, b); });
                if (lane % (32 / H) == 0) xbuf[quarter * 16 + h0 + lane / (32 / H)] = top;
            }
            group_sync(group);
#pragma unroll
            for (int h = 0; h < GP; h += 4) {
                float4 e[4];
#pragma unroll
                for (int w = 0; w < 4; ++w) e[w] = ld_shared_f4(x_addr + (16 * w + h) * 4);
                m[h] = fmaxf(fmaxf(e[0].x, e[1].x), fmaxf(e[2].x, e[3].x));
                m[h + 1] = fmaxf(fmaxf(e[0].y, e[1].y), fmaxf(e[2].y, e[3].y));
                m[h + 2] = fmaxf(fmaxf(e[0].z, e[1].z), fmaxf(e[2].z, e[3].z));
                m[h + 3] = fmaxf(fmaxf(e[0].w, e[1].w), fmaxf(e[2].w, e[3].w));
            }
            // ---- P, tile by tile
#pragma unroll 1
            for (int idx = 0; idx < x.nt; ++idx, ++t) {
                const bool vis = visible(idx);
                const int buf = group * C::NP + t % C::NP;
                const uint32_t pb = sbase + C::OFF_P + buf * C::P_BYTES;
#pragma unroll 1
                for (int h0 = 0; h0 < GP; h0 += H) {
                    float s[H];
                    scores(idx, h0, s);
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        s[h] = vis ? ex2(fmaf(s[h] - m[h], c[F8 ? h : 0], kShift)) : 0.f;
                        l[h] += s[h];
                    }
                    // the parts of two heads each
                    uint32_t part[H / 2][C::PARTS];
#pragma unroll
                    for (int h = 0; h < H; h += 2) {
                        if constexpr (F8) {
                            float a = s[h], b = s[h + 1];
#pragma unroll
                            for (int i = 0; i < 3; ++i) {
                                const uint32_t e = part[h / 2][i] = e4m3_pair(a, b);
                                if (i < 2) {
                                    const float2 f = e4m3_pair_f32(e);
                                    a = (a - f.x) * 32.f;
                                    b = (b - f.y) * 32.f;
                                }
                            }
                        } else {
                            const uint32_t hi = part[h / 2][0] = pack_bf16(s[h], s[h + 1]);
                            part[h / 2][1] = pack_bf16(s[h] - __uint_as_float(hi << 16), s[h + 1] - __uint_as_float(hi & 0xFFFF0000u));
                        }
                    }
                    // the buffer's last product is done
                    if (h0 == 0 && t >= C::NP) wait(C::B_PVDONE + buf, static_cast<uint32_t>(t / C::NP - 1) & 1u);
                    // row n of P^T (part * GP + head), key pk: 128-byte rows, swizzled by the row (h0 is 0 or whole groups of 8 rows)
                    const uint32_t pr = pb + (h0 >> 3) * 1024;
                    auto at = [&](int n) {
                        if constexpr (F8) return pr + (n >> 3) * 1024 + (n & 7) * 128 + (pk ^ ((n & 7) << 4));
                        else return pr + (pk >> 6) * C::P_CHUNK + (n >> 3) * 1024 + (n & 7) * 128 + (((pk & 63) * 2) ^ ((n & 7) << 4));
                    };
#pragma unroll
                    for (int h = 0; h < H; h += 2)
#pragma unroll
                        for (int i = 0; i < C::PARTS; ++i) {
                            const uint32_t v = part[h / 2][i];
                            if constexpr (F8) {
                                st_shared_u8(at(i * GP + h), v);
                                st_shared_u8(at(i * GP + h + 1), v >> 8);
                            } else {
                                st_shared_u16(at(i * GP + h), v);
                                st_shared_u16(at(i * GP + h + 1), v >> 16);
                            }
                        }
                    turn(m);
                    turn(l);
                    if constexpr (F8) turn(c);
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(BAR(C::B_PFULL + buf));
                    if (idx == x.nt - 1) mbar_arrive(BAR(C::B_SFREE + group));
                }
            }
            // ---- the unit's result: l of this quarter of the keys in a fixed order, O from tensor memory
            const int64_t unit = ((static_cast<int64_t>(x.row - p.held0) * p.a.hkv + x.g) * p.spans + x.span) * G;
            const float sum = reduce_each(l, [](float a, float b) { return a + b; });
            if (lane % (32 / GP) == 0 && lane / (32 / GP) < G) p.l[(unit + lane / (32 / GP)) * 4 + quarter] = sum;
            if (gt < G) {
                float mine = 0.f;
#pragma unroll
                for (int h = 0; h < GP; ++h)
                    if (gt == h) mine = m[h] * c[F8 ? h : 0];
                p.m[unit + gt] = mine;
            }
            {
                const int buf = group * C::NP + (t - 1) % C::NP;
                wait(C::B_PVDONE + buf, static_cast<uint32_t>((t - 1) / C::NP) & 1u);
            }
            tc_fence_after();
#pragma unroll(C::UNROLL)
            for (int mb = 0; mb < C::HV; ++mb) {
                float* dst = p.part + unit * D + mb * 128 + quarter * 32 + lane;
#pragma unroll 1
                for (int h0 = 0; h0 < G; h0 += H) {
                    uint32_t r[C::PARTS][H];
#pragma unroll
                    for (int part = 0; part < C::PARTS; ++part) tm_load(o_addr + mb * C::PN + part * GP + h0, r[part]);
#pragma unroll
                    for (int part = 0; part < C::PARTS; ++part) tm_wait(r[part]);
                    float o[H];
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        o[h] = __uint_as_float(r[C::PARTS - 1][h]);
#pragma unroll
                        for (int part = C::PARTS - 2; part >= 0; --part) o[h] = fmaf(o[h], F8 ? 0.03125f : 1.f, __uint_as_float(r[part][h]));
                    }
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        if (h0 + h >= G) break;
                        dst[(h0 + h) * D] = o[h];
                    }
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tbase, C::TMEM_COLS);
}

// The float64 value of 64 of a (row, head)'s dims (from col0), by the whole block: the maximum score, then weights and their sums in key order,
// 256 keys at a time; a NaN or +inf score settles the output before that.  (Without one: 2.0 ms for 4,000 keys of 128 dims, 181 ms
// for 131,072: the block's own chain.)
struct PagedRerun {
    double qd[256], wb[kRerunThreads], red[kRerunThreads / 32];
    float qf[256];
    int64_t vat[kRerunThreads];
};

__device__ __noinline__ void paged_rerun(const PagedArgs& a, PagedRerun& sm, int row, int h, int col0) {
    const int t = threadIdx.x, d = a.d, g = h / (a.hq / a.hkv);
    const int p = paged_pos(a.pos[row], a.most, a.page_log), lo = a.win > 0 ? max(0, p - a.win + 1) : 0;
    uint16_t* orow = static_cast<uint16_t*>(a.out) + row * a.o_row + static_cast<int64_t>(h) * d + col0;
    const double scale = static_cast<double>(a.scale) * (a.kv[0].scale ? static_cast<double>(a.kv[0].scale[g]) : 1.0);
    if (t < d) {
        sm.qd[t] = bf16_bits_to_f64(static_cast<const uint16_t*>(a.q)[row * a.q_row + static_cast<int64_t>(h) * d + t]);
        sm.qf[t] = static_cast<float>(sm.qd[t]) * static_cast<float>(scale);     // only the score's class matters
    }
    __syncthreads();
    // where key j's head starts in k or v; -1 in a page that is none
    auto at = [&](const PageSide& side, int j) -> int64_t {
        const int page = a.table[row * a.table_row + (j >> a.page_log)];
        if (page < 0 || page >= a.pages) return -1;
        return page * side.page + (j & ((1 << a.page_log) - 1)) * side.slot + g * side.head;
    };
    auto score = [&](int j) {
        const int64_t k = at(a.kv[0], j);
        double s = 0.0;
        for (int e = 0; e < d; ++e) s = s + sm.qd[e] * (k < 0 ? 0.0 : static_cast<double>(stored(a.kv[0].base, k + e, a.e4m3)));
        return s * scale;
    };
    // a float64 score that is NaN or +inf makes the output NaN; an fp32 one that is finite is neither
    for (int base = lo; base <= p; base += kRerunThreads) {
        const int j = base + t;
        bool hit = false;
        if (j <= p) {
            const int64_t k = at(a.kv[0], j);
            float s = 0.f;
            for (int e = 0; e < d; ++e) s = fmaf(sm.qf[e], k < 0 ? 0.f : stored(a.kv[0].base, k + e, a.e4m3), s);
            if (!isfinite(s)) {
                const double s64 = score(j);
                hit = isnan(s64) || (isinf(s64) && s64 > 0.0);
            }
        }
        if (__syncthreads_or(hit)) {
            if (t < 64) orow[t] = 0x7FC0u;
            return;
        }
    }
    double mloc = -INFINITY;
    for (int j = lo + t; j <= p; j += kRerunThreads) {
        const double s = score(j);
        mloc = (isnan(s) || isnan(mloc)) ? (s + mloc) : fmax(mloc, s);
    }
    const double M = block_reduce(mloc, true, sm.red);
    double lloc = 0.0, acc = 0.0;
    for (int base = lo; base <= p; base += kRerunThreads) {
        const int j = base + t;
        double w = 0.0;
        if (j <= p) {
            w = exp(score(j) - M);
            lloc = lloc + w;
            sm.vat[t] = at(a.kv[1], j);
        }
        sm.wb[t] = w;
        __syncthreads();
        if (t < 64) {
            const int cnt = min(kRerunThreads, p - base + 1);
            for (int jj = 0; jj < cnt; ++jj)
                acc = acc + sm.wb[jj] * (sm.vat[jj] < 0 ? 0.0 : static_cast<double>(stored(a.kv[1].base, sm.vat[jj] + col0 + t, a.e4m3)));
        }
        __syncthreads();
    }
    const double l = block_reduce(lloc, false, sm.red);
    if (t < 64) orow[t] = f64_to_bf16_rn(acc / l * (a.kv[1].scale ? static_cast<double>(a.kv[1].scale[g]) : 1.0));
}

// out = vs sum_s a_s O_s / sum_s a_s l_s, a_s = 2^(m_s - M).  Both sums run over groups of kMergeGroup spans: a group's
// in order, then the groups' in order, whichever of the two kernels below takes the row.  64 dims that hold a value that
// is not finite are worked out again.
constexpr int kMergeGroup = 4;

// The status word of the call, by the last join's first block: what the CTAs of all its launches have to report.
__device__ __forceinline__ void paged_report(WsHeader* hdr, const int* said, int ctas) {
    int bits = 0;
    for (int i = threadIdx.x; i < ctas; i += 256) bits |= said[i];
    const int bad_pos = __syncthreads_or(bits & WA_STATUS_BAD_POS), bad_page = __syncthreads_or(bits & WA_STATUS_BAD_PAGE),
              late = __syncthreads_or(bits & WA_STATUS_TIMEOUT), layout = __syncthreads_or(bits & WA_STATUS_LAYOUT);
    if (threadIdx.x == 0)
        hdr->status = (bad_pos ? WA_STATUS_BAD_POS : 0) | (bad_page ? WA_STATUS_BAD_PAGE : 0) | (late ? WA_STATUS_TIMEOUT : 0) |
                      (layout ? WA_STATUS_LAYOUT : 0);
}

struct MergeArgs {
    const float* m;
    const float4* l;
    const float* part;
    const int *said, *cut;
    int spans_most, ctas;      // ctas: to report on; 0 for a join that another one follows
    int row0, rows;            // whose partial results are held
};

// A row's spans (as many as there is room for at most, whatever is read).  Working them out from the position here, once
// more, would take 0.3 us of a short call.
__device__ __forceinline__ int spans_of(const MergeArgs& x, int row) { return max(0, min(x.cut[row], x.spans_most)); }

// (m, l) of a record, l over the quarters in order
__device__ __forceinline__ float2 record(const MergeArgs& x, int64_t at) {
    const float m = x.m[at];
    const float4 l = x.l[at];
    return make_float2(m, (l.x + l.y) + (l.z + l.w));
}

__device__ __forceinline__ void fma4(float4& x, float w, const float4& o) {
    x.x = fmaf(w, o.x, x.x);
    x.y = fmaf(w, o.y, x.y);
    x.z = fmaf(w, o.z, x.z);
    x.w = fmaf(w, o.w, x.w);
}
__device__ __forceinline__ void add4(float4& x, const float4& o) {
    x.x += o.x; x.y += o.y; x.z += o.z; x.w += o.w;
}

// Few rows: a block 64 dims of a (row, head), sixteen threads of 4 dims a group of spans.  The partial results of the first
// kWideAhead groups a thread are asked for together with their number, so a call of up to 128
// spans waits for one trip to memory.
constexpr int kWideAhead = 2;
template <int D>
__global__ void __launch_bounds__(256, 3) paged_merge_wide_kernel(const __grid_constant__ PagedArgs a, const __grid_constant__ MergeArgs x) {
    __shared__ float4 red[64][16];
    __shared__ float weight[256], sums[256], tops[8], group_den[64];
    __shared__ PagedRerun again;
    const int at = blockIdx.x / a.hq, row = x.row0 + at, h = blockIdx.x % a.hq, G = a.hq / a.hkv, g = h / G, col0 = blockIdx.y * 64;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, slice = t >> 4, quad = t & 15;
    const int64_t first = (static_cast<int64_t>(at) * a.hkv + g) * x.spans_most;
    auto rec = [&](int s) { return (first + s) * G + (h - g * G); };
    float4 ahead[kWideAhead][kMergeGroup];      // (of spans that the row does not have: whatever the workspace holds, not used)
    auto fetch = [&](int s, int most, float4 (&o)[kMergeGroup]) {
#pragma unroll
        for (int i = 0; i < kMergeGroup; ++i)
            if (s + i < most) o[i] = reinterpret_cast<const float4*>(x.part + rec(s + i) * D + col0)[quad];
    };
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // Plain loads from here on: what they read is written while this kernel is there already.  Blocks without work wait
    // too, so that nothing behind the call starts early.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int spans = spans_of(x, row);
#pragma unroll
    for (int i = 0; i < kWideAhead; ++i) fetch((16 * i + slice) * kMergeGroup, x.spans_most, ahead[i]);
    float2 mine = make_float2(-INFINITY, 0.f);
    if (t < x.spans_most) mine = record(x, rec(t));
    const float vs = a.kv[1].scale ? a.kv[1].scale[g] : 1.f;
    if (x.ctas > 0 && blockIdx.x == 0 && blockIdx.y == 0) paged_report(a.hdr, x.said, x.ctas);
    uint16_t* orow = static_cast<uint16_t*>(a.out) + row * a.o_row + static_cast<int64_t>(h) * D + col0;
    if (spans == 0) {
        if (t < 8) reinterpret_cast<uint4*>(orow)[t] = make_uint4(0u, 0u, 0u, 0u);
        return;
    }
    float M = t < spans ? mine.x : -INFINITY;
    for (int s = t + 256; s < spans; s += 256) M = fmaxf(M, x.m[rec(s)]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
    if (lane == 0) tops[warp] = M;
    __syncthreads();
    for (int w = 0; w < 8; ++w) M = fmaxf(M, tops[w]);
    float den = 0.f, o = 0.f;        // of thread t < 64: dim t
    for (int s0 = 0; s0 < spans; s0 += 256) {      // 64 groups at a time
        if (s0 + t < spans) {
            const float2 e = s0 == 0 ? mine : record(x, rec(s0 + t));
            weight[t] = exp2f(e.x - M);
            sums[t] = e.y;
        }
        __syncthreads();
        const int end = min(spans - s0, 256);
        auto group = [&](int k, const float4 (&part)[kMergeGroup]) {
            float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
            float d = 0.f;
#pragma unroll
            for (int i = 0; i < kMergeGroup; ++i) {
                const int s = k * kMergeGroup + i;
                if (s < end) {
                    fma4(num, weight[s], part[i]);
                    d = fmaf(weight[s], sums[s], d);
                }
            }
            red[k][quad] = num;
            if (quad == 0) group_den[k] = d;
        };
        int k = slice;
        if (s0 == 0) {
#pragma unroll
            for (int i = 0; i < kWideAhead; ++i, k += 16)
                if (k * kMergeGroup < end) group(k, ahead[i]);
        }
        for (; k * kMergeGroup < end; k += 16) {
            fetch(s0 + k * kMergeGroup, s0 + end, ahead[0]);
            group(k, ahead[0]);
        }
        __syncthreads();
        if (t < 64)
            for (int e = 0; e * kMergeGroup < end; ++e) {
                o += reinterpret_cast<const float*>(red[e])[t];
                den += group_den[e];
            }
        __syncthreads();
    }
    bool bad = false;
    if (t < 64) {
        o = o / den * vs;
        bad = !isfinite(o);
        orow[t] = __bfloat16_as_ushort(__float2bfloat16_rn(o));
    }
    if (__syncthreads_or(bad)) paged_rerun(a, again, row, h, col0);
}

// Many rows: a warp a (row, head), kNarrowAhead / V spans at a time.  Their number comes first here, for spans that a row does
// not have are not free when there are many rows (256 rows of 300 keys, a table for 38,400: 77 us, then 69).  (8 and 16 at
// a time: 256 rows of 300 65.9 and 66.6 us, 64 of 500 29.6 and 30.0, the 8-bit batch 163.3 and 163.0.)
constexpr int kNarrowAhead = 16;
template <int D>
__global__ void __launch_bounds__(256, 2) paged_merge_kernel(const __grid_constant__ PagedArgs a, const __grid_constant__ MergeArgs x) {
    constexpr int V = D / 128, AHEAD = kNarrowAhead / V;
    static_assert(AHEAD % kMergeGroup == 0 && 32 % AHEAD == 0, "whole groups");
    __shared__ PagedRerun again;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int item = blockIdx.x * 8 + warp, items = x.rows * a.hq;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");          // as above
    if (x.ctas > 0 && blockIdx.x == 0) paged_report(a.hdr, x.said, x.ctas);
    uint32_t bad = 0u;                          // the lane's 4 dims of each 128 that are not finite
    if (item < items) {
        const int at = item / a.hq, row = x.row0 + at, h = item % a.hq, G = a.hq / a.hkv, g = h / G;
        const int64_t first = (static_cast<int64_t>(at) * a.hkv + g) * x.spans_most;
        auto rec = [&](int s) { return (first + s) * G + (h - g * G); };
        float4 o[AHEAD][V];
        auto fetch = [&](int s, int most) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i)
                if (s + i < most) {
#pragma unroll
                    for (int v = 0; v < V; ++v) o[i][v] = reinterpret_cast<const float4*>(x.part + rec(s + i) * D)[v * 32 + lane];
                }
        };
        const int spans = spans_of(x, row);
        const float vs = a.kv[1].scale ? a.kv[1].scale[g] : 1.f;
        uint2* orow = reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * a.o_row + static_cast<int64_t>(h) * D);
        fetch(0, spans);
        float2 mine = make_float2(-INFINITY, 0.f);
        if (lane < spans) mine = record(x, rec(lane));
        float M = lane < spans ? mine.x : -INFINITY;
        for (int s = lane + 32; s < spans; s += 32) M = fmaxf(M, x.m[rec(s)]);
#pragma unroll
        for (int e = 16; e > 0; e >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, e));
        float den = 0.f, w = 0.f;
        float4 sum[V];
#pragma unroll
        for (int v = 0; v < V; ++v) sum[v] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s0 = 0; s0 < spans; s0 += AHEAD) {
            if (s0 > 0) fetch(s0, spans);
            if ((s0 & 31) == 0) {
                if (s0 > 0) mine = s0 + lane < spans ? record(x, rec(s0 + lane)) : make_float2(-INFINITY, 0.f);
                w = exp2f(mine.x - M);
            }
#pragma unroll
            for (int k = 0; k < AHEAD; k += kMergeGroup) {
                if (s0 + k >= spans) break;
                float4 num[V];
                float d = 0.f;
#pragma unroll
                for (int v = 0; v < V; ++v) num[v] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int i = k; i < k + kMergeGroup; ++i) {
                    const float wi = __shfl_sync(0xFFFFFFFFu, w, (s0 + i) & 31), li = __shfl_sync(0xFFFFFFFFu, mine.y, (s0 + i) & 31);
                    if (s0 + i < spans) {
                        d = fmaf(wi, li, d);
#pragma unroll
                        for (int v = 0; v < V; ++v) fma4(num[v], wi, o[i][v]);
                    }
                }
                den += d;
#pragma unroll
                for (int v = 0; v < V; ++v) add4(sum[v], num[v]);
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float4 r = sum[v];
            if (spans > 0) {
                r.x = r.x / den * vs; r.y = r.y / den * vs; r.z = r.z / den * vs; r.w = r.w / den * vs;
                if (!(isfinite(r.x) && isfinite(r.y) && isfinite(r.z) && isfinite(r.w))) bad |= 1u << v;
            }
            orow[v * 32 + lane] = make_uint2(pack_bf16(r.x, r.y), pack_bf16(r.z, r.w));
        }
    }
    // Of 64 dims that hold one all are computed again, and no others: what the wide kernel does.
    __shared__ uint32_t again_for[8];           // of each warp's pair, a bit for 64 dims
    uint32_t again_dims = 0u;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const uint32_t lanes = __ballot_sync(0xFFFFFFFFu, (bad >> v) & 1u);
        again_dims |= ((lanes & 0xFFFFu) != 0u ? 1u : 0u) << (2 * v) | ((lanes >> 16) != 0u ? 2u : 0u) << (2 * v);
    }
    if (lane == 0) again_for[warp] = again_dims;
    if (!__syncthreads_or(again_dims != 0u)) return;
    for (int i = 0; i < 8; ++i) {
        for (int c = 0; c < D / 64; ++c) {
            if (!((again_for[i] >> c) & 1u)) continue;
            paged_rerun(a, again, x.row0 + (blockIdx.x * 8 + i) / a.hq, (blockIdx.x * 8 + i) % a.hq, 64 * c);
            __syncthreads();
        }
    }
}

// (row, head) pairs below which the wide kernel runs.  (It, and the other one: one row of 131,072 keys, 32 heads of 128, 49.2 and
// 65.3 us, 7 ragged rows, 24 heads of 256, 36.6 and 42.9, 4 rows of 2,000, 32 heads, 13.7 and 14.1, 8 rows 19.3 and 18.7, 64 rows of
// 500 43.6 and 30.0.)
constexpr int kMergeWide = 256;

bool encode_pages(CUtensorMap* m, PageCoord* at, const PageSide& side, const PagedArgs& a, int align) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const int esz = a.e4m3 ? 1 : 2, page = 1 << a.page_log;
    const int64_t one = a.pages == 1 ? 1 : 0;          // a lone page's stride means nothing
    at->by_slots = one || side.page % (8 * side.slot) == 0;
    at->ratio = static_cast<int>(one ? 0 : at->by_slots ? side.page / (8 * side.slot) : side.page / side.head);
    const int64_t reach = static_cast<int64_t>(a.pages - 1) * at->ratio;
    const int64_t groups = page / 8 + (at->by_slots ? reach : 0), heads = a.hkv + (at->by_slots ? 0 : reach);
    at->none = static_cast<int>(groups);
    cuuint64_t dims[5] = {static_cast<cuuint64_t>(128 / esz), 8, static_cast<cuuint64_t>(a.d * esz / 128),
                          static_cast<cuuint64_t>(groups), static_cast<cuuint64_t>(heads)};
    cuuint64_t strides[4] = {static_cast<cuuint64_t>(side.slot * esz), 128, static_cast<cuuint64_t>(8 * side.slot * esz),
                             static_cast<cuuint64_t>(side.head * esz)};
    cuuint32_t box[5] = {static_cast<cuuint32_t>(128 / esz), 8, static_cast<cuuint32_t>(esz),
                         static_cast<cuuint32_t>(align / 8), 1};
    cuuint32_t es[5] = {1, 1, 1, 1, 1};
    return enc(m, a.e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, side.base, dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               a.d * esz >= 256 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class F>
cudaError_t for_each_paged(F&& f) {
    cudaError_t e;
#define WA_PAGED(D, F8, GP) \
    if ((e = f(paged_kernel<D, F8, GP>, D, F8, GP, PagedCfg<D, F8, GP>::SMEM, PagedCfg<D, F8, GP>::ROWS)) != cudaSuccess) return e
    WA_PAGED(128, false, 4); WA_PAGED(128, false, 8); WA_PAGED(128, false, 16);
    WA_PAGED(256, false, 4); WA_PAGED(256, false, 8); WA_PAGED(256, false, 16);
    WA_PAGED(128, true, 4); WA_PAGED(128, true, 8); WA_PAGED(128, true, 16);
    WA_PAGED(256, true, 4); WA_PAGED(256, true, 8); WA_PAGED(256, true, 16);
#undef WA_PAGED
    return cudaSuccess;
}

}  // namespace

PagedPlan paged_plan(int rows, int hq, int hkv, int d, int page_log, int most, int win) {
    PagedPlan pl{};
    const int align = copy_keys(page_log);
    const int64_t keys = static_cast<int64_t>(most) << page_log;
    int64_t tiles = (keys + kPTile - 1) / kPTile;
    const int64_t seen = (static_cast<int64_t>(win) + align - 2) / kPTile + 1;      // tiles of a window, wherever it begins
    if (win > 0 && seen < tiles) tiles = seen;
    // ceil(t / each) with each >= t hkv / (kFill waves(t)), and waves(t) no less for longer rows
    const int64_t fill = (kFill * row_waves(tiles, hkv) + hkv - 1) / hkv;
    pl.spans = static_cast<int>(fill < tiles ? fill : tiles);
    // a row takes hq * spans * (d + 5) floats
    const int64_t fit = kHeldBytes / (static_cast<int64_t>(hq) * pl.spans * (d + 5) * static_cast<int64_t>(sizeof(float))) / kPagedRows;
    const int64_t held = (fit > 1 ? fit : 1) * kPagedRows;
    pl.held = static_cast<int>(held < rows ? held : rows);
    const int64_t heads = static_cast<int64_t>(pl.held) * hq;
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    pl.taken = kHeaderBytes;
    pl.said = pl.taken + up((rows / kPagedFewest + 1) * sizeof(int));
    pl.cut = pl.said + up((rows / kPagedFewest + 1) * kPagedGrid * sizeof(int));
    pl.m = pl.cut + up(rows * sizeof(int));
    pl.l = pl.m + up(heads * pl.spans * sizeof(float));
    pl.part = pl.l + up(heads * pl.spans * 4 * sizeof(float));
    pl.bytes = pl.part + up(static_cast<size_t>(heads) * pl.spans * d * sizeof(float));
    return pl;
}

cudaError_t paged_prepare_device(int) {
    return for_each_paged([](auto kernel, int, bool, int, int smem, int) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
}

cudaError_t launch_paged_decode(const PagedArgs& a, cudaStream_t s) {
    const PagedPlan pl = paged_plan(a.rows, a.hq, a.hkv, a.d, a.page_log, a.most, a.win);
    const int G = a.hq / a.hkv, gp = G <= 4 ? 4 : G <= 8 ? 8 : 16;
    PagedParams p{};
    p.a = a;
    p.align = copy_keys(a.page_log);
    for (int i = 0; i < 2; ++i)
        if (!encode_pages(&p.map[i], &p.at[i], a.kv[i], a, p.align)) return cudaErrorInvalidValue;
    uint8_t* base = reinterpret_cast<uint8_t*>(a.hdr);
    int* taken = reinterpret_cast<int*>(base + pl.taken);
    int* said = reinterpret_cast<int*>(base + pl.said);
    p.cut = reinterpret_cast<int*>(base + pl.cut);
    p.m = reinterpret_cast<float*>(base + pl.m);
    p.l = reinterpret_cast<float*>(base + pl.l);
    p.part = reinterpret_cast<float*>(base + pl.part);
    p.spans = pl.spans;
    p.c = fabsf(a.scale) * 1.4426950408889634f;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return cudaErrorInvalidValue;
    // Each kernel is launched while the one before runs, sets itself up and waits for it on the GPU, the first one for
    // whatever the stream holds before.
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const int most_ctas = sms < kPagedGrid ? sms : kPagedGrid;
    // Up to kInTurn units a CTA go to them in turn, which spares the launch that clears their counter
    const bool in_turn = static_cast<int64_t>(a.rows) * a.hkv * pl.spans <= static_cast<int64_t>(kInTurn) * most_ctas;
    cudaError_t e = cudaSuccess;
    if (!in_turn) {
        cfg.gridDim = dim3(1);
        cfg.blockDim = dim3((a.rows / kPagedFewest / 32 + 1) * 32);
        e = cudaLaunchKernelEx(&cfg, paged_clear_kernel, taken, a.rows / kPagedFewest + 1);
        if (e != cudaSuccess) return e;
    }
    MergeArgs m{p.m, reinterpret_cast<const float4*>(p.l), p.part, said, p.cut, pl.spans, 0, 0, 0};
    int ctas = 0;
    e = for_each_paged([&](auto kernel, int d, bool f8, int g, int smem, int most_rows) {
        if (d != a.d || f8 != (a.e4m3 != 0) || g != gp) return cudaSuccess;
        for (int r0 = 0; r0 < a.rows; r0 += most_rows) {
            p.row0 = r0;
            p.rows = a.rows - r0 < most_rows ? a.rows - r0 : most_rows;
            p.next_unit = in_turn ? nullptr : taken + r0 / most_rows;
            p.said = said + ctas;
            const int64_t units = static_cast<int64_t>(p.rows) * a.hkv * pl.spans;
            cfg.gridDim = dim3(static_cast<unsigned>(units < most_ctas ? units : most_ctas));
            cfg.blockDim = dim3(kPThreads);
            cfg.dynamicSmemBytes = smem;
            ctas += cfg.gridDim.x;
            cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, p);
            if (err != cudaSuccess) return err;
            const bool last = r0 + p.rows == a.rows;
            m.row0 = p.held0;
            m.rows = r0 + p.rows - p.held0;
            if (!last && m.rows < pl.held) continue;
            m.ctas = last ? ctas : 0;
            p.held0 = r0 + p.rows;
            const int pairs = m.rows * a.hq;
            cfg.gridDim = pairs < kMergeWide ? dim3(pairs, a.d / 64) : dim3((pairs + 7) / 8);
            cfg.blockDim = dim3(256);
            cfg.dynamicSmemBytes = 0;
            auto merge = pairs < kMergeWide ? (a.d == 256 ? paged_merge_wide_kernel<256> : paged_merge_wide_kernel<128>)
                                            : (a.d == 256 ? paged_merge_kernel<256> : paged_merge_kernel<128>);
            err = cudaLaunchKernelEx(&cfg, merge, a, m);
            if (err != cudaSuccess) return err;
        }
        return cudaSuccess;
    });
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace wa
