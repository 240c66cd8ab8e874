// wa_tree_commit.cu — the kept nodes' keys and values into the rings of several layers.
//
// Node path[r, j] of row r goes to slot (pos[r] + 1 + j) mod ring, j < length[r]: a copy of hkv * d bf16 values a
// (layer, K or V, row, j), bound by latency for one sequence (the row's numbers, then its path, then the data) and
// by HBM for many.  A block takes kNodes nodes of one (layer, K or V, row), so the numbers are fetched once for
// them; its warps divide among the nodes, so that slots and addresses are computed once a warp and not for every 16
// bytes, which bound it before (12 layers of 48 rows, 8 heads of 256: 12.1 us, 15.1 with a division a piece, 16.5
// with a block a node; one row and layer 3.2 us; graph replays, 13.7 and 5.2 us called from Python).  Where length
// exceeds the ring, the nodes that a later one would overwrite are left out, so no two blocks write one slot.
//
// The status word is written by block 0 alone, which looks through every row's numbers, so that a call is one
// launch; for calls of more than kOneBlockEntries entries it is cleared before, and each block reports its own.
#include <cuda_runtime.h>

#include "wa_internal.h"

namespace wa {

namespace {

constexpr int kNodes = 16;
constexpr int kCommitThreads = 512;
constexpr int64_t kOneBlockEntries = 32768;

// What is wrong with row r's length and position.
__device__ __forceinline__ int row_faults(const CommitArgs& a, int r) {
    const int raw = a.length[r];
    return (raw < 0 || raw > a.most ? WA_STATUS_BAD_TREE : 0) | (a.pos[r] < -1 ? WA_STATUS_BAD_POS : 0);
}

__global__ void __launch_bounds__(kCommitThreads, 4) commit_kernel(const __grid_constant__ CommitArgs a, int groups, int one_block) {
    const int r = blockIdx.x / groups, j0 = blockIdx.x % groups * kNodes;
    const int l = blockIdx.y, kv = blockIdx.z, t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const bool first = blockIdx.x == 0 && l == 0 && kv == 0;
    const int32_t* path = a.path + static_cast<int64_t>(r) * a.most + j0;
    const int entry = lane < kNodes && j0 + lane < a.most ? path[lane] : -1;
    const int p = a.pos[r], len = min(max(a.length[r], 0), a.most);
    const int count = min(kNodes, len - j0);
    if (p >= -1 && count > 0) {
        // 16 warps: 16, 8, 4, 2 or 1 a node
        const int sh = count > 8 ? 0 : count > 4 ? 1 : count > 2 ? 2 : count > 1 ? 3 : 4;
        const int i = warp >> sh, j = j0 + i, node = __shfl_sync(0xFFFFFFFFu, entry, i), ring = a.ring[l];
        if (i < count && node >= 0 && node < a.nodes && j >= len - ring) {
            const int pieces = a.hkv * a.d / 8, step = 32 << sh;        // of 16 bytes
            const uint32_t slot = (static_cast<uint32_t>(p) + 1u + static_cast<uint32_t>(j)) % static_cast<uint32_t>(ring);
            const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.src[kv][l]) + r * a.row[kv] + node * a.tok[kv]);
            uint4* dst = reinterpret_cast<uint4*>(a.dst[kv][l]) + (static_cast<int64_t>(r) * ring + slot) * pieces;
            for (int c = (warp & ((1 << sh) - 1)) * 32 + lane; c < pieces; c += 4 * step) {
                uint4 v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c + e * step < pieces) v[e] = src[c + e * step];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c + e * step < pieces) dst[c + e * step] = v[e];
            }
        }
    }
    if (one_block ? !first : l != 0 || kv != 0) return;
    // the status: of every entry, or of this block's
    int bad = 0;
    if (one_block) {
        for (int i = t; i < a.rows; i += kCommitThreads) bad |= row_faults(a, i);
        for (int64_t i = t; i < static_cast<int64_t>(a.rows) * a.most; i += kCommitThreads) {
            const int row = static_cast<int>(i / a.most), j = static_cast<int>(i % a.most), node = a.path[i];
            if (a.pos[row] >= -1 && j < a.length[row] && (node < 0 || node >= a.nodes)) bad |= WA_STATUS_BAD_TREE;
        }
        const int tree = __syncthreads_or(bad & WA_STATUS_BAD_TREE), pos = __syncthreads_or(bad & WA_STATUS_BAD_POS);
        if (t == 0) a.hdr->status = (tree ? WA_STATUS_BAD_TREE : 0) | (pos ? WA_STATUS_BAD_POS : 0);
    } else {
        if (t == 0 && j0 == 0) bad = row_faults(a, r);
        if (p >= -1 && t < count && (entry < 0 || entry >= a.nodes)) bad |= WA_STATUS_BAD_TREE;
        if (bad) atomicOr(&a.hdr->status, bad);
    }
}

}  // namespace

cudaError_t launch_commit(const CommitArgs& a, cudaStream_t s) {
    const int groups = (a.most + kNodes - 1) / kNodes;
    const bool one_block = static_cast<int64_t>(a.rows) * a.most <= kOneBlockEntries;
    if (!one_block) {
        const cudaError_t e = cudaMemsetAsync(a.hdr, 0, kHeaderBytes, s);
        if (e != cudaSuccess) return e;
    }
    const dim3 grid(static_cast<unsigned>(a.rows) * groups, a.layers, 2);
    commit_kernel<<<grid, kCommitThreads, 0, s>>>(a, groups, one_block ? 1 : 0);
    return cudaGetLastError();
}

}  // namespace wa
