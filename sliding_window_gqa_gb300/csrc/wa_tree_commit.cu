// wa_tree_commit.cu — the kept nodes' keys and values into the rings of several layers.
//
// Node path[r, j] of row r goes to slot (pos[r] + 1 + j) mod ring, j < length[r].
// A copy of hkv * d bf16 values a (layer, K or V, row, j): one block each, 16 bytes
// a thread and pass.  Where length exceeds the ring, the nodes that a later one
// would overwrite are left out, so no two blocks write one slot.
#include <cuda_runtime.h>

#include "wa_internal.h"

namespace wa {

namespace {

__global__ void __launch_bounds__(128) commit_kernel(const __grid_constant__ CommitArgs a) {
    const int r = blockIdx.x / a.most, j = blockIdx.x % a.most;
    const int l = blockIdx.y, kv = blockIdx.z;
    const int p = a.pos[r], raw = a.length[r];
    const int len = min(max(raw, 0), a.most);
    const bool first = l == 0 && kv == 0 && threadIdx.x == 0;
    if (first && j == 0) {
        if (raw != len) atomicOr(&a.hdr->status, WA_STATUS_BAD_TREE);
        if (p < -1) atomicOr(&a.hdr->status, WA_STATUS_BAD_POS);
    }
    if (p < -1 || j >= len || j < len - a.ring[l]) return;
    const int node = a.path[static_cast<int64_t>(r) * a.most + j];
    if (node < 0 || node >= a.nodes) {
        if (first) atomicOr(&a.hdr->status, WA_STATUS_BAD_TREE);
        return;
    }
    const int64_t slot = (static_cast<int64_t>(p) + 1 + j) % a.ring[l];
    const int64_t width = static_cast<int64_t>(a.hkv) * a.d;
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.src[kv][l]) + r * a.row[kv] + node * a.tok[kv]);
    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.dst[kv][l]) + (static_cast<int64_t>(r) * a.ring[l] + slot) * width);
    for (int e = threadIdx.x; e < width / 8; e += blockDim.x) dst[e] = src[e];
}

}  // namespace

cudaError_t launch_commit(const CommitArgs& a, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>(a.rows) * a.most, a.layers, 2);
    commit_kernel<<<grid, 128, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace wa
