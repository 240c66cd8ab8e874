// wa_internal.h — launch-side structures shared by the library's translation units.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "wa.h"

namespace wa {

constexpr int kChunk = 256;     // decode: keys per chunk, at absolute positions [256c, 256c+255]
constexpr int kHeaderBytes = 256;

// First 256 bytes of every workspace.  The per-call clear resets them.
struct WsHeader {
    int status;   // WA_STATUS_* bits
    int nflag;    // (row, head) pairs queued for the float64 re-run
    int next_unit;   // tensor-core decode, tree decode: units taken so far past the first one of each CTA
    int pairs;       // tree decode: listed (row, span) pairs
    int pad[60];
};

inline int decode_chunks_max(int win, int ring) {
    return win > 0 ? (win - 1 + kChunk - 1) / kChunk + 1 : (ring + kChunk - 1) / kChunk;
}

struct DecodeArgs {
    const void* q;
    const void* k;
    const void* v;
    const int32_t* pos;
    int rows, hq, hkv, d, win, ring;
    float scale;
    void* out;
    WsHeader* hdr;
    int* flags;      // [rows * hq]
    float* part;     // [rows, hq, cmax, d + 4]
    int cmax;
};

struct PromptArgs {
    const void* q;
    const void* k;
    const void* v;
    const int32_t* hi;   // may be null
    int p0, n, hq, hkv, d, win, ring;
    float scale;
    int p32;
    int64_t q_tok, k_tok, v_tok, o_tok;   // token strides, elements
    void* out;
    WsHeader* hdr;
    int* flags;      // [n * hq]
    const int32_t* sel;   // block-sparse form: [n, hkv, nsel] selected 64-key blocks; null otherwise
    int nsel;
};

// Attention of trees of drafted tokens over ring caches.
struct TreeArgs {
    const void* q;
    const void* k;           // ring
    const void* v;
    const void* kt;          // the nodes' keys and values
    const void* vt;
    const int32_t* pos;
    const int32_t* parent;   // [rows, nodes]
    const int32_t* n;        // may be null
    int rows, nodes, hq, hkv, d, win, ring;
    float scale;
    int64_t q_row, q_tok, kt_row, kt_tok, vt_row, vt_tok, o_row, o_tok;   // elements
    void* out;
    WsHeader* hdr;
    void* part;              // partial results: l float4[units * lanes], O float[units * lanes * d], m float[units * lanes],
                             // the list of (row, span) pairs: kTreePairBytes each, rows * spans at most
};

constexpr int kTreePairBytes = 32 + WA_TREE_MAX_NODES;

// How a tree decode call is cut: nodes a query tile, query tiles a key head, spans a row at most, query rows
// kept of a tile, units = rows * hkv * mtiles * spans.
struct TreePlan {
    int npt, mtiles, spans, lanes;
    int64_t units;
};
TreePlan tree_plan(int rows, int nodes, int hq, int hkv, int win, int ring);

// Verification of drafted tokens.
struct VerifyArgs {
    const float* target;
    const float* draft;      // may be null
    const int32_t* parent;
    const int32_t* tokens;
    const int32_t* n;        // may be null
    const float* u;
    int rows, nodes, vocab;
    int64_t t_row, t_node, d_row, d_node;
    int32_t* path;
    int32_t* length;
    int32_t* token;
    WsHeader* hdr;
};

// Keys or values of a paged cache: strides in elements.
struct PageSide {
    void* base;
    const float* scale;      // may be null
    int64_t page, slot, head;
};

// Rotary positions (hkv = 0, no cache) and append to a paged cache.
struct PagedAppendArgs {
    const void* src;
    const int32_t* pos;
    const int32_t* row;      // may be null
    const float* inv_freq;
    PageSide kv[2];
    const int32_t* table;
    int64_t src_tok, q_tok, table_row;
    void* q_out;
    WsHeader* hdr;           // null: nothing to report (wa_rope)
    int n, hq, hkv, d, dims, layout, inverse, pages, page_log, rows, most, e4m3;
    float factor;
};

// Decode over a paged cache.
struct PagedArgs {
    const void* q;
    const int32_t* pos;
    PageSide kv[2];
    const int32_t* table;
    int64_t table_row, q_row, o_row;
    void* out;
    WsHeader* hdr;
    int rows, hq, hkv, d, pages, page_log, most, e4m3, win;
    float scale;
};

// The workspace of a paged decode call in bytes from its start, and the most spans of a (row, key head).
struct PagedPlan {
    int spans;
    int held;        // rows whose partial results are held at a time: of whole launches
    size_t taken;    // int[launches] units that are taken
    size_t said;     // int[launches * CTAs] what they have to report
    size_t cut;      // int[rows] spans of a row
    size_t m;        // float[held * hkv * spans * G]
    size_t l;        // float[held * hkv * spans * G * 4]
    size_t part;     // float[held * hkv * spans * G * d]
    size_t bytes;
};
PagedPlan paged_plan(int rows, int hq, int hkv, int d, int page_log, int most, int win);

// Kept nodes' keys and values into the rings of several layers.
struct CommitArgs {
    const void* src[2][WA_COMMIT_MAX_LAYERS];   // [k, v]
    void* dst[2][WA_COMMIT_MAX_LAYERS];
    int ring[WA_COMMIT_MAX_LAYERS];
    int64_t row[2], tok[2];                     // strides of the trees, elements
    int layers, rows, nodes, hkv, d, most;
    const int32_t* path;
    const int32_t* length;
    const int32_t* pos;
    WsHeader* hdr;
};

// A node's parent as every kernel uses it: a value outside [-1, i) counts as -1.
__host__ __device__ inline int tree_parent(int raw, int i) { return raw >= -1 && raw < i ? raw : -1; }

// A row's last position as every tree kernel uses it: key indices up to a span past it stay in 32 bits.
constexpr int kTreeMaxPos = INT32_MAX - 4096;
__host__ __device__ inline int tree_pos(int raw, int win, int ring) {
    const int most = win == 0 && ring - 1 < kTreeMaxPos ? ring - 1 : kTreeMaxPos;
    return raw < -1 ? -1 : raw > most ? most : raw;
}

// Float64 re-run of every flagged (row, head); mode 0 = decode, 1 = prompt, 2 = block-sparse prompt.
struct RerunArgs {
    int mode;
    const int32_t* sel;   // mode 2: [rows, hkv, nsel] selected 64-key blocks
    int nsel;
    const void* q;
    const void* k;
    const void* v;
    const int32_t* idx;  // decode: pos; prompt: hi (may be null)
    int rows, hq, hkv, d, win, ring, p0;
    float scale;
    int64_t q_tok, k_tok, v_tok, o_tok;   // prompt token strides; decode uses dense layouts
    void* out;
    WsHeader* hdr;
    const int* flags;
};

// q/k preparation and KV append (mode WA_PREP_*).
struct PrepArgs {
    const void* src;
    const int32_t* pos;
    const float* q_scale;    // may be null
    const float* inv_freq;   // WA_PREP_L2_ROPE only
    void* q_out;
    void* k_ring;
    void* v_ring;            // may be null
    int n, hq, hkv, d, ring, mode;
    int64_t src_tok, q_tok, ring_row, slot;
    WsHeader* hdr;
};

// cuTensorMapEncodeTiled from the driver, looked up once; null if unavailable.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t s);
cudaError_t launch_prompt(const PromptArgs& a, cudaStream_t s);
cudaError_t launch_prompt_sparse(const PromptArgs& a, cudaStream_t s);
cudaError_t prompt_sparse_prepare_device(int dev);
cudaError_t launch_rerun(const RerunArgs& a, cudaStream_t s);
cudaError_t launch_prep(const PrepArgs& a, cudaStream_t s);
cudaError_t launch_tree(const TreeArgs& a, cudaStream_t s);
cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t s);
cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t s);
cudaError_t launch_paged_decode(const PagedArgs& a, cudaStream_t s);
cudaError_t launch_commit(const CommitArgs& a, cudaStream_t s);
cudaError_t tree_prepare_device(int dev);
cudaError_t paged_prepare_device(int dev);
cudaError_t prompt_prepare_device(int dev);
cudaError_t decode_prepare_device(int dev);
// Decode partials on the tensor cores (query-head groups of kTcMinGroup and more); the merge is shared.
constexpr int kTcMinGroup = 3;
cudaError_t launch_decode_tc_part(const DecodeArgs& a, cudaStream_t s);
cudaError_t decode_tc_prepare_device(int dev);
// Device address of wa_decode_static's scratch on the current device (WA_OK or a WA_E* code).
int static_ws_header(void** out);

}  // namespace wa
