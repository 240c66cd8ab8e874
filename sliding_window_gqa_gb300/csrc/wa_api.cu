// wa_api.cu — the C ABI: argument checks, workspace carving, launches.
//
// Entry points and their arguments follow the operator of TensorFold pull
// request #1123, section "What this changes": decode (bullet "Decode") and
// prompt rows with an optional per-row last key (bullet "promptRows(...,
// hi)"), a scale parameter and window 0 as a linear cache (bullet "Scale is
// a parameter"), and the optional two-half P (bullet "Window.p32").  The calls
// for drafted tokens (tree decode, verification, commit) build on the decode form.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>

#include <cuda_runtime.h>

#include "wa.h"
#include "wa_internal.h"

namespace {

constexpr int kMaxDevices = 64;
std::mutex g_mu;
int g_ready[kMaxDevices];   // 0 unknown, 1 ready, negative: a WA_E* code

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool heads_ok(int32_t hq, int32_t hkv) {
    return hq > 0 && hkv > 0 && hq % hkv == 0 && hq / hkv <= 16;
}

// Once per device: capability check and kernel attributes.
int ensure_device() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return WA_ECUDA;
    if (dev < 0 || dev >= kMaxDevices) return WA_EDEVICE;
    std::lock_guard<std::mutex> lock(g_mu);
    if (g_ready[dev] != 0) return g_ready[dev] > 0 ? WA_OK : g_ready[dev];
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
        return WA_ECUDA;
    if (major != 10 || minor != 3) {
        g_ready[dev] = WA_EDEVICE;
        return WA_EDEVICE;
    }
    if (wa::decode_prepare_device(dev) != cudaSuccess || wa::prompt_prepare_device(dev) != cudaSuccess ||
        wa::prompt_sparse_prepare_device(dev) != cudaSuccess || wa::tree_prepare_device(dev) != cudaSuccess ||
        wa::paged_prepare_device(dev) != cudaSuccess)
        return WA_ECUDA;
    g_ready[dev] = 1;
    return WA_OK;
}

size_t flags_bytes(int64_t units) { return round_up(static_cast<size_t>(units) * sizeof(int), 256); }

// Whether a ring is given twice with other nodes: one slot would get two values.
bool rings_contradict(const wa::CommitArgs& a, int layers) {
    const void* all[2 * WA_COMMIT_MAX_LAYERS];
    for (int i = 0; i < 2 * layers; ++i) all[i] = a.dst[i / layers][i % layers];
    std::sort(all, all + 2 * layers);
    if (std::adjacent_find(all, all + 2 * layers) == all + 2 * layers) return false;
    for (int i = 1; i < 2 * layers; ++i)
        for (int j = 0; j < i; ++j) {
            const int ki = i / layers, li = i % layers, kj = j / layers, lj = j % layers;
            if (a.dst[ki][li] == a.dst[kj][lj] &&
                (a.src[ki][li] != a.src[kj][lj] || a.ring[li] != a.ring[lj] || a.tok[ki] != a.tok[kj] || a.row[ki] != a.row[kj]))
                return true;
        }
    return false;
}

int log2_of(int32_t x) {
    int n = 0;
    while ((1 << n) < x) ++n;
    return n;
}

// Whether no two elements of [pages][page_size][hkv][d] under these strides share memory, and all 16-byte pieces of a
// head are aligned.
bool pages_apart(const wa_pages& c, int64_t page, int64_t slot, int64_t head, int64_t align) {
    if ((page | slot | head) & (align - 1)) return false;
    struct { int64_t stride, size; } dim[3] = {{page, c.pages}, {slot, c.page_size}, {head, c.hkv}};
    std::sort(dim, dim + 3, [](auto& x, auto& y) { return x.stride < y.stride; });
    int64_t extent = c.d;        // elements that the dims so far span
    for (auto& x : dim) {
        if (x.size == 1) continue;
        if (x.stride < extent || x.stride > (int64_t{1} << 38)) return false;
        extent += x.stride * (x.size - 1);
        if (extent > (int64_t{1} << 44)) return false;
    }
    return true;
}

bool page_sizes_ok(const wa_pages& c, int32_t hq, int32_t win) {
    if (c.pages <= 0 || c.rows <= 0 || c.rows > 65535 || c.most <= 0 || !heads_ok(hq, c.hkv) || c.hkv > 65535) return false;
    if (c.page_size < 16 || c.page_size > 256 || (c.page_size & (c.page_size - 1)) || (c.d != 128 && c.d != 256)) return false;
    if (c.type != WA_PAGE_BF16 && c.type != WA_PAGE_E4M3) return false;
    if (static_cast<int64_t>(c.rows) * hq > INT32_MAX) return false;
    // positions, and those of a tile past the last, stay in 32 bits
    return win >= 0 && static_cast<int64_t>(c.most) * c.page_size <= INT32_MAX - 4096;
}

bool pages_ok(const wa_pages* c, int32_t hq, int32_t win) {
    if (!c || !c->k || !c->v || !c->table || !page_sizes_ok(*c, hq, win)) return false;
    if (!aligned16(c->k) || !aligned16(c->v) || (reinterpret_cast<uintptr_t>(c->table) & 3u)) return false;
    if (c->type == WA_PAGE_BF16 && (c->k_scale || c->v_scale)) return false;
    if (c->table_row < c->most) return false;
    const int64_t align = c->type == WA_PAGE_E4M3 ? 16 : 8;
    return pages_apart(*c, c->k_page, c->k_slot, c->k_head, align) && pages_apart(*c, c->v_page, c->v_slot, c->v_head, align);
}

// The head stride as the kernels use it: a lone head's means nothing.
int64_t head_stride(const wa_pages& c, int64_t head) { return c.hkv > 1 ? head : c.d; }

// Whether the decode's copies can name a page's keys by one index: pages apart by a whole number of 8 positions, or of heads.
bool pages_in_steps(const wa_pages& c, int64_t page, int64_t slot, int64_t head) {
    const int64_t step = page % (8 * slot) == 0 ? 8 * slot : head_stride(c, head);
    return c.pages == 1 || (page % step == 0 && (c.pages - 1) * (page / step) + c.hkv + c.page_size < INT32_MAX);
}

bool rotary_ok(const wa_rotary* r, int32_t d) {
    if (!r || r->dims == 0) return true;
    return r->inv_freq && r->dims > 0 && r->dims <= d && r->dims % 16 == 0 && std::isfinite(r->factor) &&
           (r->layout == WA_ROTARY_HALF || r->layout == WA_ROTARY_INTERLEAVED);
}

void set_rotary(wa::PagedAppendArgs& a, const wa_rotary* r) {
    if (!r || r->dims == 0) return;
    a.inv_freq = r->inv_freq;
    a.dims = r->dims;
    a.layout = r->layout;
    a.factor = r->factor;
}

}  // namespace

extern "C" {

size_t wa_decode_ws_bytes(int32_t rows, int32_t hq, int32_t d, int32_t win, int32_t ring) {
    if (rows <= 0 || hq <= 0 || (d != 128 && d != 256) || win < 0 || ring <= 0 || win > ring) return 0;
    const int64_t units = static_cast<int64_t>(rows) * hq;
    const int cmax = wa::decode_chunks_max(win, ring);
    return wa::kHeaderBytes + flags_bytes(units) +
           static_cast<size_t>(units) * cmax * static_cast<size_t>(d + 4) * sizeof(float);
}

int wa_decode(const void* q, const void* k_ring, const void* v_ring, const int32_t* pos,
              int32_t rows, int32_t hq, int32_t hkv, int32_t d, int32_t win, int32_t ring,
              float scale, void* out, void* ws, size_t ws_bytes, void* stream) {
    if (!q || !k_ring || !v_ring || !pos || !out) return WA_EINVAL;
    if (rows <= 0 || rows > 65535 || !heads_ok(hq, hkv) || hkv > 65535) return WA_EINVAL;
    if (d != 128 && d != 256) return WA_EINVAL;
    if (win < 0 || ring <= 0 || win > ring) return WA_EINVAL;
    if (!std::isfinite(scale)) return WA_EINVAL;
    if (!aligned16(q) || !aligned16(k_ring) || !aligned16(v_ring) || !aligned16(out)) return WA_EINVAL;
    const size_t need = wa_decode_ws_bytes(rows, hq, d, win, ring);
    if (!ws || ws_bytes < need || (reinterpret_cast<uintptr_t>(ws) & 255u)) return WA_EWORKSPACE;
    const int rc = ensure_device();
    if (rc != WA_OK) return rc;

    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint8_t* base = static_cast<uint8_t*>(ws);
    wa::DecodeArgs a{};
    a.q = q; a.k = k_ring; a.v = v_ring; a.pos = pos;
    a.rows = rows; a.hq = hq; a.hkv = hkv; a.d = d; a.win = win; a.ring = ring; a.scale = scale;
    a.out = out;
    a.hdr = reinterpret_cast<wa::WsHeader*>(base);
    a.flags = reinterpret_cast<int*>(base + wa::kHeaderBytes);
    a.part = reinterpret_cast<float*>(base + wa::kHeaderBytes + flags_bytes(static_cast<int64_t>(rows) * hq));
    a.cmax = wa::decode_chunks_max(win, ring);
    if (cudaMemsetAsync(base, 0, wa::kHeaderBytes, s) != cudaSuccess) return WA_ECUDA;
    if (wa::launch_decode(a, s) != cudaSuccess) return WA_ECUDA;

    wa::RerunArgs r{};
    r.mode = 0; r.q = q; r.k = k_ring; r.v = v_ring; r.idx = pos;
    r.rows = rows; r.hq = hq; r.hkv = hkv; r.d = d; r.win = win; r.ring = ring; r.p0 = 0; r.scale = scale;
    r.out = out; r.hdr = a.hdr; r.flags = a.flags;
    if (wa::launch_rerun(r, s) != cudaSuccess) return WA_ECUDA;
    return WA_OK;
}

size_t wa_prompt_ws_bytes(int32_t n, int32_t hq) {
    if (n <= 0 || hq <= 0) return 0;
    return wa::kHeaderBytes + flags_bytes(static_cast<int64_t>(n) * hq);
}

}  // extern "C"

namespace {

// wa_prompt and wa_prompt_sparse: shared checks, workspace carving, launch and re-run.
int prompt_call(const void* q, const void* k, const void* v, int32_t p0, int32_t n, const int32_t* hi, int32_t hq,
                int32_t hkv, int32_t d, int32_t win, int32_t ring, float scale, int32_t p32, const int32_t* sel,
                int32_t nsel, const wa_strides* strides, void* out, void* ws, size_t ws_bytes, void* stream) {
    if (!q || !k || !v || !out) return WA_EINVAL;
    if (n <= 0 || p0 < 0 || !heads_ok(hq, hkv) || hq > 65535) return WA_EINVAL;
    if (d != 128 && d != 256) return WA_EINVAL;
    if (win < 0 || ring <= 0 || win > ring) return WA_EINVAL;
    if (p32 < 0 || p32 > 2) return WA_EINVAL;
    if (!std::isfinite(scale)) return WA_EINVAL;
    if (static_cast<int64_t>(p0) + n > INT32_MAX) return WA_EINVAL;
    const int64_t span_lo = win > 0 && p0 - win + 1 > 0 ? p0 - win + 1 : 0;
    if (win > 0) {
        if (static_cast<int64_t>(p0) + n - 1 - span_lo >= ring) return WA_EINVAL;
    } else if (static_cast<int64_t>(p0) + n > ring) {
        return WA_EINVAL;
    }
    if (sel) {
        if (nsel < 1 || nsel > WA_SPARSE_MAX_SEL) return WA_EINVAL;
        // the kernel's union bitmap covers at most 65,536 blocks of the key span
        if ((static_cast<int64_t>(p0) + n - 1) / WA_SPARSE_BLOCK - span_lo / WA_SPARSE_BLOCK + 1 > 65536)
            return WA_EINVAL;
    }
    int64_t qs = static_cast<int64_t>(hq) * d, ks = static_cast<int64_t>(hkv) * d, vs = ks, os = qs;
    if (strides) {
        if (strides->q) qs = strides->q;
        if (strides->k) ks = strides->k;
        if (strides->v) vs = strides->v;
        if (strides->out) os = strides->out;
    }
    if (qs < static_cast<int64_t>(hq) * d || ks < static_cast<int64_t>(hkv) * d || vs < static_cast<int64_t>(hkv) * d ||
        os < static_cast<int64_t>(hq) * d)
        return WA_EINVAL;
    if ((qs | ks | vs | os) & 7) return WA_EINVAL;   // 16-byte token strides (TMA)
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out)) return WA_EINVAL;
    const size_t need = wa_prompt_ws_bytes(n, hq);
    if (!ws || ws_bytes < need || (reinterpret_cast<uintptr_t>(ws) & 255u)) return WA_EWORKSPACE;
    const int rc = ensure_device();
    if (rc != WA_OK) return rc;

    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint8_t* base = static_cast<uint8_t*>(ws);
    wa::PromptArgs a{};
    a.q = q; a.k = k; a.v = v; a.hi = hi;
    a.p0 = p0; a.n = n; a.hq = hq; a.hkv = hkv; a.d = d; a.win = win; a.ring = ring; a.scale = scale; a.p32 = p32;
    a.q_tok = qs; a.k_tok = ks; a.v_tok = vs; a.o_tok = os;
    a.out = out;
    a.hdr = reinterpret_cast<wa::WsHeader*>(base);
    a.flags = reinterpret_cast<int*>(base + wa::kHeaderBytes);
    a.sel = sel;
    a.nsel = sel ? nsel : 0;
    if (cudaMemsetAsync(base, 0, wa::kHeaderBytes, s) != cudaSuccess) return WA_ECUDA;
    const cudaError_t e = sel ? wa::launch_prompt_sparse(a, s) : wa::launch_prompt(a, s);
    if (e == cudaErrorNotSupported) return WA_EINVAL;
    if (e != cudaSuccess) return WA_ECUDA;

    wa::RerunArgs r{};
    r.mode = sel ? 2 : 1; r.q = q; r.k = k; r.v = v; r.idx = hi;
    r.sel = sel; r.nsel = a.nsel;
    r.rows = n; r.hq = hq; r.hkv = hkv; r.d = d; r.win = win; r.ring = ring; r.p0 = p0; r.scale = scale;
    r.q_tok = qs; r.k_tok = ks; r.v_tok = vs; r.o_tok = os;
    r.out = out; r.hdr = a.hdr; r.flags = a.flags;
    if (wa::launch_rerun(r, s) != cudaSuccess) return WA_ECUDA;
    return WA_OK;
}

}  // namespace

extern "C" {

int wa_prompt(const void* q, const void* k, const void* v, int32_t p0, int32_t n,
              const int32_t* hi, int32_t hq, int32_t hkv, int32_t d, int32_t win, int32_t ring,
              float scale, int32_t p32, const wa_strides* strides, void* out,
              void* ws, size_t ws_bytes, void* stream) {
    return prompt_call(q, k, v, p0, n, hi, hq, hkv, d, win, ring, scale, p32, nullptr, 0, strides, out, ws, ws_bytes,
                       stream);
}

int wa_prompt_sparse(const void* q, const void* k, const void* v, int32_t p0, int32_t n,
                     const int32_t* hi, int32_t hq, int32_t hkv, int32_t d, int32_t win, int32_t ring,
                     float scale, int32_t p32, const int32_t* sel, int32_t nsel, const wa_strides* strides,
                     void* out, void* ws, size_t ws_bytes, void* stream) {
    if (!sel) return WA_EINVAL;
    return prompt_call(q, k, v, p0, n, hi, hq, hkv, d, win, ring, scale, p32, sel, nsel, strides, out, ws, ws_bytes,
                       stream);
}

int wa_prep_append(const void* src, const int32_t* pos, int32_t n, int32_t hq, int32_t hkv, int32_t d,
                   int32_t mode, const float* q_scale, const float* inv_freq, int32_t ring,
                   const wa_prep_layout* lay, void* q_out, void* k_ring, void* v_ring,
                   void* ws, size_t ws_bytes, void* stream) {
    if (!src || !pos || !lay || !q_out || !k_ring) return WA_EINVAL;
    if (n <= 0 || !heads_ok(hq, hkv) || ring <= 0) return WA_EINVAL;
    if (d != 128 && d != 256) return WA_EINVAL;
    if (mode != WA_PREP_RMSNORM && mode != WA_PREP_L2_ROPE) return WA_EINVAL;
    if (mode == WA_PREP_L2_ROPE && !inv_freq) return WA_EINVAL;
    if (!aligned16(src) || !aligned16(q_out) || !aligned16(k_ring) || (v_ring && !aligned16(v_ring))) return WA_EINVAL;
    if (lay->src_tok < (hq + 2 * hkv) * static_cast<int64_t>(d) || lay->q_tok < hq * static_cast<int64_t>(d) ||
        lay->ring_row < 0 || lay->slot < hkv * static_cast<int64_t>(d))
        return WA_EINVAL;
    if ((lay->src_tok | lay->q_tok | lay->ring_row | lay->slot) & 7) return WA_EINVAL;
    if (!ws || ws_bytes < WA_PREP_WS_BYTES || (reinterpret_cast<uintptr_t>(ws) & 255u)) return WA_EWORKSPACE;
    const int rc = ensure_device();
    if (rc != WA_OK) return rc;

    cudaStream_t s = static_cast<cudaStream_t>(stream);
    wa::PrepArgs a{};
    a.src = src; a.pos = pos; a.q_scale = mode == WA_PREP_L2_ROPE ? q_scale : nullptr; a.inv_freq = inv_freq;
    a.q_out = q_out; a.k_ring = k_ring; a.v_ring = v_ring;
    a.n = n; a.hq = hq; a.hkv = hkv; a.d = d; a.ring = ring; a.mode = mode;
    a.src_tok = lay->src_tok; a.q_tok = lay->q_tok; a.ring_row = lay->ring_row; a.slot = lay->slot;
    a.hdr = static_cast<wa::WsHeader*>(ws);
    if (cudaMemsetAsync(ws, 0, wa::kHeaderBytes, s) != cudaSuccess) return WA_ECUDA;
    if (wa::launch_prep(a, s) != cudaSuccess) return WA_ECUDA;
    return WA_OK;
}

size_t wa_tree_decode_ws_bytes(int32_t rows, int32_t nodes, int32_t hq, int32_t hkv, int32_t d, int32_t win,
                               int32_t ring) {
    if (rows <= 0 || nodes <= 0 || nodes > WA_TREE_MAX_NODES || !heads_ok(hq, hkv) || (d != 128 && d != 256) ||
        win < 0 || ring <= 0 || win > ring)
        return 0;
    const int64_t units = static_cast<int64_t>(rows) * nodes * hq;
    const wa::TreePlan pl = wa::tree_plan(rows, nodes, hq, hkv, win, ring);
    if (units > INT32_MAX || pl.units > INT32_MAX / 2) return 0;
    return wa::kHeaderBytes + static_cast<size_t>(pl.units) * pl.lanes * (static_cast<size_t>(d) + 5) * sizeof(float) +
           static_cast<size_t>(rows) * pl.spans * wa::kTreePairBytes;
}

int wa_tree_decode(const void* q, const void* k_ring, const void* v_ring, const void* k_tree, const void* v_tree,
                   const int32_t* pos, const int32_t* parent, const int32_t* n, int32_t rows, int32_t nodes,
                   int32_t hq, int32_t hkv, int32_t d, int32_t win, int32_t ring, float scale,
                   const wa_tree_strides* strides, void* out, void* ws, size_t ws_bytes, void* stream) {
    if (!q || !k_ring || !v_ring || !k_tree || !v_tree || !pos || !parent || !out) return WA_EINVAL;
    if (rows <= 0 || rows > 65535 || nodes <= 0 || nodes > WA_TREE_MAX_NODES || !heads_ok(hq, hkv) || hkv > 65535)
        return WA_EINVAL;
    if (d != 128 && d != 256) return WA_EINVAL;
    if (win < 0 || ring <= 0 || win > ring) return WA_EINVAL;
    if (!std::isfinite(scale)) return WA_EINVAL;
    if (static_cast<int64_t>(rows) * nodes * hq > INT32_MAX) return WA_EINVAL;
    const int64_t qw = static_cast<int64_t>(hq) * d, kw = static_cast<int64_t>(hkv) * d;
    wa::TreeArgs a{};
    a.q_tok = a.o_tok = qw;
    a.kt_tok = a.vt_tok = kw;
    if (strides) {
        if (strides->q_tok) a.q_tok = strides->q_tok;
        if (strides->k_tok) a.kt_tok = strides->k_tok;
        if (strides->v_tok) a.vt_tok = strides->v_tok;
        if (strides->out_tok) a.o_tok = strides->out_tok;
    }
    a.q_row = a.q_tok * nodes; a.kt_row = a.kt_tok * nodes; a.vt_row = a.vt_tok * nodes; a.o_row = a.o_tok * nodes;
    if (strides) {
        if (strides->q_row) a.q_row = strides->q_row;
        if (strides->k_row) a.kt_row = strides->k_row;
        if (strides->v_row) a.vt_row = strides->v_row;
        if (strides->out_row) a.o_row = strides->out_row;
    }
    if (a.q_tok < qw || a.o_tok < qw || a.kt_tok < kw || a.vt_tok < kw) return WA_EINVAL;
    if (a.q_row < qw || a.o_row < qw || a.kt_row < kw || a.vt_row < kw) return WA_EINVAL;
    if ((a.q_tok | a.q_row | a.o_tok | a.o_row | a.kt_tok | a.kt_row | a.vt_tok | a.vt_row) & 7) return WA_EINVAL;
    if (!aligned16(q) || !aligned16(k_ring) || !aligned16(v_ring) || !aligned16(k_tree) || !aligned16(v_tree) ||
        !aligned16(out))
        return WA_EINVAL;
    const size_t need = wa_tree_decode_ws_bytes(rows, nodes, hq, hkv, d, win, ring);
    if (need == 0) return WA_EINVAL;
    if (!ws || ws_bytes < need || (reinterpret_cast<uintptr_t>(ws) & 255u)) return WA_EWORKSPACE;
    const int rc = ensure_device();
    if (rc != WA_OK) return rc;

    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint8_t* base = static_cast<uint8_t*>(ws);
    a.q = q; a.k = k_ring; a.v = v_ring; a.kt = k_tree; a.vt = v_tree;
    a.pos = pos; a.parent = parent; a.n = n;
    a.rows = rows; a.nodes = nodes; a.hq = hq; a.hkv = hkv; a.d = d; a.win = win; a.ring = ring; a.scale = scale;
    a.out = out;
    a.hdr = reinterpret_cast<wa::WsHeader*>(base);
    a.part = base + wa::kHeaderBytes;
    if (wa::launch_tree(a, s) != cudaSuccess) return WA_ECUDA;
    return WA_OK;
}

int wa_tree_verify(const float* target, const float* draft, const int32_t* parent, const int32_t* tokens,
                   const int32_t* n, const float* u, int32_t rows, int32_t nodes, int32_t vocab,
                   const wa_verify_strides* strides, int32_t* path, int32_t* length, int32_t* token,
                   void* ws, size_t ws_bytes, void* stream) {
    if (!target || !parent || !tokens || !u || !path || !length || !token) return WA_EINVAL;
    if (rows <= 0 || rows > 65535 || nodes <= 0 || nodes > WA_TREE_MAX_NODES || vocab <= 0 || vocab > (1 << 24))
        return WA_EINVAL;
    if ((reinterpret_cast<uintptr_t>(target) | reinterpret_cast<uintptr_t>(draft)) & 3u) return WA_EINVAL;
    wa::VerifyArgs a{};
    a.t_node = a.d_node = vocab;
    if (strides && strides->t_node) a.t_node = strides->t_node;
    if (strides && strides->d_node) a.d_node = strides->d_node;
    a.t_row = a.t_node * nodes;
    a.d_row = a.d_node * nodes;
    if (strides && strides->t_row) a.t_row = strides->t_row;
    if (strides && strides->d_row) a.d_row = strides->d_row;
    if (a.t_node < vocab || a.t_row < vocab || (draft && (a.d_node < vocab || a.d_row < vocab))) return WA_EINVAL;
    if (!ws || ws_bytes < WA_TREE_WS_BYTES || (reinterpret_cast<uintptr_t>(ws) & 255u)) return WA_EWORKSPACE;
    const int rc = ensure_device();
    if (rc != WA_OK) return rc;

    cudaStream_t s = static_cast<cudaStream_t>(stream);
    a.target = target; a.draft = draft; a.parent = parent; a.tokens = tokens; a.n = n; a.u = u;
    a.rows = rows; a.nodes = nodes; a.vocab = vocab;
    a.path = path; a.length = length; a.token = token;
    a.hdr = static_cast<wa::WsHeader*>(ws);
    if (wa::launch_verify(a, s) != cudaSuccess) return WA_ECUDA;
    return WA_OK;
}

int wa_tree_commit(int32_t layers, const void* const* k_tree, const void* const* v_tree, void* const* k_ring,
                   void* const* v_ring, const int32_t* ring, int32_t rows, int32_t nodes, int32_t hkv, int32_t d,
                   const wa_tree_strides* lay, const int32_t* path, int32_t most, const int32_t* length,
                   const int32_t* pos, void* ws, size_t ws_bytes, void* stream) {
    if (!k_tree || !v_tree || !k_ring || !v_ring || !ring || !path || !length || !pos) return WA_EINVAL;
    if (layers <= 0 || layers > WA_COMMIT_MAX_LAYERS || rows <= 0 || rows > 65535) return WA_EINVAL;
    if (nodes <= 0 || nodes > WA_TREE_MAX_NODES || most <= 0 || most > WA_TREE_MAX_NODES) return WA_EINVAL;
    if (hkv <= 0 || hkv > 65535 || (d != 128 && d != 256)) return WA_EINVAL;
    const int64_t kw = static_cast<int64_t>(hkv) * d;
    wa::CommitArgs a{};
    a.tok[0] = lay && lay->k_tok ? lay->k_tok : kw;
    a.tok[1] = lay && lay->v_tok ? lay->v_tok : kw;
    a.row[0] = lay && lay->k_row ? lay->k_row : a.tok[0] * nodes;
    a.row[1] = lay && lay->v_row ? lay->v_row : a.tok[1] * nodes;
    for (int kv = 0; kv < 2; ++kv)
        if (a.tok[kv] < kw || a.row[kv] < kw || ((a.tok[kv] | a.row[kv]) & 7)) return WA_EINVAL;
    for (int l = 0; l < layers; ++l) {
        if (!k_tree[l] || !v_tree[l] || !k_ring[l] || !v_ring[l] || ring[l] <= 0) return WA_EINVAL;
        if (!aligned16(k_tree[l]) || !aligned16(v_tree[l]) || !aligned16(k_ring[l]) || !aligned16(v_ring[l]))
            return WA_EINVAL;
        a.src[0][l] = k_tree[l]; a.src[1][l] = v_tree[l];
        a.dst[0][l] = k_ring[l]; a.dst[1][l] = v_ring[l];
        a.ring[l] = ring[l];
    }
    if (rings_contradict(a, layers)) return WA_EINVAL;
    if (!ws || ws_bytes < WA_TREE_WS_BYTES || (reinterpret_cast<uintptr_t>(ws) & 255u)) return WA_EWORKSPACE;
    const int rc = ensure_device();
    if (rc != WA_OK) return rc;

    cudaStream_t s = static_cast<cudaStream_t>(stream);
    a.layers = layers; a.rows = rows; a.nodes = nodes; a.hkv = hkv; a.d = d; a.most = most;
    a.path = path; a.length = length; a.pos = pos;
    a.hdr = static_cast<wa::WsHeader*>(ws);
    if (wa::launch_commit(a, s) != cudaSuccess) return WA_ECUDA;
    return WA_OK;
}

int wa_rope(const void* x, const int32_t* pos, int32_t n, int32_t heads, int32_t d, const wa_rotary* rot,
            int32_t inverse, int64_t x_tok, int64_t out_tok, void* out, void* stream) {
    if (!x || !pos || !out || !rot || !rotary_ok(rot, d)) return WA_EINVAL;
    if (n <= 0 || heads <= 0 || heads > 65535 || (d != 128 && d != 256) || (inverse != 0 && inverse != 1)) return WA_EINVAL;
    if (!aligned16(x) || !aligned16(out) || ((x_tok | out_tok) & 7)) return WA_EINVAL;
    const int64_t width = static_cast<int64_t>(heads) * d;
    if ((n > 1 && (x_tok < width || out_tok < width)) || (x == out && x_tok != out_tok)) return WA_EINVAL;
    const int rc = ensure_device();
    if (rc != WA_OK) return rc;
    wa::PagedAppendArgs a{};
    a.src = x; a.pos = pos; a.q_out = out;
    a.n = n; a.hq = heads; a.d = d; a.inverse = inverse;
    a.src_tok = x_tok; a.q_tok = out_tok;
    set_rotary(a, rot);
    return wa::launch_paged_append(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? WA_OK : WA_ECUDA;
}

int wa_paged_append(const void* src, const int32_t* pos, const int32_t* row, int32_t n, int32_t hq,
                    const wa_pages* cache, const wa_rotary* rot, int64_t src_tok, int64_t q_tok, void* q_out,
                    void* ws, size_t ws_bytes, void* stream) {
    if (!src || !pos || !q_out || n <= 0 || !pages_ok(cache, hq, 0) || !rotary_ok(rot, cache->d)) return WA_EINVAL;
    if (hq + 2 * cache->hkv > 65535) return WA_EINVAL;     // (a grid's second dimension)
    if ((!row && n > cache->rows) || cache->k == cache->v) return WA_EINVAL;
    if (!aligned16(src) || !aligned16(q_out) || ((src_tok | q_tok) & 7)) return WA_EINVAL;
    const int64_t width = static_cast<int64_t>(hq + 2 * cache->hkv) * cache->d;
    if (n > 1 && (src_tok < width || q_tok < static_cast<int64_t>(hq) * cache->d)) return WA_EINVAL;
    if (src == q_out && n > 1 && src_tok != q_tok) return WA_EINVAL;
    if (!ws || ws_bytes < WA_PAGED_APPEND_WS_BYTES || (reinterpret_cast<uintptr_t>(ws) & 255u)) return WA_EWORKSPACE;
    const int rc = ensure_device();
    if (rc != WA_OK) return rc;
    wa::PagedAppendArgs a{};
    a.src = src; a.pos = pos; a.row = row; a.q_out = q_out;
    a.kv[0] = {cache->k, cache->k_scale, cache->k_page, cache->k_slot, head_stride(*cache, cache->k_head)};
    a.kv[1] = {cache->v, cache->v_scale, cache->v_page, cache->v_slot, head_stride(*cache, cache->v_head)};
    a.table = cache->table; a.table_row = cache->table_row;
    a.src_tok = src_tok; a.q_tok = q_tok;
    a.hdr = static_cast<wa::WsHeader*>(ws);
    a.n = n; a.hq = hq; a.hkv = cache->hkv; a.d = cache->d;
    a.pages = cache->pages; a.page_log = log2_of(cache->page_size); a.rows = cache->rows; a.most = cache->most;
    a.e4m3 = cache->type == WA_PAGE_E4M3;
    set_rotary(a, rot);
    return wa::launch_paged_append(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? WA_OK : WA_ECUDA;
}

size_t wa_paged_decode_ws_bytes(const wa_pages* cache, int32_t hq, int32_t win) {
    if (!cache || !page_sizes_ok(*cache, hq, win)) return 0;
    return wa::paged_plan(cache->rows, hq, cache->hkv, cache->d, log2_of(cache->page_size), cache->most, win).bytes;
}

int wa_paged_decode(const void* q, const int32_t* pos, int32_t hq, const wa_pages* cache, int32_t win, float scale,
                    int64_t q_row, int64_t out_row, void* out, void* ws, size_t ws_bytes, void* stream) {
    if (!q || !pos || !out || !pages_ok(cache, hq, win) || !std::isfinite(scale)) return WA_EINVAL;
    if (!pages_in_steps(*cache, cache->k_page, cache->k_slot, cache->k_head) ||
        !pages_in_steps(*cache, cache->v_page, cache->v_slot, cache->v_head))
        return WA_EINVAL;
    if (!aligned16(q) || !aligned16(out) || ((q_row | out_row) & 7)) return WA_EINVAL;
    const int64_t width = static_cast<int64_t>(hq) * cache->d;
    if (cache->rows > 1 && (q_row < width || out_row < width)) return WA_EINVAL;
    const size_t need = wa_paged_decode_ws_bytes(cache, hq, win);
    if (!ws || ws_bytes < need || (reinterpret_cast<uintptr_t>(ws) & 255u)) return WA_EWORKSPACE;
    const int rc = ensure_device();
    if (rc != WA_OK) return rc;
    wa::PagedArgs a{};
    a.q = q; a.pos = pos; a.out = out;
    a.kv[0] = {cache->k, cache->k_scale, cache->k_page, cache->k_slot, head_stride(*cache, cache->k_head)};
    a.kv[1] = {cache->v, cache->v_scale, cache->v_page, cache->v_slot, head_stride(*cache, cache->v_head)};
    a.table = cache->table; a.table_row = cache->table_row; a.q_row = q_row; a.o_row = out_row;
    a.hdr = static_cast<wa::WsHeader*>(ws);
    a.rows = cache->rows; a.hq = hq; a.hkv = cache->hkv; a.d = cache->d;
    a.pages = cache->pages; a.page_log = log2_of(cache->page_size); a.most = cache->most;
    a.e4m3 = cache->type == WA_PAGE_E4M3;
    a.win = win; a.scale = scale;
    return wa::launch_paged_decode(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? WA_OK : WA_ECUDA;
}

int wa_status(const void* ws, void* stream) {
    if (!ws) {   // the header of wa_decode_static's scratch on the current device
        void* sws = nullptr;
        const int rc = wa::static_ws_header(&sws);
        if (rc != WA_OK) return rc;
        ws = sws;
    }
    int st = 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cudaMemcpyAsync(&st, ws, sizeof(int), cudaMemcpyDeviceToHost, s) != cudaSuccess) return WA_ECUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return WA_ECUDA;
    return st;
}

const char* wa_strerror(int code) {
    switch (code) {
        case WA_OK: return "ok";
        case WA_EINVAL: return "invalid argument";
        case WA_EWORKSPACE: return "workspace missing, misaligned or too small";
        case WA_ECUDA: return "CUDA call or launch failed";
        case WA_EDEVICE: return "device is not compute capability 10.3 (GB300)";
        case WA_ESTATIC: return "sizes need more scratch than wa_decode_static's fixed 16 MiB array";
        case WA_STATUS_BAD_POS: return "status: a decode or append position was out of range (clamped or skipped)";
        case WA_STATUS_BAD_HI: return "status: a prompt hi[i] was out of range (clamped)";
        case WA_STATUS_TIMEOUT: return "status: a device wait ran out; outputs are not valid";
        case WA_STATUS_BAD_TREE: return "status: a tree's parent, node count, token, path or length was out of range (clamped or skipped)";
        case WA_STATUS_NO_MASS: return "status: a distribution without mass; its row has no token";
        case WA_STATUS_BAD_PAGE: return "status: a page table entry or a token's row was out of range (skipped, or read as zeros)";
        case WA_STATUS_LAYOUT: return "status: shared memory misaligned; outputs were not written";
        default:
            if (code > 0) return "status: several WA_STATUS bits";
            return "unknown code";
    }
}

int wa_version(void) { return 200; }

}  // extern "C"
