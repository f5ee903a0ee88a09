// abi.hip -- the extern "C" entry points declared in include/q4moe.h:
// host-side validation (fail-closed, nothing is enqueued on error), workspace
// layout, and the launches on the caller's stream.
#include <stdarg.h>
#include <stdio.h>

#include <atomic>
#include <cmath>
#include <mutex>

#include "internal.h"
#include "lmhead.h"
#include "ops.h"

namespace {

thread_local char g_err[256] = "";

// Timing hook state (moe_trace_events): caller-owned events, next index.
thread_local hipEvent_t* g_trace = nullptr;
thread_local int g_trace_n = 0, g_trace_next = 0;

void trace_begin(hipStream_t s) {
    g_trace_next = 0;
    q4moe::trace_point(s);
}

int fail(int code, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    return code;
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

int check_ptr(const void* p, const char* what, bool allow_null = false) {
    if (!p) return allow_null ? MOE_OK : fail(MOE_EINVAL, "%s is NULL", what);
    if (!aligned16(p)) return fail(MOE_EINVAL, "%s is not 16-byte aligned", what);
    return MOE_OK;
}

int check_mat(const moe_q4mat& m, const char* name) {
    char buf[64];
    int rc;
    snprintf(buf, sizeof buf, "%s.q", name);
    if ((rc = check_ptr(m.q, buf))) return rc;
    snprintf(buf, sizeof buf, "%s.scale", name);
    if ((rc = check_ptr(m.scale, buf))) return rc;
    snprintf(buf, sizeof buf, "%s.bias", name);
    return check_ptr(m.bias, buf);
}

int check_layer_sizes(const moe_layer* L) {
    if (!L) return fail(MOE_EINVAL, "layer is NULL");
    if (L->d <= 0 || L->inter <= 0 || L->n_experts <= 0 || L->top_k <= 0)
        return fail(MOE_EINVAL, "non-positive layer size (d=%d inter=%d E=%d k=%d)", L->d,
                    L->inter, L->n_experts, L->top_k);
    if (L->d % MOE_GROUP || L->inter % MOE_GROUP)
        return fail(MOE_EUNSUPPORTED, "d=%d and inter=%d must be multiples of %d", L->d,
                    L->inter, MOE_GROUP);
    if (L->d > MOE_MAX_D || L->inter > MOE_MAX_INTER)
        return fail(MOE_EUNSUPPORTED, "d=%d > %d or inter=%d > %d", L->d, MOE_MAX_D, L->inter,
                    MOE_MAX_INTER);
    if (L->n_experts > MOE_MAX_EXPERTS)
        return fail(MOE_EUNSUPPORTED, "n_experts=%d > %d", L->n_experts, MOE_MAX_EXPERTS);
    if (L->top_k > MOE_MAX_TOPK || L->top_k > L->n_experts)
        return fail(MOE_EUNSUPPORTED, "top_k=%d must be <= min(%d, n_experts=%d)", L->top_k,
                    MOE_MAX_TOPK, L->n_experts);
    return MOE_OK;
}

int check_layer(const moe_layer* L) {
    int rc;
    if ((rc = check_layer_sizes(L))) return rc;
    if ((rc = check_ptr(L->w_router, "w_router"))) return rc;
    if ((rc = check_ptr(L->router_bias, "router_bias", true))) return rc;
    if ((rc = check_mat(L->gate, "gate")) || (rc = check_mat(L->up, "up")) ||
        (rc = check_mat(L->down, "down")) || (rc = check_mat(L->sh_gate, "sh_gate")) ||
        (rc = check_mat(L->sh_up, "sh_up")) || (rc = check_mat(L->sh_down, "sh_down")))
        return rc;
    return MOE_OK;
}

int check_tokens(int32_t T) {
    if (T <= 0) return fail(MOE_EINVAL, "T=%d must be positive", T);
    if (T > MOE_MAX_TOKENS) return fail(MOE_EUNSUPPORTED, "T=%d > %d", T, MOE_MAX_TOKENS);
    return MOE_OK;
}

int check_routing(const moe_routing* r) {
    if (!r) return fail(MOE_EINVAL, "routing is NULL");
    int rc;
    if ((rc = check_ptr(r->logits, "routing.logits")) || (rc = check_ptr(r->topk_idx, "routing.topk_idx")) ||
        (rc = check_ptr(r->topk_w, "routing.topk_w")) || (rc = check_ptr(r->counts, "routing.counts")) ||
        (rc = check_ptr(r->offsets, "routing.offsets")) || (rc = check_ptr(r->perm, "routing.perm")) ||
        (rc = check_ptr(r->inv_perm, "routing.inv_perm")) ||
        (rc = check_ptr(r->block_map, "routing.block_map")) ||
        (rc = check_ptr(r->n_blocks, "routing.n_blocks")) ||
        (rc = check_ptr(r->tile_map, "routing.tile_map")) ||
        (rc = check_ptr(r->n_tiles, "routing.n_tiles")) ||
        (rc = check_ptr(r->blk_counts, "routing.blk_counts")))
        return rc;
    return MOE_OK;
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// Workspace: [decode region | prefill region], so one workspace sized for T
// tokens serves both entry points.
struct DecodeWs {
    size_t sel_idx, sel_w, logits, partial, h, y_sh, total;
};
DecodeWs decode_ws(const moe_layer* L) {
    DecodeWs w;
    size_t o = 0;
    const size_t nt = MOE_MAX_DECODE_TOKENS;
    w.sel_idx = o; o += align256(sizeof(int32_t) * nt * MOE_MAX_TOPK);
    w.sel_w = o; o += align256(sizeof(float) * nt * MOE_MAX_TOPK);
    w.logits = o; o += align256(sizeof(float) * nt * L->n_experts);
    w.partial = o;
    o += align256(sizeof(float) * (size_t)((L->d + MOE_DECODE_ROUTER_ROWS - 1) / MOE_DECODE_ROUTER_ROWS) *
                  nt * L->n_experts);
    w.h = o; o += align256(sizeof(uint16_t) * nt * (size_t)(L->top_k + 1) * L->inter);
    w.y_sh = o; o += align256(sizeof(float) * nt * (size_t)L->d);
    w.total = o;
    return w;
}
struct PrefillWs {
    size_t h, h_sh, part, pexp, dn_pre, dn_exp, total;
};
PrefillWs prefill_ws(const moe_layer* L, int32_t T, size_t base) {
    PrefillWs w;
    const size_t A = (size_t)T * L->top_k;
    size_t o = base;
    w.h = o; o += align256(sizeof(uint16_t) * A * L->inter);
    w.h_sh = o; o += align256(sizeof(uint16_t) * (size_t)T * L->inter);
    w.part = o; o += align256(sizeof(uint16_t) * A * L->d);
    w.pexp = o; o += align256((size_t)T * (L->d / 32) * MOE_MAX_TOPK);
    const size_t n_items = (size_t)moe_block_map_capacity(T, L->top_k, L->n_experts, MOE_TILE_ROWS);
    w.dn_pre = o; o += align256(sizeof(int32_t) * (n_items + 1));
    w.dn_exp = o; o += align256(sizeof(int32_t) * n_items);
    w.total = o;
    return w;
}

q4moe::Q4 q4(const moe_q4mat& m) { return q4moe::Q4{m.q, m.scale, m.bias}; }

int check_lm(const moe_lm_head* lm) {
    if (!lm) return fail(MOE_EINVAL, "lm head is NULL");
    if (lm->V <= 0 || lm->d <= 0) return fail(MOE_EINVAL, "V=%d and d=%d must be positive", lm->V, lm->d);
    if (lm->d % MOE_GROUP || lm->d > MOE_MAX_D)
        return fail(MOE_EUNSUPPORTED, "d=%d must be a multiple of %d and <= %d", lm->d, MOE_GROUP,
                    MOE_MAX_D);
    if (lm->V > MOE_MAX_VOCAB) return fail(MOE_EUNSUPPORTED, "V=%d > %d", lm->V, MOE_MAX_VOCAB);
    return MOE_OK;
}

// Hand-off workspace: per-work-group best (logit, row) pairs.
size_t lm_part_bytes(int32_t V) { return align256(8 * (size_t)q4moe::lm_partials(V, false)); }

// Sampling workspace of B rows of V logits.
struct SampleWs {
    size_t part_max, chunk_w, hist, list, list_n, state, row, total;
    int chunk_sh, n_chunks;
};
SampleWs sample_ws(int32_t V, int32_t B) {
    SampleWs w;
    w.chunk_sh = q4moe::sample_chunk_sh(V, B);
    w.n_chunks = (V + (1 << w.chunk_sh) - 1) >> w.chunk_sh;
    const size_t rows = (size_t)B, parts = rows * (size_t)w.n_chunks;
    size_t o = 0;
    w.part_max = o; o += align256(sizeof(float) * parts);
    w.chunk_w = o; o += align256(sizeof(uint64_t) * parts);
    w.hist = o; o += align256(sizeof(uint64_t) * rows * q4moe::kSampleBins);
    w.list = o; o += align256(sizeof(uint64_t) * rows * q4moe::kSampleList);
    w.list_n = o; o += align256(sizeof(uint32_t) * rows);
    w.state = o; o += align256(sizeof(q4moe::SampleState) * rows);
    w.row = o; o += align256(sizeof(q4moe::SampleRow) * rows);
    w.total = o;
    return w;
}

int check_sample_sizes(int32_t V, int32_t B) {
    if (V <= 0 || B <= 0) return fail(MOE_EINVAL, "V=%d and B=%d must be positive", V, B);
    if (V > MOE_MAX_VOCAB) return fail(MOE_EUNSUPPORTED, "V=%d > %d", V, MOE_MAX_VOCAB);
    if (B > MOE_MAX_SAMPLE_ROWS) return fail(MOE_EUNSUPPORTED, "B=%d > %d", B, MOE_MAX_SAMPLE_ROWS);
    return MOE_OK;
}

// A per-row array: only 4-byte alignment is asked for.
int check_row_array(const void* p, const char* what, bool allow_null) {
    if (!p) return allow_null ? MOE_OK : fail(MOE_EINVAL, "%s is NULL", what);
    if ((uintptr_t)p & 3u) return fail(MOE_EINVAL, "%s is not 4-byte aligned", what);
    return MOE_OK;
}

int hip_status(hipError_t e, const char* what) {
    if (e != hipSuccess) return fail(MOE_EHIP, "%s: %s", what, hipGetErrorString(e));
    return MOE_OK;
}

}  // namespace

namespace q4moe {
void trace_point(hipStream_t s) {
    if (g_trace && g_trace_next < g_trace_n) (void)hipEventRecord(g_trace[g_trace_next++], s);
}
}  // namespace q4moe

extern "C" {

void moe_trace_events(void* const* events, int32_t n) {
    g_trace = (events && n > 0) ? (hipEvent_t*)events : nullptr;
    g_trace_n = g_trace ? n : 0;
    g_trace_next = 0;
}

int32_t moe_block_map_capacity(int32_t T, int32_t top_k, int32_t n_experts, int32_t rows) {
    if (T <= 0 || top_k <= 0 || n_experts <= 0 || rows <= 0) return 0;
    const int64_t A = (int64_t)T * top_k;
    return (int32_t)(A / rows + (n_experts < A ? n_experts : A));
}

size_t moe_workspace_bytes(const moe_layer* L, int32_t T) {
    if (check_layer(L) || check_tokens(T)) return 0;
    const DecodeWs dw = decode_ws(L);
    return prefill_ws(L, T, dw.total).total;
}

int moe_route(const moe_layer* L, const uint16_t* x, int32_t T, uint32_t flags,
              const moe_routing* r, void* stream) {
    int rc;
    if ((rc = check_layer(L)) || (rc = check_tokens(T)) || (rc = check_routing(r))) return rc;
    const bool logits_in = flags & MOE_LOGITS_IN;
    if (flags & ~MOE_LOGITS_IN) return fail(MOE_EINVAL, "unknown flags 0x%x", flags);
    if (!logits_in && (rc = check_ptr(x, "x"))) return rc;
    hipStream_t s = (hipStream_t)stream;
    trace_begin(s);
    if ((rc = hip_status(q4moe::launch_router_logits(logits_in ? nullptr : x, T, L->d,
                                                     L->w_router, L->router_bias, L->n_experts,
                                                     r->logits, r->blk_counts, s),
                         "router logits")))
        return rc;
    if ((rc = hip_status(q4moe::launch_topk(r->logits, T, L->n_experts, L->top_k, r->topk_idx,
                                            r->topk_w, r->blk_counts, s),
                         "top-k")))
        return rc;
    return hip_status(q4moe::launch_route_sort(r->topk_idx, T, L->top_k, L->n_experts, r, s),
                      "route sort");
}

int moe_route_scored(const moe_layer* L, const uint16_t* x, int32_t T, uint32_t flags,
                     const moe_router_spec* spec, const moe_routing* r, void* stream) {
    int rc;
    if ((rc = check_layer_sizes(L)) || (rc = check_tokens(T)) || (rc = check_routing(r))) return rc;
    if (flags & ~MOE_LOGITS_IN) return fail(MOE_EINVAL, "unknown flags 0x%x", flags);
    const bool logits_in = flags & MOE_LOGITS_IN;
    if (!logits_in && ((rc = check_ptr(x, "x")) || (rc = check_ptr(L->w_router, "w_router")) ||
                       (rc = check_ptr(L->router_bias, "router_bias", true))))
        return rc;
    if (!spec) return fail(MOE_EINVAL, "spec is NULL");
    if ((rc = check_ptr(spec->balance, "spec.balance", true))) return rc;
    if (spec->score != MOE_SCORE_SOFTMAX && spec->score != MOE_SCORE_SIGMOID)
        return fail(MOE_EINVAL, "spec.score=%d", spec->score);
    if (spec->renorm != 0 && spec->renorm != 1) return fail(MOE_EINVAL, "spec.renorm=%d", spec->renorm);
    if (!std::isfinite(spec->scale))
        return fail(MOE_EINVAL, "spec.scale must be finite");
    const int G = spec->n_groups;
    if (G < 1 || spec->top_groups < 1 || spec->top_groups > G)
        return fail(MOE_EINVAL, "spec.n_groups=%d spec.top_groups=%d", G, spec->top_groups);
    if (G > MOE_MAX_GROUPS || L->n_experts % G)
        return fail(MOE_EUNSUPPORTED, "n_groups=%d must be <= %d and divide n_experts=%d", G,
                    MOE_MAX_GROUPS, L->n_experts);
    if (G > 1 && spec->group_top != 1 && spec->group_top != 2)
        return fail(MOE_EUNSUPPORTED, "spec.group_top=%d must be 1 or 2", spec->group_top);
    if (spec->top_groups * (L->n_experts / G) < L->top_k)
        return fail(MOE_EUNSUPPORTED, "%d groups of %d experts hold fewer than top_k=%d",
                    spec->top_groups, L->n_experts / G, L->top_k);
    hipStream_t s = (hipStream_t)stream;
    const bool small = q4moe::route_is_small(T);
    trace_begin(s);
    // (with given logits this call only clears the histogram, which few tokens do not use)
    if (!(small && logits_in) &&
        (rc = hip_status(q4moe::launch_router_logits(logits_in ? nullptr : x, T, L->d, L->w_router,
                                                     L->router_bias, L->n_experts, r->logits,
                                                     r->blk_counts, s),
                         "router logits")))
        return rc;
    q4moe::ScoreArgs a;
    a.logits = r->logits;
    a.balance = spec->balance;
    a.T = T;
    a.E = L->n_experts;
    a.k = L->top_k;
    a.n_groups = G;
    a.top_groups = spec->top_groups;
    a.group_top = spec->group_top;
    a.sigmoid = spec->score == MOE_SCORE_SIGMOID;
    a.renorm = spec->renorm != 0;
    a.scale = spec->scale;
    a.idx = r->topk_idx;
    a.w = r->topk_w;
    a.blk_counts = r->blk_counts;
    if (small) return hip_status(q4moe::launch_route_small(a, r, s), "route small");
    if ((rc = hip_status(q4moe::launch_select(a, s), "select"))) return rc;
    return hip_status(q4moe::launch_route_sort(r->topk_idx, T, L->top_k, L->n_experts, r, s),
                      "route sort");
}

int moe_prefill(const moe_layer* L, const uint16_t* x, int32_t T, const moe_routing* r, void* ws,
                size_t ws_bytes, uint16_t* y, void* stream) {
    return moe_prefill_ex(L, x, T, r, ws, ws_bytes, y, 0u, stream);
}

int moe_prefill_ex(const moe_layer* L, const uint16_t* x, int32_t T, const moe_routing* r,
                   void* ws, size_t ws_bytes, uint16_t* y, uint32_t flags, void* stream) {
    int rc;
    if ((rc = check_layer(L)) || (rc = check_tokens(T)) || (rc = check_routing(r)) ||
        (rc = check_ptr(x, "x")) || (rc = check_ptr(y, "y")) || (rc = check_ptr(ws, "workspace")))
        return rc;
    const uint32_t rows_flags = MOE_ITEM_ROWS_64 | MOE_ITEM_ROWS_32 | MOE_ITEM_ROWS_16;
    if ((flags & ~rows_flags) || __builtin_popcount(flags & rows_flags) > 1)
        return fail(MOE_EINVAL, "prefill flags 0x%x", flags);
    const size_t need = moe_workspace_bytes(L, T);
    if (ws_bytes < need)
        return fail(MOE_EWORKSPACE, "workspace %zu bytes < %zu needed", ws_bytes, need);
    const PrefillWs pw = prefill_ws(L, T, decode_ws(L).total);
    unsigned char* base = (unsigned char*)ws;
    q4moe::PrefillArgs a;
    a.x = x;
    a.T = T;
    a.d = L->d;
    a.I = L->inter;
    a.E = L->n_experts;
    a.k = L->top_k;
    a.gate = q4(L->gate);
    a.up = q4(L->up);
    a.down = q4(L->down);
    a.sh_gate = q4(L->sh_gate);
    a.sh_up = q4(L->sh_up);
    a.sh_down = q4(L->sh_down);
    a.perm = r->perm;
    a.offsets = r->offsets;
    a.tile_map = r->tile_map;
    a.n_tiles = r->n_tiles;
    a.topk_w = r->topk_w;
    a.tile_bound = moe_block_map_capacity(T, L->top_k, L->n_experts, MOE_TILE_ROWS);
    a.item_sh = (flags & MOE_ITEM_ROWS_16)   ? 3
                : (flags & MOE_ITEM_ROWS_32) ? 2
                : (flags & MOE_ITEM_ROWS_64) ? 1
                                             : 0;
    a.h = (uint16_t*)(base + pw.h);
    a.h_sh = (uint16_t*)(base + pw.h_sh);
    a.part = (uint16_t*)(base + pw.part);
    a.pexp = (int8_t*)(base + pw.pexp);
    a.dn_pre = (int32_t*)(base + pw.dn_pre);
    a.dn_exp = (int32_t*)(base + pw.dn_exp);
    a.y = y;
    trace_begin((hipStream_t)stream);
    return hip_status(q4moe::launch_prefill(a, (hipStream_t)stream), "prefill");
}

int moe_decode(const moe_layer* L, const uint16_t* x, uint32_t flags, const moe_routing* r,
               void* ws, size_t ws_bytes, uint16_t* y, void* stream) {
    return moe_decode_tokens(L, x, 1, flags, r, ws, ws_bytes, y, stream);
}

}  // extern "C"

namespace {

// Validation shared by the decode entry points (everything but the workspace).
int check_decode(const moe_layer* L, const uint16_t* x, int32_t T, uint32_t flags,
                 const moe_routing* r, const uint16_t* y) {
    int rc;
    if ((rc = check_layer(L)) || (rc = check_ptr(y, "y"))) return rc;
    if (T < 1 || T > MOE_MAX_DECODE_TOKENS)
        return fail(MOE_EUNSUPPORTED, "decode takes 1..%d tokens, not T=%d", MOE_MAX_DECODE_TOKENS,
                    T);
    if (flags & ~(MOE_LOGITS_IN | MOE_ROUTING_IN))
        return fail(MOE_EINVAL, "unknown flags 0x%x", flags);
    const bool logits_in = flags & MOE_LOGITS_IN, routing_in = flags & MOE_ROUTING_IN;
    if ((rc = check_ptr(x, "x"))) return rc;
    if (routing_in && logits_in)
        return fail(MOE_EINVAL, "MOE_ROUTING_IN and MOE_LOGITS_IN exclude each other");
    if (routing_in && (!r || !r->topk_idx || !r->topk_w))
        return fail(MOE_EINVAL, "MOE_ROUTING_IN needs routing->topk_idx and topk_w");
    if (logits_in && (!r || !r->logits))
        return fail(MOE_EINVAL, "MOE_LOGITS_IN needs routing->logits");
    if (r) {
        if ((rc = check_ptr(r->logits, "routing.logits", true)) ||
            (rc = check_ptr(r->topk_idx, "routing.topk_idx", true)) ||
            (rc = check_ptr(r->topk_w, "routing.topk_w", true)))
            return rc;
    }
    return MOE_OK;
}

// The decode launches with the decode region of the workspace at `base`.
int decode_launch(const moe_layer* L, const uint16_t* x, int32_t T, uint32_t flags,
                  const moe_routing* r, unsigned char* base, uint16_t* y, void* stream) {
    const DecodeWs dw = decode_ws(L);
    q4moe::DecodeArgs a;
    a.x = x;
    a.T = T;
    a.d = L->d;
    a.I = L->inter;
    a.E = L->n_experts;
    a.k = L->top_k;
    a.w_router = L->w_router;
    a.router_bias = L->router_bias;
    a.gate = q4(L->gate);
    a.up = q4(L->up);
    a.down = q4(L->down);
    a.sh_gate = q4(L->sh_gate);
    a.sh_up = q4(L->sh_up);
    a.sh_down = q4(L->sh_down);
    a.logits_in = (flags & MOE_LOGITS_IN) != 0;
    a.routing_in = (flags & MOE_ROUTING_IN) != 0;
    a.logits = (r && r->logits) ? r->logits : (float*)(base + dw.logits);
    a.out_idx = r ? r->topk_idx : nullptr;
    a.out_w = r ? r->topk_w : nullptr;
    a.partial = (float*)(base + dw.partial);
    a.sel_idx = (int32_t*)(base + dw.sel_idx);
    a.sel_w = (float*)(base + dw.sel_w);
    a.h = (uint16_t*)(base + dw.h);
    a.y_sh = (float*)(base + dw.y_sh);
    a.y = y;
    trace_begin((hipStream_t)stream);
    return hip_status(q4moe::launch_decode(a, (hipStream_t)stream), "decode");
}

// Scratch of moe_decode_tokens_static: one copy per GPU, for the life of the
// process.  Host code never uses this name as an address (in host code it is
// a stand-in, not device memory); it uses the per-device address that
// hipGetSymbolAddress returns.
constexpr size_t kStaticScratchBytes = MOE_STATIC_SCRATCH_BYTES;
static __device__ __align__(256) unsigned char scratch[kStaticScratchBytes];

constexpr int kMaxDevices = 64;
std::atomic<unsigned char*> g_scratch_ptr[kMaxDevices];
std::mutex g_scratch_mutex;

// The current device's scratch address, looked up once per device with that
// device current.  NULL (and the reason in the error text) on failure.
unsigned char* static_scratch(int* rc) {
    int dev = -1;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) {
        *rc = fail(MOE_EHIP, "hipGetDevice: %s", hipGetErrorString(e));
        return nullptr;
    }
    if (dev < 0 || dev >= kMaxDevices) {
        *rc = fail(MOE_EUNSUPPORTED, "device %d is beyond the %d the library tracks", dev,
                   kMaxDevices);
        return nullptr;
    }
    unsigned char* p = g_scratch_ptr[dev].load(std::memory_order_acquire);
    if (p) return p;
    std::lock_guard<std::mutex> lock(g_scratch_mutex);
    p = g_scratch_ptr[dev].load(std::memory_order_relaxed);
    if (!p) {
        void* addr = nullptr;
        e = hipGetSymbolAddress(&addr, HIP_SYMBOL(scratch));
        if (e != hipSuccess || !addr) {
            *rc = fail(MOE_EHIP, "hipGetSymbolAddress(scratch) on device %d: %s", dev,
                       hipGetErrorString(e));
            return nullptr;
        }
        p = (unsigned char*)addr;
        g_scratch_ptr[dev].store(p, std::memory_order_release);
    }
    return p;
}

}  // namespace

extern "C" {

int moe_decode_tokens_static(const moe_layer* L, const uint16_t* x, int32_t T, uint32_t flags,
                             const moe_routing* r, uint16_t* y, void* stream) {
    int rc;
    if ((rc = check_decode(L, x, T, flags, r, y))) return rc;
    const size_t need = decode_ws(L).total;
    if (need > kStaticScratchBytes)
        return fail(MOE_EUNSUPPORTED,
                    "this layer's decode scratch (%zu bytes) exceeds the library's static %zu",
                    need, kStaticScratchBytes);
    unsigned char* base = static_scratch(&rc);
    if (!base) return rc;
    return decode_launch(L, x, T, flags, r, base, y, stream);
}

int moe_decode_tokens(const moe_layer* L, const uint16_t* x, int32_t T, uint32_t flags,
                      const moe_routing* r, void* ws, size_t ws_bytes, uint16_t* y,
                      void* stream) {
    int rc;
    if ((rc = check_decode(L, x, T, flags, r, y)) || (rc = check_ptr(ws, "workspace")))
        return rc;
    const size_t need = moe_workspace_bytes(L, 1);
    if (ws_bytes < need)
        return fail(MOE_EWORKSPACE, "workspace %zu bytes < %zu needed", ws_bytes, need);
    return decode_launch(L, x, T, flags, r, (unsigned char*)ws, y, stream);
}

int moe_dequant(const moe_q4mat* m, int32_t n_rows, int32_t K, uint16_t* w_out, void* stream) {
    int rc;
    if (!m) return fail(MOE_EINVAL, "matrix is NULL");
    if ((rc = check_mat(*m, "m")) || (rc = check_ptr(w_out, "w_out"))) return rc;
    if (n_rows <= 0 || K <= 0) return fail(MOE_EINVAL, "n_rows=%d K=%d", n_rows, K);
    if (K % MOE_GROUP) return fail(MOE_EUNSUPPORTED, "K=%d not a multiple of %d", K, MOE_GROUP);
    return hip_status(q4moe::launch_dequant(q4(*m), n_rows, K, w_out, (hipStream_t)stream),
                      "dequant");
}

size_t moe_lm_workspace_bytes(const moe_lm_head* lm) {
    if (check_lm(lm)) return 0;
    return lm_part_bytes(lm->V);
}

int moe_lm_argmax(const moe_lm_head* lm, const uint16_t* x, uint32_t flags, float* logits,
                  int32_t* token, uint16_t* x_next, void* ws, size_t ws_bytes, void* stream) {
    int rc;
    if ((rc = check_lm(lm))) return rc;
    if (flags & ~MOE_LOGITS_IN) return fail(MOE_EINVAL, "unknown flags 0x%x", flags);
    const bool logits_in = flags & MOE_LOGITS_IN;
    if (!logits_in && ((rc = check_mat(lm->head, "head")) || (rc = check_ptr(x, "x")))) return rc;
    if ((rc = check_ptr(logits, "logits")) || (rc = check_ptr(ws, "workspace"))) return rc;
    if (!token || ((uintptr_t)token & 3u))
        return fail(MOE_EINVAL, "token is NULL or not 4-byte aligned");
    if (x_next && ((rc = check_ptr(x_next, "x_next")) || (rc = check_mat(lm->embed, "embed"))))
        return rc;
    const size_t need = moe_lm_workspace_bytes(lm);
    if (ws_bytes < need)
        return fail(MOE_EWORKSPACE, "workspace %zu bytes < %zu needed", ws_bytes, need);
    unsigned char* base = (unsigned char*)ws;
    q4moe::LmArgs a;
    a.x = x;
    a.V = lm->V;
    a.d = lm->d;
    a.head = q4(lm->head);
    a.embed = q4(lm->embed);
    a.logits = logits;
    a.token = token;
    a.x_next = x_next;
    a.part = (int2*)base;
    trace_begin((hipStream_t)stream);
    return hip_status(q4moe::launch_lm_argmax(a, logits_in, (hipStream_t)stream), "lm argmax");
}

size_t moe_sample_workspace_bytes(int32_t V, int32_t B) {
    if (check_sample_sizes(V, B)) return 0;
    return sample_ws(V, B).total;
}

int moe_sample(const moe_lm_head* lm, const float* logits, int32_t B, const moe_sampling* p,
               int32_t* token, float* prob, uint16_t* x_next, void* ws, size_t ws_bytes,
               void* stream) {
    int rc;
    if (!lm) return fail(MOE_EINVAL, "lm head is NULL");
    if (!p) return fail(MOE_EINVAL, "sampling is NULL");
    if ((rc = check_sample_sizes(lm->V, B)) || (rc = check_ptr(logits, "logits")) ||
        (rc = check_row_array(p->u, "u", false)) ||
        (rc = check_row_array(p->temperature, "temperature", true)) ||
        (rc = check_row_array(p->top_k, "top_k", true)) ||
        (rc = check_row_array(p->top_p, "top_p", true)) ||
        (rc = check_row_array(p->min_p, "min_p", true)) ||
        (rc = check_row_array(token, "token", false)) ||
        (rc = check_row_array(prob, "prob", true)) || (rc = check_ptr(ws, "workspace")))
        return rc;
    if (x_next && ((rc = check_lm(lm)) || (rc = check_ptr(x_next, "x_next")) ||
                   (rc = check_mat(lm->embed, "embed"))))
        return rc;
    const SampleWs w = sample_ws(lm->V, B);
    if (ws_bytes < w.total)
        return fail(MOE_EWORKSPACE, "workspace %zu bytes < %zu needed", ws_bytes, w.total);
    unsigned char* base = (unsigned char*)ws;
    q4moe::SampleArgs a;
    a.logits = logits;
    a.B = B;
    a.V = lm->V;
    a.d = lm->d;
    a.chunk_sh = w.chunk_sh;
    a.n_chunks = w.n_chunks;
    a.temperature = p->temperature;
    a.top_k = p->top_k;
    a.top_p = p->top_p;
    a.min_p = p->min_p;
    a.temperature_all = p->temperature_all;
    a.top_k_all = p->top_k_all;
    a.top_p_all = p->top_p_all;
    a.min_p_all = p->min_p_all;
    a.u = p->u;
    a.token = token;
    a.prob = prob;
    a.x_next = x_next;
    a.embed = q4(lm->embed);
    a.part_max = (float*)(base + w.part_max);
    a.chunk_w = (uint64_t*)(base + w.chunk_w);
    a.hist = (uint64_t*)(base + w.hist);
    a.list = (uint64_t*)(base + w.list);
    a.list_n = (uint32_t*)(base + w.list_n);
    a.state = (q4moe::SampleState*)(base + w.state);
    a.row = (q4moe::SampleRow*)(base + w.row);
    trace_begin((hipStream_t)stream);
    return hip_status(q4moe::launch_sample(a, (hipStream_t)stream), "sample");
}

int moe_linear(const moe_q4mat* m, int32_t N, int32_t K, const uint16_t* x, int32_t T,
               uint32_t flags, void* y, void* stream) {
    int rc;
    if (!m) return fail(MOE_EINVAL, "matrix is NULL");
    if ((rc = check_mat(*m, "m")) || (rc = check_ptr(x, "x")) || (rc = check_ptr(y, "y"))) return rc;
    if (N <= 0 || K <= 0 || T <= 0) return fail(MOE_EINVAL, "N=%d K=%d T=%d must be positive", N, K, T);
    if (K % MOE_GROUP || K > MOE_MAX_D)
        return fail(MOE_EUNSUPPORTED, "K=%d must be a multiple of %d and <= %d", K, MOE_GROUP,
                    MOE_MAX_D);
    if (N > MOE_MAX_VOCAB) return fail(MOE_EUNSUPPORTED, "N=%d > %d", N, MOE_MAX_VOCAB);
    if (T > MOE_MAX_LINEAR_TOKENS)
        return fail(MOE_EUNSUPPORTED, "T=%d > %d", T, MOE_MAX_LINEAR_TOKENS);
    if (flags & ~MOE_OUT_BF16) return fail(MOE_EINVAL, "unknown flags 0x%x", flags);
    q4moe::LinearArgs a;
    a.w = q4(*m);
    a.x = x;
    a.y = y;
    a.T = T;
    a.N = N;
    a.K = K;
    a.out_bf16 = (flags & MOE_OUT_BF16) != 0;
    trace_begin((hipStream_t)stream);
    return hip_status(q4moe::launch_linear(a, (hipStream_t)stream), "linear");
}

int moe_add_norm(const uint16_t* x, int32_t T, int32_t d, const void* residual,
                 void* residual_out, const uint16_t* weight, float eps, uint32_t flags,
                 uint16_t* y, uint8_t* y8, float* y8_scale, void* stream) {
    int rc;
    if ((rc = check_tokens(T))) return rc;
    if (d <= 0) return fail(MOE_EINVAL, "d=%d must be positive", d);
    if (d % MOE_GROUP || d > MOE_MAX_D)
        return fail(MOE_EUNSUPPORTED, "d=%d must be a multiple of %d and <= %d", d, MOE_GROUP,
                    MOE_MAX_D);
    if (flags & ~(MOE_NORM_PLUS_ONE | MOE_NORM_RESIDUAL_FLOAT | MOE_NORM_GROUP_128))
        return fail(MOE_EINVAL, "unknown flags 0x%x", flags);
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(MOE_EINVAL, "eps must be finite and >= 0");
    if ((rc = check_ptr(x, "x")) || (rc = check_ptr(weight, "weight")) ||
        (rc = check_ptr(residual, "residual", true)) ||
        (rc = check_ptr(residual_out, "residual_out", true)) || (rc = check_ptr(y, "y", true)) ||
        (rc = check_ptr(y8, "y8", true)) || (rc = check_ptr(y8_scale, "y8_scale", true)))
        return rc;
    if (residual_out && !residual)
        return fail(MOE_EINVAL, "residual_out without a residual");
    if (!y && !y8) return fail(MOE_EINVAL, "neither y nor y8 is given");
    if (!y8 != !y8_scale) return fail(MOE_EINVAL, "y8 and y8_scale come together");
    const void* const out[] = {residual_out, y, y8, y8_scale};
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < i; ++j)
            if (out[i] && out[i] == out[j]) return fail(MOE_EINVAL, "two outputs share a buffer");
    q4moe::NormArgs a;
    a.x = x;
    a.residual = residual;
    a.residual_out = residual_out;
    a.weight = weight;
    a.y = y;
    a.y8 = y8;
    a.y8_scale = y8_scale;
    a.T = T;
    a.d = d;
    a.eps = eps;
    a.group = (flags & MOE_NORM_GROUP_128) ? 128 : 64;
    a.w_add = (flags & MOE_NORM_PLUS_ONE) ? 1.0f : 0.0f;
    a.res_f32 = (flags & MOE_NORM_RESIDUAL_FLOAT) != 0;
    trace_begin((hipStream_t)stream);
    return hip_status(q4moe::launch_add_norm(a, (hipStream_t)stream), "add norm");
}

}  // extern "C"

namespace {

// Validation shared by the 8-bit products.
int check_product(const moe_e4m3mat* m, int32_t N, int32_t K, const uint8_t* x, const float* x_scale,
                  uint32_t flags, const void* y, const float* y_scale) {
    int rc;
    if (!m) return fail(MOE_EINVAL, "matrix is NULL");
    if (N <= 0 || K <= 0) return fail(MOE_EINVAL, "N=%d and K=%d must be positive", N, K);
    if (K % MOE_GROUP || K > MOE_MAX_D)
        return fail(MOE_EUNSUPPORTED, "K=%d must be a multiple of %d and <= %d", K, MOE_GROUP,
                    MOE_MAX_D);
    if (N > MOE_MAX_VOCAB) return fail(MOE_EUNSUPPORTED, "N=%d > %d", N, MOE_MAX_VOCAB);
    if (flags & ~(MOE_OUT_BF16 | MOE_GATED)) return fail(MOE_EINVAL, "unknown flags 0x%x", flags);
    const bool gated = flags & MOE_GATED;
    if (gated && (flags & MOE_OUT_BF16))
        return fail(MOE_EINVAL, "MOE_GATED and MOE_OUT_BF16 exclude each other");
    if (gated && N % (2 * MOE_GROUP))
        return fail(MOE_EUNSUPPORTED, "N=%d: a gated product needs a multiple of %d", N, 2 * MOE_GROUP);
    if ((rc = check_ptr(m->w, "m.w")) || (rc = check_ptr(m->scale, "m.scale")) || (rc = check_ptr(x, "x")) ||
        (rc = check_ptr(x_scale, "x_scale")) || (rc = check_ptr(y, "y")) ||
        (rc = check_ptr(y_scale, "y_scale", !gated)))
        return rc;
    if (!gated && y_scale) return fail(MOE_EINVAL, "y_scale without MOE_GATED");
    if (y == (const void*)x || y == (const void*)x_scale || (gated && (y == (const void*)y_scale || y_scale == x_scale)))
        return fail(MOE_EINVAL, "an output shares a buffer with an input or another output");
    return MOE_OK;
}

q4moe::ProductArgs product_args(const moe_e4m3mat* m, int32_t N, int32_t K, const uint8_t* x,
                                const float* x_scale, int32_t rows, uint32_t flags, void* y,
                                float* y_scale) {
    q4moe::ProductArgs a{};
    a.w = m->w;
    a.w_scale = m->scale;
    a.x = x;
    a.x_scale = x_scale;
    a.y = y;
    a.y_scale = y_scale;
    a.rows = rows;
    a.gated = (flags & MOE_GATED) != 0;
    a.N = a.gated ? N / 2 : N;
    a.K = K;
    a.out_bf16 = (flags & MOE_OUT_BF16) != 0;
    a.E = 1;
    return a;
}

// Sizes and indices shared by the calls that move rows between token and expert order.
int check_sort(int32_t T, int32_t k, int32_t d, const moe_routing* r) {
    int rc;
    if ((rc = check_tokens(T))) return rc;
    if (k <= 0 || d <= 0) return fail(MOE_EINVAL, "k=%d and d=%d must be positive", k, d);
    if (k > MOE_MAX_TOPK) return fail(MOE_EUNSUPPORTED, "k=%d > %d", k, MOE_MAX_TOPK);
    if (d % MOE_GROUP || d > MOE_MAX_D)
        return fail(MOE_EUNSUPPORTED, "d=%d must be a multiple of %d and <= %d", d, MOE_GROUP,
                    MOE_MAX_D);
    if (!r) return fail(MOE_EINVAL, "routing is NULL");
    return check_ptr(r->inv_perm, "routing.inv_perm");
}

q4moe::SortArgs sort_args(int32_t T, int32_t k, int32_t d, const moe_routing* r) {
    q4moe::SortArgs a{};
    a.inv_perm = r->inv_perm;
    a.T = T;
    a.k = k;
    a.d = d;
    return a;
}

}  // namespace

extern "C" {

int moe_linear_scaled(const moe_e4m3mat* m, int32_t N, int32_t K, const uint8_t* x, const float* x_scale,
                      int32_t T, uint32_t flags, void* y, float* y_scale, void* stream) {
    int rc;
    if ((rc = check_product(m, N, K, x, x_scale, flags, y, y_scale)) || (rc = check_tokens(T))) return rc;
    const q4moe::ProductArgs a = product_args(m, N, K, x, x_scale, T, flags, y, y_scale);
    trace_begin((hipStream_t)stream);
    return hip_status(q4moe::launch_product(a, (hipStream_t)stream), "linear e4m3");
}

int moe_experts_scaled(const moe_e4m3mat* m, int32_t E, int32_t N, int32_t K, const uint8_t* x,
                       const float* x_scale, int32_t T, int32_t k, const moe_routing* r,
                       uint32_t flags, void* y, float* y_scale, void* stream) {
    int rc;
    if ((rc = check_product(m, N, K, x, x_scale, flags, y, y_scale)) || (rc = check_tokens(T))) return rc;
    if (E <= 0 || k <= 0) return fail(MOE_EINVAL, "E=%d and k=%d must be positive", E, k);
    if (E > MOE_MAX_EXPERTS) return fail(MOE_EUNSUPPORTED, "E=%d > %d", E, MOE_MAX_EXPERTS);
    if (k > MOE_MAX_TOPK || k > E)
        return fail(MOE_EUNSUPPORTED, "k=%d must be <= min(%d, E=%d)", k, MOE_MAX_TOPK, E);
    if (!r) return fail(MOE_EINVAL, "routing is NULL");
    if ((rc = check_ptr(r->offsets, "routing.offsets")) ||
        (rc = check_ptr(r->block_map, "routing.block_map")) ||
        (rc = check_ptr(r->n_blocks, "routing.n_blocks")) ||
        (rc = check_ptr(r->tile_map, "routing.tile_map")) ||
        (rc = check_ptr(r->n_tiles, "routing.n_tiles")))
        return rc;
    q4moe::ProductArgs a = product_args(m, N, K, x, x_scale, T * k, flags, y, y_scale);
    a.E = E;
    a.offsets = r->offsets;
    a.map = r->block_map;
    a.n_map = r->n_blocks;
    a.map_bound = moe_block_map_capacity(T, k, E, MOE_BLOCK_ROWS);
    a.map128 = r->tile_map;
    a.n_map128 = r->n_tiles;
    a.map128_bound = moe_block_map_capacity(T, k, E, MOE_TILE_ROWS);
    trace_begin((hipStream_t)stream);
    return hip_status(q4moe::launch_product(a, (hipStream_t)stream), "experts e4m3");
}

int moe_dispatch(const uint16_t* x, int32_t T, int32_t k, int32_t d, const moe_routing* r, void* rows,
                 float* rows_scale, void* stream) {
    int rc;
    if ((rc = check_sort(T, k, d, r)) || (rc = check_ptr(x, "x")) || (rc = check_ptr(rows, "rows")) ||
        (rc = check_ptr(rows_scale, "rows_scale", true)))
        return rc;
    if (rows == (const void*)x || rows == (void*)rows_scale || (const void*)rows_scale == (const void*)x)
        return fail(MOE_EINVAL, "an output shares a buffer with x or another output");
    q4moe::SortArgs a = sort_args(T, k, d, r);
    a.x = x;
    a.rows_out = rows;
    a.scale_out = rows_scale;
    trace_begin((hipStream_t)stream);
    return hip_status(q4moe::launch_dispatch(a, (hipStream_t)stream), "dispatch");
}

int moe_combine(const uint16_t* rows, int32_t T, int32_t k, int32_t d, const moe_routing* r,
                uint32_t flags, const uint16_t* base, uint16_t* y, void* stream) {
    int rc;
    if ((rc = check_sort(T, k, d, r))) return rc;
    if (flags & ~MOE_UNWEIGHTED) return fail(MOE_EINVAL, "unknown flags 0x%x", flags);
    const bool weighted = !(flags & MOE_UNWEIGHTED);
    if ((rc = check_ptr(rows, "rows")) || (rc = check_ptr(r->topk_w, "routing.topk_w", !weighted)) ||
        (rc = check_ptr(base, "base", true)) || (rc = check_ptr(y, "y")))
        return rc;
    if (y == rows) return fail(MOE_EINVAL, "y shares a buffer with rows");
    q4moe::SortArgs a = sort_args(T, k, d, r);
    a.rows = rows;
    a.w = weighted ? r->topk_w : nullptr;
    a.base = base;
    a.y = y;
    trace_begin((hipStream_t)stream);
    return hip_status(q4moe::launch_combine(a, (hipStream_t)stream), "combine");
}

int moe_combine_grad(const uint16_t* dy, const uint16_t* rows, int32_t T, int32_t k, int32_t d,
                     const moe_routing* r, uint16_t* d_rows, float* d_w, void* stream) {
    int rc;
    if ((rc = check_sort(T, k, d, r)) || (rc = check_ptr(dy, "dy")) ||
        (rc = check_ptr(r->topk_w, "routing.topk_w")) || (rc = check_ptr(d_rows, "d_rows")) ||
        (rc = check_ptr(rows, "rows")) || (rc = check_ptr(d_w, "d_w")))
        return rc;
    if (d_rows == dy || (const void*)d_w == dy || (const void*)d_w == rows ||
        (const void*)d_w == (const void*)d_rows)
        return fail(MOE_EINVAL, "an output shares a buffer with an input or another output");
    q4moe::SortArgs a = sort_args(T, k, d, r);
    a.dy = dy;
    a.rows = rows;
    a.w = r->topk_w;
    a.rows_out = d_rows;
    a.d_w = d_w;
    trace_begin((hipStream_t)stream);
    return hip_status(q4moe::launch_combine_grad(a, (hipStream_t)stream), "combine grad");
}

int moe_penalize(const float* logits, int32_t B, int32_t V, const moe_penalties* p, float* out,
                 void* stream) {
    int rc;
    if (!p) return fail(MOE_EINVAL, "penalties is NULL");
    if ((rc = check_sample_sizes(V, B)) || (rc = check_ptr(logits, "logits")) || (rc = check_ptr(out, "out")) ||
        (rc = check_row_array(p->tokens, "tokens", true)) ||
        (rc = check_row_array(p->n_tokens, "n_tokens", true)) ||
        (rc = check_row_array(p->n_prompt, "n_prompt", true)) ||
        (rc = check_row_array(p->repetition, "repetition", true)) ||
        (rc = check_row_array(p->frequency, "frequency", true)) ||
        (rc = check_row_array(p->presence, "presence", true)) ||
        (rc = check_row_array(p->bias_ids, "bias_ids", true)) ||
        (rc = check_row_array(p->bias, "bias", true)) || (rc = check_row_array(p->mask, "mask", true)))
        return rc;
    if (p->tokens && p->stride < 0) return fail(MOE_EINVAL, "stride=%d", p->stride);
    if (p->tokens && p->stride > MOE_MAX_HISTORY)
        return fail(MOE_EUNSUPPORTED, "stride=%d > %d", p->stride, MOE_MAX_HISTORY);
    if (!p->tokens && (p->n_tokens || p->n_prompt))
        return fail(MOE_EINVAL, "n_tokens and n_prompt need tokens");
    if (!p->bias_ids != !p->bias) return fail(MOE_EINVAL, "bias_ids and bias come together");
    if (p->bias_ids && p->n_bias < 0) return fail(MOE_EINVAL, "n_bias=%d", p->n_bias);
    if (p->bias_ids && p->n_bias > MOE_MAX_BIASES)
        return fail(MOE_EUNSUPPORTED, "n_bias=%d > %d", p->n_bias, MOE_MAX_BIASES);
    q4moe::PenalizeArgs a{};
    a.logits = logits;
    a.out = out;
    a.B = B;
    a.V = V;
    a.tokens = p->tokens;
    a.n_tokens = p->n_tokens;
    a.n_prompt = p->n_prompt;
    a.stride = p->stride;
    a.repetition = p->repetition;
    a.frequency = p->frequency;
    a.presence = p->presence;
    a.repetition_all = p->repetition_all;
    a.frequency_all = p->frequency_all;
    a.presence_all = p->presence_all;
    a.bias_ids = p->bias_ids;
    a.bias = p->bias;
    a.n_bias = p->bias_ids ? p->n_bias : 0;
    a.mask = p->mask;
    a.mask_words = (V + 31) / 32;
    trace_begin((hipStream_t)stream);
    return hip_status(q4moe::launch_penalize(a, (hipStream_t)stream), "penalize");
}

const char* moe_strerror(int code) {
    switch (code) {
        case MOE_OK: return "ok";
        case MOE_EINVAL: return "invalid argument";
        case MOE_EUNSUPPORTED: return "unsupported shape";
        case MOE_EWORKSPACE: return "workspace too small";
        case MOE_EHIP: return "HIP error";
        default: return "unknown status";
    }
}

const char* moe_last_error(void) { return g_err; }

}  // extern "C"
