// rows_op.cu -- the packed-row operators behind the C ABI (include/slm.h): slm_kv_append,
// slm_attention_paged, slm_attention_prompt.  Checks of arguments and the choice of kernels;
// nothing here reads the lengths, which live on the device.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "rows.cuh"

namespace slm {

// SMs of the current device (looked up once per device); < 0: no device, and the status code.
static int current_sms(int &dev) {
    static std::atomic<int> known[64];
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return attn_fail(SLM_ECUDA, "no CUDA device");
    }
    if (dev >= 0 && dev < 64 && known[dev].load() > 0) return known[dev].load();
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return attn_fail(SLM_ECUDA, "no CUDA device");
    }
    if (dev >= 0 && dev < 64) known[dev].store(sms);
    return sms;
}

struct PtrCheck {
    const void *p;
    const char *name;
};

// Device (or managed) memory of the current device, all of them.
static int check_pointers(int dev, const PtrCheck *list, int n) {
    for (int i = 0; i < n; i++) {
        if (!list[i].p) continue;
        cudaPointerAttributes a{};
        if (cudaPointerGetAttributes(&a, list[i].p) != cudaSuccess) {
            cudaGetLastError();
            return attn_fail(SLM_EINVAL, "%s is not device memory", list[i].name);
        }
        if (a.type == cudaMemoryTypeManaged) continue;
        if (a.type != cudaMemoryTypeDevice) return attn_fail(SLM_EINVAL, "%s is not device memory", list[i].name);
        if (a.device != dev)
            return attn_fail(SLM_EINVAL, "%s is memory of device %d, the current device is %d", list[i].name, a.device, dev);
    }
    return SLM_OK;
}

// A launch that was refused.  The runtime keeps the error for the thread's next check, which may be
// another call's: it is taken here.
static int launch_fail(const char *what, cudaError_t e) {
    cudaGetLastError();
    return attn_fail(SLM_ECUDA, "%s launch: %s", what, cudaGetErrorString(e));
}

static int elem_size(int dtype) { return dtype == SLM_F32 ? 4 : 2; }

static int check_dtype(int dtype, const char *name) {
    if (dtype != SLM_F32 && dtype != SLM_BF16) return attn_fail(SLM_EINVAL, "%s %d is neither SLM_F32 nor SLM_BF16", name, dtype);
    return SLM_OK;
}

static int check_heads(int H, int KV, int hd) {
    if (H < 1 || KV < 1 || H % KV) return attn_fail(SLM_EINVAL, "n_heads %d must be a positive multiple of n_kv_heads %d", H, KV);
    if (H > kRowsMaxHeads) return attn_fail(SLM_EINVAL, "n_heads %d above %d", H, kRowsMaxHeads);
    if (hd < 8 || hd % 8 || hd > 256) return attn_fail(SLM_EINVAL, "head_dim %d must be a multiple of 8 in [8, 256]", hd);
    return SLM_OK;
}

static int check_rows(const slm_rows *r) {
    if (!r) return attn_fail(SLM_EINVAL, "rows is NULL");
    if (r->nseq < 1 || r->nseq > kRowsMaxSeqs) return attn_fail(SLM_EINVAL, "nseq %d outside [1, %d]", r->nseq, kRowsMaxSeqs);
    if (r->rows < 0 || r->rows > kRowsMaxRows) return attn_fail(SLM_EINVAL, "rows %d outside [0, 2^30]", r->rows);
    if (!r->row_start) return attn_fail(SLM_EINVAL, "row_start is NULL");
    if ((uintptr_t)r->row_start % 4 || (uintptr_t)r->ctx_len % 4) return attn_fail(SLM_EINVAL, "row_start and ctx_len must be 4-byte aligned");
    return SLM_OK;
}

static int check_cache(const slm_kv_cache *c) {
    if (!c) return attn_fail(SLM_EINVAL, "cache is NULL");
    if (check_dtype(c->kv_dtype, "kv_dtype")) return SLM_EINVAL;
    if (c->n_kv_heads < 1 || c->n_kv_heads > kRowsMaxHeads)
        return attn_fail(SLM_EINVAL, "n_kv_heads %d outside [1, %d]", c->n_kv_heads, kRowsMaxHeads);
    if (c->head_dim < 8 || c->head_dim % 8 || c->head_dim > 256)
        return attn_fail(SLM_EINVAL, "head_dim %d must be a multiple of 8 in [8, 256]", c->head_dim);
    if (c->page_size < 16 || c->page_size > (1 << 20) || (c->page_size & (c->page_size - 1)))
        return attn_fail(SLM_EINVAL, "page_size %d must be a power of two in [16, 2^20]", c->page_size);
    if (c->n_pages < 1 || c->table_ld < 1) return attn_fail(SLM_EINVAL, "n_pages %d and table_ld %d must be positive", c->n_pages, c->table_ld);
    if (!c->k || !c->v || !c->page_table) return attn_fail(SLM_EINVAL, "k, v and page_table of the cache must be non-NULL");
    if (((uintptr_t)c->k | (uintptr_t)c->v) & 15) return attn_fail(SLM_EINVAL, "the cache's k and v must be 16-byte aligned");
    if ((uintptr_t)c->page_table % 4) return attn_fail(SLM_EINVAL, "page_table must be 4-byte aligned");
    return SLM_OK;
}

// Packed rows of `heads` heads: base and row stride (elements) on 16-byte boundaries.  Without rows
// neither means anything (an empty tensor has no address).
static int check_packed(const void *p, long long ld, int heads, int hd, int dtype, int rows, const char *name) {
    if (rows == 0) return SLM_OK;
    if (!p) return attn_fail(SLM_EINVAL, "%s is NULL", name);
    if ((uintptr_t)p & 15) return attn_fail(SLM_EINVAL, "%s must be 16-byte aligned", name);
    if (rows > 1 && (ld < (long long)heads * hd || ld > (1LL << 32)))
        return attn_fail(SLM_EINVAL, "%s: row stride %lld outside [%lld, 2^32]", name, ld, (long long)heads * hd);
    if (rows > 1 && (ld * elem_size(dtype)) % 16) return attn_fail(SLM_EINVAL, "%s: a row stride must be a multiple of 16 bytes", name);
    return SLM_OK;
}

static int check_status(const int32_t *status) {
    if (!status || (uintptr_t)status % 4) return attn_fail(SLM_EINVAL, "status must be a 4-byte aligned device int32");
    return SLM_OK;
}

static int log2i(int v) {
    int s = 0;
    while ((1 << s) < v) s++;
    return s;
}

// Positions are int32 in the kernels.
static long long cache_cap(const slm_kv_cache *c) {
    return std::min<long long>((long long)c->table_ld * c->page_size, 0x7fffff00LL);
}

// Tiling and workspace of an attention call.
struct RowsTiling {
    RowsGeom geom;
    int P, slot_rows;
    size_t ws;
};

// bf16 heads of up to 128 run on the tensor cores, one CTA per SM.
static bool on_tensor_cores(int dtype, int hd) { return dtype == SLM_BF16 && hd <= 128; }

static RowsTiling rows_tiling(int sms, int dtype, int rows, int nseq, int H, int KV, int hd) {
    RowsTiling t{};
    const int G = H / KV;
    if (on_tensor_cores(dtype, hd)) {
        // An item's start and end take about as long as one block of 64-wide heads and two of 128-wide
        // ones.  At 1 / 2: prompts of 8,192 tokens, 128: 380 / 367 us; chunks of 512 over 16,000, 128:
        // 216.2 / 215.6; decode of 64 sequences, 128: 163.2 / 164.4; prompts 16 x 512, 64: 24.0 / 29.7;
        // 2,048, 64: 35.1 / 35.3; decode of 4 x 32,768, 64: 53.3 / 53.1.
        t.geom = {KV, 2 * (128 / G), 7, 1, hd <= 64 ? 1 : 2};
        t.P = sms;
    } else {
        const int R = rows_simt_tile(rows, nseq, G, hd);
        t.geom = {KV, R / G, 6, 1, 1};
        t.P = rows_simt_ctas(sms, hd, R, nseq);
    }
    auto slot = [&](int PT) { return (int)std::min<long long>((long long)PT * G, (long long)std::max(rows, 1) * G); };
    t.slot_rows = slot(t.geom.PT);
    // A workspace serves every call of no more rows and sequences: on the CUDA cores the tile and the
    // CTAs of a launch do not only grow with them, so it is the most of both tiles, at the CTAs of one
    // sequence.
    if (on_tensor_cores(dtype, hd)) {
        t.ws = rows_ws_bytes(t.P, t.slot_rows, hd);
    } else {
        const int wide = rows_simt_wide_tile(hd);
        t.ws = rows_ws_bytes(rows_simt_ctas(sms, hd, wide, 1), slot(wide / G), hd);
        if (G <= kSimtSmallTile)
            t.ws = std::max(t.ws, rows_ws_bytes(rows_simt_ctas(sms, hd, kSimtSmallTile, 1), slot(kSimtSmallTile / G), hd));
    }
    return t;
}

static int check_group(int H, int KV, int hd) {
    const int most = hd <= 128 ? kRowsMaxGroup : kRowsMaxGroup / 2;
    if (H / KV > most) return attn_fail(SLM_EUNSUPPORTED, "%d query heads per kv head: at most %d at head_dim %d", H / KV, most, hd);
    return SLM_OK;
}

static std::atomic<int> g_lost{0};  // slm_debug_rows_faults

// The part that both attention calls share: workspace, kernel, join.
static int run_attention(RowsArgs &a, const RowsTiling &t, int dtype, long long longest, void *ws, size_t ws_bytes,
                         cudaStream_t s) {
    if (!ws || (uintptr_t)ws % 256) return attn_fail(SLM_EINVAL, "workspace must be non-NULL and 256-byte aligned");
    if (ws_bytes < t.ws) return attn_fail(SLM_EINVAL, "workspace of %zu bytes, %zu needed", ws_bytes, t.ws);
    a.ws = (uint8_t *)ws;
    a.P = t.P;
    a.slot_rows = t.slot_rows;
    a.geom = t.geom;
    // Items of a few blocks stay whole: cutting and joining them costs a short call 2 to 3 us, a block
    // about 1 us.  Whole / cut, bf16, tables of two blocks: one token, 9 / 3 heads of 64, 7.1 / 8.9 us,
    // 16 sequences 8.2 / 11.2; 32 / 8 heads of 128: 8.4 / 9.5 and 9.5 / 11.3; of four blocks 9.0 / 9.6,
    // 9.9 / 11.8, 11.2 / 9.8 and 12.0 / 13.9; of eight 12.9 / 10.2, 13.8 / 13.1, 17.2 / 11.0 and 18.3 /
    // 21.2.  `longest` is what the caller's table (for prompts: the packed rows) could hold, since the
    // lengths are not known here: a short context under a wide table is cut all the same (one token
    // over 250 positions, table for 32,768: 9.1 us).
    a.geom.split = longest > (long long)(on_tensor_cores(dtype, a.hd) ? 4 : 2) << t.geom.shift;
    a.G = a.H / a.KV;
    a.lost = g_lost.load(std::memory_order_relaxed);
    a.scale_log2 = (float)(1.4426950408889634074 / std::sqrt((double)a.hd));
    const bool bf16 = dtype == SLM_BF16;
    if (a.rows == 1) {  // one row: its stride has no meaning
        a.q_ld = a.out_ld = (long long)a.H * a.hd;
        a.kv.k_ld = a.kv.v_ld = (long long)a.KV * a.hd;
    }
    cudaError_t e = on_tensor_cores(dtype, a.hd) ? rows_tc_launch(a, s) : rows_simt_launch(a, bf16, s);
    if (e == cudaSuccess && a.geom.split) e = rows_join_launch(a, bf16, s);
    if (e != cudaSuccess) return launch_fail("attention", e);
    return SLM_OK;
}

}  // namespace slm

using namespace slm;

extern "C" int slm_kv_append(const slm_kv_cache *cache, const slm_rows *rows, int32_t dtype, const void *k, int64_t k_ld,
                             const void *v, int64_t v_ld, const float *rope, int32_t rope_len, int32_t n_heads,
                             const void *q, int64_t q_ld, void *q_out, int64_t q_out_ld, int32_t *status,
                             void *stream) {
    int rc;
    if ((rc = check_cache(cache)) || (rc = check_rows(rows)) || (rc = check_dtype(dtype, "dtype"))) return rc;
    const int KV = cache->n_kv_heads, hd = cache->head_dim;
    if ((rc = check_packed(k, k_ld, KV, hd, dtype, rows->rows, "k")) ||
        (rc = check_packed(v, v_ld, KV, hd, dtype, rows->rows, "v")) || (rc = check_status(status)))
        return rc;
    if (q || q_out) {
        if ((rc = check_heads(n_heads, KV, hd)) || (rc = check_packed(q, q_ld, n_heads, hd, dtype, rows->rows, "q")) ||
            (rc = check_packed(q_out, q_out_ld, n_heads, hd, cache->kv_dtype, rows->rows, "q_out")))
            return rc;
        if (q == q_out && (dtype != cache->kv_dtype || (rows->rows > 1 && q_ld != q_out_ld)))
            return attn_fail(SLM_EINVAL, "q can be rotated in place only in the cache's type, with one row stride");
    }
    if (rope && ((uintptr_t)rope % 16 || rope_len < 1))
        return attn_fail(SLM_EINVAL, "rope must be 16-byte aligned and hold at least one position");
    int dev = 0;
    const int sms = current_sms(dev);
    if (sms < 0) return sms;
    const PtrCheck ptrs[] = {{cache->k, "the cache's k"}, {cache->v, "the cache's v"}, {cache->page_table, "page_table"},
                             {rows->row_start, "row_start"}, {rows->ctx_len, "ctx_len"}, {k, "k"}, {v, "v"},
                             {rope, "rope"}, {q, "q"}, {q_out, "q_out"}, {status, "status"}};
    if ((rc = check_pointers(dev, ptrs, sizeof ptrs / sizeof *ptrs))) return rc;
    if (rows->rows == 0) return SLM_OK;
    AppendArgs a{};
    a.row_start = rows->row_start;
    a.ctx_len = rows->ctx_len;
    a.nseq = rows->nseq;
    a.rows = rows->rows;
    a.H = q ? n_heads : 0;
    a.KV = KV;
    a.hd = hd;
    a.cap = cache_cap(cache);
    a.q = (const uint8_t *)q;
    a.k = (const uint8_t *)k;
    a.v = (const uint8_t *)v;
    a.q_out = (uint8_t *)q_out;
    a.kc = (uint8_t *)cache->k;
    a.vc = (uint8_t *)cache->v;
    a.q_ld = q_ld;
    a.k_ld = k_ld;
    a.v_ld = v_ld;
    a.q_out_ld = q_out_ld;
    a.rope = rope;
    a.rope_len = rope_len;
    a.table = cache->page_table;
    a.table_ld = cache->table_ld;
    a.n_pages = cache->n_pages;
    a.page_shift = log2i(cache->page_size);
    a.status = status;
    const cudaError_t e = rows_append_launch(a, dtype == SLM_BF16, cache->kv_dtype == SLM_BF16, (cudaStream_t)stream);
    if (e != cudaSuccess) return launch_fail("append", e);
    return SLM_OK;
}

extern "C" size_t slm_attention_rows_workspace_bytes(int32_t dtype, int32_t rows, int32_t nseq, int32_t n_heads,
                                                     int32_t n_kv_heads, int32_t head_dim) {
    if (rows < 0 || rows > kRowsMaxRows || nseq < 1 || nseq > kRowsMaxSeqs || check_dtype(dtype, "dtype") || check_heads(n_heads, n_kv_heads, head_dim) ||
        check_group(n_heads, n_kv_heads, head_dim))
        return 0;
    int dev = 0;
    const int sms = current_sms(dev);
    return sms < 0 ? 0 : rows_tiling(sms, dtype, rows, nseq, n_heads, n_kv_heads, head_dim).ws;
}

extern "C" int slm_attention_paged(const slm_kv_cache *cache, const slm_rows *rows, int32_t n_heads, const void *q,
                                   int64_t q_ld, void *out, int64_t out_ld, void *workspace, size_t workspace_bytes,
                                   int32_t *status, void *stream) {
    int rc;
    if ((rc = check_cache(cache)) || (rc = check_rows(rows))) return rc;
    const int KV = cache->n_kv_heads, hd = cache->head_dim, dtype = cache->kv_dtype;
    if ((rc = check_heads(n_heads, KV, hd)) || (rc = check_group(n_heads, KV, hd)) ||
        (rc = check_packed(q, q_ld, n_heads, hd, dtype, rows->rows, "q")) ||
        (rc = check_packed(out, out_ld, n_heads, hd, dtype, rows->rows, "out")) || (rc = check_status(status)))
        return rc;
    int dev = 0;
    const int sms = current_sms(dev);
    if (sms < 0) return sms;
    const PtrCheck ptrs[] = {{cache->k, "the cache's k"}, {cache->v, "the cache's v"}, {cache->page_table, "page_table"},
                             {rows->row_start, "row_start"}, {rows->ctx_len, "ctx_len"}, {q, "q"}, {out, "out"},
                             {workspace, "workspace"}, {status, "status"}};
    if ((rc = check_pointers(dev, ptrs, sizeof ptrs / sizeof *ptrs))) return rc;
    if (rows->rows == 0) return SLM_OK;
    RowsArgs a{};
    a.row_start = rows->row_start;
    a.ctx_len = rows->ctx_len;
    a.nseq = rows->nseq;
    a.rows = rows->rows;
    a.H = n_heads;
    a.KV = KV;
    a.hd = hd;
    a.cap = cache_cap(cache);
    a.q = (const uint8_t *)q;
    a.out = (uint8_t *)out;
    a.q_ld = q_ld;
    a.out_ld = out_ld;
    a.kv.k = (const uint8_t *)cache->k;
    a.kv.v = (const uint8_t *)cache->v;
    a.kv.table = cache->page_table;
    a.kv.table_ld = cache->table_ld;
    a.kv.n_pages = cache->n_pages;
    a.kv.page_shift = log2i(cache->page_size);
    a.status = status;
    return run_attention(a, rows_tiling(sms, dtype, rows->rows, rows->nseq, n_heads, KV, hd), dtype, a.cap, workspace,
                         workspace_bytes, (cudaStream_t)stream);
}

extern "C" int slm_attention_prompt(const slm_rows *rows, int32_t dtype, int32_t n_heads, int32_t n_kv_heads,
                                    int32_t head_dim, const void *q, int64_t q_ld, const void *k, int64_t k_ld,
                                    const void *v, int64_t v_ld, void *out, int64_t out_ld, void *workspace,
                                    size_t workspace_bytes, int32_t *status, void *stream) {
    int rc;
    if ((rc = check_rows(rows)) || (rc = check_dtype(dtype, "dtype")) || (rc = check_heads(n_heads, n_kv_heads, head_dim)) ||
        (rc = check_group(n_heads, n_kv_heads, head_dim)))
        return rc;
    if (rows->ctx_len) return attn_fail(SLM_EINVAL, "ctx_len must be NULL: a whole prompt has no cached positions");
    if ((rc = check_packed(q, q_ld, n_heads, head_dim, dtype, rows->rows, "q")) ||
        (rc = check_packed(k, k_ld, n_kv_heads, head_dim, dtype, rows->rows, "k")) ||
        (rc = check_packed(v, v_ld, n_kv_heads, head_dim, dtype, rows->rows, "v")) ||
        (rc = check_packed(out, out_ld, n_heads, head_dim, dtype, rows->rows, "out")) || (rc = check_status(status)))
        return rc;
    int dev = 0;
    const int sms = current_sms(dev);
    if (sms < 0) return sms;
    const PtrCheck ptrs[] = {{rows->row_start, "row_start"}, {q, "q"}, {k, "k"}, {v, "v"}, {out, "out"},
                             {workspace, "workspace"}, {status, "status"}};
    if ((rc = check_pointers(dev, ptrs, sizeof ptrs / sizeof *ptrs))) return rc;
    if (rows->rows == 0) return SLM_OK;
    RowsArgs a{};
    a.row_start = rows->row_start;
    a.nseq = rows->nseq;
    a.rows = rows->rows;
    a.H = n_heads;
    a.KV = n_kv_heads;
    a.hd = head_dim;
    a.cap = rows->rows;
    a.q = (const uint8_t *)q;
    a.out = (uint8_t *)out;
    a.q_ld = q_ld;
    a.out_ld = out_ld;
    a.kv.k = (const uint8_t *)k;
    a.kv.v = (const uint8_t *)v;
    a.kv.k_ld = k_ld;
    a.kv.v_ld = v_ld;
    a.status = status;
    return run_attention(a, rows_tiling(sms, dtype, rows->rows, rows->nseq, n_heads, n_kv_heads, head_dim), dtype, rows->rows,
                         workspace, workspace_bytes, (cudaStream_t)stream);
}

extern "C" int slm_debug_rows_faults(int32_t lost) {
    if (lost < 0 || lost > 2) return attn_fail(SLM_EINVAL, "lost %d outside [0, 2]", lost);
    g_lost.store(lost);
    return SLM_OK;
}
