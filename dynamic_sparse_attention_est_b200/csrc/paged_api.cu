// paged_api.cu -- the extern "C" entry points of the paged key/value cache:
// argument checks, workspace carving and launches.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "internal.h"
#include "paged.cuh"

namespace minf {

namespace {

int bad(int code, const char *fmt, ...) {
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return api_fail(code, buf);
}

int launch_result(cudaError_t e, const char *what) {
    if (e == cudaSuccess) return MINF_OK;
    return bad(MINF_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// The caller's current device, put back when the call ends.
struct DeviceScope {
    int dev = -1;
    DeviceScope() {
        if (cudaGetDevice(&dev) != cudaSuccess) {
            cudaGetLastError();
            dev = -1;
        }
    }
    ~DeviceScope() {
        if (dev >= 0 && cudaSetDevice(dev) != cudaSuccess) cudaGetLastError();
    }
};

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

size_t round_up(size_t x) { return (x + 255) & ~size_t(255); }

int check_shape(int dtype, int hq, int hkv, int d) {
    if (dtype != MINF_BF16 && dtype != MINF_FP16) return bad(MINF_ERR_UNSUPPORTED, "data type %d (bf16 or fp16)", dtype);
    if (hq <= 0 || hkv <= 0 || hq % hkv != 0) return bad(MINF_ERR_INVALID, "bad head counts hq=%d hkv=%d", hq, hkv);
    if (hq > MINF_MAX_HEADS) return bad(MINF_ERR_INVALID, "hq=%d above %d", hq, MINF_MAX_HEADS);
    if (hq / hkv > 128) return bad(MINF_ERR_UNSUPPORTED, "%d query heads to a kv-head (at most 128)", hq / hkv);
    if (d != kD) return bad(MINF_ERR_UNSUPPORTED, "head dimension %d (only 128)", d);
    return MINF_OK;
}

int check_seqs(const minf_paged_seqs *s, PagedSeqs &S, int hq) {
    if (!s) return bad(MINF_ERR_INVALID, "null sequence description");
    if (s->n_seqs < 0 || s->total < 0 || s->max_q < 0 || s->num_pages < 0)
        return bad(MINF_ERR_INVALID, "negative count in the sequence description");
    if (s->page_size != 16 && s->page_size != 32 && s->page_size != 64 && s->page_size != 128)
        return bad(MINF_ERR_UNSUPPORTED, "page size %d (16, 32, 64 or 128)", s->page_size);
    if (s->n_seqs > kMaxSeqs) return bad(MINF_ERR_UNSUPPORTED, "%d sequences (at most %d)", s->n_seqs, kMaxSeqs);
    S = PagedSeqs{};
    S.n_seqs = s->n_seqs;
    S.total = s->total;
    S.page = s->page_size;
    S.page_log2 = S.page == 16 ? 4 : S.page == 32 ? 5 : S.page == 64 ? 6 : 7;
    if (s->n_seqs == 0 || s->total == 0) return MINF_OK;  // nothing to do
    if (!s->cu_q || !s->kv_lens || !s->block_tables) return bad(MINF_ERR_INVALID, "null cu_q, kv_lens or block_tables");
    if (s->width < 1 || s->num_pages < 1) return bad(MINF_ERR_INVALID, "width=%d num_pages=%d", s->width, s->num_pages);
    if (s->table_stride < s->width) return bad(MINF_ERR_INVALID, "block_tables rows overlap");
    if ((long long)s->width * s->page_size > (1ll << 30))
        return bad(MINF_ERR_UNSUPPORTED, "block tables of %d pages of %d tokens", s->width, s->page_size);
    if (s->max_q < 1 || s->max_q > s->total) return bad(MINF_ERR_INVALID, "max_q=%d of %d tokens", s->max_q, s->total);
    if ((long long)s->total * hq > (1ll << 30)) return bad(MINF_ERR_UNSUPPORTED, "%d tokens in a call", s->total);
    S.cu_q = s->cu_q;
    S.kv_lens = s->kv_lens;
    S.tables = s->block_tables;
    S.tstride = s->table_stride;
    S.width = s->width;
    S.max_q = s->max_q;
    S.num_pages = s->num_pages;
    return MINF_OK;
}

// Longest page list: no table names more pages (2^30 tokens in pages of 16), and its
// entries times the 16-key groups of a page fit 31 bits.
constexpr int kMaxTopk = 1 << 26;

// [tokens][heads][128] rows: 16-byte rows and strides; written ones must not overlap.
int check_rows(const minf_rows *r, const char *name, int total, int heads, bool written) {
    if (!r || !r->data) return bad(MINF_ERR_INVALID, "null %s", name);
    if (!aligned16(r->data)) return bad(MINF_ERR_INVALID, "%s not 16-byte aligned", name);
    const long long ts = r->token_stride, hs = r->head_stride;
    const long long most = 1ll << 38;  // tensor maps take byte strides below 2^40
    if ((total > 1 && (ts <= 0 || ts > most || ts % 8)) || (heads > 1 && (hs <= 0 || hs > most || hs % 8)))
        return bad(MINF_ERR_INVALID, "%s strides must be positive multiples of 8 elements", name);
    if (written) {
        const bool token_major = (heads == 1 || hs >= kD) && (total == 1 || ts >= (heads - 1) * hs + kD);
        const bool head_major = (total == 1 || ts >= kD) && (heads == 1 || hs >= (total - 1) * ts + kD);
        if (!token_major && !head_major) return bad(MINF_ERR_INVALID, "%s rows overlap", name);
    }
    return MINF_OK;
}

int check_cache(const minf_paged_cache *c, int hkv, int page) {
    if (!c || !c->k || !c->v) return bad(MINF_ERR_INVALID, "null cache");
    if (!aligned16(c->k) || !aligned16(c->v)) return bad(MINF_ERR_INVALID, "cache not 16-byte aligned");
    const long long need = (long long)hkv * page * kD, most = 1ll << 38;
    if (c->k_page_stride < need || c->v_page_stride < need || c->k_page_stride % 8 || c->v_page_stride % 8 ||
        c->k_page_stride > most || c->v_page_stride > most)
        return bad(MINF_ERR_INVALID, "cache page strides must be multiples of 8 elements and cover a page");
    return MINF_OK;
}

// Query rows (tokens x group) up to which a call takes the streaming kernel: two of
// its 8-row tiles, one read of K and V.  32 sequences of 8K tokens, four q-heads to a
// kv-head: 16 rows 185 us streaming; 20 rows 196 us with the chunk kernel (which takes
// as long for one row as for 128) and 338 us streaming, which reads K and V twice.
constexpr int kStreamMaxRows = 16;
bool streams(int max_q, int group) { return (long long)max_q * group <= kStreamMaxRows; }

struct AttnSizes {
    size_t o, ml, plan, total;
};
AttnSizes attn_sizes(long long n_slots, int rows, long long n_plan) {
    AttnSizes z{};
    size_t off = MINF_STATUS_BYTES;
    z.o = off;
    off = round_up(off + (size_t)n_slots * rows * kD * sizeof(float));
    z.ml = off;
    off = round_up(off + (size_t)n_slots * rows * sizeof(float2));
    z.plan = off;
    off = round_up(off + (size_t)n_plan * sizeof(long long));
    z.total = off;
    return z;
}

AttnSizes dense_sizes(int n_seqs, int group, int max_q) {
    if (streams(max_q, group)) {
        const StreamPlan p = paged_stream_plan(group, max_q);
        return attn_sizes(p.n_slots, p.rows, n_seqs + 1);
    }
    const ChunkPlan p = paged_chunk_plan(group, max_q);
    return attn_sizes(p.n_slots, p.part_rows, n_seqs + 2);
}

AttnSizes sparse_sizes(const StreamPlan &p) { return attn_sizes(p.n_slots, p.rows, 0); }

size_t estimate_bytes(const EstimatePlan &p, size_t *top_at) {
    const size_t a = round_up(MINF_STATUS_BYTES + p.n_scores * sizeof(float));
    if (top_at) *top_at = a;
    return round_up(a + p.n_top * sizeof(float));
}

void place(PagedAttnParams &P, const AttnSizes &z, void *ws) {
    char *b = static_cast<char *>(ws);
    P.part_o = reinterpret_cast<float *>(b + z.o);
    P.part_ml = reinterpret_cast<float2 *>(b + z.ml);
    P.plan = reinterpret_cast<long long *>(b + z.plan);
    P.hdr = static_cast<WsHeader *>(ws);
    P.wait_limit_ns = api_wait_limit_ns();
}

int fill_attn(PagedAttnParams &P, const minf_paged_seqs *seqs, int dtype, int hq, int hkv, int d, const minf_rows *q,
              const minf_paged_cache *cache, float scale, const minf_rows *out, float *lse) {
    memset(&P, 0, sizeof(P));
    int rc = check_shape(dtype, hq, hkv, d);
    if (rc) return rc;
    if ((rc = check_seqs(seqs, P.seqs, hq))) return rc;
    if (!(scale > 0.f) || !std::isfinite(scale)) return bad(MINF_ERR_INVALID, "scale must be finite and > 0");
    if (P.seqs.n_seqs == 0 || P.seqs.total == 0) return MINF_OK;
    if ((rc = check_rows(q, "q", P.seqs.total, hq, false))) return rc;
    if ((rc = check_rows(out, "out", P.seqs.total, hq, true))) return rc;
    if ((rc = check_cache(cache, hkv, P.seqs.page))) return rc;
    P.q = q->data;
    P.q_ts = q->token_stride;
    P.q_hs = q->head_stride;
    P.out = out->data;
    P.o_ts = out->token_stride;
    P.o_hs = out->head_stride;
    P.lse = lse;
    P.k = cache->k;
    P.v = cache->v;
    P.kc_ps = cache->k_page_stride;
    P.vc_ps = cache->v_page_stride;
    P.hq = hq;
    P.hkv = hkv;
    P.group = hq / hkv;
    P.scale_log2 = scale * 1.4426950408889634f;
    return MINF_OK;
}

}  // namespace

cudaError_t make_tmap_4d(CUtensorMap *map, const void *base, bool fp16, const cuuint64_t (&dims)[4],
                         const cuuint64_t (&strides)[3], const cuuint32_t (&box)[4]) {
    if (!tmap_encoder()) return cudaErrorNotSupported;
    const cuuint32_t one[4] = {1, 1, 1, 1};
    const CUresult r = tmap_encoder()(
        map, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base),
        dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t make_tmap_pages(CUtensorMap *map, const void *base, bool fp16, int page, int hkv, int num_pages,
                            long long page_stride, int rows) {
    return make_tmap_4d(map, base, fp16, {kD, (cuuint64_t)page, (cuuint64_t)hkv, (cuuint64_t)num_pages},
                        {kD * 2, (cuuint64_t)page * kD * 2, (cuuint64_t)page_stride * 2},
                        {64, (cuuint32_t)rows, 1, 1});
}

}  // namespace minf

using namespace minf;

extern "C" {

size_t minf_paged_workspace_bytes(int op, int hq, int hkv, int total, int n_seqs, int max_q, int width, int topk) {
    if (hq <= 0 || hkv <= 0 || hq % hkv || hq / hkv > 128 || hq > MINF_MAX_HEADS || total < 0 || n_seqs < 0 ||
        n_seqs > kMaxSeqs || max_q < 0 || width < 0 || (long long)total * hq > (1ll << 30))
        return 0;
    if (total == 0 || n_seqs == 0) return MINF_STATUS_BYTES;
    if (max_q < 1 || max_q > total) return 0;
    switch (op) {
    case MINF_OP_PAGED_APPEND:
        return MINF_STATUS_BYTES;
    case MINF_OP_PAGED_ATTENTION:
        return dense_sizes(n_seqs, hq / hkv, max_q).total;
    case MINF_OP_PAGED_BLOCK_ESTIMATE:
        if (topk < 1 || width < 1 || width > kMaxBlocks) return 0;
        return estimate_bytes(paged_estimate_reserve(total, hkv, width), nullptr);
    case MINF_OP_PAGED_BLOCK_ATTENTION:
        if (topk < 1 || topk > kMaxTopk) return 0;
        return sparse_sizes(paged_sparse_reserve(total, hkv, hq / hkv, topk)).total;
    }
    return 0;
}

int minf_paged_append(const minf_paged_seqs *seqs, int dtype, int hq, int hkv, int d, const minf_rows *k,
                      const minf_rows *v, const minf_rows *q, const minf_rows *q_out, const minf_paged_cache *cache,
                      void *k_bounds, const float *rope, int rope_rows, int rot, int interleaved, void *ws,
                      size_t ws_bytes, minf_stream_t stream) {
    AppendParams P;
    memset(&P, 0, sizeof(P));
    int rc = check_shape(dtype, hq, hkv, d);
    if (rc) return rc;
    if ((rc = check_seqs(seqs, P.seqs, hq))) return rc;
    if (rope) {
        if (rot < 16 || rot > kD || rot % 16 != 0) return bad(MINF_ERR_UNSUPPORTED, "rotated width %d (16, 32 .. 128)", rot);
        if (rope_rows < 1) return bad(MINF_ERR_INVALID, "rope_rows=%d", rope_rows);
        if (!aligned16(rope)) return bad(MINF_ERR_INVALID, "rope not 16-byte aligned");
    }
    if ((q == nullptr) != (q_out == nullptr)) return bad(MINF_ERR_INVALID, "q and q_out go together");
    if ((rc = api_check_ws(ws, ws_bytes, MINF_STATUS_BYTES))) return rc;
    const PagedSeqs &S = P.seqs;
    if (S.n_seqs == 0 || S.total == 0) return MINF_OK;
    if ((rc = check_rows(k, "k", S.total, hkv, false))) return rc;
    if ((rc = check_rows(v, "v", S.total, hkv, false))) return rc;
    if ((rc = check_cache(cache, hkv, S.page))) return rc;
    if (q) {
        if ((rc = check_rows(q, "q", S.total, hq, false))) return rc;
        if ((rc = check_rows(q_out, "q_out", S.total, hq, true))) return rc;
        P.q = q->data;
        P.q_ts = q->token_stride;
        P.q_hs = q->head_stride;
        P.q_out = q_out->data;
        P.qo_ts = q_out->token_stride;
        P.qo_hs = q_out->head_stride;
    }
    if (k_bounds && !aligned16(k_bounds)) return bad(MINF_ERR_INVALID, "k_bounds not 16-byte aligned");
    P.k = k->data;
    P.k_ts = k->token_stride;
    P.k_hs = k->head_stride;
    P.v = v->data;
    P.v_ts = v->token_stride;
    P.v_hs = v->head_stride;
    P.k_cache = cache->k;
    P.v_cache = cache->v;
    P.kc_ps = cache->k_page_stride;
    P.vc_ps = cache->v_page_stride;
    P.k_bounds = k_bounds;
    P.rope = rope;
    P.rope_rows = rope_rows;
    P.rot = rope ? rot : 0;
    P.hq = hq;
    P.hkv = hkv;
    P.hdr = static_cast<WsHeader *>(ws);
    const DeviceScope scope;
    if ((rc = api_select_device(cache->k))) return rc;
    return launch_result(run_paged_append(P, dtype == MINF_FP16, interleaved != 0, (cudaStream_t)stream),
                         "paged append launch");
}

int minf_paged_attention(const minf_paged_seqs *seqs, int dtype, int hq, int hkv, int d, const minf_rows *q,
                         const minf_paged_cache *cache, float scale, const minf_rows *out, float *lse, void *ws,
                         size_t ws_bytes, minf_stream_t stream) {
    PagedAttnParams P;
    int rc = fill_attn(P, seqs, dtype, hq, hkv, d, q, cache, scale, out, lse);
    if (rc) return rc;
    const PagedSeqs &S = P.seqs;
    const bool none = S.n_seqs == 0 || S.total == 0;
    const AttnSizes z = none ? AttnSizes{0, 0, 0, MINF_STATUS_BYTES} : dense_sizes(S.n_seqs, P.group, S.max_q);
    if ((rc = api_check_ws(ws, ws_bytes, z.total))) return rc;
    if (none) return MINF_OK;
    place(P, z, ws);
    const DeviceScope scope;
    if ((rc = api_select_device(cache->k))) return rc;
    if (streams(S.max_q, P.group)) {
        const StreamPlan p = paged_stream_plan(P.group, S.max_q);
        P.n_slots = p.n_slots;
        return launch_result(run_paged_stream(P, dtype == MINF_FP16, p.rows, (cudaStream_t)stream),
                             "paged attention launch");
    }
    const ChunkPlan p = paged_chunk_plan(P.group, S.max_q);
    P.n_slots = p.n_slots;
    return launch_result(run_paged_chunk(P, dtype == MINF_FP16, p.part_rows, (cudaStream_t)stream),
                         "paged attention launch");
}

int minf_paged_block_estimate(const minf_paged_seqs *seqs, int dtype, int hq, int hkv, int d, const minf_rows *q,
                              const void *k_bounds, int topk, int32_t *blk_idx, int32_t *blk_cnt, void *ws,
                              size_t ws_bytes, minf_stream_t stream) {
    EstimateParams P;
    memset(&P, 0, sizeof(P));
    int rc = check_shape(dtype, hq, hkv, d);
    if (rc) return rc;
    if ((rc = check_seqs(seqs, P.seqs, hq))) return rc;
    if (topk < 1) return bad(MINF_ERR_INVALID, "topk must be >= 1");
    const PagedSeqs &S = P.seqs;
    if (S.n_seqs == 0 || S.total == 0) return api_check_ws(ws, ws_bytes, MINF_STATUS_BYTES);
    if (S.width > kMaxBlocks) return bad(MINF_ERR_UNSUPPORTED, "more than %d blocks", kMaxBlocks);
    if ((rc = check_rows(q, "q", S.total, hq, false))) return rc;
    if (!k_bounds || !aligned16(k_bounds)) return bad(MINF_ERR_INVALID, "null or unaligned k_bounds");
    if (!blk_idx || !blk_cnt) return bad(MINF_ERR_INVALID, "null blk_idx or blk_cnt");
    const EstimatePlan p = paged_estimate_plan(S.total, S.n_seqs, hkv, S.width);
    size_t top_at = 0;
    if ((rc = api_check_ws(ws, ws_bytes, estimate_bytes(p, &top_at)))) return rc;
    P.q = q->data;
    P.q_ts = q->token_stride;
    P.q_hs = q->head_stride;
    P.bounds = k_bounds;
    P.hq = hq;
    P.hkv = hkv;
    P.group = hq / hkv;
    P.topk = topk;
    P.blk_idx = blk_idx;
    P.blk_cnt = blk_cnt;
    P.scores = reinterpret_cast<float *>(static_cast<char *>(ws) + MINF_STATUS_BYTES);
    P.top = reinterpret_cast<float *>(static_cast<char *>(ws) + top_at);
    P.score_stride = p.score_stride;
    P.batch = p.batch;
    P.hdr = static_cast<WsHeader *>(ws);
    P.wait_limit_ns = api_wait_limit_ns();
    const DeviceScope scope;
    if ((rc = api_select_device(k_bounds))) return rc;
    return launch_result(run_paged_estimate(P, dtype == MINF_FP16, (cudaStream_t)stream), "paged estimate launch");
}

int minf_paged_block_attention(const minf_paged_seqs *seqs, int dtype, int hq, int hkv, int d, const minf_rows *q,
                               const minf_paged_cache *cache, float scale, const int32_t *blk_idx,
                               const int32_t *blk_cnt, int topk, const minf_rows *out, float *lse, void *ws,
                               size_t ws_bytes, minf_stream_t stream) {
    PagedAttnParams P;
    int rc = fill_attn(P, seqs, dtype, hq, hkv, d, q, cache, scale, out, lse);
    if (rc) return rc;
    if (topk < 1) return bad(MINF_ERR_INVALID, "topk must be >= 1");
    if (topk > kMaxTopk) return bad(MINF_ERR_UNSUPPORTED, "topk=%d above %d", topk, kMaxTopk);
    const PagedSeqs &S = P.seqs;
    if (S.n_seqs == 0 || S.total == 0) return api_check_ws(ws, ws_bytes, MINF_STATUS_BYTES);
    if (!blk_idx || !blk_cnt) return bad(MINF_ERR_INVALID, "null blk_idx or blk_cnt");
    const StreamPlan p = paged_sparse_plan(S.total, hkv, P.group, topk, S.page);
    const AttnSizes z = sparse_sizes(p);
    if ((rc = api_check_ws(ws, ws_bytes, z.total))) return rc;
    place(P, z, ws);
    P.blk_idx = blk_idx;
    P.blk_cnt = blk_cnt;
    P.topk = topk;
    P.n_slots = p.n_slots;
    const DeviceScope scope;
    if ((rc = api_select_device(cache->k))) return rc;
    return launch_result(run_paged_sparse(P, dtype == MINF_FP16, p.rows, (cudaStream_t)stream),
                         "paged block attention launch");
}

}  // extern "C"
