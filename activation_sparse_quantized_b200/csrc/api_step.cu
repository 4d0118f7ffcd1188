// api_step.cu -- the extern "C" entry points around the projections: cache
// plan, cache store, tree attention and residual norm (include/sgq.h).
// Host-side argument checks, then the launches on the caller's stream. Nothing
// here allocates, frees or synchronises.
#include "sgq_launch.h"

#include <cmath>
#include <cuda_runtime.h>

namespace {

bool aligned16(const void *p)
{
    return ((uintptr_t)p & 15u) == 0;
}

int finish(cudaError_t e)
{
    return e == cudaSuccess ? SGQ_OK : sgq::record_cuda_error(e);
}

constexpr long long kMaxStride = 1ll << 40;      // elements
constexpr long long kMaxCacheStride = 1ll << 38; // elements; a tensor map takes less than 2^40 bytes

// A row stride of 2- or 4-byte elements: rows start on 16 bytes and do not overlap.
bool stride_ok(long long ld, long long width, int elem_bytes)
{
    return ld >= width && ld <= kMaxStride && (ld * elem_bytes) % 16 == 0;
}

int check_cache(const sgq_cache *c)
{
    if (!c)
        return SGQ_ERR_NULL;
    if (c->type != SGQ_TYPE_BF16 && c->type != SGQ_TYPE_E4M3)
        return SGQ_ERR_TYPE;
    if ((c->dim != 64 && c->dim != 128) || c->heads < 1 || c->heads > 65536 || c->page < 1 ||
        c->page > (1 << 20) || c->num_pages < 1)
        return SGQ_ERR_SHAPE;
    const long long unit = c->type == SGQ_TYPE_E4M3 ? 16 : 8; // elements in 16 bytes
    if (c->page_stride < 0 || c->slot_stride < 0 || c->head_stride < 0 ||
        c->page_stride > kMaxCacheStride || c->slot_stride > kMaxCacheStride ||
        c->head_stride > kMaxCacheStride)
        return SGQ_ERR_SHAPE;
    if (c->page_stride % unit || c->slot_stride % unit || c->head_stride % unit)
        return SGQ_ERR_ALIGN;
    // a dimension of more than one entry steps over at least one row of dim elements
    // (that no two of them share elements otherwise is the caller's)
    if ((c->heads > 1 && c->head_stride < c->dim) || (c->page > 1 && c->slot_stride < c->dim) ||
        (c->num_pages > 1 && c->page_stride < c->dim))
        return SGQ_ERR_SHAPE;
    if (c->type == SGQ_TYPE_BF16 ? (c->k_scale != 1.0f || c->v_scale != 1.0f)
                                 : !(c->k_scale > 0.0f && c->k_scale < 3e38f && c->v_scale > 0.0f &&
                                     c->v_scale < 3e38f))
        return SGQ_ERR_SHAPE;
    if (!c->k || !c->v)
        return SGQ_ERR_NULL;
    if (!aligned16(c->k) || !aligned16(c->v))
        return SGQ_ERR_ALIGN;
    return SGQ_OK;
}

int tree_attn(const void *q, long long ld_q, int T, int R, int Hq, const int32_t *lens,
              const int32_t *cu_new, const int32_t *table, int table_ld,
              const sgq_cache *cache_host, const uint32_t *tree, int tree_words,
              float scale, void *out, long long ld_out, float *lse, void *workspace,
              size_t ws_bytes, int32_t *status, void *stream, int withhold)
{
    int rc = check_cache(cache_host);
    if (rc)
        return rc;
    if (R < 1 || R > SGQ_MAX_REQUESTS)
        return SGQ_ERR_BATCH;
    const long long D = cache_host->dim, Hkv = cache_host->heads;
    if (T < 1 || Hq < Hkv || Hq % Hkv != 0 || table_ld < 1 ||
        (long long)table_ld * cache_host->page > (1ll << 30) ||
        Hq > 32768 || (long long)T * Hq > 0x7fffffffll || (tree && (tree_words < 1 || tree_words > (1 << 25))) ||
        !(fabsf(scale) * cache_host->k_scale <= 1e37f)) // (not a number: refused)
        return SGQ_ERR_SHAPE;
    if (!q || !lens || !cu_new || !table || !out || !workspace)
        return SGQ_ERR_NULL;
    if (!aligned16(q) || !aligned16(out) || !aligned16(workspace))
        return SGQ_ERR_ALIGN;
    if (!stride_ok(ld_q, Hq * D, 2) || !stride_ok(ld_out, Hq * D, 2))
        return SGQ_ERR_SHAPE;
    if (ws_bytes < sgq::attn_workspace_bytes(T, R, Hq, (int)Hkv, (int)D))
        return SGQ_ERR_WORKSPACE;
    const int sms = sgq::current_device_sms();
    if (sms < 0)
        return sms;
    sgq::AttnProblem p{};
    p.q = static_cast<const uint16_t *>(q);
    p.lens = lens;
    p.cu_new = cu_new;
    p.table = table;
    p.tree = tree;
    p.out = static_cast<uint16_t *>(out);
    p.lse = lse;
    p.workspace = workspace;
    p.status = status;
    p.ld_q = ld_q;
    p.ld_out = ld_out;
    p.T = T;
    p.R = R;
    p.Hq = Hq;
    p.table_ld = table_ld;
    p.tree_words = tree_words;
    p.scale = scale;
    p.cache = *cache_host;
    p.debug_withhold_scores = withhold;
    return finish(sgq::launch_attn(p, sms, static_cast<cudaStream_t>(stream)));
}

} // namespace

extern "C" {

int sgq_cache_plan(const int32_t *lens, const int32_t *news, int R, int page, int num_pages,
                   int32_t *table, int table_ld, const int32_t *held, int32_t *held_out,
                   const int32_t *free_pages, const int32_t *free_count,
                   int32_t *free_count_out, const int32_t *depth, int max_tokens,
                   int32_t *cu_new, int64_t *slots, int32_t *pos, int32_t *req,
                   int32_t *status, void *stream)
{
    if (R < 1 || R > SGQ_MAX_REQUESTS)
        return SGQ_ERR_BATCH;
    if (page < 1 || page > (1 << 20) || num_pages < 1 || table_ld < 1 ||
        (long long)table_ld * page > (1ll << 30) || max_tokens < 1 || max_tokens > (1 << 30))
        return SGQ_ERR_SHAPE;
    if (!lens || !news || !table || !held || !held_out || !free_pages || !free_count ||
        !free_count_out || !cu_new || !slots)
        return SGQ_ERR_NULL;
    const int sms = sgq::current_device_sms();
    if (sms < 0)
        return sms;
    sgq::PlanProblem p{};
    p.lens = lens;
    p.news = news;
    p.held = held;
    p.free_pages = free_pages;
    p.free_count = free_count;
    p.depth = depth;
    p.table = table;
    p.held_out = held_out;
    p.free_count_out = free_count_out;
    p.cu_new = cu_new;
    p.pos = pos;
    p.req = req;
    p.status = status;
    p.slots = slots;
    p.R = R;
    p.page = page;
    p.num_pages = num_pages;
    p.table_ld = table_ld;
    p.max_tokens = max_tokens;
    return finish(sgq::launch_plan(p, sms, static_cast<cudaStream_t>(stream)));
}

int sgq_cache_write(const void *q, long long ld_q, const void *k, long long ld_k, const void *v,
                    long long ld_v, int T, const int32_t *n_tokens, int Hq, const int32_t *pos,
                    const float *rope, int rope_len, const int64_t *slots, void *q_out,
                    long long ld_qo, const sgq_cache *cache_host, int32_t *status,
                    void *stream)
{
    int rc = check_cache(cache_host);
    if (rc)
        return rc;
    const long long D = cache_host->dim, Hkv = cache_host->heads;
    if (T < 1 || (q && (Hq < 1 || Hq > 65536)))
        return SGQ_ERR_SHAPE;
    if (!k || !v || !slots || (q && !q_out) || (rope && !pos))
        return SGQ_ERR_NULL;
    if (!aligned16(k) || !aligned16(v) || (q && (!aligned16(q) || !aligned16(q_out))) ||
        (rope && !aligned16(rope)))
        return SGQ_ERR_ALIGN;
    if (!stride_ok(ld_k, Hkv * D, 2) || !stride_ok(ld_v, Hkv * D, 2) ||
        (q && (!stride_ok(ld_q, Hq * D, 2) || !stride_ok(ld_qo, Hq * D, 2))) ||
        (rope && rope_len < 1))
        return SGQ_ERR_SHAPE;
    const int sms = sgq::current_device_sms();
    if (sms < 0)
        return sms;
    sgq::WriteProblem p{};
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.n_tokens = n_tokens;
    p.pos = pos;
    p.rope = rope;
    p.slots = slots;
    p.q_out = static_cast<uint16_t *>(q_out);
    p.status = status;
    p.ld_q = ld_q;
    p.ld_k = ld_k;
    p.ld_v = ld_v;
    p.ld_qo = ld_qo;
    p.T = T;
    p.Hq = q ? Hq : 0;
    p.rope_len = rope_len;
    p.cache = *cache_host;
    return finish(sgq::launch_write(p, sms, static_cast<cudaStream_t>(stream)));
}

size_t sgq_tree_attn_workspace_bytes(int T, int R, int Hq, int Hkv, int D)
{
    if (T < 1 || R < 1 || R > SGQ_MAX_REQUESTS || Hkv < 1 || Hq < Hkv || Hq > 32768 || Hq % Hkv != 0 ||
        (D != 64 && D != 128))
        return 0;
    // Fewer requests have more rows each and may need a larger row tile: what T rows of
    // one request need is enough for up to T rows of any number.
    return sgq::attn_workspace_bytes(T, 1, Hq, Hkv, D);
}

int sgq_tree_attn(const void *q, long long ld_q, int T, int R, int Hq, const int32_t *lens,
                  const int32_t *cu_new, const int32_t *table, int table_ld,
                  const sgq_cache *cache_host, const uint32_t *tree, int tree_words,
                  float scale, void *out, long long ld_out, float *lse, void *workspace,
                  size_t ws_bytes, int32_t *status, void *stream)
{
    return tree_attn(q, ld_q, T, R, Hq, lens, cu_new, table, table_ld, cache_host, tree, tree_words, scale, out, ld_out, lse,
                     workspace, ws_bytes, status, stream, 0);
}

int sgq_debug_tree_attn_withhold(const void *q, long long ld_q, int T, int R, int Hq, const int32_t *lens,
                                 const int32_t *cu_new, const int32_t *table, int table_ld,
                                 const sgq_cache *cache_host, const uint32_t *tree, int tree_words,
                                 float scale, void *out, long long ld_out, float *lse, void *workspace,
                                 size_t ws_bytes, int32_t *status, void *stream)
{
    return tree_attn(q, ld_q, T, R, Hq, lens, cu_new, table, table_ld, cache_host, tree, tree_words, scale, out, ld_out, lse,
                     workspace, ws_bytes, status, stream, 1);
}

int sgq_residual_norm(const void *a, long long ld_a, int a_type, const void *w_post,
                      const void *gate, long long ld_gate, float scale, const void *resid,
                      long long ld_r, int r_type, void *resid_out, long long ld_ro,
                      const void *w_pre, int w_type, float w_offset, void *x, long long ld_x,
                      int B, int H, float eps, void *stream)
{
    if ((a_type != SGQ_TYPE_BF16 && a_type != SGQ_TYPE_F32) ||
        (r_type != SGQ_TYPE_BF16 && r_type != SGQ_TYPE_F32) ||
        (w_type != SGQ_TYPE_BF16 && w_type != SGQ_TYPE_F32))
        return SGQ_ERR_TYPE;
    if (B < 1 || H < 8 || H % 8 != 0 || H > 32768 || !(eps >= 0.0f))
        return SGQ_ERR_SHAPE;
    // a block's result needs a residual to go to; without one there is only x
    if (!resid || (a && !resid_out) || (!a && (w_post || gate || !x)) || (x && !w_pre))
        return SGQ_ERR_NULL;
    if ((a && !aligned16(a)) || (w_post && !aligned16(w_post)) || (gate && !aligned16(gate)) ||
        !aligned16(resid) || (resid_out && !aligned16(resid_out)) ||
        (w_pre && !aligned16(w_pre)) || (x && !aligned16(x)))
        return SGQ_ERR_ALIGN;
    const int ab = a_type == SGQ_TYPE_F32 ? 4 : 2, rb = r_type == SGQ_TYPE_F32 ? 4 : 2;
    const int wb = w_type == SGQ_TYPE_F32 ? 4 : 2;
    if ((a && !stride_ok(ld_a, H, ab)) || !stride_ok(ld_r, H, rb) ||
        (resid_out && !stride_ok(ld_ro, H, rb)) || (x && !stride_ok(ld_x, H, 2)) ||
        (gate && ld_gate != 0 && !stride_ok(ld_gate, H, wb)))
        return SGQ_ERR_SHAPE;
    const int sms = sgq::current_device_sms();
    if (sms < 0)
        return sms;
    sgq::NormProblem p{};
    p.a = a;
    p.w_post = w_post;
    p.gate = gate;
    p.resid = resid;
    p.w_pre = w_pre;
    p.resid_out = a ? resid_out : nullptr;
    p.x = static_cast<uint16_t *>(x);
    p.ld_a = ld_a;
    p.ld_gate = ld_gate;
    p.ld_r = ld_r;
    p.ld_ro = ld_ro;
    p.ld_x = ld_x;
    p.a_type = a_type;
    p.r_type = r_type;
    p.w_type = w_type;
    p.B = B;
    p.H = H;
    p.scale = scale;
    p.w_offset = w_offset;
    p.eps = eps;
    return finish(sgq::launch_norm(p, sms, static_cast<cudaStream_t>(stream)));
}

} // extern "C"
