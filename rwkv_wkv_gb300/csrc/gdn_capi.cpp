// C-ABI entry points of the gated delta rule and of draft verification: checks
// and dispatch.  The public contract is documented in wkv7.h.
#include <cmath>
#include <new>

#include "gdn_internal.h"
#include "pool.h"

namespace {

bool head_size_ok(int32_t d) { return d == 64 || d == 128; }
bool dtype_ok(int32_t d) { return d == WKV7_F32 || d == WKV7_BF16; }

// Rows that are read: apart from each other, or one row for all (stride 0).
bool stride_ok(int64_t stride, int64_t row) { return stride == 0 || stride >= row; }

bool gdn_desc_valid(const wkv7_gdn_pool_desc *d) {
    return d && d->n_layers >= 1 && d->n_k_heads >= 1 && d->n_v_heads >= 1 && d->n_v_heads % d->n_k_heads == 0 &&
           d->head_k >= 1 && d->head_v >= 1 && d->n_slots >= 1 && d->n_snapshots >= 0 && dtype_ok(d->state_dtype) &&
           dtype_ok(d->out_dtype);
}

size_t gdn_slot_bytes(const wkv7_gdn_pool_desc *d) {
    return static_cast<size_t>(d->n_layers) * static_cast<size_t>(d->n_v_heads) * static_cast<size_t>(d->head_v) *
           static_cast<size_t>(d->head_k) * (d->state_dtype == WKV7_BF16 ? 2 : 4);
}

// The part of the description that the shared pool code reads.
wkv7_pool_desc plain_desc(const wkv7_gdn_pool_desc *d) {
    wkv7_pool_desc p{};
    p.n_layers = d->n_layers;
    p.n_heads = d->n_v_heads;
    p.head_size = d->head_v;
    p.n_slots = d->n_slots;
    p.n_snapshots = d->n_snapshots;
    p.device_buffer = d->device_buffer;
    p.buffer_bytes = d->buffer_bytes;
    p.state_dtype = d->state_dtype;
    p.out_dtype = d->out_dtype;
    return p;
}

wkv7::GdnView gdn_view(wkv7_pool *p, int32_t layer) {
    wkv7::GdnView lv;
    const wkv7_gdn_pool_desc &d = p->gdn_desc;
    lv.states = p->states;
    lv.snaps = p->snaps;
    lv.slot_stride = static_cast<long long>(d.n_layers) * d.n_v_heads * p->head_elems;
    lv.layer_off = static_cast<long long>(layer) * d.n_v_heads * p->head_elems;
    lv.n_slots = d.n_slots;
    lv.n_snaps = d.n_snapshots;
    lv.hk = d.n_k_heads;
    lv.hv = d.n_v_heads;
    lv.dk = d.head_k;
    lv.dv = d.head_v;
    lv.state_bf16 = p->state_bf16;
    lv.status = p->status;
    return lv;
}

// The checks of one call's tokens; `rows` > 0 of them are read.
wkv7_status check_tokens(const wkv7_pool *p, const wkv7_gdn_tokens *t, long long rows) {
    if (!t) return WKV7_ERR_INVALID_ARG;
    if (!dtype_ok(t->in_dtype)) return WKV7_ERR_INVALID_ARG;
    if (!(t->l2norm_eps >= 0.f) || std::isinf(t->l2norm_eps)) return WKV7_ERR_INVALID_ARG;
    if (rows == 0) return WKV7_OK;
    if (!t->q || !t->k || !t->v || !t->g || !t->beta || !t->o) return WKV7_ERR_INVALID_ARG;
    const wkv7_gdn_pool_desc &d = p->gdn_desc;
    const int64_t kw = static_cast<int64_t>(d.n_k_heads) * d.head_k, vw = static_cast<int64_t>(d.n_v_heads) * d.head_v;
    // one row alone never steps to the next, so its strides may be anything
    if (rows > 1 && (!stride_ok(t->q_stride, kw) || !stride_ok(t->k_stride, kw) || !stride_ok(t->v_stride, vw) ||
                     !stride_ok(t->g_stride, d.n_v_heads) || !stride_ok(t->beta_stride, d.n_v_heads)))
        return WKV7_ERR_INVALID_ARG;
    const int64_t esz = t->in_dtype == WKV7_BF16 ? 2 : 4;
    const void *bases[4] = {t->q, t->k, t->v, t->o};
    for (const void *b : bases)
        if (reinterpret_cast<uintptr_t>(b) % 16 != 0) return WKV7_ERR_UNSUPPORTED;
    if (reinterpret_cast<uintptr_t>(t->g) % 4 != 0 || reinterpret_cast<uintptr_t>(t->beta) % 4 != 0)
        return WKV7_ERR_UNSUPPORTED;
    if (rows > 1) {
        const int64_t strides[3] = {t->q_stride, t->k_stride, t->v_stride};
        for (int64_t s : strides)
            if (s * esz % 16 != 0) return WKV7_ERR_UNSUPPORTED;
    }
    return WKV7_OK;
}

wkv7::GdnTokens token_args(const wkv7_pool *p, const wkv7_gdn_tokens *t, long long rows) {
    wkv7::GdnTokens a;
    a.q = t->q;
    a.k = t->k;
    a.v = t->v;
    a.g = t->g;
    a.beta = t->beta;
    const wkv7_gdn_pool_desc &d = p->gdn_desc;
    const bool one = rows <= 1;  // a lone row's strides are never used: make them valid ones
    a.q_stride = one ? static_cast<long long>(d.n_k_heads) * d.head_k : t->q_stride;
    a.k_stride = one ? static_cast<long long>(d.n_k_heads) * d.head_k : t->k_stride;
    a.v_stride = one ? static_cast<long long>(d.n_v_heads) * d.head_v : t->v_stride;
    a.g_stride = one ? d.n_v_heads : t->g_stride;
    a.beta_stride = one ? d.n_v_heads : t->beta_stride;
    a.scale = t->scale;
    a.eps = t->l2norm_eps;
    a.bf16 = t->in_dtype == WKV7_BF16;
    a.o = t->o;
    a.o_bf16 = p->out_bf16;
    return a;
}

// The longest max_seqlen that runs token by token where the chunked kernel could.  A chunk of
// 64 costs the same however few of its tokens there are, and a token what its state's size says.
// Token by token against in chunks, us, 32 value heads: of 128, 1 sequence of 16 tokens 9.6 and 12.5, of
// 24 13.2 and 12.7; where they fill the 152 SMs, 16 sequences of 12 47 and 47, of 16 59 and 47; 64 of 12 171
// and 178, of 16 216 and 178.  Of 128 x 64 (64 x 128 within 10%), 1 of 16 9.3 and 11.8, of 24 12.4 and 11.7; 16 of 16
// 31 and 44, of 32 58 and 43; 64 of 16 110 and 158, of 32 207 and 162.  Of 64, 1 of 16 8.8 and 10.3, of
// 24 11.9 and 10.3; 16 of 32 34 and 37, of 48 49 and 37; 64 of 32 108 and 131, of 48 159 and 133.
// A checkpointed call always runs in chunks, so that a short tail resumed from a checkpoint
// repeats the long call's path.
int longest_by_token(const wkv7::GdnRunArgs &a) {
    if (a.cu_ckpt) return 0;
    if (static_cast<long long>(a.n) * a.lv.hv < 152) return 16;
    const int state = a.lv.dk * a.lv.dv;
    return state <= 64 * 64 ? 32 : state <= 64 * 128 ? 24 : 12;
}

}  // namespace

extern "C" {

size_t wkv7_gdn_pool_required_bytes(const wkv7_gdn_pool_desc *desc) {
    if (!gdn_desc_valid(desc)) return 0;
    const wkv7_pool_desc d = plain_desc(desc);
    return wkv7::pool_bytes(&d, gdn_slot_bytes(desc));
}

wkv7_status wkv7_gdn_pool_create(const wkv7_gdn_pool_desc *desc, wkv7_pool **out) {
    if (!out) return WKV7_ERR_INVALID_ARG;
    *out = nullptr;
    if (!gdn_desc_valid(desc)) return WKV7_ERR_INVALID_ARG;
    if (!head_size_ok(desc->head_k) || !head_size_ok(desc->head_v)) return WKV7_ERR_UNSUPPORTED;
    const size_t need = wkv7_gdn_pool_required_bytes(desc);
    if (desc->device_buffer) {
        if (desc->buffer_bytes < need) return WKV7_ERR_INVALID_ARG;
        if (reinterpret_cast<uintptr_t>(desc->device_buffer) % 256 != 0) return WKV7_ERR_INVALID_ARG;
    }
    wkv7_pool *p = new (std::nothrow) wkv7_pool();
    if (!p) return WKV7_ERR_NO_MEMORY;
    p->desc = plain_desc(desc);
    p->gdn = true;
    p->gdn_desc = *desc;
    p->head_elems = static_cast<long long>(desc->head_k) * desc->head_v;
    return wkv7::lay_out_pool(p, gdn_slot_bytes(desc), need, out);
}

wkv7_status wkv7_gdn_pool_get_desc(const wkv7_pool *pool, wkv7_gdn_pool_desc *out) {
    if (!pool || !out) return WKV7_ERR_INVALID_ARG;
    if (!pool->gdn) return WKV7_ERR_UNSUPPORTED;
    *out = pool->gdn_desc;
    out->device_buffer = pool->desc.device_buffer;
    out->buffer_bytes = pool->desc.buffer_bytes;
    return WKV7_OK;
}

wkv7_status wkv7_gdn_decode_step(wkv7_pool *pool, int32_t layer, const int32_t *slot_ids_dev, int32_t n,
                                 const wkv7_gdn_tokens *tokens, cudaStream_t stream) {
    if (!pool) return WKV7_ERR_INVALID_ARG;
    if (!pool->gdn) return WKV7_ERR_UNSUPPORTED;
    if (layer < 0 || layer >= pool->desc.n_layers || n < 0 || n > pool->desc.n_slots) return WKV7_ERR_INVALID_ARG;
    wkv7_status st = check_tokens(pool, tokens, n);
    if (st != WKV7_OK) return st;
    if (n == 0) return WKV7_OK;
    if (!slot_ids_dev) return WKV7_ERR_INVALID_ARG;
    wkv7::GdnDecodeArgs a;
    a.lv = gdn_view(pool, layer);
    a.in = token_args(pool, tokens, n);
    a.slot_ids = slot_ids_dev;
    a.n = n;
    int launches = 0;
    cudaError_t e = wkv7::launch_gdn_decode(a, stream, &launches);
    return wkv7::cuda_status("gdn_decode_step", e, launches);
}

wkv7_status wkv7_gdn_decode_multi(wkv7_pool *pool, int32_t layer, const int32_t *slot_ids_dev, int32_t n,
                                  int32_t n_tokens, const wkv7_gdn_tokens *tokens, const int32_t *step_snap_ids_dev,
                                  cudaStream_t stream) {
    if (!pool) return WKV7_ERR_INVALID_ARG;
    if (!pool->gdn) return WKV7_ERR_UNSUPPORTED;
    if (layer < 0 || layer >= pool->desc.n_layers || n < 0 || n > pool->desc.n_slots || n_tokens < 1)
        return WKV7_ERR_INVALID_ARG;
    const long long rows = static_cast<long long>(n) * n_tokens;
    if (rows > 0x7fffffffLL) return WKV7_ERR_INVALID_ARG;
    wkv7_status st = check_tokens(pool, tokens, rows);
    if (st != WKV7_OK) return st;
    if (step_snap_ids_dev && pool->desc.n_snapshots == 0) return WKV7_ERR_INVALID_ARG;
    if (n == 0) return WKV7_OK;
    if (!slot_ids_dev) return WKV7_ERR_INVALID_ARG;
    wkv7::GdnRunArgs a{};
    a.lv = gdn_view(pool, layer);
    a.in = token_args(pool, tokens, rows);
    a.slot_ids = slot_ids_dev;
    a.n = n;
    a.n_tok = n_tokens;
    a.step_snap_ids = step_snap_ids_dev;
    a.total_tokens = static_cast<int>(rows);
    a.max_seqlen = n_tokens;
    int launches = 0;
    cudaError_t e = wkv7::launch_gdn_run(a, stream, &launches);
    return wkv7::cuda_status("gdn_decode_multi", e, launches);
}

size_t wkv7_gdn_prefill_workspace_bytes(const wkv7_pool *pool, int32_t n_seqs, int32_t max_seqlen) {
    if (!pool || !pool->gdn || n_seqs < 1 || max_seqlen < 1) return 0;
    const wkv7_gdn_pool_desc &d = pool->gdn_desc;
    return wkv7::gdn_split_bytes(wkv7::gdn_plan_split(n_seqs, d.n_v_heads, max_seqlen, d.head_k, d.head_v),
                                 static_cast<long long>(n_seqs) * d.n_v_heads, d.head_k, d.head_v);
}

wkv7_status wkv7_gdn_prefill(wkv7_pool *pool, int32_t layer, const int32_t *slot_ids_dev,
                             const int32_t *cu_seqlens_dev, int32_t n_seqs, int32_t total_tokens, int32_t max_seqlen,
                             const wkv7_gdn_tokens *tokens, const int32_t *cu_ckpt_dev,
                             const int32_t *ckpt_snap_ids_dev, void *workspace_dev, size_t workspace_bytes,
                             int32_t sequential, cudaStream_t stream) {
    if (!pool) return WKV7_ERR_INVALID_ARG;
    if (!pool->gdn) return WKV7_ERR_UNSUPPORTED;
    if (layer < 0 || layer >= pool->desc.n_layers) return WKV7_ERR_INVALID_ARG;
    if (n_seqs < 0 || total_tokens < 0 || max_seqlen < 0 || n_seqs > pool->desc.n_slots) return WKV7_ERR_INVALID_ARG;
    if (max_seqlen > total_tokens) return WKV7_ERR_BAD_SEQLENS;
    wkv7_status st = check_tokens(pool, tokens, n_seqs == 0 ? 0 : total_tokens);
    if (st != WKV7_OK) return st;
    if ((cu_ckpt_dev == nullptr) != (ckpt_snap_ids_dev == nullptr)) return WKV7_ERR_INVALID_ARG;
    if (cu_ckpt_dev && n_seqs > 0 && pool->desc.n_snapshots == 0) return WKV7_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(workspace_dev) % 16 != 0) return WKV7_ERR_UNSUPPORTED;
    if (n_seqs == 0) return WKV7_OK;
    if (!slot_ids_dev || !cu_seqlens_dev) return WKV7_ERR_INVALID_ARG;
    wkv7::GdnRunArgs a{};
    a.lv = gdn_view(pool, layer);
    a.in = token_args(pool, tokens, total_tokens);
    a.slot_ids = slot_ids_dev;
    a.n = n_seqs;
    a.cu_seqlens = cu_seqlens_dev;
    a.total_tokens = total_tokens;
    a.max_seqlen = max_seqlen;
    a.cu_ckpt = cu_ckpt_dev;
    a.ckpt_ids = ckpt_snap_ids_dev;
    a.workspace = workspace_dev;
    a.workspace_bytes = workspace_bytes;
    a.test_skip_loads = wkv7::test_wait_timeout();
    a.wait_cycles = a.test_skip_loads ? wkv7::kTestWaitCycles : wkv7::kWaitCycles;
    int launches = 0;
    const bool chunks = sequential == 0 && wkv7::gdn_chunk_takes(a) && max_seqlen > longest_by_token(a);
    cudaError_t e = chunks ? wkv7::launch_gdn_chunk(a, stream, &launches) : wkv7::launch_gdn_run(a, stream, &launches);
    return wkv7::cuda_status("gdn_prefill", e, launches);
}

wkv7_status wkv7_verify_drafts(wkv7_pool *pool, const wkv7_draft_batch *d, cudaStream_t stream) {
    if (!pool || !d) return WKV7_ERR_INVALID_ARG;
    if (d->n < 0 || d->n_draft < 0 || d->vocab < 1 || !dtype_ok(d->prob_dtype)) return WKV7_ERR_INVALID_ARG;
    if (d->resume_ids && !d->step_snap_ids) return WKV7_ERR_INVALID_ARG;
    if (d->n == 0) return WKV7_OK;
    if (!d->p || !d->noise || !d->accepted || !d->tokens) return WKV7_ERR_INVALID_ARG;
    if (d->n_draft > 0 && (!d->draft_ids || !d->uniforms)) return WKV7_ERR_INVALID_ARG;
    const uintptr_t esz = d->prob_dtype == WKV7_BF16 ? 2 : 4;
    const void *words[8] = {d->draft_ids, d->n_draft_rows, d->uniforms, d->noise,
                            d->step_snap_ids, d->accepted, d->tokens, d->resume_ids};
    for (const void *w : words)
        if (reinterpret_cast<uintptr_t>(w) % 4) return WKV7_ERR_UNSUPPORTED;
    if (reinterpret_cast<uintptr_t>(d->p) % esz || reinterpret_cast<uintptr_t>(d->q) % esz || d->vocab > (1 << 30))
        return WKV7_ERR_UNSUPPORTED;
    if (d->n_draft > 0 && !stride_ok(d->p_row_stride, d->vocab)) return WKV7_ERR_INVALID_ARG;
    if (d->n_draft > 1 && d->q && !stride_ok(d->q_row_stride, d->vocab)) return WKV7_ERR_INVALID_ARG;
    if (d->n > 1 && (!stride_ok(d->noise_stride, d->vocab) || !stride_ok(d->p_batch_stride, d->vocab) ||
                     (d->q && d->n_draft > 0 && !stride_ok(d->q_batch_stride, d->vocab))))
        return WKV7_ERR_INVALID_ARG;
    wkv7::VerifyArgs a;
    a.d = *d;
    if (d->n_draft == 0) a.d.q = nullptr;
    a.n_snaps = pool->desc.n_snapshots;
    a.status = pool->status;
    int launches = 0;
    cudaError_t e = wkv7::launch_verify(a, stream, &launches);
    return wkv7::cuda_status("verify_drafts", e, launches);
}

}  // extern "C"
