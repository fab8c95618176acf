// C-ABI entry points of the state space layer's operators: checks and dispatch.
// The public contract is documented in wkv7.h.
#include <cmath>
#include <new>

#include "gdn_internal.h"
#include "pool.h"
#include "ssm_chunk.h"
#include "ssm_internal.h"

namespace {

constexpr int32_t kMaxRows = 0x7fffff00;  // kernels round row counts up to whole tiles

bool size_ok(int32_t d) { return d == 64 || d == 128; }
bool dtype_ok(int32_t d) { return d == WKV7_F32 || d == WKV7_BF16; }
int64_t bytes_of(int32_t d) { return d == WKV7_BF16 ? 2 : 4; }
bool aligned(const void *p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

// Rows that are read: apart from each other, or one row for all (stride 0).
bool stride_ok(int64_t stride, int64_t row) { return stride == 0 || stride >= row; }

// Whether `rows` rows of `row_bytes`, `stride_bytes` apart from p, share a byte with the `bytes` from o on.
bool overlaps(const void *p, int64_t rows, int64_t stride_bytes, int64_t row_bytes, const void *o, int64_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(o);
    const uintptr_t end = a + static_cast<uintptr_t>((rows - 1) * stride_bytes + row_bytes);
    return a < b + static_cast<uintptr_t>(bytes) && b < end;
}

bool desc_valid(const wkv7_ssm_pool_desc *d) {
    return d && d->n_layers >= 1 && d->n_heads >= 1 && d->n_groups >= 1 && d->n_heads % d->n_groups == 0 && d->head_p >= 1 &&
           d->d_state >= 1 && d->n_slots >= 1 && d->n_snapshots >= 0 && dtype_ok(d->state_dtype) && dtype_ok(d->out_dtype) &&
           wkv7::conv_desc_valid(d->conv);
}

size_t state_bytes(const wkv7_ssm_pool_desc *d) {
    return static_cast<size_t>(d->n_layers) * static_cast<size_t>(d->n_heads) * static_cast<size_t>(d->head_p) *
           static_cast<size_t>(d->d_state) * static_cast<size_t>(bytes_of(d->state_dtype));
}

// The part of the description that the shared pool code reads.
wkv7_pool_desc plain_desc(const wkv7_ssm_pool_desc *d) {
    wkv7_pool_desc p{};
    p.n_layers = d->n_layers;
    p.n_heads = d->n_heads;
    p.head_size = d->head_p;
    p.n_slots = d->n_slots;
    p.n_snapshots = d->n_snapshots;
    p.device_buffer = d->device_buffer;
    p.buffer_bytes = d->buffer_bytes;
    p.state_dtype = d->state_dtype;
    p.out_dtype = d->out_dtype;
    return p;
}

wkv7::SsmView view_of(wkv7_pool *p, int32_t layer) {
    const wkv7_ssm_pool_desc &d = p->ssm_desc;
    wkv7::SsmView lv;
    lv.states = p->states;
    lv.snaps = p->snaps;
    lv.slot_stride = p->slot_entries;
    lv.layer_off = static_cast<long long>(layer) * d.n_heads * p->head_elems;
    lv.n_slots = d.n_slots;
    lv.n_snaps = d.n_snapshots;
    lv.heads = d.n_heads;
    lv.groups = d.n_groups;
    lv.p = d.head_p;
    lv.ds = d.d_state;
    lv.state_bf16 = p->state_bf16;
    lv.status = p->status;
    return lv;
}

// The checks of one call's tokens; `rows` > 0 of them are read.
wkv7_status check_tokens(const wkv7_pool *p, const wkv7_ssm_tokens *t, long long rows) {
    if (!t || !dtype_ok(t->in_dtype) || !dtype_ok(t->dt_dtype)) return WKV7_ERR_INVALID_ARG;
    if (rows == 0) return WKV7_OK;
    if (!t->x || !t->b || !t->c || !t->dt || !t->a || !t->o) return WKV7_ERR_INVALID_ARG;
    const wkv7_ssm_pool_desc &d = p->ssm_desc;
    const int64_t xw = static_cast<int64_t>(d.n_heads) * d.head_p, bw = static_cast<int64_t>(d.n_groups) * d.d_state;
    // one row alone never steps to the next, so its strides may be anything
    if (rows > 1 && (!stride_ok(t->x_stride, xw) || !stride_ok(t->b_stride, bw) || !stride_ok(t->c_stride, bw) ||
                     !stride_ok(t->dt_stride, d.n_heads)))
        return WKV7_ERR_INVALID_ARG;
    const void *bases[4] = {t->x, t->b, t->c, t->o};
    for (const void *b : bases)
        if (!aligned(b, 16)) return WKV7_ERR_UNSUPPORTED;
    if (!aligned(t->dt, static_cast<uintptr_t>(bytes_of(t->dt_dtype))) || !aligned(t->a, 4) || !aligned(t->d, 4) ||
        !aligned(t->dt_bias, 4))
        return WKV7_ERR_UNSUPPORTED;
    if (rows > 1) {
        const int64_t strides[3] = {t->x_stride, t->b_stride, t->c_stride};
        for (int64_t s : strides)
            if (s * bytes_of(t->in_dtype) % 16 != 0) return WKV7_ERR_UNSUPPORTED;
    }
    const int64_t e = bytes_of(t->in_dtype), de = bytes_of(t->dt_dtype), gap = rows > 1 ? 1 : 0;
    const int64_t out = rows * xw * bytes_of(d.out_dtype);
    if (overlaps(t->x, rows, gap * t->x_stride * e, xw * e, t->o, out) || overlaps(t->b, rows, gap * t->b_stride * e, bw * e, t->o, out) ||
        overlaps(t->c, rows, gap * t->c_stride * e, bw * e, t->o, out) ||
        overlaps(t->dt, rows, gap * t->dt_stride * de, d.n_heads * de, t->o, out))
        return WKV7_ERR_INVALID_ARG;
    return WKV7_OK;
}

wkv7::SsmTokens token_args(const wkv7_pool *p, const wkv7_ssm_tokens *t, long long rows) {
    const wkv7_ssm_pool_desc &d = p->ssm_desc;
    const bool one = rows <= 1;  // a lone row's strides are never used: make them valid ones
    const long long bw = static_cast<long long>(d.n_groups) * d.d_state;
    wkv7::SsmTokens a;
    a.x = t->x;
    a.b = t->b;
    a.c = t->c;
    a.dt = t->dt;
    a.a = t->a;
    a.d = t->d;
    a.dt_bias = t->dt_bias;
    a.x_stride = one ? static_cast<long long>(d.n_heads) * d.head_p : t->x_stride;
    a.b_stride = one ? bw : t->b_stride;
    a.c_stride = one ? bw : t->c_stride;
    a.dt_stride = one ? d.n_heads : t->dt_stride;
    a.bf16 = t->in_dtype == WKV7_BF16;
    a.dt_bf16 = t->dt_dtype == WKV7_BF16;
    a.softplus = t->dt_softplus != 0;
    a.o = t->o;
    a.o_bf16 = p->out_bf16;
    return a;
}

wkv7_status ssm_pool_check(const wkv7_pool *pool, int32_t layer) {
    if (!pool) return WKV7_ERR_INVALID_ARG;
    if (!pool->ssm) return WKV7_ERR_UNSUPPORTED;
    return layer < 0 || layer >= pool->desc.n_layers ? WKV7_ERR_INVALID_ARG : WKV7_OK;
}

// The longest max_seqlen that runs token by token where the chunked kernel could.  A chunk of 128 costs the
// same however few of its tokens there are, and a token what its state's size says.  Token by token against
// in chunks, us: 1 sequence of 64 heads of 64 x 128, of 24 tokens 11.4 and 13.1, of 32 13.7 and 13.0; where the blocks of
// 64 state rows fill the 152 SMs, 4 sequences of 16 17.3 and 17.8, of 24 24.6 and 18.1, 64 of 16 128 and 135, of 24
// 186 and 132.  24 heads of 64 x 64, 1 of 24 10.6 and 11.3, of 32 12.8 and 11.2; 16 of 32 20.3 and 19.8, 64 of 32 50.9
// and 51.2, of 48 74 and 52.
int longest_by_token(const wkv7::SsmRunArgs &a) {
    if (static_cast<long long>(a.n) * a.lv.heads * (a.lv.p / 64) < 152) return 24;
    return a.lv.ds == 64 ? 32 : 16;
}

// The checks of one convolution; `rows` > 0 of them are read.
wkv7_status check_conv(const wkv7_pool *p, const wkv7_conv_tokens *t, long long rows) {
    if (!t || !dtype_ok(t->weight_dtype)) return WKV7_ERR_INVALID_ARG;
    if (t->activation != WKV7_CONV_LINEAR && t->activation != WKV7_CONV_SILU) return WKV7_ERR_INVALID_ARG;
    if (rows == 0) return WKV7_OK;
    if (!t->x || !t->weight || !t->o) return WKV7_ERR_INVALID_ARG;
    const int64_t e = bytes_of(p->conv.dtype), width = p->conv.channels;
    if (rows > 1 && !stride_ok(t->x_stride, width)) return WKV7_ERR_INVALID_ARG;
    if (!aligned(t->x, 16) || !aligned(t->weight, 16) || !aligned(t->bias, 16) || !aligned(t->o, 16)) return WKV7_ERR_UNSUPPORTED;
    if (rows > 1 && t->x_stride * e % 16 != 0) return WKV7_ERR_UNSUPPORTED;
    if (overlaps(t->x, rows, rows > 1 ? t->x_stride * e : 0, width * e, t->o, rows * width * e)) return WKV7_ERR_INVALID_ARG;
    return WKV7_OK;
}

wkv7::ConvArgs conv_args(wkv7_pool *p, int32_t layer, const wkv7_conv_tokens *t, long long rows) {
    wkv7::ConvArgs a{};
    const long long e = bytes_of(p->conv.dtype);
    a.slots = reinterpret_cast<char *>(p->states);
    a.snaps = reinterpret_cast<char *>(p->snaps);
    a.slot_bytes = p->slot_floats * 4;
    a.layer_off = static_cast<long long>(p->conv_off) + static_cast<long long>(layer) * (p->conv.width - 1) * p->conv.channels * e;
    a.n_slots = p->desc.n_slots;
    a.n_snaps = p->desc.n_snapshots;
    a.channels = p->conv.channels;
    a.width = p->conv.width;
    a.bf16 = p->conv.dtype == WKV7_BF16;
    a.x = t->x;
    a.x_stride = rows <= 1 ? p->conv.channels : t->x_stride;
    a.weight = t->weight;
    a.bias = t->bias;
    a.w_bf16 = t->weight_dtype == WKV7_BF16;
    a.silu = t->activation == WKV7_CONV_SILU;
    a.o = t->o;
    a.status = p->status;
    return a;
}

}  // namespace

namespace wkv7 {

bool conv_desc_valid(const wkv7_conv_desc &c) {
    return c.channels == 0 || (c.channels > 0 && c.channels % 8 == 0 && c.width >= 2 && c.width <= 4 && dtype_ok(c.dtype));
}
// (Rounded up to 256 bytes, so that every slot begins on such a boundary.)
size_t conv_bytes(const wkv7_conv_desc &c, int32_t n_layers) {
    if (c.channels == 0) return 0;
    const size_t tails = static_cast<size_t>(n_layers) * static_cast<size_t>(c.width - 1) * static_cast<size_t>(c.channels) *
                         static_cast<size_t>(bytes_of(c.dtype));
    return (tails + 255) / 256 * 256;
}

}  // namespace wkv7

extern "C" {

size_t wkv7_ssm_pool_required_bytes(const wkv7_ssm_pool_desc *desc) {
    if (!desc_valid(desc)) return 0;
    const wkv7_pool_desc d = plain_desc(desc);
    return wkv7::pool_bytes(&d, state_bytes(desc) + wkv7::conv_bytes(desc->conv, desc->n_layers));
}

wkv7_status wkv7_ssm_pool_create(const wkv7_ssm_pool_desc *desc, wkv7_pool **out) {
    if (!out) return WKV7_ERR_INVALID_ARG;
    *out = nullptr;
    if (!desc_valid(desc)) return WKV7_ERR_INVALID_ARG;
    if (!size_ok(desc->head_p) || !size_ok(desc->d_state)) return WKV7_ERR_UNSUPPORTED;
    const size_t need = wkv7_ssm_pool_required_bytes(desc);
    if (desc->device_buffer) {
        if (desc->buffer_bytes < need) return WKV7_ERR_INVALID_ARG;
        if (!aligned(desc->device_buffer, 256)) return WKV7_ERR_INVALID_ARG;
    }
    wkv7_pool *p = new (std::nothrow) wkv7_pool();
    if (!p) return WKV7_ERR_NO_MEMORY;
    p->desc = plain_desc(desc);
    p->ssm = true;
    p->ssm_desc = *desc;
    p->head_elems = static_cast<long long>(desc->head_p) * desc->d_state;
    p->conv = desc->conv;
    p->conv_off = state_bytes(desc);
    return wkv7::lay_out_pool(p, p->conv_off + wkv7::conv_bytes(desc->conv, desc->n_layers), need, out);
}

wkv7_status wkv7_ssm_pool_get_desc(const wkv7_pool *pool, wkv7_ssm_pool_desc *out) {
    if (!pool || !out) return WKV7_ERR_INVALID_ARG;
    if (!pool->ssm) return WKV7_ERR_UNSUPPORTED;
    *out = pool->ssm_desc;
    out->device_buffer = pool->desc.device_buffer;
    out->buffer_bytes = pool->desc.buffer_bytes;
    return WKV7_OK;
}

wkv7_status wkv7_ssm_decode_step(wkv7_pool *pool, int32_t layer, const int32_t *slot_ids_dev, int32_t n,
                                 const wkv7_ssm_tokens *tokens, cudaStream_t stream) {
    wkv7_status st = ssm_pool_check(pool, layer);
    if (st != WKV7_OK) return st;
    if (n < 0 || n > pool->desc.n_slots) return WKV7_ERR_INVALID_ARG;
    st = check_tokens(pool, tokens, n);
    if (st != WKV7_OK) return st;
    if (n == 0) return WKV7_OK;
    if (!slot_ids_dev) return WKV7_ERR_INVALID_ARG;
    wkv7::SsmRunArgs a{};
    a.lv = view_of(pool, layer);
    a.in = token_args(pool, tokens, n);
    a.slot_ids = slot_ids_dev;
    a.n = n;
    a.n_tok = 1;
    int launches = 0;
    cudaError_t e = wkv7::launch_ssm_decode(a, stream, &launches);
    return wkv7::cuda_status("ssm_decode_step", e, launches);
}

wkv7_status wkv7_ssm_decode_multi(wkv7_pool *pool, int32_t layer, const int32_t *slot_ids_dev, int32_t n, int32_t n_tokens,
                                  const wkv7_ssm_tokens *tokens, const int32_t *step_snap_ids_dev, cudaStream_t stream) {
    wkv7_status st = ssm_pool_check(pool, layer);
    if (st != WKV7_OK) return st;
    if (n < 0 || n > pool->desc.n_slots || n_tokens < 1) return WKV7_ERR_INVALID_ARG;
    const long long rows = static_cast<long long>(n) * n_tokens;
    if (rows > kMaxRows) return WKV7_ERR_INVALID_ARG;
    st = check_tokens(pool, tokens, rows);
    if (st != WKV7_OK) return st;
    if (step_snap_ids_dev && pool->desc.n_snapshots == 0) return WKV7_ERR_INVALID_ARG;
    if (n == 0) return WKV7_OK;
    if (!slot_ids_dev) return WKV7_ERR_INVALID_ARG;
    wkv7::SsmRunArgs a{};
    a.lv = view_of(pool, layer);
    a.in = token_args(pool, tokens, rows);
    a.slot_ids = slot_ids_dev;
    a.n = n;
    a.n_tok = n_tokens;
    a.step_snap_ids = step_snap_ids_dev;
    a.total_tokens = static_cast<int>(rows);
    a.max_seqlen = n_tokens;
    int launches = 0;
    cudaError_t e = wkv7::launch_ssm_run(a, stream, &launches);
    return wkv7::cuda_status("ssm_decode_multi", e, launches);
}

size_t wkv7_ssm_prefill_workspace_bytes(const wkv7_pool *pool, int32_t n_seqs, int32_t max_seqlen) {
    if (!pool || !pool->ssm || n_seqs < 1 || max_seqlen < 1) return 0;
    const wkv7_ssm_pool_desc &d = pool->ssm_desc;
    return wkv7::ssm_split_bytes(wkv7::ssm_plan_split(n_seqs, d.n_heads, d.head_p, max_seqlen),
                                 static_cast<long long>(n_seqs) * d.n_heads * (d.head_p / 64), d.d_state);
}

wkv7_status wkv7_ssm_prefill(wkv7_pool *pool, int32_t layer, const int32_t *slot_ids_dev, const int32_t *cu_seqlens_dev,
                             int32_t n_seqs, int32_t total_tokens, int32_t max_seqlen, const wkv7_ssm_tokens *tokens,
                             void *workspace_dev, size_t workspace_bytes, int32_t sequential, cudaStream_t stream) {
    wkv7_status st = ssm_pool_check(pool, layer);
    if (st != WKV7_OK) return st;
    if (n_seqs < 0 || total_tokens < 0 || total_tokens > kMaxRows || max_seqlen < 0 || n_seqs > pool->desc.n_slots)
        return WKV7_ERR_INVALID_ARG;
    if (max_seqlen > total_tokens) return WKV7_ERR_BAD_SEQLENS;
    st = check_tokens(pool, tokens, n_seqs == 0 ? 0 : total_tokens);
    if (st != WKV7_OK) return st;
    if (!aligned(workspace_dev, 16)) return WKV7_ERR_UNSUPPORTED;
    if (n_seqs == 0) return WKV7_OK;
    if (!slot_ids_dev || !cu_seqlens_dev) return WKV7_ERR_INVALID_ARG;
    wkv7::SsmRunArgs a{};
    a.lv = view_of(pool, layer);
    a.in = token_args(pool, tokens, total_tokens);
    a.slot_ids = slot_ids_dev;
    a.n = n_seqs;
    a.cu_seqlens = cu_seqlens_dev;
    a.total_tokens = total_tokens;
    a.max_seqlen = max_seqlen;
    a.all_or_none = tokens->all_or_none != 0;
    a.workspace = workspace_dev;
    a.workspace_bytes = workspace_bytes;
    a.test_skip_loads = wkv7::test_wait_timeout();
    a.wait_cycles = a.test_skip_loads ? wkv7::kTestWaitCycles : wkv7::ssm_wait_cycles(max_seqlen);
    int launches = 0;
    const bool chunks = sequential == 0 && wkv7::ssm_chunk_takes(a) && max_seqlen > longest_by_token(a);
    cudaError_t e = chunks ? wkv7::launch_ssm_chunk(a, stream, &launches) : wkv7::launch_ssm_run(a, stream, &launches);
    return wkv7::cuda_status("ssm_prefill", e, launches);
}

wkv7_status wkv7_pool_conv_desc(const wkv7_pool *pool, wkv7_conv_desc *out, size_t *slot_offset) {
    if (!pool || !out) return WKV7_ERR_INVALID_ARG;
    *out = pool->conv;
    if (slot_offset) *slot_offset = pool->conv.channels ? pool->conv_off : 0;
    return WKV7_OK;
}

wkv7_status wkv7_conv_step(wkv7_pool *pool, int32_t layer, const int32_t *slot_ids_dev, int32_t n, int32_t n_tokens,
                           const wkv7_conv_tokens *tokens, const int32_t *step_snap_ids_dev, cudaStream_t stream) {
    if (!pool) return WKV7_ERR_INVALID_ARG;
    if (pool->conv.channels == 0) return WKV7_ERR_UNSUPPORTED;
    if (layer < 0 || layer >= pool->desc.n_layers || n < 0 || n > pool->desc.n_slots || n_tokens < 1) return WKV7_ERR_INVALID_ARG;
    const long long rows = static_cast<long long>(n) * n_tokens;
    if (rows > kMaxRows) return WKV7_ERR_INVALID_ARG;
    const wkv7_status st = check_conv(pool, tokens, rows);
    if (st != WKV7_OK) return st;
    if (step_snap_ids_dev && pool->desc.n_snapshots == 0) return WKV7_ERR_INVALID_ARG;
    if (n == 0) return WKV7_OK;
    if (!slot_ids_dev) return WKV7_ERR_INVALID_ARG;
    wkv7::ConvArgs a = conv_args(pool, layer, tokens, rows);
    a.slot_ids = slot_ids_dev;
    a.n = n;
    a.n_tok = n_tokens;
    a.step_snap_ids = step_snap_ids_dev;
    int launches = 0;
    cudaError_t e = wkv7::launch_conv_step(a, stream, &launches);
    return wkv7::cuda_status("conv_step", e, launches);
}

wkv7_status wkv7_conv_prefill(wkv7_pool *pool, int32_t layer, const int32_t *slot_ids_dev, const int32_t *cu_seqlens_dev,
                              int32_t n_seqs, int32_t total_tokens, const wkv7_conv_tokens *tokens, cudaStream_t stream) {
    if (!pool) return WKV7_ERR_INVALID_ARG;
    if (pool->conv.channels == 0) return WKV7_ERR_UNSUPPORTED;
    if (layer < 0 || layer >= pool->desc.n_layers || n_seqs < 0 || total_tokens < 0 || total_tokens > kMaxRows ||
        n_seqs > pool->desc.n_slots)
        return WKV7_ERR_INVALID_ARG;
    const wkv7_status st = check_conv(pool, tokens, n_seqs == 0 ? 0 : total_tokens);
    if (st != WKV7_OK) return st;
    if (n_seqs == 0 || total_tokens == 0) return WKV7_OK;
    if (!slot_ids_dev || !cu_seqlens_dev) return WKV7_ERR_INVALID_ARG;
    wkv7::ConvArgs a = conv_args(pool, layer, tokens, total_tokens);
    a.slot_ids = slot_ids_dev;
    a.cu_seqlens = cu_seqlens_dev;
    a.n = n_seqs;
    a.total_tokens = total_tokens;
    int launches = 0;
    cudaError_t e = wkv7::launch_conv_prefill(a, stream, &launches);
    return wkv7::cuda_status("conv_prefill", e, launches);
}

wkv7_status wkv7_gated_norm(const wkv7_norm_args *args, cudaStream_t stream) {
    if (!args) return WKV7_ERR_INVALID_ARG;
    wkv7_norm_args a = *args;
    if (a.rows < 0 || a.width < 1 || a.group < 1 || a.width % a.group != 0) return WKV7_ERR_INVALID_ARG;
    if (!dtype_ok(a.x_dtype) || !dtype_ok(a.z_dtype) || !dtype_ok(a.w_dtype) || !dtype_ok(a.o_dtype)) return WKV7_ERR_INVALID_ARG;
    if (a.kind != WKV7_NORM_RMS && a.kind != WKV7_NORM_LAYER) return WKV7_ERR_INVALID_ARG;
    if (a.act != WKV7_GATE_LINEAR && a.act != WKV7_GATE_SILU && a.act != WKV7_GATE_SIGMOID) return WKV7_ERR_INVALID_ARG;
    if (!(a.eps >= 0.f) || std::isinf(a.eps)) return WKV7_ERR_INVALID_ARG;
    if (a.group % 8 != 0 || a.group > 16384) return WKV7_ERR_UNSUPPORTED;
    if (a.rows == 0) return WKV7_OK;
    if (!a.x || !a.o) return WKV7_ERR_INVALID_ARG;
    if (!aligned(a.x, 16) || !aligned(a.z, 16) || !aligned(a.weight, 16) || !aligned(a.bias, 16) || !aligned(a.o, 16))
        return WKV7_ERR_UNSUPPORTED;
    const int64_t xe = bytes_of(a.x_dtype), ze = bytes_of(a.z_dtype), oe = bytes_of(a.o_dtype);
    if (a.rows > 1) {
        if (!stride_ok(a.x_stride, a.width) || (a.z && !stride_ok(a.z_stride, a.width))) return WKV7_ERR_INVALID_ARG;
        if (a.x_stride * xe % 16 != 0 || (a.z && a.z_stride * ze % 16 != 0)) return WKV7_ERR_UNSUPPORTED;
    } else {
        a.x_stride = a.z_stride = a.width;
    }
    const int64_t out = static_cast<int64_t>(a.rows) * a.width * oe;
    if (overlaps(a.x, a.rows, a.x_stride * xe, a.width * xe, a.o, out)) return WKV7_ERR_INVALID_ARG;
    if (a.z && overlaps(a.z, a.rows, a.z_stride * ze, a.width * ze, a.o, out)) return WKV7_ERR_INVALID_ARG;
    int launches = 0;
    cudaError_t e = wkv7::launch_gated_norm(a, stream, &launches);
    return wkv7::cuda_status("gated_norm", e, launches);
}

}  // extern "C"
