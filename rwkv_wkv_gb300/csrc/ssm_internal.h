// Kernel arguments and launchers of the state space layer's operators: selective
// scan, short convolution, gated norm.
#pragma once

#include "wkv7_internal.h"

namespace wkv7 {

// One layer of a pool of scan states, as its kernels see it.  Strides count state
// entries (float32, or bf16 with state_bf16).
struct SsmView {
    float *states;
    float *snaps;
    long long slot_stride;
    long long layer_off;
    int n_slots, n_snaps;
    int heads, groups, p, ds;
    bool state_bf16;
    int *status;
};
// One call's tokens; strides count elements.
struct SsmTokens {
    const void *x, *b, *c, *dt;
    const float *a, *d, *dt_bias;  // per head; d and dt_bias may be null
    long long x_stride, b_stride, c_stride, dt_stride;
    bool bf16, dt_bf16;
    bool softplus;
    void *o;
    bool o_bf16;
};
// Runs of tokens: n units of n_tok rows each (cu_seqlens == nullptr; the state after each token
// to step_snap_ids[unit * n_tok + t] if given), or the ragged sequences of cu_seqlens.
struct SsmRunArgs {
    SsmView lv;
    SsmTokens in;
    const int *slot_ids;
    int n;
    int n_tok;
    const int *step_snap_ids;
    const int *cu_seqlens;
    int total_tokens;
    int max_seqlen;
    bool all_or_none;  // no sequence is run if cu_seqlens is inconsistent anywhere
    void *workspace;  // for cutting long sequences (may be null)
    size_t workspace_bytes;
    long long wait_cycles;  // bound of every wait in the chunked kernel (clock cycles)
    int test_skip_loads;    // test hook: 1, no input load is issued; 2, none of a cut sequence's first pass
};

cudaError_t launch_ssm_decode(const SsmRunArgs &a, cudaStream_t s, int *launches);
cudaError_t launch_ssm_run(const SsmRunArgs &a, cudaStream_t s, int *launches);

// The short convolution.  tails: the pool's slots (or snapshots) as bytes, this layer's
// [width - 1][channels] at layer_off of each.
struct ConvArgs {
    char *slots, *snaps;
    long long slot_bytes, layer_off;
    int n_slots, n_snaps;
    int channels, width;
    bool bf16;                  // of x, o and the tails
    const void *x;
    long long x_stride;         // elements
    const void *weight, *bias;  // [channels][width], [channels] (bias may be null)
    bool w_bf16;
    bool silu;
    void *o;
    const int *slot_ids;
    int n, n_tok;
    const int *step_snap_ids;
    const int *cu_seqlens;
    int total_tokens;
    int *status;
};
// How a prefill's convolution is spread: `tiles` of `tokens` each by `blocks` of `threads` threads, kConvVec
// channels a thread.  Long tiles reload less, short ones spread few tokens over the SMs.
constexpr int kConvVec = 4;
struct ConvTiles {
    int tokens;
    unsigned threads, tiles, blocks;
};
inline ConvTiles conv_tiles(int channels, int total_tokens) {
    const int vecs = channels / kConvVec;
    ConvTiles t;
    t.threads = static_cast<unsigned>(vecs >= 128 ? 128 : (vecs + 31) / 32 * 32);
    t.blocks = (static_cast<unsigned>(vecs) + t.threads - 1) / t.threads;
    auto tiles = [&](int n) { return static_cast<unsigned>((total_tokens + n - 1) / n); };
    t.tokens = static_cast<long long>(tiles(64)) * t.blocks >= 152 * 8 ? 64 : static_cast<long long>(tiles(32)) * t.blocks >= 152 * 4 ? 32 : 8;
    t.tiles = tiles(t.tokens);
    return t;
}
cudaError_t launch_conv_step(const ConvArgs &a, cudaStream_t s, int *launches);
cudaError_t launch_conv_prefill(const ConvArgs &a, cudaStream_t s, int *launches);

cudaError_t launch_gated_norm(const wkv7_norm_args &a, cudaStream_t s, int *launches);

}  // namespace wkv7
