// The chunked selective scan's launcher and how it cuts long sequences.
#pragma once

#include "ssm_internal.h"

namespace wkv7 {

// Whether the chunked kernel can run this call at all (bf16 inputs, rows apart).
bool ssm_chunk_takes(const SsmRunArgs &a);
// A call's sequences in `segments` parts of `chunks` chunks each that run side by side (below 2:
// not so), or cut wherever an SM's share of the work ends; and the workspace that takes for `units` blocks of 64 state rows.
struct SsmSplit {
    int segments, chunks;
    bool cut;
};
SsmSplit ssm_plan_split(int n_seqs, int heads, int p, int max_seqlen);
size_t ssm_split_bytes(const SsmSplit &split, long long units, int ds);
// The bound of a wait.  What a role or another CTA waits for longest is a sequence's own chain of parts: 2.45 us a chunk
// of 128 tokens, or, where its rows run again token by token, 3.5 (d_state 128) to 9.5 us (64) a token; here 20.
constexpr long long ssm_wait_cycles(int max_seqlen) { return kWaitCycles + 40000LL * max_seqlen; }
cudaError_t launch_ssm_chunk(const SsmRunArgs &a, cudaStream_t s, int *launches);

}  // namespace wkv7
