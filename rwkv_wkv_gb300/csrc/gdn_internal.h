// The gated-delta-rule kernels' launchers beyond those of wkv7_internal.h.
#pragma once

#include "wkv7_internal.h"

namespace wkv7 {

// Whether the chunked kernel can run this call at all (bf16 inputs, rows apart).
bool gdn_chunk_takes(const GdnRunArgs &a);
// A call's sequences in `segments` parts of `chunks` chunks each that run side by side (below 2:
// not so), or in 3 `pieces` that run one after the other, from chunks 0, from1 and from2 on
// (0: not so), and the workspace that takes.
struct GdnSplit {
    int segments, chunks;
    int pieces, from1, from2;
};
GdnSplit gdn_plan_split(int n_seqs, int heads, int max_seqlen, int dk, int dv);
size_t gdn_split_bytes(const GdnSplit &split, long long units, int dk, int dv);
cudaError_t launch_gdn_chunk(const GdnRunArgs &a, cudaStream_t s, int *launches);

// The test hook of wkv7_test_force_wait_timeout (0: off).
int test_wait_timeout();

}  // namespace wkv7
