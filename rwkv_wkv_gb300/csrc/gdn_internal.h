// The gated-delta-rule kernels' launchers beyond those of wkv7_internal.h.
#pragma once

#include "wkv7_internal.h"

namespace wkv7 {

// Whether the chunked kernel can run this call at all (bf16 inputs, rows apart).
bool gdn_chunk_takes(const GdnRunArgs &a);
cudaError_t launch_gdn_chunk(const GdnRunArgs &a, cudaStream_t s, int *launches);

// The test hook of wkv7_test_force_wait_timeout.
bool test_wait_timeout_on();

}  // namespace wkv7
