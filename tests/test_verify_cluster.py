"""The order of verify.cu's cluster barriers, by reading the source: a kernel may store into
another CTA's shared memory only after a cluster barrier has shown that the CTA runs, a missing
one cannot be shown by running, and every thread must come to both halves of each barrier."""
import os
import re

import rwkv_wkv_gb300.build as wbuild


def kernel_text():
    with open(os.path.join(wbuild.CSRC, "verify.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    start = text.index("verify_kernel(const VerifyArgs a) {")
    return text[start:text.index("cudaError_t launch_verify")]


def test_a_cluster_barrier_comes_before_the_first_remote_store():
    body = kernel_text()
    arrive, wait = body.index("cluster_begun();"), body.index("cluster_wait_begun();")
    assert arrive < body.index("pdl_wait();") < wait < body.index("store_remote_u64(")
    assert body.count("cluster_begun();") == body.count("cluster_wait_begun();") == 1


def test_no_thread_leaves_before_the_barrier():
    body = kernel_text()
    assert "return" not in body[:body.index("cluster_wait_begun();")]
