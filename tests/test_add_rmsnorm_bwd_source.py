"""What the cluster form of rowops_add_rmsnorm_bwd relies on, in its source.

Its CTAs exchange parts of a row's sum by st.async.  That the parts are seen rests on the
scope of the waits, which no run can show: a GPU whose shared memory happens to keep the
order gives the same bits with less."""
import os
import re

from row_wise_softmax_warp_gb300 import build


def kernel():
    with open(os.path.join(build.CSRC, "add_rmsnorm_bwd.cu")) as f:
        text = f.read()
    at = text.index("add_rmsnorm_bwd_rows(const AddNormBwdArgs a)")
    return re.sub(r"//[^\n]*", "", text[at:text.index("\n}\n", at)])


def test_a_row_waits_with_the_clusters_acquire():
    """The other CTAs' parts are read behind the wait: its acquire has to reach them."""
    body = kernel()
    assert body.index("spread_part(") < body.index("mbar_wait_cluster(&all.bar[turn]") < body.index("all.sums[turn][i]")
    assert "mbar_wait(" not in body


def test_what_a_cta_sets_up_is_released_before_the_first_row():
    """Barriers and abort flag are written by one thread: the first synchronisation has to order both."""
    body = kernel()
    made = body.index("all.abort = 0")
    behind = body[made:body.index("threadIdx.x >> 5")]
    assert "cluster_sync_all()" in behind and "relaxed" not in behind
