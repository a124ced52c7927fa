"""What the CUDA sources name."""
import glob
import os

from chunkwise_gated_delta_gdr_gb300 import build as gbuild


def test_no_copy_to_several_blocks_of_a_cluster():
    """The library is built for machines with several GPUs too: no tensor load, commit or copy
    in it is a cluster multicast."""
    sources = glob.glob(os.path.join(gbuild.CSRC, "*.cu*"))
    assert sources
    for path in sources:
        with open(path) as f:
            assert "multicast::cluster" not in f.read(), path


def _body(text, kernel):
    """The braces of a kernel's definition."""
    at = text.index("{", text.index(kernel + "("))
    depth, end = 0, at
    while True:
        depth += {"{": 1, "}": -1}.get(text[end], 0)
        end += 1
        if depth == 0:
            return text[at:end]


def test_kernels_wait_before_they_touch_memory():
    """Kernels that are launched while the one before still runs wait for it (griddepcontrol, by the
    helpers of gdr_ops.cuh) ahead of the first use of anything that the call reads or writes."""
    for path in glob.glob(os.path.join(gbuild.CSRC, "*.cu*")):
        if not path.endswith("gdr_ops.cuh"):
            with open(path) as f:
                assert "griddepcontrol" not in f.read(), path
    for name, kernel, first_uses in [
            ("gdr_paged.cu", "paged_any_kernel", ("empty_rows(", "stretch(", "a.q")),
            ("gdr_paged.cu", "paged_ring_kernel", ("empty_rows(", "stretch(", "a.kc")),
            ("gdr_paged.cu", "paged_join_kernel", ("total_tiles(", "span_of(", "a.part_ml")),
            ("gdr_prefix.cu", "prefix_any_kernel", ("prefix_row(", "any_queries<", "a.kc")),
            ("gdr_prefix.cu", "prefix_join_kernel", ("a.own_lse", "a.part_ml", "a.part_o")),
            ("gdr_prefix_tc.cuh", "prefix_tc_kernel", ("q_row(", "a.table", "prefix_row(", "a.part_ml")),
            ("gdr_norm.cuh", "column_sum_kernel", ("p[",)),
            ("gdr_qk.cu", "qk_weight_kernel", ("part[",))]:
        with open(os.path.join(gbuild.CSRC, name)) as f:
            text = f.read()
        body = _body(text, kernel)
        waits = [body.index(w) for w in ("wait_for_before()", "begin_behind()") if w in body]
        assert waits, kernel
        for use in first_uses:
            at = body.find(use)
            assert (at < 0 and use != first_uses[0]) or at > min(waits), (kernel, use)
