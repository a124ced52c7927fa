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
