"""Properties of the kernel sources that no call shows."""
import glob
import os

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "long_context_sparse_clsa_b200", "csrc")


def test_the_tensor_map_encoder_is_looked_up_in_one_place():
    """One lookup of the driver's entry point, and it tests both the call's status and the query's result."""
    found = [(f, open(f).read()) for f in sorted(glob.glob(os.path.join(CSRC, "*"))) if "cudaGetDriverEntryPoint(" in open(f).read()]
    assert [os.path.basename(f) for f, _ in found] == ["tma.cu"]
    assert found[0][1].count("cudaGetDriverEntryPoint(") == 1 and "cudaDriverEntryPointSuccess" in found[0][1]
