"""The bulk copies of the kernel sources (CPU only): each brings what it reads to
one CTA. A copy that one CTA sends to all of its cluster is for memory of the GPU
that it runs on alone, which nothing here can promise: the library takes any
pointer and is loaded by processes of several GPUs too."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "implicit_gemm_convolution_vae_gb300", "csrc")

# What may stand between the instruction's name and its operands.
QUALIFIERS = {"tensor", "2d", "3d", "4d", "5d", "shared::cluster", "shared::cta", "global", "tile", "mbarrier::complete_tx::bytes",
              "bulk_group", "commit_group", "wait_group", "read", "prefetch", "L2", "cta_group::2", "L2::cache_hint"}


def bulk_copies():
    """(file, qualifiers) of each bulk copy; an instruction may be spelt over several string literals."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        text = re.sub(r"//[^\n]*", "", open(path, encoding="utf-8").read())
        text = re.sub(r'"\s*"', "", text)
        for m in re.finditer(r"cp\.async\.bulk((?:\.[A-Za-z0-9_:]+)+)", text):
            yield os.path.basename(path), m.group(1)[1:].split(".")


def test_bulk_copies_reach_one_cta():
    copies = list(bulk_copies())
    assert {"vae_common.cuh", "vae_ln.cu", "vae_mha_bwd.cu"} <= {f for f, _ in copies}
    other = [(f, ".".join(q)) for f, q in copies if not set(q) <= QUALIFIERS]
    assert not other, other
