"""What the CUDA sources may not name.  The library is loaded by runs on
several GPUs too (one replica each), and the C entries encode tensor maps of
whatever addresses they are given, so no bulk copy may multicast: such a copy
is for the memory of the GPU that runs it alone."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_no_bulk_copy_multicasts():
    files = [f for d in ("mla_attention_kv_gb300/csrc", "include") for f in glob.glob(os.path.join(ROOT, d, "*"))]
    assert len(files) > 20
    for f in files:
        text = open(f).read()
        for m in re.finditer(r"cp\.async\.bulk[^;]*", text):
            assert "multicast" not in m.group(0), (os.path.basename(f), m.group(0))
        assert "tma_load_4d_multicast" not in text


def test_arrivals_at_another_cta_are_released_to_it():
    """A release of CTA scope does not reach a waiter in another CTA of the cluster."""
    for f in glob.glob(os.path.join(ROOT, "mla_attention_kv_gb300", "csrc", "*")):
        assert "arrive.release.cta.shared::cluster" not in open(f).read(), os.path.basename(f)
