"""What can be told of the training operators' kernels from their sources, without a GPU."""
import os
import re

from combine_ep_dispatch_02_gb300 import build


def test_arrivals_on_another_ctas_barrier_have_cluster_scope():
    """mbarrier.arrive's scope is the CTA unless it says otherwise, and that orders nothing for a thread of another CTA.  Only
    the tensor cores' commit and TMA's byte counts, which are not arrive instructions, signal other CTAs in another way."""
    seen = 0
    for name in sorted(os.listdir(build.CSRC)):
        with open(os.path.join(build.CSRC, name)) as f:
            for text in re.findall(r"mbarrier\.arrive[\w.:]*", f.read()):
                if "shared::cluster" in text:
                    seen += 1
                    assert re.search(r"\.cluster\.shared::cluster", text), (name, text)
    assert seen >= 2
