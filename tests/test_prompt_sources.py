"""What the kernel sources must not hold (CPU: the text of the sources)."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_no_copy_is_sent_to_several_ctas():
    """A bulk copy to several CTAs of a cluster must read this GPU's memory alone.  The calls take any device pointer, a peer's too, and
    processes of several GPUs load the library: no source has one.  (tcgen05.commit's arrival on several barriers is no copy.)"""
    paths = sorted(glob.glob(os.path.join(ROOT, "serving_router_softmax_gb300", "csrc", "*.cu*")))
    assert len(paths) > 20
    for path in paths:
        text = re.sub(r'"\s*\n\s*"', "", open(path).read())  # strings that go on in the next line
        for line in text.split("\n"):
            assert not ("cp.async.bulk" in line and "multicast" in line), (path, line.strip())
