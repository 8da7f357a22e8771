"""What the library's kernels may not contain, read from their sources (no GPU needed)."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_matvec_lb_gb300", "csrc")


def test_a_copy_goes_into_one_cta():
    """The library is loaded by every replica of a run on several GPUs, and its copies read memory that its callers
    own: none is sent to several CTAs of a cluster at once, which is only for a GPU's own memory."""
    files = [p for ext in ("*.cu", "*.cuh") for p in glob.glob(os.path.join(CSRC, ext))]
    assert len(files) > 20
    for path in files:
        with open(path) as f:
            text = re.sub(r'"\s*\n?\s*"', "", f.read())   # strings that go on are one
        found = re.findall(r"cp\.(?:reduce\.)?async\.bulk[^;\"]*multicast[^;\"]*", text)
        assert not found, (os.path.basename(path), found)


def test_counted_waits_last_as_long_as_the_others():
    """A try's time hint is a most, not a length: waits that count tries take their number from the one place that
    knows how long a try is."""
    counted = 0
    for path in glob.glob(os.path.join(CSRC, "*.cu*")):
        with open(path) as f:
            text = f.read()
        for first in re.findall(r"\bint tries = ([^;]*);", text):
            assert first == "kWaitTries", os.path.basename(path)
            counted += 1
    assert counted == 2
