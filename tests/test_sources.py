"""What the CUDA sources must not hold: the library is also loaded by processes
that use several GPUs, so no bulk or tensor copy in it may be a cluster multicast
(the commits' arrivals at several CTAs' barriers are none)."""

import os
import re

from backward_token_expert_gb300 import build as B


def _instructions(text):
    """The inline assembly of a source: adjacent string literals joined, one statement an entry."""
    text = re.sub(r"//[^\n]*", "", text)
    text = re.sub(r'"\s*"', "", text)
    return [s.strip() for lit in re.findall(r'"((?:[^"\\]|\\.)*)"', text) for s in re.split(r";|\\n", lit)]


def _files():
    return [os.path.join(B.CSRC, f) for f in sorted(os.listdir(B.CSRC)) if f.endswith((".cu", ".cuh"))]


def test_no_copy_is_a_cluster_multicast():
    copies = multicast = 0
    for path in _files():
        with open(path) as fh:
            for s in _instructions(fh.read()):
                if s.startswith("cp."):
                    copies += 1
                    assert ".multicast" not in s, (os.path.basename(path), s)
                multicast += ".multicast::cluster" in s
    assert copies >= 8 and multicast >= 1  # the search sees the copies, and the commits' multicast
