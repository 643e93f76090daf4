"""CPU check of how the kernels on the tensor cores wait: lanes leave mbar_wait's
loop one by one and may get different answers, while reads and writes of TMEM
have to be executed by a whole warp at once.  So a wait that a warp makes is
followed by a vote, and reads of TMEM by a warp whose lanes have stored
separately by __syncwarp."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "hierarchical_kv_cache_resolve_gb300", "csrc")
FILES = sorted(f for f in os.listdir(CSRC) if f.endswith(".cu") and
               '#include "tensor_core.cuh"' in open(os.path.join(CSRC, f)).read())


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//.*", "", f.read())


def test_the_files_are_found():
    assert {"packed_attention.cu", "latent_prefill.cu", "prefix_attention.cu"} <= set(FILES)


@pytest.mark.parametrize("name", FILES)
def test_waits_of_a_warp_are_voted(name):
    text = code(name)
    for m in re.finditer(r"\bmbar_wait\(", text):
        line = text[text.rfind("\n", 0, m.start()) + 1:text.find("\n", m.start())]
        if "mbar_wait(empty(" in line:      # a ring that one lane fills
            continue
        near = text[max(0, m.start() - 40):m.start()] + "\n".join(text[m.start():].split("\n")[:6])
        assert "__all_sync(" in near, line.strip()


def test_a_wait_that_gave_up_is_the_whole_warps():
    """What reports a wait that gave up asks lane 0, so no lane may differ from it."""
    for name in ("packed_attention.cu", "latent_prefill.cu"):
        text = code(name)
        assert re.search(r"if \(!ok && lane == 0\) atomicOr", text)
        assert not re.search(r"ok = (ok && )?mbar_wait\(", text)
