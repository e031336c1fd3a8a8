"""The attention operators' arguments and build, as far as they need no GPU:
what is refused before a kernel could see it, and what is not."""

import os
import re

from conftest import ROOT

CSRC = os.path.join(ROOT, "quantized_expert_ffn_router_gb300", "csrc")

def test_every_header_is_a_dependency_of_the_build():
    """What a source includes from the tree makes its object stale."""
    from quantized_expert_ffn_router_gb300 import build as b

    known = {os.path.basename(h) for h in b.headers()}
    for name in os.listdir(CSRC):
        if name.endswith((".cu", ".cuh", ".h")):
            text = open(os.path.join(CSRC, name)).read()
            for inc in re.findall(r'^\s*#\s*include\s+"([^"]+)"', text, flags=re.M):
                assert os.path.basename(inc) in known, (name, inc)
