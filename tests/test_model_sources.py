"""Rules that the sources of the operators of a layer in 8 bits keep, read off their text (CPU)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "collective_transport_plane_gb300", "csrc")


@pytest.mark.parametrize("name", sorted(n for n in os.listdir(CSRC) if n.endswith((".cu", ".cuh", ".h"))))
def test_no_copy_goes_to_several_ctas(name):
    # The library is one file for programs of one GPU and of several, and a product takes any pointer that the device reaches,
    # so no copy into shared memory may name more than the CTA that asks for it.  (An arrival at several barriers copies nothing.)
    text = open(os.path.join(CSRC, name)).read()
    copies = re.findall(r"cp\.(?:async|reduce)[\w.:]*", text)
    assert not [c for c in copies if "multicast" in c]
