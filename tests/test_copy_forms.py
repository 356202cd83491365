"""Every CTA copies its own tiles: no source names a copy that is multicast to the
CTAs of a cluster."""
import glob
import os

import nvfp4_block_scaled_linear_gb300 as pkg

HERE = os.path.dirname(os.path.abspath(pkg.__file__))


def test_no_multicast_copy():
    sources = [f for d in ("csrc", "csrc_attention") for f in glob.glob(os.path.join(HERE, d, "*.cu*"))]
    assert len(sources) > 15
    named = [f for f in sources if "multicast::cluster" in open(f).read()]
    assert not named, named
