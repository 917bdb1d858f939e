"""The layer operators' profile names the sources that it was taken on; figures quoted from it are stale as
soon as one of them changes."""
import glob
import hashlib
import os
import re

from conftest import ROOT

CSRC = os.path.join(ROOT, "sharded_fsdp_flatten_amd", "csrc")


def named():
    """{profile: {source: sha256 given}} of the profiles that name a layer source."""
    out = {}
    for path in glob.glob(os.path.join(ROOT, "profiles", "*.md")):
        with open(path) as f:
            hashes = dict(re.findall(r"^(\S+\.(?:hip|h|cpp)) sha256: `([0-9a-f]{64})`", f.read(), re.M))
        if "layer.hip" in hashes:
            out[os.path.basename(path)] = hashes
    return out


def test_the_layer_profile_was_taken_on_the_current_sources():
    profiles = named()
    assert profiles
    for profile, hashes in profiles.items():
        assert set(hashes) >= {"layer.hip", "layer.h", "layer_dev.h", "norm_backward.h"}, profile
        for name, given in hashes.items():
            with open(os.path.join(CSRC, name), "rb") as f:
                assert hashlib.sha256(f.read()).hexdigest() == given, (profile, name)
