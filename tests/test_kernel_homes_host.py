"""Every kernel is compiled where something launches it: a header that several sources include holds kernels only as
templates, and launches them only from templates, so that a source compiles those that it calls (no GPU)."""
import glob
import os
import re

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "glu_activation_microscaling_amd", "csrc")


def text(path):
    with open(path) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def included_by(name):
    return [p for p in glob.glob(os.path.join(CSRC, "*.hip")) if f'#include "{name}"' in text(p)]


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.h"))), ids=os.path.basename)
def test_headers(path):
    t, users = text(path), included_by(os.path.basename(path))
    for m in re.finditer(r"(template\s*<[^{};]*>\s*)?__global__[^{;]*?\bvoid\s+(k_\w+)", t):
        # a plain kernel is compiled by every source that includes the header: each has to launch it
        assert m.group(1) or all(m.group(2) in text(u) for u in users), m.group(2)
    for m in re.finditer(r"(template\s*<[^{};]*>\s*)?hipError_t\s+(launch_\w+)\s*\([^{;]*\{", t):
        assert m.group(1) or all(m.group(2) in text(u) for u in users), m.group(2)
