"""Host-only: the decode kernel's loads in the compiled gfx950 code.

The kernel waits by count: at most HALF vector-memory operations in flight
means that a block's keys have landed, because its values (HALF - 1 direct-to-
LDS loads and a scale byte) are issued behind its keys (as many).  So no load
of one may stand among those of the other, wherever a block is fetched.
"""
import os
import re
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from level_dsl_amd import build  # noqa: E402


@pytest.fixture(scope="module")
def listing(tmp_path_factory):
    try:
        cc = build.hipcc()
    except RuntimeError:
        pytest.skip("no hipcc")
    out = str(tmp_path_factory.mktemp("asm") / "decode.s")
    subprocess.run([cc, *build.HIPCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-I", build.CSRC, "-S",
                    "--cuda-device-only", os.path.join(build.CSRC, "k_attn_decode.hip"), "-o", out],
                   check=True, capture_output=True)
    with open(out) as f:
        return f.read()


@pytest.mark.parametrize("small", [0, 1])
@pytest.mark.parametrize("dim", [64, 128])
def test_keys_before_values(listing, dim, small):
    name = f"_ZN3mxg4attn13decode_kernelILi{dim}ELb{small}EE"
    body = re.search(rf"^{name}\w*:.*?s_endpgm", listing, re.M | re.S).group(0)
    loads = re.findall(r"^\s+(global_load_lds_dwordx4|global_load_ubyte)", body, re.M)
    half = dim // 16 + 1
    assert len(loads) % half == 0 and len(loads) >= 4 * half    # keys and values, before and in the loop
    groups = [loads[i:i + half] for i in range(0, len(loads), half)]
    for i, g in enumerate(groups):
        assert g.count("global_load_ubyte") == 1, f"loads of keys and values mixed in group {i}: {g}"
