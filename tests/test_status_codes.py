"""Status codes that kernels record: each has one number in the kernels, the header and the binding, and
says what happened."""
import os
import re

import pytest

ROOT = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..")
CSRC = os.path.join(ROOT, "packed_varlen_attention_modality_gb300", "csrc")


def _read(*path):
    with open(os.path.join(*path)) as f:
        return f.read()


@pytest.fixture(scope="module")
def h3():
    import __graft_entry__

    __graft_entry__.build()
    import packed_varlen_attention_modality_gb300 as h3

    h3.load_library()
    return h3


def test_device_codes_are_the_headers_and_the_bindings(h3):
    device = dict(re.findall(r"kErr(\w+) = (\d+)", _read(CSRC, "sm103_ptx.cuh")))
    header = dict(re.findall(r"(H3_ERR_\w+) = (\d+)", _read(ROOT, "include", "h3attn.h")))
    assert len(device) >= 4 and len(set(header.values())) == len(header)
    for name, number in device.items():
        public = "H3_ERR" + re.sub(r"([A-Z])", r"_\1", name).upper()
        assert header[public] == number
    for public, number in header.items():
        assert h3._STATUS[int(number)] == public
        assert h3.load_library().h3_status_string(int(number)) != b"unknown status"


def test_a_misplaced_shared_memory_block_is_no_timeout(h3):
    # the code of a timeout makes every later attention launch leave until it is read
    checks = [re.search(r"record_error\([^,]*, (\w+)\)", rest).group(1)
              for name in os.listdir(CSRC) if name.endswith(".cu")
              for rest in re.split(r"& 1023u\) != 0\)", _read(CSRC, name))[1:]]
    assert checks and all(c == "kErrSmemLayout" for c in checks)
    assert b"shared memory" in h3.load_library().h3_status_string(11)
    assert h3._STATUS[11] == "H3_ERR_SMEM_LAYOUT"
