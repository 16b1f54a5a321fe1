"""The form of the state stores in the built code (no GPU needed).

A 16-byte buffer store with a scalar register as its offset, followed at once by a vector instruction that overwrites its
data register, has stored the new value in some lanes: no wait is put between the two for that form of store. So no
kernel may hold one, whatever the compiler schedules after it.
"""

import os
import re
import subprocess

import pytest

from delta_rule_recurrent_gdn_amd import build as b

SOURCES = [n for n in sorted(os.listdir(b.CSRC))
           if n.endswith((".hip", ".h")) and "raw_buffer_store" in open(os.path.join(b.CSRC, n)).read()]


def test_every_source_with_buffer_stores_is_a_unit_of_its_own():
    assert all(n.endswith(".hip") for n in SOURCES), SOURCES  # a header's would be compiled with its users


@pytest.mark.parametrize("name", SOURCES)
def test_no_wide_buffer_store_with_a_scalar_offset(name, tmp_path):
    out = str(tmp_path / "device.s")
    subprocess.run([b._hipcc(), *b.HIPCC_FLAGS, "--cuda-device-only", "-S", os.path.join(b.CSRC, name), "-o", out],
                   check=True, capture_output=True)
    with open(out) as f:
        stores = re.findall(r"^\s*(buffer_store_dwordx[34] .*)$", f.read(), re.M)
    assert stores
    #                       data, address, resource, scalar offset
    scalar = [s for s in stores if re.search(r"s\[\d+:\d+\], s\d+", s)]
    assert not scalar, (len(scalar), len(stores), scalar[0])
