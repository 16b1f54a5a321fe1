"""The state stores in the built code (no GPU needed).

A 16-byte buffer store with a scalar register as its offset, followed at once by a vector instruction that overwrites its
data register, has stored the new value in some lanes: no wait is put between the two for that form of store. So none is
followed by any vector instruction but another store: the kernels' stores of the state are the last that they do.
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
def test_nothing_overwrites_what_a_wide_store_still_reads(name, tmp_path):
    out = str(tmp_path / "device.s")
    subprocess.run([b._hipcc(), *b.HIPCC_FLAGS, "--cuda-device-only", "-S", os.path.join(b.CSRC, name), "-o", out],
                   check=True, capture_output=True)
    stores, open_store = 0, None  # a store with a scalar offset since which nothing but scalar work and stores came
    with open(out) as f:
        for line in f:
            line = line.split(";")[0].strip()
            #                       data, address, resource, scalar offset
            if re.match(r"buffer_store_dwordx[34] .*s\[\d+:\d+\], s\d+", line):
                stores, open_store = stores + 1, line
            elif line.startswith("s_endpgm"):
                open_store = None
            elif open_store:
                assert not re.match(r"(v_|ds_|global_|flat_|scratch_|buffer_load|buffer_atomic)", line), (open_store, line)
    assert stores and open_store is None
