"""The waits between matrix products and the instructions that read their
sums, in the generated code of the row products (CPU only)."""
import concurrent.futures
import os
import re

import pytest

import submanifold_sparse_convolution_device_amd.build as lib_build
from test_mfma_waits import _assembly, early_reads


def test_row_products_wait_for_their_sums(tmp_path):
    if not os.path.exists(lib_build.HIPCC):
        pytest.skip("no hipcc")
    sources = [s for s in lib_build.SOURCES if s.startswith("linear_")]
    assert len(sources) == 3
    with concurrent.futures.ThreadPoolExecutor(len(sources)) as ex:
        texts = list(ex.map(lambda s: _assembly(s, str(tmp_path / (s + ".txt"))), sources))
    for text in texts:
        kernels = 0
        for m in re.finditer(r"^(_Z\S*):[^\n]*\n(.*?)\.end_amdhsa_kernel", text, re.S | re.M):
            kernels += "mfma" in m.group(2)
            assert not early_reads(m.group(2)), m.group(1)
        assert kernels >= 9  # three forms of three shapes or more
