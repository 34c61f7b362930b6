"""The kernels over packed slots start while the kernel ahead of them on the stream may
still write what they read (it releases its dependents at its start, and they wait).
Nothing that they read is therefore read-only for their lifetime, as loads by the
read-only path have to be."""
import os
import re

import pytest

import kv_cache_compression_c128_gb300 as kvc


@pytest.mark.parametrize("name", ["kvc_reader.cu", "kvc_store.cu", "kvc_attend.cu", "kvc_evict.cu", "kvc_join.cu", "kvc_rotate.cu",
                                  "kvc_rotation.cuh", "kvc_codes.cuh"])
def test_no_read_only_loads(name):
    with open(os.path.join(kvc._CSRC, name)) as f:
        code = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
    assert not re.findall(r"__ldg|__ldlu|\.nc\b|__restrict__|ldu\.", code)
