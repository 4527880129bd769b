"""CPU sanitizer run of the host code of the operators around the table: the
argument checks of every entry point under AddressSanitizer and
UndefinedBehaviorSanitizer, in a child process."""

import os

import pytest
from test_sanitizers import _run_child


def test_operator_entry_points_under_sanitizers(tmp_path):
    from tensor_train_compressed_gather_amd import build as hipbuild

    try:
        rt = hipbuild.asan_runtime()
    except FileNotFoundError as e:
        pytest.skip(str(e))
    lib = hipbuild.build_host_sanitized(str(tmp_path / "libtt_emb_asan.so"))
    out = _run_child([os.path.join("tests", "test_lm_abi.py")], {"TT_EMB_LIB": lib, "LD_PRELOAD": rt}, timeout=600)
    assert " passed" in out
