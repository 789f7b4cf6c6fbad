"""Properties of the 4-bit key/value cache's sources and binding that no device is
needed for."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "token_skipping_sparse_step_b200", "csrc")


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_kernels_that_start_early_do_not_read_by_the_read_only_path():
    """What a kernel reads after griddepcontrol.wait was written while it lived."""
    waiting = []
    for name in sorted(os.listdir(CSRC)):
        if not re.match(r"(kv|attention)_quant.*\.cuh$", name):
            continue
        code = _code(name)
        if "grid_dependency_wait" not in code:
            continue
        waiting.append(name)
        assert not re.search(r"__ldg\s*\(|\.global\.nc\b", code), name
        assert not re.search(r"\bconst\s+\w+\s*\*\s*__restrict__", code), name
    assert waiting == ["attention_quant_rows.cuh", "attention_quant_tc.cuh", "kv_quant.cuh"]
