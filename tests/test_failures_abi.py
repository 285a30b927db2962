"""include/moe_failures.h: the exported symbol, its exact C signature and its refusal (no GPU needed)."""
import os
import re
import shutil
import subprocess

import pytest

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "moe_failures.h")
SIGNATURES = {"moe_device_failure": "int (*)(int32_t, int32_t*, void*)"}


@pytest.fixture(scope="module")
def ops():
    from fp8_moe_layer_b200 import build
    build.build()
    from fp8_moe_layer_b200 import ops
    return ops


def test_signatures_are_those_declared_and_exported(ops, tmp_path):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    assert sorted(set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", text))) == sorted(SIGNATURES)
    for name, sig in SIGNATURES.items():
        assert len(getattr(ops.LIB, name).argtypes) == sig.count(",") + 1
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "sig.c"
    src.write_text("\n".join(['#include "moe_failures.h"'] + [
        sig.replace("(*)", f"(*p{i})", 1) + f" = {name};"
        for i, (name, sig) in enumerate(SIGNATURES.items())]) + "\n")
    res = subprocess.run([gcc, "-std=c11", "-Wall", "-Werror", "-c", str(src), "-o",
                          str(tmp_path / "sig.o"), f"-I{os.path.dirname(HEADER)}"],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr


def test_refuses_to_write_nowhere(ops):
    assert ops.LIB.moe_device_failure(0, None, None) == ops.MOE_ERR_INVALID_ARG
