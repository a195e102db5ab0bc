"""The package without a usable compiled binding of the operators: the GEMMs import and refuse as ever, the
operators raise ImportError when they are called."""
from __future__ import annotations

import pathlib
import shutil
import subprocess
import sys

import pytest

import moe_grouped_gemm_08_b200 as fg

SCRIPT = """
import torch
{before}
import moe_grouped_gemm_08_b200 as fg
assert fg.LIB_PATH.parent.parent.samefile({where!r}), fg.LIB_PATH
assert fg.lib.fp8_gemm_nt(None, None, None, None, None, 1, 8, 16, None) == 1
assert fg.moe_layout_rows(10, 4) == 4 * 128
for call in (lambda: fg.moe_route(torch.zeros(4, 8), 2),
             lambda: fg.lora_add(*[torch.zeros(1)] * 5)):
    try:
        call()
    except ImportError as e:
        assert "_operators.so" in str(e) and "build" in str(e), e
    else:
        raise AssertionError("no ImportError")
"""


def copied(tmp_path):
    """A copy of the package with its library, but not the binding."""
    package = pathlib.Path(fg.__file__).parent
    to = tmp_path / package.name
    shutil.copytree(package, to, ignore=shutil.ignore_patterns("_operators.so", "*_debug.so", "csrc", "__pycache__"))
    return to


def run(where, before=""):
    subprocess.run([sys.executable, "-c", SCRIPT.format(where=str(where), before=before)], cwd=where, check=True,
                   env={"PATH": "/usr/bin:/bin", "PYTHONPATH": str(where)})


@pytest.mark.parametrize("broken", [False, True])
def test_gemms_work_without_the_operators_binding(tmp_path, broken):
    to = copied(tmp_path)
    if broken:  # one that the loader refuses
        (to / "_operators.so").write_bytes(b"not a library")
    run(tmp_path)


def test_a_binding_built_for_another_torch_is_not_used():
    run(pathlib.Path(fg.__file__).parent.parent, 'torch.__version__ = "1.99.0+cu999"')
