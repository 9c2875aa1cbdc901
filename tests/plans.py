"""The forms that calls take, asked of the rules that the library is built with (plain C++, so no GPU is needed)."""
import functools
import os
import shutil
import subprocess
import tempfile

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "qlora_linear_layers_nf4_b200", "csrc")
SMS = 148   # of the device that the sizes in the tests are chosen for


@functools.lru_cache(maxsize=None)
def _program():
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    exe = os.path.join(tempfile.mkdtemp(), "plans")
    subprocess.run(["g++", "-O1", "-std=c++17", "-I", CSRC, "-o", exe, os.path.join(HERE, "native", "plans.cpp")], check=True)
    return exe


def ask(*queries):
    """A dict for each query, a tuple such as ("decode", m, n, k, SMS)."""
    text = "".join(" ".join(str(int(v) if not isinstance(v, str) else v) for v in q) + "\n" for q in queries)
    out = subprocess.run([_program()], input=text, capture_output=True, text=True, check=True).stdout.splitlines()
    assert len(out) == len(queries)
    words = [line.split() for line in out]
    return [{name: int(value) for name, value in zip(w[::2], w[1::2])} for w in words]
