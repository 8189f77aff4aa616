"""Compiled-code guard (host only) of the operators of a batch of many requests:
where lanes of one wave hand values to each other through LDS with no barrier,
the compiler is told so.  Without a fence it may move a lane's load over another
lane's store, as it only has to keep the order of each lane by itself; that a
build does not do it proves nothing for the next one, so this reads the code
before the optimiser."""

import os
import re
import shutil
import subprocess

import pytest

from quantized_routed_moe_amd import _build


def functions(source, tmp_path):
    """{name: body} of the device code of csrc/`source`, not optimised."""
    hipcc = _build.hipcc()
    if not os.path.exists(hipcc) and shutil.which(hipcc) is None:
        pytest.skip("hipcc not available")
    out = tmp_path / (source + ".ll")
    flags = [f for f in _build.COMMON if f != "-fPIC"]
    r = subprocess.run([hipcc, *flags, "--offload-device-only", "-S", "-emit-llvm", "-Xclang", "-disable-llvm-passes",
                        os.path.join(_build.CSRC, source), "-o", str(out)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    return {m[1]: m[2] for m in re.finditer(r"^define [^\n]*@(\w+)\([^\n]*\{\n(.*?)^\}", out.read_text(), re.M | re.S)}


def fences(body):
    return len(re.findall(r"call [^\n]*wave_lds_fence", body))


def check_fence(f):
    (body,) = [b for n, b in f.items() if "wave_lds_fence" in n]
    order = re.findall(r'fence syncscope\("wavefront"\) (\w+)|(wave\.barrier)', body)
    assert [a or b for a, b in order] == ["release", "wave.barrier", "acquire"]


def test_weights_turned_round_in_a_wave(tmp_path):
    """Every step but the first writes over the rows of the one before."""
    f = functions("lora.hip", tmp_path)
    check_fence(f)
    columns = [b for n, b in f.items() if re.match(r"_ZN5qrmoe12_GLOBAL__N_112make_columns", n)]
    assert len(columns) >= 16
    for body in columns:
        assert fences(body) == 2


def test_lists_sorted_in_a_wave(tmp_path):
    f = functions("scores.hip", tmp_path)
    check_fence(f)
    (sort,) = [b for n, b in f.items() if "TopList4sort" in n]
    assert fences(sort) == 4                    # listed, zeros behind, counted, stored
    joins = [b for n, b in f.items() if "join_row" in n]
    assert len(joins) == 2 and all(fences(b) == 1 for b in joins)
