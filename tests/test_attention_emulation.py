"""The tensor-core attention kernel's waits and barriers, its source compiled for the host.

attention_emulation/emulation.h models what the kernel synchronises with; here the kernel's
source gets calls in the place of its inline assembly. Usually no wait may run out; where one
completion comes later than the waits last the kernel has to end by itself, with nothing in
flight.
"""
import concurrent.futures
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HERE = os.path.join(ROOT, "tests", "attention_emulation")
CSRC = os.path.join(ROOT, "speculative_decoding_verification_sample_gb300", "csrc")

CALLS = [
    (r'asm volatile\("bar\.sync %0, 128;".*?;$', 'barrier(group + 1, 128, "sync", false, __LINE__);'),
    (r'asm volatile\(\s*"\{\\n\\t\.reg \.pred p, q;.*?: "memory"\);',
     'r = barrier(group + 1, 128, "red", x, __LINE__);'),
    (r'asm volatile\("bar\.sync 3, %0;" ::"n"\((.*?)\) : "memory"\);',
     r'barrier(3, \1, "sync", false, __LINE__);'),
    (r'asm volatile\("redux\.sync\.max\.f32.*?;$', "r = redux_max(x, __LINE__);"),
    (r'asm\("cvt\.rn\.f16x2\.f32.*?"=r"\((\w+(?:\[w\])?)\).*?;$', r"\1 = 0x3c003c00u;"),
    (r'asm\("sub\.rn\.f16x2.*?"=r"\((\w+)\) : "r"\((\w+)\).*?;$', r"\1 = \2;"),
    (r'asm\("add\.rn\.f16x2.*?;$', ";"),
]


def _kernel():
    """The kernel's source for the host."""
    def read(name):
        with open(os.path.join(CSRC, name)) as f:
            s = f.read()
        return s[s.index("namespace sv {"):]

    s = read("kv_q8_attention_tc.cu")
    s = s[:s.index("// ------------------------------------------------------------------ host")]
    for pattern, call in CALLS:
        s, n = re.subn(pattern, call, s, flags=re.S | re.M)
        assert n, pattern
    assert "asm" not in s
    s, n = re.subn(r"extern __shared__ .*? sm\[\];", "uint8_t* const sm = shared;", s)
    assert n == 1
    return ('#include "emulation.h"\n#include "specverify.h"\n' + read("q8_attn.cuh") + s
            + "}  // namespace sv\n")


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("emulation")
    (d / "kernel.h").write_text(_kernel())
    exe = d / "emulate"
    subprocess.run(["g++", "-O1", "-std=c++17", "-w", "-fsanitize=bounds", "-fno-sanitize-recover",
                    "-I", str(d), "-I", HERE, "-I", os.path.join(ROOT, "include"), "-o", str(exe),
                    os.path.join(HERE, "main.cpp")], check=True)
    return str(exe)


@pytest.mark.parametrize("stall", [0, 1])
def test_waits_and_barriers(program, stall):
    def run(first):
        return subprocess.run([program, str(first), str(first + 5), str(stall)], capture_output=True,
                              text=True, timeout=600)

    with concurrent.futures.ThreadPoolExecutor(os.cpu_count()) as pool:
        for r in pool.map(run, range(0, 40, 5)):
            assert r.returncode == 0 and r.stdout.endswith("done\n"), r.stdout[-600:] + r.stderr[-600:]
