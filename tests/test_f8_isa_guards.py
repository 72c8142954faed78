"""The gfx950 assembly of the 8-bit floating point products (compiled here from source, no GPU).

Their direct-to-LDS copies read M0, which only the copies' own inline asm may write: nothing else in those
kernels touches it, every copy follows a write of M0 in its basic block, and no register is spilled (a spill
in their main loops waits for every copy on its way)."""
import os
import re
import subprocess

import pytest

from tests.test_isa_guards import CSRC, FLAGS, HIPCC

SOURCES = ("f8_few.hip", "f8_tile.hip", "f8_large.hip")


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    d = tmp_path_factory.mktemp("isa")
    flags = [f for f in FLAGS if f != "-fPIC"]
    running = [(str(d / (src + ".s")), subprocess.Popen(
        [HIPCC, *flags, "--cuda-device-only", "-S", os.path.join(CSRC, src), "-o", str(d / (src + ".s"))],
        stdout=subprocess.DEVNULL, stderr=subprocess.DEVNULL)) for src in SOURCES]
    found = {}
    for out, p in running:
        assert p.wait() == 0, out
        asm = open(out).read()
        for name in re.findall(r"^(_Z\S*f8_(?:few|tile|gemm_large)_kernel\S*):", asm, flags=re.M):
            at = asm.index(name + ":")
            end = asm.index(".Lfunc_end", at)
            found[name] = asm[at:end], asm[end:end + 6000]
    return found


def test_every_source_is_there(kernels):
    for what, least in (("f8_few_kernel", 4), ("f8_tile_kernel", 10), ("f8_gemm_large_kernel", 4)):
        assert sum(what in n for n in kernels) >= least, what


def test_m0_belongs_to_the_copies(kernels):
    copies = 0
    for name, (body, _) in kernels.items():
        known = in_asm = False
        for line in body.splitlines():
            t = line.strip()
            if re.match(r"^\.LBB\w*:", t) or t.startswith(("s_cbranch", "s_branch")):
                known = False
            elif t.startswith(";;#ASMSTART"):
                in_asm = True
            elif t.startswith(";;#ASMEND"):
                in_asm = False
            elif in_asm and t.startswith("s_mov_b32 m0"):
                known = True
            elif t.startswith("global_load_lds_dword") or re.search(r"^buffer_load_dword\w*\b.*\blds\b", t):
                assert in_asm and known, f"{name}: copy without a write of M0 before it in its block: {t}"
                copies += 1
            elif not in_asm and not t.startswith(";"):
                assert not re.search(r"\bm0\b", t), f"{name}: M0 used outside the copies: {t}"
    assert copies > 100


def test_no_spills(kernels):
    for name, (_, tail) in kernels.items():
        m = re.search(r"ScratchSize: (\d+)", tail)
        assert m and int(m.group(1)) == 0, f"{name}: {m and m.group(0)}"
