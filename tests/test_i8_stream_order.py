"""The step-stream int8 kernels wait by a count of what they have issued, which holds only if each
step's copies to LDS are issued before its weight loads: the built code has them in that order.
Reads the library built here from source; no GPU."""
import os
import re
import shutil
import subprocess

import pytest

OBJDUMP = shutil.which("llvm-objdump", path="/opt/rocm/llvm/bin:" + os.environ.get("PATH", ""))


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """Symbol -> its memory operations as text: C a copy to LDS, L a load to registers, | a barrier."""
    if OBJDUMP is None:
        pytest.skip("no llvm-objdump")
    from prefill_sigmoid_router_amd import binding, build
    if not os.path.exists(binding.library_path()):
        build.build()
    folder = tmp_path_factory.mktemp("code")
    lib = shutil.copy(binding.library_path(), folder)
    subprocess.run([OBJDUMP, "--offloading", lib], cwd=folder, check=True, capture_output=True)
    found = {}
    for name in sorted(os.listdir(folder)):
        if "gfx950" not in name:
            continue
        symbols = subprocess.run([OBJDUMP, "-t", name], cwd=folder, check=True, capture_output=True, text=True)
        wanted = re.findall(r"\.text\s+\S+ .*?(\S*i8_grouped_kernel\S*)$", symbols.stdout, re.M)
        if not wanted:
            continue
        code = subprocess.run([OBJDUMP, "-d", "--disassemble-symbols=" + ",".join(wanted), name], cwd=folder,
                              check=True, capture_output=True, text=True).stdout
        symbol = None
        for line in code.splitlines():
            label = re.match(r"[0-9a-f]+ <(.*)>:", line)
            if label:
                symbol = label.group(1)
                found[symbol] = ""
                continue
            op = line.split("//")[0].split()
            if symbol is None or not op:
                continue
            if op[0] == "buffer_load_dwordx4":
                found[symbol] += "C" if "lds" in op else "L"
            elif op[0] == "s_barrier":
                found[symbol] += "|"
    return found


def test_every_step_copies_before_it_loads(kernels):
    assert len(kernels) == 24      # up, down, dense in two types; three heights; with a partial chunk or not
    for symbol, seq in kernels.items():
        rows, depth = map(int, re.search(r"4RingILi(\d+)ELi(\d+)E", symbol).groups())
        step = "C{%d}L{4}" % (rows // 64)      # copies and weight loads of a wave in a step
        first, *rest = seq.split("|")
        assert re.fullmatch("LLLL(%s){%d}" % (step, depth), first), (symbol, first)
        steps = [part for part in rest if part]
        assert len(steps) >= 2 * depth and all(re.fullmatch("(%s)+" % step, part) for part in steps), (symbol, rest)
