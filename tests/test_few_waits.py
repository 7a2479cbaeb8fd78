"""The few-token layer's waits count their own polls: a clock would run on while the whole queue is
suspended, and end a wait whose result was only suspended too.  Reads the library built here from
source; no GPU."""
import os
import re
import shutil
import subprocess

import pytest

OBJDUMP = shutil.which("llvm-objdump", path="/opt/rocm/llvm/bin:" + os.environ.get("PATH", ""))


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """Symbol -> its instructions' names."""
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
        wanted = re.findall(r"\.text\s+\S+ .*?(\S*few_layer_kernel\S*)$", symbols.stdout, re.M)
        if not wanted:
            continue
        code = subprocess.run([OBJDUMP, "-d", "--disassemble-symbols=" + ",".join(wanted), name], cwd=folder,
                              check=True, capture_output=True, text=True).stdout
        symbol = None
        for line in code.splitlines():
            label = re.match(r"[0-9a-f]+ <(.*)>:", line)
            if label:
                symbol = label.group(1)
                found[symbol] = []
                continue
            op = line.split("//")[0].split()
            if symbol is not None and op:
                found[symbol].append(op[0])
    return found


def test_waits_read_no_clock(kernels):
    assert len(kernels) == 4      # one or two row groups of a wave, up and down
    for symbol, ops in kernels.items():
        assert "s_sleep" in ops, symbol      # the waits are there
        assert not [op for op in ops if op in ("s_memrealtime", "s_memtime")], symbol
