"""The cross entropy's products in the built library. They are written as assembly, whose
results the compiler does not know to be late: this reads the machine code that it made
around them. Needs no GPU."""

import glob
import os
import re
import shutil
import subprocess

import pytest

q = pytest.importorskip("quantized_weight_backward_amd")

OBJDUMP = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "llvm-objdump")
KERNEL = "_ZN5retro2ce14product_kernel"
# of a 16 x 16 x 32 product, 8 passes, until another instruction may touch its result
WAIT = 11


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """{name: [(address, instruction, branch's target)]} of every product kernel."""
    if not os.path.exists(OBJDUMP):
        pytest.skip("llvm-objdump is not installed")
    at = tmp_path_factory.mktemp("code")
    lib = shutil.copy(q.LIB_PATH, at)
    subprocess.run([OBJDUMP, "--offloading", lib], check=True, capture_output=True, cwd=at)
    out = {}
    for path in glob.glob(str(at / "*gfx950*")):
        with open(path, "rb") as f:
            if KERNEL.encode() not in f.read():
                continue
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", path], check=True, capture_output=True, text=True).stdout
        name, base = None, 0
        for line in text.splitlines():
            head = re.match(r"([0-9a-f]+) <(\S+)>:", line)
            if head:
                name, base = head[2], int(head[1], 16)
                if name.startswith(KERNEL):
                    out[name] = []
            elif name in out and "//" in line:
                code, note = line.split("//", 1)
                to = re.search(r"<\S+?(?:\+0x([0-9a-f]+))?>", note)
                out[name].append((int(note.split(":")[0], 16), code.strip(), base + int(to[1] or "0", 16) if to else None))
    return out


def registers(text):
    found = {int(r) for r in re.findall(r"\bv(\d+)\b", text)}
    for a, b in re.findall(r"\bv\[(\d+):(\d+)\]", text):
        found.update(range(int(a), int(b) + 1))
    return found


def early(code):
    """Instructions that some path brings to a product's result before its wait is over."""
    index = {address: i for i, (address, _, _) in enumerate(code)}
    product = [c.startswith("v_mfma") for _, c, _ in code]
    result = [registers(c.split(None, 1)[1].split(",")[0]) if p else set() for (_, c, _), p in zip(code, product)]
    results = set().union(*result)
    touches = [set() if p else registers(c) & results for (_, c, _), p in zip(code, product)]
    states = [int(c.split()[1]) + 1 if c.startswith("s_nop") else 1 for _, c, _ in code]
    # wait states since each result was written, on the path that leaves fewest
    seen, work, found = [None] * len(code), [(0, {})], set()
    while work:
        i, since = work.pop()
        while i < len(code):
            if seen[i] is not None:
                if all(seen[i].get(r, WAIT) <= n for r, n in since.items()):
                    break
                since = {r: min(since.get(r, WAIT), seen[i].get(r, WAIT)) for r in since.keys() | seen[i].keys()}
            seen[i] = since
            _, text, to = code[i]
            if any(r in since for r in touches[i]):
                found.add(text)
            since = {r: n + states[i] for r, n in since.items() if n + states[i] < WAIT}
            since.update(dict.fromkeys(result[i], 0))
            if to is not None and "branch" in text:
                work.append((index[to], since))
            if text.startswith(("s_endpgm", "s_branch")):
                break
            i += 1
    return found


def test_results_stay_where_they_are(kernels):
    """No result is spilled or moved to the other register file, and none is read or written by
    another instruction until it is there."""
    assert len(kernels) >= 40
    for name, code in kernels.items():
        products = [c for _, c, _ in code if c.startswith("v_mfma")]
        assert products, name
        for c in products:  # one register is both what is added to and what becomes of it
            parts = [p.strip() for p in c.split(None, 1)[1].split(",")]
            assert parts[0] == parts[3], (name, c)
        assert not [c for _, c, _ in code if c.startswith(("scratch_", "v_accvgpr"))], name
        assert not early(code), (name, early(code))


def test_the_reader_finds_what_is_early():
    """The same reading of code that is wrong, made up here."""
    product = "v_mfma_f32_16x16x32_f16 v[4:7], v[8:11], v[12:15], v[4:7]"
    end = "s_endpgm"

    def code(*lines):
        return [(4 * i, c, None) if isinstance(c, str) else (4 * i, c[0], 4 * c[1]) for i, c in enumerate(lines)]

    assert early(code(product, "v_mov_b32_e32 v0, v5", end))
    assert early(code(product, "s_nop 9", "v_mov_b32_e32 v5, v0", end))
    assert not early(code(product, "s_nop 10", "v_mov_b32_e32 v0, v5", end))
    assert not early(code(product, product, "v_mov_b32_e32 v0, v8", end))
    # a path around the wait; a loop's second turn
    assert early(code(product, ("s_cbranch_scc0 1", 3), "s_nop 15", "v_mov_b32_e32 v0, v5", end))
    assert early(code("v_mov_b32_e32 v4, 0", product, ("s_cbranch_scc0 65533", 0), end))
    assert not early(code(product, ("s_branch 1", 3), "v_mov_b32_e32 v0, v5", end))
