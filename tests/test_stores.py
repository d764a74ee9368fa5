"""Wait states behind wide stores, in the code that was built here (no GPU).

A store of more than 8 bytes reads its data registers late: on gfx950 two wait states must pass before a VALU
instruction writes one of them.  The compiler keeps them after its own stores; after a store written in inline
assembly the text of the assembly has to."""
import os
import re
import shutil
import subprocess

import pytest

from dispatch_grouped_gemm_moe_amd import build

STATES = 2
WIDE = re.compile(r"^(global|flat|scratch|buffer)_store_(dwordx[34]|format_xyzw?)\b")
REGS = re.compile(r"\bv\[(\d+):(\d+)\]|\bv(\d+)\b")


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """{kernel: its instructions' text} of the library."""
    objdump = os.path.join(os.path.dirname(build.HIPCC), "..", "llvm", "bin", "llvm-objdump")
    if not os.path.exists(objdump):
        pytest.skip("no llvm-objdump beside hipcc")
    if not os.path.exists(build.lib_path()):
        build.build()
    at = tmp_path_factory.mktemp("code")
    shutil.copy(build.lib_path(), at)
    run = lambda *a: subprocess.run([objdump, *a], cwd=at, check=True, capture_output=True, text=True).stdout
    run("--offloading", build.LIB_NAME)
    found = {}
    for f in sorted(os.listdir(at)):
        if not f.endswith("gfx950"):
            continue
        for line in run("-d", f).splitlines():
            name = re.match(r"^[0-9a-f]+ <(.+)>:$", line)
            if name:
                code = found.setdefault(name[1], [])
            elif line.startswith("\t"):
                code.append(line.split("//")[0].strip())
    assert any("block_gemm_kernel" in k for k in found)
    return found


def _operands(instr):
    return [x.strip() for x in instr.split(None, 1)[1].split(",")] if " " in instr else []


def _registers(operand):
    m = REGS.match(operand)
    return set() if not m else {int(m[3])} if m[3] else set(range(int(m[1]), int(m[2]) + 1))


def _states(instr):
    nop = re.match(r"s_nop (\d+)", instr)
    return int(nop[1]) + 1 if nop else 1


def _early_writes(code):
    """(store, VALU instruction) pairs with fewer than STATES wait states between them, up to the next jump."""
    for i, instr in enumerate(code):
        if not WIDE.match(instr):
            continue
        ops = _operands(instr)
        data, waited = _registers(ops[0] if instr.startswith("buffer") else ops[1]), 0
        for after in code[i + 1:]:
            if waited >= STATES or after.startswith(("s_branch", "s_endpgm", "s_setpc")):
                break
            if after.startswith("v_") and _operands(after) and _registers(_operands(after)[0]) & data:
                yield instr, after
            waited += _states(after)


def test_the_check_itself():
    store = "global_store_dwordx4 v[2:3], v[4:7], off nt"
    assert list(_early_writes([store, "s_nop 0", "v_mov_b32_e32 v7, v1"]))
    assert list(_early_writes([store, "v_add_u32_e32 v4, v1, v2"]))
    assert list(_early_writes(["buffer_store_dwordx4 v[4:7], v2, s[0:3], 0 offen", "s_nop 0", "v_pk_mul_f16 v[6:7], v1, v2"]))
    assert not list(_early_writes([store, "s_nop 1", "v_mov_b32_e32 v7, v1"]))
    assert not list(_early_writes([store, "v_mov_b32_e32 v3, v1", "s_nop 0", "v_mov_b32_e32 v4, v1"]))
    assert not list(_early_writes([store, "s_branch 65496", "v_mov_b32_e32 v4, v1"]))
    assert not list(_early_writes(["global_store_dwordx2 v[2:3], v[4:5], off", "v_mov_b32_e32 v4, v1"]))


def test_no_wide_store_loses_its_data(kernels):
    bad = [(k, *pair) for k, code in kernels.items() for pair in _early_writes(code)]
    assert not bad, bad[:5]


def test_stores_in_asm_wait_whatever_follows(kernels):
    """Those of the products that leave the caches alone: both wait states stand in the asm, not in what the
    compiler happens to put behind it."""
    seen = 0
    for k, code in kernels.items():
        if "block_gemm_kernel" not in k:
            continue
        for i, instr in enumerate(code):
            if WIDE.match(instr) and re.search(r"\bnt\b", instr):
                seen += 1
                assert code[i + 1].startswith("s_nop") and _states(code[i + 1]) >= STATES, (k, instr, code[i + 1])
    assert seen
