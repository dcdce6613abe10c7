"""The built libraries leave every matrix instruction the time that it takes
(on the host, from their listings)."""
import os
import shutil
import subprocess

import pytest

import matrix_waits
import state_space_model_ssm_amd as ssm
from state_space_model_ssm_amd.build import HIPCC

OBJDUMP = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(HIPCC))), "llvm", "bin", "llvm-objdump")
PATHS = {"libssm": ssm.library_path, "libssm_block": ssm.block_library_path, "libssm_delta": ssm.delta_library_path}


def listings(path, folder):
    """Of each source's device code in a library."""
    shutil.copy(path, folder)
    subprocess.check_output([OBJDUMP, "--offloading", os.path.basename(path)], cwd=folder)
    for name in sorted(os.listdir(folder)):
        if name.endswith("gfx950"):
            yield subprocess.check_output([OBJDUMP, "-d", os.path.join(folder, name)], text=True)


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no llvm-objdump")
@pytest.mark.parametrize("name", PATHS)
def test_no_result_is_read_too_soon(name, tmp_path):
    matrix = 0
    for listing in listings(PATHS[name](), tmp_path):
        for function, code in matrix_waits.functions(listing):
            matrix += sum(text.startswith("v_mfma") for text, _ in code)
            assert not matrix_waits.too_soon(code), function
    assert matrix > 500   # the listings were read


def listing(*lines):
    """As llvm-objdump prints it; `name:` marks a place, `-> name` a branch to it."""
    at, places, rows = 0x100, {}, []
    for line in lines:
        if line.endswith(":"):
            places[line[:-1]] = at
        else:
            rows.append((at, line))
            at += 4
    text = "0000000000000100 <kernel>:\n"
    for at, line in rows:
        line, _, to = line.partition(" -> ")
        text += f"\t{line:60} // {at:012X}: 00000000" + (f" <kernel+{places[to] - 0x100:#x}>" if to else "") + "\n"
    return text


MATRIX = "v_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[12:15], 0"
READ = "v_add_f32_e32 v20, v3, v20"


@pytest.mark.parametrize("lines,between", [
    ([MATRIX, "s_nop 7", READ], None), ([MATRIX, "s_nop 6", READ], 7), ([MATRIX, READ], 0),
    ([MATRIX, "s_nop 4", "v_mov_b32_e32 v30, 0", "global_store_dwordx4 v30, v[0:3], s[2:3]"], 6),
    # Over a branch, on the one side or the other, and around a loop.
    ([MATRIX, "s_cbranch_scc0 1 -> near", "s_nop 7", "near:", READ], 1),
    ([MATRIX, "s_cbranch_scc0 1 -> far", READ, "far:", "s_nop 7", "s_endpgm"], 1),
    ([MATRIX, "s_branch 1 -> end", READ, "end:", "s_endpgm"], None),
    (["head:", "s_nop 1", READ, "s_nop 7", MATRIX, "s_cbranch_scc1 0 -> head", "s_endpgm"], 3),
    # Another matrix instruction may add to the result, not multiply it.
    ([MATRIX, "v_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[12:15], v[0:3]", "s_nop 7", READ], None),
    ([MATRIX, "v_mfma_f32_16x16x32_bf16 v[4:7], v[0:3], v[12:15], 0"], 0),
    (["v_mfma_f32_32x32x16_bf16 v[0:15], v[20:23], v[24:27], 0", "s_nop 9", "ds_write_b128 v30, v[12:15]"], 10),
    (["v_mfma_f32_16x16x4_f32 a[0:3], v8, v9, 0", "s_nop 8", "v_accvgpr_read_b32 v1, a2"], 9),
    (["v_readfirstlane_b32 s4, v0", "s_nop 3", "global_load_dword v1, v2, s[4:5]"], 4),
    (["v_readfirstlane_b32 s4, v0", "s_nop 4", "global_load_dword v1, v2, s[4:5]"], None)])
def test_a_missing_wait_is_found(lines, between):
    (_, code), = matrix_waits.functions(listing(*lines, "s_endpgm"))
    assert {n for _, _, n in matrix_waits.too_soon(code)} == (set() if between is None else {between})
