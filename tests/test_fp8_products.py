"""The scaled matrix instructions of the FP8 GEMMs are read in the basic block
they stand in: across blocks the compiler has left too few wait states."""
import os
import re
import subprocess

import pytest

from bit_quantized_video_amd import build

REGS = re.compile(r"v\[(\d+):(\d+)\]|v(\d+)")


def registers(text):
    return {r for a, b, c in REGS.findall(text) for r in range(int(a or c), int(b or c) + 1)}


def products_read_elsewhere(listing):
    """(number of scaled products, those whose first reader or overwriter is in
    another block than they are) of an assembly listing."""
    code = [t.strip() for t in (line.split(";")[0] for line in listing.splitlines())]
    code = [t for t in code if t and (t.endswith(":") or not t.startswith("."))]
    count, bad = 0, []
    for i, t in enumerate(code):
        if not t.startswith("v_mfma_scale"):
            continue
        count += 1
        result = registers(t.split(None, 1)[1].split(",")[0])
        for u in code[i + 1:]:
            if u.endswith(":") or re.match(r"s_(c?branch|endpgm|setpc)", u):
                bad.append((i, t, u))
                break
            if registers(u) & result:
                break
    return count, bad


def test_the_check_sees_a_reader_in_another_block():
    product = "v_mfma_scale_f32_16x16x128_f8f6f4 v[0:3], v[8:15], v[16:23], 0, v40, v40 op_sel_hi:[0,0,0]\n"
    read = "v_fmac_f32_e32 v50, v2, v60\n"
    assert products_read_elsewhere(product + "s_nop 7\nv_mov_b32_e32 v9, v10\n" + read) == (1, [])
    for between in (".LBB0_1:\n", "s_cbranch_scc1 .LBB0_2\n"):
        count, bad = products_read_elsewhere(product + between + read)
        assert count == 1 and len(bad) == 1


def test_products_are_read_in_their_block(tmp_path):
    if not os.path.exists(build.HIPCC):
        pytest.skip("hipcc not found")
    out = tmp_path / "gemm_fp8.s"
    subprocess.check_call([build.HIPCC, *[f for f in build.FLAGS if f not in ("-shared", "-fPIC")], "-S",
                           "--offload-device-only", "-I", build.INCLUDE, "-I", build.CSRC,
                           os.path.join(build.CSRC, "gemm_fp8.hip"), "-o", str(out)], stderr=subprocess.DEVNULL)
    count, bad = products_read_elsewhere(out.read_text())
    assert count >= 100 and bad == []
