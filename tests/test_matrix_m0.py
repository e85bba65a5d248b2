"""The loads straight into the LDS set m0 in inline assembly, where no compiler can
be told of it: nothing else in the kernels that make them may hold a value there (no
GPU needed)."""
import os
import re
import shutil
import subprocess

import pytest

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
# instructions that read m0 without naming it
IMPLICIT = re.compile(r"^\s*(s_movrel\w*|v_movrel\w*|s_sendmsg\w*|ds_gws\w*|ds_\w*addtid\w*|ds_append|ds_consume|v_interp\w*|s_set_gpr_idx\w*|(?:global|buffer)_load_lds\w*)\b", re.M)
BLOCK = re.compile(r"^\s*;+#ASMSTART\n(.*?)^\s*;+#ASMEND\n", re.M | re.S)


def offences(body):
    """What of a kernel's assembly, outside its inline blocks, touches m0."""
    rest = BLOCK.sub("", body)
    rest = re.sub(r";[^\n]*", "", rest)
    return [m.group(0).strip() for m in re.finditer(r"^[^\n]*\bm0\b[^\n]*", rest, re.M)] + [m.group(1) for m in IMPLICIT.finditer(rest)]


def test_the_check_sees_other_uses():
    """On lines of assembly with a mistake in them."""
    block = "\t;;#ASMSTART\n\ts_mov_b32 m0, s4\n\ts_nop 0\n\tglobal_load_lds_dwordx4 v1, s[2:3]\n\t;;#ASMEND\n"
    assert offences("\tv_add_f32 v0, v1, v2\n" + block + "\ts_endpgm ; m0\n") == []
    for line in ("s_mov_b32 m0, s7", "s_mov_b32 s7, m0", "v_movrels_b32 v0, v1", "s_sendmsg sendmsg(1)", "global_load_lds_dwordx4 v1, s[2:3]"):
        assert offences("\t" + line + "\n" + block), line
        assert offences(block + "\t" + line + "\n" + block), line


def test_only_the_loads_use_m0(tmp_path):
    if not (os.path.exists(HIPCC) or shutil.which("hipcc")):
        pytest.skip("hipcc not available")
    from zero_sharded_mixed_partition_amd import build as B
    out = str(tmp_path / "orthogonalize.s")
    subprocess.run([HIPCC, f"--offload-arch={B.ARCH}", "-O3", "-std=c++17", "-fno-math-errno", f"-I{B.INCLUDE}", f"-I{B.CSRC}",
                    *B.DEVICE_FLAGS, "--cuda-device-only", "-S", os.path.join(B.CSRC, "orthogonalize.hip"), "-o", out],
                   check=True, capture_output=True)
    text, seen = open(out).read(), 0
    for m in re.finditer(r"^(_Z\S+):\s*; @", text, re.M):
        body = text[m.end():text.find(".section", m.end())]
        if "ortho_product" not in m.group(1):
            continue
        blocks = [b for b in BLOCK.findall(body) if "m0" in b]
        assert blocks and all("global_load_lds_dwordx4" in b and "s_mov_b32 m0" in b for b in blocks), m.group(1)
        assert offences(body) == [], m.group(1)
        seen += 1
    assert seen == 9
