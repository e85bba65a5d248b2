"""The generated gfx950 code of the list and 8-bit kernels (no GPU needed):
wide accesses carry the non-temporal hint and stay global (pointers read from a
table are generic to the compiler), nothing spills, and the 16-bit copy rounds
the stored float32 master (no fused fp16 mix instruction)."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
STREAMING = ("adam8_update", "pack8", "unpack8", "multi_adam", "multi_adam_devcoef", "multi_sqnorm")


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    if not (os.path.exists(HIPCC) or shutil.which("hipcc")):
        pytest.skip("hipcc not available")
    from zero_sharded_mixed_partition_amd import build as B
    found = {}
    for src in ("adam8", "multi_step"):
        out = str(tmp_path_factory.mktemp("asm") / f"{src}.s")
        subprocess.run([HIPCC, f"--offload-arch={B.ARCH}", "-O3", "-std=c++17", "-fno-math-errno", f"-I{B.INCLUDE}",
                        f"-I{B.CSRC}", *B.DEVICE_FLAGS, "--cuda-device-only", "-S", os.path.join(B.CSRC, src + ".hip"),
                        "-o", out], check=True, capture_output=True)
        text = open(out).read()
        for m in re.finditer(r"^(_Z\S+):\s*; @", text, re.M):
            meta = re.search(r"\.amdhsa_kernel " + re.escape(m.group(1)) + r"\n(.*?)\.end_amdhsa_kernel", text, re.S)
            found[m.group(1)] = (text[m.end():text.find(".section", m.end())], meta.group(1) if meta else "")
    return found


def kind(name):
    return next((k for k in sorted(STREAMING, key=len, reverse=True) if re.search(r"\d" + k + r"(I|E)", name)), None)


def test_every_kernel_is_present(kernels):
    assert set(STREAMING) <= {kind(n) for n in kernels}


def test_wide_accesses_are_global_and_non_temporal(kernels):
    for name, (body, _) in kernels.items():
        if kind(name) is None:
            continue
        assert not re.findall(r"^\s*(flat_\w+)", body, re.M), f"{name}: flat accesses"
        ops = re.findall(r"^\s*(global_(?:load|store)_dwordx[234])\b([^\n]*)", body, re.M)
        if kind(name) == "multi_sqnorm":                  # its stores are the partials
            ops = [o for o in ops if o[0].startswith("global_load")]
        assert ops, name
        assert all(o[1].rstrip().endswith(" nt") for o in ops), name


def test_nothing_spills(kernels):
    for name, (_, meta) in kernels.items():
        m = re.search(r"\.amdhsa_private_segment_fixed_size (\d+)", meta)
        assert m and int(m.group(1)) == 0, f"{name} uses scratch memory"


def test_the_copy_rounds_the_stored_master(kernels):
    for name, (body, _) in kernels.items():
        assert not re.findall(r"^\s*(v_(?:fma|mad)_mix(?:lo|hi)_f16)\b", body, re.M), name


def test_eight_bit_kernels_convert_in_hardware(kernels):
    for name, (body, _) in kernels.items():
        if kind(name) == "adam8_update" or re.search(r"multi_adam(_devcoef)?ILi8E", name):
            assert "v_cvt_scalef32_sr_fp8_f32" in body and "v_cvt_scalef32_pk_f32_fp8" in body, name
