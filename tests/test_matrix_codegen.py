"""The generated gfx950 code of the kernels over a list of matrices (no GPU
needed): nothing spills, no access is flat, the streaming passes' wide accesses
carry the non-temporal hint, the products run on the matrix cores and load
straight into the LDS, and the copies round the stored float32 master."""
import os
import re
import shutil
import subprocess

import pytest

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
KERNELS = {"matrix_momentum": 2, "matrix_update": 1, "ortho_squares": 1, "ortho_load": 1, "ortho_product": 9,
           "thin_gram": 3, "thin_steps": 3, "thin_apply": 3}


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    if not (os.path.exists(HIPCC) or shutil.which("hipcc")):
        pytest.skip("hipcc not available")
    from zero_sharded_mixed_partition_amd import build as B
    found = {}
    for src in ("matrix_step", "orthogonalize", "orthogonalize_thin"):
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
    return next((k for k in KERNELS if re.search(r"\d" + k + r"(I|E)", name)), None)


def test_every_kernel_is_present(kernels):
    count = {}
    for n in kernels:
        count[kind(n)] = count.get(kind(n), 0) + 1
    assert {k: count.get(k) for k in KERNELS} == KERNELS


def test_nothing_spills_and_nothing_is_flat(kernels):
    for name, (body, meta) in kernels.items():
        m = re.search(r"\.amdhsa_private_segment_fixed_size (\d+)", meta)
        assert m and int(m.group(1)) == 0, f"{name} uses scratch memory"
        assert not re.findall(r"^\s*(flat_\w+)", body, re.M), f"{name}: flat accesses"


def test_streams_are_non_temporal(kernels):
    for name, (body, _) in kernels.items():
        if kind(name) not in ("matrix_momentum", "matrix_update"):
            continue
        ops = re.findall(r"^\s*(global_(?:load|store)_dwordx[24])\b([^\n]*)", body, re.M)
        assert ops and all(o[1].rstrip().endswith(" nt") for o in ops), name
        assert not re.findall(r"^\s*(v_(?:fma|mad)_mix(?:lo|hi)_f16)\b", body, re.M), name


def test_products_run_on_the_matrix_cores(kernels):
    for name, (body, _) in kernels.items():
        if kind(name) in ("ortho_product", "thin_gram", "thin_steps", "thin_apply"):
            assert "v_mfma_f32_16x16x32_f16" in body, name
        if kind(name) == "ortho_product":
            assert "global_load_lds_dwordx4" in body, name
        if kind(name) == "ortho_product" and re.search(r"ILi\d+ELi\dELi\dELi2E", name):
            assert "ds_read_b64_tr_b16" in body, name
