"""GPU: the short root and quotient of the 8-bit update equal sqrtf and / bit for
bit, on every float the root is used for and on every quotient that the bound of
test_short_forms.py leaves in doubt (tests/kernels/short_forms.hip, built by
__graft_entry__.build())."""
import ctypes
import os
import random
import struct

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SO = os.path.join(ROOT, "tests", "kernels", "short_forms.so")


@pytest.fixture(scope="module")
def compare():
    """(values compared, values that differ) of one check."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    assert os.path.exists(SO), "tests/kernels/short_forms.so is not built: run __graft_entry__.build()"
    lib = ctypes.CDLL(SO)
    counts = torch.zeros(2, dtype=torch.int64, device="cuda")

    def run(name, *args):
        counts.zero_()
        torch.cuda.synchronize()
        assert getattr(lib, name)(*args, ctypes.c_void_p(counts.data_ptr())) == 0
        torch.cuda.synchronize()
        return tuple(counts.tolist())
    return run


def bits(x):
    return struct.unpack("<I", struct.pack("<f", x))[0]


def test_every_root(compare):
    lo, hi = bits(2.0 ** -96), bits(float("inf"))
    assert compare("check_roots", ctypes.c_uint32(lo), ctypes.c_uint32(hi)) == (hi - lo, 0)


def test_every_reciprocal(compare):
    assert compare("check_reciprocals") == (1 << 23, 0)


@pytest.mark.parametrize("radius", [6, 64])
def test_every_quotient_near_a_middle(compare, radius):
    """The bound is 5.01/(2D) (radius 6 covers it); 64 is far beyond."""
    compared, differ = compare("check_hard_quotients", ctypes.c_int(radius))
    # an odd D (2^22 of them) leaves radius offsets of its parity, of which ln 2 have a numerator in range (2.9M a
    # unit of radius); D = 2^j Do has 2^-j of the offsets and 2^j of the numerators, so all even ones add as many
    assert compared > radius << 22 and differ == 0


def test_every_numerator_of_some_divisors(compare):
    rng = random.Random(5)
    for d in [0, 1, 0x3FFFFF, 0x400000, 0x7FFFFE, 0x7FFFFF] + [rng.randrange(1 << 23) for _ in range(100)]:
        assert compare("check_numerators", ctypes.c_uint32(d)) == (1 << 23, 0), d


def test_exponents_of_the_usual_range(compare):
    n = 1 << 30
    assert compare("check_exponents", ctypes.c_uint64(n), ctypes.c_uint64(11)) == (n, 0)
