"""The int8 quantiser's quotient, exhaustively: the corrected product by the
reciprocal gives the code of the IEEE quotient (no GPU)."""
import ctypes
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def emu(tmp_path_factory):
    lib = str(tmp_path_factory.mktemp("int8") / "libint8emu.so")
    subprocess.check_call(["gcc", "-O2", "-ffp-contract=off", "-shared", "-fPIC", "-o", lib,
                           os.path.join(HERE, "int8_emulation.c"), "-lm"])
    dll = ctypes.CDLL(lib)
    for fn in (dll.int8_quick_mismatches, dll.int8_tiny_mismatches):
        fn.restype, fn.argtypes = ctypes.c_int64, [ctypes.c_uint32] * 2
    return dll


def amax(exponent):
    """The bf16 bits of amax in [2^exponent, 2^(exponent + 1))."""
    return (exponent + 127) << 7, (exponent + 128) << 7


@pytest.mark.parametrize("exponent", [-64, -63, -20, -1, 0, 1, 40, 126, 127])
def test_quick_codes_of_every_value(emu, exponent):
    """Quotients depend on the significands and on how far the exponents are apart, unless
    something underflows or overflows: the ends of the range, and exponents inside it."""
    assert emu.int8_quick_mismatches(*amax(exponent)) == 0


def test_tiny_rows(emu):
    assert emu.int8_tiny_mismatches(1, 0x1F80) == 0
