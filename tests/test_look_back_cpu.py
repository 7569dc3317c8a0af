"""The look-back's choice of the state it starts from, under random orders of publication."""
import ctypes
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "causal_prefix_scan_gb300", "csrc")


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("look_back") / "model.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-ffp-contract=off", "-Wall", "-shared", "-fPIC", f"-I{CSRC}",
                    os.path.join(HERE, "look_back_model.cpp"), "-o", out], check=True)
    fn = ctypes.CDLL(out).look_back_model
    fn.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_uint64, ctypes.c_float, ctypes.c_void_p]
    fn.restype = ctypes.c_int
    return fn


@pytest.mark.parametrize("gate", [1.0, 0.999])
@pytest.mark.parametrize("tiles,behind", [(1, 0), (7, 7), (63, 63), (64, 64), (65, 64), (256, 40), (256, 57), (256, 60),
                                          (256, 62), (256, 64), (256, 66), (256, 100), (256, 256)])
def test_every_channel_gets_the_state_before_its_tile(model, tiles, behind, gate):
    want = 0.0
    for _ in range(tiles):
        want = gate * want + 1.0  # exact in fp32 with a gate of one, the same operations otherwise
    rounds = set()
    for seed in range(200):
        out = (ctypes.c_float * 64)()
        rounds.add(model(tiles, 64, behind, seed, gate, out))
        if gate == 1.0:
            assert list(out) == [want] * 64, (seed, rounds)
        else:
            assert max(abs(x - want) for x in out) <= want * 256 * 2.0 ** -24, (seed, rounds)
    if (tiles, behind) == (256, 256):
        assert max(rounds) > 8  # the last window was read again
