"""The shapes that the GPU tests of gdn_linear multiply reach every kernel that
it has (the choice is made on the host, so this runs without a GPU)."""
import ctypes
import os

import pytest

import gated_deltanet_tree_gdn_amd as gdn
from gated_deltanet_tree_gdn_amd import layer

THIN, ANY, TILE64_TWO, TILE64, TILE128_TWO, TILE128, TILE256 = range(7)

# M, N, K, elements between rows of x and w (None: K), kernel, with the code for ends of K, tiles cut
SHAPES = [
    (5, 300, 512, None, THIN, False, 0),
    (16, 8192, 264, None, THIN, False, 0),
    (7, 1000, 333, None, THIN, True, 0),
    (100, 200, 333, 333, ANY, True, 0),
    (40, 130, 4096, (1 << 21) + 8, ANY, True, 0),    # too far apart for direct loads
    (1, 12352, 4096, None, TILE64_TWO, False, 0),
    (100, 1000, 1088, None, TILE64_TWO, False, 0),
    (100, 1000, 1096, None, TILE64_TWO, True, 0),
    (100, 1000, 1091, 1096, TILE64_TWO, True, 0),
    (1100, 4100, 256, None, TILE64, False, 0),
    (1100, 4100, 248, None, TILE64, True, 0),
    (1100, 4100, 243, 248, TILE64, True, 0),
    (777, 4096, 4096, None, TILE128_TWO, False, 0),
    (777, 4096, 4104, None, TILE128_TWO, True, 0),
    (777, 4096, 4095, 4096, TILE128_TWO, True, 0),
    (777, 4096, 4095, 4095, TILE128_TWO, False, 0),  # both copied to rows of 4096
    (2048, 3900, 2048, None, TILE128, False, 0),
    (2048, 3900, 2056, None, TILE128, True, 0),
    (2048, 3900, 2045, 2048, TILE128, True, 0),
    (3900, 4000, 1024, None, TILE256, False, 0),
    (4300, 4096, 1024, None, TILE256, False, 16),
    (4300, 4096, 1032, None, TILE256, True, 16),
    (4300, 4096, 1027, 1032, TILE256, True, 16),
    (3900, 4000, 1027, 1032, TILE256, True, 0),
]


class Choice(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int), ("tail", ctypes.c_bool), ("cut", ctypes.c_int)]


def choice(M, N, K, stride):
    if not os.path.exists(gdn.LIB_PATH):
        pytest.fail("libgdn_tree.so is not built: run __graft_entry__.build()")
    fn = layer.layer_library()._ZN3gdn13linear_choiceERK15gdn_linear_dims
    fn.argtypes, fn.restype = [ctypes.POINTER(layer.LinearDims)], Choice
    s = stride or K
    c = fn(layer.LinearDims(M, N, K, 1, 1, 0, 1.0, s, s, N, N))
    return c.kernel, c.tail, c.cut


@pytest.mark.parametrize("M,N,K,stride,kernel,tail,cut", SHAPES)
def test_choice(M, N, K, stride, kernel, tail, cut):
    assert choice(M, N, K, stride) == (kernel, tail, cut)


def test_every_kernel_is_reached():
    got = {(kernel, tail, cut > 0) for _, _, _, _, kernel, tail, cut in SHAPES}
    both = {(k, t, False) for k in (THIN, TILE64_TWO, TILE64, TILE128_TWO, TILE128, TILE256) for t in (False, True)}
    assert got == both | {(ANY, True, False), (TILE256, False, True), (TILE256, True, True)}
