"""What the channel operators' host side launches, and what it makes of launches
that fail: their translation units linked to a runtime that only writes launches
down.  No GPU is touched."""
import ctypes
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
UNITS = ("channel_desc.cpp", "linear.cu", "product.cu", "product_rows.cu", "layer_norm.cu")


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    from int8_conv2d_fprop_gb300 import _build, channel
    objects = [os.path.join(_build.OBJDIR, u + ".o") for u in UNITS]
    _build.build_library(force=not all(os.path.exists(o) for o in objects))
    so = str(tmp_path_factory.mktemp("fake") / "libfake.so")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_build.nvcc())))
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-o", so, os.path.join(HERE, "fake_cuda_runtime.cpp"),
                    "-I", _build.INCLUDE, "-I", _build.CSRC, "-I", os.path.join(cuda, "include")] + objects +
                   ["-Wl,-z,defs", "-Wl,-Bsymbolic"], check=True)
    lib = ctypes.CDLL(so)
    for name, args in (("conv_linear", 15), ("conv_linear_grad", 17), ("conv_layer_norm", 10), ("conv_layer_norm_grad", 17)):
        f = getattr(lib, name)
        f.restype = ctypes.c_int
        f.argtypes = [ctypes.c_void_p] * args
    lib.matrix = channel.MatrixDesc
    lib.linear_params, lib.norm_params = channel.LinearParams, channel.LayerNormParams
    return lib


FIRST, APART = 1 << 40, 1 << 36  # addresses that are never dereferenced
F32, F16, BF16 = 3, 4, 5
OK, ERR_CUDA = 0, 11


class Operand:
    """A matrix descriptor and an address for it."""
    count = 0

    def __init__(self, fake, rows, cols, dtype=BF16, row_stride=None, col_stride=1, shift=0):
        Operand.count += 1
        self.desc = fake.matrix(dtype, 0, rows, cols, row_stride or cols, col_stride, 1 << 50)
        self.at = FIRST + Operand.count * APART + shift

    def args(self):
        return ctypes.addressof(self.desc), self.at


def address():
    Operand.count += 1
    return FIRST + Operand.count * APART


def launches(fake):
    """(blocks, threads, shared memory, kernel, cluster size or 0) of each."""
    out = (ctypes.c_int64 * 80)()
    n = fake.fake_launches(out, 16)
    return [tuple(out[5 * i:5 * i + 5]) for i in range(n)]


def linear(fake, m, k, n, dtype=BF16, act=2, out=None, pad=0, residual=True, preact=True):
    ld = lambda c: c + pad  # noqa: E731
    x, w = Operand(fake, m, k, dtype, ld(k)), Operand(fake, n, k, dtype, ld(k))
    y = Operand(fake, m, n, out or dtype, ld(n))
    r, z = Operand(fake, m, n, out or dtype, ld(n)), Operand(fake, m, n, dtype, ld(n))
    none = (None, None)
    p = fake.linear_params(act, F32)
    return fake.conv_linear(*x.args(), *w.args(), address(), *(r.args() if residual else none),
                            *(z.args() if preact else none), *y.args(), ctypes.addressof(p), address(), APART, None)


def linear_grad(fake, m, k, n, dtype=BF16, act=2, pad=0):
    ld = lambda c: c + pad  # noqa: E731
    dy, z = Operand(fake, m, n, dtype, ld(n)), Operand(fake, m, n, dtype, ld(n))
    x, w = Operand(fake, m, k, dtype, ld(k)), Operand(fake, n, k, dtype, ld(k))
    dx, dw = Operand(fake, m, k, dtype), Operand(fake, n, k, dtype)
    p = fake.linear_params(act, F32)
    return fake.conv_linear_grad(*dy.args(), *x.args(), *w.args(), *z.args(), *dx.args(), *dw.args(), address(),
                                 ctypes.addressof(p), address(), APART, None)


def norm(fake, m, c, dtype=BF16):
    x, y = Operand(fake, m, c, dtype), Operand(fake, m, c, dtype)
    p = fake.norm_params(1e-5, 1.0, F32, 0)
    return fake.conv_layer_norm(*x.args(), address(), address(), *y.args(), address(), address(), ctypes.addressof(p), None)


def norm_grad(fake, m, c, dtype=BF16, col_stride=1):
    x, dy, dx = (Operand(fake, m, c, dtype, c * col_stride, col_stride) for _ in range(3))
    p = fake.norm_params(1e-5, 1.0, F32, 0)
    return fake.conv_layer_norm_grad(*dy.args(), *x.args(), address(), address(), address(), None, None, *dx.args(),
                                     address(), address(), ctypes.addressof(p), address(), APART, None)


CALLS = [lambda f: linear(f, 1, 1024, 1024), lambda f: linear(f, 300, 1024, 520, pad=1),
         lambda f: linear(f, 300, 20488, 520), lambda f: linear_grad(f, 40, 64, 64, act=0),
         lambda f: linear_grad(f, 40, 64, 64), lambda f: linear_grad(f, 5000, 65, 128),
         lambda f: linear_grad(f, 5000, 64, 129, pad=3), lambda f: linear_grad(f, 50176, 256, 1024),
         lambda f: norm(f, 100, 512), lambda f: norm(f, 100, 40000), lambda f: norm_grad(f, 100, 512),
         lambda f: norm_grad(f, 100, 5000), lambda f: norm_grad(f, 100, 512, col_stride=2)]


@pytest.mark.parametrize("call", range(len(CALLS)))
def test_a_failed_launch_ends_the_call(fake, call):
    fake.fake_reset(-1, 0)
    assert CALLS[call](fake) == OK
    count = len(launches(fake))
    assert count > 0
    for i in range(count):
        fake.fake_reset(i, 0)
        assert CALLS[call](fake) == ERR_CUDA
        assert len(launches(fake)) == i + 1  # nothing behind it


@pytest.mark.parametrize("call", range(len(CALLS)))
def test_an_earlier_error_is_not_this_calls(fake, call):
    fake.fake_reset(-1, 1)
    assert CALLS[call](fake) == OK
    assert fake.cudaGetLastError() != 0  # left for whose it is


def test_sizes_reach_the_forms_they_are_tested_for(fake):
    """The product's forms by what they launch: a cluster of 2 for each pair's
    tile, clusters of single CTAs that share one, a joining kernel behind sums
    cut into runs."""
    import channel_sizes as sizes

    def made(size):
        fake.fake_reset(-1, 0)
        assert linear(fake, *size) == OK
        return launches(fake)

    single, pairs = made((100, 64, 64))[0][3], made((50176, 512, 2048))[0][3]
    assert single != pairs
    for size in sizes.PAIR_TILES:
        (_, _, _, kernel, cluster), = made(size)
        assert kernel == pairs and cluster == 2, size
    for size in sizes.WIDE_SINGLE_TILES:
        (_, _, _, kernel, cluster), = made(size)
        assert kernel == single and cluster == 1, size
    for size in sizes.JOINED_RUNS + sizes.CUT_LAST_ROUND:
        first, join = made(size)
        assert first[3] == pairs and first[4] == 2 and join[3] not in (single, pairs), size
        tiles = -(-size[0] // 256) * -(-size[2] // 256)
        assert (tiles < 76) == (size in sizes.JOINED_RUNS), size
    for split, size in sizes.CLUSTERS:
        (_, _, _, kernel, cluster), = made(size)
        assert kernel == single and cluster == split, size
    for size in sizes.FEW_ROWS:
        _, threads, _, kernel, cluster = made(size)[-1]  # (behind the copies of rows that are not aligned)
        assert threads == 256 and cluster == 0, size
