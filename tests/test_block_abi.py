"""Host-side tests of the learner's block entry points (no GPU, nothing
launched): argument checks before any device work, and what the compiled
kernels hold."""

import ctypes
import inspect
import os
import re

import pytest

from test_device_code import ASM_MEM, _compile, needs_hipcc
from invariant_token_logprobs_lm_amd import build

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
v = ctypes.c_void_p
M = 1 << 24  # arrays of the calls below lie this far apart


@pytest.fixture(scope="module")
def itl():
    import invariant_token_logprobs_lm_amd as itl

    return itl


def _spec(itl, p=0.1, seed=64 * M, site=0, first_row=0):
    return itl._DropoutSpec(seed, first_row, site, p)


def test_dropout_arguments(itl):
    def f(x=M, y=2 * M, dt=0, n=4, d=64, **spec):
        return itl.lib.itl_dropout(v(x), dt, n, d, _spec(itl, **spec), v(y), None)

    assert f(n=0, x=0, y=0) == OK
    assert f(n=-1) == INVALID and f(d=0) == INVALID and f(dt=2) == UNSUPPORTED
    assert f(n=1 << 31) == UNSUPPORTED and f(d=(1 << 24) + 1) == UNSUPPORTED
    assert f(x=0) == INVALID and f(y=0) == INVALID and f(x=M + 8) == INVALID and f(y=2 * M + 1, d=63) == INVALID
    for p in (-0.1, 1.1, float("nan"), float("inf")):
        assert f(p=p) == INVALID and "p must be" in itl.lib.itl_last_error().decode()
    assert f(seed=0) == INVALID and f(seed=64 * M + 4) == INVALID
    assert f(first_row=-1) == INVALID and f(first_row=2 ** 63 - 4) == INVALID
    assert f(y=M + 16) == INVALID and f(seed=2 * M) == INVALID  # y over part of x, over the seed
    assert itl.lib.itl_dropout(v(M), 0, 4, 64, None, v(M), None) == INVALID


def test_norm_with_dropout_arguments(itl):
    def f(x=M, y=2 * M, h=3 * M, u=4 * M, d=64, spec=True, **kw):
        return itl.lib.itl_residual_norm_dropout(v(x), v(y), None, 0, None, v(5 * M), 0, 4, d, 1.0, 1e-6,
                                                 _spec(itl, **kw) if spec else None, v(h), v(u), None, None, None)

    assert f(spec=False) == INVALID and f(p=2.0) == INVALID and f(seed=0) == INVALID and f(first_row=-1) == INVALID
    assert f(y=0) == INVALID and f(u=0) == INVALID and f(seed=4 * M) == INVALID

    def b(y=2 * M, dy=3 * M, spec=True, ws=7 * M, **kw):
        return itl.lib.itl_residual_norm_dropout_backward(v(M), 1, None, v(4 * M), v(y), None, 0, None, v(5 * M), v(6 * M),
                                                          None, 0, 4, 64, 1.0, _spec(itl, **kw) if spec else None, v(8 * M),
                                                          v(dy), None, v(9 * M), None, v(ws), 1 << 20, None)

    assert b(spec=False) == INVALID and b(p=-1.0) == INVALID and b(y=0) == INVALID and b(dy=0) == INVALID
    assert b(seed=0) == INVALID and b(ws=0) == WORKSPACE and b(seed=8 * M) == INVALID

    def q(d=128, codes=4 * M, scale=6 * M, y=2 * M, spec=None, n=4):
        return itl.lib.itl_residual_norm_blocks_fp8(v(M), v(y), None, 0, None, v(5 * M), 0, n, d, 1.0, 1e-6, spec, v(3 * M),
                                                    v(codes), v(scale), None, None, None)

    assert q(n=0) == OK and q(d=64) == UNSUPPORTED and q(codes=4 * M + 4) == INVALID and q(scale=0) == INVALID
    assert q(scale=4 * M) == INVALID and q(y=0, spec=_spec(itl)) == INVALID and q(spec=_spec(itl, p=3.0)) == INVALID
    assert q(scale=3 * M + 4 * 2048 - 60, d=1024) == INVALID  # the first of them lie in h's last row


@pytest.mark.parametrize("name", ["itl_quantize_blocks_fp8", "itl_quantize_tiles_fp8"])
def test_quantize_arguments(itl, name):
    def f(X=M, dt=0, n=4, d=100, Xq=2 * M, s=3 * M, Xtq=4 * M, ts=5 * M):
        return getattr(itl.lib, name)(v(X), dt, n, d, v(Xq), v(s), v(Xtq), v(ts), None)

    assert f(n=0, X=0, Xq=0, Xtq=0) == OK
    assert f(n=-1) == INVALID and f(d=0) == INVALID and f(dt=9) == UNSUPPORTED
    assert f(n=1 << 31) == UNSUPPORTED and f(d=(1 << 23) + 1) == UNSUPPORTED
    assert f(X=0) == INVALID and f(Xq=0, Xtq=0) == INVALID and f(s=0) == INVALID and f(ts=0) == INVALID
    assert f(X=M + 1) == INVALID and f(Xq=2 * M + 8) == INVALID and f(Xtq=4 * M + 8) == INVALID
    assert f(Xq=M) == INVALID and f(Xtq=2 * M + 496) == INVALID and f(s=M + 796) == INVALID
    assert f(ts=4 * M + 128 * 99 + 124) == INVALID  # inside Xtq's last row


def test_product_arguments(itl):
    def f(A=M, sa=2 * M, B=3 * M, sb=4 * M, m=4, n=5, k=128, dt=0, C=5 * M):
        return itl.lib.itl_matmul_fp8_blocks(v(A), v(sa), v(B), v(sb), m, n, k, dt, v(C), None)

    assert f(m=0, A=0, C=0) == OK and f(n=0, B=0, C=0) == OK
    assert f(m=-1) == INVALID and f(n=-1) == INVALID and f(k=-128) == INVALID
    assert f(k=64) == UNSUPPORTED and f(dt=7) == UNSUPPORTED and f(k=(1 << 23) + 128) == UNSUPPORTED
    assert f(m=1 << 31) == UNSUPPORTED and f(n=1 << 31) == UNSUPPORTED and f(m=1 << 30, n=1 << 11) == UNSUPPORTED
    for name in ("A", "sa", "B", "sb", "C"):
        assert f(**{name: 0}) == INVALID, name
    assert f(A=M + 8) == INVALID and f(B=3 * M + 8) == INVALID and f(C=5 * M + 1) == INVALID and f(dt=1, C=5 * M + 2) == INVALID
    assert f(C=M + 511) == INVALID and f(C=M + 510) == INVALID and f(C=2 * M) == INVALID and f(C=4 * M + 2) == INVALID


def test_bindings_refuse(itl):
    import torch

    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    seed = torch.zeros(1, dtype=torch.int64)
    for call in (lambda: itl.dropout(x, itl.Dropout(0.1, seed)), lambda: itl.quantize_blocks_fp8(x),
                 lambda: itl.quantize_tiles_fp8(x), lambda: itl.residual_norm_blocks_fp8(x, x, x[0])):
        with pytest.raises(ValueError):  # host tensors
            call()
    codes = torch.zeros(4, 128, dtype=torch.uint8)
    with pytest.raises(ValueError):
        itl.matmul_fp8_blocks(codes, torch.zeros(1, 4), codes, torch.zeros(1, 1))
    with pytest.raises(TypeError):
        itl.dropout([1.0], None)


def test_which_norms_take_dropout(itl):
    """Those that the package's documentation names, and no other."""
    norms = ("residual_norm", "residual_norm_fp8", "residual_norm_blocks_fp8", "residual_norm_backward")
    takes = {name for name in norms if "dropout" in inspect.signature(getattr(itl, name)).parameters}
    entry = next(e for e in itl.__doc__.split("\n* ") if "``dropout=``" in e)
    named = set(re.findall(r"``(residual_\w+)", entry.split("``dropout=``")[1]))
    assert named == takes and "norms above" not in entry


@needs_hipcc
@pytest.mark.parametrize("src,kernels", [("matmul_fp8.hip", ["product_"]), ("quantize_blocks.hip", ["quantize_"]),
                                         ("dropout.hip", ["dropout_"])])
def test_kernels_have_no_scratch(tmp_path, src, kernels):
    r = _compile(os.path.join(build.CSRC, src), str(tmp_path),
                 ("-c", "-o", str(tmp_path / "x.o"), "-Rpass-analysis=kernel-resource-usage"))
    seen, current = set(), None
    for line in r.stderr.splitlines():
        m = re.search(r"Function Name: (\S+)", line)
        if m:
            current = m.group(1)
        m = re.search(r"ScratchSize \[bytes/lane\]: (\d+)", line)
        if m and current:
            for k in kernels:
                if k in current:
                    assert int(m.group(1)) == 0, (current, line)
                    seen.add(k)
    assert seen == set(kernels)


@needs_hipcc
@pytest.mark.parametrize("src", ["norm_dropout.hip", "norm_codes.hip"])
def test_norms_with_dropout_and_codes_have_no_scratch(tmp_path, src):
    """The norms' other instances: those of two groups with dropout are at the registers' end."""
    test_kernels_have_no_scratch(tmp_path, src, ["norm_"])


@needs_hipcc
def test_inline_asm_loads_write_lds_only(tmp_path):
    out = str(tmp_path / "k.s")
    _compile(os.path.join(build.CSRC, "matmul_fp8.hip"), str(tmp_path), ("-S", "-o", out))
    in_asm, loads = False, 0
    for line in open(out):
        if ";;#ASMSTART" in line or ";;#ASMEND" in line:
            in_asm = ";;#ASMSTART" in line
            continue
        text = line.split(";")[0]
        if in_asm and (m := ASM_MEM.match(text)):
            assert m.group(2) == "load" and m.group(1) == "buffer" and text.rstrip().endswith(" lds"), line.strip()
            loads += 1
    assert loads > 0
