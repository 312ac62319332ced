"""The block-scaled E4M3 codes and their product against the definitions in 64
bits: sizes of one, odd, around the tiles' ends and past one tile's steps, zero
lengths, both result types, rows alone and in a batch, odd outputs' alignment,
replayed graphs, other streams.

Tolerances, from the arithmetic. fp32 results: a block's products are exact in
fp32 and their 128 additions lose at most a step (2^-23) of the magnitudes each;
the scales' product and the chain over b blocks half a step each: (256 + b + 3)
2^-24 of the summed magnitudes. bf16 results: the matrix cores add eight products
at a time keeping 13 bits below the largest, seven of them each off by at most
2^-13 of it: 7 2^-13 of the magnitudes; and half a step of the result. That
covers the worst case; on random operands the errors of a row of C are
independent, and the whole is within 2^-8 of its norm by far.
"""

import pytest
import torch

import block_refs as B
import learner_refs as R
from helpers import same_bits, say

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float32]
SIZES = [(1, 1, 128), (1, 16, 256), (1, 1536, 1536), (2, 100, 384), (5, 127, 128), (15, 129, 1024), (16, 300, 8960),
         (17, 65, 512), (31, 1000, 256), (33, 128, 640), (64, 129, 384), (65, 250, 1536), (100, 77, 128), (127, 255, 256),
         (128, 256, 512), (129, 257, 384), (200, 1001, 1536), (256, 256, 128), (257, 513, 256), (300, 200, 8448),
         (777, 1001, 1536), (1024, 1536, 640), (8, 40, 16640), (3, 5000, 256), (16, 9000, 384), (30, 8000, 128),
         (33, 70000, 128), (90, 70000, 256), (4000, 1100, 128), (2100, 4100, 384), (4353, 4097, 640), (16900, 600, 512), (2900, 6100, 2560),
         (5400, 2600, 2560), (4200, 4100, 2560), (300, 3001, 8576), (700, 999, 384)]


@pytest.fixture(scope="module")
def itl():
    import invariant_token_logprobs_lm_amd as itl

    return itl


def _bits(t):
    return t.contiguous().view(torch.uint8)


def _matrix(n, d, seed, scale=1.0):
    """Columns of different sizes, a row and a stretch of zeros, odd rows of large values."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, d, generator=g) * torch.exp(0.7 * torch.randn(d, generator=g)) * scale
    if n > 2:
        x[n // 2] = 0
    x[:, : d // 3 : 5] = 0
    return x


# ------------------------------------------------------------------ the codes

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d", [(1, 1), (1, 128), (1, 7168), (3, 7), (2, 100), (5, 136), (127, 129), (128, 128), (129, 257),
                                 (300, 1001), (260, 2560), (1000, 64), (33, 8960)])
def test_codes(cuda, itl, n, d, dtype):
    x = _matrix(n, d, n + d).to(dtype)
    for make, ref in ((itl.quantize_blocks_fp8, B.blocks), (itl.quantize_tiles_fp8, B.tiles)):
        say("codes", n, d, dtype, make.__name__)
        q, s, qt, ts = make(x.to(cuda), columns=True)
        for got, scale, (want, wscale) in ((q, s, ref(x)), (qt, ts, ref(x.t().contiguous()))):
            assert got.shape == want.shape and scale.shape == wscale.shape
            assert same_bits(scale.cpu(), wscale)
            assert torch.equal(got.cpu(), want)
        alone, sa, none, _ = make(x.to(cuda))
        assert none is None and torch.equal(alone, q) and same_bits(sa, s)
        none, _, alone, sa = make(x.to(cuda), rows=False, columns=True)
        assert none is None and torch.equal(alone, qt) and same_bits(sa, ts)


def test_codes_of_odd_alignment_and_small_values(cuda, itl):
    flat = torch.randn(64 * 137 + 3, device=cuda).bfloat16()
    for at in (1, 2, 3):
        x = flat[at:at + 64 * 136].view(64, 136)
        q, s, qt, ts = itl.quantize_blocks_fp8(x, columns=True)
        want = itl.quantize_blocks_fp8(x.clone(), columns=True)
        assert all(torch.equal(_bits(a), _bits(b)) for a, b in zip((q, s, qt, ts), want))
    tiny = torch.full((2, 128), 1e-40, device=cuda)
    q, s, _, _ = itl.quantize_blocks_fp8(tiny)
    assert bool((s == 2.0 ** -126).all()) and bool(torch.isfinite(B.values(q)).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d", [(2, 128), (3, 100), (130, 264)])
def test_zeros_keep_their_sign(cuda, itl, n, d, dtype):
    """A code's bits are the quotient's, negative zeros among them."""
    x = _matrix(n, d, 5).to(dtype)
    x[:, ::2] = torch.where(torch.arange(d)[::2] % 4 == 0, 0.0, -0.0).to(dtype)
    x[0] = -0.0
    for make, ref in ((itl.quantize_blocks_fp8, B.blocks), (itl.quantize_tiles_fp8, B.tiles)):
        say("zeros", n, d, dtype, make.__name__)
        q, _, qt, _ = make(x.to(cuda), columns=True)
        assert torch.equal(q.cpu(), ref(x)[0]) and torch.equal(qt.cpu(), ref(x.t().contiguous())[0])
        assert torch.equal(make(x.to(cuda))[0], q)


def test_nothing_beyond_the_codes_is_written(cuda, itl):
    n, d = 130, 200
    x = torch.randn(n, d, device=cuda)
    room = {}

    def guarded(shape, dtype):
        k = 1
        for v in shape:
            k *= v
        flat = torch.full((k + 128,), 77, dtype=dtype, device=cuda)
        room[len(room)] = (flat, k)
        return flat[64:64 + k].view(shape)

    for make, tiles in ((itl.quantize_blocks_fp8, False), (itl.quantize_tiles_fp8, True)):
        make(x, columns=True, Xq=guarded((n, 256), torch.uint8), scale=guarded((2, 2) if tiles else (2, n), torch.float32),
             Xtq=guarded((d, 256), torch.uint8), t_scale=guarded((2, 2) if tiles else (2, d), torch.float32))
    for flat, k in room.values():
        assert bool((flat[:64] == 77).all()) and bool((flat[64 + k:] == 77).all())


def test_codes_do_not_depend_on_other_rows(cuda, itl):
    x = torch.randn(300, 1000, device=cuda)
    q, s, _, _ = itl.quantize_blocks_fp8(x, columns=True)
    q1, s1, _, _ = itl.quantize_blocks_fp8(x[200:203].contiguous())
    assert torch.equal(q1, q[200:203]) and same_bits(s1, s[:, 200:203])


# ---------------------------------------------------------------- the product

def _operands(itl, m, n, k, device, seed=0):
    a, sa, _, _ = itl.quantize_blocks_fp8(_matrix(m, k, seed + m).to(device))
    b, sb, _, _ = itl.quantize_tiles_fp8(_matrix(n, k, seed + n + 1, 0.02).to(device))
    return a, sa, b, sb


def _check(got, ops):
    want, mag = B.product(*(t.cpu() for t in ops))
    blocks = ops[1].shape[0]
    off = (R.f64(got) - want).abs()
    chain = (256 + blocks + 3) * R.EPS24
    if got.dtype == torch.float32:
        assert bool((off <= chain * mag).all())
        return
    assert bool((off <= R.half_step(torch.bfloat16) * want.abs() + (chain + 7 * 2.0 ** -13) * mag).all())
    assert float(off.norm()) <= 2.0 ** -8 * float(want.norm())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", SIZES)
def test_product(cuda, itl, m, n, k, dtype):
    say("product", m, n, k, dtype)
    ops = _operands(itl, m, n, k, cuda)
    _check(itl.matmul_fp8_blocks(*ops, out_dtype=dtype), ops)


@pytest.mark.parametrize("m,n,k", [(1, 100, 256), (40, 130, 1024), (300, 300, 640)])
def test_small_whole_numbers_are_exact(cuda, itl, m, n, k):
    """Codes of -2 .. 2 and scales of powers of two: every sum is exact in both types' arithmetic."""
    g = torch.Generator().manual_seed(k)
    a, b = torch.randint(-2, 3, (m, k), generator=g), torch.randint(-2, 3, (n, k), generator=g)
    code = lambda x: x.float().to(torch.float8_e4m3fn).view(torch.uint8).to(cuda)
    sa = 2.0 ** torch.randint(-2, 3, (k // 128, m), generator=g)
    sb = 2.0 ** torch.randint(-2, 3, (-(-n // 128), k // 128), generator=g)
    ops = (code(a), sa.to(cuda), code(b), sb.to(cuda))
    want, _ = B.product(*ops)
    assert torch.equal(R.f64(itl.matmul_fp8_blocks(*ops, out_dtype=torch.float32)), want)
    assert torch.equal(itl.matmul_fp8_blocks(*ops).cpu(), want.to(torch.bfloat16))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,k", [(1001, 1536), (256, 8448), (1536, 384)])
def test_rows_do_not_depend_on_their_batch(cuda, itl, n, k, dtype):
    """One token, a few and many: the same bits, as tiles and kernels change."""
    a, sa, b, sb = _operands(itl, 1300, n, k, cuda)
    whole = itl.matmul_fp8_blocks(a, sa, b, sb, out_dtype=dtype)
    for i, m in ((0, 1), (650, 1), (3, 2), (640, 16), (17, 17), (100, 33), (5, 64), (1200, 100), (128, 129), (1, 300), (700, 600)):
        some = itl.matmul_fp8_blocks(a[i:i + m].contiguous(), sa[:, i:i + m].contiguous(), b, sb, out_dtype=dtype)
        assert torch.equal(_bits(some), _bits(whole[i:i + m])), (i, m)


@pytest.mark.parametrize("k", [384, 512])
def test_rows_of_a_large_product(cuda, itl, k):
    """Rows that large tiles made, several per workgroup, and those of smaller calls: the same bits."""
    m, n = 4300, 4000
    a, sa, b, sb = _operands(itl, m, n, k, cuda)
    whole = itl.matmul_fp8_blocks(a, sa, b, sb)
    for i, some in ((0, 1), (4200, 100), (1000, 700), (255, 33)):
        got = itl.matmul_fp8_blocks(a[i:i + some].contiguous(), sa[:, i:i + some].contiguous(), b, sb)
        assert torch.equal(_bits(got), _bits(whole[i:i + some])), i
    # run to run, beside another stream's work
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        other = itl.matmul_fp8_blocks(a, sa, b, sb)
    again = itl.matmul_fp8_blocks(a, sa, b, sb)
    torch.cuda.synchronize()
    assert torch.equal(_bits(other), _bits(whole)) and torch.equal(_bits(again), _bits(whole))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", [(2560, 6656, 1024), (2550, 6601, 1024), (1500, 5601, 2560), (2049, 8200, 2560), (120, 70000, 2560)])
def test_products_of_more_than_whole_rounds(cuda, itl, m, n, k, dtype):
    """Tiles just past a whole number of rounds, by rows or by columns: some of the rows and
    columns against 64 bits, all of them against smaller calls' bits, nothing beyond written."""
    say("rounds", m, n, k, dtype)
    a, sa, b, sb = _operands(itl, m, n, k, cuda)
    flat = torch.full((m * n + 32,), 7.0, dtype=dtype, device=cuda)
    out = itl.matmul_fp8_blocks(a, sa, b, sb, out_dtype=dtype, out=flat[16:16 + m * n].view(m, n))
    assert bool((flat[:16] == 7).all()) and bool((flat[16 + m * n:] == 7).all())
    rows = torch.unique(torch.tensor([0, 1, m // 3, m // 2, m - 200, m - 130, m - 2, m - 1]).clamp(min=0))
    _check(out[rows.to(cuda)], (a[rows.to(cuda)], sa[:, rows.to(cuda)], b, sb))
    for i in range(0, m, 700):
        some = itl.matmul_fp8_blocks(a[i:i + 700], sa[:, i:i + 700].contiguous(), b, sb, out_dtype=dtype)
        assert torch.equal(_bits(some), _bits(out[i:i + 700])), i
    for j in range(0, n, 1280):
        some = itl.matmul_fp8_blocks(a, sa, b[j:j + 1280], sb[j // 128:j // 128 + 10], out_dtype=dtype)
        assert torch.equal(_bits(some), _bits(out[:, j:j + 1280])), j


def test_columns_do_not_depend_on_the_width(cuda, itl):
    """The first columns of a wider B, down to a few: the same bits."""
    for m in (3, 40, 300):
        a, sa, b, sb = _operands(itl, m, 1300, 512, cuda)
        whole = itl.matmul_fp8_blocks(a, sa, b, sb)
        for n in (1, 17, 128, 200, 700):
            some = itl.matmul_fp8_blocks(a, sa, b[:n].contiguous(), sb[:-(-n // 128)].contiguous())
            assert torch.equal(_bits(some), _bits(whole[:, :n]))


@pytest.mark.parametrize("dtype", DTYPES)
def test_outputs_of_any_alignment_and_nothing_beyond(cuda, itl, dtype):
    for m, n in ((1, 12), (3, 13), (20, 64), (130, 260), (300, 258), (2048, 4090), (2048, 4096), (2050, 4092)):
        ops = _operands(itl, m, n, 384, cuda)
        want = itl.matmul_fp8_blocks(*ops, out_dtype=dtype)
        for at in (8, 9, 10, 12):
            flat = torch.full((m * n + 32,), 7.0, dtype=dtype, device=cuda)
            out = flat[at:at + m * n].view(m, n)
            assert itl.matmul_fp8_blocks(*ops, out_dtype=dtype, out=out) is out
            assert torch.equal(_bits(out), _bits(want))
            assert bool((flat[:at] == 7).all()) and bool((flat[at + m * n:] == 7).all())


def test_lengths_of_zero(cuda, itl):
    f = lambda *s: torch.zeros(*s, device=cuda)
    u = lambda *s: torch.zeros(*s, dtype=torch.uint8, device=cuda)
    out = torch.full((5, 7), 3.0, device=cuda)
    itl.matmul_fp8_blocks(u(5, 0), f(0, 5), u(7, 0), f(1, 0), out_dtype=torch.float32, out=out)
    assert not bool(out.any())
    assert not bool(itl.matmul_fp8_blocks(u(300, 0), f(0, 300), u(257, 0), f(3, 0)).any())
    assert itl.matmul_fp8_blocks(u(0, 128), f(1, 0), u(7, 128), f(1, 1)).shape == (0, 7)
    assert itl.matmul_fp8_blocks(u(5, 128), f(1, 5), u(0, 128), f(0, 1)).shape == (5, 0)
    # no tokens: the weight gradient is zeros
    _, _, dyt, ds = itl.quantize_blocks_fp8(f(0, 100), columns=True)
    _, _, xt, xs = itl.quantize_tiles_fp8(f(0, 200), columns=True)
    assert not bool(itl.matmul_fp8_blocks(dyt, ds, xt, xs, out_dtype=torch.float32).any())


def test_values_that_are_not_finite_stay_in_their_row(cuda, itl):
    a, sa, b, sb = _operands(itl, 20, 130, 256, cuda)
    want = itl.matmul_fp8_blocks(a, sa, b, sb, out_dtype=torch.float32)
    a[3, 7] = 0x7F  # E4M3's NaN
    got = itl.matmul_fp8_blocks(a, sa, b, sb, out_dtype=torch.float32)
    assert bool(torch.isnan(got[3]).all())
    keep = torch.arange(20, device=cuda) != 3
    assert same_bits(got[keep], want[keep])


def test_linear_layer_and_its_gradients(cuda, itl):
    """Y, dX and dW of Y = X W^T from X, W and dY, against the layer in 64 bits:
    each operand's codes are within 2^-4 of a value, rms 2.6 %, the products' errors
    independent, so each result is within 5 % of its norm."""
    n, d, f = 391, 600, 777
    g = torch.Generator().manual_seed(4)
    X, W, dY = torch.randn(n, d, generator=g), 0.02 * torch.randn(f, d, generator=g), torch.randn(n, f, generator=g)
    Xc, Wc, dYc = (t.to(torch.bfloat16).to(cuda) for t in (X, W, dY))
    xq, xs, _, _ = itl.quantize_blocks_fp8(Xc)
    wq, ws, wt, wts = itl.quantize_tiles_fp8(Wc, columns=True)
    dq, ds, dt, dts = itl.quantize_blocks_fp8(dYc, columns=True)
    _, _, xt, xts = itl.quantize_tiles_fp8(Xc, rows=False, columns=True)
    Y = itl.matmul_fp8_blocks(xq, xs, wq, ws)
    dX = itl.matmul_fp8_blocks(dq, ds, wt, wts)
    dW = itl.matmul_fp8_blocks(dt, dts, xt, xts, out_dtype=torch.float32)
    Xd, Wd, dYd = R.f64(Xc), R.f64(Wc), R.f64(dYc)
    for got, want in ((Y, Xd @ Wd.t()), (dX, dYd @ Wd), (dW, dYd.t() @ Xd)):
        assert got.shape == want.shape
        assert float((R.f64(got) - want).norm()) <= 0.05 * float(want.norm())


@pytest.mark.parametrize("m", [1, 40, 300, 33000])
def test_replays_and_other_streams(cuda, itl, m):
    x, w = torch.randn(m, 1000, device=cuda), torch.randn(520, 1000, device=cuda).mul_(0.02)
    wq, ws, _, _ = itl.quantize_tiles_fp8(w)

    def step():
        q, s, _, _ = itl.quantize_blocks_fp8(x)
        return itl.matmul_fp8_blocks(q, s, wq, ws), itl.matmul_fp8_blocks(q, s, wq, ws, out_dtype=torch.float32)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for rep in range(3):
        x.normal_()
        graph.replay()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(_bits(a), _bits(b)) for a, b in zip(out, want)), rep
    torch.cuda.synchronize()
    got = []
    for s in [torch.cuda.Stream() for _ in range(2)]:
        with torch.cuda.stream(s):
            got.append(step())
    torch.cuda.synchronize()
    assert all(torch.equal(_bits(a), _bits(b)) for g in got for a, b in zip(g, want))


def test_refusals(cuda, itl):
    a, sa, b, sb = _operands(itl, 4, 130, 256, cuda)
    for bad in ((a, sa.t().contiguous(), b, sb), (a, sa, b, sb.t().contiguous().t()), (a, sa, b[:, :128].contiguous(), sb),
                (a.float(), sa, b, sb), (a, sa.double(), b, sb), (a.cpu(), sa, b, sb), (a, sa, b, sb[:1])):
        with pytest.raises(ValueError):
            itl.matmul_fp8_blocks(*bad)
    with pytest.raises(ValueError):
        itl.matmul_fp8_blocks(a, sa, b, sb, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        itl.matmul_fp8_blocks(a, sa, b, sb, out=torch.empty(4, 129, dtype=torch.bfloat16, device=cuda))
    with pytest.raises(itl.ItlError):  # not whole blocks
        itl.matmul_fp8_blocks(a[:, :192].contiguous(), sa, b[:, :192].contiguous(), sb)
    x = torch.randn(4, 64, device=cuda)
    with pytest.raises(ValueError):
        itl.quantize_blocks_fp8(x, rows=False)
    with pytest.raises(ValueError):
        itl.quantize_tiles_fp8(x, Xtq=torch.empty(64, 128, dtype=torch.uint8, device=cuda))
    with pytest.raises(ValueError):
        itl.quantize_blocks_fp8(x.t())
