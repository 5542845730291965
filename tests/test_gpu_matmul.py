"""ob_matmul on the GPU against products in 64 bits.

Tolerances: a sum of K products of 16-bit values has exact products in fp32; an fp32 sum of K terms in any order, whatever
its tree, is off by at most (K - 1) u sum|a b| with u = 2^-24 (a fused multiply-add rounds once per term), the matrix cores may
truncate where the bound rounds, which doubles u.  alpha and beta * C add three roundings of the result's parts, and the
result is rounded to its type: half a step, eps / 2 of it.
"""
import pytest
import torch

import adam_ob_compress_amd as ob

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = 2.0 ** -24


def operand(gen, batch, rows, cols, dtype, transposed=False, pad=0):
    """[batch, rows, cols] (or [rows, cols]) as a view with `pad` elements between lines."""
    x, y = (cols, rows) if transposed else (rows, cols)
    t = torch.randn(batch or 1, x, y + pad, generator=gen, device="cuda").to(dtype)[:, :, :y]
    t = t.transpose(1, 2) if transposed else t
    return t if batch else t[0]


def check(a, b, out, alpha, beta, c, symmetric=False):
    """Run the product and compare every element with the one in 64 bits."""
    want = alpha * (a.double() @ b.double())
    size = abs(alpha) * (a.double().abs() @ b.double().abs())
    if c is not None and beta:
        want, size = want + beta * c.double(), size + abs(beta) * c.double().abs()
    ob.ob_matmul(a, b, out, alpha=alpha, beta=beta, c=c, symmetric=symmetric)
    K = a.shape[-1]
    tol = (2 * K + 4) * U * size + torch.finfo(out.dtype).eps / 2 * want.abs() + torch.finfo(out.dtype).tiny
    far = (out.double() - want).abs() - tol
    assert not out.isnan().any()
    assert float(far.max()) <= 0, (float(far.max()), tuple(a.shape), tuple(b.shape))


SHAPES = [(3, 2, 1000), (5, 6, 333), (1, 1, 1), (1, 5, 3), (16, 16, 32), (33, 17, 65), (64, 64, 64), (65, 127, 129), (96, 200, 136), (128, 256, 320),
          (129, 300, 77), (1, 512, 4096), (520, 8, 1000), (264, 520, 72)]


@pytest.mark.parametrize("layout", ["nn", "nt", "tn", "tt"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_layouts_and_odd_sizes(m, n, k, layout):
    gen = torch.Generator("cuda").manual_seed(m * 1000003 + n * 1009 + k)
    a = operand(gen, 0, m, k, torch.bfloat16, layout[0] == "t")
    b = operand(gen, 0, k, n, torch.bfloat16, layout[1] == "t")
    c = torch.randn(m, n, generator=gen, device="cuda")
    check(a, b, torch.empty(m, n, device="cuda"), 0.75, -1.5, c)


@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_types(dtype, out):
    gen = torch.Generator("cuda").manual_seed(3)
    a, b = operand(gen, 0, 200, 104, DT[dtype]), operand(gen, 0, 104, 136, DT[dtype])
    c = torch.randn(200, 136, generator=gen, device="cuda").to(DT[out])
    check(a, b, torch.empty_like(c), 0.3, 1.0, c)
    check(a, b, torch.empty_like(c), -2.0, 0.0, None)
    check(a, b, torch.empty_like(c), 1.0, 0.0, torch.full_like(c, float("nan")))   # not read with beta = 0


@pytest.mark.parametrize("layout", ["nn", "nt", "tn", "tt"])
@pytest.mark.parametrize("pad", [0, 3, 8])
def test_batches_and_strides(pad, layout):
    gen = torch.Generator("cuda").manual_seed(pad)
    a = operand(gen, 5, 72, 88, torch.float16, layout[0] == "t", pad)
    b = operand(gen, 5, 88, 56, torch.float16, layout[1] == "t", pad)
    flat = torch.zeros(5, 72, 56 + 5, device="cuda")
    out = flat[:, :, :56]
    c = torch.randn(5, 72, 64, generator=gen, device="cuda")[:, :, 4:60]
    check(a, b, out, 1.0, 0.5, c)
    assert not flat[:, :, 56:].any()   # what lies between the rows is left alone


@pytest.mark.parametrize("layout", ["nn", "nt", "tn", "tt"])
@pytest.mark.parametrize("m,n,k", [(2048, 1792, 192), (1800, 2056, 520), (3000, 1000, 64)])
def test_large_tiles(m, n, k, layout):
    """Sizes whose tiles of 256 and 128 fill the card, with parts of a tile at each end."""
    gen = torch.Generator("cuda").manual_seed(k)
    for batch in (0, 6):
        a = operand(gen, batch, m, k, torch.bfloat16, layout[0] == "t")
        b = operand(gen, batch, k, n, torch.bfloat16, layout[1] == "t")
        check(a, b, torch.empty(*a.shape[:-1], n, device="cuda", dtype=torch.bfloat16), 1.0, 0.0, None)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["nt", "tn"])
@pytest.mark.parametrize("m,k", [(1, 9), (40, 64), (130, 136), (257, 77), (700, 1024), (5000, 128)])
def test_symmetric(m, k, layout, out):
    gen = torch.Generator("cuda").manual_seed(m)
    a = operand(gen, 0, m, k, torch.bfloat16, layout == "tn")
    c = torch.randn(m, m, generator=gen, device="cuda")
    c = (c + c.t()).to(DT[out])
    got = c.clone()
    check(a, a.t(), got, 0.5, 0.9, c.clone(), symmetric=True)
    assert torch.equal(got, got.t())
    ob.ob_matmul(a, a.t(), c, alpha=0.5, beta=0.9, c=c, symmetric=True)   # in place: the same bits
    assert torch.equal(got, c)


@pytest.mark.parametrize("layout", ["nn", "nt", "tn", "tt"])
@pytest.mark.parametrize("m,n,k,batch", [(64, 64, 65536, 0), (40, 24, 40_000, 0), (300, 520, 20_008, 0), (257, 129, 9999, 0),
                                         (512, 512, 8192, 3), (1100, 1030, 4096, 0), (4096, 4224, 1024, 0)])
def test_long_sums_and_rests(m, n, k, batch, layout):
    """Tiles that several work groups share: few tiles, or a rest behind full rounds; with and without a workspace, in place."""
    gen = torch.Generator("cuda").manual_seed(k)
    a = operand(gen, batch, m, k, torch.bfloat16, layout[0] == "t")
    b = operand(gen, batch, k, n, torch.bfloat16, layout[1] == "t")
    c = torch.randn(*a.shape[:-1], n, generator=gen, device="cuda")
    out = torch.empty_like(c)
    check(a, b, out, 0.5, 0.25, c)
    room = torch.full((1 << 28,), 255, dtype=torch.uint8, device="cuda")   # of any content: NaN
    again = c.clone()
    ob.ob_matmul(a, b, again, alpha=0.5, beta=0.25, c=again, workspace=room)
    assert torch.equal(out, again)
    half = torch.empty_like(c, dtype=torch.float16)
    check(a, b, half, 1.0, 0.0, None)
    if m == 512:
        check(a, a.transpose(1, 2), c[:, :, :m].contiguous(), 1.0, 0.0, None, symmetric=True)


def test_shared_tiles_in_a_graph_and_on_a_stream():
    gen = torch.Generator("cuda").manual_seed(6)
    a, b = operand(gen, 0, 100, 30_000, torch.float16), operand(gen, 0, 30_000, 72, torch.float16)
    want, out = torch.empty(100, 72, device="cuda"), torch.empty(100, 72, device="cuda")
    side = torch.cuda.Stream()
    ob.ob_matmul(a, b, want)
    side.wait_stream(torch.cuda.current_stream())
    ob.ob_matmul(a, b, out, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(want, out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ob.ob_matmul(a, b, out)
    for k in range(3):
        a.mul_(0.5)
        g.replay()
        ob.ob_matmul(a, b, want)
        junk = torch.full((1 << 24,), 2.0 ** 100, device="cuda")   # what the allocator hands out between replays
        torch.cuda.synchronize()
        assert torch.equal(want, out) and bool((junk == 2.0 ** 100).all()), k


def test_in_place_and_zero_extents():
    gen = torch.Generator("cuda").manual_seed(1)
    a, b = operand(gen, 0, 130, 70, torch.float16), operand(gen, 0, 70, 300, torch.float16)
    c = torch.randn(130, 300, generator=gen, device="cuda")
    want = torch.empty_like(c)
    ob.ob_matmul(a, b, want, beta=2.0, c=c)
    ob.ob_matmul(a, b, c, beta=2.0, c=c)
    assert torch.equal(c, want)
    # no k: the residual alone; no rows, no columns, no matrices: nothing
    ob.ob_matmul(a[:, :0], b[:0], c, beta=0.5, c=want)
    assert torch.equal(c, want * 0.5)
    ob.ob_matmul(a[:, :0], b[:0], c)
    assert not c.any()
    ob.ob_matmul(a[:0], b, c[:0])
    ob.ob_matmul(a, b[:, :0], c[:, :0])
    ob.ob_matmul(a.expand(0, 130, 70), b.expand(0, 70, 300), c.expand(0, 130, 300))


def test_repeated_operands_and_infinities():
    gen = torch.Generator("cuda").manual_seed(2)
    a, b = operand(gen, 3, 40, 24, torch.bfloat16), operand(gen, 0, 24, 48, torch.bfloat16).expand(3, 24, 48)
    check(a, b, torch.empty(3, 40, 48, device="cuda"), 1.0, 0.0, None)
    column = operand(gen, 0, 40, 1, torch.bfloat16).expand(40, 200)   # one column for every k
    check(column, operand(gen, 0, 200, 48, torch.bfloat16), torch.empty(40, 48, device="cuda"), 1.0, 0.0, None)
    row = operand(gen, 0, 1, 24, torch.bfloat16).expand(40, 24)
    check(row, b[0], torch.empty(40, 48, device="cuda"), 1.0, 0.0, None)
    # an infinity and a NaN stay in their rows and columns; what lies beyond an operand never enters
    wide = torch.full((40, 100), float("nan"), device="cuda", dtype=torch.bfloat16)
    wide[:, :72] = 1.0
    wide[7, 3] = float("inf")
    wide[9, 5] = float("nan")
    for cut in (72, 69):
        for view in (wide[:, :cut], wide.t().contiguous().t()[:, :cut]):
            out = torch.empty(40, 40, device="cuda")
            ob.ob_matmul(view, torch.ones(cut, 40, device="cuda", dtype=torch.bfloat16), out)
            assert out[7].isinf().all() and out[9].isnan().all()
            rest = torch.cat([out[:7], out[8:9], out[10:]])
            assert torch.equal(rest, torch.full_like(rest, float(cut)))


def test_graph_streams_and_equal_bits():
    gen = torch.Generator("cuda").manual_seed(4)
    a, b = operand(gen, 0, 300, 520, torch.bfloat16), operand(gen, 0, 520, 264, torch.bfloat16, True)
    want, out = torch.empty(300, 264, device="cuda"), torch.empty(300, 264, device="cuda")
    ob.ob_matmul(a, b, want, beta=0.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ob.ob_matmul(a, b, out, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ob.ob_matmul(a, b, out)
    for k in range(3):
        a.mul_(0.5)
        g.replay()
        ob.ob_matmul(a, b, want)
        torch.cuda.synchronize()
        assert torch.equal(out, want), k


def test_offsets_past_2_31():
    """Rows that start past 2^31 elements of their operand, result and residual."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    ld = (1 << 27) + 8
    big = torch.empty(17 * ld + 64, dtype=torch.bfloat16, device="cuda")
    a = big.as_strided((18, 40), (ld, 1))
    a.copy_(torch.randn(18, 40, generator=torch.Generator("cuda").manual_seed(1), device="cuda"))
    b = torch.randn(40, 56, generator=torch.Generator("cuda").manual_seed(2), device="cuda").to(torch.bfloat16)
    out = torch.empty(17 * ld + 64, dtype=torch.bfloat16, device="cuda").as_strided((18, 56), (ld, 1))
    check(a, b, out, 1.0, 0.0, None)
    out.copy_(torch.randn(18, 56, device="cuda"))
    check(a, b, out, 1.0, 1.0, out.clone())
    bt = big.as_strided((40, 18), (1, ld))
    bt.copy_(a.t())
    check(b.t().contiguous(), bt, torch.empty(56, 18, device="cuda"), 1.0, 0.0, None)


def test_refusals():
    a, b = (torch.zeros(8, 8, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    out = torch.zeros(8, 8, device="cuda")
    with pytest.raises(TypeError, match="b must be"):
        ob.ob_matmul(a, b.half(), out)
    with pytest.raises(TypeError, match="a must be"):
        ob.ob_matmul(a.float(), b, out)
    with pytest.raises(TypeError, match="out must be"):
        ob.ob_matmul(a, b, out.double())
    with pytest.raises(ValueError, match="no product"):
        ob.ob_matmul(a[:, :4], b, out)
    with pytest.raises(ValueError, match="dimensions"):
        ob.ob_matmul(a[None], b, out)
    with pytest.raises(ValueError, match="by rows"):
        ob.ob_matmul(a, b, torch.zeros(8, 16, device="cuda")[:, ::2])
    with pytest.raises(TypeError, match="c must be"):
        ob.ob_matmul(a, b, out, beta=1.0, c=out.half())
    with pytest.raises(ValueError, match="shape"):
        ob.ob_matmul(a, b, out, beta=1.0, c=out[:4])
    with pytest.raises(ob.ObError):
        ob.ob_matmul(a, b, out, beta=1.0)
    with pytest.raises(ob.ObError):
        ob.ob_matmul(a, b, out, alpha=float("nan"))
    with pytest.raises(ob.ObError):   # neither stride is one
        ob.ob_matmul(torch.zeros(16, 16, device="cuda", dtype=torch.bfloat16)[::2, ::2], b, out)
    with pytest.raises(ob.ObError):   # rows of the result that overlap
        ob.ob_matmul(a, b, out.view(-1).as_strided((8, 8), (4, 1)))
    with pytest.raises(ob.ObError):
        ob.ob_matmul(a, b[:, :4], out[:, :4], symmetric=True)
    with pytest.raises(ValueError, match="GPU"):
        ob.ob_matmul(a.cpu(), b, out)
    long = torch.zeros(8, 1 << 16, device="cuda", dtype=torch.bfloat16)
    for bad in (torch.zeros(16, device="cuda", dtype=torch.uint8), torch.zeros(1 << 26, device="cuda"), torch.zeros(1 << 26, dtype=torch.uint8)):
        with pytest.raises(ValueError, match="workspace"):
            ob.ob_matmul(long, long.t(), out, workspace=bad)
    assert not out.any()
