"""TensorList: the norm of many tensors and clipping by it, against 64 bits.

Tolerance of the norm: a 16-bit chunk's fp32 sum goes through at most 16
additions of a chain and 11 of trees, each rounding a sum of non-negative
numbers, so it is off by at most 27 * 2^-24 of itself; the square root halves
that, the result rounds once: REL = 8.7e-7.  (An fp32 chunk's chains are 32
long, which bounds it by 42 * 2^-24; the tolerance for it is the same, tighter
one: roundings of both signs do not reach either.)  A clipped number: that, four
roundings of the factor and the product, and the rounding to its type."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DTYPES = [torch.float32, torch.float16, torch.bfloat16]
REL = 8.7e-7
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}


@pytest.fixture(scope="module")
def sq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import parity_binade_chunked_gb300 as sq
    return sq


def make(shapes, dtype, seed, scale=0.1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(s, device="cuda", generator=g) * scale).to(dtype) for s in shapes]


def norm_64(tensors):
    return math.sqrt(math.fsum(float(t.double().square().sum()) for t in tensors))


def check_clip(before, after, norm, max_norm, scale):
    f = scale * min(1.0, max_norm / (norm + 1e-6))
    for b, t in zip(before, after):
        want = b.double() * f
        tol = (REL + 5 * 2.0 ** -24 + HALF[t.dtype]) * want.abs() + TINY[t.dtype]
        assert (t.double() - want).abs().le(tol).all()


SHAPES = [(1,), (7,), (0,), (3, 5, 11), (16384,), (16385,), (1000, 129), (2, 0, 3), (50000,), (8,)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("out", [None] + DTYPES)
def test_types(sq, dtype, out):
    g = make(SHAPES, dtype, 1)
    outs = None if out is None else [torch.full(t.shape, 7.0, device="cuda", dtype=out) for t in g]
    before = [t.clone() for t in g]
    want = norm_64(g)
    with sq.TensorList(g, outs) as tl:
        assert tl.norm().item() == pytest.approx(want, rel=REL)
        assert tl.norm(scale=0.25).item() == pytest.approx(want / 4, rel=REL)
        n = tl.clip(0.5, scale=0.5)
        assert n.item() == pytest.approx(want / 2, rel=REL)
        check_clip(before, outs or g, want / 2, 0.5, 0.5)
        if outs:
            assert all(torch.equal(a, b) for a, b in zip(before, g))
            tl.clip(1e9)   # nothing to clip: the numbers as they are
            check_clip(before, outs, want, 1e9, 1.0)


@pytest.mark.parametrize("n", [1, 2, 3, 7, 8, 9, 255, 2048, 2049, 16383, 16384, 16385, 1000003])
@pytest.mark.parametrize("dtype", DTYPES)
def test_one_tensor(sq, dtype, n):
    g = make([(n,)], dtype, n)
    tl = sq.TensorList(g)
    want = norm_64(g)
    assert tl.norm().item() == pytest.approx(want, rel=REL)
    before = [g[0].clone()]
    tl.clip(want / 3)
    check_clip(before, g, want, want / 3, 1.0)


def test_mixed_types_and_misaligned(sq):
    base = torch.randn(40001, device="cuda")
    h = torch.randn(70003, device="cuda").half()
    b = torch.randn(30007, device="cuda").bfloat16()
    g = [base[1:20002], h[3:60000], b[1:], base[20003:], torch.randn(13, 17, device="cuda").t(),
         torch.randn(4, 6, 8, device="cuda").permute(2, 0, 1)]
    outs = [torch.zeros_like(t, dtype=torch.bfloat16) for t in g]
    copies = [t.clone() for t in g]
    want = norm_64(g)
    tl = sq.TensorList(g, outs)
    n = tl.clip(1.0)
    assert n.item() == pytest.approx(want, rel=REL)
    check_clip(g, outs, want, 1.0, 1.0)
    # the bits do not depend on the tensors' alignment
    assert sq.TensorList([c.reshape(-1) if c.dim() == 1 else c for c in copies]).norm().item() == n.item()
    inside = torch.full((90,), 5.0, device="cuda")
    sq.TensorList([inside[3:80]]).clip(1.0)
    assert (inside[:3] == 5).all() and (inside[80:] == 5).all() and (inside[3:80] < 1).all()


def test_bits_are_the_same_every_time(sq):
    shapes = [(1 << 20,), (300001,), (5, 100003)] + [(97,)] * 50
    g = make(shapes, torch.bfloat16, 3)
    tl = sq.TensorList(g)
    first = tl.norm().item()
    for _ in range(20):
        assert tl.norm().item() == first
    assert sq.TensorList([t.clone() for t in g]).norm().item() == first


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_squares_outside_fp32(sq, dtype):
    for scale in (1e30, 1e-30, 3e-38, 1e-42):
        g = make([(20000,), (1000,), (1,)], dtype, 5, scale=scale)
        want = norm_64(g)
        if want > 0:
            got = sq.TensorList(g).norm().item()
            assert abs(got - want) <= REL * want + 2.0 ** -149, scale
    g = make([(20000,)], dtype, 6, scale=1e25) + make([(20000,)], dtype, 7, scale=1e-3)
    assert sq.TensorList(g).norm().item() == pytest.approx(norm_64(g), rel=REL)
    g = [torch.full((1 << 20,), 3e38, device="cuda", dtype=dtype)]
    assert sq.TensorList(g).norm().item() == math.inf


def test_nothing_zeros_and_what_is_no_number(sq):
    assert sq.TensorList([]).norm().item() == 0
    assert sq.TensorList([]).clip(1.0).item() == 0
    z = [torch.zeros(100000, device="cuda"), torch.empty(0, device="cuda")]
    assert sq.TensorList(z).clip(1.0).item() == 0 and not z[0].any()
    for bad, norm in ((math.inf, math.inf), (-math.inf, math.inf), (math.nan, math.nan)):
        g = make([(40000,), (10,)], torch.float16, 7)
        g[0][39999] = bad
        clean = g[1].clone()
        n = sq.TensorList(g).clip(1.0).item()
        assert n == norm or (n != n and norm != norm)
        if norm == math.inf:   # the factor is 0
            assert not g[1].any() and g[0][39999].isnan()
        else:
            assert g[1].isnan().all() and clean.isfinite().all()


def test_not_clipped_in_place_is_untouched(sq):
    g = make(SHAPES, torch.bfloat16, 9)
    before = [t.clone() for t in g]
    tl = sq.TensorList(g)
    tl.clip(1e6)
    assert all(torch.equal(a, b) for a, b in zip(before, g))


def test_many_tensors(sq):
    rng = np.random.RandomState(1)
    g = make([(int(n),) for n in rng.randint(0, 3000, 3000)], torch.float16, 11)
    want = norm_64(g)
    before = [t.clone() for t in g]
    tl = sq.TensorList(g)
    assert tl.clip(2.0).item() == pytest.approx(want, rel=REL)
    check_clip(before, g, want, 2.0, 1.0)


def test_other_stream_and_graph(sq):
    g = make(SHAPES, torch.float32, 13)
    outs = [torch.empty_like(t) for t in g]
    tl = sq.TensorList(g, outs)
    want = tl.clip(0.5).item()
    kept = [o.clone() for o in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    n = tl.clip(0.5, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert n.item() == want and all(torch.equal(a, b) for a, b in zip(outs, kept))
    norm = torch.empty(1, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tl.clip(0.5, out=norm)
    for t in g:
        t.mul_(3.0)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert norm.item() == pytest.approx(3 * want, rel=4 * REL)
    check_clip(g, outs, norm_64(g), 0.5, 1.0)


def test_refusals(sq):
    t = torch.zeros(10, 10, device="cuda")
    for bad in ([t.cpu()], [t.double()], [t[:, :5]], [t.expand(3, 10, 10)], [None]):
        with pytest.raises(TypeError):
            sq.TensorList(bad)
    for outs in ([t.double()], [t[:5]], [t.cpu()], [torch.zeros(2, 10, 10, device="cuda").permute(0, 2, 1)[0]]):
        with pytest.raises(TypeError):
            sq.TensorList([t], outs)
    with pytest.raises(ValueError):
        sq.TensorList([t], [])
    tl = sq.TensorList([t])
    with pytest.raises(TypeError):
        tl.norm(out=torch.zeros(1, device="cuda", dtype=torch.float64))
    tl.close()
    with pytest.raises(sq.SeqsumError):
        tl.norm()
    tl.close()
