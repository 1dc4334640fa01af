"""Rotary positions on the GPU against the oracle, bit for bit (fp32 results; bf16 ones are these rounded
once), and against fp64 within
    (|a c| + |b s|) (2 x 2^-24 for the rounded cosine and product, 2^-24 of the sum)  <=  (|a| + |b|) 2^-22.
A cosine in fp64 is off by 2^-52 or so and an fp32 rounding border lies as near with probability 2^-27: a few
hundred thousand of them are the same on both sides."""
import numpy as np
import pytest

from oracle import msq_rotary as R

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def msq():
    import block_wise_mixed_amd as m
    m.load_library()
    assert torch.cuda.is_available()
    return m


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def same_bits(a, b):
    a, b = np.ascontiguousarray(a, np.float32), np.ascontiguousarray(b, np.float32)
    return np.array_equal(a.view(np.uint32), b.view(np.uint32))


def make(rng, rows, heads, dim, dtype):
    t = torch.from_numpy(rng.normal(size=(rows, heads, dim)).astype(np.float32)).to(dtype)
    return t.float().numpy(), t.cuda()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rows,heads,dim,part,dtype,out", [
    (1, 1, 16, 16, torch.float32, None), (1, 32, 128, 128, torch.bfloat16, None), (3, 5, 64, 48, torch.float32, torch.bfloat16),
    (77, 8, 128, 64, torch.bfloat16, torch.float32), (130, 3, 256, 256, torch.float32, None),
    (9, 71, 64, 16, torch.bfloat16, None), (5, 2, 1024, 1008, torch.float32, None), (700, 1, 80, 80, torch.bfloat16, None),
    (33, 128, 128, 32, torch.bfloat16, torch.float32)])
def test_bit_exact(msq, rows, heads, dim, part, dtype, out, interleaved):
    print("rotary", rows, heads, dim, part, dtype, out, interleaved, flush=True)
    rng = np.random.default_rng(rows + dim)
    x, xt = make(rng, rows, heads, dim, dtype)
    f = msq.rotary_frequencies(part, base=500000.0, factor=4.0, original=2048)
    at = rng.integers(-5, 200000, size=rows)
    rot = msq.Rotary(f, interleaved, 1.25)
    got = msq.rotary(xt, i32(at), rot, out_dtype=out)
    torch.cuda.synchronize()
    assert got.dtype == (out or dtype) and got.is_contiguous()
    want = R.rotate(x, at, f.cpu().numpy(), interleaved, 1.25)
    full = R.rotate64(x, at, f.cpu().numpy(), interleaved, 1.25)
    lo, hi = R.pairs(part, interleaved)
    size = 1.25 * (np.abs(x[..., lo]) + np.abs(x[..., hi]))
    assert (np.abs(want[..., lo] - full[..., lo]) <= size * 2.0 ** -22).all()
    if got.dtype == torch.float32:
        assert same_bits(got.cpu().numpy(), want)
    else:
        assert torch.equal(got.cpu(), torch.from_numpy(want).to(torch.bfloat16))


def test_far_positions(msq):
    """Up to the ends of int32, frequencies up to 2 radians: fp64 angles."""
    rng = np.random.default_rng(3)
    at = np.concatenate([[2 ** 31 - 1, -2 ** 31, 2 ** 31 - 2, 0], rng.integers(-2 ** 31, 2 ** 31, size=300)])
    x, xt = make(rng, len(at), 2, 64, torch.float32)
    f = torch.linspace(1e-9, 2.0, 32, dtype=torch.float64).cuda()
    got = msq.rotary(xt, i32(at), msq.Rotary(f))
    assert same_bits(got.cpu().numpy(), R.rotate(x, at, f.cpu().numpy()))


def test_special_values(msq):
    """Zeros, infinities and NaN go their way through the formula; other pairs do not see them."""
    x = np.ones((2, 1, 32), np.float32)
    x[0, 0, 0], x[0, 0, 1], x[1, 0, 2] = np.inf, np.nan, -0.0
    f = torch.full((16,), 0.5, dtype=torch.float64).cuda()
    got = msq.rotary(torch.from_numpy(x).cuda(), i32([1, 0]), msq.Rotary(f)).cpu().numpy()
    want = R.rotate(x, [1, 0], np.full(16, 0.5))
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[~np.isnan(want)], want[~np.isnan(want)])
    assert np.isfinite(got[..., 3:16]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strides_in_place_and_out(msq, dtype):
    rng = np.random.default_rng(5)
    f = msq.rotary_frequencies(64)
    rot = msq.Rotary(f)
    x, xt = make(rng, 20, 12, 128, dtype)
    at = rng.integers(0, 5000, size=20)
    want = msq.rotary(xt, i32(at), rot)
    # a slice of a fused product, in place: its neighbours stay
    fused = torch.zeros(20, 20, 128, dtype=dtype, device="cuda")
    fused[:, 3:15] = xt
    y = fused[:, 3:15]
    assert msq.rotary(y, i32(at), rot, out=y) is y
    assert torch.equal(y, want) and not fused[:, :3].any() and not fused[:, 15:].any()
    # head-major, and strides that the kernel does not read
    assert torch.equal(msq.rotary(xt.transpose(0, 1).contiguous().transpose(0, 1), i32(at), rot), want)
    odd = torch.zeros(20, 12, 129, dtype=dtype, device="cuda")[..., 1:]
    odd.copy_(xt)
    assert torch.equal(msq.rotary(odd, i32(at), rot), want)
    with pytest.raises(ValueError):
        msq.rotary(odd, i32(at), rot, out=odd)
    to = torch.full((12, 20, 128), 7.0, dtype=torch.float32, device="cuda").transpose(0, 1)
    assert torch.equal(msq.rotary(xt, i32(at), rot, out=to), msq.rotary(xt, i32(at), rot, out_dtype=torch.float32))
    assert msq.rotary(xt[:0], i32([]), rot).shape == (0, 12, 128)
    for overlapping in (xt[:1].expand(20, 12, 128), xt[:, :1].expand(20, 12, 128), xt.view(-1)[:20 * 128 + 11 * 64]
                        .as_strided((20, 12, 128), (128, 64, 1))):
        with pytest.raises(ValueError):
            msq.rotary(xt, i32(at), rot, out=overlapping)
    wide = torch.zeros(20, 12, 256, dtype=dtype, device="cuda")[..., :128]
    assert torch.equal(msq.rotary(xt, i32(at), rot, out=wide), want)


def test_inverse_is_the_gradient(msq):
    """rotary(g, -p) is the rotation's transpose: <rotary(x, p), g> = <x, rotary(g, -p)>, and central
    differences of the former agree (the rotation is linear, so they are exact but for rounding)."""
    rng = np.random.default_rng(6)
    f = msq.rotary_frequencies(32, base=100.0)
    for interleaved in (False, True):
        rot = msq.Rotary(f, interleaved, 1.5)
        x, xt = make(rng, 6, 3, 64, torch.float32)
        g, gt = make(rng, 6, 3, 64, torch.float32)
        at = i32(rng.integers(0, 1000, size=6))
        grad = msq.rotary(gt, -at, rot)
        full = R.rotate64(g, -at.cpu().numpy(), f.cpu().numpy(), interleaved, 1.5)
        assert np.abs(grad.cpu().numpy() - full).max() <= 1.5 * 2 * np.abs(g).max() * 2.0 ** -22
        loss = lambda t: float((msq.rotary(t, at, rot).double() * gt.double()).sum())
        for _ in range(10):
            d = torch.from_numpy(rng.normal(size=x.shape).astype(np.float32)).cuda()
            num = (loss(xt + d) - loss(xt - d)) / 2
            # each result rounded a few times: 2^-22 of its size, 1152 of them with g of about 1
            assert abs(num - float((grad.double() * d.double()).sum())) <= 1152 * 40 * 2.0 ** -22


def test_stream_and_graph(msq):
    rng = np.random.default_rng(7)
    rot = msq.Rotary(msq.rotary_frequencies(128))
    x, xt = make(rng, 16, 8, 128, torch.bfloat16)
    at = i32(np.arange(16))
    want = msq.rotary(xt, at, rot)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = msq.rotary(xt, at, rot, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = msq.rotary(xt, at, rot)
    for k in range(4):
        xt.copy_(torch.randn_like(xt))
        at += 3
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, msq.rotary(xt, at, rot)), k
