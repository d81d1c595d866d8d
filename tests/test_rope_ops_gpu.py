"""lla_rope_table_scaled and lla_rope_apply against 64-bit statements of the same operators."""
import numpy as np
import pytest
import torch

from looped_transformer_cross_gb300 import lla
from oracle import q4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from looped_transformer_cross_gb300 import build
    build.build()


def _ws():
    return torch.zeros(256, dtype=torch.uint8, device="cuda")


# An fp32 value of sincospi is within 1 ulp (2^-23 at 1) of its argument's; the argument, at most an
# eighth of a turn, carries the half step of its own fp32 rounding (2^-24 relative, pi/4 * 2^-24
# absolute); the fp64 frequency and its 64-bit turn carry 2^-52 relative and pos/2^64 turns.
def _table_tol(last):
    return 2**-23 + 2**-24 + 2 * last * 2**-52 + last * 2 * np.pi * 2**-54


@pytest.mark.parametrize("kind,factor,orig", [("plain", 1.0, 0), ("linear", 4.0, 0), ("base", 8.0, 0),
                                               ("by_parts", 8.0, 4096), ("by_parts", 0.5, 1)])
@pytest.mark.parametrize("d,n,pos0", [(128, 1000, 0), (64, 257, 4095), (2, 33, 0), (6, 1, 7), (256, 70, 1 << 20),
                                      (34, 129, (1 << 31) - 129), (126, 40, 123456)])
def test_table(kind, factor, orig, d, n, pos0):
    if kind == "base" and d < 4:
        pytest.skip("no base scaling of one pair")
    dm = lla.dims(1, 1, 16, 16, d_head=d, rope_base=10000.0)
    c, s = lla.rope_table_scaled(dm, n, lla.rope_scaling(kind, factor, orig), pos0=pos0)
    th = q4.thetas(d, 10000.0, kind, factor, orig)
    ang = (np.arange(n, dtype=np.float64) + pos0)[:, None] * th
    tol = _table_tol(pos0 + n)
    assert c.shape == s.shape == (n, d // 2)
    assert np.abs(c.cpu().numpy() - np.cos(ang)).max() <= tol
    assert np.abs(s.cpu().numpy() - np.sin(ang)).max() <= tol


def test_table_equals_the_host_table():
    dm = lla.dims(4, 2, 96, 160)
    c, s = lla.rope_table(dm, 5000)
    gc, gs = lla.rope_table_scaled(dm, 5000)
    assert (gc.cpu() - c).abs().max() <= 2**-23 and (gs.cpu() - s).abs().max() <= 2**-23


def test_table_leaves_the_rest():
    """Nothing is written past the last row, and zero rows write nothing."""
    dm = lla.dims(1, 1, 16, 16, d_head=64)
    buf = torch.full((2, 40, 32), 9.0, device="cuda")
    lla.rope_table_scaled(dm, 37, cos=buf[0, :37], sin=buf[1, :37])
    assert (buf[:, 37:] == 9.0).all() and (buf[:, :37].abs() <= 1.0).all()
    lla.rope_table_scaled(dm, 0, cos=buf[0, :0], sin=buf[1, :0])


def _tables(d_rope, n=300, seed=0):
    """Any rows serve as a table (scaled ones need not have unit length)."""
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n, d_rope // 2, generator=g).cuda(), torch.randn(n, d_rope // 2, generator=g).cuda()


def _check(y, x, pos, cos, sin, off, style, scale, inv):
    want = q4.rope_apply(x.double().cpu().numpy(), pos.cpu().numpy(), cos.cpu().numpy(), sin.cpu().numpy(), off, style,
                         scale, inv)
    got = y.double().cpu().numpy()
    # each output: two products, a sum and a scale in fp32 (half a step each, on terms of the size
    # |x0 c| + |x1 s|), then half a step of the storage type
    half = cos.shape[1]
    rot = slice(off, off + 2 * half)
    xs = np.abs(x.double().cpu().numpy()[..., rot])
    size = xs.max(-1, keepdims=True) * (np.abs(cos.cpu().numpy()).max() + np.abs(sin.cpu().numpy()).max()) * scale
    step = torch.finfo(y.dtype).eps / 2
    tol = step * np.abs(want[..., rot]) + 4 * 2**-24 * size
    assert (np.abs(got[..., rot] - want[..., rot]) <= tol).all()
    keep = np.ones(x.shape[-1], bool)
    keep[rot] = False
    np.testing.assert_array_equal(got[..., keep], x.double().cpu().numpy()[..., keep])


@pytest.mark.parametrize("style", [0, 1])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,heads,d_x,off,d_rope", [(1, 1, 2, 0, 2), (5, 16, 128, 0, 128), (33, 3, 192, 128, 64),
                                                    (7, 2, 100, 3, 90), (64, 1, 96, 32, 16), (2, 5, 128, 8, 48)])
def test_apply(style, dtype, N, heads, d_x, off, d_rope):
    dm = lla.dims(1, heads, 16, 16, dtype=lla.LLA_BF16 if dtype == "bf16" else lla.LLA_F32, rope_style=style)
    sd = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator().manual_seed(N + d_x)
    x = torch.randn(N, heads, d_x, generator=g).to(sd).cuda()
    pos = torch.randint(0, 300, (N,), generator=g, dtype=torch.int32).cuda()
    cos, sin = _tables(d_rope)
    ws = _ws()
    for inv, scale in ((False, 1.0), (True, 1.0), (False, 1.25)):
        y = lla.rope_apply(dm, x, pos, cos, sin, offset=off, scale=scale, inverse=inv, workspace=ws)
        _check(y, x, pos, cos, sin, off, style, scale, inv)
        z = x.clone()
        assert lla.rope_apply(dm, z, pos, cos, sin, out=z, offset=off, scale=scale, inverse=inv, workspace=ws) is z
        assert torch.equal(z, y)                                    # in place: the same values
    assert lla.device_status(ws) == lla.LLA_OK


@pytest.mark.parametrize("style", [0, 1])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,heads,d_x,off,d_rope", [(3, 71, 64, 0, 32), (2, 530, 16, 0, 16), (9, 2, 2100, 4, 2080),
                                                    (2, 3, 1031, 5, 1020), (1000, 1, 32, 16, 16)])
def test_apply_many_heads_and_wide_rows(style, dtype, N, heads, d_x, off, d_rope):
    """More heads than a block's threads take at once, rows of more than a block's threads; table
    rows that begin on a 16-byte boundary and no wider one."""
    dm = lla.dims(1, heads, 16, 16, dtype=lla.LLA_BF16 if dtype == "bf16" else lla.LLA_F32, rope_style=style)
    sd = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator().manual_seed(N + d_x)
    x = torch.randn(N, heads, d_x, generator=g).to(sd).cuda()
    pos = torch.randint(0, 300, (N,), generator=g, dtype=torch.int32).cuda()
    cos, sin = (torch.cat([t.new_zeros(4), t.flatten()])[4:].view_as(t) for t in _tables(d_rope))
    ws = _ws()
    y = lla.rope_apply(dm, x, pos, cos, sin, offset=off, workspace=ws)
    _check(y, x, pos, cos, sin, off, style, 1.0, False)
    lla.rope_apply(dm, x, pos, cos, sin, out=x, offset=off, workspace=ws)
    assert torch.equal(x, y) and lla.device_status(ws) == lla.LLA_OK


def test_apply_strided_slices():
    """q and k as slices of one fused projection, rotated in place and into each other's buffer."""
    dm = lla.dims(1, 4, 16, 16)
    buf = torch.randn(9, 3 * 4 * 128, device="cuda").bfloat16()
    ref = buf.clone()
    q, k = buf[:, :512].view(9, 4, 128), buf[:, 512:1024].view(9, 4, 128)
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    cos, sin = _tables(128)
    ws = _ws()
    lla.rope_apply(dm, q, pos, cos, sin, out=q, workspace=ws)
    _check(q, ref[:, :512].view(9, 4, 128), pos, cos, sin, 0, 0, 1.0, False)
    assert torch.equal(buf[:, 512:], ref[:, 512:])
    lla.rope_apply(dm, q, pos, cos, sin, out=k, workspace=ws)
    _check(k, q, pos, cos, sin, 0, 0, 1.0, False)
    assert torch.equal(buf[:, 1024:], ref[:, 1024:])
    # head-major output, an odd base address, broadcast heads
    out = torch.empty(4, 9, 128, device="cuda", dtype=torch.bfloat16).transpose(0, 1)
    lla.rope_apply(dm, k, pos, cos, sin, out=out, workspace=ws)
    _check(out, k, pos, cos, sin, 0, 0, 1.0, False)
    odd = torch.randn(9 * 4 * 128 + 1, device="cuda").bfloat16()[1:].view(9, 4, 128)
    _check(lla.rope_apply(dm, odd, pos, cos, sin, workspace=ws), odd, pos, cos, sin, 0, 0, 1.0, False)
    one = torch.randn(9, 1, 128, device="cuda").bfloat16().expand(9, 4, 128)
    _check(lla.rope_apply(dm, one, pos, cos, sin, workspace=ws), one, pos, cos, sin, 0, 0, 1.0, False)


def test_apply_gradient():
    """The inverse rotation is the gradient: against differences of the forward call in fp32, and
    against the adjoint identity <R x, g> = <x, R' g>."""
    dm = lla.dims(1, 2, 16, 16, dtype=lla.LLA_F32, rope_style=1)
    cos, sin = _tables(12)
    ws = _ws()
    pos = torch.tensor([3, 299, 0], dtype=torch.int32, device="cuda")
    x, g = torch.randn(3, 2, 16, device="cuda"), torch.randn(3, 2, 16, device="cuda")
    f = lambda v: lla.rope_apply(dm, v, pos, cos, sin, offset=4, scale=0.75, workspace=ws)
    dx = lla.rope_apply(dm, g, pos, cos, sin, offset=4, scale=0.75, inverse=True, workspace=ws)
    # the untouched part passes through unscaled in both directions
    lhs, rhs = (f(x).double() * g.double()).sum(), (x.double() * dx.double()).sum()
    assert abs(lhs - rhs) <= 1e-5 * (f(x).double().abs() * g.double().abs()).sum()
    for n, h, e in ((0, 0, 0), (0, 1, 5), (1, 0, 10), (2, 1, 15)):
        a, b = x.clone(), x.clone()
        a[n, h, e] += 0.5
        b[n, h, e] -= 0.5
        diff = ((f(a).double() - f(b).double()) * g.double()).sum()
        assert abs(diff - dx[n, h, e].double()) <= 1e-4 * (1 + g.abs().max() * cos.abs().max())


def test_apply_positions_out_of_range():
    """Positions outside the table are clamped and reported; the other tokens are right."""
    dm = lla.dims(1, 2, 16, 16)
    cos, sin = _tables(128, n=10)
    x = torch.randn(4, 2, 128, device="cuda").bfloat16()
    ws = _ws()
    y = lla.rope_apply(dm, x, torch.tensor([-5, 3, 10, 1 << 30], dtype=torch.int32, device="cuda"), cos, sin, workspace=ws)
    assert lla.device_status(ws) == lla.LLA_ERR_DEVICE_ARG
    _check(y, x, torch.tensor([0, 3, 9, 9], dtype=torch.int32), cos, sin, 0, 0, 1.0, False)
    assert lla.device_status(ws) == lla.LLA_OK
    lla.rope_apply(dm, x[:0], torch.zeros(0, dtype=torch.int32, device="cuda"), cos, sin, workspace=ws)


def test_apply_large_and_captured():
    """More than 2^31 elements apart: 64-bit addressing; then a captured call on another stream."""
    dm = lla.dims(1, 1, 16, 16)
    big = torch.empty((1 << 31) + 4096, device="cuda", dtype=torch.bfloat16)
    x = big.as_strided((2, 1, 128), (1 << 31, 128, 1))
    x.copy_(torch.randn(2, 1, 128))
    cos, sin = _tables(128)
    ws = _ws()
    pos = torch.tensor([1, 200], dtype=torch.int32, device="cuda")
    ref = x.clone()
    _check(lla.rope_apply(dm, x, pos, cos, sin, out=x, workspace=ws), ref, pos, cos, sin, 0, 0, 1.0, False)
    del big, x
    x = torch.randn(5, 1, 128, device="cuda").bfloat16()
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    y = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        lla.rope_apply(dm, x, pos, cos, sin, out=y, workspace=ws)
    x.copy_(torch.randn(5, 1, 128))
    pos += 7
    graph.replay()
    torch.cuda.synchronize()
    _check(y, x, pos, cos, sin, 0, 0, 1.0, False)
