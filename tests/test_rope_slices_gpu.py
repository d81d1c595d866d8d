"""lla_rope_apply from one slice of a buffer into another: every layout whose rows lie apart is taken,
every other is refused before a launch."""
import random

import pytest
import torch

from looped_transformer_cross_gb300 import lla

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from looped_transformer_cross_gb300 import build
    build.build()


def _quarter_turn(x, out, ws):
    """A rotation by a table of cos = 0, sin = 1: out = (-x1, x0), exactly."""
    n, heads, d = x.shape
    dm = lla.dims(1, heads, 16, 16)
    c = torch.zeros(1, d // 2, device="cuda")
    lla.rope_apply(dm, x, torch.zeros(n, dtype=torch.int32, device="cuda"), c, c + 1, out=out, workspace=ws)


def _turned(x):
    h = x.shape[-1] // 2
    return torch.cat((-x[..., h:], x[..., :h]), -1)


@pytest.mark.parametrize("shape,view", [((9, 4, 2, 128), lambda b, i: b[:, :, i]),                  # per head
                                        ((9, 2, 4, 128), lambda b, i: b[:, i]),                     # per token
                                        ((2, 9, 4, 128), lambda b, i: b[i]),                        # halves
                                        ((4, 9, 2, 128), lambda b, i: b[:, :, i].transpose(0, 1)),  # head-major
                                        ((4, 2, 9, 128), lambda b, i: b[:, i].transpose(0, 1)),
                                        ((5, 3, 2, 6), lambda b, i: b[:, :, i])])
def test_slices_that_lie_apart(shape, view):
    buf, ws = torch.randn(shape, device="cuda").bfloat16(), torch.zeros(256, dtype=torch.uint8, device="cuda")
    for a, b in ((0, 1), (1, 0)):
        x, out = view(buf, a), view(buf, b)
        want = _turned(x.clone())
        rest = x.clone()
        _quarter_turn(x, out, ws)
        assert torch.equal(out, want) and torch.equal(x, rest)
    assert lla.device_status(ws) == lla.LLA_OK


def test_every_layout_of_small_rows():
    """Random strides and distances: refused exactly where a row of x meets a row of out."""
    r, taken, refused = random.Random(4), 0, 0
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    for _ in range(1500):
        n, heads, d = r.randint(1, 4), r.randint(1, 4), r.choice([2, 4, 6])
        s, t = sorted((r.randint(d, 3 * d), r.randint(d, 14 * d)))
        if r.random() < 0.7:
            t = max(t, ((heads if s <= t else n) - 1) * s + d)
        strides = (t, s) if r.random() < 0.5 else (s, t)
        at = lambda base: {base + i * strides[0] + j * strides[1] + e for i in range(n) for j in range(heads)  # noqa: E731
                           for e in range(d)}
        if len(at(0)) < n * heads * d:
            continue                                            # rows of out meet each other: another refusal
        x0, o0 = r.randint(0, 20), r.randint(0, 60)
        if x0 == o0:
            continue
        buf = torch.randn(600, device="cuda").bfloat16()
        x, out = (buf.as_strided((n, heads, d), (*strides, 1), base) for base in (x0, o0))
        want, before = _turned(x.clone()), buf.clone()
        if at(x0) & at(o0):
            with pytest.raises(lla.LLAError):
                _quarter_turn(x, out, ws)
            assert torch.equal(buf, before)
            refused += 1
            continue
        # (interleaved rows that no pair of sorted strides describes are refused as rows of out that meet)
        try:
            _quarter_turn(x, out, ws)
        except lla.LLAError:
            spread = max(strides) < (min(strides) * ((n if strides[0] <= strides[1] else heads) - 1) + d)
            assert spread and n > 1 and heads > 1, (n, heads, d, strides, x0, o0)
            continue
        assert torch.equal(out, want)
        before.as_strided((n, heads, d), (*strides, 1), o0).copy_(want)
        assert torch.equal(buf, before)
        taken += 1
    assert taken > 200 and refused > 200
