"""lla_page_plan against the plan written out request by request."""
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


def _i32(x):
    return torch.as_tensor(np.asarray(x, np.int32)).cuda()


def _both(P, mp, num, ctx, new, free, table, n_tok, head=None):
    B = len(ctx)
    plan = lla.PagePlan(B, n_tok)
    for t in (plan.seq_lens, plan.granted, plan.tok_start, plan.seq_idx, plan.pos, plan.slots, plan.counts):
        t.fill_(-77)
    bt = _i32(table).reshape(B, mp).clone()
    plan(P, num, _i32(ctx), _i32(new), _i32(free), bt, None if head is None else _i32([head]))
    st = lla.device_status(plan.workspace)
    want = q4.page_plan(P, mp, num, ctx, new, free, 0 if head is None else head, np.asarray(table), n_tok)
    for name in ("seq_lens", "tok_start", "granted", "seq_idx", "pos", "slots", "counts"):
        np.testing.assert_array_equal(getattr(plan, name).cpu().numpy(), np.asarray(want[name]), err_msg=name)
    np.testing.assert_array_equal(bt.cpu().numpy(), want["table"])
    return st, want


def _case(seed, B, P, ctx_hi, new_hi, share=1.0, slack=0, n_slack=0):
    g = np.random.default_rng(seed)
    ctx, new = g.integers(0, ctx_hi + 1, B), g.integers(0, new_hi + 1, B)
    mp = (ctx_hi + new_hi) // P + 1
    held = -(-ctx // P)
    need = int((-(-(ctx + new) // P) - held).sum())
    n_free = int(need * share) + slack
    num = int(held.sum()) + max(n_free, 1)
    perm = g.permutation(num)
    table = np.full((B, mp), -1)
    k = 0
    for b in range(B):
        table[b, :held[b]] = perm[k:k + held[b]]
        k += held[b]
    return P, mp, num, ctx, new, perm[k:k + n_free], table, int(new.sum()) + n_slack


@pytest.mark.parametrize("B,P,ctx_hi,new_hi", [(1, 1, 0, 1), (1, 16, 100, 1), (3, 24, 50, 60), (511, 16, 300, 1),
                                               (513, 1, 5, 3), (700, 64, 900, 40), (64, 16, 0, 2000), (8192, 8, 20, 2)])
@pytest.mark.parametrize("share", [1.0, 0.6])
def test_plan(B, P, ctx_hi, new_hi, share):
    st, want = _both(*_case(B + P, B, P, ctx_hi, new_hi, share, slack=2 if share == 1.0 else 0, n_slack=5))
    assert st == lla.LLA_OK
    if share == 1.0:
        assert all(want["granted"])


def test_plan_nothing_to_do():
    e = np.zeros(0, np.int32)
    assert _both(16, 4, 8, e, e, e, np.zeros((0, 4)), 3)[0] == lla.LLA_OK              # no request
    assert _both(16, 4, 8, [3, 0], [0, 0], e, np.ones((2, 4)), 0)[0] == lla.LLA_OK     # no token, no free page
    st, w = _both(16, 4, 8, [16, 15], [1, 1], e, np.ones((2, 4)), 2)                   # no free page
    assert st == lla.LLA_OK and w["granted"] == [0, 1]


def test_plan_refuses_requests():
    """A request beyond its table row, or beyond the token maps, is left out; later ones are not."""
    st, w = _both(4, 2, 9, [6, 8, 1, 0], [3, 0, 2, 4], [0, 1, 2], np.full((4, 2), 8), 20)
    assert st == lla.LLA_OK and w["granted"] == [0, 1, 1, 1]
    st, w = _both(4, 4, 9, [0, 0, 0], [3, 9, 1], [0, 1, 2, 3, 4], np.full((3, 4), 8), 7)
    assert st == lla.LLA_OK and w["granted"] == [1, 0, 0]
    # the largest lengths: sums past 32 bits saturate the starts and grant nothing
    big = 2**31 - 1
    st, w = _both(4, 4, 9, [0, big, big], [big, big, 1], [0, 1], np.full((3, 4), 8), 7)
    assert st == lla.LLA_OK and w["granted"] == [0, 0, 0]


def test_plan_reports_bad_values():
    ok = dict(P=4, mp=2, num=9, free=[0, 1, 2], table=np.full((2, 2), 8), n_tok=6)
    bad = lla.LLA_ERR_DEVICE_ARG
    assert _both(4, 2, 9, [-3, 1], [2, 2], [0, 1, 2], np.full((2, 2), 8), 6)[0] == bad       # negative lengths
    assert _both(4, 2, 9, [1, 1], [-2, 2], [0, 1, 2], np.full((2, 2), 8), 6)[0] == bad
    assert _both(4, 2, 9, [1, 1], [1, 1], [0], np.array([[9, 8], [-1, 8]]), 2)[0] == bad      # held pages outside
    assert _both(4, 2, 9, [0, 4], [1, 1], [0, 9], np.full((2, 2), 8), 2)[0] == bad            # a free page outside
    for head in (-1, 4):
        st, w = _both(4, 2, 9, [0, 1], [1, 1], [0, 1, 2], ok["table"], 2, head)
        assert st == bad and w["granted"] == [0, 1]


def test_plan_steps_on_the_gpu():
    """Three steps chained on the device (lengths and the list's head alternate between two
    plans), eagerly and replayed from one captured graph."""
    B, P, mp, n_free = 37, 4, 8, 120
    g = np.random.default_rng(3)
    ctx, new = g.integers(0, 9, B), g.integers(0, 4, B)
    held = -(-ctx // P)
    num = int(held.sum()) + n_free
    perm = g.permutation(num)
    table = np.full((B, mp), -1)
    k = 0
    for b in range(B):
        table[b, :held[b]] = perm[k:k + held[b]]
        k += held[b]
    free = perm[k:]
    n_tok = int(new.sum())
    d_ctx, d_new, d_free = _i32(ctx), _i32(new), _i32(free)

    def steps(a, b, bt, zero):
        a(P, num, d_ctx, d_new, d_free, bt, zero)
        b(P, num, a.seq_lens, d_new, d_free, bt, a.counts[:1])
        a(P, num, b.seq_lens, d_new, d_free, bt, b.counts[:1])

    want_t, c, head = table, ctx, 0
    for _ in range(3):
        w = q4.page_plan(P, mp, num, c, new, free, head, want_t, n_tok)
        want_t, c, head = w["table"], w["seq_lens"], w["counts"][0]
    for captured in (False, True):
        a, b = lla.PagePlan(B, n_tok), lla.PagePlan(B, n_tok)
        bt, zero = _i32(table), _i32([0])
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                steps(a, b, bt, zero)
            bt.copy_(_i32(table))
            graph.replay()
        else:
            steps(a, b, bt, zero)
        torch.cuda.synchronize()
        np.testing.assert_array_equal(bt.cpu().numpy(), want_t)
        np.testing.assert_array_equal(a.slots.cpu().numpy(), w["slots"])
        np.testing.assert_array_equal(a.seq_lens.cpu().numpy(), w["seq_lens"])
        assert a.counts.tolist() == w["counts"] and lla.device_status(a.workspace) == lla.LLA_OK
