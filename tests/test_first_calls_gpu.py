"""Calls whose shared memory lies near the size that needs an opt-in, as the first ones of a process,
and calls of two host threads at once: a launch must not depend on what ran before or beside it.
"""
import os
import subprocess
import sys
import threading

import pytest
import torch

from looped_transformer_cross_gb300 import lla

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from looped_transformer_cross_gb300 import build
    build.build()


def _in_new_process(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout


def fp32_decode(rk, rv, stream=None, B=2, L=40):
    """A closure that makes one fp32 4-bit decode call; its output tensor."""
    dm = lla.dims(1, 1, rk, rv, dtype=lla.LLA_F32)
    g = torch.Generator(device="cuda").manual_seed(rk + rv)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    pool, ws = lla.q4_pool(dm, B, 64), lla.q4_workspace(dm, B, 64)
    lla.q4_store(dm, rnd(B * 64, 1, rk), rnd(B * 64, 1, rv), torch.arange(B * 64, device="cuda"), pool, ws)
    i32 = dict(dtype=torch.int32, device="cuda")
    args = (rnd(B, 1, 128), pool, torch.arange(B, **i32)[:, None].contiguous(), torch.full((B,), L, **i32),
            torch.full((B,), L - 1, **i32), rnd(1, 1, 128, rk), rnd(1, 1, 128, rv), rnd(1, 128), rnd(1, 128))
    cos, sin = lla.rope_table_scaled(lla.dims(1, 1, 16, 16), 128)
    out = torch.empty(B, 1, 128, device="cuda")
    torch.cuda.synchronize()

    def call():
        lla.decode_attn_q4(dm, 0, *args, cos, sin, out, None, ws, stream)
    return call, out


def test_fp32_decode_of_any_rank_first():
    """Ranks around the size at which shared memory has to be asked for, smallest first."""
    code = """
import sys
sys.path.insert(0, "tests")
import torch
from test_first_calls_gpu import fp32_decode
ranks = sorted(((k, v) for k in range(16, 129, 16) for v in range(16, 257, 16) if k * 512 + 128 * v < 60000), key=lambda r: 512 * r[0] + 64 * r[1])
for rk, rv in ranks:
    call, out = fp32_decode(rk, rv)
    call()
    assert out.isfinite().all()
print(len(ranks))
"""
    assert int(_in_new_process(code)) > 40


@pytest.mark.parametrize("rk,rv", [(64, 128), (48, 256)])
def test_fp32_decode_first_call(rk, rv):
    _in_new_process("""
import sys
sys.path.insert(0, "tests")
from test_first_calls_gpu import fp32_decode
call, out = fp32_decode(%d, %d)
call()
assert out.isfinite().all()
""" % (rk, rv))


def test_page_plan_of_any_number_of_requests_first():
    """Request counts around the size at which shared memory has to be asked for, in rising order."""
    _in_new_process("""
import torch
from looped_transformer_cross_gb300 import lla
for B in (3000, 3050, 3055, 3056, 3060, 3065, 3071, 3080, 4000, 8192):
    i32 = dict(dtype=torch.int32, device="cuda")
    plan = lla.PagePlan(B, B)
    table = torch.full((B, 1), -1, **i32)
    plan(4, B, torch.zeros(B, **i32), torch.ones(B, **i32), torch.arange(B, **i32), table)
    assert torch.equal(plan.slots, 4 * torch.arange(B, device="cuda")), B
    assert torch.equal(table[:, 0], torch.arange(B, **i32)) and plan.counts.tolist() == [B, B]
    assert lla.device_status(plan.workspace) == lla.LLA_OK
""")


def test_two_threads_with_different_ranks(monkeypatch):
    """Three host threads call the same kernel with different shared memory at once (the C call itself,
    which runs without Python's lock)."""
    calls, kept, fails = [], [], []
    ranks = ((256, 256), (112, 64), (256, 16))
    for rk, rv in ranks:
        stream = torch.cuda.Stream()
        call, out = fp32_decode(rk, rv, stream)
        kept.append(call)                                      # (and with it the tensors that the addresses belong to)
        call()
        torch.cuda.synchronize()
        with monkeypatch.context() as m:
            m.setattr(lla, "_run", lambda what, f, index, s, *args: calls.append((f, args, s, out, out.clone())))
            call()
    torch.cuda.synchronize()

    def work(f, args, stream, out, want):
        status = {f(*args, stream.cuda_stream) for _ in range(20000)}
        stream.synchronize()
        if status != {lla.LLA_OK} or not torch.equal(out, want):
            fails.append(status)

    threads = [threading.Thread(target=work, args=c) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not fails, fails
