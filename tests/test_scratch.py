"""The scratch that the Python calls keep: threads on one stream, and graphs."""
import threading
import time

import pytest
import torch

import selective_state_space_conv1d_gb300 as m
from selective_state_space_conv1d_gb300 import _binding


# ------------------------------------------------------- on the CPU, with a fake library

class _Fake:
    """A library whose prefill takes a while and notes who was in it with which scratch."""

    def __init__(self):
        self.lock, self.inside, self.met, self.scratch = threading.Lock(), [], False, []

    def mamba_gated_delta_workspace_bytes(self, *a):
        return 4096

    def mamba_gated_delta_prefill(self, *a):
        ws, nbytes = a[-3], a[-2]
        assert nbytes >= 4096
        with self.lock:
            self.met |= ws in self.inside
            self.inside.append(ws)
            self.scratch.append(ws)
        time.sleep(0.02)
        with self.lock:
            self.inside.remove(ws)
        return 0


@pytest.fixture
def fake(monkeypatch):
    lib, empty = _Fake(), torch.empty
    monkeypatch.setattr(_binding, "load", lambda: lib)
    monkeypatch.setattr(_binding, "_ws_cache", {})
    monkeypatch.setattr(_binding, "_capturing", lambda dev, st: False, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: empty(*a, **{k: v for k, v in kw.items() if k != "device"}))
    return lib


def _call(stream, **kw):
    q, v, a, w = torch.zeros(1, 32, 1, 8), torch.zeros(1, 32, 1, 8), torch.zeros(1, 32, 1), torch.zeros(1)
    m.mamba_gated_delta_prefill(torch.zeros_like(v), q, q, v, a, a, w, w, stream=stream, **kw)


def _threads(*calls):
    failed = []

    def run(f):
        try:
            f()
        except BaseException as e:
            failed.append(e)

    ts = [threading.Thread(target=run, args=(f,)) for f in calls]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not failed, failed


def test_threads_on_one_stream_take_turns(fake):
    _threads(*[lambda: [_call(7) for _ in range(4)]] * 3)
    assert len(fake.scratch) == 12 and not fake.met


def test_streams_have_their_own(fake):
    _threads(*[lambda s=s: [_call(s) for _ in range(3)] for s in (7, 8, 9)])
    assert len(set(fake.scratch)) == 3 and not fake.met


def test_a_failed_call_gives_the_scratch_back(fake):
    good = fake.mamba_gated_delta_prefill
    fake.mamba_gated_delta_prefill = lambda *a: -1
    fake.mamba_last_error = lambda: b"no"
    with pytest.raises(m.MambaError):
        _call(7)
    fake.mamba_gated_delta_prefill = good
    _threads(lambda: _call(7))


def test_a_workspace_given_or_declined(fake, monkeypatch):
    got = []
    monkeypatch.setattr(fake, "mamba_gated_delta_prefill", lambda *a: got.append(a[-3:-1]) or 0)
    ws = torch.zeros(8192, dtype=torch.uint8)
    _call(7, workspace=ws)
    _call(7, workspace=False)
    assert got == [(ws.data_ptr(), 8192), (None, 0)] and not _binding._ws_cache


def test_a_captured_call_keeps_none(fake, monkeypatch):
    monkeypatch.setattr(_binding, "_capturing", lambda dev, st: True, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 7, raising=False)
    _call(7)
    assert len(fake.scratch) == 1 and not _binding._ws_cache


# ------------------------------------------------------------------ on the GPU

def _prefills(B, T, H, d):
    """Two calls of different inputs, as (function, their outputs, what they give)."""
    out = []
    for seed in (1, 2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        q, k = (torch.nn.functional.normalize(r(B, T, H, d), dim=-1).bfloat16() for _ in range(2))
        v, a, b = r(B, T, H, d).bfloat16(), r(B, T, H).bfloat16(), r(B, T, H).bfloat16()
        w, bias, s = torch.zeros(H, device="cuda"), torch.full((H,), -4.0, device="cuda"), r(B, H, d, d)
        y, s_out = torch.empty_like(v), torch.empty_like(s)

        def call(x=(y, q, k, v, a, b, w, bias, s, s_out)):
            m.mamba_gated_delta_prefill(*x)

        call()
        torch.cuda.synchronize()
        out.append((call, (y, s_out), (y.clone(), s_out.clone())))
    return out


SIZES = [(1, 2048, 4, 128), (2, 200, 90, 64)]  # in parts; items handed from SM to SM


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,H,d", SIZES)
def test_graphs_of_one_capture_stream_replay_side_by_side(cuda_lib, B, T, H, d):
    calls = _prefills(B, T, H, d)
    graphs = []
    for call, _, _ in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):
        for _, out, _ in calls:
            [t.zero_() for t in out]
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
                g.replay()
        torch.cuda.synchronize()
        for _, out, want in calls:
            assert all(torch.equal(t, w) for t, w in zip(out, want))
    assert m.mamba_device_faults() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,H,d", SIZES)
def test_threads_on_one_stream_do_not_mix(cuda_lib, B, T, H, d):
    calls = _prefills(B, T, H, d)
    for _ in range(3):
        for _, out, _ in calls:
            [t.zero_() for t in out]
        torch.cuda.synchronize()
        _threads(*[lambda call=call: [call() for _ in range(50)] for call, _, _ in calls])  # each on the default stream
        torch.cuda.synchronize()
        for _, out, want in calls:
            assert all(torch.equal(t, w) for t, w in zip(out, want))
    assert m.mamba_device_faults() == 0


@pytest.mark.gpu
def test_a_stream_given_by_its_handle_while_another_is_current(cuda_lib):
    (call, out, want), _ = _prefills(1, 2048, 4, 128)
    x = call.__defaults__[0]
    st = torch.cuda.Stream()
    for t in out:
        t.zero_()
    torch.cuda.synchronize()
    m.mamba_gated_delta_prefill(*x, stream=st.cuda_stream)
    st.synchronize()
    assert all(torch.equal(t, w) for t, w in zip(out, want))
