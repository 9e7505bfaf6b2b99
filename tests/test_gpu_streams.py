"""Calls with `stream=`: what a call allocates belongs to the stream that its kernels run on, and stays
safe where the caller uses it. (A tile list that went back to the current stream's pool while the
kernels still read it would be overwritten by that stream's next tensors.)"""
import inspect

import pytest
import torch

import moe_nvfp4_gemm_gb300 as m

FP8 = torch.float8_e4m3fn


def calls_with_a_stream():
    return [n for n in m.EXPORTS if hasattr(m, n) and "stream" in inspect.signature(getattr(m, n)).parameters]


def test_every_call_with_a_stream_runs_on_it(monkeypatch):
    names = calls_with_a_stream()
    assert len(names) == 21
    monkeypatch.setattr(m, "_on_stream", lambda stream, fn, args: (stream, fn, args))
    for n in names:
        fn = getattr(m, n)
        given = {p: i for i, p in enumerate(inspect.signature(fn).parameters)}
        assert fn(**given) == (given["stream"], fn, given)  # before anything is looked at or allocated


class FakeTensor:
    def __init__(self, log):
        self.log = log

    def record_stream(self, s):
        self.log.append(("recorded", s))


def test_allocation_rule(monkeypatch):
    """On fakes: the call runs with its stream current, its outputs are recorded for the caller's stream."""
    log, current = [], ["main"]

    class use:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            self.before, current[0] = current[0], self.s

        def __exit__(self, *a):
            current[0] = self.before

    monkeypatch.setattr(m.torch.cuda, "stream", use)
    monkeypatch.setattr(m.torch.cuda, "current_stream", lambda: current[0])

    def call(x, y=None, stream=None):
        assert stream is None
        log.append(("allocated on", current[0], x, y))
        return FakeTensor(log), None

    def run(stream):
        log.clear()
        m._on_stream(stream, call, {"x": 1, "y": 2, "stream": stream})
        return list(log)

    assert run("main") == [("allocated on", "main", 1, 2)]
    assert run("side") == [("allocated on", "side", 1, 2), ("recorded", "main")]
    assert current == ["main"]


def owner(t):
    """The stream that an allocation of torch's caching allocator belongs to."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not an allocation of torch's")


def fp8_experts(E, N, K, counts):
    g = torch.Generator(device="cuda").manual_seed(1)
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[1:] = torch.tensor(counts).cumsum(0)
    rows = int(off[-1])
    a, sa = m.nvfp4_fp8_quantize(torch.randn(rows, K, generator=g, device="cuda").bfloat16())
    b = torch.empty(E, N, K, dtype=FP8, device="cuda")
    sb = torch.empty(E, (N + 127) // 128, (K + 127) // 128, device="cuda")
    for e in range(E):
        b[e], sb[e] = m.nvfp4_fp8_quantize(torch.randn(N, K, generator=g, device="cuda").bfloat16(), 128)
    return a, sa, b, sb, off.cuda(), E, rows, N, K


@pytest.mark.gpu
def test_allocations_belong_to_the_stream(monkeypatch):
    args = fp8_experts(4, 256, 512, [3, 0, 70, 40])
    x = torch.randn(64, 512, device="cuda").bfloat16()
    logits = torch.randn(300, 16, device="cuda")
    gs = m.nvfp4_amax(x)[1]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    seen, empty = [], torch.empty

    def spy(*a, **k):
        seen.append(torch.cuda.current_stream() == s)
        return empty(*a, **k)

    monkeypatch.setattr(torch, "empty", spy)
    r = m.nvfp4_moe_route(logits, 2, stream=s)
    outs = [r.topk_w, r._buf, m.nvfp4_fp8_grouped_gemm(*args, stream=s), m.nvfp4_amax(x, stream=s)[0],
            *m.nvfp4_quantize(x, gs, stream=s), *m.nvfp4_fp8_quantize(x, transposed=True, stream=s),
            m.nvfp4_moe_route_backward(logits, r, d_loss=torch.ones(1, device="cuda"), stream=s)]
    s.synchronize()
    assert len(seen) >= 10 and all(seen)
    assert all(owner(t) == s.cuda_stream for t in outs[:3])


@pytest.mark.gpu
def test_results_hold_while_the_current_stream_allocates():
    """Many calls on a side stream, each followed by tensors on the current stream that would take over a
    workspace given back too early and overwrite it."""
    args = fp8_experts(8, 384, 1024, [3, 0, 70, 40, 1, 200, 16, 9])
    g = torch.Generator(device="cuda").manual_seed(2)
    logits = torch.randn(5000, 64, generator=g, device="cuda")
    want = m.nvfp4_fp8_grouped_gemm(*args)
    routed = m.nvfp4_moe_route(logits, 4, renormalize=True)
    ws = m.nvfp4_fp8_grouped_gemm_workspace_bytes(*args[5:])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(30):
        got.append(m.nvfp4_fp8_grouped_gemm(*args, stream=s))
        got.append(m.nvfp4_moe_route(logits, 4, renormalize=True, stream=s))
        junk = [torch.full((ws,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
        del junk
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(got[::2], got[1::2]):
        assert torch.equal(a, want)
        assert all(torch.equal(x, y) for x, y in zip(b, routed))
