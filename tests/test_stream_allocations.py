"""Calls on another stream than the current one: what they allocate belongs to that stream's pool, so that
neither the block's earlier users nor its next ones on the current stream run beside the call."""
import contextlib

import pytest
import torch

from linear_attention_recurrence_kda_gb300 import binding as B


class Side:
    cuda_stream = 0


class Library:
    """In the library's place: every call is refused, nothing is launched (a Grace-based GPU would address the host's
    tensors)."""

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return lambda *a: 256
        if name == "kda_status_string":
            return lambda status: b"KDA_ERR_INVALID_ARG"
        return lambda *a: B.KDA_ERR_INVALID_ARG


@pytest.fixture
def watched(monkeypatch):
    """(where, recorded): the stream of every allocation, and the tensors handed to the current stream."""
    now, where, recorded = ["current"], [], []
    real = torch.empty

    @contextlib.contextmanager
    def on(stream):
        now.append(stream)
        yield
        now.pop()

    def empty(*a, **kw):
        where.append(now[-1])
        return real(*a, **kw)

    monkeypatch.setattr(B, "lib", Library)
    monkeypatch.setattr(B, "_stream", lambda stream=None: None)
    B._decode_workspace_bytes.cache_clear()
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: "current")
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append(s), raising=False)
    yield where, recorded
    B._decode_workspace_bytes.cache_clear()


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def refused(call, *a, **kw):
    with pytest.raises(B.KdaError):
        call(*a, **kw)


def test_attention(watched):
    where, recorded = watched
    side = Side()
    q, k = t(8, 4, 64), t(8, 2, 64)
    cache = B.kda_cache_alloc(3, 16, 2, 64, device="cpu")
    lengths, table = t(8, dtype=torch.int32), t(8, 1, dtype=torch.int32)
    refused(B.kda_attention_prefill, q, k, k, stream=side)
    refused(B.kda_attention_decode, q, cache, table, lengths, stream=side)
    assert where == [side] * 3, where           # two results and a workspace
    assert recorded == ["current"] * 2, recorded  # the results go on to the current stream
    where.clear()
    refused(B.kda_attention_decode, q, cache, table, lengths)
    assert where == ["current"] * 2 and len(recorded) == 2


T, H, D = 8, 2, 64
F32 = torch.float32
QKVZ = lambda: [t(T, H, D) for _ in range(4)] + [t(H, dtype=F32), t(T, H, dtype=F32)]  # noqa: E731
STATE = lambda n=1: t(n, H, D, D, dtype=F32)  # noqa: E731
CALLS = {  # name: (call, results that it allocates, workspaces)
    "forward": (lambda s: B.kda_forward(*QKVZ(), stream=s), 2, 1),
    "forward_static_scratch": (lambda s: B.kda_forward_static_scratch(*QKVZ(), stream=s), 2, 0),
    "backward": (lambda s: B.kda_backward(*QKVZ(), t(T, H, D), stream=s), 7, 1),
    "forward_summary": (lambda s: B.kda_forward_summary(*QKVZ(), stream=s), 2, 1),
    "state_scan": (lambda s: B.kda_state_scan(t(2, 1, H, D, D, dtype=F32), t(2, 1, H, D, D, dtype=F32), stream=s), 1, 0),
    "decode_step": (lambda s: B.kda_decode_step(*QKVZ(), STATE(T), stream=s), 1, 0),
    "decode_replay": (lambda s: B.kda_decode_replay(*QKVZ(), STATE(), stream=s), 2, 0),
    "prologue": (lambda s: B.kda_prologue(*[t(T, H, D)] * 3, *[t(H, D, 4, dtype=F32)] * 3, stream=s), 3, 0),
    "epilogue": (lambda s: B.kda_epilogue(t(T, H, D), t(T, H, D), t(D, dtype=F32), stream=s), 1, 0),
}


@pytest.mark.parametrize("name", CALLS)
def test_every_call(watched, name):
    where, recorded = watched
    call, results, workspaces = CALLS[name]
    side = Side()
    refused(call, side)
    assert where == [side] * (results + workspaces), where
    assert recorded == ["current"] * results, recorded


def test_epilogue_refuses_a_strided_input():
    with pytest.raises(ValueError):
        B.kda_epilogue(t(H, T, D).transpose(0, 1), t(T, H, D), t(D, dtype=F32))


@pytest.mark.gpu
def test_blocks_that_the_current_stream_still_writes():
    """Blocks of the sizes that a call allocates are freed with work on them pending; the call on another stream is right."""
    N, hq, hkv, d, page, cols = 64, 8, 2, 128, 64, 12
    g = torch.Generator(device="cuda").manual_seed(0)
    cache = B.kda_cache_alloc(N * cols, page, hkv, d)
    table = torch.arange(N * cols, dtype=torch.int32, device="cuda").view(N, cols)
    lengths = torch.arange(1, N + 1, dtype=torch.int32, device="cuda") * (cols * page // N)
    k = torch.randn(int(lengths.sum()), 2 * hkv, d, generator=g, device="cuda").bfloat16()
    cu = torch.cat([lengths.new_zeros(1), lengths.cumsum(0, dtype=torch.int32)])
    B.kda_cache_append(k[:, :hkv], k[:, hkv:], cache, table, lengths, cu_seqlens=cu)
    q = torch.randn(N, hq, d, generator=g, device="cuda").bfloat16()
    want = B.kda_attention_decode(q, cache, table, lengths)
    ws = B._decode_workspace_bytes(N, N, hq, hkv, d, B.KDA_BF16, q.device)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        pending = [torch.empty(ws, dtype=torch.uint8, device="cuda"), torch.empty_like(q)]
        torch.cuda._sleep(20_000_000)  # about ten milliseconds, far longer than the call
        for x in pending:
            x.fill_(1)
        del x, pending
        got = B.kda_attention_decode(q, cache, table, lengths, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, want)
