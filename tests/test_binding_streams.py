"""A call of the binding that is given a stream and no workspace works in memory of that stream.

The caching allocator hands memory out again in the order of the stream it was allocated on.  A workspace of the
current stream, dropped when the call returns, could be another tensor's while kernels on the given stream still use it.
"""

import contextlib

import pytest
import torch


S, HQ, HKV, D, B, NB, MB = 2, 4, 2, 64, 16, 12, 5
CTX = [70, 33]


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_382_b200 import build

    build.build()
    from paged_kv_cache_382_b200 import pa as binding

    return binding


def arguments(device):
    g = torch.Generator().manual_seed(3)
    t = lambda *shape: torch.randn(shape, generator=g).to(torch.bfloat16).to(device)  # noqa: E731
    i = lambda x, dt=torch.int32: torch.tensor(x, dtype=dt, device=device)  # noqa: E731
    tables = torch.randperm(NB, generator=g)[: S * MB].reshape(S, MB).to(torch.int32).to(device)
    return dict(q=t(S, HQ, D), k=t(NB, HKV, B, D), v=t(NB, HKV, B, D), new=t(S, HKV, D), tables=tables, lens=i(CTX),
                slots=i([-1, -1], torch.int64), start=i([0, 1, 2]), mask=i([[1], [1]], torch.int64))


def calls(pa, a, device):
    # not filled: that would be work of the current stream
    out = lambda: torch.empty((S, HQ, D), dtype=torch.float32, device=device)  # noqa: E731
    totals = torch.empty(S, HKV, MB * B, device=device)   # outlives the calls, as outputs have to
    base = (a["k"], a["v"], a["tables"], a["lens"])
    return {
        "decode": lambda **kw: pa.decode(out(), a["q"], *base, 0.2, **kw),
        "decode_step": lambda **kw: pa.decode_step(out(), a["q"], a["new"], a["new"], a["k"], a["v"], a["slots"], a["tables"], a["lens"],
                                                   0.2, **kw),
        "prefill": lambda **kw: pa.prefill(out(), a["q"], *base, a["start"], 0.2, **kw),
        "tree_decode": lambda **kw: pa.tree_decode(out(), a["q"], *base, a["start"], a["mask"], 0.2, **kw),
        "decode_weights": lambda **kw: pa.decode_weights(out(), totals, a["q"], *base, 0.2, **kw),
    }


NAMES = ["decode", "decode_step", "prefill", "tree_decode", "decode_weights"]


@pytest.mark.parametrize("name", NAMES)
def test_workspace_is_allocated_under_the_given_stream(pa, name, monkeypatch):
    """On the CPU, with a library that launches nothing."""
    under, seen, given = [None], [], object()

    @contextlib.contextmanager
    def on(stream):
        under[0] = stream
        yield
        under[0] = None

    class Library:
        def __getattr__(self, entry):
            return lambda *args: 4096 if entry.endswith("bytes") else 0

    empty = torch.empty

    def recorded(*args, **kw):
        if kw.get("dtype") == torch.uint8:
            seen.append(under[0])
        return empty(*args, **kw)

    call = calls(pa, arguments("cpu"), "cpu")[name]
    monkeypatch.setattr(pa, "lib", Library())
    monkeypatch.setattr(pa, "_dev", lambda t, name, dtype=None: t.data_ptr())
    monkeypatch.setattr(pa, "_stream_handle", lambda stream: 0)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", recorded)
    call(stream=given)
    assert seen == [given]
    call()
    assert seen == [given, None]


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_memory_of_the_current_stream_is_not_the_calls(pa, name):
    """A call queued behind other work of a side stream; meanwhile the current stream allocates and fills memory."""
    a = arguments("cuda")
    call = calls(pa, a, "cuda")[name]
    expected = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)        # 10 ms
        got = call(stream=side)
        filled = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (1 << 14, 1 << 18, 1 << 20, 1 << 22, 1 << 24, 1 << 25)]
        torch.cuda.synchronize()
        assert all(bool((f == 255).all()) for f in filled)
        assert torch.equal(got, expected)
