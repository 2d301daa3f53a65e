"""Where a call on a stream of its own makes its tensors: on that stream. Memory
taken from the current stream's pool may still be read by that stream's kernels,
and a workspace would go back to it while the call's kernels use it. The library
is replaced here; no kernel runs."""
import contextlib

import pytest
import torch

tt = pytest.importorskip("exact_inner_product_b200")


class Stream:
    cuda_stream = 0x55


class Lib:
    """Every entry point answers TT_OK."""

    def __getattr__(self, name):
        if name.startswith("tt_"):
            return lambda *args: tt.TT_OK
        raise AttributeError(name)


@pytest.fixture
def made(monkeypatch):
    """The streams on which torch.empty is called."""
    at, now = [], []

    @contextlib.contextmanager
    def on(stream):
        now.append(stream)
        yield
        now.pop()

    empty, strided = torch.empty, torch.empty_strided
    monkeypatch.setattr(tt, "_lib", Lib())
    monkeypatch.setattr(tt, "_on", on)
    monkeypatch.setattr(tt.torch, "empty", lambda *a, **k: at.append(now[-1] if now else None) or empty(*a, **k))
    monkeypatch.setattr(tt.torch, "empty_strided", lambda *a, **k: at.append(now[-1] if now else None) or strided(*a, **k))
    return at


class FakeIndex:
    handle, n, d = None, 40, 16


def _calls():
    q = torch.ones((3, 16))
    index, stream = FakeIndex(), Stream()
    ids, scores = torch.zeros((2, 3, 5), dtype=torch.int32), torch.zeros((2, 3, 5))
    users, items = torch.ones((3, 64)).bfloat16(), torch.ones((4, 64)).bfloat16()
    return stream, {
        "tt_score_topk": lambda: tt.tt_score_topk(index, q, 5, stream=stream),
        "tt_score_topk_noalloc": lambda: tt.tt_score_topk_noalloc(torch.ones((40, 16)), q, 5, stream=stream),
        "tt_merge_topk": lambda: tt.tt_merge_topk(ids, scores, [0, 20], 5, stream=stream),
        "tt_score_topk_ranges": lambda: tt.tt_score_topk_ranges(index, q, 5, [(0, 20)], stream=stream),
        "tt_score_topk_types": lambda: tt.tt_score_topk_types(index, q, 5, torch.zeros(40, dtype=torch.uint8), [0],
                                                              stream=stream),
        "tt_inbatch_softmax": lambda: tt.tt_inbatch_softmax(users, items, stream=stream, check=False),
    }


@pytest.mark.parametrize("name", list(_calls()[1]))
def test_made_on_the_calls_stream(made, name):
    stream, calls = _calls()
    del made[:]
    calls[name]()
    assert made and all(s is stream for s in made), made
