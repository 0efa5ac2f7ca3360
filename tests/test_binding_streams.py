"""Tensors that a call makes itself are made on the stream that it runs on (no GPU needed: the library, the allocator and
the streams are stood in for).  A block that was just freed on another stream may still be read or written there."""
import contextlib

import pytest
import torch

from fp4_sparse_attention_gb300 import binding as B


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


HERE, SIDE = Stream(11), Stream(22)


class OnDevice(torch.Tensor):
    """A host tensor that says it is on device 0."""

    def get_device(self):
        return 0


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32).as_subclass(OnDevice)


class Recorder:
    """Current stream, tensors made and on which stream, tensors recorded and for which, streams of the calls."""

    def __init__(self, monkeypatch, workspace):
        self.now, self.made, self.recorded, self.calls = HERE, [], [], []
        empty, empty_like = torch.empty, torch.empty_like

        @contextlib.contextmanager
        def made_on(stream):
            before, self.now = self.now, stream
            yield
            self.now = before

        def note(make):
            def f(*args, **kwargs):
                x = make(*args, **kwargs)
                self.made.append((x, self.now))
                return x
            return f

        class Library:
            def __getattr__(_, name):
                if name.endswith("workspace_bytes"):
                    return lambda *args: workspace
                return lambda *args: self.calls.append(args[-1]) or 0

        monkeypatch.setattr(B, "load_library", Library)
        monkeypatch.setattr(B, "_on_current", lambda device: None)
        monkeypatch.setattr(B, "_raw_stream", None)
        monkeypatch.setattr(B, "_pages_workspace", lambda *args: workspace)
        monkeypatch.setattr(torch, "empty", note(empty))
        monkeypatch.setattr(torch, "empty_like", note(empty_like))
        monkeypatch.setattr(torch.cuda, "stream", made_on)
        monkeypatch.setattr(torch.cuda, "Stream", Stream)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda: self.now)
        monkeypatch.setattr(torch.Tensor, "record_stream", lambda x, stream: self.recorded.append((x, stream)))


def problem():
    cache = torch.zeros((3, 1, 64, 64), dtype=torch.uint8)
    return B.DeviceProblem(format=0, num_heads=2, num_kv_heads=1, page_size=64, q=torch.zeros((2, 2, 64), dtype=torch.uint8),
                           q_scale=torch.zeros((2, 2, 4), dtype=torch.uint8), k=cache, k_scale=torch.zeros((3, 1, 64, 4), dtype=torch.uint8),
                           cu_seqlens_q=i32(2), cu_seqlens_k=i32(2), block_table=i32(1, 2), max_seqlen_q=2, max_seqlen_k=128)


N, T = i32(4), i32(4, 3)
W, SCORES = torch.zeros((2, 2)), torch.zeros((2, 5, 3))
CALLS = {  # name: (call, tensors that are returned, scratch that is not)
    "fork": (lambda s, **kw: B.fp4idx_fork_requests(N, N, N, T, N, 64, stream=s, **kw), 3, 0),
    "release": (lambda s, **kw: B.fp4idx_release_pages(N, N, T, 64, 9, stream=s, **kw), 2, 1),
    "compact": (lambda s, **kw: B.fp4idx_compact_pages(N, T, 64, 9, 3, stream=s, **kw), 4, 1),
    "tables": (lambda s, **kw: B.fp4idx_build_tables(N, N, T, N, 64, 9, stream=s, **kw), 5, 0),
    "token table": (lambda s: B.fp4idx_pages_from_token_table(i32(3), i32(2, 70), 64, 9, stream=s), 3, 0),
    "logits": (lambda s, **kw: B.fp4idx_logits(problem(), W, 128, stream=s, **kw), 1, 0),
    "block scores": (lambda s, **kw: B.fp4idx_block_scores(problem(), stream=s, **kw), 1, 0),
    "block top-k": (lambda s: B.fp4idx_block_topk(SCORES, 3, stream=s), 3, 0),
    "slots": (lambda s: B.fp4idx_topk_slots(problem(), i32(2, 3), stream=s), 1, 0),
    "queries": (lambda s: B.fp4idx_quantize_q(torch.zeros((2, 3, 128), dtype=torch.bfloat16), stream=s), 2, 0),
    "top-k": (lambda s: B.fp4idx_topk(problem(), W, 3, stream=s), 3, 1),
    "logits and top-k": (lambda s: B.fp4idx_logits_topk(problem(), W, 3, stream=s), 4, 0),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("stream", [SIDE, None])
def test_what_a_call_makes_is_made_on_its_stream(monkeypatch, name, stream):
    call, outputs, scratch = CALLS[name]
    r = Recorder(monkeypatch, workspace=160)
    got = call(stream)
    at = stream or HERE
    assert r.calls == [at.cuda_stream] and r.now is HERE
    assert len(r.made) == outputs + scratch and all(s is at for _, s in r.made)
    given = {id(N), id(T)}
    mine = [x for x in (got if isinstance(got, tuple) else (got,)) if isinstance(x, torch.Tensor) and id(x) not in given]
    assert len(mine) == outputs
    # the caller uses them on the stream that is current outside
    assert {id(x) for x, s in r.recorded if s is HERE} == ({id(x) for x in mine} if stream else set())


def test_given_tensors_are_used_as_they_are(monkeypatch):
    r = Recorder(monkeypatch, workspace=160)
    ws = torch.zeros(160, dtype=torch.uint8)
    ws_of = N.device
    assert ws.device == ws_of
    B.fp4idx_fork_requests(N, N, N, T, N, 64, out=(i32(4), i32(4), i32(1)), stream=SIDE)
    B.fp4idx_release_pages(N, N, T, 64, 9, out=(i32(9), i32(1)), workspace=ws, stream=SIDE)
    B.fp4idx_compact_pages(N, T, 64, 9, 3, out=(i32(3), i32(3), i32(1), i32(1)), workspace=ws, stream=SIDE)
    B.fp4idx_logits(problem(), W, out=torch.zeros((2, 128)), stream=SIDE)
    given = (i32(2, 3), torch.zeros((2, 3)), i32(2))
    B.fp4idx_topk(problem(), W, 3, False, *given, ws, stream=SIDE)
    assert r.calls == [22] * 5 and r.made == [] and r.recorded == []
    B.fp4idx_topk(problem(), W, 3, False, given[0], stream=SIDE)  # some are given
    assert len(r.made) == 3 and all(s is SIDE for _, s in r.made) and len(r.recorded) == 2


def test_scratch_of_a_call_with_given_outputs(monkeypatch):
    r = Recorder(monkeypatch, workspace=160)
    B.fp4idx_release_pages(N, N, T, 64, 9, out=(i32(9), i32(1)), stream=SIDE)
    assert r.calls == [22] and [s for _, s in r.made] == [SIDE] and r.recorded == []
