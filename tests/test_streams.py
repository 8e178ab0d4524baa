"""Calls on another stream than the current one, which allocate what the caller
does not give: no memory that the current stream has still to write is used,
accumulators are zero when the kernels add to them, and tensors that the caller
drops are not handed out again before their last use.

Each hazard is made to last by a delay on one of the streams; the results are
compared with those of the same calls on the current stream.
"""
import pytest
import torch

from long_context_causal_gb300 import dfa
from long_context_causal_gb300.inputs import make

DELAY = 40_000_000      # cycles, about 20 ms: longer than what the host does meanwhile
CU = [0, 300, 300, 1000]


def chain(q, k, v, do, stream=None, cu=CU):
    """Every call that allocates; dQ (fp32 atomics) apart from what has the same bits each time."""
    same, near = [], []
    kw = dict(stream=stream)
    part = dfa.dfa_chunk_attn_fwd(q, k, v, **kw)
    grads = dfa.dfa_chunk_attn_bwd(q, k, v, part[0].to(q.dtype) if stream is None else chain.O, part[1], do, **kw)
    same += [*part, *dfa.dfa_merge_partials(*part, *part, **kw)]
    near += grads
    O, lse = dfa.dfa_attn_fwd(q, k, v, **kw)
    grads = dfa.dfa_attn_bwd(q, k, v, O, lse, do, **kw)
    same += [O, lse, *grads[1:]]
    near += grads[:1]
    O, lse = dfa.dfa_attn_fwd_local(q, k, v, 4, 2, **kw)
    grads = dfa.dfa_attn_bwd_local(q, k, v, O, lse, do, 4, 2, **kw)
    same += [O, lse, *grads[1:]]
    near += grads[:1]
    O, lse = dfa.dfa_attn_fwd_varlen(q[0], k[0], v[0], cu, **kw)
    grads = dfa.dfa_attn_bwd_varlen(q[0], k[0], v[0], O, lse, do[0], cu, **kw)
    same += [O, lse, *grads[1:]]
    near += grads[:1]
    return same, near


def agree(got, want):
    for a, b in zip(got[0], want[0]):
        assert torch.equal(a, b)
    for a, b in zip(got[1], want[1]):     # fp32 sums in another order, rounded to bf16 at most once
        torch.testing.assert_close(a.float(), b.float(), rtol=2.0 ** -7, atol=2e-3)


@pytest.mark.gpu
@pytest.mark.parametrize("raw", [False, True])
def test_memory_of_calls_on_another_stream(raw):
    q, k, v, do = make(1, 4, 2, 1000, 128, torch.bfloat16, device="cuda", seed=3)
    chain.O = dfa.dfa_chunk_attn_fwd(q, k, v)[0].to(q.dtype)
    want, now, s = chain(q, k, v, do), torch.cuda.current_stream(), torch.cuda.Stream()
    stream = s.cuda_stream if raw else s
    for _ in range(3):
        # blocks of the outputs' sizes that the current stream is about to fill
        torch.cuda.synchronize()
        blocks = [torch.empty_like(t) for part in want for t in part]
        torch.cuda._sleep(DELAY)
        for t in blocks:
            t.fill_(7)
        del blocks
        got = chain(q, k, v, do, stream)
        torch.cuda.synchronize()
        agree(got, want)
        # inputs that are dropped while the other stream has still to read them
        held = [t.clone() for t in (q, k, v)]
        s.wait_stream(now)
        with torch.cuda.stream(s):
            torch.cuda._sleep(DELAY)
        O, lse = dfa.dfa_attn_fwd(*held, stream=stream)
        del held
        blocks = [torch.full_like(t, 1) for t in (q, k, v)]
        torch.cuda.synchronize()
        del blocks
        assert torch.equal(O, want[0][4]) and torch.equal(lse, want[0][5])
        # an output that is dropped while the current stream has still to read it
        other = q.flip(1).contiguous()
        torch.cuda.synchronize()
        O = dfa.dfa_attn_fwd(q, k, v, stream=stream)[0]
        s.synchronize()
        torch.cuda._sleep(DELAY)
        seen = O.clone()
        del O
        dfa.dfa_attn_fwd(other, k, v, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(seen, want[0][4])
    # offsets that the current stream has still to write
    cu = torch.zeros(len(CU), dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(DELAY)
    cu.copy_(torch.tensor(CU, dtype=torch.int32).pin_memory(), non_blocking=True)
    got = chain(q, k, v, do, stream, cu)
    torch.cuda.synchronize()
    agree(got, want)
    dfa.dfa_check_errors()


def test_a_call_on_the_current_stream_stays_as_it_was(monkeypatch):
    """The wrapper passes a call without a stream straight on (CPU)."""
    seen = []

    @dfa._on_its_stream
    def call(a, b=2, stream=None):
        seen.append((a, b, stream))
        return (a,)

    monkeypatch.setattr(torch.cuda, "current_stream", lambda: pytest.fail("not asked"))
    assert call(1) == (1,) and call(1, b=3, stream=None) == (1,) and call(5, 6, None) == (5,)
    assert seen == [(1, 2, None), (1, 3, None), (5, 6, None)]
    assert list(__import__("inspect").signature(call).parameters) == ["a", "b", "stream"]


def test_a_stream_of_another_device_is_refused(monkeypatch):
    """Before anything is allocated or launched (CPU, with stand-ins for the streams)."""
    class Stream:
        def __init__(self, device, cuda_stream):
            self.device, self.cuda_stream = torch.device("cuda", device), cuda_stream

    @dfa._on_its_stream
    def call(a, stream=None):
        return (a, stream)

    now = Stream(0, 16)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: now)
    with pytest.raises(ValueError, match="cuda:1"):
        call(1, Stream(1, 32))
    same = Stream(0, 16)
    assert call(1, stream=same) == (1, same)
