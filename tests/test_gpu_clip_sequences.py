"""The sequences of gradients that the norm and the clipping take: held for the call."""
import math

import pytest
import torch

import scaled_quantize_gemm_amax_gb300 as fq
from gpu_util import require_gpu
from row_util import gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def gradients(seed=1):
    return [torch.randn(n, generator=gen(seed + n), device="cuda") for n in (70000, 33, 5000)]


class Emptying:
    """A stream whose handle is asked for in the middle of the call, and which then empties the caller's lists."""

    def __init__(self, *lists):
        self.lists = lists

    @property
    def cuda_stream(self):
        for x in self.lists:
            x.clear()
        return torch.cuda.current_stream().cuda_stream


def expected(grads, max_norm):
    outs = [torch.empty_like(g) for g in grads]
    return fq.clip_grad_norm(grads, max_norm, out=outs), outs


def test_a_list_emptied_during_the_call():
    norm, want = expected(gradients(), 0.5)
    grads, kept = gradients(), gradients()
    grads[:] = kept
    assert torch.equal(fq.grad_norm(grads, stream=Emptying(grads)), norm) and not grads
    grads[:] = kept
    outs = [torch.empty_like(g) for g in kept]
    held = list(outs)
    assert torch.equal(fq.clip_grad_norm(grads, 0.5, out=outs, stream=Emptying(grads, outs)), norm)
    assert all(torch.equal(a, b) for a, b in zip(held, want)) and not grads and not outs
    grads[:] = kept
    versions = [g._version for g in kept]
    assert torch.equal(fq.clip_grad_norm(grads, 0.5, stream=Emptying(grads)), norm)
    assert all(torch.equal(a, b) for a, b in zip(kept, want)) and all(g._version > v for g, v in zip(kept, versions))


def test_gradients_that_nothing_else_holds():
    """What the list alone held is still read by the call that emptied it."""
    norm, want = expected(gradients(), 0.5)
    for _ in range(3):
        grads, outs = gradients(), [torch.empty_like(g) for g in want]
        held = list(outs)
        got = fq.clip_grad_norm(grads, 0.5, out=outs, stream=Emptying(grads, outs))
        torch.full((70000,), 9.0, device="cuda")   # takes the memory of the first one, behind the call
        assert torch.equal(got, norm) and all(torch.equal(a, b) for a, b in zip(held, want))


def test_through_the_c_names():
    norm, want = expected(gradients(), 0.5)
    ws = torch.empty(fq.fp8_grad_norm_workspace(3), dtype=torch.uint8, device="cuda")
    got = torch.empty(1, device="cuda")
    grads, outs = gradients(), [torch.empty_like(g) for g in want]
    held = list(outs)
    fq.fp8_clip_grad_norm(grads, outs, 0.5, ws, got, stream=Emptying(grads, outs))
    assert torch.equal(got, norm) and all(torch.equal(a, b) for a, b in zip(held, want))
    grads = gradients()
    got.zero_()
    fq.fp8_grad_norm(grads, ws, got, stream=Emptying(grads))
    assert torch.equal(got, norm)
    assert abs(float(got) / math.sqrt(sum(float(g.double().square().sum()) for g in gradients())) - 1) < 1e-6


def test_generators():
    """Every kind of sequence gives what a list gives, in place and not."""
    norm, want = expected(gradients(), 0.5)
    for make in (lambda ts: (t for t in ts), tuple, lambda ts: {i: t for i, t in enumerate(ts)}.values()):
        grads = gradients()
        assert torch.equal(fq.grad_norm(make(grads)), norm)
        outs = [torch.empty_like(g) for g in grads]
        assert torch.equal(fq.clip_grad_norm(make(grads), 0.5, out=make(outs)), norm)
        assert torch.equal(fq.clip_grad_norm(make(grads), 0.5), norm)
        for a, b, c in zip(outs, grads, want):
            assert torch.equal(a, c) and torch.equal(b, c)


def test_refuses_memory_shared_by_another_storage():
    """A tensor taken over by DLPack has a storage of its own in the other's memory."""
    b = torch.randn(1000, generator=gen(9), device="cuda")
    other = torch.from_dlpack(b)
    assert other.untyped_storage().data_ptr() == b.untyped_storage().data_ptr() and other.data_ptr() == b.data_ptr()
    was = b.clone()
    for grads, out in (([b, other], None), ([other, b], None), ([b[:600], torch.from_dlpack(b[500:])], None),
                       ([torch.from_dlpack(b[500:]), b[:600]], None), ([b[:500]], [other[250:750]]), ([other[:500]], [b[250:750]])):
        with pytest.raises(ValueError, match="share memory"):
            fq.clip_grad_norm(grads, 0.1, out=out)
        assert torch.equal(b, was)
    norm, want = expected([was[:500], was[500:]], 0.1)
    assert torch.equal(fq.clip_grad_norm([b[:500], torch.from_dlpack(b[500:])], 0.1), norm)    # apart
    assert torch.equal(b, torch.cat(want))
    b.copy_(was)
    assert torch.equal(fq.clip_grad_norm([b[:500], b[500:]], 0.1, out=[other[:500], other[500:]]), norm)   # each in itself
    assert torch.equal(b, torch.cat(want))
