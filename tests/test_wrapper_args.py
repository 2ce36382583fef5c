"""What the binding does with its arguments before anything is launched: no GPU needed."""
import contextlib

import pytest
import torch

import bit_nf4_quantized_double_b200 as q


def test_copies_are_made_on_the_calls_stream(monkeypatch):
    # a copy queued on another stream than the kernel's could still be running, or not have begun, when the kernel reads it
    now, made_on = [None], []

    @contextlib.contextmanager
    def stream(s):
        before, now[0] = now[0], s
        yield
        now[0] = before

    class Strided(torch.Tensor):
        def contiguous(self, *a, **kw):
            made_on.append(now[0])
            return super().contiguous(*a, **kw)

    monkeypatch.setattr(torch.cuda, "stream", stream)
    x = torch.arange(24.0).view(4, 6)[:, ::2].as_subclass(Strided)
    dense, = q._dense("s", x)
    assert dense.is_contiguous() and torch.equal(dense, x) and made_on == ["s"]
    y = torch.zeros(3)
    assert q._dense("s", y)[0] is y
