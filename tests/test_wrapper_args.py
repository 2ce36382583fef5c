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


def buffers(rows, cols):
    t = q.nf4_empty(rows, cols, "cpu")
    return dict(codes=t.codes, scale8=t.scale8, scale2=t.scale2, offset=t.offset)


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 16421), (256, 128)])
def test_stored_tensor_takes_its_buffers(rows, cols):
    q.NF4Tensor(rows, cols, **buffers(rows, cols))
    more = {k: torch.cat((t, t)) for k, t in buffers(rows, cols).items()}      # longer ones are fine
    q.NF4Tensor(rows, cols, **more)


@pytest.mark.parametrize("name", ["codes", "scale8", "scale2", "offset"])
def test_stored_tensor_refuses_wrong_buffers(name):
    # 256 x 1024: 131072 bytes of codes, 4096 and 16 constants
    good = buffers(256, 1024)
    t = good[name]
    for bad in (t[:-1], t.to(torch.int32), torch.stack((t, t), 1)[:, 0][:max(t.numel(), 2)] if t.numel() > 1 else t[:0],
                torch.empty_like(t, device="meta")):
        with pytest.raises(ValueError, match=name if bad.device.type == "cpu" or name != "codes" else "scale8"):
            q.NF4Tensor(256, 1024, **{**good, name: bad})


def test_moe_refuses_more_experts_per_token_than_there_are():
    # 2^32 + 2 would reach the C call as 2
    x, router = torch.zeros(1, 128, dtype=torch.bfloat16), torch.zeros(4, 128)
    t = [q.nf4_empty(r, c, "cpu") for r, c in ((256, 128), (256, 128), (512, 64))]
    for k in (5, -1, 2 ** 32 + 2):
        with pytest.raises(ValueError, match="k must be"):
            q.qlora_moe_fwd(x, router, *t, k)


def test_workspace_with_strides_or_elsewhere_is_refused():
    cpu = torch.device("cpu")
    ws = torch.zeros(64, 2, dtype=torch.uint8)
    assert q._workspace(100, cpu, ws)[0] is ws
    with pytest.raises(ValueError, match="contiguous"):       # its 64 bytes would be taken from 64 in a row
        q._workspace(64, cpu, ws[:, 0])
    with pytest.raises(ValueError, match="device"):
        q._workspace(64, torch.device("meta"), ws)
