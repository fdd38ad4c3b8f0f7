"""What the binding hands to the library for an 8-bit matrix, on the host: its tensors stand in for
device tensors, and no call reaches the library."""
import pytest
import torch

import fsdp_sharded_optimizer_zs_amd as zs
from fsdp_sharded_optimizer_zs_amd import _binding as B


@pytest.fixture
def calls(monkeypatch):
    """The arguments of every call that the binding makes."""
    seen = []
    typed = B._typed

    def on_host(t, what, dtype, numel=None, dev=None):
        if t.dtype != dtype or not t.is_contiguous() or numel not in (None, t.numel()):
            typed(t, what, dtype, numel, dev)            # raises

    monkeypatch.setattr(B, "_typed", on_host)
    monkeypatch.setattr(B, "_matrix", lambda t, *a: (zs.ZS_BF16, t.shape[1]))
    monkeypatch.setattr(B, "_enqueue", lambda f, ref, stream, *args: seen.append(args))
    return seen


def made(rows=128, cols=256):
    return zs.F8Matrix(*(torch.zeros(n, dtype=torch.uint8) for n in zs.zs_f8_layout(rows, cols, 128)), rows, cols,
                       block_rows=128)


def handed(calls, m):
    """Codes' and scales' addresses that a call with m passes on."""
    zs.zs_dequantize_f8(m, torch.zeros(m.rows, m.cols, dtype=torch.bfloat16))
    c = calls.pop()[0]._obj
    assert (c.rows, c.cols, c.type, c.block_rows) == (m.rows, m.cols, m.type, m.block_rows)
    return c.codes, c.scales


def test_calls_take_the_buffers_where_they_are(calls):
    """A gathered matrix whose storage is freed between the passes and taken again."""
    m, kept = made(), []
    for k in range(3):
        assert handed(calls, m) == (m.codes.data_ptr(), m.scales.data_ptr())
        before = m.codes.data_ptr()
        for t in (m.codes, m.scales):
            n = t.untyped_storage().nbytes()
            t.untyped_storage().resize_(0)
            kept.append(torch.zeros(n, dtype=torch.uint8))      # somebody else's by now
            t.untyped_storage().resize_(n)
        if k == 0:
            m.codes.data = torch.zeros_like(m.codes)
            assert m.codes.data_ptr() != before
    assert handed(calls, m) == (m.codes.data_ptr(), m.scales.data_ptr())


def test_freed_and_exchanged_buffers_are_refused(calls):
    m = made()
    m.codes.untyped_storage().resize_(0)
    with pytest.raises(ValueError, match="codes"):
        handed(calls, m)
    m = made()
    m.scales.data = torch.zeros(m.scales.numel() - 4, dtype=torch.uint8)
    with pytest.raises(ValueError, match="scales"):
        handed(calls, m)
    assert not calls
    empty = made(0, 256)                                        # has no buffers to lose
    assert handed(calls, empty) is not None
