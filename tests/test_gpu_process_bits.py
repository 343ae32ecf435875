"""Entries that no penalty, bias or mask touches keep their bits, NaN's too, at rows' and slices' edges and inside."""
import pytest
import torch

import semi_autoregressive_drafting_gb300 as ds

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,ints,payload", [(torch.bfloat16, torch.int16, [0x7F81, 0x7FAB, -0x006F, -0x0001]),
                                                (torch.float32, torch.int32, [0x7F800001, 0x7FABCDEF, -0x007FFFFF, -1])])
@pytest.mark.parametrize("off", range(8))
@pytest.mark.parametrize("V", [9, 9001, 33003])
def test_nan_bits(dtype, ints, payload, off, V):
    B, R = 2, 3
    buf = torch.randn(B * R * V + off, generator=torch.Generator().manual_seed(V)).to(dtype)
    bits = buf.view(ints)
    # every row all NaN, of several kinds
    bits[off:] = torch.tensor(payload, dtype=ints)[torch.arange(B * R * V) % 4]
    z = buf.cuda()[off:].view(B, R, V)
    assert torch.equal(z.view(ints).cpu().flatten(), bits[off:])
    h = torch.full((B, 2), 5, dtype=torch.int32, device="cuda")
    freq = torch.tensor([0.5, 0.0], device="cuda")
    for pad in (0, 3, 8):
        wide = torch.zeros(B * R * (V + pad) + off, dtype=dtype, device="cuda")
        out = wide[off:].view(B, R, V + pad)[..., :V]
        ds.process_logits(z, history=h, frequency=freq, out=out)
        got, want = out.reshape(-1, V).view(ints).cpu(), bits[off:].view(-1, V)
        keep = torch.ones(V, dtype=torch.bool)
        keep[5] = False                                  # (the text's token)
        assert torch.equal(got[:, keep], want[:, keep]) and torch.equal(got[R:], want[R:])
        ds.process_logits_grad(z, torch.zeros_like(z), history=h, repetition=freq + 1.0, out=out)
        got = out.reshape(-1, V).view(ints).cpu()
        assert torch.equal(got[:, keep], want[:, keep]) and torch.equal(got[R:], want[R:])
