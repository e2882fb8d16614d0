"""The convolution's prompts and tokens of more channels than its gradients take, against the definition in 64 bits
(tolerances: those of a row, fp32 16 2^-24 with room for a sum of W terms, bf16 one rounding of 2^-8)."""
import pytest
import torch

from linear_token_mixer_gb300 import fw

import mixer_ref as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 4e-6), (torch.bfloat16, 4.1e-3)])
@pytest.mark.parametrize("H,d,T", [(32, 65536, 3), (1, 65535 * 32 + 1, 2), (1, 65535 * 32 + 8, 9)])
def test_many_channels(H, d, T, dtype, tol):
    W, gen = 4, torch.Generator().manual_seed(T)
    x, state = (torch.randn(1, H, n, d, generator=gen).to(dtype) for n in (T, W - 1))
    w, b = 0.5 * torch.randn(H, d, W, generator=gen), torch.randn(H, d, generator=gen)
    want, end = R.conv(*[R.f64(t) for t in (x, w, b, state)])
    x, w, b, state = (t.cuda() for t in (x, w, b, state))
    y, so = fw.conv_prefill(x, w, b, state)
    first, past = fw.conv_prefill(x[:, :, :-1].clone(memory_format=torch.contiguous_format), w, b, state)
    last = fw.conv_step(x[:, :, -1].clone(), w, b, past)      # (rows of an odd width: an address of its own)
    fw.check()
    assert R.rel(y, want) <= tol and torch.equal(so.cpu().double(), end)
    assert torch.equal(torch.cat([first, last.unsqueeze(2)], 2), y) and torch.equal(past, so)
    with pytest.raises(fw.FwError, match="SHAPE"):
        fw.conv_backward(x, x, w, b)
