"""Attention over 8-bit caches and with capped or biased scores at the ends of its range, against 64 bits."""
import pytest
import torch

from score_ref import Pair, bits_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [8, 16])
def test_first_slopes_set_on_a_side_stream(cuda_device, bits):
    """Work queued on the default stream comes between the allocation of the slopes and their use on another one."""
    p = Pair(2, 4, 2, 64, 2, 8, [200, 131], 3, bits=bits, seed=5).load().append(3)
    p.slopes = [0.5, 0.125, 0.3, 1.0]
    q, lse = p.queries(3), p.lse(3)
    qd = bits_dev(q)
    out = torch.empty_like(qd)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # about a tenth of a second
    p.gpu.set_scores(0.0, p.slopes, stream=s)
    p.gpu.verify_attn(0, 0, qd, out=out, lse=lse, stream=s)
    s.synchronize()
    p.check(out, lse, q, 0)
    torch.cuda.synchronize()  # the default stream has run dry
    out.zero_()
    torch.cuda.synchronize()
    p.gpu.verify_attn(0, 0, qd, out=out, lse=lse, stream=s)
    s.synchronize()
    p.check(out, lse, q, 0)
    p.close()
