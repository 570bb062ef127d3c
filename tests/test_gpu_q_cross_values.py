"""GPU tests of what cross-attention and its gradient answer where values are not finite."""
import pytest
import torch

from exact_attention_68_gb300 import binding, cross
from test_gpu_o_cross import problem

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")

# B, Hq, Hkv, Sq, Sk, lens, D: each gradient kernel, a tile or more with keys that are not there beside ones that are
GRADS = [
    ((2, 2, 2, 30, 40, [33, 5]), 64), ((2, 4, 2, 20, 64, [50, 17]), 128), ((2, 2, 1, 7, 60, [3, 59]), 256),
    ((2, 2, 2, 300, 400, [333, 5]), 64), ((2, 4, 2, 70, 900, [800, 130]), 128), ((2, 2, 2, 150, 300, [290, 70]), 256),
]


@pytest.mark.parametrize("shape,D", GRADS, ids=str)
@pytest.mark.parametrize("what", ["q", "dout"])
@pytest.mark.parametrize("value", [NAN, INF])
def test_keys_that_are_not_there_have_no_gradient_whatever_the_queries_are(cuda_device, shape, D, what, value):
    """A query or upstream gradient that is not finite: its own dq and the keys of its head take it, keys behind
    the end get 0 all the same, and other rows and heads what they get without it."""
    B, Hq, Hkv, Sq, Sk, lens = shape
    q, k, v, dout, ln = problem(B, Hq, Hkv, Sq, Sk, D, lens, torch.bfloat16, seed=Sq + D)
    out, lse = cross.cross_fwd(q, k, v, ln)
    clean = cross.cross_bwd(q, k, v, out, lse, dout, ln)
    (q if what == "q" else dout)[1, 0, 2, 3] = value
    dq, dk, dv, _ = cross.cross_bwd(q, k, v, out, lse, dout, ln)
    torch.cuda.synchronize()
    assert binding.device_status() == binding.ATTN_OK
    for b, n in enumerate(lens):
        assert (dk[b, :, n:] == 0).all() and (dv[b, :, n:] == 0).all()
    assert not dq[1, 0, 2].isfinite().all() and not (dk[1, 0, :lens[1]].isfinite().all() and dv[1, 0, :lens[1]].isfinite().all())
    for got, want in zip((dk, dv), clean[1:3]):
        got = got.clone()
        got[1, 0] = want[1, 0]
        assert torch.equal(got, want)
    dq = dq.clone()
    dq[1, 0, 2] = clean[0][1, 0, 2]
    assert torch.equal(dq, clean[0])
