"""Cross-attention and the heads' norm and rotation on the debug build (-DATTN_DEBUG,
see test_gpu_i_debug_checks): its in-kernel index checks find nothing over ragged
shapes, every kernel, width and route, and it gives the release build's bits."""
import pytest
import torch

from exact_attention_68_gb300 import binding, cross, rope
from exact_attention_68_gb300.build import build_debug_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dbg(cuda_device):
    lib = binding.load_library(build_debug_library())
    return rope.declare(cross.declare(lib))


def _status(lib):
    return lib.attn_device_status(torch.cuda.current_stream().cuda_stream)


CROSS = [  # B, Hq, Hkv, Sq, Sk, lens: few queries with clusters and runs, tiles, runs of tiles, small gradients, many
    (5, 4, 2, 1, 900, [900, 0, 1, 511, 64]), (1, 8, 1, 3, 20000, [19999]), (2, 2, 2, 20, 300, [300, 7]),
    (1, 4, 2, 64, 4000, [3333]), (2, 2, 2, 1000, 100, [100, 3]), (2, 3, 3, 30, 60, [60, 0]), (1, 2, 2, 300, 5000, None),
    (3, 8, 4, 500, 700, [700, 0, 129]), (2, 16, 16, 1500, 300, [300, 130]),
]


@pytest.mark.parametrize("shape", CROSS, ids=str)
@pytest.mark.parametrize("D", [64, 72, 128, 192, 256])
def test_cross_no_check_fails(dbg, monkeypatch, shape, D):
    B, Hq, Hkv, Sq, Sk, lens = shape
    g = torch.Generator().manual_seed(Sq + Sk + D)
    dt = torch.float16 if D == 72 else torch.bfloat16
    q, dout = (torch.randn(B, Hq, Sq, D, generator=g).to(dt).cuda() for _ in "qd")
    k, v = (torch.randn(B, Hkv, Sk, D, generator=g).to(dt).cuda() for _ in "kv")
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda()
    want = cross.cross_fwd(q, k, v, ln)
    want += cross.cross_bwd(q, k, v, *want, dout, ln)
    assert binding.device_status() == binding.ATTN_OK
    monkeypatch.setattr(cross, "_lib", dbg)
    got = cross.cross_fwd(q, k, v, ln)
    got += cross.cross_bwd(q, k, v, *got, dout, ln)
    assert _status(dbg) == binding.ATTN_OK
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("D,pairs,interleaved", [(64, 32, False), (72, 36, True), (128, 64, False), (80, 17, False),
                                                 (256, 128, True), (200, 50, False), (8, 0, False)])
def test_rope_no_check_fails(dbg, monkeypatch, D, pairs, interleaved):
    g = torch.Generator().manual_seed(D)
    for B, S, heads in ((2, 37, (4, 1, 1)), (1, 700, (3, 3, 3)), (16, 1, (32, 8, 8))):
        x = torch.randn(B, S, sum(heads), D, generator=g).to(torch.bfloat16).cuda()
        xs = x.split(heads, dim=2)
        w = [torch.randn(D, generator=g).cuda() for _ in "qk"] + [None]
        plan = rope.Rope(torch.rand(pairs, generator=g, dtype=torch.float64), None, interleaved)
        pos = torch.arange(S, dtype=torch.int32).cuda()[None]
        dys = [torch.randn(B, h, S, D, generator=g).to(torch.bfloat16).cuda() for h in heads]
        turn = (True, True, False)

        def both():
            ys = rope.rope_fwd(xs, plan, pos, w, 1e-6, turn)
            dxs, dws = rope.rope_bwd(dys, xs, plan, pos, w, 1e-6, turn)
            return ys + dxs + dws[:2]

        want = both()
        with monkeypatch.context() as m:
            m.setattr(rope, "_lib", dbg)
            got = both()
        assert _status(dbg) == binding.ATTN_OK
        assert all(torch.equal(a, b) for a, b in zip(got, want))
