"""GPU checks of the 8-bit cache on unusual values: NaN and infinities in queries
and keys, padding rows that hold anything, bounds of NaN-only channels, and every
kernel of the attention by width, rows of a pass and route."""
import numpy as np
import pytest
import torch

from exact_attention_68_gb300 import binding, cache as kv
from oracle import cache as oc
from test_gpu_l_cache import BF, DEV, FP, check_fwd, clean_status, filled, ints, pool, rows, same_cache, to_np  # noqa: F401

pytestmark = pytest.mark.gpu

# The ways the attention's work is cut (152 SMs): lengths, heads and the table's
# width in pages of 64 tokens.  2817 = 44 chunks and one token, whose chunk is a
# worker's only one where chunks are dealt to CTAs (20 units a worker, 16 of them
# the segment's lead) and alone in its warp everywhere.
ROUTES = {
    "one CTA": ([65, 129, 1], 3),
    "cluster": ([2817, 65, 1], 45),
    "dealt to CTAs": ([2817, 65, 1], 2000),
    "dealt to warps": ([65, 129, 1] * 60, 3),
}


def call(c, q, table, lens, fresh, mass=True, fill=7.0):
    B, Hq, T, D = q.shape
    out = torch.full(q.shape, fill, dtype=q.dtype, device=DEV)
    lse = torch.full((B, Hq, T), fill, device=DEV)
    m = torch.zeros((B, c.k.shape[1], table.shape[1] * c.k.shape[2]), device=DEV) if mass else None
    kv.cache_fwd(q.to(DEV), c, ints(table), ints(lens), fresh=ints(fresh), mass=m, out=out, lse=lse)
    torch.cuda.synchronize()
    return out, lse, m


# ---------------------------------------------------------------- padding rows
@pytest.mark.parametrize("G", [2, 16])  # one pass of 6 rows, three of 16
@pytest.mark.parametrize("route", ROUTES)
def test_rows_behind_the_fresh_tokens_may_hold_anything(route, G):
    """Queries of tokens from fresh[b] on are not part of the step: no output or weight depends on them."""
    lens, width = ROUTES[route]
    T, D = 3, 128
    c, _, table, _ = filled(lens, 1, D, 64, BF, 11, width=width)
    fresh = np.minimum([[1, 3, 1][b % 3] for b in range(len(lens))], lens)
    q = rows((len(lens), G, T, D), BF, 12)
    want = call(c, q, table, lens, fresh)
    bad = q.clone()
    for b, n in enumerate(fresh):
        bad[b, :, n:] = torch.tensor([float("nan"), float("inf"), -float("inf"), 3e38]).to(BF).repeat(D // 4)
        bad[b, ::2, n:, 5:] = q[b, ::2, n:, 5:]
    got = call(c, bad, table, lens, fresh)
    assert all(torch.isfinite(w).all() for w in (want[0].float(), want[1], want[2]))
    for g, w in zip(got, want):
        assert torch.equal(g, w)
    assert binding.device_status() == binding.ATTN_OK
