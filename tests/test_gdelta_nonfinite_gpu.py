"""A live token that is not finite: what the header says it touches, and nothing else."""
from __future__ import annotations

import pytest
import torch

from xlstm_mlstm_cell_b200 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("name", ["q", "k", "v", "g", "beta"])
@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
def test_other_items_heads_and_earlier_chunks_keep_their_bits(name, dt, poison):
    B, NH, NHV, S, DK, DV, at = 3, 2, 4, 200, 64, 64, 100
    gen = torch.Generator().manual_seed(70)
    r = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    unit = lambda x: torch.nn.functional.normalize(x, dim=-1).to(dt).cuda()   # noqa: E731
    x = dict(q=unit(r(B, NH, S, DK)), k=unit(r(B, NH, S, DK)), v=r(B, NHV, S, DV).to(dt).cuda(),
             g=-torch.rand(B, NHV, S, generator=gen).cuda(), beta=torch.rand(B, NHV, S, generator=gen).cuda())
    do = r(B, NHV, S, DV).to(dt).cuda()
    o, state = binding.gdelta_fwd(**x)
    grads = binding.gdelta_bwd(**x, do=do)
    x[name][1, 0, at] = poison
    po, pstate = binding.gdelta_fwd(**x)
    pgrads = binding.gdelta_bwd(**x, do=do)
    torch.cuda.synchronize()
    heads = 2 if name in "qk" else 1            # value heads 0 and 1 read key head 0
    clean = torch.ones(B, NHV, dtype=torch.bool)
    clean[1, :heads] = False
    assert torch.equal(o[clean], po[clean]) and torch.equal(state[clean], pstate[clean])
    assert torch.equal(o[1, :, :64], po[1, :, :64])                      # the chunk in front of the token's
    assert not torch.isfinite(po[1, :heads, at]).all()
    for n, a, b in zip(("dq", "dk", "dv", "dg", "dbeta"), grads, pgrads):
        same = clean if a.shape[1] == NHV else clean.view(B, NH, -1).all(-1)
        assert torch.equal(a[same], b[same]), n
