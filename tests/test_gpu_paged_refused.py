"""GPU: calls over a paged cache that are refused, or of which a part is, leave
the rest as it was."""
import math

import pytest
import torch

import bit_kv_cache_jfa_b200 as jfa
from bit_kv_cache_jfa_b200 import JfaError
from test_gpu_paged import D, check_cache, gen, make, rand_q

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [
    dict(out="float"), dict(out="odd"), dict(lse="short"), dict(window=-1), dict(window=2.5), dict(sinks=2**31),
    dict(scale=0.0), dict(scale=1e-60), dict(scale=math.nan)], ids=str)
def test_refused_decode_step_changes_nothing(bad):
    """At lengths where a page completes; then the step goes through."""
    lens = [64, 0, 128, 30]
    table, cache, ws, rows = make(lens, 4, 2, seed=83)
    plan = jfa.RotaryPlan(128)
    table.grow(1)
    new = torch.randn(4, 8, D, generator=gen(83)).bfloat16().cuda()
    kw = dict(bad)
    if kw.get("out") == "float":
        kw["out"] = torch.zeros(4, 4, D, device="cuda")
    if kw.get("out") == "odd":
        kw["out"] = torch.zeros(4 * 4 * D + 8, dtype=torch.bfloat16, device="cuda")[4:4 + 4 * 4 * D].view(4, 4, D)
    if kw.get("lse") == "short":
        kw["lse"] = torch.zeros(4, 3, device="cuda")
    kept = [x.clone() for x in (cache.pages, cache.tail_k, cache.tail_v, table.table, table.seq_lens)]
    args = (cache, new[:, :4], new[:, 4:6], new[:, 6:], table.seq_lens - 1, plan, ws)
    with pytest.raises((JfaError, TypeError)):
        jfa.paged_decode_step(*args, **kw)
    torch.cuda.synchronize()
    for a, b in zip(kept, (cache.pages, cache.tail_k, cache.tail_v, table.table, table.seq_lens)):
        assert torch.equal(a, b)
    jfa.paged_decode_step(*args)
    _, k = jfa.qk_norm_rope(new[:, :4], new[:, 4:6], table.seq_lens - 1, plan)
    torch.cuda.synchronize()
    assert ws.error_flag(cache) == 0
    check_cache(table, cache, [(torch.cat((a, k[b:b + 1].cpu())), torch.cat((c, new[b:b + 1, 6:].cpu())))
                               if lens[b] else (a, c) for b, (a, c) in enumerate(rows)])


def test_rotation_in_place_between_other_heads():
    """Every other head of seven, in place: no two rows share a byte."""
    plan = jfa.RotaryPlan(128)
    wide = torch.randn(9, 7, D, generator=gen(85)).bfloat16().cuda()
    pos = torch.arange(9, device="cuda")
    before = wide.clone()
    k = wide[:, 1::2]
    want = jfa.qk_norm_rope(wide[:, ::2], k, pos, plan)
    got = jfa.qk_norm_rope(wide[:, ::2], k, pos, plan, q_out=wide[:, ::2], k_out=torch.empty_like(want[1]))
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(wide[:, 1::2], before[:, 1::2]) and torch.equal(wide[:, ::2], want[0])
