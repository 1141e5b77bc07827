"""GPU: calls over a paged cache that are refused, or of which a part is, leave
the rest as it was."""
import math

import pytest
import torch

import bit_kv_cache_jfa_b200 as jfa
from bit_kv_cache_jfa_b200 import JfaError, _lib
from test_gpu_paged import D, check_cache, gen, make, make_rows

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


def state(table, cache):
    return [x.clone() for x in (cache.pages, cache.tail_k, cache.tail_v, table.table, table.seq_lens)]


def flag_of(cache, ws):
    torch.cuda.synchronize()
    flag = ws.error_flag(cache)
    ws.clear_error(cache)
    return flag


@pytest.mark.parametrize("n", [-1, -2**31, 2**31 - 1, 64 * 5 + 65])
def test_fork_of_a_parent_of_bad_length_leaves_the_child(n):
    """The pair is skipped whole; the call's other pair is made."""
    lens = [130, 200, 70, 64]
    table, cache, ws, rows = make(lens, 2, 2, seed=87)      # rows of 5 entries
    assert table.max_pages == 5
    table.seq_lens[0] = n
    before = state(table, cache)
    jfa.paged_fork(cache, torch.tensor([[0, 1], [2, 3]], dtype=torch.int32).cuda(), ws)
    assert flag_of(cache, ws) == _lib.DEVERR_BAD_INDEX
    after = state(table, cache)
    assert torch.equal(before[0], after[0])
    for a, b in zip(before[1:], after[1:]):
        assert torch.equal(a[:3], b[:3])                    # parent, its child, the other parent
    table.seq_lens[0] = 130
    table.rows[3], rows[3] = list(table.rows[2]), rows[2]
    assert int(table.seq_lens[3]) == 70
    check_cache(table, cache, rows)


@pytest.mark.parametrize("pairs", [[[0, 5]], [[-1, 1]], [[0, 0]], [[0, 1], [1, 2]], [[0, 2], [1, 2]],
                                   [[2**31 - 1, 1]], [[0, -2**31]]])
def test_refused_forks_change_nothing(pairs):
    """Pairs that are bad by themselves, or that meet (then each of them), beside a good one."""
    lens = [130, 200, 0, 64, 30]
    table, cache, ws, rows = make(lens, 2, 2, seed=89)
    before = state(table, cache)
    jfa.paged_fork(cache, torch.tensor(pairs + [[3, 4]], dtype=torch.int32).cuda()[:5], ws)
    assert flag_of(cache, ws) == _lib.DEVERR_BAD_INDEX
    after = state(table, cache)
    assert torch.equal(before[0], after[0])
    for a, b in zip(before[1:], after[1:]):
        assert torch.equal(a[:4], b[:4])
    assert int(table.seq_lens[4]) == 64
    rows[4] = rows[3]
    check_cache(table, cache, rows)


@pytest.mark.parametrize("cu", [[0, 11, 21, 30], [-1, 5, 15, 25], [16, 5, 15, 25], [0, -3, 10, 20],
                                [0, 2**31 - 1, 10, 20]])
def test_refused_ranges_change_nothing(cu):
    """Row ranges outside their tensors are skipped, in the append and in the
    read-back; a good one of the same call is brought in."""
    good = [i for i in range(3) if 0 <= cu[i] <= cu[i + 1] <= 24]
    lens = [130, 200, 300]
    table, cache, ws, rows = make(lens, 2, 2, seed=90)
    before = state(table, cache)
    c = torch.tensor(cu, dtype=torch.int32).cuda()
    outs = [torch.full((24, 2, D), 77.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    jfa.paged_gather(cache, c, 24, ws, k_out=outs[0], v_out=outs[1])
    assert flag_of(cache, ws) == _lib.DEVERR_BAD_INDEX
    whole = jfa.paged_gather(cache, torch.tensor([0, 130, 330, 630], dtype=torch.int32).cuda(), 630, ws)
    seen = torch.zeros(24, dtype=torch.bool)
    first = [0, 130, 330]
    for i in good:
        seen[cu[i]:cu[i + 1]] = True
        for x, w in zip(outs, whole):
            assert torch.equal(x[cu[i]:cu[i + 1]], w[first[i]:first[i] + cu[i + 1] - cu[i]])
    assert all((x[~seen.cuda()] == 77).all() for x in outs)
    # the append of these ranges: the table has grown by each good one's rows
    counts = [cu[i + 1] - cu[i] if i in good else 0 for i in range(3)]
    table.grow(counts)
    before = state(table, cache)
    k, v = (torch.randn(24, 2, D, generator=gen(s)).bfloat16() for s in (91, 92))
    jfa.paged_append(cache, k.cuda(), v.cuda(), ws, c)
    assert flag_of(cache, ws) == _lib.DEVERR_BAD_INDEX
    after = state(table, cache)
    for i in range(3):
        if i in good:
            rows[i] = tuple(torch.cat((a, x[cu[i]:cu[i + 1]])) for a, x in zip(rows[i], (k, v)))
        else:
            assert all(torch.equal(a[i], b[i]) for a, b in zip(before[1:3], after[1:3]))
    assert torch.equal(before[4], after[4]) and torch.equal(before[3], after[3])
    check_cache(table, cache, rows)


@pytest.mark.parametrize("sign", [1, -1])
def test_nan_rows_are_flagged_once_packed(sign):
    """A NaN in the tail is kept as it is; when its group is packed the flag
    shows it, its code is 0 and the others' are as without it."""
    n, hkv = 64, 2
    nan = torch.tensor([sign * math.nan]).bfloat16()
    for keys in (True, False):
        for token, channel in ((0, 0), (5, 77), (63, 127), (31, 64)):
            table = jfa.PageTable(2, 6, 4)
            cache = jfa.PagedKVCache(table, hkv, hkv)
            ws = jfa.PagedWorkspace(cache)
            k, v = make_rows(2 * n + 2, hkv, 95 + token)
            clean = (k, v)[0 if keys else 1][:n].clone()
            # what a code of 0 stands for: the smallest of the others it shares a scale with
            x = clean[:, 1, channel] if keys else clean[token, 1, channel // 32 * 32:channel // 32 * 32 + 32]
            others = torch.cat((x[:token], x[token + 1:])) if keys else \
                torch.cat((x[:channel % 32], x[channel % 32 + 1:]))
            (k, v)[0 if keys else 1][token, 1, channel] = nan
            clean[token, 1, channel] = others.min()
            jfa.paged_append(cache, k[:2 * n].cuda(), v[:2 * n].cuda(), ws, table.grow([n, n]))
            assert flag_of(cache, ws) == 0, "in the tail"
            assert torch.isnan(cache.tail_k if keys else cache.tail_v).sum() == 1
            table.grow(1)
            jfa.paged_append(cache, k[2 * n:].cuda(), v[2 * n:].cuda(), ws)
            assert flag_of(cache, ws) == _lib.DEVERR_NONFINITE_QUANT
            rows = []
            for b in range(2):
                kk, vv = k[n * b:n * b + n], v[n * b:n * b + n]
                if b == 0:
                    kk, vv = (clean, vv) if keys else (kk, clean)
                rows.append((torch.cat((kk, k[2 * n + b:][:1])), torch.cat((vv, v[2 * n + b:][:1]))))
            check_cache(table, cache, rows)
