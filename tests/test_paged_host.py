"""CPU checks of the paged cache's host side: the page book-keeping, the rotary
frequencies, the workspace's size, and the refusals of every entry point before
any launch."""
import math
import random

import pytest
import torch

import bit_kv_cache_jfa_b200 as jfa
from bit_kv_cache_jfa_b200 import JfaError, _lib

BAD = _lib.JFA_ERR_INVALID_ARG
UNSUPPORTED = _lib.JFA_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def built():
    from bit_kv_cache_jfa_b200 import build
    build.build()


def _split(n):
    return 0 if n <= 0 else (n - 1) // 64


def _check_book(t):
    """Device copies as the host's book; every page counted once per row that lists it."""
    assert t.seq_lens.tolist() == t.lens
    count = [0] * t.n_pages
    for b, row in enumerate(t.rows):
        assert len(row) == _split(t.lens[b])
        for p in row:
            count[p] += 1
    assert count == t._refs
    assert sorted(t._free) == [p for p in range(t.n_pages) if count[p] == 0]


def _check_table(t):
    for b, row in enumerate(t.rows):
        assert t.table[b, :len(row)].tolist() == row


def test_grow_gives_pages_when_groups_complete():
    t = jfa.PageTable(3, 8, 4, device="cpu")
    cu = t.grow([64, 0, 65])
    assert cu.tolist() == [0, 64, 64, 129] and cu.dtype == torch.int32
    assert t.rows == [[], [], [0]] and t.lens == [64, 0, 65]
    assert t.grow(1) is None                         # the idle row stays idle
    assert t.lens == [65, 0, 66] and t.rows == [[1], [], [0]]
    _check_book(t)
    _check_table(t)
    t.grow([130, 1, 0])
    assert t.lens == [195, 1, 66] and t.rows[0] == [1, 2, 3]
    _check_book(t)
    _check_table(t)


def test_grow_refuses_without_changing_anything():
    t = jfa.PageTable(2, 3, 2, device="cpu")
    t.grow([100, 30])
    before = (list(t.lens), [list(r) for r in t.rows], t.table.clone())
    for counts in ([100, 0], [0, 200], [-1, 0], [1], [60, 100]):
        with pytest.raises(JfaError) as e:
            t.grow(counts)
        assert e.value.status == BAD
        assert (t.lens, t.rows) == before[:2] and torch.equal(t.table, before[2])
        _check_book(t)


def test_grow_takes_whole_numbers_of_any_kind():
    import numpy as np
    t = jfa.PageTable(2, 4, 4, device="cpu")
    t.grow(np.array([3, 0]))
    t.grow(np.int64(2))
    assert t.lens == [5, 0]
    _check_book(t)


def test_fork_shares_and_free_counts():
    t = jfa.PageTable(4, 10, 4, device="cpu")
    t.grow([200, 70, 0, 0])
    pairs = t.fork([(0, 2), (0, 1)])
    assert pairs.tolist() == [[0, 2], [0, 1]] and pairs.dtype == torch.int32
    assert t.rows[1] == t.rows[2] == t.rows[0] and t.lens == [200, 200, 200, 0]
    assert t.free_pages == 7                         # row 1's own page is free again
    t.free([0])
    assert t.free_pages == 7 and t.lens[0] == 0
    t.free([1, 2])
    assert t.free_pages == 10
    for bad in ([(1, 1)], [(0, 1), (1, 2)], [(0, 1), (2, 1)], [(0, 4)], [(-1, 0)]):
        with pytest.raises(JfaError):
            t.fork(bad)
    with pytest.raises(JfaError):
        t.free([4])


def test_compact_moves_pages_in_use_to_the_front():
    t = jfa.PageTable(4, 40, 8, device="cpu")
    t.grow([300, 200, 500, 0])
    t.fork([(2, 3)])
    t.free([0, 1])
    rows = [list(r) for r in t.rows]
    moves, remap = t.compact()
    n_used = 7
    assert sorted({p for r in t.rows for p in r}) == list(range(n_used))
    remap = remap.tolist()
    assert [[remap[p] for p in r] for r in rows] == t.rows
    src, dst = zip(*moves.tolist())
    assert not set(src) & set(dst) and len(set(src)) == len(src) and len(set(dst)) == len(dst)
    for a, b in moves.tolist():
        assert remap[a] == b and remap[b] == b
    assert all(remap[p] == p for p in range(40) if p not in src)
    assert t.seq_lens.tolist() == t.lens == [0, 0, 500, 500]
    moves, _ = t.compact()
    assert moves.shape == (0, 2)


def test_random_book_keeping():
    rng = random.Random(5)
    t = jfa.PageTable(6, 60, 12, device="cpu")
    for _ in range(300):
        op = rng.randrange(4)
        try:
            if op == 0:
                t.grow([rng.choice([0, 1, 5, 64, 130]) for _ in range(6)])
            elif op == 1:
                t.grow(1)
            elif op == 2:
                a, b = rng.sample(range(6), 2)
                t.fork([(a, b)])
                # what paged_fork does on the device
                t.table[b], t.seq_lens[b] = t.table[a].clone(), t.lens[b]
            else:
                t.free([rng.randrange(6)])
        except JfaError:
            pass
        _check_book(t)
        _check_table(t)


@pytest.mark.parametrize("scaling,kw", [
    ("none", {}), ("linear", dict(factor=4.0)),
    ("llama3", dict(factor=8.0, low_freq_factor=1.0, high_freq_factor=4.0, original=8192)),
    ("yarn", dict(factor=16.0, original=16384))])
@pytest.mark.parametrize("rotary", [2, 6, 64, 128])
def test_rotary_frequencies(scaling, kw, rotary):
    base = 500000.0
    plan = jfa.RotaryPlan(rotary, base=base, scaling=scaling, device="cpu", **kw)
    for i, (f, turn) in enumerate(zip(plan.frequencies, plan.freq.tolist())):
        w = base ** (-2 * i / rotary)
        if scaling == "linear":
            want = w / 4
        elif scaling == "llama3":
            length = 2 * math.pi / w
            if length < 8192 / 4:
                want = w
            elif length > 8192:
                want = w / 8
            else:
                u = (8192 / length - 1) / 3
                want = (1 - u) * w / 8 + u * w
        elif scaling == "yarn":
            lo, hi = (rotary * math.log(16384 / (b * 2 * math.pi)) / (2 * math.log(base)) for b in (32, 1))
            lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), rotary - 1)
            u = min(max((i - lo) / max(hi - lo, 1e-3), 0), 1)
            want = u * w / 16 + (1 - u) * w
        else:
            want = w
        assert math.isclose(f, want, rel_tol=1e-13)
        # a whole number of units of 2 pi 2^-64: half a unit off, 1e-12 of the slowest frequency here
        assert math.isclose((turn % 2**64) / 2**64 * 2 * math.pi, f, rel_tol=1e-13, abs_tol=math.pi * 2.0**-64)
    assert plan.freq.shape == (rotary // 2,)
    assert math.isclose(plan.amplitude, 0.1 * math.log(16) + 1 if scaling == "yarn" else 1.0)


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=0), dict(rotary_dim=130), dict(rotary_dim=7), dict(base=1.0), dict(factor=0.0),
    dict(scaling="other"), dict(scaling="llama3"), dict(scaling="yarn"),
    dict(scaling="llama3", original=8192, low_freq_factor=4.0),
    dict(scaling="yarn", original=8192, beta_slow=40.0), dict(amplitude=math.inf)])
def test_rotary_plan_refusals(kw):
    with pytest.raises(JfaError) as e:
        jfa.RotaryPlan(device="cpu", **kw)
    assert e.value.status == BAD


def _paged(**kw):
    d = dict(batch=2, num_heads=8, num_kv_heads=2, n_pages=10, max_pages=5, reserved=0, pages=256,
             tail_k=256, tail_v=256, table=256, seq_lens=256)
    d.update(kw)
    return _lib.Paged(*d.values())


def test_workspace_bytes():
    n = _lib.jfa_paged_workspace_bytes(_paged())
    part = 8 * 132 * 4                               # a partial of 8 heads
    # flag, tickets, two partials of each block and one of each of its 12 warps
    assert n == 256 + 256 + 192 * (2 + 12) * part
    assert _lib.jfa_paged_workspace_bytes(_paged(batch=256, num_kv_heads=8)) == n + 256 * 8 * 4 - 256


@pytest.mark.parametrize("bad,status", [
    (dict(batch=0), BAD), (dict(batch=257), BAD), (dict(num_heads=9), BAD), (dict(num_kv_heads=0), BAD),
    (dict(num_heads=18, num_kv_heads=2), BAD), (dict(n_pages=0), BAD), (dict(max_pages=0), BAD),
    (dict(max_pages=1 << 26), UNSUPPORTED), (dict(num_heads=1 << 17, num_kv_heads=1 << 16), UNSUPPORTED),
    (dict(batch=256, num_heads=256, num_kv_heads=256, max_pages=1 << 16), UNSUPPORTED)])
def test_bad_sizes_refused(bad, status):
    c = _paged(**bad)
    with pytest.raises(JfaError) as e:
        _lib.jfa_paged_workspace_bytes(c)
    assert e.value.status == status
    assert _lib.jfa_paged_append(c, 256, 8, 8, 256, 8, 8, 256, 2, 256) == status
    assert _lib.jfa_paged_gather(c, 256, None, 2, 256, 256, 256) == status
    assert _lib.jfa_paged_attend(c, 256, 1024, 0.1, 0, 0, 256, 256) == status
    assert _lib.jfa_paged_fork(c, 256, 1, 256) == status
    assert _lib.jfa_paged_move(c, 256, 1, 256, 256) == status


@pytest.mark.parametrize("bad", [dict(pages=0), dict(pages=264), dict(tail_k=0), dict(tail_v=8), dict(table=0),
                                 dict(table=258), dict(seq_lens=0)])
def test_bad_buffers_refused(bad):
    c = _paged(**bad)
    assert _lib.jfa_paged_append(c, 256, 8, 8, 256, 8, 8, 256, 2, 256) == BAD
    assert _lib.jfa_paged_attend(c, 256, 1024, 0.1, 0, 0, 256, 256) == BAD
    assert _lib.jfa_paged_move(c, 256, 1, None, 256) == BAD


def test_bad_arguments_refused_before_launch():
    c = _paged()
    # append: count, uniform split, pointers, strides, workspace
    assert _lib.jfa_paged_append(c, 256, 8, 8, 256, 8, 8, 256, -1, 256) == BAD
    assert _lib.jfa_paged_append(c, 256, 8, 8, 256, 8, 8, None, 3, 256) == BAD
    assert _lib.jfa_paged_append(c, None, 8, 8, 256, 8, 8, 256, 2, 256) == BAD
    assert _lib.jfa_paged_append(c, 256, 12, 8, 256, 8, 8, 256, 2, 256) == BAD
    assert _lib.jfa_paged_append(c, 256, 8, 8, 260, 8, 8, 256, 2, 256) == BAD
    assert _lib.jfa_paged_append(c, 256, 8, 8, 256, 8, 8, 256, 2, 128) == BAD
    assert _lib.jfa_paged_append(c, 256, 8, 8, 256, 8, 8, 256, 2, None) == BAD
    assert _lib.jfa_paged_append(c, None, 8, 8, None, 8, 8, None, 0, 256) == 0     # nothing to do
    # gather
    assert _lib.jfa_paged_gather(c, None, None, 2, 256, 256, 256) == BAD
    assert _lib.jfa_paged_gather(c, 256, 258, 2, 256, 256, 256) == BAD
    assert _lib.jfa_paged_gather(c, 256, None, -2, 256, 256, 256) == BAD
    assert _lib.jfa_paged_gather(c, 256, None, 2, 256, 264, 256) == BAD
    assert _lib.jfa_paged_gather(c, 256, None, 0, None, None, 256) == 0
    # attend
    for args in ((None, 1024, 0.1, 0, 0, 256, 256), (256, 1028, 0.1, 0, 0, 256, 256),
                 (256, 1024, 0.0, 0, 0, 256, 256), (256, 1024, math.nan, 0, 0, 256, 256),
                 (256, 1024, 0.1, -1, 0, 256, 256), (256, 1024, 0.1, 0, -1, 256, 256),
                 (256, 1024, 0.1, 0, 0, 256, None), (256, 1024, 0.1, 0, 0, 64, 256)):
        assert _lib.jfa_paged_attend(c, *args) == BAD
    assert _lib.jfa_paged_attend(c, 256, 1024, 0.1, 0, 0, 256, 256, 258) == BAD    # lse
    # fork and move
    assert _lib.jfa_paged_fork(c, 256, 3, 256) == BAD
    assert _lib.jfa_paged_fork(c, None, 1, 256) == BAD
    assert _lib.jfa_paged_fork(c, None, 0, 256) == 0
    assert _lib.jfa_paged_move(c, 256, 11, None, 256) == BAD
    assert _lib.jfa_paged_move(c, None, 1, None, 256) == BAD
    assert _lib.jfa_paged_move(c, None, 0, None, 256) == 0


def _rope(**kw):
    d = dict(n_tokens=3, num_heads=4, num_kv_heads=2, rotary_dim=128, interleaved=0, positions64=0, eps=1e-6,
             amplitude=1.0, q=256, k=256, q_out=256, k_out=256, q_tok=512, q_head=128, k_tok=256, k_head=128,
             qo_tok=512, qo_head=128, ko_tok=256, ko_head=128, q_weight=0, k_weight=0, positions=256, freq=256)
    d.update(kw)
    return _lib.Rope(*d.values())


@pytest.mark.parametrize("bad", [
    dict(n_tokens=-1), dict(num_heads=-1), dict(rotary_dim=0), dict(rotary_dim=129), dict(rotary_dim=130),
    dict(eps=-1.0), dict(eps=math.nan), dict(amplitude=math.nan), dict(q=0), dict(q=264), dict(k_out=0),
    dict(q_tok=513), dict(k_head=4), dict(ko_tok=130), dict(q_weight=264), dict(positions=0),
    dict(positions=258), dict(positions=260, positions64=1), dict(freq=0), dict(freq=260)])
def test_rope_refusals(bad):
    assert _lib.jfa_qk_norm_rope(_rope(**bad)) == BAD


def test_rope_nothing_to_do():
    assert _lib.jfa_qk_norm_rope(_rope(n_tokens=0, q=0, k=0, positions=0)) == 0
    assert _lib.jfa_qk_norm_rope(_rope(num_heads=0, num_kv_heads=0, q=0, k=0)) == 0
    assert _lib.jfa_qk_norm_rope(_rope(num_heads=(1 << 20) + 1)) == UNSUPPORTED


def test_python_layer_refusals():
    for args in ((0, 4, 4), (257, 4, 4), (2, 0, 4), (2, 4, 0)):
        with pytest.raises(JfaError):
            jfa.PageTable(*args, device="cpu")
    t = jfa.PageTable(2, 4, 4, device="cpu")
    with pytest.raises(JfaError):
        jfa.PagedKVCache(t, 9, 2)
    cache = jfa.PagedKVCache(t, 8, 2)
    ws = jfa.PagedWorkspace(cache)
    rows = torch.zeros(2, 2, 128, dtype=torch.bfloat16)
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    cu = torch.zeros(3, dtype=torch.int32)
    # a workspace of fewer KV heads, and one of more
    other = jfa.PagedWorkspace(jfa.PagedKVCache(t, 8, 4))
    plan = jfa.RotaryPlan(device="cpu")
    refused = [
        lambda: jfa.paged_append(cache, rows.float(), rows, ws),
        lambda: jfa.paged_append(cache, rows[:, :1], rows, ws),
        lambda: jfa.paged_append(cache, rows, rows[:1], ws),
        lambda: jfa.paged_append(cache, rows, rows, ws, cu.long()),
        lambda: jfa.paged_append(cache, rows, rows, ws, cu[:2]),
        lambda: jfa.paged_append(cache, rows.transpose(1, 2).contiguous().transpose(1, 2), rows, ws),
        lambda: jfa.paged_gather(cache, cu, -1, ws),
        lambda: jfa.paged_gather(cache, cu, 2, ws, k_out=rows[:1]),
        lambda: jfa.paged_gather(cache, cu, 2, ws, start=cu),
        lambda: jfa.paged_attend(cache, q[:1], ws),
        lambda: jfa.paged_attend(cache, q[:, :4], ws),
        lambda: jfa.paged_attend(cache, q.transpose(0, 1).contiguous().transpose(0, 1), ws),
        lambda: jfa.paged_attend(cache, q, ws, scale=-1.0),
        lambda: jfa.paged_attend(cache, q, ws, window=-1),
        lambda: jfa.paged_attend(cache, q, ws, window=2**32 + 5),
        lambda: jfa.paged_attend(cache, q, ws, window=5, sinks=2**31),
        lambda: jfa.paged_attend(cache, q, other),
        lambda: jfa.qk_norm_rope(q, rows, cu[:2], plan, q_out=q[:1].expand(2, 8, 128)),
        lambda: jfa.qk_norm_rope(q, rows, cu[:2], plan, k_out=rows[:, :1].expand(2, 2, 128)),
        lambda: jfa.qk_norm_rope(q, rows, cu[:2], plan, q_out=q.as_strided((2, 8, 128), (256, 128, 1))),
        lambda: jfa.qk_norm_rope(q, rows, cu[:2], plan, q_out=q.as_strided((2, 8, 128), (128, 128, 1))),
        lambda: jfa.paged_attend(cache, q, ws, scale=math.inf),
        lambda: jfa.paged_attend(cache, q, ws, out=q.float()),
        lambda: jfa.paged_attend(cache, q, ws, lse=torch.zeros(2, 4)),
        lambda: jfa.paged_fork(cache, torch.zeros(3, 2, dtype=torch.int32), ws),
        lambda: jfa.paged_fork(cache, torch.zeros(1, 2), ws),
        lambda: jfa.paged_move(cache, torch.zeros(5, 2, dtype=torch.int32), ws),
        lambda: jfa.paged_move(cache, torch.zeros(1, 2, dtype=torch.int32), ws, cu),
        lambda: jfa.qk_norm_rope(q, rows[:1], cu[:2], plan),
        lambda: jfa.qk_norm_rope(q, rows, cu, plan),
        lambda: jfa.qk_norm_rope(q, rows, cu[:2].float(), plan),
        lambda: jfa.qk_norm_rope(q, rows, cu[:2], plan, q_weight=torch.zeros(64, dtype=torch.bfloat16)),
        lambda: jfa.qk_norm_rope(q, rows, cu[:2], plan, q_out=rows),
        lambda: jfa.paged_decode_step(cache, q[:1], rows[:1], rows[:1], cu[:1], plan, ws),
    ]
    for i, call in enumerate(refused):
        with pytest.raises(JfaError) as e:
            call()
        assert e.value.status == BAD, i


def test_refused_decode_step_launches_nothing(monkeypatch):
    """Whatever a decode step refuses, it refuses before its first launch: the
    append cannot be taken back."""
    from bit_kv_cache_jfa_b200 import paged
    launched = []
    monkeypatch.setattr(paged, "_run", lambda where, *a: launched.append(where))
    t = jfa.PageTable(2, 4, 4, device="cpu")
    t.grow([64, 3])
    cache = jfa.PagedKVCache(t, 8, 2)
    ws = jfa.PagedWorkspace(cache)
    t.grow(1)
    q, k = torch.zeros(2, 8, 128, dtype=torch.bfloat16), torch.zeros(2, 2, 128, dtype=torch.bfloat16)
    plan = jfa.RotaryPlan(device="cpu")
    pos = t.seq_lens - 1
    flat = torch.zeros(2 * 8 * 128 + 8, dtype=torch.bfloat16)
    at = 4 if flat.data_ptr() % 16 == 0 else 0
    for kw in (dict(out=q.float()), dict(out=q[:1]), dict(out=flat[at:at + 2048].view(2, 8, 128)),
               dict(lse=torch.zeros(2, 4)), dict(lse=torch.zeros(2, 8).double()), dict(window=-1),
               dict(window=2**31), dict(window=4, sinks=-1), dict(sinks=2**31), dict(window=2.5), dict(scale=0.0),
               dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(scale=1e-60), dict(scale=1e60)):
        with pytest.raises((JfaError, TypeError)):
            jfa.paged_decode_step(cache, q, k, k, pos, plan, ws, **kw)
        assert "jfa_paged_append" not in launched, kw
    with pytest.raises(JfaError):
        jfa.paged_decode_step(cache, q[:, :4], k, k, pos, plan, ws)
    with pytest.raises(JfaError):
        jfa.paged_decode_step(cache, q, k, k[:, :1], pos, plan, ws)
    assert "jfa_paged_append" not in launched
    launched.clear()
    jfa.paged_decode_step(cache, q, k, k, pos, plan, ws, scale=0.1, window=5, sinks=1)
    assert launched == ["jfa_qk_norm_rope", "jfa_paged_append", "jfa_paged_attend"]


def test_outputs_overlap_exactly_when_two_rows_share_an_element():
    from bit_kv_cache_jfa_b200 import paged
    rng = random.Random(11)
    seen = [0, 0]
    for _ in range(3000):
        n0, n1 = rng.randint(1, 6), rng.randint(1, 6)
        s0, s1 = (rng.choice([8 * rng.randint(0, 130), 128 * rng.randint(0, 8)]) for _ in range(2))
        at = sorted(i * s0 + j * s1 for i in range(n0) for j in range(n1))
        want = any(b - a < 128 for a, b in zip(at, at[1:]))
        assert paged._overlap(s0, n0, s1, n1) == want, (s0, n0, s1, n1)
        seen[want] += 1
    assert min(seen) > 300


def test_outputs_between_other_rows_are_taken(monkeypatch):
    """Every other head of an odd number, heads before tokens, and rows that lie
    between one another without sharing a byte."""
    from bit_kv_cache_jfa_b200 import paged
    monkeypatch.setattr(paged, "_run", lambda *a: None)
    plan = jfa.RotaryPlan(device="cpu")
    wide = torch.zeros(6, 7, 128, dtype=torch.bfloat16)
    pos = torch.zeros(6, dtype=torch.int32)
    k = torch.zeros(6, 1, 128, dtype=torch.bfloat16)
    for out in (wide[:, ::2], wide.view(7, 6, 128).transpose(0, 1)[:, :4], wide[:, 1:5]):
        got, _ = jfa.qk_norm_rope(out, k, pos, plan, q_out=out)
        assert got is out
    between = wide.as_strided((2, 4, 128), (384, 256, 1))
    assert jfa.qk_norm_rope(between, k[:2], pos[:2], plan, q_out=between)[0] is between


def test_calls_on_host_tensors_are_refused():
    """The book of a table without a device works; the calls name what is missing."""
    t = jfa.PageTable(2, 4, 4, device="cpu")
    cu = t.grow([64, 3])
    cache = jfa.PagedKVCache(t, 8, 2)
    ws = jfa.PagedWorkspace(cache)
    rows, q = torch.zeros(67, 2, 128, dtype=torch.bfloat16), torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    plan = jfa.RotaryPlan(device="cpu")
    pos = torch.zeros(2, dtype=torch.int32)
    for call in (lambda **kw: jfa.paged_append(cache, rows, rows, ws, cu, **kw),
                 lambda **kw: jfa.paged_gather(cache, cu, 67, ws, **kw),
                 lambda **kw: jfa.paged_attend(cache, q, ws, **kw),
                 lambda **kw: jfa.paged_fork(cache, torch.zeros(1, 2, dtype=torch.int32), ws, **kw),
                 lambda **kw: jfa.paged_move(cache, torch.zeros(1, 2, dtype=torch.int32), ws, **kw),
                 lambda **kw: jfa.qk_norm_rope(q, rows[:2], pos, plan, **kw),
                 lambda **kw: jfa.paged_decode_step(cache, q, rows[:2], rows[:2], pos, plan, ws, **kw),
                 lambda **kw: ws.error_flag(cache, **kw), lambda **kw: ws.clear_error(cache, **kw)):
        for kw in ({}, dict(stream=256)):
            with pytest.raises(JfaError) as e:
                call(**kw)
            assert e.value.status == BAD and "CUDA" in str(e.value)


def test_counts_past_32_bits_are_refused(monkeypatch):
    """They would wrap: an append of 2^32 rows (of one row's memory) did nothing."""
    from bit_kv_cache_jfa_b200 import paged
    monkeypatch.setattr(paged, "_run", lambda *a: None)
    t = jfa.PageTable(2, 4, 4, device="cpu")
    cache = jfa.PagedKVCache(t, 8, 2)
    ws = jfa.PagedWorkspace(cache)
    cu = torch.zeros(3, dtype=torch.int32)
    plan = jfa.RotaryPlan(device="cpu")
    row, pos = torch.zeros(1, 2, 128, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
    some = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    for n in (2**31, 2**32, 2**32 + 4):
        many = row.expand(n, 2, 128)
        for call in (lambda: jfa.paged_append(cache, many, many, ws, cu), lambda: jfa.paged_append(cache, many, many, ws),
                     lambda: jfa.paged_gather(cache, cu, n, ws, k_out=some, v_out=some),
                     lambda: jfa.qk_norm_rope(many, many, pos.expand(n), plan, q_out=some, k_out=some),
                     lambda: jfa.PageTable(2, n, 4, device="cpu"), lambda: jfa.PageTable(2, 4, n, device="cpu"),
                     lambda: jfa.PagedKVCache(t, n, 2), lambda: jfa.PagedKVCache(t, n, n)):
            with pytest.raises(JfaError) as e:
                call()
            assert e.value.status == BAD
    jfa.paged_append(cache, row.expand(2**31 - 1, 2, 128), row.expand(2**31 - 1, 2, 128), ws, cu)


@pytest.mark.parametrize("kw", [
    dict(scaling="linear", factor=1e-320), dict(scaling="linear", factor=1e-300), dict(base=math.nan),
    dict(scaling="yarn", original=math.inf, factor=2.0), dict(scaling="yarn", original=8192, base=math.inf),
    dict(scaling="llama3", original=8192, low_freq_factor=-math.inf),
    dict(scaling="yarn", original=8192, beta_fast=math.inf), dict(scaling="llama3", original=math.nan),
    dict(amplitude=1e39), dict(amplitude=-1e300), dict(amplitude=math.nan)], ids=str)
def test_rotary_plan_refuses_what_no_frequency_comes_of(kw):
    with pytest.raises(JfaError) as e:
        jfa.RotaryPlan(device="cpu", **kw)
    assert e.value.status == BAD


def test_rotary_plan_of_extreme_factors():
    """Frequencies of many turns a position are whole numbers of 2^-64 turns as well."""
    plan = jfa.RotaryPlan(4, base=10000.0, scaling="linear", factor=1e-200, device="cpu")
    assert plan.frequencies[0] == 1 / 1e-200
    assert jfa.RotaryPlan(4, scaling="linear", factor=1e300, device="cpu").freq.tolist() == [0, 0]


def test_read_back_into_one_place_is_refused(monkeypatch):
    from bit_kv_cache_jfa_b200 import paged
    monkeypatch.setattr(paged, "_run", lambda *a: None)
    t = jfa.PageTable(2, 4, 4, device="cpu")
    cache = jfa.PagedKVCache(t, 8, 2)
    ws = jfa.PagedWorkspace(cache)
    cu = torch.zeros(3, dtype=torch.int32)
    both = torch.zeros(10, 2, 128, dtype=torch.bfloat16)
    for k, v in ((both[:5], both[:5]), (both[:5], both[4:9]), (both[4:9], both[:5])):
        with pytest.raises(JfaError) as e:
            jfa.paged_gather(cache, cu, 5, ws, k_out=k, v_out=v)
        assert e.value.status == BAD
    jfa.paged_gather(cache, cu, 5, ws, k_out=both[:5], v_out=both[5:])
    jfa.paged_gather(cache, cu, 5, ws, k_out=both[5:], v_out=both[:5])
    jfa.paged_gather(cache, cu, 0, ws)
