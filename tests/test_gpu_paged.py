"""GPU parity of the paged 4-bit cache: append, read-back, attention (whole and
windowed), forks, page moves, and a run of them together, against 64-bit
references built from the oracle's quantization."""
import math

import numpy as np
import pytest
import torch

import bit_kv_cache_jfa_b200 as jfa
import oracle.jfa_oracle as O
from bit_kv_cache_jfa_b200 import _lib

pytestmark = pytest.mark.gpu

D = 128
BF16 = 2.0**-8     # half a step of bf16, relative to the value


def split(n):
    return 64 * ((n - 1) // 64) if n > 0 else 0


def gen(seed):
    return torch.Generator().manual_seed(seed)


def make_rows(n, hkv, seed, outliers=4, k_scale=1.0, v_scale=1.0):
    """bf16 keys and values [n, hkv, 128] on the CPU; some key channels ten times as large."""
    g = gen(seed)
    big = torch.ones(D)
    big[torch.randperm(D, generator=g)[:outliers]] = 10.0
    k = (torch.randn(n, hkv, D, generator=g) * big * k_scale).bfloat16()
    v = (torch.randn(n, hkv, D, generator=g) * v_scale).bfloat16()
    return k, v


class Ref:
    """A sequence's cache in 64 bits: packed codes, scales and zero points, exact tail."""

    def __init__(self, k, v):
        kk, vv = (x.double().numpy().transpose(1, 0, 2)[None] for x in (k, v))
        self.n = k.shape[0]
        self.c = O.pack_cache(kk, vv, self.n, 4, 4)
        self.nq = self.c.n_quant
        self.k = np.concatenate((self.c.k_hat(), self.c.tail_k), 2)[0]   # [hkv][n][128]
        self.v = np.concatenate((self.c.v_hat(), self.c.tail_v), 2)[0]

    def attend(self, q, scale, window=0, sinks=0):
        """(out, lse, bound, lse_bound): outputs of q [H][128] and bounds of
        what the kernel's roundings may do to them."""
        hkv, h = self.k.shape[0], q.shape[0]
        t = np.arange(self.n)
        seen = (t >= self.n - window) | (t < sinks) if window else t >= 0
        out, bound, lse, lse_bound = np.zeros((h, D)), np.zeros((h, D)), np.full(h, -np.inf), np.zeros(h)
        if self.n == 0:
            return out, lse, bound, lse_bound
        for i in range(h):
            j = i // (h // hkv)
            k, v = self.k[j][seen], self.v[j][seen]
            x = scale * (k @ q[i])
            m = x.max()
            p = np.exp(x - m)
            lse[i] = m + np.log(p.sum())
            p /= p.sum()
            out[i] = p @ v
            # Errors of a logit: the fp32 sums (256 products and additions of
            # terms |q_c k_c| and of the zero points', 2^-24 each) and, for a
            # packed token, fp16(q_c s_c): 2^-11 |q_c s_c| |k' - 7.5|, plus the
            # remainder's own rounding, 2^-22 of 7.5 |q_c s_c|, and what falls
            # under fp16's smallest step 2^-25 of q's largest power of two
            # (times 8 and 15).
            a = np.abs(q[i])
            size = np.abs(k) @ a
            e = np.zeros(self.n)
            if self.nq:
                s = np.repeat(self.c.k_scale[0, j].astype(float), 64, 0)
                z = np.repeat(np.abs(self.c.k_zero[0, j].astype(float)), 64, 0)
                code = self.c.k_codes[0, j].astype(float)
                e[:self.nq] = 2.0**-11 * ((np.abs(code - 7.5) * s) @ a) + 2.0**-22 * 7.5 * (s @ a) \
                    + 2.0**-16 * ((s * code + z) @ a) + 2.0**-22 * 15 * 128 * a.max()
            e = scale * (e[seen] + 2.0**-16 * size) + 2.0**-20 * (1 + np.abs(x))
            # Errors of a weight: the logit's, fp16's rounding of the weight
            # and of its product with the scale.  The largest weight lies
            # between 2^(sh - 5) and 2^sh, sh = 15 and less where value scales
            # are 2 and more; 2^-25 is lost at the bottom of fp16, of a weight
            # and of its product with a scale (times the code's 15).
            w = 2.0**-11
            top = 0 if not self.nq else np.floor(np.log2(max(float(self.c.v_scale[0, j].max()), 1.0)))
            lost = 2.0**-(25 + 15 - top - 5) * p.max()
            ce = np.abs(v)
            if self.nq:
                vs = np.repeat(self.c.v_scale[0, j].astype(float), 32, -1) * self.c.v_codes[0, j]
                vz = np.repeat(np.abs(self.c.v_zero[0, j].astype(float)), 32, -1)
                full = np.abs(self.v[j]).copy()
                full[:self.nq] = vs + vz
                ce = full[seen]
            bound[i] = p @ ((np.expm1(e) + 2 * w + 2.0**-16)[:, None] * (ce + np.abs(out[i]))) \
                + lost * (15 + np.abs(v) + np.abs(out[i])).sum(0) + (BF16 + 2.0**-16) * np.abs(out[i]) + 1e-38
            lse_bound[i] = -np.log1p(-min(p @ (np.expm1(e) + w) + lost * len(p), 0.9)) + 2.0**-20 * (1 + abs(lse[i]))
        return out, lse, bound, lse_bound


def make(lens, heads, hkv, seed=0, spare=3, **kw):
    """A filled cache: (table, cache, ws, refs, rows)."""
    need = sum(split(n) // 64 for n in lens)
    table = jfa.PageTable(len(lens), need + spare, max(1, max(split(n) // 64 for n in lens) + 2))
    rng = np.random.default_rng(seed)
    cache = jfa.PagedKVCache(table, heads, hkv)
    ws = jfa.PagedWorkspace(cache)
    k, v = make_rows(sum(lens), hkv, seed, **kw)
    cu = table.grow(lens)
    # scatter the pages over the pool: what grow gave, permuted
    perm = rng.permutation(table.n_pages)
    table.rows = [[int(perm[p]) for p in r] for r in table.rows]
    refs = [0] * table.n_pages
    for r in table.rows:
        for p in r:
            refs[p] += 1
    table._refs = refs
    table._free = sorted(p for p in range(table.n_pages) if refs[p] == 0)
    for b, r in enumerate(table.rows):
        if r:
            table.table[b, :len(r)] = torch.tensor(r, dtype=torch.int32)
    jfa.paged_append(cache, k.cuda(), v.cuda(), ws, cu)
    at = np.concatenate(([0], np.cumsum(lens)))
    rows = [(k[a:z], v[a:z]) for a, z in zip(at[:-1], at[1:])]
    return table, cache, ws, rows


def swizzled(x):
    """Tail slots [..., slots, 128] with chunk c of slot t at c ^ (t % 8)."""
    n = x.shape[-2]
    at = torch.arange(16) ^ (torch.arange(n) % 8)[:, None]
    y = x.reshape(*x.shape[:-1], 16, 8)
    return y.gather(-2, at[..., None].expand(y.shape)).reshape(x.shape)


def check_cache(table, cache, rows):
    """Records and tails of every sequence, bit for bit."""
    tk, tv = cache.tail_k.cpu(), cache.tail_v.cpu()
    tab = table.table.cpu()
    for b, (k, v) in enumerate(rows):
        n = k.shape[0]
        if n == 0:
            continue
        ref = Ref(k, v).c
        nq = ref.n_quant
        for h in range(cache.num_kv_heads):
            for g in range(nq // 64):
                kc, ks, kz, vc, vs, vz = _lib.jfa_unpack_record(4, 4, cache.record(int(tab[b, g]), h))
                t = slice(64 * g, 64 * g + 64)
                assert np.array_equal(ks, ref.k_scale[0, h, g].view(np.uint16)), (b, h, g)
                assert np.array_equal(kz, ref.k_zero[0, h, g].view(np.uint16)), (b, h, g)
                assert np.array_equal(kc, ref.k_codes[0, h, t]), (b, h, g)
                assert np.array_equal(vs, ref.v_scale[0, h, t].view(np.uint16)), (b, h, g)
                assert np.array_equal(vz, ref.v_zero[0, h, t].view(np.uint16)), (b, h, g)
                assert np.array_equal(vc, ref.v_codes[0, h, t]), (b, h, g)
        assert torch.equal(swizzled(tk[b])[:, :n - nq], k[nq:].transpose(0, 1))
        assert torch.equal(swizzled(tv[b])[:, :n - nq], v[nq:].transpose(0, 1))


def check_attend(cache, ws, rows, q, window=0, sinks=0, scale=None, out=None, rms=None):
    s = 1 / math.sqrt(D) if scale is None else scale
    lse = torch.full((len(rows), cache.num_heads), 7.0, device="cuda")
    out = jfa.paged_attend(cache, q.cuda(), ws, scale=scale, window=window, sinks=sinks, lse=lse, out=out)
    torch.cuda.synchronize()
    assert ws.error_flag(cache) == 0
    got, lse = out.cpu().double().numpy(), lse.cpu().double().numpy()
    qd = q.double().numpy()
    want = np.zeros_like(got)
    for b, (k, v) in enumerate(rows):
        o, l, bound, l_bound = Ref(k, v).attend(qd[b], s, window, sinks)
        want[b] = o
        assert np.isfinite(got[b]).all(), b
        err = np.abs(got[b] - o)
        assert (err <= bound).all(), (b, k.shape[0], (err / np.maximum(bound, 1e-300)).max(), err.max())
        if k.shape[0] == 0:
            assert np.all(lse[b] == -np.inf)
        else:
            assert (np.abs(lse[b] - l) <= l_bound).all(), (b, lse[b] - l, l_bound)
    if rms is not None and np.linalg.norm(want):
        assert np.linalg.norm(got - want) <= rms * np.linalg.norm(want)
    return out


def rand_q(b, h, seed, scale=1.0):
    return (torch.randn(b, h, D, generator=gen(1000 + seed)) * scale).bfloat16()


# ---------------------------------------------------------------------------
# append and read-back
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("hkv", [1, 2, 8])
def test_append_prompts(hkv):
    lens = [1, 63, 64, 65, 0, 128, 129, 300, 193]
    table, cache, ws, rows = make(lens, hkv, hkv, seed=hkv)
    torch.cuda.synchronize()
    assert ws.error_flag(cache) == 0
    check_cache(table, cache, rows)


@pytest.mark.parametrize("chunks", [[1] * 70, [63, 1, 1, 64, 2], [64, 64, 64], [65, 65, 200], [300, 7, 57, 1]])
def test_append_in_chunks_equals_at_once(chunks):
    """Two sequences that grow by the chunks (one begins 31 tokens later), strided rows."""
    hkv, total = 2, sum(chunks) + 31
    k, v = make_rows(2 * total, hkv, seed=len(chunks))
    both = torch.stack((k, v), 2).cuda()              # [rows][hkv][2][128]: strides of their own
    table = jfa.PageTable(2, 20, 10)
    cache = jfa.PagedKVCache(table, 4, hkv)
    ws = jfa.PagedWorkspace(cache)
    done = [0, 0]
    for first, counts in [(True, [31, 0])] + [(False, [c, c]) for c in chunks]:
        cu = table.grow(counts)
        pick = torch.cat([torch.arange(total * b + done[b], total * b + done[b] + c) for b, c in enumerate(counts)])
        x = both[pick.cuda()]
        jfa.paged_append(cache, x[:, :, 0], x[:, :, 1], ws, cu)
        done = [a + c for a, c in zip(done, counts)]
    torch.cuda.synchronize()
    assert ws.error_flag(cache) == 0
    check_cache(table, cache, [(k[total * b:total * b + n], v[total * b:total * b + n]) for b, n in enumerate(done)])


def test_uniform_append_leaves_idle_rows():
    lens = [64, 0, 100, 127]
    table, cache, ws, rows = make(lens, 4, 2, seed=9)
    before = cache.tail_k[1].clone()
    for step in range(3):
        table.grow(1)
        k, v = make_rows(4, 2, 50 + step)
        jfa.paged_append(cache, k.cuda(), v.cuda(), ws)
        rows = [(torch.cat((a, k[b:b + 1])), torch.cat((c, v[b:b + 1]))) if lens[b] else (a, c)
                for b, (a, c) in enumerate(rows)]
    torch.cuda.synchronize()
    assert ws.error_flag(cache) == 0
    check_cache(table, cache, rows)
    assert torch.equal(cache.tail_k[1], before)


@pytest.mark.parametrize("ranges", [False, True])
def test_append_padded_in_front(ranges):
    """Rows of one length for every sequence, the shorter ones padded in front."""
    lens, wide, hkv = [130, 1, 0, 64, 200], 200, 2
    table = jfa.PageTable(5, 12, 5)
    cache = jfa.PagedKVCache(table, 2, hkv)
    ws = jfa.PagedWorkspace(cache)
    k, v = make_rows(5 * wide, hkv, 14)
    rows = [(k[wide * (b + 1) - n:wide * (b + 1)], v[wide * (b + 1) - n:wide * (b + 1)]) for b, n in enumerate(lens)]
    table.grow(lens)
    cu = torch.arange(6, dtype=torch.int32, device="cuda") * wide if ranges else None
    jfa.paged_append(cache, k.cuda(), v.cuda(), ws, cu)
    torch.cuda.synchronize()
    assert ws.error_flag(cache) == 0
    check_cache(table, cache, rows)


def test_append_ties_and_constant_groups():
    """Rows whose quotients lie on borders between codes, constant groups
    (scale 0), the type's smallest steps."""
    n, hkv = 129, 1
    g = gen(3)
    k = torch.randint(0, 31, (n, hkv, D), generator=g).float() / 2   # halves over a range of 15
    k[0], k[1] = 0.0, 15.0
    v = torch.randint(0, 31, (n, hkv, D), generator=g).float() / 2
    v[..., 0::32], v[..., 1::32] = 0.0, 15.0
    v[5], v[6] = 1.5, 0.0
    k[:, 0, 7] = -2.25
    k[:, 0, 8] = 0.0
    k[:, 0, 9] *= 2.0**-24
    k[:, 0, 10] *= 2.0**-40
    v[7] *= 2.0**-30
    k, v = k.bfloat16(), v.bfloat16()
    table = jfa.PageTable(1, 4, 4)
    cache = jfa.PagedKVCache(table, 1, 1)
    ws = jfa.PagedWorkspace(cache)
    jfa.paged_append(cache, k.cuda(), v.cuda(), ws, table.grow([n]))
    torch.cuda.synchronize()
    assert ws.error_flag(cache) == 0
    check_cache(table, cache, [(k, v)])


def test_append_flags_values_past_fp16():
    table = jfa.PageTable(2, 4, 2)
    cache = jfa.PagedKVCache(table, 1, 1)
    ws = jfa.PagedWorkspace(cache)
    k, v = make_rows(130, 1, 4)
    k[3, 0, 5] = 1e30
    jfa.paged_append(cache, k.cuda(), v.cuda(), ws, table.grow([65, 65]))
    assert ws.error_flag(cache) == _lib.DEVERR_NONFINITE_QUANT
    ws.clear_error(cache)
    assert ws.error_flag(cache) == 0


@pytest.mark.parametrize("lens,start,count", [
    ([1, 64, 65, 200, 0], None, [1, 64, 65, 200, 0]),
    ([300, 129, 64], [0, 128, 63], [300, 1, 1]),
    ([300, 129, 64], [63, 64, 0], [2, 65, 0]),
    ([500, 191], [257, 190], [100, 1])])
def test_gather(lens, start, count):
    table, cache, ws, rows = make(lens, 6, 3, seed=sum(lens))
    first = 5                                          # rows before and behind belong to nobody
    cu = torch.tensor(np.concatenate(([first], first + np.cumsum(count))), dtype=torch.int32).cuda()
    total = first + sum(count) + 9
    outs = [torch.full((total, 3, D), 77.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    st = None if start is None else torch.tensor(start, dtype=torch.int32).cuda()
    got = jfa.paged_gather(cache, cu, total, ws, start=st, k_out=outs[0], v_out=outs[1])
    torch.cuda.synchronize()
    assert ws.error_flag(cache) == 0 and got[0] is outs[0]
    at = first
    for b, c in enumerate(count):
        s = start[b] if start else 0
        ref = Ref(*rows[b])
        for x, want, orig in ((outs[0], ref.k, rows[b][0]), (outs[1], ref.v, rows[b][1])):
            x = x[at:at + c].cpu()
            w = want[:, s:s + c].transpose(1, 0, 2)
            # one fp32 rounding of code * scale + zero, one to bf16
            assert (np.abs(x.double().numpy() - w) <= (BF16 + 2.0**-23) * np.abs(w) + 2.0**-133).all()
            tail = max(ref.nq - s, 0)
            assert torch.equal(x[tail:], orig[s + tail:s + c])
        at += c
    for x in outs:
        assert (x[:first] == 77).all() and (x[at:] == 77).all()


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
# Relative error over all outputs, root mean square, at unit normal data with
# four outlier channels: bf16's rounding, at most 2^-8 and uniform, 2.3e-3;
# fp16(q s), 2^-11 / sqrt(3) of q s (k' - 7.5), over 128 channels 8e-4 of a
# logit; the weights' two roundings 4e-4: 2.5e-3 together.
RMS = 4e-3


@pytest.mark.parametrize("heads,hkv", [(1, 1), (2, 1), (3, 1), (8, 1), (10, 2), (32, 8), (14, 2)])
def test_attend_ragged(heads, hkv):
    lens = [1, 2, 0, 15, 16, 17, 63, 64, 65, 66, 128, 129, 0, 200, 577, 1000]
    table, cache, ws, rows = make(lens, heads, hkv, seed=heads)
    check_attend(cache, ws, rows, rand_q(len(lens), heads, heads), rms=RMS)


@pytest.mark.parametrize("lens", [[1], [64], [65], [300], [5000], [20001], [9, 4999, 1, 70, 1, 1, 12001]])
def test_attend_lengths(lens):
    table, cache, ws, rows = make(lens, 8, 2, seed=len(lens))
    check_attend(cache, ws, rows, rand_q(len(lens), 8, 5), rms=RMS)


def test_attend_largest_batch():
    lens = [(37 * b) % 150 for b in range(256)]
    table, cache, ws, rows = make(lens, 4, 2, seed=8)
    check_attend(cache, ws, rows, rand_q(256, 4, 8), rms=RMS)


@pytest.mark.parametrize("window", [1, 15, 63, 64, 65, 100, 128, 577, 2000])
@pytest.mark.parametrize("sinks", [0, 1, 4, 64, 70, 128, 700])
def test_attend_window_and_sinks(window, sinks):
    lens = [1, 0, 64, 65, 130, 192, 193, 600, 1001]
    table, cache, ws, rows = make(lens, 4, 2, seed=window + sinks)
    check_attend(cache, ws, rows, rand_q(len(lens), 4, window), window=window, sinks=sinks)


def test_attend_strided_query_scale_and_given_out():
    lens = [100, 0, 333]
    table, cache, ws, rows = make(lens, 8, 4, seed=6)
    wide = torch.zeros(3, 14, D, dtype=torch.bfloat16)
    wide[:, 3:11] = rand_q(3, 8, 6)
    q = wide.cuda()[:, 3:11]
    out = torch.full((3, 8, D), 9.0, dtype=torch.bfloat16, device="cuda")
    a = jfa.paged_attend(cache, q, ws, scale=0.05, out=out)
    assert a is out
    b = check_attend(cache, ws, rows, wide[:, 3:11], scale=0.05)
    assert torch.equal(a, b)


@pytest.mark.parametrize("k_scale,v_scale,q_scale", [
    (1.0, 1e-4, 1.0), (1.0, 300.0, 1.0), (1e-3, 1.0, 30.0), (300.0, 1.0, 1e-3), (1.0, 1e-6, 1.0),
    (1.0, 8000.0, 1.0), (3.0, 1.0, 4.0), (1.0, 1.0, 1e-20), (1000.0, 1.0, 2e-4)])
def test_attend_value_ranges(k_scale, v_scale, q_scale):
    lens = [700, 64, 1]
    table, cache, ws, rows = make(lens, 4, 1, seed=11, k_scale=k_scale, v_scale=v_scale)
    check_attend(cache, ws, rows, rand_q(3, 4, 11, q_scale))


def test_attend_values_of_unlike_groups():
    """Value scales that grow by powers of two along a sequence: the weights'
    reference follows."""
    n = 1500
    table = jfa.PageTable(2, 60, 30)
    cache = jfa.PagedKVCache(table, 2, 1)
    ws = jfa.PagedWorkspace(cache)
    k, v = make_rows(2 * n, 1, 21)
    ramp = torch.exp2(torch.arange(n) // 100 - 3.0)[:, None, None]
    v[:n] = (v[:n].float() * ramp).bfloat16()
    v[n:] = (v[n:].float() * ramp.flip(0)).bfloat16()
    jfa.paged_append(cache, k.cuda(), v.cuda(), ws, table.grow([n, n]))
    check_attend(cache, ws, [(k[:n], v[:n]), (k[n:], v[n:])], rand_q(2, 2, 21))


def test_attend_one_token_above_many_far_below():
    """One weight of 1 and 20000 of about 2e-6: together they count."""
    n = 20001
    k, v = make_rows(n, 1, 31, outliers=0)
    k *= 0.02
    v = (v.float() * 0.01 + 0.05).bfloat16()
    q = torch.ones(1, 1, D).bfloat16()
    k[n // 2] = 13.2 * math.sqrt(D) / D
    table = jfa.PageTable(1, 320, 320)
    cache = jfa.PagedKVCache(table, 1, 1)
    ws = jfa.PagedWorkspace(cache)
    v[n // 2] = -0.1
    jfa.paged_append(cache, k.cuda(), v.cuda(), ws, table.grow([n]))
    check_attend(cache, ws, [(k, v)], q)


@pytest.mark.parametrize("fill", [math.nan, math.inf, -math.inf, torch.finfo(torch.bfloat16).min])
def test_attend_what_is_masked_does_not_matter(fill):
    """Slots past the length, groups outside the window, free pages and table
    entries past the length hold anything."""
    lens = [200, 333, 70, 64, 0]
    table, cache, ws, rows = make(lens, 4, 2, seed=13)
    q = rand_q(5, 4, 13)
    window, sinks = 100, 5
    want = check_attend(cache, ws, rows, q, window=window, sinks=sinks).clone()
    whole = check_attend(cache, ws, rows, q).clone()
    for b, n in enumerate(lens):
        cache.tail_k[b, :, n - split(n):] = fill
        cache.tail_v[b, :, n - split(n):] = fill
        table.table[b, split(n) // 64:] = 2**31 - 1
    free = [p for p in range(table.n_pages) if not table._refs[p]]
    cache.pages[free] = 0xFF                           # NaN scales
    assert torch.equal(whole, check_attend(cache, ws, rows, q))
    # groups that neither the window nor the first tokens touch
    tab = table.table.cpu()
    for b, n in enumerate(lens):
        for g in range(split(n) // 64):
            if 64 * (g + 1) <= n - window and 64 * g >= sinks:
                cache.pages[int(tab[b, g])] = 0xFF
                table.table[b, g] = -5
    # in the first group and the window's first: values of the tokens in between
    for b, n in enumerate(lens):
        for g in range(split(n) // 64):
            for t in range(64):
                if sinks <= 64 * g + t < n - window and not (64 * (g + 1) <= n - window and 64 * g >= sinks):
                    kk, tig, hi, e = t // 16, t % 8 // 2, t % 16 // 8, t % 2
                    for j in range(4):
                        at = 4608 + kk * 128 + tig * 32 + j * 8 + hi * 4 + 2 * e
                        for part in (at, at + 512):
                            cache.pages[int(tab[b, g]), :, part:part + 2] = 0xFF
    got = jfa.paged_attend(cache, q.cuda(), ws, window=window, sinks=sinks)
    torch.cuda.synchronize()
    assert ws.error_flag(cache) == 0
    # The logits are the same; a NaN scale in a masked place may lower the
    # weights' reference, which changes their two fp16 roundings (2^-11 each,
    # on both sides, of values of 4 and less) and then bf16's.
    a, b = got.double().cpu(), want.double().cpu()
    assert torch.isfinite(a).all()
    assert ((a - b).abs() <= 2 * BF16 * b.abs() + 4 * 2.0**-11 * 4).all()


def test_attend_is_reproducible():
    lens = [3000, 100, 0, 9000, 64]
    table, cache, ws, rows = make(lens, 8, 2, seed=17)
    q = rand_q(5, 8, 17).cuda()
    a = jfa.paged_attend(cache, q, ws).clone()
    for _ in range(5):
        assert torch.equal(a, jfa.paged_attend(cache, q, ws))


def test_attend_nonfinite_query_and_keys_show():
    """An infinite key among the visible tokens gives NaN for its sequence, none for others."""
    lens = [100, 100]
    table, cache, ws, rows = make(lens, 4, 2, seed=19)
    cache.tail_k[0, 0, 3] = math.inf
    out = jfa.paged_attend(cache, rand_q(2, 4, 19).cuda(), ws)
    torch.cuda.synchronize()
    assert torch.isnan(out[0, :2]).any()
    assert torch.isfinite(out[1]).all() and torch.isfinite(out[0, 2:]).all()


# ---------------------------------------------------------------------------
# pages: forks, moves
# ---------------------------------------------------------------------------
def test_fork_shares_then_diverges():
    lens = [200, 65, 0, 64, 30]
    table, cache, ws, rows = make(lens, 4, 2, seed=23, spare=12)
    pairs = table.fork([(0, 2), (1, 3)])
    jfa.paged_fork(cache, pairs, ws)
    rows[2], rows[3] = rows[0], rows[1]
    torch.cuda.synchronize()
    assert ws.error_flag(cache) == 0
    assert table.seq_lens.tolist() == table.lens == [200, 65, 200, 65, 30]
    check_cache(table, cache, rows)
    for step in range(3):                              # groups complete at different pages
        k, v = make_rows(5 * 40, 2, 60 + step)
        cu = table.grow([40] * 5)
        jfa.paged_append(cache, k.cuda(), v.cuda(), ws, cu)
        rows = [(torch.cat((a, k[40 * b:40 * b + 40])), torch.cat((c, v[40 * b:40 * b + 40])))
                for b, (a, c) in enumerate(rows)]
    torch.cuda.synchronize()
    assert ws.error_flag(cache) == 0
    check_cache(table, cache, rows)
    check_attend(cache, ws, rows, rand_q(5, 4, 23), rms=RMS)


@pytest.mark.parametrize("hkv", [1, 8])
def test_compact_keeps_every_row(hkv):
    lens = [500, 300, 0, 700, 64, 129]
    table, cache, ws, rows = make(lens, hkv, hkv, seed=29, spare=20)
    other = jfa.PagedKVCache(table, hkv, hkv)          # another layer on the same table
    ws2 = jfa.PagedWorkspace(other)
    other.pages.random_(0, 256)
    old = other.pages.clone()
    table.free([1])
    rows[1] = (rows[1][0][:0], rows[1][1][:0])
    before = [list(r) for r in table.rows]
    moves, remap = table.compact()
    assert moves.shape[0] > 0
    jfa.paged_move(other, moves, ws2)
    jfa.paged_move(cache, moves, ws, remap)
    torch.cuda.synchronize()
    assert ws.error_flag(cache) == 0 and ws2.error_flag(other) == 0
    check_cache(table, cache, rows)
    for b, row in enumerate(table.rows):
        assert table.table[b, :len(row)].tolist() == row
        assert torch.equal(other.pages[row], old[before[b]])
    check_attend(cache, ws, rows, rand_q(6, hkv, 29), rms=RMS)


def test_empty_page_calls():
    table, cache, ws, rows = make([100, 0], 2, 1, seed=2)
    none = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    jfa.paged_fork(cache, none, ws)
    jfa.paged_move(cache, none, ws)
    _, remap = table.compact()
    empty = torch.zeros(0, 1, D, dtype=torch.bfloat16, device="cuda")
    jfa.paged_append(cache, empty, empty, ws)
    k, v = jfa.paged_gather(cache, torch.zeros(3, dtype=torch.int32, device="cuda"), 0, ws)
    assert k.shape == (0, 1, D) and ws.error_flag(cache) == 0


def test_pages_past_32_bit_offsets():
    """A pool of 4.7 GB whose last pages are in use: append, read-back,
    attention, move."""
    hkv, n = 8, 400
    table = jfa.PageTable(2, 60000, 16)
    cache = jfa.PagedKVCache(table, 8, hkv)
    assert cache.pages.numel() > 2**32
    ws = jfa.PagedWorkspace(cache)
    k, v = make_rows(2 * n, hkv, 67)
    rows = [(k[:n], v[:n]), (k[n:], v[n:])]
    pages = list(range(59988, 60000))
    table.grow([n, n])
    table.rows = [pages[:6], pages[6:]]
    table._refs = [0] * 60000
    for p in pages:
        table._refs[p] = 1
    table.table[:, :6] = torch.tensor(table.rows, dtype=torch.int32)
    cu = torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
    jfa.paged_append(cache, k.cuda(), v.cuda(), ws, cu)
    check_cache(table, cache, rows)
    q = rand_q(2, 8, 67)
    check_attend(cache, ws, rows, q, rms=RMS)
    got = jfa.paged_gather(cache, cu, 2 * n, ws)
    want = np.concatenate([Ref(*r).k.transpose(1, 0, 2) for r in rows])
    err = np.abs(got[0].cpu().double().numpy() - want)
    assert (err <= (BF16 + 2.0**-23) * np.abs(want) + 2.0**-133).all()
    moves, remap = table.compact()
    jfa.paged_move(cache, moves, ws, remap)
    torch.cuda.synchronize()
    assert ws.error_flag(cache) == 0 and sorted(table.rows[0] + table.rows[1]) == list(range(12))
    check_cache(table, cache, rows)
    check_attend(cache, ws, rows, q, rms=RMS)


# ---------------------------------------------------------------------------
# what the kernels themselves refuse
# ---------------------------------------------------------------------------
def flagged(cache, ws):
    torch.cuda.synchronize()
    flag = ws.error_flag(cache)
    ws.clear_error(cache)
    return flag == _lib.DEVERR_BAD_INDEX


@pytest.mark.parametrize("page", [-1, -2**31, 10**6, 2**31 - 1])
def test_bad_page_is_skipped_and_flagged(page):
    lens = [130, 200]
    table, cache, ws, rows = make(lens, 2, 1, seed=37)
    q = rand_q(2, 2, 37).cuda()
    want = jfa.paged_attend(cache, q, ws).clone()
    pages = cache.pages.clone()
    good = table.table.clone()
    table.table[0, 1] = page
    out = jfa.paged_attend(cache, q, ws)
    assert flagged(cache, ws)
    assert torch.equal(out[1], want[1]) and torch.isfinite(out[0]).all()
    cu = torch.tensor([0, 130, 330], dtype=torch.int32, device="cuda")
    outs = [torch.full((330, 1, D), 77.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    jfa.paged_gather(cache, cu, 330, ws, k_out=outs[0], v_out=outs[1])
    assert flagged(cache, ws)
    assert (outs[0][64:128] == 77).all() and not (outs[0][:64] == 77).any()
    # a page to be written
    table.table.copy_(good)
    table.grow([0, 60])
    table.table[1, 3] = page
    k, v = make_rows(60, 1, 38)
    cu = torch.tensor([0, 0, 60], dtype=torch.int32, device="cuda")
    jfa.paged_append(cache, k.cuda(), v.cuda(), ws, cu)
    assert flagged(cache, ws)
    assert torch.equal(cache.pages, pages)
    # an entry that a move should follow
    table.table[1, 3] = page
    remap = torch.arange(table.n_pages, dtype=torch.int32, device="cuda")
    jfa.paged_move(cache, torch.zeros(0, 2, dtype=torch.int32, device="cuda"), ws, remap)
    assert flagged(cache, ws)
    assert int(table.table[1, 3]) == page


@pytest.mark.parametrize("n", [-1, -2**31, 2**31 - 1, 64 * 5 + 65])
def test_bad_length_is_flagged(n):
    lens = [130, 200]
    table, cache, ws, rows = make(lens, 2, 1, seed=41)      # rows of 5 entries
    assert table.max_pages == 5
    q = rand_q(2, 2, 41).cuda()
    want = jfa.paged_attend(cache, q, ws).clone()
    table.seq_lens[0] = n
    out = jfa.paged_attend(cache, q, ws)
    assert flagged(cache, ws)
    assert torch.equal(out[1], want[1]) and (out[0] == 0).all()
    k, v = make_rows(2, 1, 42)
    pages, tails = cache.pages.clone(), cache.tail_k.clone()
    table.seq_lens[1] = 200
    jfa.paged_append(cache, k[:2].cuda(), v[:2].cuda(), ws, torch.tensor([0, 2, 2], dtype=torch.int32).cuda())
    assert flagged(cache, ws)
    assert torch.equal(cache.pages, pages) and torch.equal(cache.tail_k, tails)
    jfa.paged_gather(cache, torch.tensor([0, 2, 2], dtype=torch.int32).cuda(), 2, ws)
    assert flagged(cache, ws)


@pytest.mark.parametrize("cu", [[0, 5, 11], [-1, 5, 10], [6, 5, 10], [0, -3, 10], [0, 2**31 - 1, 10], [0, 10, 4]])
def test_bad_ranges_are_flagged(cu):
    lens = [130, 200]
    table, cache, ws, rows = make(lens, 2, 1, seed=43)
    k, v = make_rows(10, 1, 44)
    c = torch.tensor(cu, dtype=torch.int32).cuda()
    jfa.paged_gather(cache, c, 10, ws)
    assert flagged(cache, ws)
    jfa.paged_append(cache, k.cuda(), v.cuda(), ws, c)
    assert flagged(cache, ws)


def test_bad_starts_are_flagged():
    table, cache, ws, rows = make([130, 200], 2, 1, seed=45)
    cu = torch.tensor([0, 5, 10], dtype=torch.int32).cuda()
    for start in ([126, 0], [-1, 0], [0, 2**31 - 1]):
        jfa.paged_gather(cache, cu, 10, ws, start=torch.tensor(start, dtype=torch.int32).cuda())
        assert flagged(cache, ws)


@pytest.mark.parametrize("pairs", [[[0, 4]], [[-1, 1]], [[0, 0]], [[0, 1], [1, 2]], [[0, 2], [1, 2]],
                                   [[2**31 - 1, 1]]])
def test_bad_forks_are_flagged(pairs):
    table, cache, ws, rows = make([130, 200, 0, 64], 2, 1, seed=47)
    jfa.paged_fork(cache, torch.tensor(pairs, dtype=torch.int32).cuda(), ws)
    assert flagged(cache, ws)


@pytest.mark.parametrize("moves,remap", [
    ([[0, 100]], None), ([[-1, 2]], None), ([[3, 3]], None), ([[0, 2]], [0, 1, 2]), ([[0, 2]], [2, 1, 1])])
def test_bad_moves_are_flagged(moves, remap):
    table, cache, ws, rows = make([1], 2, 1, seed=49, spare=6)
    cache.pages.random_(0, 256)
    pages = cache.pages.clone()
    if remap is not None:
        remap = torch.tensor(remap + [3, 4, 5], dtype=torch.int32).cuda()
    jfa.paged_move(cache, torch.tensor(moves, dtype=torch.int32).cuda(), ws, remap)
    assert flagged(cache, ws)
    assert torch.equal(cache.pages, pages)


# ---------------------------------------------------------------------------
# together, as a program uses them
# ---------------------------------------------------------------------------
def rotate(x, pos, plan, w, eps):
    """In 64 bits, half layout: [T, heads, 128]."""
    y = x.double()
    if w is not None:
        y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    a = pos.double()[:, None, None] * torch.tensor(plan.frequencies, dtype=torch.float64)
    h = plan.rotary_dim // 2
    u, v = y[..., :h].clone(), y[..., h:2 * h].clone()
    y[..., :h], y[..., h:2 * h] = u * a.cos() - v * a.sin(), u * a.sin() + v * a.cos()
    return y


@pytest.mark.parametrize("graph", [False, True])
def test_prompts_then_decode_steps(graph):
    """Prompts enter, sequences fork, decode steps (eager, or one captured
    graph replayed as the cache grows), the pool is compacted in between."""
    heads, hkv, batch, steps = 8, 2, 4, 70
    plan = jfa.RotaryPlan(128, base=10000.0)
    g = gen(71)
    wq, wk = ((1 + 0.2 * torch.randn(D, generator=g)).bfloat16() for _ in range(2))
    table = jfa.PageTable(batch, 30, 12)
    cache = jfa.PagedKVCache(table, heads, hkv)
    ws = jfa.PagedWorkspace(cache)
    lens = [190, 60, 0, 1]
    cu = table.grow(lens)
    total = sum(lens)
    qkv = torch.randn(total, heads + 2 * hkv, D, generator=g).bfloat16().cuda()
    pos = torch.cat([torch.arange(n) for n in lens]).cuda()
    _, k = jfa.qk_norm_rope(qkv[:, :heads], qkv[:, heads:heads + hkv], pos, plan, wq.cuda(), wk.cuda())
    jfa.paged_append(cache, k, qkv[:, heads + hkv:], ws, cu)
    at = np.concatenate(([0], np.cumsum(lens)))
    kept = [(k[a:z].cpu(), qkv[a:z, heads + hkv:].cpu()) for a, z in zip(at[:-1], at[1:])]
    want = rotate(qkv[:, heads:heads + hkv].cpu(), pos.cpu(), plan, wk, 1e-6)
    err = (k.cpu().double() - want).abs()
    assert (err <= BF16 * want.abs() + 2.0**-18 * want.abs().amax(-1, keepdim=True)).all()
    jfa.paged_fork(cache, table.fork([(0, 2)]), ws)
    kept[2] = kept[0]

    wq_d, wk_d = wq.cuda(), wk.cuda()
    x = torch.empty(batch, heads + 2 * hkv, D, dtype=torch.bfloat16, device="cuda")
    where = torch.zeros(batch, dtype=torch.int32, device="cuda")
    out = torch.empty(batch, heads, D, dtype=torch.bfloat16, device="cuda")

    def step():
        torch.sub(table.seq_lens, 1, out=where)
        jfa.paged_decode_step(cache, x[:, :heads], x[:, heads:heads + hkv], x[:, heads + hkv:], where, plan, ws,
                              wq_d, wk_d, window=150, sinks=4, out=out)

    captured = None
    for i in range(steps):
        fresh = torch.randn(batch, heads + 2 * hkv, D, generator=g).bfloat16()
        x.copy_(fresh)
        table.grow(1)
        if graph and captured is None and i == 1:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            captured = torch.cuda.CUDAGraph()
            with torch.cuda.graph(captured, stream=side):
                step()
        if captured is not None:
            captured.replay()
        else:
            step()
        p = torch.tensor(table.lens) - 1
        kr = rotate(fresh[:, heads:heads + hkv], p, plan, wk, 1e-6)
        torch.cuda.synchronize()
        # the stored key: within a rounding of the formula's, then taken as it is
        rows = jfa.paged_gather(cache, torch.arange(batch + 1, dtype=torch.int32, device="cuda"), batch, ws,
                                start=(table.seq_lens - 1))
        torch.cuda.synchronize()
        knew = rows[0].cpu()
        assert ((knew.double() - kr).abs() <= BF16 * kr.abs() + 2.0**-18 * kr.abs().amax(-1, keepdim=True)).all()
        assert torch.equal(rows[1].cpu(), fresh[:, heads + hkv:])
        kept = [(torch.cat((a, knew[b:b + 1])), torch.cat((c, fresh[b:b + 1, heads + hkv:])))
                for b, (a, c) in enumerate(kept)]
        if i % 10 == 3 or i == steps - 1:
            q, _ = jfa.qk_norm_rope(x[:, :heads], x[:, heads:heads + hkv], where, plan, wq_d, wk_d)
            qd = q.cpu().double()
            qr = rotate(fresh[:, :heads], p, plan, wq, 1e-6)
            assert ((qd - qr).abs() <= BF16 * qr.abs() + 2.0**-18 * qr.abs().amax(-1, keepdim=True)).all()
            for b in range(batch):
                o, _, bound, _ = Ref(*kept[b]).attend(qd[b].numpy(), 1 / math.sqrt(D), 150, 4)
                assert (np.abs(out[b].cpu().double().numpy() - o) <= bound).all()
        if i == 30:
            table.free([1])
            jfa.paged_fork(cache, table.fork([(0, 1)]), ws)
            kept[1] = kept[0]
            moves, remap = table.compact()
            jfa.paged_move(cache, moves, ws, remap)
    assert ws.error_flag(cache) == 0
    check_cache(table, cache, kept)


def test_decode_step_with_idle_rows():
    lens = [64, 0, 70, 0]
    table, cache, ws, rows = make(lens, 4, 2, seed=73)
    plan = jfa.RotaryPlan(64)
    table.grow(1)
    new = torch.randn(4, 8, D, generator=gen(73)).bfloat16().cuda()
    pos = table.seq_lens - 1
    out = jfa.paged_decode_step(cache, new[:, :4], new[:, 4:6], new[:, 6:], pos, plan, ws)
    q, k = jfa.qk_norm_rope(new[:, :4], new[:, 4:6], pos, plan)
    torch.cuda.synchronize()
    assert ws.error_flag(cache) == 0
    kept = [(torch.cat((a, k[b:b + 1].cpu())), torch.cat((c, new[b:b + 1, 6:].cpu()))) if lens[b] else (a, c)
            for b, (a, c) in enumerate(rows)]
    check_cache(table, cache, kept)
    assert torch.equal(out, check_attend(cache, ws, kept, q.cpu()))
    assert (out[1] == 0).all() and (out[3] == 0).all()


def test_side_stream_and_two_graphs_on_one_workspace():
    lens = [500, 64, 3000]
    table, cache, ws, rows = make(lens, 8, 2, seed=53)
    qs = [rand_q(3, 8, 53 + i).cuda() for i in range(2)]
    want = [jfa.paged_attend(cache, q, ws).clone() for q in qs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        a = jfa.paged_attend(cache, qs[0], ws)
    side.synchronize()
    assert torch.equal(a, want[0])
    graphs, outs = [], []
    for q in qs:
        g = torch.cuda.CUDAGraph()
        out = torch.empty_like(want[0])
        with torch.cuda.graph(g):
            jfa.paged_attend(cache, q, ws, out=out)
        graphs.append(g)
        outs.append(out)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for out, w in zip(outs, want):
        assert torch.equal(out, w)


def test_calls_on_a_given_stream():
    """Stream objects and handles; outputs come from that stream's memory."""
    lens = [300, 70]
    table, cache, ws, rows = make(lens, 4, 2, seed=59)
    q = rand_q(2, 4, 59).cuda()
    want = jfa.paged_attend(cache, q, ws).clone()
    cu = torch.tensor([0, 300, 370], dtype=torch.int32, device="cuda")
    k, v = jfa.paged_gather(cache, cu, 370, ws)
    plan = jfa.RotaryPlan(128)
    pos = torch.arange(2, device="cuda")
    turned = jfa.qk_norm_rope(q, k[:2], pos, plan)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        a = jfa.paged_attend(cache, q, ws, stream=stream)
        b = jfa.paged_gather(cache, cu, 370, ws, stream=stream)
        c = jfa.qk_norm_rope(q, k[:2], pos, plan, stream=stream)
        side.synchronize()
        assert torch.equal(a, want) and torch.equal(b[0], k) and torch.equal(b[1], v)
        assert torch.equal(c[0], turned[0]) and torch.equal(c[1], turned[1])


def test_one_sequence_of_odd_strides():
    """The stride of a dimension of one element means nothing."""
    table, cache, ws, rows = make([100], 1, 1, seed=61)
    q = rand_q(1, 1, 61).cuda()
    want = jfa.paged_attend(cache, q, ws).clone()
    odd = q.as_strided((1, 1, D), (3, 5, 1))
    assert torch.equal(jfa.paged_attend(cache, odd, ws), want)
    table.grow(1)
    jfa.paged_append(cache, odd, odd, ws)
    kept = [(torch.cat((rows[0][0], q.cpu())), torch.cat((rows[0][1], q.cpu())))]
    torch.cuda.synchronize()
    assert ws.error_flag(cache) == 0
    check_cache(table, cache, kept)


def test_output_in_the_query_s_place():
    lens = [3000, 0, 64]
    table, cache, ws, rows = make(lens, 8, 2, seed=63)
    q = rand_q(3, 8, 63).cuda()
    want = jfa.paged_attend(cache, q, ws).clone()
    got = jfa.paged_attend(cache, q, ws, out=q)
    torch.cuda.synchronize()
    assert got is q and torch.equal(q, want)


def test_two_workspaces_at_the_same_time():
    lens = [9000, 64, 3000]
    table, cache, ws, rows = make(lens, 8, 2, seed=57)
    q = rand_q(3, 8, 57).cuda()
    want = jfa.paged_attend(cache, q, ws).clone()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [ws, jfa.PagedWorkspace(cache)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(jfa.paged_attend(cache, q, spaces[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for xs in got for x in xs)
