"""GPU: how exact the attention over the paged 4-bit cache is, whatever the
ranges of keys and values: bounds in which logits are of 32 bits."""
import math

import numpy as np
import pytest
import torch

import bit_kv_cache_jfa_b200 as jfa
from test_gpu_paged import BF16, D, Ref, gen, make, make_rows, rand_q

pytestmark = pytest.mark.gpu


def reference(ref, q, scale):
    """(out, lse, bound, lse_bound) of queries [H][128] over ref's cache, in 64
    bits.

    A logit is a sum of products that are exact in 32 bits (the query times a
    key's scale is held in two halves, 2^-25 of 8 max|q| lost under fp16's
    smallest step, times a code of at most 15), of codes and zero points apart:
    about 20 additions, cut to 32 bits each, are 20 * 2^-23 < 2^-18 of the terms'
    size, scaling and the rest 2^-20 of the logit.
    A weight is rounded to fp16, and once more times its value's scale (2^-11
    each at most).  The largest lies in [2^10, 2^15], so that what is lost at
    fp16's bottom, 2^-25, is 2^-35 of the largest; of a weight times a scale
    (which counts for a code of 15 at most), that times 8 of the largest scale
    of the 64 tokens, and times 8 of it again where it is 2 or more."""
    hkv, h = ref.k.shape[0], q.shape[0]
    out, bound, lse, lse_bound = np.zeros((h, D)), np.zeros((h, D)), np.zeros(h), np.zeros(h)
    c, nq = ref.c, ref.nq
    for i in range(h):
        j = i // (h // hkv)
        k, v, a = ref.k[j], ref.v[j], np.abs(q[i])
        x = scale * (k @ q[i])
        m = x.max()
        p = np.exp(x - m)
        lse[i] = m + np.log(p.sum())
        p /= p.sum()
        out[i] = p @ v
        size, ce = np.abs(k) @ a, np.abs(v).copy()
        lost = np.zeros((len(p), D))
        if nq:
            s = np.repeat(c.k_scale[0, j].astype(float), 64, 0)
            z = np.repeat(np.abs(c.k_zero[0, j].astype(float)), 64, 0)
            size[:nq] += (s * c.k_codes[0, j] + z) @ a
            vs = np.repeat(c.v_scale[0, j].astype(float), 32, -1)
            vz = np.repeat(np.abs(c.v_zero[0, j].astype(float)), 32, -1)
            ce[:nq] = vs * c.v_codes[0, j] + vz
            top = c.v_scale[0, j].astype(float).reshape(-1, 64 * 4).max(1).repeat(64)[:, None]
            lost[:nq] = 15 * 8 * top * np.maximum(8 * top, 1) + vz
        e = scale * (2.0**-18 * size + 2.0**-22 * 15 * 128 * a.max()) + 2.0**-20 * (1 + np.abs(x))
        w = 2.0**-11
        bound[i] = p @ ((np.expm1(e) + 2 * w + 2.0**-16)[:, None] * (ce + np.abs(out[i]))) \
            + 2.0**-35 * p.max() * (lost + np.abs(out[i])).sum(0) + (BF16 + 2.0**-16) * np.abs(out[i])
        lse_bound[i] = -np.log1p(-min(p @ (np.expm1(e) + w) + 2.0**-35 * p.max() * len(p), 0.9)) \
            + 2.0**-20 * (1 + abs(lse[i]))
    return out, lse, bound, lse_bound


# Relative error over all outputs, root mean square: bf16's rounding, at most
# 2^-8 and uniform, 2^-8 / sqrt(3) = 2.26e-3; the weights' two, 2^-11 / sqrt(3)
# each, of codes times scales, which are about three times the values'
# size: 8.5e-4 and 2.8e-4; a logit's 32 bits 2e-4.  Together 2.45e-3.
RMS = 2.5e-3


def check(lens, k, v, q, rms=RMS, scale=1 / math.sqrt(D)):
    heads, hkv = q.shape[1], k.shape[1]
    n_pages = sum(n // 64 + 1 for n in lens)
    table = jfa.PageTable(len(lens), n_pages, max(lens) // 64 + 1)
    cache = jfa.PagedKVCache(table, heads, hkv)
    ws = jfa.PagedWorkspace(cache)
    jfa.paged_append(cache, k.cuda(), v.cuda(), ws, table.grow(lens))
    lse = torch.zeros(len(lens), heads, device="cuda")
    out = jfa.paged_attend(cache, q.cuda(), ws, scale=scale, lse=lse)
    torch.cuda.synchronize()
    assert ws.error_flag(cache) == 0
    got, lse, at, want = out.cpu().double().numpy(), lse.cpu().double().numpy(), 0, []
    for b, n in enumerate(lens):
        o, l, bound, l_bound = reference(Ref(k[at:at + n], v[at:at + n]), q[b].double().numpy(), scale)
        at += n
        want.append(o)
        assert (np.abs(lse[b] - l) <= l_bound).all(), (b, np.abs(lse[b] - l) / l_bound)
        assert (np.abs(got[b] - o) <= bound).all(), (b, (np.abs(got[b] - o) / bound).max())
    want = np.stack(want)
    assert np.linalg.norm(got - want) <= rms * np.linalg.norm(want)


@pytest.mark.parametrize("big,q_scale", [(1.0, 1.0), (10.0, 1.0), (30.0, 1.0), (100.0, 1.0), (100.0, 4.0),
                                         (1000.0, 0.5)])
@pytest.mark.parametrize("heads,hkv", [(8, 1), (6, 2), (1, 1)])
def test_keys_of_any_range(big, q_scale, heads, hkv):
    """A few key channels far larger than the others: what their products are
    rounded to must not grow with them."""
    lens = [257, 4000, 641, 1]
    k, v = make_rows(sum(lens), hkv, int(big) + heads, outliers=0)
    wide = torch.ones(D)
    wide[torch.randperm(D, generator=gen(int(big)))[:4]] = big
    q = (torch.randn(len(lens), heads, D, generator=gen(heads)) * q_scale).bfloat16()
    check(lens, (k.float() * wide).bfloat16(), v, q)


def test_wide_keys_of_a_long_sequence():
    lens = [32768]
    k, v = make_rows(lens[0], 1, 77, outliers=0)
    wide = torch.ones(D)
    wide[[3, 40, 77, 120]] = 30.0
    q = torch.randn(1, 8, D, generator=gen(78)).bfloat16()
    check(lens, (k.float() * wide).bfloat16(), v, q)


@pytest.mark.parametrize("size,loud", [(1.0, False), (1.0, True), (2.0**-9, False), (2.0**-14, False)])
def test_mass_spread_over_many_tokens_far_below_one(size, loud):
    """One token of value 0 above 20000 of a weight of 2^-24 each, which alone
    make the output: with values of about 1, with values thousands of times as
    large among them (which no weight reaches), with small values.  256
    sequences share the pages, so that a warp goes over most of one."""
    n, batch, hkv = 20001, 256, 8
    k, v = make_rows(n, hkv, 91, outliers=0)
    k *= 0.02
    k[n // 2] = 16.6 * math.sqrt(D) / D
    v = ((v.float() * 0.5 + 3) * size).bfloat16()
    v[n // 2] = 0
    if loud:
        for g in range(0, n // 64, 8):
            k[64 * g:64 * g + 64] = -3.0
            v[64 * g:64 * g + 64] *= 2048
    q = torch.ones(1, hkv, D).bfloat16()
    table = jfa.PageTable(batch, 320, 320)
    cache = jfa.PagedKVCache(table, hkv, hkv)
    ws = jfa.PagedWorkspace(cache)
    jfa.paged_append(cache, k.cuda(), v.cuda(), ws, table.grow([n] + [0] * (batch - 1)))
    jfa.paged_fork(cache, table.fork([(0, b) for b in range(1, batch)]), ws)
    lse = torch.zeros(batch, hkv, device="cuda")
    got = jfa.paged_attend(cache, q.cuda().expand(batch, hkv, D), ws, lse=lse).cpu().double().numpy()
    assert ws.error_flag(cache) == 0
    out, l, bound, l_bound = reference(Ref(k, v), q[0].double().numpy(), 1 / math.sqrt(D))
    for b in range(batch):
        assert np.linalg.norm(got[b] - out) <= RMS * np.linalg.norm(out), b
        assert (np.abs(got[b] - out) <= bound).all(), b
        assert (np.abs(lse[b].cpu().double().numpy() - l) <= l_bound).all(), b


@pytest.mark.parametrize("q_value", [-2.0**97, -2.0**99, 2.0**99, -2.0**60, 0.0])
def test_logits_of_any_size(q_value):
    """Equal logits far below and above zero: the mean of the values.  Keys of 1
    and powers of two, so that every logit is the same number exactly."""
    lens = [200, 1, 64, 1000]
    table = jfa.PageTable(len(lens), 30, 17)
    cache = jfa.PagedKVCache(table, 4, 2)
    ws = jfa.PagedWorkspace(cache)
    _, v = make_rows(sum(lens), 2, 99)
    jfa.paged_append(cache, torch.ones_like(v).cuda(), v.cuda(), ws, table.grow(lens))
    lse = torch.zeros(len(lens), 4, device="cuda")
    out = jfa.paged_attend(cache, torch.full((len(lens), 4, D), q_value).bfloat16().cuda(), ws, lse=lse)
    torch.cuda.synchronize()
    assert ws.error_flag(cache) == 0
    at = 0
    for b, n in enumerate(lens):
        ref = Ref(torch.ones(n, 2, D).bfloat16(), v[at:at + n])
        at += n
        want = np.repeat(ref.v.mean(1), 2, 0)
        # 1 / n of each: the value's sum in 32 bits, its product with fp16 weights
        # exact or rounded once, the mass; bf16 at the end
        size = np.repeat(np.abs(ref.v).max(1), 2, 0)
        assert (np.abs(out[b].cpu().double().numpy() - want) <= BF16 * np.abs(want) + 2.0**-10 * 3 * size).all()
        x = q_value * D / math.sqrt(D)
        assert (np.abs(lse[b].cpu().double().numpy() - (x + math.log(n))) <= 2.0**-20 * (abs(x) + 8)).all()


@pytest.mark.parametrize("fill", [0xFFFF, 0x7C00, 0x7BFF, 0x7000, 0x3C00, 0x0001])
@pytest.mark.parametrize("window,sinks", [(100, 5), (100, 0), (1, 70), (130, 64), (65, 129)])
def test_masked_values_change_no_bit(fill, window, sinks):
    """Value scales and zero points of masked tokens, in groups that are seen in
    part: NaN, infinite, the largest numbers, large and small ones."""
    lens = [200, 333, 70, 64, 600]
    table, cache, ws, rows = make(lens, 4, 2, seed=101)
    q = rand_q(5, 4, 101).cuda()
    want = jfa.paged_attend(cache, q, ws, window=window, sinks=sinks).clone()
    tab, pages = table.table.cpu(), cache.pages.clone().cpu()
    changed = 0
    for b, n in enumerate(lens):
        for t in range(64 * ((n - 1) // 64)):
            if sinks <= t < n - window:
                s = t % 64
                for j in range(4):
                    at = 4608 + s // 16 * 128 + s % 8 // 2 * 32 + j * 8 + s % 16 // 8 * 4 + 2 * (s % 2)
                    for part in (at, at + 512):
                        pages[int(tab[b, t // 64]), :, part] = fill & 0xFF
                        pages[int(tab[b, t // 64]), :, part + 1] = fill >> 8
                changed += 1
    assert changed > 100
    cache.pages.copy_(pages)
    lse = torch.zeros(5, 4, device="cuda")
    got = jfa.paged_attend(cache, q, ws, window=window, sinks=sinks, lse=lse)
    torch.cuda.synchronize()
    assert ws.error_flag(cache) == 0
    assert torch.equal(got, want) and torch.isfinite(lse).all()


def test_read_back_to_16_byte_aligned_rows():
    """Outputs that begin 16 bytes past a 32-byte border, or one of them."""
    lens = [200, 0, 129, 64]
    table, cache, ws, rows = make(lens, 3, 3, seed=103)
    cu = torch.tensor(np.concatenate(([0], np.cumsum(lens))), dtype=torch.int32).cuda()
    total = sum(lens)
    want = jfa.paged_gather(cache, cu, total, ws)
    for offs in ((8, 8), (8, 0), (0, 8), (24, 16)):
        flat = [torch.full((total * 3 * D + 64,), 77.0, dtype=torch.bfloat16, device="cuda") for _ in offs]
        outs = [f[o:o + total * 3 * D].view(total, 3, D) for f, o in zip(flat, offs)]
        jfa.paged_gather(cache, cu, total, ws, k_out=outs[0], v_out=outs[1])
        torch.cuda.synchronize()
        assert ws.error_flag(cache) == 0
        for f, o, x, w in zip(flat, offs, outs, want):
            assert torch.equal(x, w)
            assert (f[:o] == 77).all() and (f[o + total * 3 * D:] == 77).all()
