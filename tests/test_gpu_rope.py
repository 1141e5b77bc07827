"""GPU parity of the head norms and rotary positions against the formula in 64 bits."""
import math

import pytest
import torch

import bit_kv_cache_jfa_b200 as jfa

pytestmark = pytest.mark.gpu

D = 128
BF16 = 2.0**-8     # half a step of bf16, relative to the value
SCALINGS = {"none": {}, "linear": dict(factor=4.0), "llama3": dict(factor=8.0, original=8192),
            "yarn": dict(factor=16.0, original=16384)}


def formula(x, pos, plan, w, eps):
    """(y, size): the outputs in 64 bits and the size of what is added for each."""
    y = x.double()
    if w is not None:
        y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    r, h = plan.rotary_dim, plan.rotary_dim // 2
    a = pos.double()[:, None, None] * torch.tensor(plan.frequencies, dtype=torch.float64)
    cos, sin = plan.amplitude * a.cos(), plan.amplitude * a.sin()
    first, second = (slice(0, r, 2), slice(1, r, 2)) if plan.interleaved else (slice(0, h), slice(h, r))
    u, v = y[..., first].clone(), y[..., second].clone()
    size = y.abs()
    size[..., first] = size[..., second] = plan.amplitude * (u.abs() + v.abs())
    y[..., first], y[..., second] = u * cos - v * sin, u * sin + v * cos
    return y, size


def check(got, x, pos, plan, w, eps=1e-6):
    want, size = formula(x.cpu(), pos.cpu(), plan, None if w is None else w.cpu(), eps)
    # One rounding to bf16; before it fp32: the angle's fraction of a turn to
    # 2^-24 of half a turn (2e-7), sine and cosine, the norm's sum of 128
    # squares (64 * 2^-24 of it at most) and a few products: 2^-17 of the terms.
    err = (got.cpu().double() - want).abs()
    assert (err <= BF16 * want.abs() + 2.0**-17 * size + 2.0**-133).all(), \
        (err / (BF16 * want.abs() + 2.0**-17 * size + 1e-300)).max()


def inputs(t, h, hkv, seed, far=100000, dtype=torch.int32):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(t, h + 2 * hkv, D, generator=g).bfloat16().cuda()
    pos = torch.randint(0, far, (t,), generator=g).to(dtype).cuda()
    w = [(1 + 0.2 * torch.randn(D, generator=g)).bfloat16().cuda() for _ in range(2)]
    return qkv[:, :h], qkv[:, h:h + hkv], pos, w


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary", [2, 6, 16, 24, 48, 50, 64, 96, 126, 128])
@pytest.mark.parametrize("norm", [False, True])
def test_layouts(rotary, interleaved, norm):
    q, k, pos, w = inputs(19, 5, 3, rotary)
    plan = jfa.RotaryPlan(rotary, interleaved=interleaved)
    wq, wk = w if norm else (None, None)
    qo, ko = jfa.qk_norm_rope(q, k, pos, plan, wq, wk)
    torch.cuda.synchronize()
    assert qo.is_contiguous() and qo.shape == (19, 5, D) and ko.shape == (19, 3, D)
    check(qo, q, pos, plan, wq)
    check(ko, k, pos, plan, wk)
    if not norm:                                       # channels past the rotary ones pass as they are
        assert torch.equal(qo[..., rotary:], q[..., rotary:])


@pytest.mark.parametrize("scaling", sorted(SCALINGS))
@pytest.mark.parametrize("far", [10, 200000, 2**31 - 1])
def test_scalings_and_far_positions(scaling, far):
    q, k, pos, w = inputs(65, 8, 2, 7, far)
    pos[0], pos[1] = 0, far - 1
    plan = jfa.RotaryPlan(128, base=500000.0, scaling=scaling, **SCALINGS[scaling])
    qo, ko = jfa.qk_norm_rope(q, k, pos, plan, w[0], w[1], eps=1e-5)
    torch.cuda.synchronize()
    check(qo, q, pos, plan, w[0], 1e-5)
    check(ko, k, pos, plan, w[1], 1e-5)


@pytest.mark.parametrize("tokens,heads,hkv", [(1, 1, 1), (1, 64, 8), (2, 3, 1), (1000, 7, 1), (33, 16, 16), (4, 0, 2),
                                              (4, 2, 0), (300, 40, 1)])
def test_sizes_and_wide_positions(tokens, heads, hkv):
    q, k, pos, w = inputs(tokens, heads, hkv, tokens + heads, dtype=torch.int64)
    plan = jfa.RotaryPlan(64)
    qo, ko = jfa.qk_norm_rope(q, k, pos, plan, w[0], None)    # a norm on one side only
    torch.cuda.synchronize()
    check(qo, q, pos, plan, w[0])
    check(ko, k, pos, plan, None)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary", [10, 128])
def test_in_place_and_strided(rotary, interleaved):
    q, k, pos, w = inputs(50, 6, 2, 3)
    plan = jfa.RotaryPlan(rotary, interleaved=interleaved)
    want = jfa.qk_norm_rope(q, k, pos, plan, *w)
    heads_first = q.transpose(0, 1).contiguous().transpose(0, 1)     # [heads][tokens][128] in memory
    got = jfa.qk_norm_rope(heads_first, k, pos, plan, *w, q_out=heads_first, k_out=k)
    torch.cuda.synchronize()
    assert got[0] is heads_first and got[1] is k
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_negative_positions_turn_back():
    q, k, pos, _ = inputs(40, 2, 1, 5, dtype=torch.int64)
    plan = jfa.RotaryPlan(128)
    qo, _ = jfa.qk_norm_rope(q, k, -pos, plan)
    torch.cuda.synchronize()
    check(qo, q, -pos, plan, None)


def test_extreme_rows():
    """Zero rows (eps alone), rows of tiny and of large values, infinities
    past the rotary channels and in them."""
    q, k, pos, w = inputs(6, 2, 1, 9)
    q[0] = 0
    q[1] *= 1e-15
    q[2] *= 1e15
    q[3, :, 100] = math.inf
    q[4, :, 3] = math.nan
    plan = jfa.RotaryPlan(64)
    qo, _ = jfa.qk_norm_rope(q, k, pos, plan, None, None)
    qn, _ = jfa.qk_norm_rope(q, k, pos, plan, w[0], None)
    torch.cuda.synchronize()
    assert (qn[0] == 0).all() and (qo[0] == 0).all()
    check(qo[:3], q[:3], pos[:3], plan, None)
    check(qn[:3], q[:3], pos[:3], plan, w[0])
    assert (qo[3, :, 100] == math.inf).all()
    keep = [c for c in range(D) if c != 100]
    assert torch.isfinite(qo[3][:, keep]).all()
    assert torch.isnan(qo[4][:, [3, 35]]).all()
    keep = [c for c in range(D) if c not in (3, 35)]
    assert torch.isfinite(qo[4][:, keep]).all()


def test_on_another_stream_and_captured():
    q, k, pos, w = inputs(100, 8, 2, 13)
    plan = jfa.RotaryPlan(128)
    want = jfa.qk_norm_rope(q, k, pos, plan, *w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = jfa.qk_norm_rope(q, k, pos, plan, *w)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    outs = [torch.empty_like(x) for x in want]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        jfa.qk_norm_rope(q, k, pos, plan, *w, q_out=outs[0], k_out=outs[1])
    pos += 1
    g.replay()
    again = jfa.qk_norm_rope(q, k, pos, plan, *w)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], again[0]) and torch.equal(outs[1], again[1])
