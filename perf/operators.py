"""Cases of the operators of one decode layer over a paged 4-bit KV cache: the
head norms and rotary positions in front of the cache, the cache's append and
read-back, the single-token attention over it (whole, or a sliding window with
the first tokens kept), and the page operations (fork, compaction).

Each case runs in its plain form (elementary torch operations) or, with
``own`` set, through the package's calls, on the same inputs; ``exact`` gives
the outputs in 64 bits from the operators' definitions.

The cache, as both forms find it: 64-token pages of one 9728-byte K4V4 record
per KV head (4-bit codes in the record's order, fp16 scales and zero points),
a page table and a length per sequence, and a bf16 tail of the newest 1..64
tokens of each sequence, whose 16-byte chunk c of slot t sits at chunk
position c ^ (t % 8) of its row."""
import functools
import math

import numpy as np
import torch

own = False

D = 128             # head size
PAGE = 64           # tokens of a page
REC = 9728          # bytes of a record: 64 tokens of one KV head
O_KC, O_VS, O_VC = 512, 4608, 5632   # key codes, value scales, value codes (key scales at 0)


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    def rope(name, **kw):
        return {"name": name, "op": "rope", **kw}

    def attend(name, **kw):
        return {"name": name, "op": "attend", "window": 0, "sinks": 0, "idle": False, **kw}

    return [
        # one decode step of a batch of 64, a layer with head norms (32 heads, 4 KV heads)
        rope("rope_norm_64_rows", tokens=64, heads=32, kv_heads=4, norm=True, rotary=128,
             interleaved=False, scaling="none", far=32768),
        # a prompt of 8192 tokens, 32/8 heads, no norm, frequencies scaled by parts, q and k as
        # slices of one projection's output
        rope("rope_prompt_8192", tokens=8192, heads=32, kv_heads=8, norm=False, rotary=128,
             interleaved=False, scaling="llama3", far=131072),
        # an odd chunk far into a long context, interleaved pairs on half of the head, 64/8 heads
        rope("rope_far_interleaved", tokens=1021, heads=64, kv_heads=8, norm=True, rotary=64,
             interleaved=True, scaling="yarn", far=262144),
        # five prompts of odd lengths enter the cache and are read back for their attention
        {"name": "append_prompts", "op": "append", "batch": 5, "kv_heads": 8, "lo": 900,
         "hi": 3000, "new": 1601},
        # a decode batch: two tokens a sequence over short histories, read back whole
        {"name": "append_rows", "op": "append", "batch": 33, "kv_heads": 4, "lo": 1, "hi": 700,
         "new": 2},
        # the smallest call: one sequence of 300 tokens, 8/2 heads
        attend("attend_300", batch=1, heads=8, kv_heads=2, lo=300, hi=300),
        # 64 sequences of very unlike lengths, some slots idle, 32/8 heads
        attend("attend_ragged_64", batch=64, heads=32, kv_heads=8, lo=1, hi=6000, idle=True),
        # one sequence of 131072 tokens, 32/8 heads
        attend("attend_128k", batch=1, heads=32, kv_heads=8, lo=131072, hi=131072),
        # 16 sequences about 32768 tokens long, 8 query heads a KV head
        attend("attend_32k_gqa8", batch=16, heads=32, kv_heads=4, lo=30001, hi=32768),
        # a layer with a window of 4000 tokens and 70 first tokens kept, 24 long sequences
        attend("attend_window_4000", batch=24, heads=64, kv_heads=8, lo=5000, hi=16001,
               window=4000, sinks=70),
        # one sequence of a handful forked into the others (parallel samples), a small pool compacted
        {"name": "pages_small", "op": "pages", "batch": 6, "kv_heads": 2, "pages": 300,
         "parents": 1, "moves": 41},
        # 8 parents forked to 64 slots; a third of a pool of 3000 pages moved to its front
        {"name": "pages_large", "op": "pages", "batch": 64, "kv_heads": 8, "pages": 3001,
         "parents": 8, "moves": 1000},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "pages"])
    if op == "rope":
        hkv = rng.choice([1, 2, 4, 8])
        return {"op": op, "tokens": _log(rng, 1, 6000), "heads": hkv * rng.randint(1, 8),
                "kv_heads": hkv, "norm": rng.random() < 0.5, "rotary": 2 * rng.randint(1, 64),
                "interleaved": rng.random() < 0.5,
                "scaling": rng.choice(["none", "linear", "llama3", "yarn"]),
                "far": _log(rng, 100, 1000000)}
    if op == "append":
        lo = _log(rng, 1, 1500)
        return {"op": op, "batch": _log(rng, 1, 40), "kv_heads": rng.choice([1, 2, 4, 8]),
                "lo": lo, "hi": lo + _log(rng, 1, 700), "new": _log(rng, 1, min(lo, 500))}
    if op == "pages":
        pages = _log(rng, 60, 3000)
        batch = rng.randint(2, 60)
        return {"op": op, "batch": batch, "kv_heads": rng.choice([1, 2, 4, 8]), "pages": pages,
                "parents": rng.randint(1, max(1, batch // 4)), "moves": rng.randint(1, pages // 3)}
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.randint(1, 8)
    total = _log(rng, 100, 900000) // hkv + 1   # tokens of all sequences together
    batch = max(1, min(96, total // _log(rng, 50, 60000)))
    hi = max(1, min(131072, total // batch))
    lo = rng.randint(1, hi)
    window = _log(rng, 1, 2 * hi) if rng.random() < 0.5 else 0
    return {"op": op, "batch": batch, "heads": hkv * g, "kv_heads": hkv, "lo": lo, "hi": hi,
            "window": window, "sinks": _log(rng, 1, 200) - 1 if window else 0,
            "idle": batch > 3 and rng.random() < 0.5}


def _lens(case):
    """The sequences' lengths: spread over [lo, hi] by multiples of the golden
    section; with idle slots every seventh length is 0."""
    b = np.arange(case["batch"])
    n = case["lo"] + np.floor((case["hi"] - case["lo"] + 1) * np.modf((b + 1) * 0.6180339887498949)[0])
    n = np.minimum(n, case["hi"]).astype(np.int64)
    if case.get("idle"):
        n[b % 7 == 3] = 0
    return n


def _packed(n):
    """Packed tokens of a sequence of n: whole pages, the newest 1..64 tokens left out."""
    return PAGE * (np.maximum(n - 1, 0) // PAGE)


def _seen(n, window, sinks):
    """(first windowed token, end of the kept first tokens) of a query at n - 1."""
    lo = np.maximum(n - window, 0) if window else np.zeros_like(n)
    return lo, np.minimum(lo, sinks)


def work(case):
    if case["op"] == "rope":
        rows = case["tokens"] * (case["heads"] + case["kv_heads"])
        return {"bytes": rows * D * 4 + 4 * case["tokens"], "flops": rows * (3 * case["rotary"] + 4 * D * case["norm"])}
    if case["op"] == "append":
        n = _lens(case)
        n0 = n - case["new"]
        hkv = case["kv_heads"]
        flushed, old = (_packed(n) - _packed(n0)).sum(), (n0 - _packed(n0))[_packed(n) > _packed(n0)].sum()
        put = 512 * (case["batch"] * case["new"] + old) + 152 * flushed \
            + 512 * np.minimum(case["new"], n - _packed(n)).sum()
        got = 152 * _packed(n).sum() + 512 * (n - _packed(n)).sum() + 512 * n.sum()
        return {"bytes": float(hkv * (put + got)), "flops": float(hkv * D * 4 * (flushed + n.sum()))}
    if case["op"] == "pages":
        tails = sum(_tail_of(case, p) for p in _pairs(case)[:, 0])
        return {"bytes": float(2 * case["moves"] * case["kv_heads"] * REC + 2 * 512 * case["kv_heads"] * tails), "flops": 0}
    n = _lens(case)
    lo, sink = _seen(n, case["window"], case["sinks"])
    nq = _packed(n)
    packed = np.minimum(sink, nq) + np.maximum(nq - lo, 0)
    tail = np.maximum(sink - nq, 0) + n - np.maximum(lo, nq)
    b = case["kv_heads"] * (152.0 * packed.sum() + 512.0 * tail.sum()) + case["batch"] * case["heads"] * D * 4
    return {"bytes": float(b), "flops": float(4 * D * case["heads"] * (packed + tail).sum())}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rows(case, seed):
    """Keys and values of every sequence's tokens, in turn, bf16 [sum n][H_kv][128]:
    unit normals, four key channels ten times as large (outlier channels)."""
    g = _gen(seed)
    total, hkv = int(_lens(case).sum()), case["kv_heads"]
    big = torch.ones(D, device="cuda")
    big[torch.randperm(D, generator=g, device="cuda")[:4]] = 10.0
    k, v = (torch.empty(total, hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for a in range(0, total, 1 << 16):
        m = min(1 << 16, total - a)
        k[a:a + m] = _normal(g, m, hkv, D) * big
        v[a:a + m] = _normal(g, m, hkv, D)
    return k, v


def _q(case, seed):
    return _normal(_gen(seed + 7), case["batch"], case["heads"], D).bfloat16()


def _ints(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@functools.cache
def _key_nibbles():
    """Place of the code of (token, channel) among a record's 8192 key codes."""
    t, c = torch.meshgrid(torch.arange(PAGE), torch.arange(D), indexing="ij")
    half, lane = c % 16 // 8, t % 8 * 4 + c % 8 // 2
    slot = c // 16 * 2 + half
    word = t // 16 * 256 + lane * 8 + slot % 8
    return (word * 8 + slot // 8 + t % 16 // 8 * 2 + c % 2 * 4).cuda()


@functools.cache
def _value_nibbles():
    t, c = torch.meshgrid(torch.arange(PAGE), torch.arange(D), indexing="ij")
    lane, w = c % 8 * 4 + t % 8 // 2, c // 16 % 4 * 2 + t % 16 // 8
    word = (t // 16 * 2 + w // 4) * 128 + lane * 4 + w % 4
    return (word * 8 + c // 64 + c % 16 // 8 * 2 + t % 2 * 4).cuda()


@functools.cache
def _key_params():
    """Place of channel c's scale among the record's 16-bit key numbers (its zero point 128 on)."""
    c = torch.arange(D)
    pair = c // 16 * 2 + c % 16 // 8
    return (pair // 4 * 32 + c % 8 // 2 * 8 + pair % 4 * 2 + c % 2).cuda()


@functools.cache
def _value_params():
    """Place of (token, 32-channel group)'s scale among the 16-bit value numbers (zero point 256 on)."""
    t, j = torch.meshgrid(torch.arange(PAGE), torch.arange(D // 32), indexing="ij")
    return (t // 16 * 64 + t % 8 // 2 * 16 + j * 4 + t % 16 // 8 * 2 + t % 2).cuda()


def _round_to_half(x, up):
    """fp16 neighbour of a float64 at or above (up) or at or below it."""
    h = x.half()
    off = h.double() < x if up else h.double() > x
    bits = h.view(torch.int16).int()
    order = torch.where(bits < 0, -(bits & 0x7FFF), bits) + (1 if up else -1)  # the halves in order, as whole numbers
    near = torch.where(order < 0, -order - 0x8000, order).to(torch.int16).view(torch.float16)
    return torch.where(off, near, h)


def _quantise(x, dim):
    """(codes, scale, zero) of x along dim: zero the minimum rounded down, scale the
    fifteenth part of the range rounded up, codes to nearest even (all in 64 bits)."""
    x = x.double()
    zero = _round_to_half(x.amin(dim, True), False)
    scale = _round_to_half((x.amax(dim, True) - zero.double()) / 15, True)
    s = scale.double()
    code = torch.round((x - zero.double()) / torch.where(s == 0, 1.0, s)).clamp(0, 15)
    return torch.where(s == 0, 0.0, code).to(torch.uint8), scale, zero


def _records(k, v):
    """Records uint8 [...][9728] of k, v [...][64][128]."""
    lead = k.shape[:-2]
    kc, ks, kz = _quantise(k, -2)
    vc, vs, vz = _quantise(v.reshape(*lead, PAGE, 4, 32), -1)
    rec = torch.empty(*lead, REC, dtype=torch.uint8, device=k.device)
    for off, codes, at in ((O_KC, kc, _key_nibbles()), (O_VC, vc.reshape(*lead, PAGE, D), _value_nibbles())):
        nib = torch.empty(*lead, PAGE * D, dtype=torch.uint8, device=k.device)
        nib[..., at.reshape(-1)] = codes.reshape(*lead, -1)
        rec[..., off:off + 4096] = nib[..., 0::2] | nib[..., 1::2] << 4
    for off, s, z, at in ((0, ks, kz, _key_params()), (O_VS, vs, vz, _value_params())):
        n = at.numel()
        both = torch.empty(*lead, 2 * n, dtype=torch.float16, device=k.device)
        both[..., at.reshape(-1)] = s.reshape(*lead, n)
        both[..., at.reshape(-1) + n] = z.reshape(*lead, n)
        rec[..., off:off + 4 * n] = both.view(torch.uint8)
    return rec


def _values(rec):
    """fp32 keys and values [...][64][128] of records."""
    lead = rec.shape[:-1]

    def codes(off, at):
        b = rec[..., off:off + 4096]
        return torch.stack((b & 15, b >> 4), -1).reshape(*lead, PAGE * D)[..., at.reshape(-1)].reshape(*lead, PAGE, D).float()

    def params(off, at):
        n = at.numel()
        both = rec[..., off:off + 4 * n].contiguous().view(torch.float16).float()
        return (both[..., at.reshape(-1) + i * n].reshape(*lead, *at.shape) for i in (0, 1))

    ks, kz = params(0, _key_params())
    vs, vz = params(O_VS, _value_params())
    k = codes(O_KC, _key_nibbles()) * ks.unsqueeze(-2) + kz.unsqueeze(-2)
    v = codes(O_VC, _value_nibbles()) * vs.repeat_interleave(32, -1) + vz.repeat_interleave(32, -1)
    return k, v


def _swizzle(x):
    """Tail rows [...][slots][128] with chunk c of slot t at c ^ (t % 8) (its own inverse)."""
    at = torch.arange(16, device=x.device) ^ (torch.arange(x.shape[-2], device=x.device) % 8)[:, None]
    y = x.reshape(*x.shape[:-1], 16, 8)
    return y.gather(-2, at[..., None].expand(y.shape)).reshape(x.shape)


def _cache(case, seed, n, k, v, starts):
    """Pages, table, tails and lengths of sequences whose first n[b] tokens, from row
    starts[b] of k and v on, are cached; some pages of the pool stay free."""
    nq = _packed(n)
    b, hkv = len(n), k.shape[1]
    used = int(nq.sum()) // PAGE
    room = int(nq.max()) // PAGE + 32
    n_pages = used + 40 * b
    order = torch.randperm(n_pages, generator=_gen(seed + 3), device="cuda")
    table = torch.full((b, room), -1, dtype=torch.int32, device="cuda")
    pages = torch.zeros(n_pages, hkv, REC, dtype=torch.uint8, device="cuda")
    tail_k, tail_v = (torch.zeros(b, hkv, PAGE, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    at = 0
    for i in range(b):
        groups = int(nq[i]) // PAGE
        mine = order[at:at + groups + 32]
        at += groups + 32
        table[i, :groups + 32] = mine.int()
        for g in range(0, groups, 256):
            m = min(256, groups - g)
            rows = slice(int(starts[i]) + g * PAGE, int(starts[i]) + (g + m) * PAGE)
            kg, vg = (x[rows].view(m, PAGE, hkv, D).transpose(1, 2) for x in (k, v))
            pages[mine[g:g + m]] = _records(kg, vg)
        rest = slice(int(starts[i] + nq[i]), int(starts[i] + n[i]))
        tail_k[i, :, :int(n[i] - nq[i])] = k[rest].transpose(0, 1)
        tail_v[i, :, :int(n[i] - nq[i])] = v[rest].transpose(0, 1)
    return {"pages": pages, "table": table, "tail_k": _swizzle(tail_k), "tail_v": _swizzle(tail_v)}


def _positions(case, seed):
    return torch.randint(0, case["far"], (case["tokens"],), generator=_gen(seed + 1), device="cuda", dtype=torch.int32)


def _rope_inputs(case, seed):
    g = _gen(seed)
    h, hkv = case["heads"], case["kv_heads"]
    qkv = _normal(g, case["tokens"], h + 2 * hkv, D).bfloat16()   # one projection's output: q, k, v heads
    w = [(1 + 0.2 * _normal(g, D)).bfloat16() if case["norm"] else None for _ in range(2)]
    return qkv[:, :h], qkv[:, h:h + hkv], w[0], w[1], _positions(case, seed)


SCALINGS = {"none": {}, "linear": {"factor": 4.0},
            "llama3": {"factor": 8.0, "low_freq_factor": 1.0, "high_freq_factor": 4.0, "original": 8192},
            "yarn": {"factor": 16.0, "beta_fast": 32.0, "beta_slow": 1.0, "original": 16384}}
BASE = 500000.0
EPS = 1e-6


def _pairs(case):
    """(parent, child) rows of a fork: the first rows are the parents, taken in turn."""
    child = np.arange(case["parents"], case["batch"])
    return np.stack((child % case["parents"], child), 1)


def _tail_of(case, row):
    return 1 + row * 37 % PAGE


def prepare(case, seed):
    s = {"case": case}
    if case["op"] == "rope":
        q, k, wq, wk, pos = _rope_inputs(case, seed)
        s.update(q=q, k=k, wq=wq, wk=wk, pos=pos, freq=_frequencies(case))
    elif case["op"] == "append":
        n = _lens(case)
        new = case["new"]
        k, v = _rows(case, seed)
        starts = np.cumsum(n) - n
        s.update(_cache(case, seed, n - new, k, v, starts))
        fresh = torch.as_tensor((starts[:, None] + n[:, None] - new + np.arange(new)).reshape(-1), device="cuda")
        both = torch.stack((k[fresh], v[fresh]), 1)               # k and v of one projection, side by side
        s.update(k=both[:, 0], v=both[:, 1], lens=_ints(n), cu=_ints(np.arange(case["batch"] + 1) * new),
                 out_cu=_ints(np.concatenate(([0], np.cumsum(n)))), total=int(n.sum()))
        s["plan"] = _append_plan(n, new)
    elif case["op"] == "attend":
        n = _lens(case)
        k, v = _rows(case, seed)
        s.update(_cache(case, seed, n, k, v, np.cumsum(n) - n), lens=_ints(n), q=_q(case, seed))
    else:
        g = _gen(seed)
        b, hkv, p = case["batch"], case["kv_heads"], case["pages"]
        words = torch.randint(-2**31, 2**31, (p, hkv, REC // 4), generator=g, device="cuda", dtype=torch.int32)
        tails = [_normal(g, b, hkv, PAGE, D).bfloat16() for _ in range(2)]
        order = torch.randperm(p, generator=g, device="cuda").cpu().numpy()
        src = np.sort(order)[::-1][:case["moves"]]                # the last pages in use ...
        dst = np.sort(order)[:case["moves"]]                      # ... to the first free ones
        live = np.setdiff1d(order, dst)
        per = max(1, len(live) // b)
        table = np.full((b, per), -1)
        flat = np.random.RandomState(seed % 2**32).permutation(live)
        for i in range(b):
            row = flat[i * per:(i + 1) * per]
            table[i, :len(row)] = row
        lens = np.array([(table[i] >= 0).sum() * PAGE + _tail_of(case, i) for i in range(b)])
        goes = np.arange(p)
        goes[src] = dst
        s.update(pages=words.view(torch.uint8), tail_k=tails[0], tail_v=tails[1], table=_ints(table), lens=_ints(lens),
                 pairs=_ints(_pairs(case)), moves=_ints(np.stack((src, dst), 1)), goes=_ints(goes),
                 wide=torch.arange(PAGE, device="cuda"))
    if own:
        _handle(s)
    return s


# --------------------------------------------------------------------------
# the package's calls
# --------------------------------------------------------------------------
def _handle(s):
    """The objects a program keeps between calls: rotary plan, cache, workspace."""
    import bit_kv_cache_jfa_b200 as jfa

    case = s["case"]
    s["jfa"] = jfa
    if case["op"] == "rope":
        s["rotary"] = jfa.RotaryPlan(case["rotary"], base=BASE, interleaved=case["interleaved"],
                                     scaling=case["scaling"], **SCALINGS[case["scaling"]])
        return
    rows, room = s["table"].shape
    table = jfa.PageTable(rows, s["pages"].shape[0], room)
    cache = jfa.PagedKVCache(table, case.get("heads", case["kv_heads"]), case["kv_heads"])
    for to, of in ((table.table, "table"), (table.seq_lens, "lens"), (cache.pages, "pages"),
                   (cache.tail_k, "tail_k"), (cache.tail_v, "tail_v")):
        to.copy_(s.pop(of))
    s["cache"], s["ws"] = cache, jfa.PagedWorkspace(cache)


def _own(s):
    jfa, case = s["jfa"], s["case"]
    if case["op"] == "rope":
        return jfa.qk_norm_rope(s["q"], s["k"], s["pos"], s["rotary"], s["wq"], s["wk"], eps=EPS)
    cache, ws = s["cache"], s["ws"]
    if case["op"] == "attend":
        return jfa.paged_attend(cache, s["q"], ws, window=case["window"], sinks=case["sinks"])
    if case["op"] == "append":
        jfa.paged_append(cache, s["k"], s["v"], ws, s["cu"])
        k, v = jfa.paged_gather(cache, s["out_cu"], s["total"], ws)
        return k, v, cache.tail_k, cache.tail_v
    jfa.paged_fork(cache, s["pairs"], ws)
    jfa.paged_move(cache, s["moves"], ws, s["goes"])
    return cache.pages.view(torch.int32), cache.tail_k, cache.tail_v, cache.table.table, cache.table.seq_lens


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------
def _frequencies(case):
    """Angles per position, float64 [rotary / 2]."""
    r, a = case["rotary"], SCALINGS[case["scaling"]]
    i = torch.arange(r // 2, dtype=torch.float64, device="cuda")
    f = BASE ** (-2 * i / r)
    if case["scaling"] == "linear":
        return f / a["factor"]
    if case["scaling"] == "llama3":
        turns = a["original"] * f / (2 * math.pi)                  # of the original context
        mix = ((turns - a["low_freq_factor"]) / (a["high_freq_factor"] - a["low_freq_factor"])).clamp(0, 1)
        return f * (mix + (1 - mix) / a["factor"])
    if case["scaling"] == "yarn":
        at = [r * math.log(a["original"] / (b * 2 * math.pi)) / (2 * math.log(BASE))
              for b in (a["beta_fast"], a["beta_slow"])]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), r - 1)
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return f * (1 - ramp + ramp / a["factor"])
    return f


def _amplitude(case):
    return 0.1 * math.log(SCALINGS["yarn"]["factor"]) + 1 if case["scaling"] == "yarn" else 1.0


def _rope(x, w, cos, sin, rotary, interleaved):
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * w.float()
    turned, rest = y[..., :rotary], y[..., rotary:]
    if interleaved:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = turned[..., :rotary // 2], turned[..., rotary // 2:]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turned, rest), -1).bfloat16()


def _append_plan(n, new):
    """Where the rows of every page to be packed, and of the new tails, come from:
    places among the old tails' rows (64 a sequence) with the new rows behind them."""
    b, n0 = len(n), n - new
    q0, q1 = _packed(n0), _packed(n)

    def source(row, t):
        return np.where(t < n0[row], row * PAGE + t - q0[row], b * PAGE + row * new + t - n0[row])

    row = np.repeat(np.arange(b), (q1 - q0) // PAGE)
    group = np.concatenate([np.arange(a // PAGE, z // PAGE) for a, z in zip(q0, q1)])
    page = source(row[:, None], group[:, None] * PAGE + np.arange(PAGE))
    slot = q1[:, None] + np.arange(PAGE)
    kept = slot < n[:, None]
    tail = source(np.arange(b)[:, None], np.where(kept, slot, n[:, None] - 1))
    out_row = np.repeat(np.arange(b), n)
    out_t = np.concatenate([np.arange(m) for m in n])
    return {key: torch.as_tensor(x, device="cuda") for key, x in dict(
        row=row, group=group, page=page, kept=kept[:, None, :, None], tail=tail, out_row=out_row, out_t=out_t,
        out_packed=(out_t < q1[out_row])[:, None, None], out_slot=np.maximum(out_t - q1[out_row], 0),
        out_group=np.minimum(out_t, np.maximum(q1[out_row] - 1, 0)) // PAGE).items()}


def _plain_append(s):
    p, fresh = s["plan"], {}
    for name, tail in (("k", "tail_k"), ("v", "tail_v")):
        old = _swizzle(s[tail]).transpose(1, 2).flatten(0, 1)      # [B * 64][H_kv][128]
        fresh[name] = torch.cat((old, s[name]))
        put = fresh[name][p["tail"]].transpose(1, 2)
        s[tail].copy_(_swizzle(torch.where(p["kept"], put, old.view(-1, PAGE, *old.shape[1:]).transpose(1, 2))))
    where = s["table"].long()
    if p["row"].numel():
        pages = _records(*(fresh[x][p["page"]].transpose(1, 2) for x in "kv"))
        s["pages"][where[p["row"], p["group"]]] = pages
    # read back: the pages of every sequence in turn, then each row from its page or tail
    held, place = torch.unique(where[p["out_row"], p["out_group"]], return_inverse=True)
    got = []
    for x, tail in zip(_values(s["pages"][held]), ("tail_k", "tail_v")):
        packed = x.transpose(1, 2)[place, p["out_t"] % PAGE]
        exact_rows = _swizzle(s[tail]).transpose(1, 2)[p["out_row"], p["out_slot"]]
        got.append(torch.where(p["out_packed"], packed.bfloat16(), exact_rows))
    return got[0], got[1], s["tail_k"], s["tail_v"]


def _plain_attend(s):
    case = s["case"]
    q, lens = s["q"].float(), s["lens"].long()
    b, hkv = q.shape[0], case["kv_heads"]
    groups = s["table"].shape[1] - 32
    nq = torch.clamp(lens - 1, min=0) // PAGE * PAGE
    k, v = (x.permute(0, 2, 1, 3, 4).flatten(2, 3) for x in _values(s["pages"][s["table"][:, :groups].long().clamp(min=0)]))
    k = torch.cat((k, _swizzle(s["tail_k"]).float()), 2)
    v = torch.cat((v, _swizzle(s["tail_v"]).float()), 2)
    at = torch.arange(groups * PAGE + PAGE, device="cuda")
    in_tail = at >= groups * PAGE
    t = torch.where(in_tail, at - groups * PAGE + nq[:, None], at)  # the token in each place, by sequence
    there = torch.where(in_tail, t < lens[:, None], t < nq[:, None])
    if case["window"]:
        there = there & ((t >= lens[:, None] - case["window"]) | (t < case["sinks"]))
    there = there[:, None, None, :]
    x = (q.view(b, hkv, -1, D) / math.sqrt(D)) @ k.transpose(2, 3)
    x = x.masked_fill(~there, -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(x - m)
    out = p @ v / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return out.view(b, -1, D).bfloat16()


def _plain_pages(s):
    src, dst = s["pairs"].long().unbind(1)
    count = (s["lens"].long() - 1) % PAGE + 1
    kept = (s["wide"] < count[src, None])[:, None, :, None]
    for tail in (s["tail_k"], s["tail_v"]):
        tail[dst] = torch.where(kept, tail[src], tail[dst])
    s["table"][dst] = s["table"][src]
    s["lens"][dst] = s["lens"][src]
    src, dst = s["moves"].long().unbind(1)
    s["pages"][dst] = s["pages"][src]
    held = torch.arange(s["table"].shape[1], device="cuda") < (s["lens"].long()[:, None] - 1) // PAGE
    s["table"].copy_(torch.where(held, s["goes"][s["table"].long().clamp(min=0)], s["table"]))
    return s["pages"].view(torch.int32), s["tail_k"], s["tail_v"], s["table"], s["lens"]


def run(state):
    if own:
        return _own(state)
    case = state["case"]
    if case["op"] == "rope":
        angle = state["pos"].double()[:, None] * state["freq"]
        cos, sin = (f(angle).float()[:, None] * _amplitude(case) for f in (torch.cos, torch.sin))
        return tuple(_rope(x, w, cos, sin, case["rotary"], case["interleaved"])
                     for x, w in ((state["q"], state["wq"]), (state["k"], state["wk"])))
    return {"append": _plain_append, "attend": _plain_attend, "pages": _plain_pages}[case["op"]](state)


# --------------------------------------------------------------------------
# in 64 bits, from the definitions
# --------------------------------------------------------------------------
def _exact_rope(case, seed):
    q, k, wq, wk, pos = _rope_inputs(case, seed)
    r, a = case["rotary"], SCALINGS[case["scaling"]]
    f = []
    for i in range(r // 2):
        w = BASE ** (-2.0 * i / r)
        if case["scaling"] == "linear":
            w /= a["factor"]
        elif case["scaling"] == "llama3":
            length = 2 * math.pi / w
            if length > a["original"] / a["low_freq_factor"]:
                w /= a["factor"]
            elif length >= a["original"] / a["high_freq_factor"]:
                u = (a["original"] / length - a["low_freq_factor"]) / (a["high_freq_factor"] - a["low_freq_factor"])
                w = (1 - u) * w / a["factor"] + u * w
        elif case["scaling"] == "yarn":
            def dim(turns):
                return r * math.log(a["original"] / (turns * 2 * math.pi)) / (2 * math.log(BASE))
            first, last = max(math.floor(dim(a["beta_fast"])), 0), min(math.ceil(dim(a["beta_slow"])), r - 1)
            u = min(max((i - first) / max(last - first, 1e-3), 0), 1)
            w = u * w / a["factor"] + (1 - u) * w
        f.append(w)
    turn = torch.polar(torch.full((len(f),), _amplitude(case), dtype=torch.float64, device="cuda"),
                       pos.double()[:, None, None] * torch.tensor(f, dtype=torch.float64, device="cuda"))
    outs = []
    for x, w in ((q, wq), (k, wk)):
        y = x.double()
        if w is not None:
            y = w.double() * y / (y.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt()
        shape = y.shape[:-1]
        first = y[..., :r].reshape(*shape, r // 2, 2) if case["interleaved"] else \
            y[..., :r].reshape(*shape, 2, r // 2).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(first.contiguous()) * turn)
        z = z if case["interleaved"] else z.transpose(-1, -2)
        y[..., :r] = z.reshape(*shape, r)
        outs.append(y)
    return tuple(outs)


def _stored(x, cols):
    """What 4 bits keep of x [m][64][H_kv][128]: groups of 64 tokens of a channel
    (cols = False) or of 32 channels of a token, in 64 bits."""
    y = x.double()
    m, _, h, _ = y.shape
    y = y.reshape(m, PAGE, h, 4, 32) if cols else y
    dim = 4 if cols else 1

    def half(z, up):
        # 11 significant bits, at least 2^-24 apart
        unit = torch.exp2((torch.frexp(z)[1] - 11).clamp(min=-24).double())
        return (torch.ceil(z / unit) if up else torch.floor(z / unit)) * unit

    zero = half(y.min(dim, keepdim=True).values, False)
    step = half((y.max(dim, keepdim=True).values - zero) / 15, True)
    code = ((y - zero) / step.clamp(min=2.0**-24)).round().clamp(0, 15)
    return (zero + torch.where(step > 0, code * step, 0.0)).reshape(x.shape)


def _kept_rows(k, v, n, starts):
    """Per sequence its rows as the cache stands for them, float64 [n][H_kv][128]."""
    for length, a in zip(n.tolist(), starts.tolist()):
        nq = int(_packed(np.int64(length)))
        both = []
        for x, cols in ((k, False), (v, True)):
            y = x[a:a + length]
            packed = y[:nq].reshape(nq // PAGE, PAGE, *y.shape[1:])
            both.append(torch.cat((_stored(packed, cols).reshape(nq, *y.shape[1:]), y[nq:].double())))
        yield both


def _exact_append(case, seed):
    n = _lens(case)
    k, v = _rows(case, seed)
    rows = list(_kept_rows(k, v, n, np.cumsum(n) - n))
    return torch.cat([r[0] for r in rows]), torch.cat([r[1] for r in rows]), None, None


def _exact_attend(case, seed):
    n = _lens(case)
    k, v = _rows(case, seed)
    q = _q(case, seed).double()
    hkv = case["kv_heads"]
    out = torch.zeros(case["batch"], case["heads"], D, dtype=torch.float64, device="cuda")
    lo, sink = _seen(n, case["window"], case["sinks"])
    for i, (kk, vv) in enumerate(_kept_rows(k, v, n, np.cumsum(n) - n)):
        if n[i] == 0:
            continue
        seen = torch.cat((torch.arange(sink[i], device="cuda"), torch.arange(lo[i], n[i], device="cuda")))
        kk, vv = kk[seen].transpose(0, 1), vv[seen].transpose(0, 1)
        x = q[i].view(hkv, -1, D) @ kk.transpose(1, 2) * D ** -0.5
        out[i] = (torch.softmax(x, -1) @ vv).view(-1, D)
    return out


def exact(case, seed):
    """What run() returns on these inputs, from the definitions in 64 bits; whole
    numbers and copied bits (the page operations, the tails) have no such value."""
    if case["op"] == "rope":
        return _exact_rope(case, seed)
    if case["op"] == "append":
        return _exact_append(case, seed)
    if case["op"] == "attend":
        return _exact_attend(case, seed)
    return None
