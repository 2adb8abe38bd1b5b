"""Plain forms and timed cases of the operators that a hybrid model's layers need around a replay.

The recurrences: a gated linear recurrence over packed sequences (``linrec``) and its gradients
(``linrec_back``).  The full-attention layers between two replay groups: appending rotated keys and
values to a paged 8-bit cache (``append``) and attention over that cache (``attend``), for single
tokens and for the unmatched tokens behind a cached prefix.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
# A block's scale is the least power of two with amax <= 449 scale: what lies between 448 and 449 rounds to 448, and no
# 16-bit input lies on that border.
BORDER = 449.0
SCALE_EXP_MIN, SCALE_EXP_MAX = -32, 32
ROPE_THETA = 1.0e6


# ---------------------------------------------------------------- cases


def listed():
    rec = dict(op="linrec", lens=1, dtype="bf16", g="fp32", h0=True)
    back = dict(rec, op="linrec_back")
    app = dict(op="append", lens=1, rot=64, axes=1, interleaved=False, page=64)
    att = dict(op="attend", lens=1, page=64)
    return [
        # one token for each of 64 running requests: the latency of a decode step
        dict(rec, name="linrec_step", seqs=64, lo=1, hi=1, channels=2560),
        # eight replayed suffixes of unequal lengths, as wide as 32 heads of 128
        dict(rec, name="linrec_ragged", seqs=8, lo=512, hi=2048, channels=4096),
        # one long prefill in 32 bits: the scan along one sequence
        dict(rec, name="linrec_long_fp32", seqs=1, lo=32768, hi=32768, channels=2560, dtype="fp32", h0=False),
        # training on packed samples of unequal lengths, every tensor in 16 bits
        dict(back, name="linrec_back_ragged", seqs=8, lo=512, hi=2048, channels=4096, g="bf16"),
        # training on one long sample
        dict(back, name="linrec_back_long", seqs=1, lo=32768, hi=32768, channels=2560),
        # one new token for each of 64 running requests
        dict(app, name="append_step", seqs=64, new_lo=1, new_hi=1, past_lo=255, past_hi=4095, h_q=16, h_kv=4, d=256),
        # the new tokens of eight requests, positions along time, height and width
        dict(app, name="append_extend_axes", seqs=8, new_lo=512, new_hi=2048, past_lo=0, past_hi=4096, h_q=32, h_kv=8,
             d=128, rot=128, axes=3),
        # one request's next token over a short prefix: latency
        dict(att, name="attend_step_one", seqs=1, new_lo=1, new_hi=1, past_lo=819, past_hi=819, h_q=16, h_kv=4, d=256),
        # the next token of 64 running requests of unequal lengths
        dict(att, name="attend_step_ragged", seqs=64, new_lo=1, new_hi=1, past_lo=255, past_hi=4095, h_q=16, h_kv=4, d=256),
        # a few long requests, 32K tokens cached each
        dict(att, name="attend_step_long", seqs=8, new_lo=1, new_hi=1, past_lo=30000, past_hi=32768, h_q=32, h_kv=8, d=128),
        # fresh prompts of unequal lengths, nothing cached before them
        dict(att, name="attend_prompts", seqs=8, new_lo=512, new_hi=2048, past_lo=0, past_hi=0, h_q=32, h_kv=8, d=128),
        # 1639 unmatched tokens behind a cached prefix of 32K
        dict(att, name="attend_extend_32k", seqs=1, new_lo=1639, new_hi=1639, past_lo=32768, past_hi=32768, h_q=16, h_kv=4, d=256),
    ]


def draw(rng):
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    op = rng.choice(["linrec", "linrec_back", "append", "attend", "attend"])
    lens = rng.randrange(1 << 30)
    if op.startswith("linrec"):
        seqs, channels = log(1, 128), log(64, 5120)
        if rng.random() < 0.7:
            channels = max(64, channels // 8 * 8)
        hi = max(1, min(32768, (80 << 20) // (seqs * channels)))
        hi = 1 if rng.random() < 0.2 else log(1, hi)
        dtype = rng.choice(["bf16", "fp32"])
        return dict(op=op, lens=lens, seqs=seqs, lo=max(1, hi // log(1, 16)), hi=hi, channels=channels, dtype=dtype,
                    g="fp32" if dtype == "fp32" else rng.choice(["bf16", "fp32"]), h0=rng.random() < 0.5)
    d = rng.choice([64, 128, 256])
    h_kv = rng.choice([1, 2, 4, 8])
    h_q = h_kv * rng.choice([1, 2, 3, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    if rng.random() < 0.5:
        seqs, new_hi, past_hi = log(1, 64), rng.choice([1, 1, 2, 4]), log(16, 32768)
    else:
        seqs, new_hi, past_hi = log(1, 16), log(8, 2048), log(16, 32768)
    # bounds of the cached bytes and of the scores
    while seqs > 1 and (seqs * (past_hi + new_hi) * h_kv * d > (1 << 28) or
                        seqs * (past_hi + new_hi) * new_hi * h_q > (13 << 26)):
        seqs //= 2
    while (past_hi + new_hi) * new_hi * h_q > (13 << 26):
        past_hi //= 2
        new_hi = (new_hi + 1) // 2
    case = dict(op=op, lens=lens, seqs=seqs, new_lo=max(1, new_hi // 4), new_hi=new_hi, past_lo=past_hi // log(1, 16),
                past_hi=past_hi, h_q=h_q, h_kv=h_kv, d=d, page=page)
    if op == "append":
        case.update(rot=rng.choice([d, d // 2, d // 4]), axes=rng.choice([1, 3]), interleaved=rng.random() < 0.5)
    return case


def _lengths(case, lo, hi, salt):
    r = random.Random(case["lens"] * 2 + salt)
    return [r.randint(case[lo], case[hi]) for _ in range(case["seqs"])]


def _sections(case):
    """Rotated pairs of each position axis: time takes what height and width leave."""
    half = case["rot"] // 2
    if case["axes"] == 1:
        return [half]
    side = half * 3 // 8
    return [half - 2 * side, side, side]


_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp32": 4}


# ---------------------------------------------------------------- inputs


def _cu(lens, dev):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device=dev)


def _quantise(x, dims):
    """x as e4m3 times a power of two, one for each block (the dims reduced over)."""
    m, e = torch.frexp(x.abs().amax(dims, keepdim=True))
    e = torch.where(m <= BORDER / 512, e - 9, e - 8).clamp(SCALE_EXP_MIN, SCALE_EXP_MAX)
    scale = torch.ldexp(torch.ones_like(m), e)
    return (x / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    randn = lambda *shape: torch.randn(*shape, generator=gen, device=dev)
    if case["op"].startswith("linrec"):
        lens = _lengths(case, "lo", "hi", 0)
        T, D, N = sum(lens), case["channels"], case["seqs"]
        st = dict(case=case, cu=_cu(lens, dev), max_len=max(lens), h0=None)
        x = randn(T, D).to(_TYPES[case["dtype"]])
        # decays from a thousand tokens' memory down to one token's
        u = torch.rand(T, D, generator=gen, device=dev)
        g = (-torch.exp(u * math.log(1e3) - math.log(1e3))).to(_TYPES[case["g"]])
        if case["h0"]:
            st["h0"] = randn(N, D)
        st.update(x=x, g=g)
        if case["op"] == "linrec_back":
            # the outputs that the forward pass kept, and the gradients that arrive
            st["y"] = _linrec(st)[0]
            st["dy"] = randn(T, D).to(x.dtype)
            st["ds"] = randn(N, D)
        return st
    new, past = _lengths(case, "new_lo", "new_hi", 0), _lengths(case, "past_lo", "past_hi", 1)
    N, page, h_kv, d = case["seqs"], case["page"], case["h_kv"], case["d"]
    T, total = sum(new), [a + b for a, b in zip(new, past)]
    per = [(n + page - 1) // page for n in total]
    n_pages = sum(per) + 3
    order = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    table = torch.zeros(N, max(per), dtype=torch.int32, device=dev)
    at = 0
    for n, p in enumerate(per):
        table[n, :p] = order[at:at + p]
        at += p
    # keys and values differ in size from head to head and drift along the pages
    size = torch.exp(0.5 * randn(n_pages, h_kv, 1, 1))
    kc, ks = _quantise(randn(n_pages, h_kv, page, d) * size, (2, 3))
    vc, vs = _quantise(randn(n_pages, h_kv, page, d) * size, (2, 3))
    st = dict(case=case, cu=_cu(new, dev), kv_lens=torch.tensor(total, dtype=torch.int32, device=dev), table=table,
              k_cache=kc, v_cache=vc, k_scale=ks.view(n_pages, h_kv), v_scale=vs.view(n_pages, h_kv), max_new=max(new),
              max_kv=max(total))
    st["q"] = (1.5 * randn(T, case["h_q"], d)).to(torch.bfloat16)
    if case["op"] == "append":
        st["k"] = (2.0 * randn(T, h_kv, d)).to(torch.bfloat16)
        st["v"] = randn(T, h_kv, d).to(torch.bfloat16)
        half = case["rot"] // 2
        st["inv_freq"] = (ROPE_THETA ** (-torch.arange(half, dtype=torch.float64) / half)).float().to(dev)
        # text goes on along all axes; a picture's tokens share a time and spread over height and width
        time = torch.cat([torch.arange(p, p + n) for p, n in zip(past, new)])
        axes = [time] if case["axes"] == 1 else [time - time % 256, time // 16 % 16 + time, time % 16 + time]
        st["positions"] = torch.stack(axes).to(torch.int32).to(dev)
    return st


# ---------------------------------------------------------------- plain forms


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 0, by doubling: after step s every row holds the last 2s tokens."""
    s = 1
    while s < a.shape[0]:
        b = torch.cat([b[:s], torch.addcmul(b[s:], a[s:], b[:-s])])
        a = torch.cat([a[:s], a[s:] * a[:-s]])
        s *= 2
    return b


def _linrec(st):
    x, cu = st["x"].float(), st["cu"].long()
    a = torch.exp(st["g"].float())
    first, last = cu[:-1], cu[1:] - 1
    b = x
    if st["h0"] is not None:
        b = x.clone()
        b[first] += a[first] * st["h0"]
    a[first] = 0.0
    h = _scan(a, b)
    return h.to(st["x"].dtype), h[last].clone()


def _linrec_back(st):
    cu, dt = st["cu"].long(), st["x"].dtype
    first, last = cu[:-1], cu[1:] - 1
    a = torch.exp(st["g"].float())
    b = st["dy"].float()
    b[last] += st["ds"]
    nxt = torch.cat([a[1:], a[:1]])
    nxt[last] = 0.0
    dh = _scan(nxt.flip(0), b.flip(0)).flip(0)
    y = st["y"].float()
    prev = torch.cat([y[:1], y[:-1]])
    prev[first] = 0.0 if st["h0"] is None else st["h0"]
    pull = dh * a
    return dh.to(dt), (pull * prev).to(st["g"].dtype), pull[first].clone()


def _rotate(x, st):
    """x [T, heads, d] turned pair by pair by its token's angles; the angles in 64 bits, as positions are far."""
    case = st["case"]
    half = case["rot"] // 2
    axis = torch.repeat_interleave(torch.arange(case["axes"], device=x.device),
                                   torch.tensor(_sections(case), device=x.device))
    angle = st["positions"].double()[axis].T * st["inv_freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    x = x.float()
    r = x[..., :2 * half]
    if case["interleaved"]:
        lo, hi = r[..., 0::2], r[..., 1::2]
        r = torch.stack([lo * cos - hi * sin, lo * sin + hi * cos], -1).flatten(-2)
    else:
        lo, hi = r[..., :half], r[..., half:]
        r = torch.cat([lo * cos - hi * sin, lo * sin + hi * cos], -1)
    return torch.cat([r, x[..., 2 * half:]], -1)


def _put(x, cache, scale, st):
    """Writes x [T, h_kv, d] behind the cached tokens: a page keeps the larger of its scale and what the new tokens
    need, and its older values are rounded again where that grew."""
    page = st["case"]["page"]
    T, h, d = x.shape
    cu, dev = st["cu"].long(), x.device
    new = cu[1:] - cu[:-1]
    seq = torch.repeat_interleave(torch.arange(new.numel(), device=dev), new)
    start = st["kv_lens"].long() - new
    pos = start[seq] + torch.arange(T, device=dev) - cu[seq]
    at = st["table"].long()[seq, pos // page]
    amax = torch.full_like(scale, 2.0 ** -40).index_reduce_(0, at, x.abs().amax(-1), "amax")
    m, e = torch.frexp(amax)
    e = torch.where(m <= BORDER / 512, e - 9, e - 8).clamp(SCALE_EXP_MIN, SCALE_EXP_MAX)
    need = torch.ldexp(torch.ones_like(m), e)
    touched = torch.zeros(scale.shape[0], dtype=torch.bool, device=dev).index_fill_(0, at, True)
    # tokens that a page held before this call
    held = torch.zeros(scale.shape[0], dtype=torch.long, device=dev)
    held[st["table"].long()[torch.arange(new.numel(), device=dev), start // page]] = start % page
    kept = torch.where((held > 0)[:, None], torch.maximum(scale, need), need)
    kept = torch.where(touched[:, None], kept, scale)
    rows = torch.nonzero(touched & (held > 0))[:, 0]
    old = cache[rows].float() * (scale[rows] / kept[rows])[..., None, None]
    older = (torch.arange(page, device=dev) < held[rows][:, None])[:, None, :, None]
    raw = cache.view(torch.uint8)
    raw[rows] = torch.where(older, old.to(cache.dtype).view(torch.uint8), raw[rows])
    raw[at[:, None], torch.arange(h, device=dev), (pos % page)[:, None]] = (
        (x / kept[at][..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(cache.dtype).view(torch.uint8))
    scale.copy_(kept)


def _append(st):
    k = _rotate(st["k"], st)
    _put(k, st["k_cache"], st["k_scale"], st)
    _put(st["v"].float(), st["v_cache"], st["v_scale"], st)
    return _rotate(st["q"], st).to(torch.bfloat16)


def _attend(st):
    case, dev = st["case"], st["q"].device
    h_q, h_kv, d = case["h_q"], case["h_kv"], case["d"]
    cu, kv = st["cu"].long(), st["kv_lens"].long()
    new = cu[1:] - cu[:-1]
    N, Lq = new.numel(), st["max_new"]
    table = st["table"].long()
    k = (st["k_cache"][table].float() * st["k_scale"][table][..., None, None]).transpose(1, 2).reshape(N, h_kv, -1, d)
    v = (st["v_cache"][table].float() * st["v_scale"][table][..., None, None]).transpose(1, 2).reshape(N, h_kv, -1, d)
    i = torch.arange(Lq, device=dev)
    row = (cu[:-1, None] + torch.minimum(i, (new - 1)[:, None]))
    q = st["q"][row].float().view(N, Lq, h_kv, h_q // h_kv, d).permute(0, 2, 3, 1, 4).reshape(N, h_kv, -1, d)
    s = (q @ k.transpose(-1, -2)).view(N, h_kv, -1, Lq, k.shape[2]) * (d ** -0.5)
    seen = torch.arange(k.shape[2], device=dev) <= ((kv - new)[:, None] + i)[..., None]
    s = s.masked_fill_(~seen[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (top + torch.log(total)).squeeze(-1)
    o = (p.view(N, h_kv, -1, k.shape[2]) @ v).view(N, h_kv, -1, Lq, d) / total
    real = i < new[:, None]
    o = o.permute(0, 3, 1, 2, 4)[real].reshape(-1, h_q, d)
    return o.to(torch.bfloat16), lse.permute(0, 3, 1, 2)[real].reshape(-1, h_q)


# ---------------------------------------------------------------- one pass


def run(st):
    case = st["case"]
    if own:
        import gated_deltanet_state_sr_b200 as sr
    if case["op"] == "linrec":
        if own:
            y, s = sr.linrec_replay(st["x"], st["g"], st["cu"], max_seqlen=st["max_len"], h0=st["h0"])
        else:
            y, s = _linrec(st)
        return {"y": y, "state": s}
    if case["op"] == "linrec_back":
        if own:
            dx, dg, dh0 = sr.linrec_backward(st["g"], st["y"], st["dy"], st["cu"], max_seqlen=st["max_len"], h0=st["h0"],
                                             ds=st["ds"])
        else:
            dx, dg, dh0 = _linrec_back(st)
        return {"dx": dx, "dg": dg, "dh0": dh0}
    if case["op"] == "append":
        if own:
            q = sr.kv_append(st["k"], st["v"], st["cu"], st["kv_lens"], st["table"], st["k_cache"], st["v_cache"],
                             st["k_scale"], st["v_scale"], max_seqlen=st["max_new"], q=st["q"], inv_freq=st["inv_freq"],
                             positions=st["positions"], sections=_sections(case), interleaved=case["interleaved"])
        else:
            q = _append(st)
        return {"q": q, "k_cache": st["k_cache"], "v_cache": st["v_cache"], "k_scale": st["k_scale"],
                "v_scale": st["v_scale"]}
    if own:
        o, lse = sr.paged_attention(st["q"], st["cu"], st["kv_lens"], st["table"], st["k_cache"], st["v_cache"],
                                    st["k_scale"], st["v_scale"], max_seqlen=st["max_new"], max_kvlen=st["max_kv"],
                                    want_lse=True)
    else:
        o, lse = _attend(st)
    return {"o": o, "lse": lse}


def work(case):
    if case["op"].startswith("linrec"):
        n = sum(_lengths(case, "lo", "hi", 0)) * case["channels"]
        states = case["seqs"] * case["channels"] * 4
        x, g = _BYTES[case["dtype"]], _BYTES[case["g"]]
        if case["op"] == "linrec":
            return {"bytes": n * (2 * x + g) + states * (2 if case["h0"] else 1), "flops": 3 * n}
        return {"bytes": n * (3 * x + 2 * g) + states * (3 if case["h0"] else 2), "flops": 5 * n}
    new, past = _lengths(case, "new_lo", "new_hi", 0), _lengths(case, "past_lo", "past_hi", 1)
    h_q, h_kv, d, page = case["h_q"], case["h_kv"], case["d"], case["page"]
    T = sum(new)
    if case["op"] == "append":
        pages = sum((a + b + page - 1) // page - b // page for a, b in zip(new, past))
        # 16-bit queries there and back, keys and values read in 16 bits and written in 8, a page's scales
        return {"bytes": T * d * (4 * h_q + 6 * h_kv) + 16 * pages * h_kv + 4 * T * case["axes"],
                "flops": 3 * T * case["rot"] * (h_q + h_kv) + 4 * T * d * h_kv}
    pairs = sum(a * b + a * (a + 1) // 2 for a, b in zip(new, past))
    pages = sum((a + b + page - 1) // page for a, b in zip(new, past))
    return {"bytes": sum(new + past) * h_kv * d * 2 + pages * (h_kv * 8 + 4) + T * h_q * (4 * d + 4),
            "flops": 4 * pairs * h_q * d}


# ---------------------------------------------------------------- the definitions in 64 bits


def _exact_linrec(st):
    """Token by token, all sequences at a time."""
    cu = st["cu"].long()
    lens = cu[1:] - cu[:-1]
    x, g = st["x"], st["g"]
    h = torch.zeros(lens.numel(), x.shape[1], dtype=torch.float64, device=x.device)
    if st["h0"] is not None:
        h += st["h0"]
    y = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    order = torch.argsort(lens, descending=True, stable=True)
    starts, sizes = cu[:-1][order], lens[order].tolist()
    h = h[order]
    live = len(sizes)
    for t in range(max(sizes)):
        while sizes[live - 1] <= t:
            live -= 1
        at = starts[:live] + t
        h[:live] = torch.addcmul(x[at].double(), g[at].double().exp_(), h[:live])
        y[at] = h[:live]
    out = torch.empty_like(h)
    out[order] = h
    return {"y": y, "state": out}


def _exact_linrec_back(st):
    cu = st["cu"].long()
    lens = cu[1:] - cu[:-1]
    g, y, dy = st["g"], st["y"], st["dy"]
    order = torch.argsort(lens, descending=True, stable=True)
    ends, starts, sizes = cu[1:][order] - 1, cu[:-1][order], lens[order].tolist()
    dh = st["ds"].double()[order]
    h0 = torch.zeros_like(dh) if st["h0"] is None else st["h0"].double()[order]
    dx = torch.empty(y.shape, dtype=torch.float64, device=y.device)
    dg = torch.empty_like(dx)
    live = len(sizes)
    for t in range(max(sizes)):
        while sizes[live - 1] <= t:
            live -= 1
        at = ends[:live] - t
        grad = dh[:live] + dy[at].double()
        dx[at] = grad
        dh[:live] = grad * g[at].double().exp_()
        before = torch.where((at == starts[:live])[:, None], h0[:live], y[(at - 1).clamp_(min=0)].double())
        dg[at] = dh[:live] * before
    out = torch.empty_like(dh)
    out[order] = dh
    return {"dx": dx, "dg": dg, "dh0": out}


def _exact_turned(x, st):
    case = st["case"]
    half, x = case["rot"] // 2, x.double().clone()
    i = 0
    for axis, count in enumerate(_sections(case)):
        for _ in range(count):
            angle = st["positions"][axis].double() * float(st["inv_freq"][i])
            c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
            a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
            u, w = x[..., a].clone(), x[..., b].clone()
            x[..., a] = u * c - w * s
            x[..., b] = u * s + w * c
            i += 1
    return x


def _exact_e4m3(x):
    """Nearest multiple of the step at each value's binade, half to even; the least binade is 2**-6."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_put(x, cache, scale, st):
    page = st["case"]["page"]
    values, scale = cache.double(), scale.double().clone()
    cu, kv = st["cu"].tolist(), st["kv_lens"].tolist()
    for n, total in enumerate(kv):
        begin = total - (cu[n + 1] - cu[n])
        p = begin // page
        while p * page < total:
            a, b = max(begin, p * page), min(total, (p + 1) * page)
            at = int(st["table"][n, p])
            part = x[cu[n] + a - begin:cu[n] + b - begin].transpose(0, 1)
            old = a - p * page
            top = (part.abs().amax((1, 2)) / BORDER).clamp(min=2.0 ** -40)
            need = torch.ldexp(torch.ones_like(top), torch.ceil(torch.log2(top)).long().clamp(SCALE_EXP_MIN, SCALE_EXP_MAX))
            kept = torch.maximum(need, scale[at]) if old else need
            if old:
                values[at, :, :old] = _exact_e4m3(values[at, :, :old] * (scale[at] / kept)[:, None, None])
            values[at, :, old:old + b - a] = _exact_e4m3(part / kept[:, None, None])
            scale[at] = kept
            p += 1
    return values, scale


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "linrec":
        return _exact_linrec(st)
    if case["op"] == "linrec_back":
        return _exact_linrec_back(st)
    if case["op"] == "append":
        kc, ks = _exact_put(_exact_turned(st["k"], st), st["k_cache"], st["k_scale"], st)
        vc, vs = _exact_put(st["v"].double(), st["v_cache"], st["v_scale"], st)
        return {"q": _exact_turned(st["q"], st), "k_cache": kc, "v_cache": vc, "k_scale": ks, "v_scale": vs}
    group, page, d = case["h_q"] // case["h_kv"], case["page"], case["d"]
    cu, kv = st["cu"].tolist(), st["kv_lens"].tolist()
    o = torch.empty(st["q"].shape, dtype=torch.float64, device=st["q"].device)
    lse = torch.empty(st["q"].shape[:2], dtype=torch.float64, device=st["q"].device)
    for n, total in enumerate(kv):
        pages = st["table"][n, :(total + page - 1) // page].long()
        count = cu[n + 1] - cu[n]
        limit = torch.arange(total - count, total, device=o.device)[:, None]
        hidden = torch.arange(total, device=o.device)[None] > limit
        for h in range(case["h_kv"]):
            k = (st["k_cache"][pages, h].double() * st["k_scale"][pages, h].double()[:, None, None]).reshape(-1, d)[:total]
            v = (st["v_cache"][pages, h].double() * st["v_scale"][pages, h].double()[:, None, None]).reshape(-1, d)[:total]
            for j in range(h * group, (h + 1) * group):
                s = (st["q"][cu[n]:cu[n + 1], j].double() @ k.T) / math.sqrt(d)
                s = s.masked_fill_(hidden, -math.inf)
                lse[cu[n]:cu[n + 1], j] = torch.logsumexp(s, -1)
                o[cu[n]:cu[n + 1], j] = torch.softmax(s, -1) @ v
    return {"o": o, "lse": lse}
