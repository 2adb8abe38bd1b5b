"""sr_paged_attention on the GPU against the fp64 definition (oracle.paged).

Bounds.  A weight meets the tensor cores in half precision: 2^-11 of itself.  A
score is an fp32 sum of d products (2^-23 of their magnitudes' sum each, in
whatever order), its query element exact down to 2^-9 of the row's largest and
off by 2^-17 of that below (two e4m3 numbers; half precision, for few rows, is
closer); a score's error e moves its
weight by e (1 + e).  With three roundings of fp32 sums and factors beside
(2^-20 covers them), o is within (2^-11 + 2 e + 2^-20) sum p |v| and a last
rounding to bf16, 2^-8 of itself; weights under 2^-35 of the largest are lost,
2^-35 of the largest |v| each.  lse is within e + 2^-20 (1 + |lse|)."""
import numpy as np
import pytest
import torch

from oracle import paged as O

pytestmark = pytest.mark.gpu
TABLE = O.e4m3_table()


@pytest.fixture(scope="module")
def sr():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_deltanet_state_sr_b200 as m
    return m


def np64(t):
    return t.detach().double().cpu().numpy()


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def make(new, kv, h_q=4, h_kv=2, d=64, page=16, seed=0, spare=3, q_std=2.0, scale_lo=-9, scale_hi=-6):
    gen = torch.Generator().manual_seed(seed)
    N, T = len(new), sum(new)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(int).tolist()
    per = [(t + page - 1) // page for t in kv]
    n_pages = sum(per) + spare
    order = torch.randperm(n_pages, generator=gen).tolist()
    table, at = np.full((N, max(max(per, default=0), 1)), n_pages + 7, int), 0  # entries behind the end are not read
    for n, p in enumerate(per):
        table[n, :p] = order[at:at + p]
        at += p
    c = dict(cu=cu, kv=list(kv), table=table, new=list(new), page=page, d=d, group=h_q // h_kv)
    for name in ("k", "v"):
        x = torch.randn(n_pages, h_kv, page, d, generator=gen) * 100
        c[name + "_cache"] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        e = torch.randint(scale_lo, scale_hi + 1, (n_pages, h_kv), generator=gen)
        c[name + "_scale"] = torch.ldexp(torch.ones(n_pages, h_kv), e)
    # what lies behind a sequence's end, and in pages of nobody, is garbage: NaN bytes and scales
    used = np.zeros((n_pages, page), bool)
    for n in range(N):
        for t in range(kv[n]):
            used[table[n, t // page], t % page] = True
    free = torch.tensor(~used)
    for name in ("k", "v"):
        c[name + "_cache"].transpose(1, 2)[free] = 0x7f
        c[name + "_scale"][torch.tensor(~used.any(1))] = float("nan")
    c["q"] = (q_std * torch.randn(T, h_q, d, generator=gen)).bfloat16()
    return {k: v.cuda() if torch.is_tensor(v) else v for k, v in c.items()}


def call(sr, c, **kw):
    args = dict(max_seqlen=max(c["new"]), max_kvlen=max(c["kv"]), want_lse=True)
    args.update(kw)
    return sr.paged_attention(c["q"], i32(c["cu"]), i32(c["kv"]), i32(c["table"]), c["k_cache"], c["v_cache"],
                              c["k_scale"], c["v_scale"], **args)


def check(sr, c, scale=None, **kw):
    o, lse = call(sr, c, scale=0.0 if scale is None else scale, **kw)
    q, k, v = np64(c["q"]), TABLE[c["k_cache"].cpu().numpy()], TABLE[c["v_cache"].cpu().numpy()]
    ks, vs = (np.clip(np64(c[n]), 2.0 ** -32, 2.0 ** 32) for n in ("k_scale", "v_scale"))
    used = (c["cu"], c["kv"], c["table"])
    o_ref, lse_ref = O.attention(q, *used, k, v, ks, vs, scale)
    size, _ = O.attention(q, *used, k, np.abs(v), ks, vs, scale)
    # magnitude of a score's products: |q| against the largest key magnitude of the sequence, column by column
    e = np.zeros(q.shape[:2])
    v_most = np.zeros(q.shape[:2])
    sc = c["d"] ** -0.5 if scale is None else scale
    for n in range(len(c["kv"])):
        rows = slice(c["cu"][n], c["cu"][n + 1])
        pages = c["table"][n, :(c["kv"][n] + c["page"] - 1) // c["page"]]
        if len(pages) == 0:
            continue
        kk = np.nan_to_num(np.abs(k[pages]) * ks[pages][..., None, None]).max((0, 2))
        vv = np.nan_to_num(np.abs(v[pages]) * vs[pages][..., None, None]).max((0, 2, 3))
        for h in range(q.shape[1]):
            g = h // c["group"]
            qa = np.abs(q[rows, h])
            e[rows, h] = abs(sc) * (c["d"] * 2.0 ** -23 * (qa @ kk[g]) + 2.0 ** -17 * qa.max(-1) * kk[g].sum())
            v_most[rows, h] = vv[g]
    assert e.max() < 0.05, "the bound says nothing"
    longest = max(c["kv"])
    tol = (2.0 ** -11 + 2 * e[..., None] + 2.0 ** -20) * size + 2.0 ** -8 * np.abs(o_ref) + longest * 2.0 ** -35 * v_most[..., None]
    got = np64(o)
    assert np.array_equal(np.isnan(got), np.isnan(o_ref))
    off = np.abs(got - o_ref)
    bad = off > tol
    assert not bad.any(), f"o: {bad.sum()} of {bad.size} off, worst {np.nanmax(off / np.maximum(tol, 1e-300)):.2f} bounds"
    if lse is not None:
        empty = np.isneginf(lse_ref)
        got = np64(lse)
        assert np.array_equal(np.isneginf(got), empty) and np.array_equal(np.isnan(got), np.isnan(lse_ref))
        fine = np.isfinite(lse_ref)
        assert (np.abs(got[fine] - lse_ref[fine]) <= e[fine] + 2.0 ** -20 * (1 + np.abs(lse_ref[fine]))).all()
    return o, lse


SHAPES = [(64, 16, 4, 2), (64, 64, 8, 1), (128, 64, 8, 2), (128, 16, 3, 3), (128, 128, 16, 1), (256, 32, 4, 1), (256, 64, 12, 4),
          (128, 32, 32, 1)]


@pytest.mark.parametrize("d,page,h_q,h_kv", SHAPES, ids=str)
@pytest.mark.parametrize("kv", [[1], [2, 15, 16, 17], [63, 64, 65, 128, 129], [1000, 3], [0, 40, 0]], ids=str)
def test_single_tokens(sr, d, page, h_q, h_kv, kv):
    check(sr, make([1] * len(kv), kv, h_q, h_kv, d, page, seed=d + page + len(kv)))


@pytest.mark.parametrize("d,page,h_q,h_kv", SHAPES, ids=str)
@pytest.mark.parametrize("new,kv", [([2, 4, 3], [2, 300, 64]), ([5, 0, 1], [70, 30, 9]), ([40, 7], [40, 200]),
                                    ([9, 3, 130], [5, 0, 131])], ids=str)
def test_several_tokens(sr, d, page, h_q, h_kv, new, kv):
    """Causal edges inside a step, a stage and a page; rows that see nothing (fewer cached than new tokens)."""
    check(sr, make(new, kv, h_q, h_kv, d, page, seed=d + page + len(kv)))


@pytest.mark.parametrize("d,page", [(64, 64), (128, 16), (256, 128)], ids=str)
def test_long_caches_are_shared_and_joined(sr, d, page):
    check(sr, make([1], [20011], 4, 2, d, page, seed=1))
    check(sr, make([1, 2, 1], [9000, 100, 12345], 4, 1, d, page, seed=2))


@pytest.mark.parametrize("d,h_q,h_kv,new", [(256, 8, 1, 1), (256, 9, 1, 1), (256, 4, 1, 2), (256, 4, 1, 3), (128, 8, 2, 8),
                                            (128, 8, 2, 9), (64, 32, 1, 1), (64, 33, 1, 1), (64, 4, 1, 8), (128, 8, 2, 12),
                                            (128, 8, 2, 13), (64, 48, 1, 1), (64, 49, 1, 1), (64, 6, 1, 8)], ids=str)
def test_either_side_of_the_kernels_border(sr, d, h_q, h_kv, new):
    """Eight query rows and more at head dimension 256, 32 and more below; several row tiles of the few-rows kernel."""
    check(sr, make([new, 1, new], [new, 777, 130], h_q, h_kv, d, 32, seed=h_q + new))


def test_many_requests(sr):
    rng = np.random.default_rng(3)
    kv = rng.integers(0, 400, 500).tolist()
    check(sr, make([1] * 500, kv, 4, 2, 64, 32, seed=3))
    new = rng.integers(0, 3, 500).tolist()
    check(sr, make(new, kv, 4, 2, 128, 64, seed=4))


@pytest.mark.parametrize("d,h_q,h_kv", [(256, 16, 4), (256, 16, 1), (128, 32, 8), (128, 16, 1), (64, 8, 4), (64, 12, 1)], ids=str)
def test_many_stages_in_flight(sr, d, h_q, h_kv):
    """Long and short sequences after one another in a CTA, their loads overtaking each other, several times over."""
    rng = np.random.default_rng(21)
    c = make([1] * 40, rng.integers(1, 1500, 40).tolist(), h_q, h_kv, d, 64, seed=21)
    ref = check(sr, c)
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for _ in range(5):
        flush.zero_()
        o, lse = call(sr, c)
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


def test_prompts(sr):
    check(sr, make([300, 1, 129], [300, 50, 400], 8, 2, 128, 64, seed=5))
    check(sr, make([200], [200], 4, 1, 256, 16, seed=6))


def test_sharp_and_flat_scores_and_a_scale(sr):
    check(sr, make([1, 3], [700, 80], 4, 2, 128, 64, seed=7, q_std=30.0))
    check(sr, make([1, 3], [700, 80], 4, 2, 128, 64, seed=8, q_std=1e-3))
    check(sr, make([1, 3], [700, 80], 4, 2, 128, 64, seed=9), scale=0.3)
    check(sr, make([1, 3], [700, 80], 4, 2, 128, 64, seed=10), scale=-0.05)


def test_pages_whose_scales_differ_by_much(sr):
    c = make([1, 4], [500, 300], 4, 2, 128, 16, seed=11)
    gen = torch.Generator().manual_seed(11)
    c["v_scale"] = torch.ldexp(torch.ones(c["v_scale"].shape), torch.randint(-32, 33, c["v_scale"].shape, generator=gen)).cuda()
    check(sr, c)
    c["k_scale"] = c["k_scale"] * 1.37  # a scale need not be a power of two
    c["v_scale"] = c["v_scale"].clamp(2.0 ** -20, 2.0 ** 20) * 0.77
    check(sr, c)


def test_one_token_outweighs_the_others(sr):
    """A sink: one key far above the rest, whose weights are then small but many."""
    c = make([1, 2], [6000, 3000], 2, 1, 128, 64, seed=12, q_std=0.5)
    q = c["q"].float()
    for n, t in ((0, 0), (1, 17)):
        at, s = c["table"][n, t // 64], t % 64
        row = c["cu"][n]
        k = q[row, 0] / c["k_scale"][at, 0] / q[row, 0].norm() ** 2 * 12 * 128 ** 0.5
        c["k_cache"][at, 0, s] = k.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    check(sr, c)


def test_nan_bytes_reach_the_rows_that_see_them_and_no_others(sr):
    for new, d, h_q in ((4, 128, 4), (4, 64, 2), (4, 256, 2), (150, 128, 4)):
        c = make([new, 1], [200, 90], h_q, 2, d, 64, seed=13)
        at = c["table"][0, 197 // 64]
        c["v_cache"][at, 1, 197 % 64, 5] = 0xff   # the last but two of 200: rows new-3.. of the first sequence see it
        c["v_cache"][at, 0, 199 % 64, 40] = 0x7f  # the last row alone
        o, _ = check(sr, c)
        assert bool(torch.isnan(o[new - 1]).any()) and not bool(torch.isnan(o[:new - 3]).any())
        c["k_cache"][at, 0, 198 % 64, 3] = 0x7f   # a key: the whole row of every head that it serves
        o, lse = check(sr, c)
        assert bool(torch.isnan(o[new - 1, 0]).all()) and bool(torch.isnan(lse[new - 1, 0]))


def test_nan_bytes_beside_many_rows_that_see_nothing(sr):
    """More query tiles without a cached token, between those that have some, than any ring of the kernel holds."""
    new = [200] + [130] * 40 + [200]
    c = make(new, [200] + [0] * 40 + [200], 4, 2, 128, 64, seed=22)
    for n in (0, 41):
        c["v_cache"][c["table"][n, 3], 1, 5, 9] = 0x7f  # token 197
    o, _ = check(sr, c)
    assert bool(torch.isnan(o[197:200, 2:, 9]).all()) and bool(torch.isnan(o[-3:, 2:, 9]).all()) and int(torch.isnan(o).sum()) == 12


def test_queries_that_are_not_finite_spoil_their_own_rows(sr):
    for new in ([3, 1], [40, 1]):
        c = make(new, [100, 90], 4, 2, 128, 64, seed=14)
        clean, _ = call(sr, c)
        c["q"][1, 2, 7], c["q"][new[0], 0, 0], c["q"][2, 1, 100] = float("nan"), float("inf"), float("-inf")
        o, lse = call(sr, c)
        spoilt = torch.zeros(sum(new), 4, dtype=torch.bool, device="cuda")
        spoilt[1, 2] = spoilt[new[0], 0] = spoilt[2, 1] = True
        assert bool(torch.isnan(o[spoilt]).all()) and bool(torch.isnan(lse[spoilt]).all())
        assert torch.equal(o[~spoilt], clean[~spoilt])


def test_strided_queries_no_lse_and_given_outputs(sr):
    c = make([3, 40], [100, 90], 4, 2, 128, 64, seed=15)
    o_ref, lse_ref = call(sr, c)
    wide = torch.zeros(43, 9, 128, dtype=torch.bfloat16, device="cuda")
    wide[:, 2:6] = c["q"]
    out = torch.empty_like(o_ref)
    o, lse = call(sr, dict(c, q=wide[:, 2:6]), o=out, want_lse=False)
    assert o is out and lse is None and torch.equal(o, o_ref)
    ll = torch.empty_like(lse_ref)
    assert call(sr, c, lse=ll)[1] is ll and torch.equal(ll, lse_ref)


def test_a_cache_of_more_than_4_gb(sr):
    """Pages whose bytes lie beyond 2^32."""
    page, d = 128, 128
    n_pages = (1 << 32) // (page * d) + 1000
    c = make([1, 3], [300, 129], 4, 1, d, page, seed=16)
    small = {k: c[k] for k in ("k_cache", "v_cache", "k_scale", "v_scale")}
    old = c["k_cache"].shape[0]
    far = [n_pages - 1 - 3 * i for i in range(old)]
    far[0] = 0
    o_ref, lse_ref = check(sr, c)
    for name in small:
        big = torch.zeros(n_pages, *small[name].shape[1:], dtype=small[name].dtype, device="cuda")
        big[torch.tensor(far, device="cuda")] = small[name]
        c[name] = big
    c["table"] = np.array([[far[p] if p < old else p for p in row] for row in c["table"].tolist()])
    o, lse = call(sr, c)
    assert torch.equal(o, o_ref) and torch.equal(lse, lse_ref)


@pytest.mark.parametrize("new,kv", [([1, 1, 1], [5000, 64, 900]), ([130, 1, 60], [700, 64, 60])], ids=str)
def test_same_bits_again_captured_and_on_two_streams(sr, new, kv):
    c = make(new, kv, 8, 2, 128, 64, seed=17)
    ref = call(sr, c)
    dev = dict(cu=i32(c["cu"]), kv=i32(c["kv"]), table=i32(c["table"]))
    kw = dict(max_seqlen=max(new), max_kvlen=max(kv))
    rest = (c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"])
    o, lse = torch.zeros_like(ref[0]), torch.zeros_like(ref[1])
    ws = sr.workspace(64 << 20)
    ws.fill_(255)  # whatever a workspace held before
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):  # one workspace, two calls after one another
            sr.paged_attention(c["q"], dev["cu"], dev["kv"], dev["table"], *rest, o=o, lse=lse, ws=ws, **kw)
    for _ in range(3):
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])
    assert sr.device_status(ws) == 0
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        for s in streams:  # overlapping calls, a workspace each
            outs.append(sr.paged_attention(c["q"], dev["cu"], dev["kv"], dev["table"], *rest, want_lse=True, stream=s, **kw))
    torch.cuda.synchronize()
    for a, b in outs:
        assert torch.equal(a, ref[0]) and torch.equal(b, ref[1])


def test_bad_pages_and_lengths_skip_their_sequence(sr):
    for new in ([1, 1, 1], [40, 3, 200]):
        c = make(new, [400, 90, 300], 4, 2, 128, 64, seed=18)
        ref = call(sr, c)
        ws = sr.workspace(64 << 20)

        def skips(n, flag, same_bits=True, **kw):
            o, lse = torch.full_like(ref[0], 7.0), torch.full_like(ref[1], 7.0)
            call(sr, {**c, **kw}, o=o, lse=lse, ws=ws, max_kvlen=400)
            assert sr.device_status(ws) == flag
            rows = slice(c["cu"][n], c["cu"][n + 1])
            want = [t.clone() for t in ref]
            want[0][rows], want[1][rows] = 7.0, 7.0
            if same_bits:
                assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
                return
            # a length out of range takes its blocks out of the line that the CTAs share, so the other sequences may be
            # cut elsewhere: two results, each within (2^-11 + 2^-12) sum p |v| + 2^-8 |o| of the definition (as above,
            # e < 2^-14 here), where |v| <= 448 / 64 = 7
            assert torch.equal(o[rows], want[0][rows]) and torch.equal(lse[rows], want[1][rows])
            assert bool(((o.double() - want[0].double()).abs() <= 2 * (7 * (2.0 ** -11 + 2.0 ** -12) + 2.0 ** -8 * want[0].double().abs())).all())
            assert bool(((lse - want[1]).abs() <= 2.0 ** -13 + 2.0 ** -19 * (1 + want[1].abs())).all())

        for n, p, bad in ((0, 6, c["k_cache"].shape[0]), (1, 0, -1), (2, 4, 1 << 30)):
            table = c["table"].copy()
            table[n, p] = bad
            skips(n, sr.SR_DEV_BAD_INDEX, table=table)
        skips(0, sr.SR_DEV_BAD_LENGTH, same_bits=False, kv=[401, 90, 300])
        skips(1, sr.SR_DEV_BAD_LENGTH, same_bits=False, kv=[400, -1, 300])
        o = torch.full_like(ref[0], 7.0)
        call(sr, c, o=o, ws=ws, max_seqlen=max(new) - 1 if max(new) > 1 else 0)
        assert sr.device_status(ws) & sr.SR_DEV_SEQ_TOO_LONG


def test_the_cache_as_it_is_used(sr):
    """Prompts are appended and attended, then single tokens, over pages that fill up: every step's o is the definition's
    over the bytes that the cache holds by then, and near the attention over the keys and values before they were
    rounded to 8 bits."""
    gen = torch.Generator().manual_seed(19)
    h_q, h_kv, d, page, n_pages = 8, 2, 128, 64, 20
    cache = {k: torch.zeros(n_pages, h_kv, page, d, dtype=torch.float8_e4m3fn, device="cuda") for k in ("k_cache", "v_cache")}
    cache.update({k: torch.zeros(n_pages, h_kv, device="cuda") for k in ("k_scale", "v_scale")})
    table = np.array([[3, 8, 1, 17], [0, 2, 4, 6], [19, 5, 7, 9]])
    freq = (1e4 ** (-torch.arange(32).double() / 32)).float().cuda()
    held = [0, 0, 0]
    keys, values = [[] for _ in held], [[] for _ in held]
    for new in ([100, 1, 70], [1, 1, 1], [1, 2, 1], [27, 0, 60], [1, 1, 1]):
        T = sum(new)
        q, k, v = (torch.randn(T, h, d, generator=gen).bfloat16().cuda() for h in (h_q, h_kv, h_kv))
        held = [a + b for a, b in zip(held, new)]
        cu = np.concatenate([[0], np.cumsum(new)])
        args = (i32(cu), i32(held), i32(table))
        store = (cache["k_cache"], cache["v_cache"], cache["k_scale"], cache["v_scale"])
        turned = sr.kv_append(k, v, *args, *store, max_seqlen=max(new), q=q, inv_freq=freq)
        c = dict(cu=cu.tolist(), kv=held, table=table, new=new, page=page, d=d, group=h_q // h_kv, q=turned,
                 **{n: t.view(torch.uint8) if "cache" in n else t for n, t in cache.items()})
        o, _ = check(sr, c)
        pos = np.concatenate([np.arange(held[n] - new[n], held[n]) for n in range(3)])[None]
        kr, qr = (O.rotate(np64(x), pos, np64(freq), [32]) for x in (k, q))
        for n in range(3):
            keys[n] += list(kr[cu[n]:cu[n + 1]])
            values[n] += list(np64(v)[cu[n]:cu[n + 1]])
            for i in range(new[n]):
                row, seen = cu[n] + i, held[n] - new[n] + i + 1
                for h in range(h_q):
                    kk, vv = np.array(keys[n][:seen])[:, h // 4], np.array(values[n][:seen])[:, h // 4]
                    s = kk @ qr[row, h] * d ** -0.5
                    # a key or value is off by 2^-4 of itself at most, twice that where its page's scale grew: a score
                    # by e, a weight by a factor within exp(2 e) of the others
                    e = 2.0 ** -3 * (np.abs(kk) @ np.abs(qr[row, h])).max() * d ** -0.5
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    bound = (np.expm1(2 * e) + 2.0 ** -3 * np.exp(2 * e)) * (p @ np.abs(vv)) + 0.02
                    assert (np.abs(np64(o[row, h]) - p @ vv) <= bound).all()


def test_refusals(sr):
    c = make([3, 4], [20, 30], seed=20)
    with pytest.raises(ValueError, match="kv_lens"):
        call(sr, dict(c, kv=[20]), max_kvlen=30)
    with pytest.raises(ValueError, match="block_table"):
        call(sr, dict(c, table=c["table"][:1]))
    with pytest.raises(ValueError, match="q must be"):
        call(sr, dict(c, q=c["q"].float()))
    with pytest.raises(ValueError, match="v_cache"):
        call(sr, dict(c, v_cache=c["v_cache"][:, :, :8].contiguous()))
    with pytest.raises(sr.SrError, match="page_size"):
        call(sr, dict(c, k_cache=c["k_cache"][:, :, :8].contiguous(), v_cache=c["v_cache"][:, :, :8].contiguous()))
    with pytest.raises(sr.SrError, match="multiple"):
        call(sr, dict(c, q=torch.zeros(7, 3, 64, dtype=torch.bfloat16, device="cuda")))
    with pytest.raises(sr.SrError, match="finite"):
        call(sr, c, scale=float("nan"))
    with pytest.raises(sr.SrError, match="workspace"):
        call(sr, c, ws=sr.workspace(256))
