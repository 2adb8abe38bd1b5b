"""sr_kv_append on the GPU against the fp64 definition (oracle.paged).

Bounds.  Values are stored with one rounding: a stored value times its scale is
within half an e4m3 step of the row that was appended.  A rotated key carries
fp32 roundings before that: the cosine and sine (two half steps each, and the
angle reduced in 64 bits: one half step of a fraction of a turn times 2 pi,
under 4 in all) and three of the product and sum, so under 2^-21 of the pair's
length.  A rotated query is that far off and rounded once to bf16 (2^-8)."""
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
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def make(new, past, h_q=4, h_kv=2, d=64, page=16, rot=None, axes=1, seed=0, spare=3):
    """A cache with `past` tokens of every sequence in it (random bytes, scales of mixed size) and new rows."""
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    N, T = len(new), sum(new)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(int).tolist()
    kv = [a + b for a, b in zip(new, past)]
    per = [(t + page - 1) // page for t in kv]
    n_pages = sum(per) + spare
    order = torch.randperm(n_pages, generator=gen).tolist()
    table, at = np.zeros((N, max(max(per, default=0), 1)), int), 0
    for n, p in enumerate(per):
        table[n, :p] = order[at:at + p]
        at += p
    rot = d if rot is None else rot
    c = dict(cu=cu, kv=kv, table=table, new=new, past=past, max_new=max(new), page=page, d=d, rot=rot, order=order)
    byte = lambda: torch.randint(0, 256, (n_pages, h_kv, page, d), generator=gen, dtype=torch.uint8)
    c["k_cache"], c["v_cache"] = byte().cuda(), byte().cuda()
    sc = lambda: torch.ldexp(torch.ones(n_pages, h_kv), torch.randint(-12, 2, (n_pages, h_kv), generator=gen))
    c["k_scale"], c["v_scale"] = sc().cuda(), sc().cuda()
    size = torch.exp(2 * r(T, 1, 1))
    c["k"], c["v"] = (r(T, h_kv, d) * size).bfloat16().cuda(), (r(T, h_kv, d) * size).bfloat16().cuda()
    c["q"] = r(T, h_q, d).bfloat16().cuda()
    half = rot // 2
    c["inv_freq"] = (1e6 ** (-torch.arange(half).double() / max(half, 1))).float().cuda()
    side = half // 4
    c["sections"] = [half] if axes == 1 else [half - side * (axes - 1)] + [side] * (axes - 1)
    c["positions"] = torch.randint(0, 1 << 20, (axes, T), generator=gen, dtype=torch.int32).cuda()
    return c


def call(sr, c, **kw):
    args = dict(max_seqlen=c["max_new"], q=c["q"], inv_freq=c["inv_freq"] if c["rot"] else None,
                positions=c["positions"], sections=c["sections"])
    args.update(kw)
    return sr.kv_append(c["k"], c["v"], i32(c["cu"]), i32(c["kv"]), i32(c["table"]), c["k_cache"], c["v_cache"],
                        c["k_scale"], c["v_scale"], **args)


def check(sr, c, positions=None, interleaved=False, **kw):
    """Runs the call and compares the queries, every byte and every scale."""
    before = {k: c[k].clone() for k in ("k_cache", "v_cache", "k_scale", "v_scale")}
    k0, q0 = np64(c["k"]), np64(c["q"])
    q = call(sr, c, interleaved=interleaved, **kw)
    pos = np64(c["positions"]) if positions is None else positions
    freq = np64(c["inv_freq"])
    turn = lambda x: O.rotate(x, pos, freq, c["sections"], interleaved)
    if q is not None:
        want = turn(q0)
        length = np.sqrt((q0 ** 2).max(-1, keepdims=True) * 2)
        assert (np.abs(np64(q) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * length).all()
    for name, rows in (("k", turn(k0)), ("v", np64(c["v"]))):
        values = TABLE[before[name + "_cache"].cpu().numpy()]
        scales = np64(before[name + "_scale"])
        new = O.append(rows, c["cu"], c["kv"], c["table"], values, scales)
        assert np.array_equal(np64(c[name + "_scale"]), scales), name
        got = TABLE[c[name + "_cache"].cpu().numpy()]
        if name == "k":
            # rows that were rotated: half a step of the stored value, and the rotation's own error
            for (p, h, s), row in new.items():
                with np.errstate(invalid="ignore"):
                    off = np.abs(got[p, h, s] * scales[p, h] - row)
                    clip = np.clip(row / scales[p, h], -O.E4M3_MAX, O.E4M3_MAX)
                    tol = (O.e4m3_step(clip) / 2 + np.abs(row / scales[p, h] - clip)) * scales[p, h]
                    tol = tol + 2.0 ** -20 * np.sqrt(2) * np.nanmax(np.abs(np.where(np.isfinite(row), row, 0)))
                fine = np.isfinite(row)
                assert np.array_equal(np.isnan(got[p, h, s]), ~fine)
                assert (off[fine] <= tol[fine]).all(), (name, p, h, s)
                values[p, h, s] = got[p, h, s]
        assert np.array_equal(np.nan_to_num(got, nan=1e9), np.nan_to_num(values, nan=1e9)), name
    return q


NEW_PAST = [([1], [0]), ([1, 1, 1], [15, 16, 17]), ([5, 0, 40], [3, 20, 0]), ([16, 32], [16, 8]), ([70, 1, 33], [0, 31, 15]),
            ([0, 2], [4, 0])]


@pytest.mark.parametrize("new,past", NEW_PAST, ids=str)
@pytest.mark.parametrize("d,page,rot,axes,inter", [(64, 16, 64, 1, False), (64, 32, 16, 3, True), (128, 64, 128, 3, False),
                                                   (128, 16, 64, 2, True), (256, 128, 64, 1, False), (256, 16, 256, 3, False),
                                                   (128, 32, 0, 1, False)], ids=str)
def test_append(sr, new, past, d, page, rot, axes, inter):
    check(sr, make(new, past, d=d, page=page, rot=rot, axes=axes, seed=d + page), interleaved=inter)


def test_many_heads_and_long(sr):
    check(sr, make([300, 700, 129], [1000, 0, 63], h_q=12, h_kv=3, d=128, page=64, axes=3, seed=1))
    check(sr, make([400], [5], h_q=32, h_kv=1, d=256, page=128, rot=256, seed=2))


def test_cache_positions_by_default(sr):
    c = make([3, 50], [7, 100], seed=4)
    pos = np.array([[7, 8, 9] + list(range(100, 150))], float)
    c["positions"] = None
    check(sr, c, positions=pos)


def test_far_and_negative_positions(sr):
    """An fp32 product would be off by radians at 2^30."""
    c = make([64], [0], seed=5)
    c["positions"] = torch.randint(-(1 << 30), 1 << 30, (1, 64), dtype=torch.int32, generator=torch.Generator().manual_seed(5)).cuda()
    check(sr, c)


def test_without_queries_and_with_strided_rows_in_place(sr):
    c = make([9, 20], [3, 0], seed=6)
    c["q"] = c["q"].clone()
    q = c["q"]
    ref = {k: v.clone() if torch.is_tensor(v) else v for k, v in c.items()}
    q_ref = call(sr, ref)
    assert call(sr, {**{k: v.clone() if torch.is_tensor(v) else v for k, v in c.items()}, "q": q}, q=None) is None
    # q, k and v as slices of one projection, queries rotated in place
    T, h_q, d = q.shape
    h_kv = c["k"].shape[1]
    fused = torch.cat([q.flatten(1), c["k"].flatten(1), c["v"].flatten(1)], 1).contiguous()
    view = lambda a, n: fused[:, a * d:(a + n) * d].unflatten(1, (n, d))
    c["q"], c["k"], c["v"] = view(0, h_q), view(h_q, h_kv), view(h_q + h_kv, h_kv)
    out = call(sr, c, q_out=c["q"])
    assert out is c["q"] and torch.equal(out, q_ref)
    for name in ("k_cache", "v_cache", "k_scale", "v_scale"):
        assert torch.equal(c[name], ref[name])


def test_a_reused_page_starts_afresh_and_zeros_take_the_least_scale(sr):
    c = make([4], [0], seed=7)
    c["k_scale"].fill_(float("nan"))
    c["v_scale"].fill_(1e30)
    c["v"].zero_()
    call(sr, c)
    at = c["table"][0, 0]
    assert bool((c["v_scale"][at] == 2.0 ** -32).all()) and bool(torch.isfinite(c["k_scale"][at]).all())
    assert not bool(c["v_cache"][at][:, :4].any())


def test_values_that_are_not_finite(sr):
    c = make([20], [5], seed=8, rot=16, d=64)
    c["k"][3, 0, 40], c["k"][4, 1, 2], c["v"][6, 1, 7], c["v"][2, 0, 0] = float("inf"), float("nan"), float("-inf"), float("nan")
    with np.errstate(invalid="ignore"):
        check(sr, c)


def test_huge_and_tiny_values_meet_the_scale_limits(sr):
    c = make([2, 2], [0, 0], seed=9, rot=0)
    c["v"][:2] = 1e30
    c["v"][2:] = 1e-30
    check(sr, c)
    assert float(c["v_scale"][c["table"][0, 0], 0]) == 2.0 ** 32
    assert float(c["v_scale"][c["table"][1, 0], 0]) == 2.0 ** -32


def test_token_by_token_is_within_the_roundings_of_its_scales(sr):
    """Each growth of a page's scale rounds its older values once more, by half a step of the value at that scale, and
    the steps halve going back: under one step of the last scale in all."""
    c = make([60], [0], d=64, page=16, seed=10)
    one = dict(c, max_new=1)
    for t in range(60):
        step = dict(one, cu=[0, 1], kv=[t + 1], positions=c["positions"][:, t:t + 1].contiguous(),
                    k=c["k"][t:t + 1], v=c["v"][t:t + 1], q=c["q"][t:t + 1])
        call(sr, step)
    v = np64(c["v"])
    got = TABLE[c["v_cache"].cpu().numpy()]
    s = np64(c["v_scale"])
    for t in range(60):
        at = c["table"][0, t // 16]
        x = got[at, :, t % 16] * s[at][:, None]
        assert (np.abs(x - v[t]) <= O.e4m3_step(v[t] / s[at][:, None]) * s[at][:, None]).all()
    want = np.array([[O.scale_of(np.abs(v[16 * p:16 * p + 16, h]).max()) for h in range(2)] for p in range(4)])
    assert np.array_equal(s[c["table"][0]], want)


def test_captured_on_a_side_stream_and_again(sr):
    c = make([1, 1, 30], [15, 40, 0], seed=11)
    ref = {k: v.clone() if torch.is_tensor(v) else v for k, v in c.items()}
    q_ref = call(sr, ref)
    q_out, ws = torch.zeros_like(c["q"]), sr.workspace(256)
    cu, kv, table = i32(c["cu"]), i32(c["kv"]), i32(c["table"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sr.kv_append(c["k"], c["v"], cu, kv, table, c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"],
                     max_seqlen=30, q=c["q"], q_out=q_out, inv_freq=c["inv_freq"], positions=c["positions"], ws=ws)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(q_out, q_ref)
        for name in ("k_cache", "v_cache", "k_scale", "v_scale"):
            assert torch.equal(c[name], ref[name])
    assert sr.device_status(ws) == 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert torch.equal(call(sr, ref, stream=side).cpu(), q_ref.cpu())


def test_bad_pages_and_lengths_are_left_out(sr):
    c = make([20, 6, 6], [0, 3, 4], seed=12)
    ref = {k: v.clone() if torch.is_tensor(v) else v for k, v in c.items()}
    call(sr, ref)
    n_pages = c["k_cache"].shape[0]
    good = c["table"].copy()
    c["table"][0, 1], c["table"][2, 0] = n_pages, -1
    ws = sr.workspace(256)
    before = {k: c[k].clone() for k in ("k_cache", "v_cache", "k_scale", "v_scale")}
    call(sr, c, ws=ws)
    assert sr.device_status(ws) == sr.SR_DEV_BAD_INDEX
    for name in before:
        want = ref[name].clone()
        for at in (good[0, 1], good[2, 0]):
            want[at] = before[name][at]
        assert torch.equal(c[name], want), name
    c["table"] = good
    for kv in ([10, 9, 10], [20, 9, 33]):  # fewer tokens than the new ones; more than the table's two pages hold
        for name in before:
            c[name].copy_(before[name])
        q_out = torch.full_like(c["q"], 7.0)
        call(sr, dict(c, kv=kv), ws=ws, q_out=q_out)
        assert sr.device_status(ws) == sr.SR_DEV_BAD_LENGTH
        lost = 0 if kv[0] == 10 else 2
        rows = slice(c["cu"][lost], c["cu"][lost + 1])
        assert bool((q_out[rows] == 7.0).all()) and int((q_out == 7.0).all(-1).all(-1).sum()) == c["new"][lost]
        for name in before:
            want = ref[name].clone()
            for at in good[lost]:
                want[at] = before[name][at]
            assert torch.equal(c[name], want), (kv, name)


def test_refusals(sr):
    c = make([4], [0], seed=13)
    with pytest.raises(ValueError, match="sections"):
        call(sr, c, sections=[16, 16])
    with pytest.raises(sr.SrError, match="add up"):
        call(sr, c, sections=[16])
    with pytest.raises(ValueError, match="q_out needs q"):
        call(sr, c, q=None, q_out=c["q"])
    with pytest.raises(ValueError, match="lie together"):
        call(sr, dict(c, k=c["k"].transpose(0, 1).contiguous().transpose(0, 1)))
    with pytest.raises(ValueError, match="v_scale"):
        call(sr, dict(c, v_scale=c["v_scale"].double()))
    with pytest.raises(ValueError, match="kv_lens"):
        call(sr, dict(c, kv=[4, 4]))
    with pytest.raises(sr.SrError, match="rot_dim"):
        call(sr, c, inv_freq=c["inv_freq"][:6].contiguous(), sections=[6])
    with pytest.raises(sr.SrError, match="max_seqlen"):
        call(sr, c, max_seqlen=5)
