"""The elementwise gated linear recurrence and its gradients on the GPU,
against the fp64 definition (oracle.linrec).

Bounds.  A state carries one rounding of its decay (expf: two half steps) and
of its fma (one) per remembered token, and the fold over warps and CTAs at
most three more per level, so with M = min(len, 1 / (1 - max a)) remembered
tokens an fp32 result is within (3 M + 12) 2^-24 of the largest magnitude that
its sum passes through, sum |a ... a x|; a bf16 result rounds once more, by
2^-8 of itself at most (torch.finfo(t).eps / 2)."""
import numpy as np
import pytest
import torch

from oracle import linrec as O

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def sr():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_deltanet_state_sr_b200 as m
    return m


def np64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def make(lens, D, dtype=F32, g_dtype=F32, h0=True, seed=0, g_lo=-1.0, g_hi=-0.02):
    gen = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)
    r = lambda *s: torch.randn(*s, generator=gen)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    g = torch.rand(T, D, generator=gen) * (g_hi - g_lo) + g_lo
    c = dict(x=r(T, D).to(dtype), g=g.to(g_dtype), dy=r(T, D).to(dtype), h0=r(N, D) if h0 else None, ds=r(N, D))
    c = {k: None if v is None else v.cuda() for k, v in c.items()}
    c.update(cu=cu, cu_dev=torch.tensor(cu, dtype=torch.int32, device="cuda"), max_len=max(lens, default=0))
    return c


def bound(c, dtype, ref, size):
    """Elementwise bound of a result `ref` whose sums pass through `size`."""
    a = np.exp(np64(c["g"]).max()) if c["g"].numel() else 0.0
    m = min(c["max_len"], 1 / (1 - a) if a < 1 else np.inf)
    return (3 * m + 12) * 2.0 ** -24 * size + (2.0 ** -8 * np.abs(ref) if dtype == BF else 0.0)


def check(got, ref, tol, what):
    # fp32 has no values between 0 and 2^-149: a decay below that is 0, which moves a term by 2^-149 of its other
    # factors; those stay under 2^23 here
    off = np.abs(np64(got) - ref)
    assert off.shape == ref.shape
    tol = tol + 2.0 ** -126
    bad = ~(off <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(off - tol):.3e} over its bound"


def check_forward(sr, c, **kw):
    y, s = sr.linrec_replay(c["x"], c["g"], c["cu_dev"], max_seqlen=c["max_len"], h0=c["h0"], **kw)
    x, g, h0 = np64(c["x"]), np64(c["g"]), np64(c["h0"])
    y_ref, s_ref = O.replay(x, g, c["cu"], h0)
    y_size, s_size = O.replay(np.abs(x), g, c["cu"], None if h0 is None else np.abs(h0))
    check(y, y_ref, bound(c, c["x"].dtype, y_ref, y_size), "y")
    check(s, s_ref, bound(c, F32, s_ref, s_size), "s")
    return y, s


def check_backward(sr, c, y, **kw):
    got = sr.linrec_backward(c["g"], y, c["dy"], c["cu_dev"], max_seqlen=c["max_len"], h0=c["h0"], ds=c["ds"], **kw)
    g, yy, dy, h0, ds = (np64(t) for t in (c["g"], y, c["dy"], c["h0"], c["ds"]))
    ref = O.backward(g, yy, dy, c["cu"], h0, ds)
    size = O.backward(g, np.abs(yy), np.abs(dy), c["cu"], None if h0 is None else np.abs(h0), np.abs(ds))
    for name, dt, a, r, z in zip(("dx", "dg", "dh0"), (y.dtype, c["g"].dtype, F32), got, ref, size):
        assert a.dtype == dt
        # dg multiplies by a stored h once more: one half step
        check(a, r, bound(c, dt, r, z) + 2.0 ** -24 * z, name)
    return got


LENGTHS = [
    [1], [2], [8], [9], [64], [65], [63, 1, 0, 7], [0, 0], [513], [1, 1, 1, 1, 1], [130, 0, 64, 1, 1000, 3],
    [4097], [20, 700, 511, 512],
]


@pytest.mark.parametrize("lens", LENGTHS, ids=str)
@pytest.mark.parametrize("D", [1, 8, 37, 64, 130, 200])
@pytest.mark.parametrize("types", [(BF, BF), (BF, F32), (F32, F32)], ids=["bf16", "bf16_g32", "fp32"])
def test_forward_and_backward(sr, lens, D, types):
    c = make(lens, D, *types, h0=D != 37, seed=D)
    y, _ = check_forward(sr, c)
    check_backward(sr, c, y)


@pytest.mark.parametrize("lens,D", [([32768], 64), ([3000] * 5, 2560), ([5000, 1, 9000], 520)], ids=str)
def test_long(sr, lens, D):
    """Several waves of every cluster size, long memories."""
    c = make(lens, D, BF, F32, seed=3, g_lo=-0.5, g_hi=-1e-3)
    y, _ = check_forward(sr, c)
    check_backward(sr, c, y)


def test_many_sequences(sr):
    """More sequences than the longest-first order covers."""
    lens = [(7 * i) % 23 for i in range(300)]
    c = make(lens, 66, seed=4)
    y, _ = check_forward(sr, c)
    check_backward(sr, c, y)


def test_many_short_sequences_beside_a_long_one(sr):
    lens = [(5 * i) % 7 for i in range(299)]
    lens.insert(150, 2500)
    for D in (64, 37):
        c = make(lens, D, BF, BF, seed=14)
        y, _ = check_forward(sr, c)
        check_backward(sr, c, y)


def test_unaligned_rows_take_single_channels(sr):
    """Rows whose pairs of channels straddle the alignment: a view that starts one element into its storage."""
    c = make([33, 70], 6, BF, BF, seed=5)
    for k in ("x", "g", "dy"):
        buf = torch.empty(c[k].numel() + 1, dtype=c[k].dtype, device="cuda")
        buf[1:] = c[k].flatten()
        c[k] = buf[1:].view(c[k].shape)
    y, _ = check_forward(sr, c)
    check_backward(sr, c, y)


def test_gates_that_close_and_gates_that_stay_open(sr):
    """exp(-inf) = 0 forgets everything before, whatever it was; g = 0 sums."""
    c = make([40, 600], 34, seed=6, g_lo=-0.1, g_hi=-0.01)
    c["g"][10] = -np.inf
    c["g"][300, 5:9] = -np.inf
    c["g"][500] = -200.0
    c["g"][20:24] = 0.0
    y, s = sr.linrec_replay(c["x"], c["g"], c["cu_dev"], max_seqlen=600, h0=c["h0"])
    with np.errstate(invalid="ignore"):
        ref = O.replay(np64(c["x"]), np64(c["g"]), c["cu"], np64(c["h0"]))
    size = O.replay(np.abs(np64(c["x"])), np64(c["g"]), c["cu"], np.abs(np64(c["h0"])))
    for a, r, z in zip((y, s), ref, size):
        check(a, r, (3 * 104 + 12) * 2.0 ** -24 * z, "closed gates")
    got = sr.linrec_backward(c["g"], y, c["dy"], c["cu_dev"], max_seqlen=600, h0=c["h0"], ds=c["ds"])
    args = [np64(t) for t in (c["g"], y, c["dy"])]
    ref = O.backward(*args, c["cu"], np64(c["h0"]), np64(c["ds"]))
    size = O.backward(args[0], np.abs(args[1]), np.abs(args[2]), c["cu"], np.abs(np64(c["h0"])), np.abs(np64(c["ds"])))
    for a, r, z in zip(got, ref, size):
        check(a, r, (3 * 104 + 13) * 2.0 ** -24 * z, "closed gates, gradients")


def test_nan_and_inf_stay_in_their_sequence_and_channel(sr):
    c = make([50, 700, 9], 32, seed=7)
    c["x"][60, 3] = float("nan")
    c["x"][400, 5] = float("inf")
    y, s = sr.linrec_replay(c["x"], c["g"], c["cu_dev"], max_seqlen=700, h0=c["h0"])
    ref = O.replay(np64(c["x"]), np64(c["g"]), c["cu"], np64(c["h0"]))
    for a, r in zip((y, s), ref):
        a = np64(a)
        assert np.array_equal(np.isnan(a), np.isnan(r)) and np.array_equal(np.isposinf(a), np.isposinf(r))


def test_gradients_are_the_differences_of_the_definition(sr):
    c = make([5, 90, 1], 8, seed=8, g_lo=-0.8, g_hi=-0.05)
    y, _ = sr.linrec_replay(c["x"], c["g"], c["cu_dev"], max_seqlen=90, h0=c["h0"])
    grads = sr.linrec_backward(c["g"], y, c["dy"], c["cu_dev"], max_seqlen=90, h0=c["h0"], ds=c["ds"])
    base = [np64(c[k]) for k in ("x", "g", "h0")]
    dy, ds = np64(c["dy"]), np64(c["ds"])

    def loss(v):
        yy, ss = O.replay(v[0], v[1], c["cu"], v[2])
        return (yy * dy).sum() + (ss * ds).sum()

    rng = np.random.default_rng(9)
    size = sum(np.abs(np64(a)).sum() for a in grads)
    for k in range(3):
        for _ in range(4):
            u = rng.normal(size=base[k].shape)
            e = 1e-5
            hi, lo = list(base), list(base)
            hi[k], lo[k] = base[k] + e * u, base[k] - e * u
            # the y that the gradients read is fp32, as are they: (3 * 21 + 12) 2^-24 of the terms' size, |u| <= 5
            assert abs((loss(hi) - loss(lo)) / (2 * e) - (np64(grads[k]) * u).sum()) < 80 * 2.0 ** -24 * 5 * size


def test_a_split_sequence_continues_and_the_step_is_in_place(sr):
    """A prefill, then single tokens with s_out = h0, gives the states of one call over all tokens."""
    c = make([300], 256, BF, F32, seed=10)
    y_all, s_all = check_forward(sr, c)
    state = c["h0"].clone()
    cu = torch.tensor([0, 290], dtype=torch.int32, device="cuda")
    y0, _ = sr.linrec_replay(c["x"][:290], c["g"][:290], cu, max_seqlen=290, h0=state, s_out=state)
    ys = [y0]
    one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    for t in range(290, 300):
        y, s = sr.linrec_replay(c["x"][t:t + 1], c["g"][t:t + 1], one, max_seqlen=1, h0=state, s_out=state)
        assert s is state
        ys.append(y)
    x, g, h0 = np64(c["x"]), np64(c["g"]), np64(c["h0"])
    ref, s_ref = O.replay(x, g, c["cu"], h0)
    size, s_size = O.replay(np.abs(x), g, c["cu"], np.abs(h0))
    check(torch.cat(ys), ref, bound(c, BF, ref, size), "y")
    check(state, s_ref, bound(c, F32, s_ref, s_size), "s")


def test_same_bits_again_captured_and_on_another_stream(sr):
    c = make([700, 3, 1200], 320, BF, BF, seed=11)
    kw = dict(max_seqlen=1200, h0=c["h0"])
    y, s = sr.linrec_replay(c["x"], c["g"], c["cu_dev"], **kw)
    grads = sr.linrec_backward(c["g"], y, c["dy"], c["cu_dev"], ds=c["ds"], **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, s2 = sr.linrec_replay(c["x"], c["g"], c["cu_dev"], stream=side, **kw)
    side.synchronize()
    assert torch.equal(y, y2) and torch.equal(s, s2)
    out = [torch.zeros_like(t) for t in (y, s, *grads)]
    ws = [sr.workspace(256), sr.workspace(256)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sr.linrec_replay(c["x"], c["g"], c["cu_dev"], y=out[0], s_out=out[1], ws=ws[0], **kw)
        sr.linrec_backward(c["g"], out[0], c["dy"], c["cu_dev"], ds=c["ds"], dx=out[2], dg=out[3], dh0=out[4],
                           ws=ws[1], **kw)
    for _ in range(2):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, (y, s, *grads)))
    assert sr.device_status(ws[0]) == 0 and sr.device_status(ws[1]) == 0


def test_bad_sequences_are_skipped_and_rows_behind_the_last_are_left(sr):
    c = make([30, 40, 30], 64, seed=12)
    y_ref, s_ref = sr.linrec_replay(c["x"], c["g"], c["cu_dev"], max_seqlen=40, h0=c["h0"])
    for max_len, cu, flag, skipped in ((35, [0, 30, 70, 100], sr.SR_DEV_SEQ_TOO_LONG, [1]),
                                       (40, [0, 30, 70, 200], sr.SR_DEV_BAD_CU_SEQLENS, [2]),
                                       (40, [0, 30, 70, 69], sr.SR_DEV_BAD_CU_SEQLENS, [2])):
        y, s, ws = torch.full_like(y_ref, 7.0), torch.full_like(s_ref, 7.0), sr.workspace(256)
        sr.linrec_replay(c["x"], c["g"], torch.tensor(cu, dtype=torch.int32, device="cuda"), max_seqlen=max_len,
                         h0=c["h0"], y=y, s_out=s, ws=ws)
        assert sr.device_status(ws) & flag
        for n in range(3):
            rows = slice(c["cu"][n], c["cu"][n + 1])
            want_y, want_s = (torch.full_like(y[rows], 7.0), torch.full_like(s[n], 7.0)) if n in skipped else (
                y_ref[rows], s_ref[n])
            assert torch.equal(y[rows], want_y) and torch.equal(s[n], want_s), (cu, n)
    # cu[n_seqs] below total_tokens: the rows behind it belong to no sequence
    y = torch.full_like(y_ref, 7.0)
    sr.linrec_replay(c["x"], c["g"], torch.tensor([0, 30, 70], dtype=torch.int32, device="cuda"), max_seqlen=40,
                     h0=c["h0"][:2].contiguous(), y=y)
    assert torch.equal(y[:70], y_ref[:70]) and bool((y[70:] == 7.0).all())


def test_refusals(sr):
    c = make([30, 40], 64, BF, F32, seed=13)
    ok = dict(max_seqlen=40)
    with pytest.raises(ValueError, match="shape"):
        sr.linrec_replay(c["x"], c["g"][:, :32].contiguous(), c["cu_dev"], **ok)
    with pytest.raises(ValueError, match="contiguous"):
        sr.linrec_replay(c["x"], c["g"].t().contiguous().t(), c["cu_dev"], **ok)
    with pytest.raises(ValueError, match="CUDA"):
        sr.linrec_replay(c["x"].cpu(), c["g"], c["cu_dev"], **ok)
    with pytest.raises(ValueError, match="int32"):
        sr.linrec_replay(c["x"], c["g"], c["cu_dev"].long(), **ok)
    with pytest.raises(ValueError, match="h0"):
        sr.linrec_replay(c["x"], c["g"], c["cu_dev"], h0=c["h0"].bfloat16(), **ok)
    with pytest.raises(sr.SrError, match="fp32 g"):
        sr.linrec_replay(c["x"].float(), c["g"].bfloat16(), c["cu_dev"], **ok)
    with pytest.raises(sr.SrError, match="max_seqlen"):
        sr.linrec_replay(c["x"], c["g"], c["cu_dev"], max_seqlen=71)
    with pytest.raises(sr.SrError, match="workspace"):
        sr.linrec_replay(c["x"], c["g"], c["cu_dev"], ws=sr.workspace(256)[:128], **ok)
    with pytest.raises(ValueError, match="dy"):
        sr.linrec_backward(c["g"], c["x"], c["dy"].float(), c["cu_dev"], **ok)
