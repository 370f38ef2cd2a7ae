"""Sampling and the filtered distribution against the fp64 oracle.

Tolerance.  A weight e^d, d = (x - m) fl(1/T), carries three roundings of d (3 2^-24
|d|) and expf's error (2^-22).  Weights below 2^-44 do not count, so |d| <= 31 where it
matters: below 2^-17 relative.  Sums are exact to V 2^-44 <= 2^-26.  A border or a
draw compares two such sums: it may go either way within 2^-16.  Log probabilities:
|d| 3 2^-24 + 2^-16 (the sum's) and one rounding.
"""

import numpy as np
import pytest

from oracle import sampling as osa

pytestmark = pytest.mark.gpu
TOL = 2.0 ** -16


@pytest.fixture(scope="module")
def tsd():
    import tree_speculative_decoding_virtual_gb300 as m
    return m


def T(a, dtype=None):
    from _gpu_path import dev_tensor
    return dev_tensor(a, dtype)


def rows_of(rng, R, V, kind):
    x = rng.standard_normal((R, V)).astype(np.float32) * 2
    if kind == "peaked":
        up = rng.integers(0, V, (R, max(1, V // 500)))
        np.put_along_axis(x, up, (3 * rng.exponential(size=up.shape) + 2).astype(np.float32), 1)
    elif kind == "ties":
        x = np.round(x)
    elif kind == "equal":
        x[:] = 1.5
    elif kind == "masked":
        x[rng.random((R, V)) < 0.9] = -np.inf
        x[:, V // 2] = 0.0
    elif kind == "wide":
        x *= 40
    elif kind == "lowest":  # masked with the type's lowest value
        x[rng.random((R, V)) < 0.5] = np.finfo(np.float32).min
        x[:, V // 3] = 1.0
    return x


SETTINGS = [(1.0, 0, 1.0, 0.0), (0.7, 50, 1.0, 0.0), (1.0, 0, 0.9, 0.0), (1.3, 1000, 0.95, 0.0), (1.0, 0, 1.0, 0.05),
            (0.8, 40, 0.5, 0.02), (0.0, 0, 0.9, 0.5), (1.0, 1, 1.0, 0.0), (1.0, 0, 0.0, 0.0), (1.0, 0, 1e-6, 0.0),
            (1.0, 0, 0.99999, 0.0), (2.0, 0, 1.0, 1.0), (1e-3, 0, 0.99, 0.0), (1.0, 7, 0.999, 0.0), (1.0, 0, 1.0, 3.0)]


def check_row(x, setting, row, probs, tokens, logprob, u):
    """The filtered row, the probabilities and the draws of one row."""
    t, k, p, m = setting
    order = osa.ranking(x)
    kept = np.flatnonzero(row > -np.inf)
    n = len(kept)
    assert set(kept) == set(order[:n]), "not a prefix of the ranking"
    lo, hi = osa.kept_bounds(x, t, k, p, m, TOL)
    assert lo <= n <= hi, (setting, lo, n, hi)
    d, w = osa.weights(x, t)
    assert (np.abs(row[kept] - d[kept]) <= 3 * 2.0 ** -24 * np.abs(d[kept])).all()
    total = w[kept].sum()
    d = np.where(x > -np.inf, d, 0.0)
    want = np.zeros(len(x))
    want[kept] = w[kept] / total
    assert (np.abs(probs - want) <= (TOL + 3 * 2.0 ** -24 * np.abs(d)) * want + 2.0 ** -100).all()
    for token, lp, v in zip(tokens, logprob, u):
        assert osa.draw_ok(x, kept, token, float(v), t, TOL), (setting, token, v)
        ref = d[token] - np.log(total)
        assert abs(lp - ref) <= 3 * 2.0 ** -24 * abs(d[token]) + TOL + 2.0 ** -22 * abs(ref)


@pytest.mark.parametrize("V,kind,bf16", [
    (1, "plain", False), (2, "plain", False), (33, "plain", True), (1000, "ties", False), (1000, "equal", True),
    (4097, "peaked", False), (5003, "masked", True), (32000, "peaked", False), (32000, "ties", True),
    (32768, "equal", False), (50257, "wide", False), (128256, "peaked", False), (128256, "plain", False),
    (128256, "plain", True), (20001, "lowest", False), (262144, "peaked", True), (262144, "ties", False)])
def test_filters_and_draws(tsd, V, kind, bf16):
    import torch
    R = len(SETTINGS)
    rng = np.random.default_rng(V + R + len(kind))
    x = rows_of(rng, R, V, kind)
    if bf16:
        x = torch.from_numpy(x).bfloat16().float().numpy()
    logits = T(x).bfloat16() if bf16 else T(x)
    t, k, p, m = [T(np.array([s[i] for s in SETTINGS], np.int32 if i == 1 else np.float32)) for i in range(4)]
    u = rng.random((R, 5)).astype(np.float32)
    u[:, 0], u[:, 1] = 0.0, np.float32(1 - 2.0 ** -24)
    args = dict(temperature=t, top_k=k, top_p=p, min_p=m)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tokens, lp = tsd.token_sample(logits, T(u), status=st, **args)
    rows = tsd.logits_filter(logits, status=st, **args)
    probs = tsd.logits_filter(logits, probs=True, status=st, **args)
    assert int(st.item()) == 0
    tokens, lp, rows, probs = [a.cpu().numpy() for a in (tokens, lp, rows, probs)]
    for r, setting in enumerate(SETTINGS):
        f32 = tuple(float(np.float32(s)) if i != 1 else s for i, s in enumerate(setting))
        check_row(x[r].astype(np.float64), f32, rows[r].astype(np.float64), probs[r].astype(np.float64), tokens[r], lp[r], u[r])
    # ties are cut by id, exactly, and in-place filtering gives the same
    if not bf16:
        again = logits.clone()
        assert tsd.logits_filter(again, out=again, **args) is again
        assert np.array_equal(again.cpu().numpy(), rows)


@pytest.mark.parametrize("V,k,p", [(1000, 10, 1.0), (30000, 777, 1.0), (30000, 0, 0.25), (262144, 100000, 1.0), (1024, 0, 0.5)])
def test_equal_logits_are_cut_by_id(tsd, V, k, p):
    """All weights are 1, sums are whole: the kept ids are exactly the first ones, and so is a draw's."""
    x = T(np.full((2, V), -3.25, np.float32))
    args = dict(top_k=T(np.array([k, k], np.int32)), top_p=T(np.array([p, p], np.float32)))
    n = k if k else int(np.ceil(p * V))
    row = tsd.logits_filter(x, **args).cpu().numpy()
    assert (row[:, :n] == 0).all() and np.isneginf(row[:, n:]).all()
    u = np.array([[0.0, 0.5, 1 - 2.0 ** -24], [0.25, 0.75, 0.125]], np.float32)
    tokens, _ = tsd.token_sample(x, T(u), **args)
    assert np.array_equal(tokens.cpu().numpy(), np.floor(u.astype(np.float64) * n).astype(np.int32))


def test_zero_signs_tie(tsd):
    x = np.full((1, 64), -5.0, np.float32)
    x[0, [10, 20, 30]] = [-0.0, 0.0, -0.0]
    row = tsd.logits_filter(T(x), top_k=T(np.array([2], np.int32))).cpu().numpy()
    assert list(np.flatnonzero(row[0] > -np.inf)) == [10, 20]


def test_special_rows(tsd):
    import torch
    V = 5000
    x = np.random.default_rng(0).standard_normal((6, V)).astype(np.float32)
    x[0] = -np.inf
    x[1, 4000] = np.nan
    x[2, 17] = np.inf
    x[3] = -np.inf
    x[3, V - 1] = -7.0  # a single token
    x[4, :] = np.finfo(np.float32).max
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    u = T(np.full((6, 2), 0.5, np.float32))
    p = T(np.full(6, 0.9, np.float32))
    tokens, lp = [a.cpu().numpy() for a in tsd.token_sample(T(x), u, top_p=p, status=st)]
    assert int(st.item()) == tsd.STATUS_NONFINITE
    assert (tokens[:3] == -1).all() and np.isneginf(lp[0]).all() and np.isnan(lp[1:3]).all()
    assert (tokens[3] == V - 1).all() and (lp[3] == 0).all()
    assert (tokens[4] == int(0.5 * np.ceil(np.float64(np.float32(0.9)) * V))).all() and (tokens[5] >= 0).all()
    row = tsd.logits_filter(T(x), top_p=p).cpu().numpy()
    pr = tsd.logits_filter(T(x), top_p=p, probs=True).cpu().numpy()
    assert np.isneginf(row[0]).all() and np.isnan(row[1:3]).all() and (pr[0] == 0).all() and np.isnan(pr[1:3]).all()
    assert row[3, V - 1] == 0 and np.isneginf(row[3, :-1]).all() and pr[3, V - 1] == 1
    # masked by the lowest value and by -inf alike: what is not masked is drawn
    st.zero_()
    tokens, _ = tsd.token_sample(T(x[4:]), u[4:], status=st)
    assert int(st.item()) == 0


def test_chosen_rows_and_shared_settings(tsd):
    import torch
    rng = np.random.default_rng(3)
    x = rows_of(rng, 12, 3001, "peaked")  # odd: rows start at every alignment
    u = rng.random((12, 1)).astype(np.float32)
    t = np.array([0.5, 0.0, 1.5], np.float32)
    whole, lp = tsd.token_sample(T(x), T(u), temperature=T(np.repeat(t, 4)))
    grouped, lp2 = tsd.token_sample(T(x.reshape(3, 4, -1)), T(u.reshape(3, 4)), temperature=T(t))
    assert torch.equal(whole.view(3, 4), grouped) and torch.equal(lp.view(3, 4), lp2)
    rows = np.array([5, -1, 0, 11, 12, -3], np.int32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    some, lp3 = tsd.token_sample(T(x), T(u[[5, 0, 0, 11, 0, 0], 0]), rows=T(rows), status=st)
    plain, lp4 = tsd.token_sample(T(x), T(u[:, 0]))
    assert int(st.item()) == tsd.STATUS_BAD_PATH
    assert some.tolist()[:4] == [plain[5].item(), -1, plain[0].item(), plain[11].item()] and some.tolist()[4:] == [-1, -1]
    assert lp3.tolist() == [lp4[5].item(), 0.0, lp4[0].item(), lp4[11].item(), 0.0, 0.0]
    none, _ = tsd.token_sample(T(x)[:0], T(u)[:0])
    assert none.shape == (0, 1)


def test_draws_follow_the_distribution(tsd):
    """Evenly spread numbers draw each token in proportion to its weight, to one draw."""
    rng = np.random.default_rng(4)
    V, n = 40, 64
    x = rng.standard_normal((32, V)).astype(np.float32)
    x[:] = x[0]
    u = ((np.arange(32 * n) + 0.5) / (32 * n)).astype(np.float32).reshape(32, n)
    tokens, _ = tsd.token_sample(T(x), T(u))
    count = np.bincount(tokens.cpu().numpy().ravel(), minlength=V)
    w = np.exp(x[0].astype(np.float64))
    assert (np.abs(count - 32 * n * w / w.sum()) <= 1 + 32 * n * TOL).all()


def test_filter_draw_verify_and_score(tsd):
    """A step: the drafter's children are drawn from its filtered distribution, the verification divides by the same one."""
    import torch
    rng = np.random.default_rng(12)
    B, N, V, D_max = 2, 7, 1500, 3
    parent = np.array([[-1, 0, 0, 1, 1, 2, 2]] * B, np.int32)
    target, draft = [T(rows_of(rng, B * N, V, "peaked").reshape(B, N, V)) for _ in range(2)]
    t, p = T(np.array([0.9, 0.0], np.float32)), T(np.array([0.8, 0.9], np.float32))
    q = tsd.logits_filter(draft, temperature=t, top_p=p, probs=True)
    drawn, _ = tsd.token_sample(draft, T(rng.random((B, N, 2)).astype(np.float32)), temperature=t, top_p=p)
    tokens = torch.zeros((B, N), dtype=torch.int32, device="cuda")
    tokens[:, 1:3], tokens[:, 3:5], tokens[:, 5:7] = drawn[:, 0], drawn[:, 1], drawn[:, 2]
    x = tsd.logits_filter(target, temperature=t, top_p=p)
    anc, depth, mask, err = tsd.tree_build_ancestors(T(parent), None, D_max)
    u1, u2 = [T(rng.random((B, N)).astype(np.float32)) for _ in range(2)]
    nxt, draw, A, leaf, path, bonus = tsd.tree_verify_stochastic(x, q, tokens, T(parent), None, err, u1, u2, D_max)
    emitted, lp, _, _, _ = tsd.tree_path_logprobs(x, tokens, path, A, bonus, err, D_max)
    for b in range(B):
        for i in range(int(A[b]) + 1):  # nothing is emitted that the target's filters removed
            node = int(path[b, i]) - 1
            assert x[b, node, emitted[b, i]] > -np.inf and np.isfinite(lp[b, i].item())
    # temperature 0 is greedy verification with the most probable tokens
    node = 0
    best = target[1].argmax(-1)
    assert int(emitted[1, 0]) == int(best[node])


def test_replayed_with_other_settings(tsd):
    import torch
    rng = np.random.default_rng(13)
    x = T(rows_of(rng, 3, 9000, "peaked"))
    u, t = T(rng.random((3, 2)).astype(np.float32)), T(np.ones(3, np.float32))
    k = T(np.zeros(3, np.int32))
    tokens = torch.empty((3, 2), dtype=torch.int32, device="cuda")
    lp = torch.empty((3, 2), device="cuda")
    tsd.token_sample(x, u, temperature=t, top_k=k, tokens=tokens, logprob=lp)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tsd.token_sample(x, u, temperature=t, top_k=k, tokens=tokens, logprob=lp)
    t.fill_(0.6)
    k.fill_(30)
    x.mul_(-1)
    g.replay()
    want, want_lp = tsd.token_sample(x, u, temperature=t, top_k=k)
    assert torch.equal(tokens, want) and torch.equal(lp, want_lp)


@pytest.mark.parametrize("V,R,bf16", [(900, 700, False), (8000, 508, False), (32000, 64, True), (32000, 300, False),
                                      (32000, 1300, True), (128256, 60, True), (128256, 160, True), (128256, 60, False)])
def test_many_rows_are_as_each_alone(tsd, V, R, bf16):
    """How many CTAs share a row depends on how many rows there are; the results do not:
    sums are exact."""
    import torch
    rng = np.random.default_rng(V + R)
    some = rows_of(rng, 12, V, "peaked")
    x = T(some)[torch.arange(R, device="cuda") % 12]
    x = x + 0.25 * torch.randint(0, 5, (R, 1), device="cuda") + torch.arange(V, device="cuda") % 7 * 0.125
    if bf16:
        x = x.bfloat16()
    t, k, p, m = [T(np.array([SETTINGS[r % len(SETTINGS)][i] for r in range(R)], np.int32 if i == 1 else np.float32))
                  for i in range(4)]
    u = T(rng.random((R, 3)).astype(np.float32))
    tokens, lp = tsd.token_sample(x, u, temperature=t, top_k=k, top_p=p, min_p=m)
    rows = tsd.logits_filter(x, temperature=t, top_k=k, top_p=p, min_p=m)
    probs = tsd.logits_filter(x, temperature=t, top_k=k, top_p=p, min_p=m, probs=True)
    for r in list(range(0, R, max(1, R // 40))) + [R - 1]:
        one = dict(temperature=t[r:r + 1], top_k=k[r:r + 1], top_p=p[r:r + 1], min_p=m[r:r + 1])
        alone, alone_lp = tsd.token_sample(x[r:r + 1], u[r:r + 1], **one)
        assert torch.equal(tokens[r:r + 1], alone) and torch.equal(lp[r:r + 1], alone_lp), r
        assert torch.equal(rows[r:r + 1], tsd.logits_filter(x[r:r + 1], **one)), r
        assert torch.equal(probs[r:r + 1], tsd.logits_filter(x[r:r + 1], probs=True, **one)), r


def test_two_streams_at_once(tsd):
    import torch
    rng = np.random.default_rng(21)
    x = [T(rows_of(rng, 40, 32000, "peaked")), T(rows_of(rng, 40, 32000, "plain"))]
    u = T(rng.random((40, 2)).astype(np.float32))
    k, p = T(np.full(40, 40, np.int32)), T(np.full(40, 0.9, np.float32))
    want = [tsd.token_sample(x[0], u, top_k=k), tsd.token_sample(x[1], u, top_p=p)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = tsd.token_sample(x[i], u, **(dict(top_p=p) if i else dict(top_k=k)))
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(got[i][0], want[i][0]) and torch.equal(got[i][1], want[i][1])


def test_settings_out_of_range(tsd):
    """An infinite temperature is uniform over what is not masked; NaN settings are off."""
    import torch
    x = T(rows_of(np.random.default_rng(31), 4, 5000, "masked"))
    inf, nan = T(np.full(4, np.inf, np.float32)), T(np.full(4, np.nan, np.float32))
    finite = (x > -torch.inf).float()
    probs = tsd.logits_filter(x, inf, probs=True)
    assert torch.allclose(probs, finite / finite.sum(1, keepdim=True), rtol=2.0 ** -20, atol=0)
    assert torch.equal(probs, tsd.logits_filter(x, nan, probs=True))
    tokens, lp = tsd.token_sample(x, T(np.array([[0.0, 0.3, 0.999]] * 4, np.float32)), inf)
    assert (finite.gather(1, tokens.long()) == 1).all() and torch.isfinite(lp).all()
    for kw in (dict(top_k=T(np.full(4, 10, np.int32))), {}):  # with another filter, and alone
        want = tsd.logits_filter(x, **kw)
        assert torch.equal(tsd.logits_filter(x, top_p=nan, min_p=nan, **kw), want)
    last = tsd.logits_filter(x, inf, top_p=T(np.full(4, 0.5, np.float32)), probs=True)
    half = (finite.sum(1) + 1).div(2, rounding_mode="floor")  # ranks before r: r of n equal weights < n / 2
    assert torch.equal((last > 0).sum(1).float(), half)


@pytest.mark.parametrize("V,width", [(100000, 0.05), (262144, 1e-3), (50000, 2.0)])
def test_dense_logits(tsd, V, width):
    """Thousands of different logits in each of the first bins, which are cut again."""
    import torch
    settings = [(1.0, 0, 0.5, 0.0), (1.0, 20000, 1.0, 0.0), (0.5, 30000, 0.3, 0.0), (1.0, 0, 0.999, 0.0), (0.1, 700, 0.9, 0.5)]
    rng = np.random.default_rng(V)
    x = (rng.random((len(settings), V)) * width).astype(np.float32)
    t, k, p, m = [T(np.array([s[i] for s in settings], np.int32 if i == 1 else np.float32)) for i in range(4)]
    args = dict(temperature=t, top_k=k, top_p=p, min_p=m)
    u = rng.random((len(settings), 4)).astype(np.float32)
    tokens, lp = tsd.token_sample(T(x), T(u), **args)
    rows, probs = tsd.logits_filter(T(x), **args), tsd.logits_filter(T(x), probs=True, **args)
    tokens, lp, rows, probs = [a.cpu().numpy() for a in (tokens, lp, rows, probs)]
    for r, setting in enumerate(settings):
        f32 = tuple(float(np.float32(s)) if i != 1 else s for i, s in enumerate(setting))
        check_row(x[r].astype(np.float64), f32, rows[r].astype(np.float64), probs[r].astype(np.float64), tokens[r], lp[r], u[r])


def drawn(tsd, x, u, **args):
    """token_sample into outputs that hold what no call writes."""
    import torch
    tokens = torch.full(u.shape, -7, dtype=torch.int32, device="cuda")
    lp = torch.full(u.shape, 7.0, device="cuda")
    tsd.token_sample(T(x), T(u), tokens=tokens, logprob=lp, **args)
    return tokens.cpu().numpy(), lp.cpu().numpy()


@pytest.mark.parametrize("R", [1, 3])
def test_short_lists_behind_many_kept(tsd, R):
    """More is kept than a list holds, and the border's bins hold a few logits: those of every CTA of a row, whose
    weights the draws need by run."""
    rng = np.random.default_rng(51)
    V, n, draws = 262144, 2000, 64
    x = np.full((R, V), -np.inf, np.float32)
    for r in range(R):
        x[r, np.sort(rng.permutation(V)[:n])] = rng.permutation(n).astype(np.float32) * np.float32(-0.001)
    u = ((np.arange(R * draws) + rng.random(R * draws)) / (R * draws)).astype(np.float32).reshape(R, draws)
    args = dict(top_p=T(np.full(R, 0.9, np.float32)))
    tokens, lp = drawn(tsd, x, u, **args)
    rows = tsd.logits_filter(T(x), **args).cpu().numpy()
    probs = tsd.logits_filter(T(x), probs=True, **args).cpu().numpy()
    for r in range(R):
        check_row(x[r].astype(np.float64), (1.0, 0, float(np.float32(0.9)), 0.0), rows[r].astype(np.float64), probs[r].astype(np.float64), tokens[r], lp[r], u[r])
    for _ in range(20):
        again, again_lp = drawn(tsd, x, u, **args)
        assert np.array_equal(again, tokens) and np.array_equal(again_lp, lp)


@pytest.mark.parametrize("top_k", [0, 50, 700])
@pytest.mark.parametrize("V,p", [(200, -np.inf), (1000, -1e6), (5003, -1.0), (5003, -3e38), (32000, -np.inf), (262144, -1e6)])
def test_top_p_below_zero_keeps_rank_zero(tsd, V, p, top_k):
    """include/tsd.h: rank 0 is kept whatever p is.  Hundreds of logits lie within 32 of the maximum."""
    rng = np.random.default_rng(V)
    R = 3
    x = rows_of(rng, R, V, "plain")
    x[1] = np.round(x[1])  # the largest one more than once
    args = dict(top_p=T(np.full(R, p, np.float32)), top_k=T(np.full(R, top_k, np.int32)))
    best = x.argmax(1)  # (the lowest id of equal ones)
    tokens, lp = drawn(tsd, x, rng.random((R, 3)).astype(np.float32), **args)
    assert (tokens == best[:, None]).all() and (lp == 0).all()
    rows = tsd.logits_filter(T(x), **args).cpu().numpy()
    probs = tsd.logits_filter(T(x), probs=True, **args).cpu().numpy()
    want = np.full((R, V), -np.inf, np.float32)
    want[np.arange(R), best] = 0
    assert np.array_equal(rows, want) and np.array_equal(probs, np.exp(want))


def gap_row():
    """A maximum, 480 equal logits half a unit in front of what top-p 0.999 may still reach (a weight of 0.001 / V
    and 5%), 2099 behind it: nothing lies between, and the weight of all but the maximum is the share that
    top-p leaves out, to 10^-6."""
    V, n, p = 2580, 480, float(np.float32(0.999))
    near = np.log(V) - np.log(1 - p) + 0.05
    far = np.float32(near + 0.002)
    tail = lambda d: n * np.exp(-np.float64(np.float32(d))) + (V - 1 - n) * np.exp(-np.float64(far))
    lo, hi = near - 0.6, near  # the tail falls with d
    for _ in range(60):
        d = (lo + hi) / 2
        lo, hi = (d, hi) if tail(d) > (1 - p) * (1 + tail(d)) else (lo, d)
    assert abs(tail(lo) - (1 - p) * (1 + tail(lo))) < 1e-6 * tail(lo) and near - lo < 0.3
    x = np.full(V, -far, np.float32)
    x[1000:1000 + n] = -np.float32(lo)
    x[17] = 0.0
    return x, p


def thin_row():
    """A maximum, and 262143 logits behind it that together weigh less than the 2^-24 that top-p leaves out."""
    x = np.full(262144, -29.165, np.float32)
    x[200000] = 0.0
    assert np.exp(np.float64(x)).sum() * 2.0 ** -24 > 262143 * np.exp(np.float64(x[0])) * (1 + 2.0 ** -5)
    return x, 1 - 2.0 ** -24


@pytest.mark.parametrize("row", [gap_row, thin_row])
def test_top_p_next_to_what_it_cannot_reach(tsd, row):
    """Thousands of logits just below any that top-p may keep, in reach of the border's bins."""
    one, p = row()
    x = np.stack([one, one + np.float32(2), one])
    x[2, [0, 1]] = -np.inf
    args = dict(top_p=T(np.full(3, p, np.float32)))
    u = np.array([[0.0, 0.5, 1 - 2.0 ** -24]] * 3, np.float32)
    tokens, lp = drawn(tsd, x, u, **args)
    rows = tsd.logits_filter(T(x), **args).cpu().numpy()
    probs = tsd.logits_filter(T(x), probs=True, **args).cpu().numpy()
    for r in range(3):
        check_row(x[r].astype(np.float64), (1.0, 0, p, 0.0), rows[r].astype(np.float64), probs[r].astype(np.float64), tokens[r], lp[r], u[r])
