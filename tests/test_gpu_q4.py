"""The 4-bit cache's kernels, the slot map kernels and the log probability
kernels against the fp64 oracle, bit for bit where the result is a choice or a
stored value.

Attention tolerance.  Every value of K and V is exact; what rounds is
- q after its power-of-two scaling, to fp16: exact for elements within 2^-27 of
  the row's largest, else 2^-25 absolute where the row's largest is 2^13, i.e.
  2^-38 of it: nothing next to the fp32 sums;
- a score's fp32 sum of D products: at most D 2^-24 times sum |q||k| |scale|,
  which is a relative change of a probability by the same amount, and an
  absolute change of lse by at most it;
- ex2.approx, the scale's product and the fp32 row sums: together below
  2^-20 relative;
- P to fp16: 2^-11 relative, or 2^-25 absolute below 2^-14; the P of a row sum
  to 2^8 or more (the reference score's alone is 2^8), so a key's probability
  is off by at most 2^-33, and out by 2^-33 sum |v|;
- out to bf16: 2^-8 relative.
So |out - ref| <= 2^-8 |ref| + (2^-11 + 2^-19 + 2 D 2^-24 score) sum p|v| +
2^-33 sum |v| (times 1 + 2^-8 for the rounding of what is off), and
|lse - ref| <= D 2^-24 score + 2^-19 + 2^-22 |ref|, with score the largest sum
|q||k| |scale| of the row's keys.
"""

import numpy as np
import pytest

import gen
import oracle
from oracle import logprobs as ologp
from oracle import q4 as oq4
from oracle import slots as oslots

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tsd():
    import tree_speculative_decoding_virtual_gb300 as m
    return m


def T(a, dtype=None):
    from _gpu_path import dev_tensor
    return dev_tensor(a, dtype)


def bf(bits):
    import torch
    return T(bits, torch.bfloat16)


def status_word():
    import torch
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def np_of(t, dtype=None):
    from _gpu_path import to_np
    return to_np(t, dtype)


# ---------------------------------------------------------------------------
# writer and reader
# ---------------------------------------------------------------------------


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("tokens,Hkv,spread", [(1, 1, 0), (37, 3, 0), (200, 8, 0), (64, 2, 20)])
def test_write_and_read(tsd, tokens, Hkv, D, spread):
    rng = np.random.default_rng(tokens * D + spread)
    blocks = tokens // 16 + 3
    pools = [rng.integers(0, 256, (blocks, Hkv, 9 * D)).astype(np.uint8) for _ in range(2)]
    rows = []
    for _ in range(2):
        x = rng.standard_normal((tokens, Hkv, D)).astype(np.float32)
        if spread:  # magnitudes far beyond both ends of the scales
            x *= np.exp2(rng.integers(-spread, spread, (tokens, Hkv, D // 8, 1)).astype(np.float32)).repeat(8, -1).reshape(x.shape)
        rows.append(gen.bf16_bits(x))
    slots = rng.permutation(blocks * 16)[:tokens].astype(np.int32)
    slots[::7] = np.where(np.arange(0, tokens, 7) % 2 == 1, -1, slots[::7])
    kc, vc = T(pools[0]), T(pools[1])
    st = status_word()
    tsd.kv_write_q4(bf(rows[0]), bf(rows[1]), T(slots), kc, vc, status=st)
    for got, pool, x in zip((kc, vc), pools, rows):
        assert np.array_equal(np_of(got), oq4.write_rows(pool, x, slots))
    k, v = tsd.kv_read_q4(kc, vc, T(slots), status=st)
    for got, pool in zip((k, v), (kc, vc)):
        assert np.array_equal(oracle.bf16_to_f64(np_of(got, np.uint16)), oq4.read_rows(np_of(pool), slots))
    assert int(st.item()) == 0


def test_write_every_tie_and_special(tsd):
    """Each group: a largest value that fixes the scale, and the values around
    every code boundary of that scale; scale ties; NaN and infinities."""
    groups = []
    for byte in list(range(0, 0xE3, 5)) + [1, 7, 8, 9, 0xE1, 0xE2]:
        s = oq4.scale_values()[byte]
        mids = s * np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
        groups.append(np.concatenate([[6 * s], mids, -mids, [-0.0]]))
        for f in (6.375, 6.1875, 5.8125):
            groups.append(np.concatenate([[f * s], np.zeros(15)]))
    groups.append(np.array([np.nan, np.inf, -np.inf] + [1.0] * 13))
    groups.append(np.array([3.3e38, -3.3e38] + [1e-40] * 14))
    while len(groups) % 8:
        groups.append(np.zeros(16))
    x = gen.bf16_bits(np.array(groups, np.float32).reshape(-1, 1, 128))
    slots = np.arange(len(x), dtype=np.int32)
    pool = np.zeros(((len(x) + 15) // 16, 1, 9 * 128), np.uint8)
    kc, vc = T(pool), T(pool)
    st = status_word()
    tsd.kv_write_q4(bf(x), bf(x), T(slots), kc, vc, status=st)
    assert np.array_equal(np_of(kc), oq4.write_rows(pool, x, slots))
    assert np.array_equal(np_of(vc), np_of(kc))
    assert int(st.item()) == tsd.STATUS_NONFINITE


@pytest.mark.parametrize("amax", [6e-6, 3e-5, 3.7e-4, 0.011, 1.0, 5.8125, 100.0, 61440.0, 3e38])
def test_write_every_bf16(tsd, amax):
    """Groups of one largest value and 15 others, which together are every bf16
    value up to it, both signs and zeros."""
    top = int(gen.bf16_bits(np.array([amax], np.float32))[0])
    vals = np.concatenate([np.arange(top + 1), np.arange(top + 1) | 0x8000]).astype(np.uint16)
    vals = np.concatenate([vals, np.zeros(-len(vals) % (15 * 64), np.uint16)]).reshape(-1, 15)
    x = np.concatenate([np.full((len(vals), 1), top, np.uint16), vals], 1).reshape(-1, 8, 128)
    slots = np.arange(len(x), dtype=np.int32)
    pool = np.zeros(((len(x) + 15) // 16, 8, 9 * 128), np.uint8)
    kc, vc = T(pool), T(pool)
    flipped = x ^ 0x8000
    st = status_word()
    tsd.kv_write_q4(bf(x), bf(flipped), T(slots), kc, vc, status=st)
    assert np.array_equal(np_of(kc), oq4.write_rows(pool, x, slots))
    assert np.array_equal(np_of(vc), oq4.write_rows(pool, flipped, slots))
    assert int(st.item()) == 0


def test_write_strided_and_bad_slots(tsd):
    import torch
    rng = np.random.default_rng(5)
    fused = gen.normal_bf16(rng, (9, 3 * 256))
    f = bf(fused)
    k, v = f[:, 256:512].unflatten(1, (2, 128)), f[:, 512:].unflatten(1, (2, 128))
    pool = rng.integers(0, 256, (2, 2, 9 * 128)).astype(np.uint8)
    kc, vc = T(pool), T(pool)
    slots = np.array([31, 0, -1, 32, -7, 5, 2 ** 31 - 1, 17, 16], np.int32)
    st = status_word()
    tsd.kv_write_q4(k, v, T(slots), kc, vc, status=st)
    assert np.array_equal(np_of(kc), oq4.write_rows(pool, fused[:, 256:512].reshape(9, 2, 128), slots))
    assert np.array_equal(np_of(vc), oq4.write_rows(pool, fused[:, 512:].reshape(9, 2, 128), slots))
    assert int(st.item()) == tsd.STATUS_BAD_PAGE
    st.zero_()
    k1, _ = tsd.kv_read_q4(kc, vc, T(slots), status=st)
    assert np.array_equal(oracle.bf16_to_f64(np_of(k1, np.uint16)), oq4.read_rows(np_of(kc), slots))
    assert int(st.item()) == tsd.STATUS_BAD_PAGE
    empty = torch.empty((0, 2, 128), dtype=torch.bfloat16, device="cuda")
    tsd.kv_write_q4(empty, empty, T(slots[:0]), kc, vc)
    assert tsd.kv_read_q4(kc, vc, T(slots[:0]))[0].shape == (0, 2, 128)


# ---------------------------------------------------------------------------
# slots
# ---------------------------------------------------------------------------


@pytest.mark.parametrize("B,N,P_max", [(1, 1, 0), (1, 63, 4096), (3, 7, 50), (64, 31, 300), (65, 31, 300), (64, 128, 90), (3, 2001, 5000), (64, 700, 900), (1, 8192, 100), (2, 4099, 40),
                                       (5, 4097, 2000), (1500, 3, 60), (2, 0, 70), (300, 37, 0)])
@pytest.mark.parametrize("tight", [False, True])
def test_slots_build_and_release(tsd, B, N, P_max, tight):
    rng = np.random.default_rng(B + N)
    P = rng.integers(0, P_max + 1, B).astype(np.int32)
    n = rng.integers(0, N + 1, B).astype(np.int32) if N % 2 else None
    new = n if n is not None else np.full(B, N)
    have = (P + 15) // 16
    # some sequences hold more than their prefix needs, some nothing at all
    held = np.where(rng.random(B) < 0.2, have + 2, np.where(rng.random(B) < 0.1, 0, have)).astype(np.int32)
    max_blocks = int(max((P + new + 15).max() // 16, held.max(), 1))
    need = np.maximum(0, (P + new + 15) // 16 - held)
    total = int(held.sum() + need.sum()) + 5
    ids = rng.permutation(total).astype(np.int32)
    table = np.full((B, max_blocks), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    count = total - at
    if tight:
        count = int(need.sum()) // 2
        if B > 2:
            P[B // 2] = -3
    free = rng.integers(0, total, total).astype(np.int32)
    free[:count] = ids[at:at + count]
    d = [T(x) for x in (table, held, free, np.array([count], np.int32))]
    st = status_word()
    got = tsd.kv_slots_build(T(P), None if n is None else T(n), N, *d, status=st)
    slots, t1, h1, c1, s1 = oslots.slots_build(P, n, N, table, held, free, count)
    assert np.array_equal(np_of(got), slots) and np.array_equal(np_of(d[0]), t1)
    assert np.array_equal(np_of(d[1]), h1) and int(d[3].item()) == c1 and int(st.item()) == s1
    assert np.array_equal(np_of(d[2]), free)
    keep = np.where(rng.random(B) < 0.3, 0, np.maximum(P, 0)).astype(np.int32)
    st.zero_()
    tsd.kv_blocks_release(T(keep), *d, status=st)
    t2, h2, f2, c2, s2 = oslots.blocks_release(keep, t1, h1, free, c1)
    assert np.array_equal(np_of(d[0]), t2) and np.array_equal(np_of(d[1]), h2)
    assert np.array_equal(np_of(d[2]), f2) and int(d[3].item()) == c2 and int(st.item()) == s2


@pytest.mark.parametrize("B", [3, 70])
def test_slots_fail_closed(tsd, B):
    """Bad free lists, counts, held numbers and tables: nothing out of range is
    handed out, and the status says what was wrong."""
    rng = np.random.default_rng(B)
    for case in ["count high", "count low", "bad ids", "held", "full list", "table"]:
        P = np.full(B, 16, np.int32)
        held = np.ones(B, np.int32)
        table = np.full((B, 4), -1, np.int32)
        table[:, 0] = np.arange(B)
        free = rng.permutation(np.arange(B, 4 * B)).astype(np.int32)
        free = np.concatenate([free, np.zeros(B, np.int32)])
        count = 3 * B
        if case == "count high":
            count = 4 * B + 1
        elif case == "count low":
            count = -1
        elif case == "bad ids":
            free[1::2] = 10 ** 6
        elif case == "held":
            held[1] = 9
            held[2] = -1
        elif case == "table":
            P[:] = 14
            table[0, 0] = -5
            table[1, 0] = 4 * B
        if case == "full list":
            keep = np.zeros(B, np.int32)
            count = 3 * B + 1
            d = [T(x) for x in (table, held, free, np.array([count], np.int32))]
            st = status_word()
            tsd.kv_blocks_release(T(keep), *d, status=st)
            t, h, f, c, s = oslots.blocks_release(keep, table, held, free, count)
            assert s == tsd.STATUS_BAD_LEN and int(st.item()) == s and int(d[3].item()) == c
            assert np.array_equal(np_of(d[0]), t) and np.array_equal(np_of(d[1]), h) and np.array_equal(np_of(d[2]), f)
            continue
        d = [T(x) for x in (table, held, free, np.array([count], np.int32))]
        st = status_word()
        got = tsd.kv_slots_build(T(P), None, 18, *d, status=st)
        slots, t, h, c, s = oslots.slots_build(P, None, 18, table, held, free, count)
        assert s != 0 and int(st.item()) == s, case
        assert np.array_equal(np_of(got), slots) and np.array_equal(np_of(d[0]), t), case
        assert np.array_equal(np_of(d[1]), h) and int(d[3].item()) == c, case


@pytest.mark.parametrize("count_ok", [True, False])
@pytest.mark.parametrize("B", [3, 70])  # one block, and scan and fill
def test_slots_of_a_sequence_that_needs_no_block(tsd, B, count_ok):
    """Behind sequences whose needs no longer fit, and with a count that is refused."""
    P = np.where(np.arange(B) % 3 == 2, 10, 16).astype(np.int32)
    table, held = np.full((B, 3), -1, np.int32), np.ones(B, np.int32)
    table[:, 0] = np.arange(B)
    free, count = np.full(B + 1, B, np.int32), 1 if count_ok else -1
    n = np.where(np.arange(B) % 3 == 2, 6, 20).astype(np.int32)
    d = [T(x) for x in (table, held, free, np.array([count], np.int32))]
    st = status_word()
    got = np_of(tsd.kv_slots_build(T(P), T(n), 20, *d, status=st))
    slots, t, h, c, s = oslots.slots_build(P, n, 20, table, held, free, count)
    assert int(st.item()) == s == (tsd.STATUS_NO_BLOCK if count_ok else tsd.STATUS_BAD_LEN)
    assert np.array_equal(got, slots) and np.array_equal(np_of(d[0]), t) and np.array_equal(np_of(d[1]), h)
    assert int(d[3].item()) == c == count and (got[2::3, :6] >= 0).all() and (got[0::3] == -1).all()


@pytest.mark.parametrize("B", [3, 70])  # a cluster, and scan and fill
def test_release_reports_bad_blocks(tsd, B):
    """A block id outside the pool that comes back is reported, keeps its place on
    the list as it stands, and is met again by the build that takes it."""
    rng = np.random.default_rng(B)
    blocks = 4 * B
    table, held = np.full((B, 4), -1, np.int32), np.ones(B, np.int32)
    table[:, 0] = np.arange(B)
    free = np.concatenate([rng.permutation(np.arange(B, blocks)), np.zeros(B)]).astype(np.int32)
    count = blocks - B
    free[[count - 1, count - 2 * B]] = [10 ** 6, -7]  # taken first and last
    table[B - 1, 0] = blocks
    d = [T(x) for x in (table, held, free, np.array([count], np.int32))]
    P = np.full(B, 16, np.int32)
    zero = np.zeros(B, np.int32)

    def build():
        nonlocal table, held, count
        st = status_word()
        got = tsd.kv_slots_build(T(P), None, 32, *d, status=st)
        slots, table, held, count, s = oslots.slots_build(P, None, 32, table, held, free, count)
        assert int(st.item()) == s == tsd.STATUS_BAD_PAGE
        assert np.array_equal(np_of(got), slots) and np.array_equal(np_of(d[0]), table)

    def release(keep):
        nonlocal table, held, free, count
        st = status_word()
        tsd.kv_blocks_release(T(keep), *d, status=st)
        table, held, free, count, s = oslots.blocks_release(keep, table, held, free, count)
        assert int(st.item()) == s
        for a, b in zip(d, (table, held, free, np.array([count]))):
            assert np.array_equal(np_of(a), b)
        return s

    build()
    assert release(np.full(B, 16, np.int32)) == tsd.STATUS_BAD_PAGE
    assert free[count - 1] == -1 and free[count - 2 * B] == -1
    build()
    assert release(zero) == tsd.STATUS_BAD_PAGE and count == blocks and (free == blocks).sum() == 1
    assert release(zero) == 0  # nothing comes back


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------


def _mask(parent, n_nodes, D_max=32):
    _, _, mask, err = oracle.build_ancestors(parent, n_nodes, D_max)
    return mask, err


def _attn_inputs(seed, B, N, Hq, Hkv, D, prefix, nodes, spare=1):
    rng = np.random.default_rng(seed)
    P = np.array(prefix, np.int32)
    n = np.array(nodes, np.int32)
    parent = np.full((B, N), -1, np.int32)
    for b in range(B):
        parent[b, :n[b]] = gen.relabel(rng, gen.random_tree(rng, int(n[b]), 20)) if n[b] > 2 else gen.chain_tree(int(n[b]))
    mask, err = _mask(parent, n)
    assert (err == 0).all()
    need = (P + n + 15) // 16
    blocks = int(need.sum()) + spare
    ids = rng.permutation(blocks).astype(np.int32)
    table = np.full((B, int(need.max()) + 1), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :need[b]] = ids[at:at + need[b]]
        at += need[b]
    pools = []
    for _ in range(2):
        # pages start as garbage (scale bytes above the largest among it), then
        # every slot of a sequence's range is written
        pool = rng.integers(0, 256, (blocks, Hkv, 9 * D)).astype(np.uint8)
        codes, scales = oq4.split_pages(pool)
        x = gen.normal_bf16(rng, (blocks, Hkv, 16, D))
        c, s = oq4.quantise_rows(x)
        for b in range(B):
            for t in range(int(P[b] + n[b])):
                pg = table[b, t // 16]
                codes[pg, :, t % 16], scales[pg, :, t % 16] = c[pg, :, t % 16], s[pg, :, t % 16]
        pools.append(pool)
    q = gen.normal_bf16(rng, (B, N, Hq, D))
    return dict(q=q, k=pools[0], v=pools[1], table=table, P=P, n=n, mask=mask, err=err, D=D,
                max_slots=int((P + n).max()), scale=1.0 / D ** 0.5)


def _run(tsd, x, mask="tree", max_slots=None, status=None, **kw):
    import torch
    m = T(x["mask"].view(np.int32)) if mask == "tree" else None
    out = torch.full(x["q"].shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full(x["q"].shape[:3], float("nan"), dtype=torch.float32, device="cuda")
    tsd.tree_attn_fwd_q4(bf(x["q"]), T(x["k"]), T(x["v"]), T(x["table"]), T(x["P"]), T(x["n"]), m, T(x["err"]),
                         max_slots or x["max_slots"], scale=x["scale"], out=out, lse=lse, status=status, **kw)
    return oracle.bf16_to_f64(np_of(out, np.uint16)), np_of(lse).astype(np.float64)


def _check(x, got, lse, ref):
    r_out, r_lse, weight, total, score = ref
    D = x["D"]
    off = (2.0 ** -11 + 2.0 ** -19 + 2 * D * 2.0 ** -24 * score[..., None]) * weight + 2.0 ** -33 * total
    tol = 2.0 ** -8 * np.abs(r_out) + (1 + 2.0 ** -8) * off
    seen = np.isfinite(r_lse)
    assert np.array_equal(seen, np.isfinite(lse)) and np.isneginf(lse[~seen]).all()
    assert (got[~seen] == 0).all()
    d = np.abs(got - r_out) - tol
    assert not (d > 0).any(), (np.abs(got - r_out).max(), d.max())
    d = np.abs(lse[seen] - r_lse[seen]) - (D * 2.0 ** -24 * score[seen] + 2.0 ** -19 + 2.0 ** -22 * np.abs(r_lse[seen]))
    assert not (d > 0).any(), d.max()


def _ref(x, mask="tree"):
    return oq4.tree_attention_q4(x["q"], x["k"], x["v"], x["table"], x["P"], x["n"], x["mask"] if mask == "tree" else None,
                                 x["err"], x["scale"])


SHAPES = [
    # B, N, Hq, Hkv, D, prefix, nodes
    (1, 1, 1, 1, 64, [0], [1]),
    (1, 1, 1, 1, 128, [0], [1]),
    (1, 1, 8, 1, 128, [15], [1]),
    (2, 1, 6, 2, 128, [16, 300], [1, 1]),
    (3, 1, 32, 2, 128, [1000, 31, 0], [1, 1, 1]),
    (1, 1, 4, 4, 64, [2049], [1]),
    (2, 2, 6, 2, 128, [77, 130], [2, 1]),
    (2, 5, 7, 1, 64, [45, 3], [5, 4]),
    (1, 9, 4, 2, 128, [639], [9]),
    (2, 16, 8, 2, 128, [100, 511], [16, 3]),
    (1, 33, 4, 1, 128, [63], [33]),
    (2, 31, 8, 4, 128, [512, 7], [31, 30]),
    (1, 64, 4, 2, 64, [129], [64]),
    (1, 127, 2, 1, 128, [200], [127]),
    (1, 256, 2, 2, 128, [90], [256]),
    (1, 40, 16, 1, 128, [260], [37]),
    (1, 100, 5, 1, 128, [255], [100]),
    (1, 130, 16, 8, 128, [1], [129]),
]


@pytest.fixture(params=[None, 262144], ids=["close", "far"])
def bound(request):
    """max_slots: the longest sequence, or far above it.  It decides which kernel
    runs: with the far one more than 16 rows always are the many-row kernel's."""
    return request.param


@pytest.mark.parametrize("B,N,Hq,Hkv,D,prefix,nodes", SHAPES)
def test_attention(tsd, B, N, Hq, Hkv, D, prefix, nodes):
    x = _attn_inputs(N * Hq + D, B, N, Hq, Hkv, D, prefix, nodes)
    st = status_word()
    got, lse = _run(tsd, x, status=st)
    _check(x, got, lse, _ref(x))
    assert int(st.item()) == 0
    # a looser bound on the lengths cuts the keys differently, and takes many rows to
    # the kernel for them
    for loose in (x["max_slots"] * 7 + 3000, 262144):
        got, lse = _run(tsd, x, max_slots=loose, status=st)
        _check(x, got, lse, _ref(x))
    assert int(st.item()) == 0


def _ref_on_gpu(x, chain=False):
    """tree_attention_q4 for long sequences, fp64 on the GPU (torch)."""
    import torch
    q = bf(x["q"]).double()
    B, N, Hq, D = q.shape
    Hkv = x["k"].shape[1]
    g = Hq // Hkv
    out, weight, total = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((B, N, Hq), -np.inf, dtype=torch.float64, device="cuda")
    score = torch.zeros_like(lse)
    for b in range(B):
        P, n = int(x["P"][b]), int(x["n"][b])
        slots = [int(x["table"][b, t // 16]) * 16 + t % 16 for t in range(P + n)]
        k, v = (T(oq4.read_rows(x[c], slots)) for c in "kv")
        seen = np.ones((n, P + n), bool)
        for i in range(n):
            seen[i, P:] = oq4.visible(None if chain else x["mask"], b, i, n, N)
        rows = q[b, :n].reshape(n, Hkv, g, D)
        s = torch.einsum("ihgd,thd->hgit", rows, k) * x["scale"]
        s = s.masked_fill(~T(seen), -np.inf)
        z = torch.logsumexp(s, -1)
        pr = torch.exp(s - z[..., None])
        out[b, :n] = torch.einsum("hgit,thd->ihgd", pr, v).reshape(n, Hq, D)
        weight[b, :n] = torch.einsum("hgit,thd->ihgd", pr, v.abs()).reshape(n, Hq, D)
        total[b, :n] = torch.einsum("it,thd->ihd", T(seen).double(), v.abs()).repeat_interleave(g, 1)
        lse[b, :n] = z.permute(2, 0, 1).reshape(n, Hq)
        for h in range(Hkv):
            top = torch.einsum("igd,td->igt", rows[:, h].abs(), k[:, h].abs()).amax(-1) * x["scale"]
            score[b, :n, h * g:(h + 1) * g] = top
    return tuple(t.cpu().numpy() for t in (out, lse, weight, total, score))


def _long_inputs(seed, B, N, Hq, Hkv, D, prefix, nodes):
    """_attn_inputs with whole pages of quantised values (fast for long
    sequences)."""
    rng = np.random.default_rng(seed)
    x = _attn_inputs(seed, B, N, Hq, Hkv, D, [0] * B, nodes)
    P, n = np.array(prefix, np.int32), np.array(nodes, np.int32)
    need = (P + n + 15) // 16
    ids = rng.permutation(int(need.sum()) + 3).astype(np.int32)
    table = np.full((B, int(need.max())), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :need[b]] = ids[at:at + need[b]]
        at += need[b]
    for name in "kv":
        pool = np.zeros((len(ids), Hkv, 9 * D), np.uint8)
        codes, scales = oq4.split_pages(pool)
        codes[:], scales[:] = oq4.quantise_rows(gen.normal_bf16(rng, (len(ids), Hkv, 16, D)))
        x[name] = pool
    x.update(P=P, table=table, max_slots=int((P + n).max()))
    return x


@pytest.mark.parametrize("B,N,Hq,Hkv,D,prefix,nodes", [
    (1, 1, 8, 1, 128, [20011], [1]),
    (3, 1, 32, 8, 128, [9000, 17, 4100], [1, 1, 1]),
    (64, 1, 16, 8, 64, list(range(3, 3 + 64 * 29, 29)), [1] * 64),
    (20, 4, 16, 8, 128, list(range(1000, 1000 + 20 * 61, 61)), [4, 1] * 10),
    (16, 31, 32, 8, 128, list(range(64, 64 + 16 * 190, 190)), [31, 17] * 8),
    (2, 127, 64, 8, 128, [5000, 2047], [127, 126]),
    (40, 33, 16, 4, 128, list(range(700, 700 + 40 * 37, 37)), [33, 9] * 20),
    (12, 100, 24, 8, 64, list(range(300, 300 + 12 * 333, 333)), [100, 65] * 6),
    (1, 256, 16, 1, 128, [12345], [255]),
    (5, 256, 128, 8, 128, [900, 1, 2000, 127, 128], [256, 255, 129, 1, 128]),
    (70, 1, 4, 1, 128, list(range(1, 1 + 70 * 37, 37)), [1] * 70),
    (66, 20, 4, 2, 64, list(range(5, 5 + 66 * 23, 23)), [20, 7, 1] * 22),
    (70, 20, 16, 4, 128, list(range(0, 70 * 3, 3)), [20, 7] * 35),  # one piece a range
    (3, 40, 16, 8, 128, [300, 40, 128], [40, 1, 39]),               # row blocks of 16, in clusters
    (1, 20, 8, 2, 64, [16000], [20]),
])
def test_attention_long(tsd, B, N, Hq, Hkv, D, prefix, nodes):
    x = _long_inputs(B + N, B, N, Hq, Hkv, D, prefix, nodes)
    st = status_word()
    got, lse = _run(tsd, x, status=st)
    _check(x, got, lse, _ref_on_gpu(x))
    assert int(st.item()) == 0
    got, lse = _run(tsd, x, mask=None, max_slots=2 * x["max_slots"])
    _check(x, got, lse, _ref_on_gpu(x, chain=True))


@pytest.mark.parametrize("B,N,Hq,Hkv,prefix", [
    (16, 31, 32, 8, list(range(64, 64 + 16 * 190, 190))),   # 128-row blocks: alternate key tiles
    (6, 100, 32, 8, [2000, 130, 900, 4000, 17, 1200]),      # 256-row blocks: two row tiles
    (24, 2, 32, 8, list(range(100, 100 + 24 * 173, 173))),  # the few-row kernel
])
def test_attention_repeats_exactly(tsd, B, N, Hq, Hkv, prefix):
    """The same call many times over, other work between: every result is the
    first one, bit for bit (a missing wait shows as a rare wrong tile)."""
    import torch
    x = _long_inputs(B, B, N, Hq, Hkv, 128, prefix, [N] * B)
    a = {k: T(v) for k, v in x.items() if k in ("k", "v", "table", "P", "n", "err")}
    q, m = bf(x["q"]), T(x["mask"].view(np.int32))
    noise = torch.empty(1 << 24, device="cuda")

    def call():
        return tsd.tree_attn_fwd_q4(q, a["k"], a["v"], a["table"], a["P"], a["n"], m, a["err"], x["max_slots"])

    out, lse = call()
    _check(x, oracle.bf16_to_f64(np_of(out, np.uint16)), np_of(lse).astype(np.float64), _ref_on_gpu(x))
    wrong = torch.zeros(1, dtype=torch.int64, device="cuda")
    for i in range(200):
        if i % 3 == 0:
            noise.normal_()  # other lines in L2
        o2, l2 = call()
        wrong += (o2.view(torch.int16) != out.view(torch.int16)).sum() + (l2 != lse).sum()
    assert int(wrong.item()) == 0


@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-30, 3.0])
@pytest.mark.parametrize("N", [1, 40])
def test_attention_scale(tsd, N, scale, bound):
    x = _attn_inputs(3, 1, N, 2, 1, 128, [150], [N])
    x["scale"] = scale
    got, lse = _run(tsd, x, max_slots=bound)
    _check(x, got, lse, _ref(x))


@pytest.mark.parametrize("N,Hq", [(1, 4), (6, 4), (40, 8), (200, 2)])
def test_attention_chain_mask(tsd, N, Hq, bound):
    x = _attn_inputs(N, 2, N, Hq, 2, 128, [70, 0], [N, max(1, N - 1)])
    got, lse = _run(tsd, x, mask=None, max_slots=bound)
    _check(x, got, lse, _ref(x, mask=None))


@pytest.mark.parametrize("N,Hq", [(3, 2), (20, 2), (90, 4)])
def test_attention_rows_that_see_nothing(tsd, N, Hq, bound):
    """No prefix and mask rows without a bit: 0 and -inf, whatever the other
    rows see."""
    x = _attn_inputs(N + 3, 2, N, Hq, 2, 64, [0, 40], [N, N])
    x["mask"][:, 1::2] = 0
    got, lse = _run(tsd, x, max_slots=bound)
    _check(x, got, lse, _ref(x))
    assert np.isneginf(lse[0, 1::2]).all() and np.isfinite(lse[1]).all()


@pytest.mark.parametrize("N,Hq", [(1, 8), (20, 8), (64, 8)])
def test_attention_value_ranges(tsd, N, Hq, bound):
    """Rows of q from 2^-130 to 2^100, all zero, and scores that rise along the
    keys so that the reference moves many times."""
    x = _attn_inputs(7 + N, 1, N, Hq, 1, 128, [700], [N])
    q = oracle.bf16_to_f64(x["q"])
    q[0, :, 0] *= 2.0 ** -130
    q[0, :, 1] = 0
    q[0, :, 2] *= 2.0 ** 30
    q[0, :, 3] *= 2.0 ** -20
    q[0, :, 4, ::2] *= 2.0 ** -24
    q[0, :, 5] = 1.0
    x["q"] = gen.bf16_bits(q.astype(np.float32))
    rng = np.random.default_rng(1)
    rows = rng.standard_normal((700 + N, 1, 128)).astype(np.float32) * 0.05
    rows += (np.arange(700 + N, dtype=np.float32) / 60)[:, None, None]
    slots = [int(x["table"][0, t // 16]) * 16 + t % 16 for t in range(700 + N)]
    x["k"] = oq4.write_rows(x["k"], gen.bf16_bits(rows), slots)
    got, lse = _run(tsd, x, max_slots=bound)
    _check(x, got, lse, _ref(x))


def test_attention_nan_query_stays_in_its_row(tsd, bound):
    for N in (1, 30, 64):
        x = _attn_inputs(11, 1, N, 4, 1, 128, [50], [N])
        ref = _ref(x)
        x["q"][0, 0, 2, 5] = 0x7FC0
        got, lse = _run(tsd, x, max_slots=bound)
        assert np.isnan(got[0, 0, 2]).all() and np.isnan(lse[0, 0, 2])
        keep = np.ones(lse.shape, bool)
        keep[0, 0, 2] = False
        got[~keep], lse[~keep] = ref[0][~keep], ref[1][~keep]
        _check(x, got, lse, ref)


@pytest.mark.parametrize("N,Hq", [(1, 4), (40, 8), (130, 4)])
def test_attention_skips_bad_sequences(tsd, N, Hq, bound):
    """Tree errors, lengths that do not fit and bad block ids: 0 / -inf rows and
    the status bit, the other sequences unharmed."""
    x = _attn_inputs(13 + N, 5, N, Hq, 2, 128, [100, 40, 333, 64, 20], [N] * 5)
    x["err"] = np.array([0, 4, 0, 0, 0], np.int32)
    x["table"][2, 7] = x["k"].shape[0]
    x["table"][3, 0] = -1
    x["n"][4] = N + 1
    st = status_word()
    got, lse = _run(tsd, x, max_slots=bound, status=st)
    assert int(st.item()) == tsd.STATUS_BAD_PAGE | tsd.STATUS_BAD_LEN
    y = dict(x, err=np.array([0, 1, 1, 1, 1], np.int32))
    _check(y, got, lse, _ref(y))
    # blocks past the sequence's range are never looked at
    z = dict(x, err=np.array([0, 1, 1, 1, 1], np.int32), table=x["table"].copy())
    z["table"][0, (100 + N + 15) // 16:] = 10 ** 9
    st.zero_()
    got, lse = _run(tsd, z, max_slots=bound, status=st)
    assert int(st.item()) == 0
    _check(z, got, lse, _ref(y))


def test_attention_is_deterministic_and_capturable(tsd, bound):
    import torch
    x = _attn_inputs(17, 2, 40, 8, 2, 128, [900, 333], [40, 22])
    a = {k: T(v) for k, v in x.items() if k in ("k", "v", "table", "P", "n", "err")}
    q, m = bf(x["q"]), T(x["mask"].view(np.int32))

    def call(stream=None):
        return tsd.tree_attn_fwd_q4(q, a["k"], a["v"], a["table"], a["P"], a["n"], m, a["err"], bound or x["max_slots"],
                                    stream=stream)

    out, lse = call()
    for _ in range(3):
        o2, l2 = call()
        assert torch.equal(out, o2) and torch.equal(lse, l2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o3, l3 = call(stream=side)
    o4, l4 = call(stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(out, o3) and torch.equal(lse, l3) and torch.equal(out, o4) and torch.equal(lse, l4)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o5, l5 = call()
    for _ in range(2):
        o5.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, o5) and torch.equal(lse, l5)


@pytest.mark.parametrize("N,Hq", [(1, 8), (5, 8), (40, 16)])
def test_attention_replayed_with_other_lengths(tsd, N, Hq, bound):
    """A captured call is cut up on the device: it holds for whatever lengths,
    errors and block tables its buffers have when it is replayed."""
    import torch
    prefixes = ([900, 333, 64], [1, 1200, 700], [15, 16, 17], [0, 1300, 0])
    x = _long_inputs(N, 3, N, Hq, 2, 128, [1300] * 3, [N] * 3)
    x["P"] = np.array(prefixes[0], np.int32)
    a = {k: T(v) for k, v in x.items() if k in ("k", "v", "table", "P", "n", "err")}
    q, m = bf(x["q"]), T(x["mask"].view(np.int32))
    out, lse = (torch.empty(x["q"].shape, dtype=torch.bfloat16, device="cuda"),
                torch.empty(x["q"].shape[:3], dtype=torch.float32, device="cuda"))

    def call():
        tsd.tree_attn_fwd_q4(q, a["k"], a["v"], a["table"], a["P"], a["n"], m, a["err"], bound or x["max_slots"],
                             scale=x["scale"], out=out, lse=lse)

    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for i, prefix in enumerate(prefixes):
        x["P"][:] = prefix
        x["n"][:] = [N, max(1, N - i), 1]
        x["err"][:] = [0, i == 2, 0]
        x["table"] = np.ascontiguousarray(np.roll(x["table"], 1, 0))
        for k in ("P", "n", "err", "table"):
            a[k].copy_(T(x[k]))
        out.fill_(float("nan"))
        lse.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        _check(x, oracle.bf16_to_f64(np_of(out, np.uint16)), np_of(lse).astype(np.float64), _ref(x))


def test_two_streams_at_once(tsd):
    """The calls of two streams overlap, each with what it allocates, and give what
    they give alone."""
    import torch
    xs = [_long_inputs(5, 8, 3, 16, 4, 128, list(range(500, 500 + 8 * 211, 211)), [3] * 8),
          _long_inputs(6, 6, 60, 16, 4, 128, list(range(700, 700 + 6 * 307, 307)), [60] * 6)]
    logits = torch.randn(40, 50000, device="cuda")
    tokens = torch.arange(40, dtype=torch.int32, device="cuda")
    args = []
    for x in xs:
        a = {k: T(v) for k, v in x.items() if k in ("k", "v", "table", "P", "n", "err")}
        args.append((bf(x["q"]), a["k"], a["v"], a["table"], a["P"], a["n"], T(x["mask"].view(np.int32)), a["err"],
                     x["max_slots"]))
    alone = [tsd.tree_attn_fwd_q4(*a) + tsd.token_logprobs(logits, tokens, k=7) for a in args]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i in (0, 1):
            got[i].append(tsd.tree_attn_fwd_q4(*args[i], stream=streams[i])
                          + tsd.token_logprobs(logits, tokens, k=7, stream=streams[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        for one in got[i]:
            assert all(torch.equal(x, y) for x, y in zip(one, alone[i]))


def test_blocks_beyond_four_gigabytes(tsd):
    """Blocks at the end of a pool of 4.6 GB: the byte offsets pass 32 bits."""
    import torch
    blocks, Hkv, D, P, N = 500000, 8, 128, 200, 6
    k, v = (torch.empty((blocks, Hkv, 9 * D), dtype=torch.uint8, device="cuda") for _ in range(2))
    need = (P + N + 15) // 16
    table = np.arange(blocks - 1, blocks - 1 - 7 * need, -7, dtype=np.int32)[None]
    slots = np.array([table[0, t // 16] * 16 + t % 16 for t in range(P + N)], np.int32)
    rng = np.random.default_rng(2)
    rows = [gen.normal_bf16(rng, (P + N, Hkv, D)) for _ in range(2)]
    st = status_word()
    tsd.kv_write_q4(bf(rows[0]), bf(rows[1]), T(slots), k, v, status=st)
    # the oracle has the last blocks only
    first = int(table.min())
    near = slots - first * 16
    pools = [oq4.write_rows(np.zeros((blocks - first, Hkv, 9 * D), np.uint8), r, near) for r in rows]
    for got, pool in zip(tsd.kv_read_q4(k, v, T(slots), status=st), pools):
        assert np.array_equal(oracle.bf16_to_f64(np_of(got, np.uint16)), oq4.read_rows(pool, near))
    mask, err = _mask(np.array([[-1, 0, 0, 1, 1, 2]], np.int32), np.array([N], np.int32))
    x = dict(q=gen.normal_bf16(rng, (1, N, 32, D)), k=pools[0], v=pools[1], table=table - first,
             P=np.array([P], np.int32), n=np.array([N], np.int32), mask=mask, err=err, D=D, max_slots=P + N,
             scale=0.09)
    ref = _ref(x)
    for bound in (P + N, 262144):
        out, lse = tsd.tree_attn_fwd_q4(bf(x["q"]), k, v, T(table), T(x["P"]), T(x["n"]), T(mask.view(np.int32)),
                                        T(err), bound, scale=0.09, status=st)
        _check(x, oracle.bf16_to_f64(np_of(out, np.uint16)), np_of(lse).astype(np.float64), ref)
    path, accept = np.array([[1, 3, 6, 0, 0]], np.int32), np.array([2], np.int32)
    new_len, moved = tsd.kv_commit_path_q4(k, v, T(table), T(x["P"]), T(x["n"]), T(accept), T(path), T(err), N, 4,
                                           status=st)
    ok, ov, o_len, o_moved = oq4.commit_path(pools[0], pools[1], x["table"], x["P"], accept, path, err)[:4]
    assert np.array_equal(np_of(new_len), o_len) and np.array_equal(np_of(moved), o_moved)
    for got, pool in zip((k, v), (ok, ov)):
        assert np.array_equal(np_of(got[table[0].astype(np.int64)]), pool[x["table"][0]])
    assert int(st.item()) == 0


@pytest.mark.parametrize("B,N,Hq,prefix", [(6, 100, 32, [2000, 130, 900, 4000, 17, 1200]),
                                           (16, 31, 32, list(range(64, 64 + 16 * 190, 190)))])
def test_attention_wait_limit(tsd, B, N, Hq, prefix):
    """A wait of the many-row kernel that runs out: the status says so, the kernel
    returns, and the next call is right."""
    import torch
    x = _long_inputs(B, B, N, Hq, 8, 128, prefix, [N] * B)
    st = status_word()
    old = tsd.get_option(tsd.OPT_WAIT_LIMIT_NS)
    try:
        tsd.set_option(tsd.OPT_WAIT_LIMIT_NS, 1_000_000)
        tsd.set_option(tsd.OPT_TEST_STALL, 1)
        _run(tsd, x, status=st)
        torch.cuda.synchronize()
    finally:
        tsd.set_option(tsd.OPT_TEST_STALL, 0)
        tsd.set_option(tsd.OPT_WAIT_LIMIT_NS, old)
    assert int(st.item()) == tsd.STATUS_TIMEOUT
    st.zero_()
    got, lse = _run(tsd, x, status=st)
    assert int(st.item()) == 0
    _check(x, got, lse, _ref_on_gpu(x))


# ---------------------------------------------------------------------------
# commit
# ---------------------------------------------------------------------------


@pytest.mark.parametrize("layers,B,N,Hkv,D,D_max", [(1, 1, 2, 1, 64, 1), (1, 5, 31, 3, 128, 5), (3, 4, 63, 2, 64, 8),
                                                    (2, 2, 200, 8, 128, 32)])
@pytest.mark.parametrize("own_base", [False, True])
def test_commit(tsd, layers, B, N, Hkv, D, D_max, own_base):
    rng = np.random.default_rng(N + D)
    P = rng.integers(0, 70, B).astype(np.int32)
    tail = (P + rng.integers(0, 40, B)).astype(np.int32) if own_base else None
    base = tail if own_base else P
    need = (base + N + 15) // 16
    ids = rng.permutation(int(need.sum()) + 2).astype(np.int32)
    table = np.zeros((B, int(need.max())), np.int32)
    path = np.zeros((B, D_max + 1), np.int32)
    A = np.zeros(B, np.int32)
    at = 0
    for b in range(B):
        table[b, :need[b]] = ids[at:at + need[b]]
        at += need[b]
        A[b] = rng.integers(0, min(D_max, N - 1) + 1)
        path[b, 0] = 1
        path[b, 1:A[b] + 1] = 2 + np.sort(rng.permutation(N - 1)[:A[b]])
    err = np.zeros(B, np.int32)
    if B > 2:
        err[1] = 2
    pools = [rng.integers(0, 256, (layers, len(ids), Hkv, 9 * D)).astype(np.uint8) for _ in range(2)]
    kc, vc = T(pools[0]), T(pools[1])
    st = status_word()
    new_len, moved = tsd.kv_commit_path_q4(kc, vc, T(table), T(P), None, T(A), T(path), T(err), N, D_max,
                                           tail_base=None if tail is None else T(tail), status=st)
    assert int(st.item()) == 0
    for layer in range(layers):
        k1, v1, r_len, r_moved = oq4.commit_path(pools[0][layer], pools[1][layer], table, P, A, path, err, tail)
        assert np.array_equal(np_of(kc)[layer], k1) and np.array_equal(np_of(vc)[layer], v1)
    assert np.array_equal(np_of(new_len), r_len) and np.array_equal(np_of(moved), r_moved)


def test_commit_fails_closed(tsd):
    rng = np.random.default_rng(3)
    pool = rng.integers(0, 256, (6, 2, 576)).astype(np.uint8)
    kc, vc = T(pool), T(pool)
    table = np.array([[0, 1], [2, 99], [3, 4]], np.int32)
    path = np.array([[1, 9, 0], [1, 4, 0], [1, 3, 2]], np.int32)  # node past the tree, bad block, fine
    st = status_word()
    new_len, _ = tsd.kv_commit_path_q4(kc, vc, T(table), T(np.array([5, 14, 3], np.int32)), None,
                                       T(np.array([1, 1, 2], np.int32)), T(path), None, 5, 2, status=st)
    assert int(st.item()) == tsd.STATUS_BAD_PATH | tsd.STATUS_BAD_PAGE
    assert np_of(new_len).tolist() == [5, 14, 6]
    k1, v1, _, _ = oq4.commit_path(pool, pool, table, [5, 14, 3], [1, 1, 2], path, [1, 1, 0])
    assert np.array_equal(np_of(kc), k1) and np.array_equal(np_of(vc), v1)


# ---------------------------------------------------------------------------
# log probabilities
# ---------------------------------------------------------------------------


def _check_rows(x, tokens, k, got):
    """x [R][V] fp64 (what the kernel read).  A logit difference and log S are
    rounded to fp32 (2^-24 relative each), ex2's argument too (d log2 e up to
    2^-24 relative, a probability's weight vanishing as |d| grows): below
    2^-20 absolute plus 2^-22 relative for |logits| up to 2^6."""
    lp, ent, ids, top = [np_of(t) for t in got]
    big = max(1.0, float(np.abs(x[np.isfinite(x)]).max()) if np.isfinite(x).any() else 1.0)
    tol = big * 2.0 ** -22 + 2.0 ** -20
    for r in range(len(x)):
        e_lp, e_ent, e_ids, e_top = ologp.row_logprobs(x[r], int(tokens[r]), k)
        assert np.array_equal(ids[r], e_ids), (r, ids[r], e_ids)
        for a, e in ((lp[r], e_lp), (ent[r], e_ent), (top[r], e_top)):
            a, e = np.atleast_1d(a).astype(np.float64), np.atleast_1d(e)
            fine = np.isfinite(e)
            assert np.array_equal(np.isnan(a), np.isnan(e)) and np.array_equal(np.isneginf(a), np.isneginf(e)), (r, a, e)
            assert (np.abs(a[fine] - e[fine]) <= tol + np.abs(e[fine]) * 2.0 ** -22).all(), (r, a[fine] - e[fine])


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("R,V,k", [(1, 1, 1), (1, 1, 0), (3, 7, 7), (2, 32, 32), (5, 1000, 5), (4, 8192, 20), (2, 8193, 32),
                                   (3, 32000, 8), (2, 128256, 20), (2, 151937, 32), (2, 262144, 4), (40, 333, 3)])
def test_logprobs(tsd, R, V, k, bf16):
    rng = np.random.default_rng(R + V)
    x = rng.standard_normal((R, V)).astype(np.float32) * 2
    tokens = rng.integers(0, V, R).astype(np.int32)
    if bf16:
        bits = gen.bf16_bits(x)
        logits, x = bf(bits), oracle.bf16_to_f64(bits)
    else:
        logits, x = T(x), x.astype(np.float64)
    _check_rows(x, tokens, k, tsd.token_logprobs(logits, T(tokens), k=k))


def test_logprobs_special_rows(tsd):
    """Ties of every length, masked vocabularies, ascending and descending rows,
    infinities, NaN, signed zeros and tokens out of range."""
    rng = np.random.default_rng(9)
    V, k = 20011, 32
    rows, tokens = [], []

    def add(row, token=5):
        rows.append(np.asarray(row, np.float32))
        tokens.append(token)

    add(np.zeros(V))
    add(np.full(V, -np.inf))
    add(np.full(V, -1e4))
    x = np.full(V, -np.inf)
    x[[7, 9000, 19999]] = [1, 3, 2]
    add(x, 9000)
    add(x, 8)
    x = np.full(V, -1e30)
    x[rng.permutation(V)[:40]] = rng.standard_normal(40)
    add(x)
    add(np.arange(V) * 1e-3, V - 1)
    add(-np.arange(V) * 1e-3, 0)
    add(np.where(np.arange(V) < V // 2, -50.0, rng.standard_normal(V)))
    add(np.round(rng.standard_normal(V) * 2))
    x = np.full(V, -1.0)
    x[::3] = 0.0
    x[::2] = -0.0
    add(x)
    x = rng.standard_normal(V)
    x[[3, 15000]] = np.nan
    add(x, 3)
    add(x, 100)
    x = rng.standard_normal(V)
    x[[4, 16000]] = np.inf
    add(x, 4)
    add(x, 100)
    add(rng.standard_normal(V), -1)
    add(rng.standard_normal(V), V)
    x = rng.standard_normal(V)
    x[12] = 60
    add(x, 12)
    add(x, 13)
    x = np.array(rows)
    got = tsd.token_logprobs(T(x), T(np.array(tokens, np.int32)), k=k)
    lp, ent, ids, top = [np_of(t) for t in got]
    for r in range(len(x)):  # logits up to 2^6 around the maximum, as _check_rows; far ones relative to themselves
        e = ologp.row_logprobs(x[r], tokens[r], k)
        assert np.array_equal(ids[r], e[2]), r
        for a, b in ((lp[r], e[0]), (ent[r], e[1]), (top[r], e[3])):
            a, b = np.atleast_1d(a).astype(np.float64), np.atleast_1d(b)
            assert np.array_equal(np.isnan(a), np.isnan(b)) and np.array_equal(np.isneginf(a), np.isneginf(b)), r
            fine = np.isfinite(b)
            assert (np.abs(a[fine] - b[fine]) <= 65 * 2.0 ** -22 + np.abs(b[fine]) * 2.0 ** -22).all(), (r, a, b)


def _masked_rows(rng, V, mask, n):
    """n rows of V logits, `mask` but for allowed ids that leave out the first
    chunk of 4096: twelve runs of 32 ids with logits in [0, 8], the even rows'
    largest ones before id 16384 (before a first settlement can raise the
    threshold) and all others 2 at most."""
    x = np.full((n, V), mask, np.float32)
    for r in range(n):
        for run in range(12):
            early = run < 6
            at = rng.integers(4096, 16384 - 32) if early else rng.integers(16384, V - 32)
            top = 8.0 if r % 2 or early else 2.0
            x[r, at:at + 32] = rng.uniform(6.0 if early and r % 2 == 0 else 0.0, top, 32)
    x[0] = mask  # and two ids alone
    x[0, [5000, 20000]] = [2, 1]
    return x


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("mask", [-np.inf, -100.0, -1e4, -1e30, -3.38e38])
@pytest.mark.parametrize("R,V", [(1, 128256), (20, 128256), (20, 128251), (160, 128256), (1, 262144)])
def test_logprobs_masked_vocabulary(tsd, R, V, mask, bf16):
    """Tolerance, in units of 2^-24: a term e^d of a sum has d from -8 to 8 (a
    reference is the mask, which has no weight next to an allowed logit, or an
    allowed logit), so 2 * 8 for d and its product with log2 e and 4 for ex2;
    as much for the factor of a warp and of a CTA; 384 terms and 24 levels of
    joining: 468 relative in S, so absolute in log S, and with logf's last place
    (16 at 14), the difference's (16) and the logits' (8) below 512.  The
    entropy's quotient is 8 at most and off by that much relative in numerator and
    denominator: 16 * 468 + 512 < 2^13.  Results far off zero round to 2^-24 of
    themselves, twice."""
    n = min(R, 6)
    x = _masked_rows(np.random.default_rng(R + V), V, mask, n)
    if bf16:
        bits = gen.bf16_bits(x)
        x = oracle.bf16_to_f64(bits)
    rows = np.arange(R) % n
    logits = bf(bits[rows]) if bf16 else T(x[rows])
    x = x.astype(np.float64)
    tokens = np.where(np.arange(n) % 3 == 0, 5000, np.argmax(x, axis=1)).astype(np.int32)
    want = [ologp.row_logprobs(x[r], int(tokens[r]), 32) for r in range(n)]
    for k in (0, 1, 5, 20, 32):
        lp, ent, ids, top = [np_of(t) for t in tsd.token_logprobs(logits, T(tokens[rows]), k=k)]
        for r in range(R):
            e_lp, e_ent, e_ids, e_top = want[rows[r]]
            assert np.array_equal(ids[r], e_ids[:k]), (k, r)
            for a, e, units in ((lp[r], e_lp, 512), (ent[r], e_ent, 8192), (top[r], e_top[:k], 512)):
                a, e = np.atleast_1d(a).astype(np.float64), np.atleast_1d(e)
                fine = np.isfinite(e)
                assert np.array_equal(np.isneginf(a), np.isneginf(e)), (k, r, a, e)
                assert (np.abs(a[fine] - e[fine]) <= units * 2.0 ** -24 + np.abs(e[fine]) * 2.0 ** -23).all(), (k, r, a, e)


def test_path_logprobs_masked_vocabulary(tsd):
    """The same rows on an accepted path (tolerance as above)."""
    V, D_max = 262144, 3
    x = _masked_rows(np.random.default_rng(4), V, -np.inf, 4).reshape(1, 4, V)
    best = np.argmax(x, axis=2).astype(np.int32)
    tokens = np.array([[9, best[0, 0], best[0, 1], best[0, 2]]], np.int32)
    path, A, bonus = np.array([[1, 2, 3, 4]], np.int32), np.array([3], np.int32), best[:, 3].copy()
    for k in (0, 1, 5):
        emitted, lp, ent, ids, top = [np_of(t) for t in tsd.tree_path_logprobs(T(x), T(tokens), T(path), T(A), T(bonus),
                                                                               None, D_max, k=k)]
        assert np.array_equal(emitted, best)
        for s in range(4):
            e_lp, e_ent, e_ids, e_top = ologp.row_logprobs(x[0, s], int(best[0, s]), k)
            assert abs(lp[0, s] - e_lp) <= 512 * 2.0 ** -24 and abs(ent[0, s] - e_ent) <= 8192 * 2.0 ** -24, (k, s)
            fine = np.isfinite(e_top)
            assert np.array_equal(ids[0, s], e_ids) and np.array_equal(np.isneginf(top[0, s]), ~fine), (k, s)
            assert (np.abs(top[0, s][fine] - e_top[fine]) <= 512 * 2.0 ** -24).all(), (k, s)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("V", [40008, 40011])  # through shared memory, and unaligned
@pytest.mark.parametrize("alone", [True, False])  # a cluster a row, and a CTA a row
def test_logprobs_special_rows_every_form(tsd, V, alone, bf16):
    """Masked first chunks, ties, infinities and NaN under every k and in every
    form of the kernel.  Tolerance, in units of 2^-24 (as for the masked rows):
    rows climb up to 40 above their reference, so d and its product 80, ex2 4, as much
    for two factors, 80 terms of a thread's sum, 24 levels: 356; logf, the
    difference and the logits 96 more: 512.  Entropy: two terms of up to 48, the quotient
    off by 2 * 356 relative: 48 * 712 + 512 < 2^16."""
    rng = np.random.default_rng(V)
    late = np.arange(V) >= 4096
    rows = []
    for mask in (-np.inf, -100.0, -1e4, -3.38e38):
        x = np.full(V, mask)
        x[[5000, 9001, 20128, 33000]] = [5, 4.5, 4, 3]
        rows.append(x)
        rows.append(np.where(late & (rng.random(V) < 0.01), rng.uniform(0, 8, V), mask))
        rows.append(np.where(late, np.minimum(np.round(rng.standard_normal(V) * 2), 4), mask))
        x = np.full(V, mask)
        x[7] = -60
        x[[4100, 16390, 39990]] = [0, 60, -20]
        rows.append(x)
    rows.append(np.full(V, -np.inf))
    rows.append(np.zeros(V))
    rows.append(np.arange(V) * (40 / V))
    rows.append(np.arange(V) * (-40 / V))
    rows.append(np.arange(V) * (300 / V))
    for special, at in ((np.nan, 3), (np.nan, 20000), (np.inf, 4), (np.inf, 20000)):
        x = rng.standard_normal(V)
        x[[at, 39999]] = special
        rows.append(x)
        rows.append(np.where(np.arange(V) == at, special, -np.inf))
    x = np.array(rows, np.float32)
    if bf16:
        bits = gen.bf16_bits(x)
        x = oracle.bf16_to_f64(bits)
    n = len(x)
    x64 = x.astype(np.float64)
    tokens = np.where(np.arange(n) % 2 == 0, 5000, 20128).astype(np.int32)
    want = [ologp.row_logprobs(x64[r], int(tokens[r]), 32) for r in range(n)]
    if alone:
        calls = [(np.array([r]), (bf(bits[r:r + 1]) if bf16 else T(x[r:r + 1]))) for r in range(n)]
    else:
        which = np.arange(3 * n) % n
        calls = [(which, bf(bits[which]) if bf16 else T(x[which]))]
    for which, logits in calls:
        for k in (0, 1, 5, 32):
            lp, ent, ids, top = [np_of(t) for t in tsd.token_logprobs(logits, T(tokens[which]), k=k)]
            for i, r in enumerate(which):
                e_lp, e_ent, e_ids, e_top = want[r]
                assert np.array_equal(ids[i], e_ids[:k]), (k, r)
                for a, e, units in ((lp[i], e_lp, 512), (ent[i], e_ent, 65536), (top[i], e_top[:k], 512)):
                    a, e = np.atleast_1d(a).astype(np.float64), np.atleast_1d(e)
                    fine = np.isfinite(e)
                    assert np.array_equal(np.isnan(a), np.isnan(e)), (k, r, a, e)
                    assert np.array_equal(np.isneginf(a), np.isneginf(e)), (k, r, a, e)
                    assert (np.abs(a[fine] - e[fine]) <= units * 2.0 ** -24 + np.abs(e[fine]) * 2.0 ** -23).all(), (k, r, a, e)


def test_logprobs_chosen_rows(tsd):
    rng = np.random.default_rng(10)
    x = rng.standard_normal((6, 501)).astype(np.float32)
    rows = np.array([5, -1, 0, 5, 6, -2], np.int32)
    tokens = np.array([1, 2, 3, 4, 5, 6], np.int32)
    st = status_word()
    lp, ent, ids, top = [np_of(t) for t in tsd.token_logprobs(T(x), T(tokens), rows=T(rows), k=3, status=st)]
    assert int(st.item()) == tsd.STATUS_BAD_PATH
    good = [0, 2, 3]
    _check_rows(x[rows[good]].astype(np.float64), tokens[good], 3,
                [T(np.ascontiguousarray(a[good])) for a in (lp, ent, ids, top)])
    for r in (1, 4, 5):
        assert lp[r] == 0 and ent[r] == 0 and (ids[r] == -1).all() and np.isneginf(top[r]).all()


@pytest.mark.parametrize("B,N,V,D_max,k", [(1, 5, 50, 3, 2), (4, 31, 3001, 6, 5), (3, 8, 40000, 0, 0)])
def test_path_logprobs(tsd, B, N, V, D_max, k):
    rng = np.random.default_rng(B * N)
    x = rng.standard_normal((B, N, V)).astype(np.float32)
    tokens = rng.integers(0, V, (B, N)).astype(np.int32)
    path = np.zeros((B, D_max + 1), np.int32)
    A = np.zeros(B, np.int32)
    for b in range(B):
        A[b] = min(D_max, N - 1) if b == 0 else rng.integers(0, min(D_max, N - 1) + 1)
        path[b, :A[b] + 1] = 1 + np.concatenate([[0], 1 + rng.permutation(N - 1)[:A[b]]])
    bonus = rng.integers(0, V, B).astype(np.int32)
    err = np.zeros(B, np.int32)
    if B > 1:
        err[B - 1] = 1
    emitted, lp, ent, ids, top = tsd.tree_path_logprobs(T(x), T(tokens), T(path), T(A), T(bonus), T(err), D_max, k=k)
    want = ologp.emitted_tokens(tokens, path, A, bonus, err)
    e = np.full((B, D_max + 1), -1, np.int32)
    for b, s, node, token in want:
        e[b, s] = token
    assert np.array_equal(np_of(emitted), e)
    at = ([w[0] for w in want], [w[1] for w in want])
    _check_rows(np.array([x[w[0], w[2]] for w in want], np.float64), [w[3] for w in want], k,
                [T(np.ascontiguousarray(np_of(t)[at])) for t in (lp, ent, ids, top)])
    none = e == -1
    assert (np_of(lp)[none] == 0).all() and (np_of(ids)[none] == -1).all()
    if B > 1:
        bad = path.copy()
        bad[0, A[0]] = N + 1
        st = status_word()
        out = tsd.tree_path_logprobs(T(x), T(tokens), T(bad), T(A), T(bonus), T(err), D_max, status=st)
        assert int(st.item()) == tsd.STATUS_BAD_PATH and int(out[0][0, A[0]].item()) == -1


# ---------------------------------------------------------------------------
# together, as a server's loop would use them
# ---------------------------------------------------------------------------


def test_verify_steps_over_a_4_bit_cache(tsd):
    """Prompts and two verify steps: every length, table, slot and cache byte
    stays on the GPU and equals the oracle's."""
    import torch
    rng = np.random.default_rng(21)
    B, N, Hq, Hkv, D, V, D_max, blocks, max_blocks = 4, 20, 8, 2, 64, 500, 6, 60, 12
    pools = [np.zeros((blocks, Hkv, 9 * D), np.uint8) for _ in range(2)]
    table, held = np.full((B, max_blocks), -1, np.int32), np.zeros(B, np.int32)
    free, count = rng.permutation(blocks).astype(np.int32), blocks
    kc, vc = T(pools[0]), T(pools[1])
    d = [T(x) for x in (table, held, free, np.array([count], np.int32))]
    st = status_word()

    def write(P, n, N_max, P_dev):
        nonlocal table, held, count
        slots = tsd.kv_slots_build(P_dev, T(n), N_max, *d, status=st)
        want, table, held, count, s = oslots.slots_build(P, n, N_max, table, held, free, count)
        assert s == 0 and np.array_equal(np_of(slots), want)
        k, v = gen.normal_bf16(rng, (B, N_max, Hkv, D)), gen.normal_bf16(rng, (B, N_max, Hkv, D))
        tsd.kv_write_q4(bf(k), bf(v), slots, kc, vc, status=st)
        for i, x in enumerate((k, v)):
            pools[i] = oq4.write_rows(pools[i], x.reshape(-1, Hkv, D), want.reshape(-1))

    prompt = np.array([37, 1, 90, 16], np.int32)
    P = np.zeros(B, np.int32)
    P_dev = T(P)
    write(P, prompt, 90, P_dev)
    P, P_dev = prompt, T(prompt)
    for step in range(2):
        parent = np.stack([gen.random_tree(rng, N, D_max) for _ in range(B)])
        n = np.full(B, N, np.int32)
        write(P, n, N, P_dev)
        anc, depth, mask, err = tsd.tree_build_ancestors(T(parent), T(n), D_max)
        _, _, o_mask, o_err = oracle.build_ancestors(parent, n, D_max)
        q = gen.normal_bf16(rng, (B, N, Hq, D))
        out, lse = tsd.tree_attn_fwd_q4(bf(q), kc, vc, d[0], P_dev, T(n), mask, err, max_blocks * 16, status=st)
        x = dict(q=q, k=pools[0], v=pools[1], table=table, P=P, n=n, mask=o_mask, err=o_err, D=D, scale=D ** -0.5)
        _check(x, oracle.bf16_to_f64(np_of(out, np.uint16)), np_of(lse).astype(np.float64), _ref(x))
        logits = rng.standard_normal((B, N, V)).astype(np.float32)
        targets = rng.integers(0, V, (B, N))
        gen.plant_targets(logits, targets)
        tokens = np.stack([gen.draft_tokens(rng, parent[b], targets[b], 0.8, V) for b in range(B)])
        am, A, leaf, path, bonus = tsd.tree_verify_greedy(T(logits), T(tokens), T(parent), anc, depth, mask, T(n), err,
                                                          D_max)
        _, o_A, _, o_path, o_bonus = oracle.verify_greedy(logits, tokens, parent, n, o_err, D_max)
        emitted, lp, ent, ids, top = tsd.tree_path_logprobs(T(logits), T(tokens), path, A, bonus, err, D_max, k=3,
                                                            status=st)
        for b, s, node, token in ologp.emitted_tokens(tokens, o_path, o_A, o_bonus, o_err):
            assert int(emitted[b, s]) == token
            assert token == int(ids[b, s, 0])  # greedy: what is emitted is the most probable token
            assert abs(float(lp[b, s]) - ologp.row_logprobs(logits[b, node], token, 0)[0]) < 1e-5
        new_len, moved = tsd.kv_commit_path_q4(kc, vc, d[0], P_dev, T(n), A, path, err, N, D_max, status=st)
        k1, v1, o_len, _ = oq4.commit_path(pools[0], pools[1], table, P, o_A, o_path, o_err)
        pools = [k1, v1]
        assert np.array_equal(np_of(kc), k1) and np.array_equal(np_of(vc), v1) and np.array_equal(np_of(new_len), o_len)
        tsd.kv_blocks_release(new_len, *d, status=st)
        table, held, free, count, s = oslots.blocks_release(o_len, table, held, free, count)
        assert np.array_equal(np_of(d[0]), table) and np.array_equal(np_of(d[2]), free) and int(d[3].item()) == count
        P, P_dev = o_len, new_len
    assert int(st.item()) == 0
    torch.cuda.synchronize()
