"""Attention with shared prefixes against the definition in fp64.

Tolerance.  K, V and q are exact; what rounds is
- a score's fp32 sum of D products: at most D 2^-24 times sum |q||k| scale, a relative
  change of a probability, and an absolute one of lse, by as much;
- the scores' product with the scale, ex2.approx, the fp32 row sums and the join:
  together below 2^-18 relative;
- P to bf16: 2^-8 relative, while the row sum adds it unrounded;
- out to bf16: 2^-8 relative.
So |out - ref| <= 2^-8 |ref| + (1 + 2^-8) (2^-8 + 2^-18 + 2 D 2^-24 score) sum p|v|, and
|lse - ref| <= D 2^-24 score + 2^-18 + 2^-22 |ref|, with score the largest sum
|q||k| scale of the row's keys.
"""

import numpy as np
import pytest

import gen
import oracle

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


NAN = 0x7FC0


def inputs(seed, N, Hq, Hkv, D, groups, nodes=None, hide=NAN):
    """groups: (S, own lengths of its sequences).  Whole shared blocks are the same
    blocks, a last, partly shared one is each sequence's copy; slots that hold no
    key are `hide`."""
    rng = np.random.default_rng(seed)
    first = np.concatenate([[0], np.cumsum([len(own) for _, own in groups])]).astype(np.int32)
    S = np.array([s for s, _ in groups], np.int32)
    P = np.array([s + o for s, own in groups for o in own], np.int32)
    B = len(P)
    n = np.array(nodes if nodes is not None else [N] * B, np.int32)
    parent = np.full((B, N), -1, np.int32)
    for b in range(B):
        parent[b, :n[b]] = gen.relabel(rng, gen.random_tree(rng, int(n[b]), 20)) if n[b] > 2 else gen.chain_tree(int(n[b]))
    _, _, mask, err = oracle.build_ancestors(parent, n, 32)
    assert (err == 0).all()
    need = (P + n + 15) // 16
    whole = S // 16
    total = int(whole.sum() + sum(need[b] - whole[g] for g in range(len(S)) for b in range(first[g], first[g + 1]))) + 3
    ids = list(rng.permutation(total))
    table = np.full((B, int(need.max()) + 1), -1, np.int32)
    pools = [np.full((total, Hkv, 16, D), hide, np.uint16) for _ in range(2)]
    for g in range(len(S)):
        if first[g] == first[g + 1]:
            continue
        common = [ids.pop() for _ in range(whole[g])]
        t = np.arange(S[g])
        shared = [gen.normal_bf16(rng, (len(t), Hkv, D)) for _ in pools]
        for b in range(first[g], first[g + 1]):
            table[b, :whole[g]] = common
            table[b, whole[g]:need[b]] = [ids.pop() for _ in range(need[b] - whole[g])]
            e = np.arange(S[g], P[b] + n[b])
            s = t if b == first[g] else t[whole[g] * 16:]  # (a copy of what the last block shares)
            for pool, x in zip(pools, shared):
                pool[table[b, s // 16], :, s % 16] = x[s]
                pool[table[b, e // 16], :, e % 16] = gen.normal_bf16(rng, (len(e), Hkv, D))
    return dict(q=gen.normal_bf16(rng, (B, N, Hq, D)), k=pools[0], v=pools[1], table=table, P=P, n=n, mask=mask, err=err,
                first=first, S=S, scale=1.0 / D ** 0.5, D=D)


def run(tsd, x, mask="tree", status=None, **kw):
    import torch
    out = torch.full(x["q"].shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full(x["q"].shape[:3], float("nan"), dtype=torch.float32, device="cuda")
    tsd.tree_attn_fwd_shared(bf(x["q"]), bf(x["k"]), bf(x["v"]), T(x["table"]), T(x["P"]), T(x["n"]),
                             T(x["mask"].view(np.int32)) if mask == "tree" else None, T(x["err"]), T(x["first"]), T(x["S"]),
                             scale=x["scale"], out=out, lse=lse, status=status, **kw)
    return out.double(), lse.double()


def reference(x, mask="tree"):
    """out, lse, sum p|v| and the largest sum |q||k| scale, fp64 on the GPU."""
    import torch
    q = bf(x["q"]).double()
    B, N, Hq, D = q.shape
    Hkv = x["k"].shape[1]
    g = Hq // Hkv
    kp, vp = bf(x["k"]), bf(x["v"])
    out, weight = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((B, N, Hq), -np.inf, dtype=torch.float64, device="cuda")
    score = torch.zeros_like(lse)
    for b in range(B):
        if x["err"][b]:
            continue
        P, n = int(x["P"][b]), int(x["n"][b])
        t = np.arange(P + n)
        page, row = T(x["table"][b][t // 16].astype(np.int64)), T(t % 16)
        k, v = (c[page, :, row].double() for c in (kp, vp))
        seen = np.ones((n, P + n), bool)
        j = np.arange(n)
        seen[:, P:] = (x["mask"][b, :n][:, j // 32] >> (j % 32)) & 1 if mask == "tree" else j[None, :] <= j[:, None]
        seen = T(seen)
        rows = q[b, :n].reshape(n, Hkv, g, D)
        s = torch.einsum("ihgd,thd->hgit", rows, k) * x["scale"]
        s = s.masked_fill(~seen, -np.inf)
        z = torch.logsumexp(s, -1)
        pr = torch.exp(s - z[..., None]).nan_to_num(0.0)
        out[b, :n] = torch.einsum("hgit,thd->ihgd", pr, v).reshape(n, Hq, D)
        weight[b, :n] = torch.einsum("hgit,thd->ihgd", pr, v.abs()).reshape(n, Hq, D)
        lse[b, :n] = z.permute(2, 0, 1).reshape(n, Hq)
        for h in range(Hkv):
            top = torch.einsum("igd,td->igt", rows[:, h].abs(), k[:, h].abs()).amax(-1) * x["scale"]
            score[b, :n, h * g:(h + 1) * g] = top
    return out, lse, weight, score


def check(x, got, lse, ref, rows=None):
    import torch
    r_out, r_lse, weight, score = ref
    D = x["D"]
    if rows is not None:
        got, lse, r_out, r_lse, weight, score = (a[rows] for a in (got, lse, r_out, r_lse, weight, score))
    off = (2.0 ** -8 + 2.0 ** -18 + 2 * D * 2.0 ** -24 * score[..., None]) * weight
    tol = 2.0 ** -8 * r_out.abs() + (1 + 2.0 ** -8) * off
    seen = torch.isfinite(r_lse)
    assert torch.equal(seen, torch.isfinite(lse)) and torch.isneginf(lse[~seen]).all()
    assert (got[~seen] == 0).all()
    d = (got - r_out).abs() - tol
    assert not (d > 0).any(), ((got - r_out).abs().max().item(), d.max().item())
    assert torch.isfinite(got).all()
    d = (lse[seen] - r_lse[seen]).abs() - (D * 2.0 ** -24 * score[seen] + 2.0 ** -18 + 2.0 ** -22 * r_lse[seen].abs())
    assert not (d > 0).any(), d.max().item()


SHAPES = [
    # N, Hq, Hkv, D, groups, nodes
    (1, 1, 1, 64, [(0, [0])], None),
    (1, 8, 1, 128, [(16, [0, 0])], None),
    (1, 8, 2, 128, [(1, [0, 5])], None),
    (1, 32, 8, 128, [(128, [1, 17, 300])], None),
    (1, 6, 2, 64, [(130, [0, 15, 16]), (77, [3])], None),
    (4, 16, 1, 128, [(300, [7, 0, 129, 64])], [4, 1, 3, 2]),
    (5, 7, 1, 64, [(0, [45, 3]), (31, [0, 1, 2])], [5, 4, 1, 2, 5]),
    (9, 4, 2, 128, [(639, [1, 1])], None),
    (16, 8, 2, 128, [(100, [0, 11]), (0, []), (257, [30, 31, 32])], [16, 3, 1, 16, 9]),
    (33, 4, 1, 128, [(63, [0, 63])], None),
    (31, 8, 4, 128, [(512, [7, 130]), (15, [1, 0])], [31, 30, 29, 1]),
    (64, 4, 2, 64, [(129, [127, 0, 1])], [64, 33, 2]),
    (127, 2, 1, 128, [(200, [10, 500])], [127, 65]),
    (256, 2, 2, 128, [(90, [40, 6])], [256, 255]),
    (256, 16, 1, 64, [(33, [0, 2])], [256, 17]),
    (40, 16, 1, 128, [(260, [0, 300, 17, 4])], [37, 40, 1, 9]),
    (100, 5, 1, 128, [(255, [1, 2])], None),
]


@pytest.mark.parametrize("N,Hq,Hkv,D,groups,nodes", SHAPES)
def test_shared_prefixes(tsd, N, Hq, Hkv, D, groups, nodes):
    x = inputs(N * Hq + D, N, Hq, Hkv, D, groups, nodes)
    st = status_word()
    check(x, *run(tsd, x, status=st), reference(x))
    assert int(st.item()) == 0
    if N <= 16:  # without a mask: chains
        check(x, *run(tsd, x, mask=None, status=st), reference(x, mask=None))
        assert int(st.item()) == 0


@pytest.mark.parametrize("N,Hq,Hkv,D,groups,nodes", [
    (1, 64, 8, 128, [(6000, list(range(3, 3 + 40 * 29, 29)))], None),
    (1, 16, 8, 64, [(3000, [40] * 30), (517, list(range(40))), (0, [200, 9000])], None),
    (31, 32, 8, 128, [(2048, [64, 300, 1, 700]), (777, [5, 900])], [31, 17, 20, 1, 31, 16]),
    (127, 64, 8, 128, [(9001, [500, 3])], [127, 126]),
    (20, 48, 4, 64, [(1500, [0] * 12)], [20, 7, 1] * 4),
    (2, 8, 8, 128, [(40000, [1, 2, 3])], None),
])
def test_long_ranges(tsd, N, Hq, Hkv, D, groups, nodes):
    x = inputs(N * Hq + D, N, Hq, Hkv, D, groups, nodes, hide=0)
    got = run(tsd, x)
    check(x, *got, reference(x))
    again = run(tsd, x)  # the cuts do not depend on what runs when
    assert all((a == b).all() for a, b in zip(got, again))


def test_many_sequences(tsd):
    """The plan's largest batch, groups of every size among them."""
    rng = np.random.default_rng(0)
    groups, left = [], 1024
    while left:
        m = min(left, int(rng.integers(0, 40)))
        groups.append((int(rng.integers(0, 200)), list(rng.integers(0, 40, m))))
        left -= m
    x = inputs(1, 1, 2, 1, 64, groups, hide=0)
    check(x, *run(tsd, x), reference(x))


def test_same_as_without_sharing(tsd):
    x = inputs(3, 31, 8, 2, 128, [(700, [10, 40]), (64, [200, 1, 0])], [31, 9, 1, 30, 2])
    got, lse = run(tsd, x)
    ref = reference(x)
    alone = dict(x, S=np.zeros(2, np.int32))  # every sequence reads its own slots
    got2, lse2 = run(tsd, alone)
    check(x, got2, lse2, ref)
    each = dict(x, first=np.arange(6, dtype=np.int32), S=x["P"].copy())  # groups of one
    got3, lse3 = run(tsd, each)
    check(x, got3, lse3, ref)
    out, lse4 = tsd.tree_attn_fwd(bf(x["q"]), bf(np.where(x["k"] == NAN, 0, x["k"]).astype(np.uint16)),
                                  bf(np.where(x["v"] == NAN, 0, x["v"]).astype(np.uint16)), T(x["table"]), T(x["P"]), T(x["n"]),
                                  T(x["mask"].view(np.int32)), T(x["err"]), int((x["P"] + x["n"]).max()), scale=x["scale"])
    check(x, out.double(), lse4.double(), ref)


def test_rows_that_see_nothing(tsd):
    x = inputs(4, 8, 4, 2, 64, [(0, [0, 20]), (40, [0, 0])])
    x["mask"][0, 3] = 0
    x["mask"][1, 2] = 0
    x["mask"][2, 5] = 0
    got, lse = run(tsd, x)
    check(x, got, lse, reference(x))
    assert (lse[0, 3] == -np.inf).all() and (got[0, 3] == 0).all() and (lse[1, 2] > -np.inf).all()


@pytest.mark.parametrize("N,nodes", [(1, None), (40, [40, 12, 1])])
def test_nonfinite_tree_nodes_stay_in_their_branch(tsd, N, nodes):
    import torch
    x = inputs(5, N, 8, 2, 128, [(150, [9, 30, 0])], nodes)
    ref = reference(x)
    clean, _ = run(tsd, x)
    b, slot = 1, int(x["P"][1]) + (5 if N > 1 else 0)
    j = slot - int(x["P"][b])
    for bits, pool in ((0x7F80, "v"), (0xFF80, "v"), (NAN, "v"), (NAN, "k")):
        y = dict(x)
        y[pool] = x[pool].copy()
        y[pool][x["table"][b, slot // 16], 0, slot % 16, 77] = bits  # kv head 0
        got, lse = run(tsd, y)
        sees = torch.zeros(got.shape[:3], dtype=torch.bool, device="cuda")
        for i in range(int(x["n"][b])):
            sees[b, i, :4] = bool((int(x["mask"][b, i, j // 32]) >> (j % 32)) & 1)
        assert sees.any() and torch.isnan(got[sees]).all()
        assert torch.equal(got[~sees], clean[~sees])
        check(x, torch.where(sees[..., None], ref[0], got), torch.where(sees, ref[1], lse), ref)


def test_nan_query_stays_in_its_row(tsd):
    import torch
    x = inputs(6, 4, 8, 2, 64, [(150, [9, 30])])
    clean, _ = run(tsd, x)
    x["q"][1, 2, 3, 5] = NAN
    got, _ = run(tsd, x)
    rows = torch.ones(got.shape[:3], dtype=torch.bool, device="cuda")
    rows[1, 2, 3] = False
    assert torch.isnan(got[~rows]).all() and torch.equal(got[rows], clean[rows])


@pytest.mark.parametrize("scale", [1e-30, 1e-3, 30.0, 1e4])
def test_scales(tsd, scale):
    x = inputs(7, 6, 8, 2, 64, [(200, [9, 300])])
    x["scale"] = scale
    check(x, *run(tsd, x), reference(x))


def test_large_scores_move_the_reference(tsd):
    """Keys that grow along the pool: scores far above those of a chain's first tile."""
    x = inputs(8, 3, 4, 1, 64, [(1008, [500, 300])], hide=0)
    ramp = (np.arange(x["k"].shape[0]) % 61 * 3.0).astype(np.float32).reshape(-1, 1, 1, 1)
    x["k"] = gen.bf16_bits((oracle.bf16_to_f64(x["k"]) * ramp).astype(np.float32))
    check(x, *run(tsd, x), reference(x))


def test_skipped_sequences(tsd):
    import torch
    x = inputs(9, 4, 8, 2, 64, [(100, [9, 30, 2]), (20, [1, 2, 3]), (64, [5, 5])])
    x["err"] = x["err"].copy()
    x["err"][0] = 1   # the first of its group: another's table is read
    st = status_word()
    got, lse = run(tsd, x, status=st)
    ref = reference(x)
    check(x, got, lse, ref)
    assert int(st.item()) == 0
    bad = dict(x, P=x["P"].copy(), n=x["n"].copy())
    bad["P"][3] = 19          # shorter than the shared prefix
    bad["n"][4] = 0
    bad["P"][6] = 1 << 30     # beyond its table
    st = status_word()
    got, lse = run(tsd, bad, status=st)
    assert int(st.item()) == tsd.STATUS_BAD_LEN
    fine = [b for b in range(8) if b not in (0, 3, 4, 6)]
    check(x, got, lse, ref, rows=fine)
    for b in (0, 3, 4, 6):
        assert (got[b] == 0).all() and torch.isneginf(lse[b]).all()
    # a bad block in one's own range, and in a shared one
    for b, block, value, out in ((2, 100 // 16, -5, [0, 2]), (1, 2, x["k"].shape[0], [0, 1, 2]), (7, 64 // 16, 1 << 20, [0, 7])):
        y = dict(x, table=x["table"].copy())
        y["table"][b, block] = value
        st = status_word()
        got, lse = run(tsd, y, status=st)
        assert int(st.item()) == tsd.STATUS_BAD_PAGE
        check(x, got, lse, ref, rows=[c for c in range(8) if c not in out])
        for c in out:
            assert (got[c] == 0).all() and torch.isneginf(lse[c]).all()
    # entries past a sequence's range, and those that another sequence's table stands for, are not looked at
    y = dict(x, table=x["table"].copy())
    y["table"][2, :100 // 16] = -9
    y["table"][:, -1] = 1 << 29
    st = status_word()
    got, lse = run(tsd, y, status=st)
    assert int(st.item()) == 0
    check(x, got, lse, ref)


def test_bad_groups_skip_everything(tsd):
    import torch
    x = inputs(10, 2, 4, 2, 64, [(40, [1, 2]), (30, [3, 4, 5])])
    for first in ([1, 2, 5], [0, 2, 4], [0, 6, 5], [0, -1, 5], [0, 2, 1 << 30]):
        st = status_word()
        got, lse = run(tsd, dict(x, first=np.array(first, np.int32)), status=st)
        assert int(st.item()) == tsd.STATUS_BAD_LEN
        assert (got == 0).all() and torch.isneginf(lse).all()
    st = status_word()
    got, _ = run(tsd, dict(x, S=np.array([-1, 30], np.int32)), status=st)
    assert int(st.item()) == tsd.STATUS_BAD_LEN and (got[:2] == 0).all() and (got[2:] != 0).any()


def test_captured_and_replayed_with_other_lengths(tsd):
    import torch
    a = inputs(11, 5, 8, 2, 64, [(300, [20, 40, 3]), (50, [2])], [5, 3, 1, 4], hide=0)
    b = inputs(12, 5, 8, 2, 64, [(33, [5]), (700, [1, 100, 7])], [2, 5, 5, 1], hide=0)
    pages, cols = max(len(a["k"]), len(b["k"])), max(a["table"].shape[1], b["table"].shape[1])
    for x in (a, b):
        for name in "kv":
            x[name] = np.concatenate([x[name], np.zeros((pages - len(x[name]),) + x[name].shape[1:], np.uint16)])
        x["table"] = np.concatenate([x["table"], np.full((4, cols - x["table"].shape[1]), -1, np.int32)], 1)
    names = ["q", "k", "v", "table", "P", "n", "mask", "err", "first", "S"]
    load = lambda x: [bf(x[i]) if i in "qkv" else T(x[i].view(np.int32)) for i in names]  # noqa: E731
    args = load(a)
    ws = [torch.empty(tsd.tree_attn_shared_workspace_bytes(4, 5, 8, 2, 64, 2), dtype=torch.uint8, device="cuda") for _ in range(2)]
    out = [torch.empty_like(args[0]) for _ in range(2)]
    lse = [torch.empty((4, 5, 8), device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs = []
    tsd.tree_attn_fwd_shared(*args, out=out[0], lse=lse[0], workspace=ws[0])
    torch.cuda.synchronize()
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tsd.tree_attn_fwd_shared(*args, out=out[i], lse=lse[i], workspace=ws[i])
        graphs.append(g)
    for t, new in zip(args, load(b)):
        t.copy_(new)
    torch.cuda.synchronize()
    for g, s in zip(graphs, streams):  # two at once, each with its workspace
        with torch.cuda.stream(s):
            for _ in range(3):
                g.replay()
    torch.cuda.synchronize()
    ref = reference(b)
    for i in range(2):
        check(b, out[i].double(), lse[i].double(), ref)


def test_a_workspace_is_needed(tsd):
    import torch
    x = inputs(13, 1, 2, 1, 64, [(20, [1, 2])])
    with pytest.raises(tsd.TsdError):
        run(tsd, x, workspace=torch.empty(100, dtype=torch.uint8, device="cuda"))


def test_append_attend_commit(tsd):
    """Two steps of a group over one prompt: slots, the append with its rotation, the shared
    attention, the verification and the commit."""
    import torch
    rng = np.random.default_rng(14)
    B, N, Hq, Hkv, D, D_max, S = 3, 6, 8, 2, 64, 3, 75
    own = np.array([3, 20, 0], np.int32)
    P = T(S + own)
    blocks, max_blocks = 64, 10
    whole = S // 16
    held = (S + own + 15) // 16
    table = np.full((B, max_blocks), -1, np.int32)
    ids = list(range(blocks))
    common = [ids.pop() for _ in range(whole)]
    for b in range(B):
        table[b, :whole] = common
        table[b, whole:held[b]] = [ids.pop() for _ in range(held[b] - whole)]
    table, held = T(table), T(held.astype(np.int32))
    free = T(np.array(ids + [0] * (blocks - len(ids)), np.int32))
    count = T(np.array([len(ids)], np.int32))
    kc, vc = [torch.full((blocks, Hkv, 16, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    inv = T((10000.0 ** (-np.arange(D // 2) * 2.0 / D)).astype(np.float32))
    rows = lambda *s: bf(gen.normal_bf16(rng, s))  # noqa: E731

    def slots_of(b, t):
        return (table[b, t // 16] * 16 + t % 16).int().contiguous()

    t = torch.arange(S, device="cuda")
    prompt_k, prompt_v = rows(S, Hkv, D), rows(S, Hkv, D)
    for b in range(B):  # (the last, partly filled block is each sequence's own)
        tsd.kv_append_rope(None, prompt_k, prompt_v, slots_of(b, t), kc, vc, inv, t.int())
        if own[b]:
            e = torch.arange(S, S + int(own[b]), device="cuda")
            tsd.kv_append_rope(None, rows(int(own[b]), Hkv, D), rows(int(own[b]), Hkv, D), slots_of(b, e), kc, vc, inv, e.int())
    first, shared = T(np.array([0, B], np.int32)), T(np.array([S], np.int32))
    parent = T(np.array([[-1, 0, 0, 1, 1, 2], [-1, 0, 1, 2, -1, -1], [-1, 0, 0, 0, 1, 4]], np.int32))
    n = T(np.array([6, 4, 6], np.int32))
    tokens = T(rng.integers(0, 50, (B, N)).astype(np.int32))
    for _ in range(2):
        anc, depth, mask, err = tsd.tree_build_ancestors(parent, n, D_max)
        st = status_word()
        slots = tsd.kv_slots_build(P, n, N, table, held, free, count, status=st)
        q = tsd.kv_append_rope(rows(B, N, Hq, D), rows(B, N, Hkv, D), rows(B, N, Hkv, D), slots, kc, vc, inv, depth, base=P,
                               status=st)
        out, lse = tsd.tree_attn_fwd_shared(q, kc, vc, table, P, n, mask, err, first, shared, status=st)
        x = dict(q=q.view(torch.int16).cpu().numpy().view(np.uint16), table=table.cpu().numpy(), P=P.cpu().numpy(),
                 n=n.cpu().numpy(), mask=mask.cpu().numpy().view(np.uint32), err=err.cpu().numpy(), scale=D ** -0.5, D=D)
        x["k"], x["v"] = [c.view(torch.int16).cpu().numpy().view(np.uint16) for c in (kc, vc)]
        check(x, out.double(), lse.double(), reference(x))
        logits = T(rng.standard_normal((B, N, 50)).astype(np.float32))
        _, A, _, path, _ = tsd.tree_verify_greedy(logits, tokens, parent, anc, depth, mask, n, err, D_max)
        P, _ = tsd.kv_commit_path(kc, vc, table, P, n, A, path, err, N, D_max, status=st)
        assert int(st.item()) == 0


def test_wait_limit(tsd):
    """A wait that runs out (on a barrier that nothing signals) ends the call with a status; the next call is as before."""
    import torch
    x = inputs(15, 40, 8, 2, 128, [(300, [9, 30, 2])])
    before = run(tsd, x)
    old = tsd.get_option(tsd.OPT_WAIT_LIMIT_NS)
    st = status_word()
    try:
        tsd.set_option(tsd.OPT_WAIT_LIMIT_NS, 1_000_000)
        tsd.set_option(tsd.OPT_TEST_STALL, 1)
        run(tsd, x, status=st)
        torch.cuda.synchronize()
    finally:
        tsd.set_option(tsd.OPT_TEST_STALL, 0)
        tsd.set_option(tsd.OPT_WAIT_LIMIT_NS, old)
    assert int(st.item()) == tsd.STATUS_TIMEOUT
    after = run(tsd, x)
    assert all(torch.equal(a, b) for a, b in zip(before, after))


def test_pool_past_32_bit_offsets(tsd):
    """The same blocks 2^32 bytes further on: the same rows, bit for bit."""
    import torch
    x = inputs(51, 5, 16, 8, 128, [(300, [20, 40]), (17, [30])], hide=0)
    far = 2 ** 32 // (8 * 16 * 128 * 2)
    args = [bf(x["q"]), bf(x["k"]), bf(x["v"]), T(x["table"]), T(x["P"]), T(x["n"]), T(x["mask"].view(np.int32)), T(x["err"]),
            T(x["first"]), T(x["S"])]
    want = tsd.tree_attn_fwd_shared(*args)
    for i in (1, 2):
        small = args[i]
        args[i] = torch.empty((far + len(small),) + small.shape[1:], dtype=small.dtype, device="cuda")
        args[i][:len(small)] = float("nan")
        args[i][far:] = small
    args[3] = torch.where(args[3] >= 0, args[3] + far, args[3])
    got = tsd.tree_attn_fwd_shared(*args)
    live = torch.arange(5, device="cuda")[None] < args[5][:, None]
    for a, b in zip(want, got):
        assert torch.equal(a[live], b[live])


def test_one_prompt_of_many_tokens_in_two_groups_at_once(tsd):
    """Two calls at once on two streams, each with a workspace of its own."""
    import torch
    xs = [inputs(52, 3, 8, 2, 64, [(900, [1, 5, 9, 30])]), inputs(53, 7, 8, 2, 64, [(64, [2, 2]), (128, [700, 3])])]
    want = [run(tsd, x) for x in xs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run(tsd, xs[i]))
    torch.cuda.synchronize()
    for i, x in enumerate(xs):
        live = torch.arange(x["q"].shape[1], device="cuda")[None] < T(x["n"])[:, None]
        for out, lse in got[i]:
            assert torch.equal(out[live], want[i][0][live]) and torch.equal(lse[live], want[i][1][live])


@pytest.mark.parametrize("N,Hq,Hkv,D", [(31, 32, 8, 128), (40, 32, 8, 128), (9, 64, 8, 64), (70, 16, 16, 64)])
def test_more_ranges_than_blocks(tsd, N, Hq, Hkv, D):
    """Trees of many sequences: a block takes several ranges, or the ends of two."""
    rng = np.random.default_rng(N + Hq)
    groups = [(int(rng.integers(0, 900)), [int(o) for o in rng.integers(0, 400, m)]) for m in (9, 1, 0, 14)]
    x = inputs(N * Hq + D, N, Hq, Hkv, D, groups, [int(i) for i in rng.integers(1, N + 1, 24)])
    st = status_word()
    got = run(tsd, x, status=st)
    check(x, *got, reference(x))
    assert int(st.item()) == 0
    again = run(tsd, x)
    assert all((a.nan_to_num(7.0) == b.nan_to_num(7.0)).all() for a, b in zip(got, again))
