"""CPU checks of the append's and the sampling's oracles, and of the refusals of their
entry points and binding."""

import numpy as np
import pytest
import torch

import gen
from oracle import append, sampling
from oracle.attention import bf16_to_f64


def test_rotation_keeps_lengths_and_distances():
    rng = np.random.default_rng(0)
    x = gen.bf16_bits(rng.standard_normal((6, 2, 64)).astype(np.float32))
    inv = (10000.0 ** (-np.arange(32) / 32)).astype(np.float32)
    pos = np.arange(6)[None] * 7
    axis = np.zeros(32, np.int32)
    for pairs in (False, True):
        y = append.rotate(x, pos, inv, axis, interleaved=pairs)
        assert np.allclose((y ** 2).sum(-1), (bf16_to_f64(x) ** 2).sum(-1))
        # a product of two rotated rows depends on the distance of their positions alone
        z = append.rotate(x, pos + 1000, inv, axis, interleaved=pairs)
        assert np.allclose((y[0] * y[3]).sum(-1), (z[0] * z[3]).sum(-1))
        assert np.allclose(append.rotate(x, 0 * pos, inv, axis, interleaved=pairs), bf16_to_f64(x))


def test_norm_is_the_root_mean_square():
    rng = np.random.default_rng(1)
    x = gen.bf16_bits(rng.standard_normal((3, 1, 64)).astype(np.float32))
    one = gen.bf16_bits(np.ones(64, np.float32))
    y = append.rotate(x, np.zeros((1, 3), int), np.zeros(32, np.float32), np.zeros(32, int), one)
    assert np.allclose((y ** 2).mean(-1), 1.0)


def test_axes_turn_their_own_frequencies():
    x = gen.bf16_bits(np.ones((1, 1, 64), np.float32))
    inv = np.ones(32, np.float32)
    axis = np.arange(32) % 3
    y = append.rotate(x, np.array([[0], [1], [2]]), inv, axis)
    assert np.allclose(y[0, 0, :32], np.cos(axis) - np.sin(axis))


def test_kept_sets_against_definitions():
    rng = np.random.default_rng(2)
    for _ in range(50):
        x = np.round(rng.standard_normal(30), 1)
        x[rng.random(30) < 0.2] = -np.inf
        order = sampling.ranking(x)
        assert all(x[a] > x[b] or (x[a] == x[b] and a < b) for a, b in zip(order, order[1:]))
        k, p, m = int(rng.integers(0, 30)), float(rng.random()), float(rng.random() * 0.2)
        lo, hi = sampling.kept_bounds(x, 0.7, k, p, m)
        probs = torch.softmax(torch.from_numpy(x) / 0.7, -1).numpy()[order]
        n = len(order) if k == 0 else min(k, len(order))
        q = probs[:n] / probs[:n].sum()
        keep = [r == 0 or (q[:r].sum() < p and probs[r] >= m * probs[0]) for r in range(n)]
        assert lo == hi == sum(keep)
    assert sampling.kept_bounds(x, 0.0, 0, 0.5, 0.0) == (1, 1)
    assert sampling.kept_bounds(np.full(4, -np.inf)) == (0, 0)


def test_draws_tile_the_unit_interval():
    x = np.log(np.array([1.0, 2.0, 4.0, 1.0]))
    for u, token in ((0.0, 0), (0.124, 0), (0.126, 1), (0.4, 2), (0.99, 3)):
        assert [sampling.draw_ok(x, np.arange(4), t, u, 1.0, 1e-9) for t in range(4)] == [t == token for t in range(4)]


def _i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _append(t, q=(3, 4, 64), k=(3, 2, 64), v=(3, 2, 64), slots=3, pool=(4, 2, 16, 64), **kw):
    return t.kv_append_rope(_bf(*q), _bf(*k), _bf(*v), _i32(slots), _bf(*pool), _bf(*pool), **kw)


def _shared(t, q=(2, 1, 4, 64), pool=(4, 2, 16, 64), first=(2,)):
    return t.tree_attn_fwd_shared(_bf(*q), _bf(*pool), _bf(*pool), _i32(2, 3), _i32(2), None, None, None, _i32(*first),
                                  _i32(1))


REFUSED = {
    "cpu": lambda t: _append(t),
    "pool page": lambda t: _append(t, pool=(4, 2, 8, 64)),
    "heads": lambda t: _append(t, k=(3, 1, 64)),
    "tokens": lambda t: _append(t, q=(2, 4, 64)),
    "slots": lambda t: _append(t, slots=4),
    "4-bit page": lambda t: t.kv_append_rope_q4(None, _bf(3, 2, 64), _bf(3, 2, 64), _i32(3),
                                                *[torch.zeros(4, 2, 500, dtype=torch.uint8)] * 2),
    "4-bit layers": lambda t: t.kv_append_rope_q4(None, _bf(3, 2, 64), _bf(3, 2, 64), _i32(3),
                                                  *[torch.zeros(2, 4, 2, 576, dtype=torch.uint8)] * 2),
    "sample cpu": lambda t: t.token_sample(torch.zeros(2, 9), torch.zeros(2)),
    "sample dtype": lambda t: t.token_sample(torch.zeros(2, 9, dtype=torch.float16), torch.zeros(2)),
    "sample numbers": lambda t: t.token_sample(torch.zeros(2, 9), torch.zeros(3)),
    "sample settings": lambda t: t.token_sample(torch.zeros(6, 9), torch.zeros(6), temperature=torch.ones(4)),
    "sample settings differ": lambda t: t.token_sample(torch.zeros(6, 9), torch.zeros(6), temperature=torch.ones(3),
                                                       top_k=_i32(2)),
    "shared cpu": lambda t: _shared(t),
    "shared pool": lambda t: _shared(t, pool=(4, 2, 8, 64)),
    "shared head dim": lambda t: _shared(t, q=(2, 1, 4, 128)),
    "shared groups": lambda t: _shared(t, first=(3,)),
    "filter row": lambda t: t.logits_filter(torch.zeros(9)),
    "filter cpu": lambda t: t.logits_filter(torch.zeros(2, 9)),
}


@pytest.mark.parametrize("what", sorted(REFUSED))
def test_binding_refuses(what):
    import tree_speculative_decoding_virtual_gb300 as tsd
    with pytest.raises(tsd.TsdError):
        REFUSED[what](tsd)


def test_c_entry_points_check_before_any_launch():
    import tree_speculative_decoding_virtual_gb300 as tsd
    L, p = tsd.lib, 1 << 20  # a pointer that is never followed
    ARG, LIMIT = tsd.TSD_ERR_ARG, tsd.TSD_ERR_LIMIT

    def app(T=2, Hq=4, Hkv=2, D=64, R=64, axes=1, q=p, qs=256, ks=128, per=2, blocks=4, inv=p, eps=0.0, qo=p, fn=None):
        return (fn or L.tsd_kv_append_rope)(q, qs, p, ks, p, 128, p, T, Hq, Hkv, D, inv, R, None, axes, 0, 1.0, None,
                                            None, per, None, None, eps, blocks, p, p, qo, 256, None, None)

    for fn in (L.tsd_kv_append_rope, L.tsd_kv_append_rope_q4):
        assert app(T=0, fn=fn) == 0
        assert app(D=96, fn=fn) == LIMIT and app(R=48, fn=fn) == LIMIT and app(R=96, fn=fn) == LIMIT
        assert app(axes=5, fn=fn) == LIMIT and app(blocks=1 << 27, fn=fn) == LIMIT and app(T=1 << 31, fn=fn) == LIMIT
        assert app(T=-1, fn=fn) == ARG and app(q=None, fn=fn) == ARG and app(qo=None, fn=fn) == ARG
        assert app(q=p + 2, fn=fn) == ARG and app(qs=250, fn=fn) == ARG and app(ks=64, fn=fn) == ARG
        assert app(inv=None, fn=fn) == ARG and app(per=0, fn=fn) == ARG and app(axes=0, fn=fn) == ARG
        assert app(eps=-1.0, fn=fn) == ARG and app(eps=float("nan"), fn=fn) == ARG and app(blocks=0, fn=fn) == ARG

    def sample(R=1, rows=1, V=9, draws=1, per=1, x=p, u=p, chosen=None):
        return L.tsd_token_sample(x, 0, chosen, R, rows, V, u, draws, None, None, None, None, per, p, p, None, None)

    assert sample(R=0) == 0 and sample(R=2) == ARG and sample(V=0) == ARG and sample(V=262145) == LIMIT
    assert sample(draws=0) == ARG and sample(draws=65) == LIMIT and sample(per=0) == ARG and sample(x=None) == ARG
    assert sample(u=None) == ARG and sample(x=p + 2) == ARG and sample(R=-1) == ARG and sample(R=1 << 25, rows=1 << 25) == LIMIT

    def filt(R=1, V=9, x=p, out=p):
        return L.tsd_logits_filter(x, 0, R, V, 0, None, None, None, None, 1, out, None, None)

    assert filt(R=0) == 0 and filt(V=262145) == LIMIT and filt(x=None) == ARG and filt(out=None) == ARG
    assert filt(out=p + 2) == ARG and filt(R=-1) == ARG

    def attn(B=1, N=1, Hq=2, Hkv=2, D=64, G=1, scale=1.0, q=p, ws=None, ws_bytes=0, blocks=4, first=p):
        return L.tsd_tree_attn_fwd_shared(q, p, p, p, 2, blocks, p, None, None, None, first, p, G, B, N, Hq, Hkv, D, scale,
                                          p, None, ws, ws_bytes, None, None)

    assert attn(B=0, G=0) == 0
    assert attn(D=96) == LIMIT and attn(N=257) == LIMIT and attn(Hq=3) == LIMIT and attn(Hq=34) == LIMIT
    assert attn(B=1025) == LIMIT and attn(blocks=1 << 27) == LIMIT
    assert attn(G=0) == ARG and attn(G=2) == ARG and attn(q=None) == ARG and attn(q=p + 2) == ARG and attn(first=None) == ARG
    assert attn(scale=0.0) == ARG and attn(scale=float("nan")) == ARG and attn(blocks=0) == ARG
    need = L.tsd_tree_attn_shared_workspace_bytes(1, 1, 2, 2, 64, 1)
    assert need > 0 and L.tsd_tree_attn_shared_workspace_bytes(1, 1, 2, 2, 96, 1) == 0
    assert attn() == tsd.TSD_ERR_WORKSPACE and attn(ws=p, ws_bytes=need - 1) == tsd.TSD_ERR_WORKSPACE
    assert attn(ws=p + 4, ws_bytes=need) == ARG
