"""The append of rotated keys against the fp64 oracle.

Tolerance.  The fp32 work on a value: the norm's sum of D squares (D + 2 roundings,
half of it through the root), its reciprocal root (2^-22) and two products; cosine and
sine off by 2^-22 of 1 (the fraction of a turn is exact to 2^-24 before sincospif,
which is good to 2^-22); two products and a sum.  Together below 2^-16 of the pair's
magnitude |a| + |b|, times |scale|; then one rounding to bf16, 2^-8 relative.
"""

import numpy as np
import pytest

import gen
import oracle
from oracle import append as oap
from oracle import q4 as oq4

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


def np_of(t, dtype=None):
    from _gpu_path import to_np
    return to_np(t, dtype)


def status_word():
    import torch
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def freqs(R, theta=500000.0):
    return (theta ** (-np.arange(R // 2) * 2.0 / max(R, 1))).astype(np.float32)


def inputs(rng, tokens, Hq, Hkv, D, spread=0):
    def rows(H):
        x = rng.standard_normal((tokens, H, D)).astype(np.float32)
        if spread:
            x *= np.exp2(rng.integers(-spread, spread, (tokens, H, 1)).astype(np.float32))
        return gen.bf16_bits(x)
    return rows(Hq), rows(Hkv), rows(Hkv)


def near(got_bits, ref, mag):
    got = oracle.bf16_to_f64(got_bits)
    bound = np.abs(ref) * 2.0 ** -8 + mag * 2.0 ** -16
    assert (np.abs(got - ref) <= bound).all(), float((np.abs(got - ref) - bound).max())


def magnitude(x, weight, eps):
    """The largest |value| of a row after its norm: bounds any pair's |a| + |b| by twice it."""
    y = np.abs(oracle.bf16_to_f64(x))
    if weight is not None:
        y = y / np.sqrt((y ** 2).mean(-1, keepdims=True) + eps) * np.abs(oracle.bf16_to_f64(weight))
    return 2 * y.max(-1, keepdims=True)


@pytest.mark.parametrize("tokens,Hq,Hkv,D,R,axes,norm,pairs", [
    (1, 32, 8, 128, 128, 1, False, False), (1, 1, 1, 64, 64, 1, True, False), (31, 7, 1, 128, 64, 1, True, False),
    (33, 5, 5, 64, 32, 2, False, True), (257, 8, 2, 128, 128, 3, True, True), (1000, 16, 4, 128, 96, 3, True, False),
    (5000, 3, 3, 64, 64, 1, True, True), (16, 0, 8, 128, 128, 1, True, False), (77, 4, 2, 128, 0, 1, True, False),
    (40, 4, 2, 64, 0, 1, False, False)])
def test_append(tsd, tokens, Hq, Hkv, D, R, axes, norm, pairs):
    rng = np.random.default_rng(tokens + D + R)
    q, k, v = inputs(rng, tokens, Hq, Hkv, D, spread=3)
    blocks = tokens // 16 + 3
    pools = [gen.bf16_bits(rng.standard_normal((blocks, Hkv, 16, D)).astype(np.float32)) for _ in range(2)]
    slots = rng.permutation(blocks * 16)[:tokens].astype(np.int32)
    if tokens > 8:
        slots[::5] = -1
    # positions over the whole range, negative ones (a picture's offsets) among them
    pos = rng.integers(-1000, 262144, (axes, tokens)).astype(np.int32)
    inv = freqs(R)
    axis = rng.integers(0, axes, R // 2).astype(np.int32)
    eps = 1e-6
    qw, kw = [gen.bf16_bits((1 + 0.3 * rng.standard_normal(D)).astype(np.float32)) if norm else None for _ in range(2)]
    kc, vc = bf(pools[0]), bf(pools[1])
    st = status_word()
    out = tsd.kv_append_rope(bf(q) if Hq else None, bf(k), bf(v), T(slots), kc, vc, T(inv) if R else None,
                             T(pos if axes > 1 else pos[0]), freq_axis=T(axis) if axes > 1 else None,
                             q_weight=bf(qw) if norm else None, k_weight=bf(kw) if norm else None, eps=eps,
                             interleaved=pairs, status=st)
    assert int(st.item()) == 0
    at = axis if axes > 1 else np.zeros(R // 2, np.int32)
    if Hq:
        near(np_of(out, np.uint16), oap.rotate(q, pos, inv, at, qw, eps, pairs), magnitude(q, qw, eps))
    else:
        assert out is None
    got_k, got_v = np_of(kc, np.uint16), np_of(vc, np.uint16)
    here = slots >= 0
    page, row = slots[here] // 16, slots[here] % 16
    near(got_k[page, :, row], oap.rotate(k, pos, inv, at, kw, eps, pairs)[here], magnitude(k, kw, eps)[here])
    want_v = pools[1].copy()
    want_v[page, :, row] = v[here]
    assert np.array_equal(got_v, want_v)
    untouched = np.ones((blocks, 16), bool)
    untouched[page, row] = False
    assert np.array_equal(got_k.transpose(0, 2, 1, 3)[untouched], pools[0].transpose(0, 2, 1, 3)[untouched])


@pytest.mark.parametrize("tokens,Hkv,D,R,norm,pairs", [(1, 8, 128, 128, False, False), (61, 2, 64, 64, True, False),
                                                       (200, 3, 128, 64, True, False), (50, 2, 128, 96, False, True)])
def test_append_to_a_4_bit_cache(tsd, tokens, Hkv, D, R, norm, pairs):
    """The 4-bit pool is, byte for byte, what kv_write_q4 makes of the bf16 pool's rows."""
    rng = np.random.default_rng(tokens + D)
    q, k, v = inputs(rng, tokens, 2 * Hkv, Hkv, D, spread=5)
    blocks = tokens // 16 + 2
    slots = rng.permutation(blocks * 16)[:tokens].astype(np.int32)
    slots[3::7] = -1
    kw = bf(gen.bf16_bits((1 + 0.3 * rng.standard_normal(D)).astype(np.float32))) if norm else None
    pos = T(rng.integers(0, 262144, tokens).astype(np.int32))
    kc, vc = [bf(np.zeros((blocks, Hkv, 16, D), np.uint16)) for _ in range(2)]
    pool = rng.integers(0, 200, (blocks, Hkv, 9 * D)).astype(np.uint8)
    k4, v4 = T(pool), T(pool)
    args = dict(q_weight=kw, k_weight=kw, interleaved=pairs)
    q1 = tsd.kv_append_rope(bf(q), bf(k), bf(v), T(slots), kc, vc, T(freqs(R)), pos, **args)
    q2 = tsd.kv_append_rope_q4(bf(q), bf(k), bf(v), T(slots), k4, v4, T(freqs(R)), pos, **args)
    assert np.array_equal(np_of(q1, np.uint16), np_of(q2, np.uint16))
    here = slots >= 0
    for four, two in ((k4, kc), (v4, vc)):
        rows = np.zeros((tokens, Hkv, D), np.uint16)
        rows[here] = np_of(two, np.uint16)[slots[here] // 16, :, slots[here] % 16]
        assert np.array_equal(np_of(four), oq4.write_rows(pool, rows, slots))


def test_positions_of_trees_chains_and_far_tokens(tsd):
    """base + depth, base + place, and positions where an fp32 angle would be off by far more than the tolerance."""
    rng = np.random.default_rng(5)
    B, N, H, D = 3, 5, 2, 64
    q, k, v = inputs(rng, B * N, H, H, D)
    slots = np.full((B, N), -1, np.int32)
    base = np.array([0, 262139, 2 ** 31 - 100], np.int32)
    depth = rng.integers(0, 5, (B, N)).astype(np.int32)
    inv = freqs(D)
    kc = bf(np.zeros((1, H, 16, D), np.uint16))
    zero = np.zeros(D // 2, np.int32)
    shape = (B, N, H, D)
    for pos, want in ((depth, depth), (None, np.tile(np.arange(N), (B, 1)))):
        out = tsd.kv_append_rope(bf(q.reshape(shape)), bf(k.reshape(shape)), bf(v.reshape(shape)), T(slots), kc, kc,
                                 T(inv), T(pos) if pos is not None else None, base=T(base))
        p = (base[:, None].astype(np.int64) + want).reshape(1, -1)
        near(np_of(out, np.uint16).reshape(q.shape), oap.rotate(q, p, inv, zero), magnitude(q, None, 0))
    # without base: the place in each sequence, from the shape of slots
    out = tsd.kv_append_rope(bf(q.reshape(shape)), bf(k.reshape(shape)), bf(v.reshape(shape)), T(slots), kc, kc, T(inv))
    p = np.tile(np.arange(N), (B, 1)).reshape(1, -1)
    near(np_of(out, np.uint16).reshape(q.shape), oap.rotate(q, p, inv, zero), magnitude(q, None, 0))


def test_scale_and_large_frequencies(tsd):
    rng = np.random.default_rng(6)
    q, k, v = inputs(rng, 9, 2, 1, 64)
    inv = (rng.standard_normal(32) * 50).astype(np.float32)  # negative, and several turns a position
    pos = rng.integers(0, 4096, 9).astype(np.int32)
    kc = bf(np.zeros((1, 1, 16, 64), np.uint16))
    out = tsd.kv_append_rope(bf(q), bf(k), bf(v), T(np.full(9, -1, np.int32)), kc, kc, T(inv), T(pos), rot_scale=1.25)
    near(np_of(out, np.uint16), oap.rotate(q, pos[None], inv, np.zeros(32, np.int32), scale=1.25), 1.25 * magnitude(q, None, 0))


def test_strided_in_place_and_bad_slots(tsd):
    import torch
    rng = np.random.default_rng(7)
    tokens, Hq, Hkv, D = 50, 8, 2, 128
    qkv = bf(gen.bf16_bits(rng.standard_normal((tokens, Hq + 2 * Hkv, D)).astype(np.float32)))
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    slots = np.arange(tokens, dtype=np.int32)
    slots[4], slots[9] = 64, -7  # outside the pool of 4 blocks
    pos, inv = T(np.arange(tokens, dtype=np.int32)), T(freqs(D))
    pools = [bf(np.zeros((4, Hkv, 16, D), np.uint16)) for _ in range(4)]
    st = status_word()
    want = tsd.kv_append_rope(q.contiguous(), k.contiguous(), v.contiguous(), T(slots), pools[0], pools[1], inv, pos,
                              status=st)
    assert int(st.item()) == tsd.STATUS_BAD_PAGE
    before = qkv[:, Hq:].clone()
    got = tsd.kv_append_rope(q, k, v, T(slots), pools[2], pools[3], inv, pos, q_out=q)
    assert got.data_ptr() == q.data_ptr() and torch.equal(q, want)
    assert torch.equal(qkv[:, Hq:], before)
    assert torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])
    stored = np_of(pools[1], np.uint16).transpose(0, 2, 1, 3).reshape(64, Hkv, D)
    assert not stored[[4, 9]].any() and not stored[50:].any() and stored[[3, 5]].any()
    empty = tsd.kv_append_rope(q[:0], k[:0], v[:0], T(slots[:0]), pools[2], pools[3], inv, pos[:0])
    assert empty.shape == (0, Hq, D)


def test_nonfinite_rows_are_reported_by_the_4_bit_cache(tsd):
    rng = np.random.default_rng(8)
    q, k, v = inputs(rng, 4, 1, 1, 64)
    v[2, 0, 5] = 0x7FC0
    pool = T(np.zeros((1, 1, 9 * 64), np.uint8))
    st = status_word()
    tsd.kv_append_rope_q4(bf(q), bf(k), bf(v), T(np.arange(4, dtype=np.int32)), pool, pool.clone(), T(freqs(64)),
                          T(np.arange(4, dtype=np.int32)), status=st)
    assert int(st.item()) == tsd.STATUS_NONFINITE


def test_captured_and_replayed(tsd):
    import torch
    rng = np.random.default_rng(9)
    q, k, v = [bf(x) for x in inputs(rng, 20, 4, 2, 64)]
    slots, pos, inv = T(np.arange(20, dtype=np.int32)), T(np.arange(20, dtype=np.int32)), T(freqs(64))
    kc, vc = [bf(np.zeros((2, 2, 16, 64), np.uint16)) for _ in range(2)]
    out = torch.empty_like(q)
    tsd.kv_append_rope(q, k, v, slots, kc, vc, inv, pos, q_out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tsd.kv_append_rope(q, k, v, slots, kc, vc, inv, pos, q_out=out)
    pos += 1000
    slots += 7
    g.replay()
    got, gk = out.clone(), kc.clone()
    kc2, vc2 = [bf(np.zeros((2, 2, 16, 64), np.uint16)) for _ in range(2)]
    tsd.kv_append_rope(q, k, v, slots - 7, kc2, vc2, inv, pos - 1000)
    want = tsd.kv_append_rope(q, k, v, slots, kc2, vc2, inv, pos)
    assert torch.equal(got, want) and torch.equal(gk, kc2)


@pytest.mark.parametrize("q4", [False, True])
def test_pool_past_32_bit_offsets(tsd, q4):
    """Blocks whose byte offsets wrap to block 0 at 2^32 (bf16: 32 KB a block; 4 bits: 9 KB)."""
    import torch
    rng = np.random.default_rng(41)
    Hkv, D, few = 8, 128, 4
    shape = (Hkv, 9 * D) if q4 else (Hkv, 16, D)
    kind, block = (torch.uint8, Hkv * 9 * D) if q4 else (torch.bfloat16, Hkv * 16 * D * 2)
    far = -(-2 ** 32 // block)
    append = tsd.kv_append_rope_q4 if q4 else tsd.kv_append_rope
    q, k, v = [bf(x) for x in inputs(rng, 50, 4, Hkv, D)]
    slots = T(rng.permutation(few * 16)[:50].astype(np.int32))
    pos, inv = T(np.arange(50, dtype=np.int32)), T(freqs(D))
    small = [torch.zeros((few,) + shape, dtype=kind, device="cuda") for _ in range(2)]
    want = append(q, k, v, slots, *small, inv, pos)
    big = [torch.empty((far + few,) + shape, dtype=kind, device="cuda") for _ in range(2)]
    for pool in big:
        pool[:2 * few] = 0
        pool[far:] = 0
    got = append(q, k, v, slots + far * 16, *big, inv, pos)
    assert torch.equal(want, got)
    for a, b in zip(small, big):
        assert torch.equal(a, b[far:]) and not b[:2 * few].any()


def test_two_streams_at_once(tsd):
    import torch
    rng = np.random.default_rng(42)
    q, k, v = [bf(x) for x in inputs(rng, 300, 8, 2, 64)]
    pos, inv = T(np.arange(300, dtype=np.int32)), T(freqs(64))
    slots = [T(np.arange(300, dtype=np.int32) + 400 * i) for i in range(2)]
    pools = [torch.zeros((50, 2, 16, 64), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    want = [tsd.kv_append_rope(q, k, v, s, pools[0], pools[1], inv, pos) for s in slots]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [None, None]
    for i in range(2):  # into the same pool, other slots
        with torch.cuda.stream(streams[i]):
            got[i] = tsd.kv_append_rope(q, k, v, slots[i], pools[2], pools[3], inv, pos)
    torch.cuda.synchronize()
    assert torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def turn_fraction():
    """floor(2^400 / (2 pi)), pi by Machin's formula in whole numbers."""
    bits = 460

    def atan_inverse(n):
        total, term, k, sign = 0, (1 << bits) // n, 1, 1
        while term:
            total += sign * (term // k)
            term //= n * n
            k += 2
            sign = -sign
        return total

    pi = 4 * (4 * atan_inverse(5) - atan_inverse(239))
    return (1 << (400 + bits)) // (2 * pi)


@pytest.mark.parametrize("D,pairs", [(128, False), (64, True)])
def test_angles_of_far_positions_and_high_frequencies(tsd, D, pairs):
    """Rows of ones and zeros turn into cosines and sines of position times frequency.  The angle is exact to 2^-24
    of a turn (below 2^-21 radians), sincospif to 2^-22, and the result is rounded to bf16."""
    rng = np.random.default_rng(D)
    half, tokens = D // 2, 96
    inv = (10.0 ** rng.uniform(-8, 7, half) * rng.choice([-1, 1], half)).astype(np.float32)
    inv[:6] = [1.0, -100.0, 0.0, 1e-42, 1e18, -1e15]
    pos = rng.integers(-2 ** 31, 2 ** 31, tokens).astype(np.int32)
    pos[:4] = [2 ** 31 - 1, -2 ** 31, 0, 262144]
    x = np.zeros((tokens, 1, D), np.float32)
    x[..., np.arange(half) * 2 if pairs else np.arange(half)] = 1.0
    bits = gen.bf16_bits(x)
    kc = bf(np.zeros((1, 1, 16, D), np.uint16))
    out = tsd.kv_append_rope(bf(bits), bf(bits), bf(bits), T(np.full(tokens, -1, np.int32)), kc, kc, T(inv), T(pos),
                             interleaved=pairs)
    got = oracle.bf16_to_f64(np_of(out, np.uint16))[:, 0]
    got_cos, got_sin = (got[:, ::2], got[:, 1::2]) if pairs else (got[:, :half], got[:, half:])
    turn = turn_fraction()
    for f in range(half):
        num, den = float(inv[f]).as_integer_ratio()
        for t in range(tokens):
            # a fraction of a turn in 2^64ths, then in [-1/2, 1/2)
            z = ((num * int(pos[t]) * turn << 64) // (den << 400)) % (1 << 64)
            angle = 2 * np.pi * (z - (1 << 64) * (z >> 63)) / 2.0 ** 64
            for g, ref in ((got_cos[t, f], np.cos(angle)), (got_sin[t, f], np.sin(angle))):
                assert abs(g - ref) <= 2.0 ** -8 * abs(ref) + 2.0 ** -21 + 2.0 ** -22, (inv[f], pos[t], g, ref)


@pytest.mark.parametrize("tokens,Hkv,D,R,pairs", [(5003, 1, 128, 128, False), (2500, 2, 64, 32, True)])
def test_prompts_into_a_4_bit_cache(tsd, tokens, Hkv, D, R, pairs):
    """Prompts whose blocks take several tokens each, queries among them: as the smaller ones."""
    test_append_to_a_4_bit_cache(tsd, tokens, Hkv, D, R, True, pairs)
