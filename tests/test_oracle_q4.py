"""Pins of the 4-bit cache, slot map and log probability oracles (CPU), and the
refusals of the calls that need no GPU."""

import numpy as np
import pytest
import torch

import gen
from oracle import logprobs, q4, slots
from oracle.attention import bf16_to_f64


def test_scale_grid_is_the_half_grid():
    v = q4.scale_values()
    assert v[0] == 0 and v[1] == 2.0 ** -17 and v[8] == 2.0 ** -14 and v[0xE2] == 10240
    assert (np.diff(v) > 0).all() and 6 * v[-1] <= np.finfo(np.float16).max


def test_quantise_is_nearest_and_idempotent():
    rng = np.random.default_rng(0)
    x = gen.normal_bf16(rng, (64, 4, 128), 3.0)
    codes, scales = q4.quantise_rows(x)
    y = q4.dequantise_rows(codes, scales)
    xf = bf16_to_f64(x)
    s = np.repeat(q4.scale_values()[scales], 16, axis=-1)
    grid = np.concatenate([-q4.MAGNITUDES[::-1], q4.MAGNITUDES])
    best = np.abs(xf[..., None] - s[..., None] * grid).min(-1)
    assert np.allclose(np.abs(xf - y), best, rtol=0, atol=0)
    # values are exact in bf16, and storing them again changes nothing unless
    # the group's largest value moved
    again = q4.dequantise_rows(*q4.quantise_rows(gen.bf16_bits(y.astype(np.float32))))
    same = np.abs(y).reshape(-1, 16).max(-1) == 6 * q4.scale_values()[scales].reshape(-1)
    assert np.array_equal(again.reshape(-1, 16)[same], y.reshape(-1, 16)[same])


def test_ties_go_to_the_even_code_and_byte():
    # group maximum 6 -> scale 1: ties at the midpoints between codes
    vals = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5, -0.0]
    x = gen.bf16_bits(np.array(vals + [0] * 48, np.float32))[None]
    y = q4.dequantise_rows(*q4.quantise_rows(x))[0, :16]
    assert y.tolist() == [6, 0, 1, 1, 2, 2, 4, 4, 0, -1, -1, -2, -2, -4, -4, 0]
    # scale ties: 6 * 1.0625 lies between bytes 0x78 (1) and 0x79 (1.125)
    x = gen.bf16_bits(np.array([6.375] + [0] * 15 + [7.125] + [0] * 15 + [0] * 32, np.float32))[None]
    _, s = q4.quantise_rows(x)
    assert s[0, :3].tolist() == [0x78, 0x7A, 0]


def test_nonfinite_and_huge_inputs_stay_finite():
    x = gen.bf16_bits(np.array([np.nan, np.inf, -np.inf, 1.0] + [0] * 12 + [3e38] + [0] * 15 + [1e-30] + [0] * 31,
                               np.float32))[None]
    y = q4.dequantise_rows(*q4.quantise_rows(x))[0]
    assert y[:4].tolist() == [0, 61440, -61440, 0] and y[16] == 61440 and y[32] == 0


def test_attention_without_a_tree_is_softmax():
    rng = np.random.default_rng(1)
    pool = q4.write_rows(np.zeros((3, 2, 9 * 64), np.uint8), gen.normal_bf16(rng, (48, 2, 64)), np.arange(48))
    q = gen.normal_bf16(rng, (1, 1, 2, 64))
    table = np.array([[2, 0, 1]], np.int32)
    out, lse, _, _, _ = q4.tree_attention_q4(q, pool, pool, table, [36], None, None, None, 0.125)
    rows = torch.from_numpy(q4.read_rows(pool, [32 + i for i in range(16)] + list(range(16)) + list(range(16, 21))))
    x = torch.einsum("hd,thd->ht", torch.from_numpy(bf16_to_f64(q))[0, 0], rows) * 0.125
    ref = torch.einsum("ht,thd->hd", torch.softmax(x, -1), rows)
    assert np.allclose(out[0, 0], ref.numpy()) and np.allclose(lse[0, 0], torch.logsumexp(x, -1).numpy())


def test_slots_and_release_are_inverse():
    rng = np.random.default_rng(2)
    table = np.full((4, 9), -1, np.int32)
    free = rng.permutation(32).astype(np.int32)
    held = np.zeros(4, np.int32)
    P, n = np.array([0, 5, 40, 100]), np.array([17, 0, 3, 44])
    s, t2, h2, c2, st = slots.slots_build(P, n, 64, table, held, free, 32)
    assert st == 0 and h2.tolist() == [2, 1, 3, 9] and c2 == 32 - 15
    used = t2[t2 >= 0]
    assert len(set(used)) == 15 and set(used) == set(free[c2:])
    assert s[0, 16] == t2[0, 1] * 16 and s[3, 43] == t2[3, 8] * 16 + 15 and (s[1] == -1).all()
    t3, h3, f3, c3, st = slots.blocks_release(np.zeros(4, int), t2, h2, free, c2)
    assert st == 0 and c3 == 32 and (f3 == free).all() and (t3 == -1).all() and (h3 == 0).all()


def test_slots_fail_closed():
    free = np.arange(4, dtype=np.int32)
    table = np.full((3, 8), -1, np.int32)
    s, t, h, c, st = slots.slots_build([0, 0, 0], [32, 48, 0], 64, table, [0, 0, 0], free, 4)
    assert st == slots.NO_BLOCK and h.tolist() == [2, 0, 0] and c == 2 and (s[1] == -1).all()
    _, _, h, c, st = slots.slots_build([-1, 0, 200], None, 16, table, [0, 9, 0], free, 4)
    assert st == slots.BAD_LEN and h.tolist() == [0, 9, 0] and c == 4


def test_slots_of_a_sequence_that_needs_no_block():
    table, free = np.array([[0, -1, -1], [1, -1, -1], [2, -1, -1]], np.int32), np.array([3, 0, 0, 0], np.int32)
    s, t, h, c, st = slots.slots_build([16, 16, 10], [20, 4, 4], 20, table, [1, 1, 1], free, 1)
    assert st == slots.NO_BLOCK and (s[0] == -1).all() and (s[1] == -1).all()  # (the first one's need counts on)
    assert s[2].tolist() == [42, 43, 44, 45] + [-1] * 16 and h.tolist() == [1, 1, 1] and c == 1


def test_release_reports_bad_blocks():
    table, free = np.array([[2, -1, 9], [7, 1, 0]], np.int32), np.array([3, 0, 0, 0, 0, 0, 0], np.int32)
    t, h, f, c, st = slots.blocks_release([16, 32], table, np.array([3, 3]), free, 1)
    assert st == slots.BAD_PAGE and c == 4 and f[:4].tolist() == [3, 0, 9, -1]
    assert t.tolist() == [[2, -1, -1], [7, 1, -1]] and h.tolist() == [1, 2]  # (the bad id 7 stays held)
    assert slots.blocks_release([48, 32], table, np.array([3, 3]), free, 1)[4] == 0


def test_logprobs_against_torch():
    rng = np.random.default_rng(3)
    x = rng.standard_normal(1000) * 3
    lp, ent, ids, top = logprobs.row_logprobs(x, 17, 5)
    ref = torch.log_softmax(torch.from_numpy(x), -1)
    assert abs(lp - ref[17].item()) < 1e-12
    assert abs(ent - torch.distributions.Categorical(logits=torch.from_numpy(x)).entropy().item()) < 1e-10
    assert ids.tolist() == torch.topk(ref, 5).indices.tolist() and np.allclose(top, ref[ids].numpy())
    assert logprobs.row_logprobs(np.zeros(9), 3, 4)[2].tolist() == [0, 1, 2, 3]
    assert logprobs.row_logprobs(np.full(9, -np.inf), 3, 2)[:2] == (-np.inf, 0.0)


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------


def _i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _pool(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


REFUSED = {
    "cpu tensors": lambda t: t.kv_slots_build(_i32(2), None, 4, _i32(2, 3), _i32(2), _i32(6), _i32(1)),
    "table rows": lambda t: t.kv_slots_build(_i32(2), None, 4, _i32(3, 3), _i32(2), _i32(6), _i32(1)),
    "held dtype": lambda t: t.kv_slots_build(_i32(2), None, 4, _i32(2, 3), _i32(2).long(), _i32(6), _i32(1)),
    "release table": lambda t: t.kv_blocks_release(_i32(2), _i32(6), _i32(2), _i32(6), _i32(1)),
    "page size": lambda t: t.kv_write_q4(_bf(3, 2, 64), _bf(3, 2, 64), _i32(3), _pool(4, 2, 500), _pool(4, 2, 500)),
    "pools differ": lambda t: t.kv_write_q4(_bf(3, 2, 64), _bf(3, 2, 64), _i32(3), _pool(4, 2, 576), _pool(5, 2, 576)),
    "heads": lambda t: t.kv_write_q4(_bf(3, 1, 64), _bf(3, 2, 64), _i32(3), _pool(4, 2, 576), _pool(4, 2, 576)),
    "tokens": lambda t: t.kv_write_q4(_bf(3, 2, 64), _bf(3, 2, 64), _i32(4), _pool(4, 2, 576), _pool(4, 2, 576)),
    "head stride": lambda t: t.kv_write_q4(_bf(3, 4, 64)[:, ::2], _bf(3, 2, 64), _i32(3), _pool(4, 2, 576),
                                           _pool(4, 2, 576)),
    "uneven tokens": lambda t: t.kv_write_q4(_bf(2, 5, 2, 64)[:, :3], _bf(2, 3, 2, 64), _i32(6), _pool(4, 2, 576),
                                             _pool(4, 2, 576)),
    "a layer axis": lambda t: t.kv_write_q4(_bf(3, 2, 64), _bf(3, 2, 64), _i32(3), _pool(2, 4, 2, 576),
                                            _pool(2, 4, 2, 576)),
    "read on cpu": lambda t: t.kv_read_q4(_pool(4, 2, 576), _pool(4, 2, 576), _i32(3)),
    "commit path": lambda t: t.kv_commit_path_q4(_pool(4, 2, 576), _pool(4, 2, 576), _i32(1, 2), _i32(1), None, _i32(1),
                                                 _i32(1, 3), None, 4, 4),
    "q head dim": lambda t: t.tree_attn_fwd_q4(_bf(1, 1, 2, 128), _pool(4, 2, 576), _pool(4, 2, 576), _i32(1, 2),
                                               _i32(1), None, None, None, 16),
    "mask words": lambda t: t.tree_attn_fwd_q4(_bf(1, 33, 2, 64), _pool(4, 2, 576), _pool(4, 2, 576), _i32(1, 2),
                                               _i32(1), None, _i32(1, 33, 1), None, 16, out=_bf(1, 33, 2, 64)),
    "logits dtype": lambda t: t.token_logprobs(torch.zeros(2, 9, dtype=torch.float16), _i32(2)),
    "logits on cpu": lambda t: t.token_logprobs(torch.zeros(2, 9), _i32(2)),
    "path shape": lambda t: t.tree_path_logprobs(torch.zeros(1, 2, 9), _i32(1, 2), _i32(1, 3), _i32(1), _i32(1), None, 3),
}


@pytest.mark.parametrize("what", sorted(REFUSED))
def test_binding_refuses(what):
    import tree_speculative_decoding_virtual_gb300 as tsd
    with pytest.raises(tsd.TsdError):
        REFUSED[what](tsd)


def test_strided_tokens_are_understood():
    import tree_speculative_decoding_virtual_gb300 as tsd
    x = _bf(6, 512)[:, 128:256].unflatten(1, (2, 64))  # K inside a fused projection
    assert tsd._token_rows(x, 2, 64, "k") == (6, 512)
    assert tsd._token_rows(_bf(2, 3, 2, 64), 2, 64, "k") == (6, 128)
    assert tsd._token_rows(_bf(1, 2, 64), 2, 64, "k") == (1, 128)
    assert tsd._token_rows(_bf(0, 2, 64), 2, 64, "k")[0] == 0


def test_c_entry_points_check_before_any_launch():
    import tree_speculative_decoding_virtual_gb300 as tsd
    L, p = tsd.lib, 1 << 20  # a pointer that is never followed
    ARG, LIMIT, WS = tsd.TSD_ERR_ARG, tsd.TSD_ERR_LIMIT, tsd.TSD_ERR_WORKSPACE

    def attn(B=1, N=1, Hq=2, Hkv=2, D=64, slots=16, scale=1.0, q=p, ws=None, ws_bytes=0, num_blocks=4):
        return L.tsd_tree_attn_fwd_q4(q, p, p, p, 2, num_blocks, p, None, None, None, B, N, Hq, Hkv, D, slots, scale, p,
                                      None, ws, ws_bytes, None, None)

    assert attn(B=0) == 0
    assert attn(D=96) == LIMIT and attn(N=257) == LIMIT and attn(Hq=3) == LIMIT and attn(Hq=34) == LIMIT
    assert attn(slots=262145) == LIMIT and attn(B=65536) == LIMIT
    assert attn(q=None) == ARG and attn(q=p + 2) == ARG and attn(scale=float("nan")) == ARG and attn(num_blocks=0) == ARG
    assert attn(slots=65536) == WS
    assert L.tsd_tree_attn_q4_workspace_bytes(1, 1, 2, 2, 64, 65536) > 0
    assert L.tsd_tree_attn_q4_workspace_bytes(1, 1, 2, 2, 96, 65536) == 0

    def slots(B=1, N=4, max_blocks=2, num_blocks=4, out=p, ws=None):
        return L.tsd_kv_slots_build(p, None, B, N, p, max_blocks, p, p, p, num_blocks, out, ws, 0, None, None)

    assert slots(B=0) == 0
    assert slots(B=-1) == ARG and slots(out=None) == ARG and slots(out=p + 4) == ARG and slots(max_blocks=0) == ARG
    assert slots(B=65536) == LIMIT and slots(N=262145) == LIMIT and slots(num_blocks=1 << 27) == LIMIT
    assert slots(B=65) == WS
    assert L.tsd_kv_slots_workspace_bytes(64, 128) == 0 and L.tsd_kv_slots_workspace_bytes(64, 129) > 0
    assert L.tsd_kv_blocks_release(p, 65, p, 2, p, p, p, 4, None, 0, None, None) == WS
    assert L.tsd_kv_blocks_release(None, 1, p, 2, p, p, p, 4, None, 0, None, None) == ARG

    def write(T=3, ks=128, D=64, k=p, num_blocks=4):
        return L.tsd_kv_write_q4(k, ks, p, 128, p, T, num_blocks, 2, D, p, p, None, None)

    assert write(T=0) == 0 and write(T=-1) == ARG and write(D=80) == LIMIT and write(ks=120) == ARG
    assert write(ks=132) == ARG and write(k=p + 8) == ARG and write(k=None) == ARG and write(num_blocks=1 << 27) == LIMIT
    assert L.tsd_kv_read_q4(p, p, None, 1, 4, 2, 64, p, p, None, None) == ARG

    def commit(layers=1, stride=0, D=64, N=4, Dm=4):
        return L.tsd_kv_commit_path_q4(p, p, layers, stride, p, 2, 4, p, None, p, p, None, None, 1, N, 2, D, Dm, None,
                                       None, None, None)

    assert commit(layers=0) == 0 and commit() == ARG and commit(D=32) == LIMIT and commit(N=257) == LIMIT
    assert commit(Dm=33) == LIMIT

    def lp(R=1, rows=1, V=9, k=2, ids=p):
        return L.tsd_token_logprobs(p, 0, p, None, R, rows, V, k, p, p, ids, p, None, None)

    assert lp(R=0) == 0 and lp(R=2) == ARG and lp(V=0) == ARG and lp(k=33) == LIMIT and lp(k=10) == LIMIT
    assert lp(ids=None) == ARG and lp(k=-1) == ARG
    assert L.tsd_tree_path_logprobs(p, 0, p, p, p, p, None, 4096, 4, 9, 31, 0, p, p, p, None, None, None, None) == LIMIT
    assert L.tsd_tree_path_logprobs(p, 0, p, p, p, p, None, 1, 4, 9, 3, 0, None, p, p, None, None, None, None) == ARG
