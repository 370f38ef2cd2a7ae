"""Cases of one verify step over a 4-bit paged cache: block tables and slot maps,
the cache's writer and reader, tree attention over it, its commit, and the log
probabilities of the emitted tokens.

``own`` false: the operators in elementary torch operations; true: the library's
entry points.  Cache format: groups of 16 values along the head axis share a
scale byte b (the half with bits ``min(b, 0xE2) << 7``); a value is its scale
times an E2M1 code (nibble: sign, two exponent bits, one fraction bit).  A page
holds 16 slots of one head: 16 rows of D/2 code bytes (even column in the low
nibble), then 16 rows of D/16 scale bytes.
"""

import math

import numpy as np
import torch

own = False

PAGE = 16
GROUP = 16
MAX_SCALE = 0xE2  # 10240: six times it is still a finite half
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------


def listed():
    return [
        # one request's tree of 63 nodes behind a 4096-token prefix: what every
        # step of a single 8B-shaped request pays before its K/V are written
        dict(name="slots_step", op="slots", B=1, N=63, n_min=63, P_min=4096, P_max=4096),
        # 64 prompts of up to 8192 tokens enter the cache at once
        dict(name="slots_prompts", op="slots", B=64, N=8192, n_min=37, P_min=0, P_max=0),
        # the K/V of 16 ragged trees of up to 31 nodes, written each step
        dict(name="write_trees", op="write", T=496, Hkv=8, D=128, spare=64),
        # a prompt chunk of 32768 tokens
        dict(name="write_prompt", op="write", T=32768, Hkv=8, D=128, spare=512),
        # plain decoding of one request, one token: the latency end
        dict(name="attn_token", op="attn", B=1, N=1, n_min=1, Hq=32, Hkv=8, D=128, P_min=4096, P_max=4096),
        # plain decoding of 32 requests of very different lengths: bound by the cache's bytes
        dict(name="attn_token_ragged", op="attn", B=32, N=1, n_min=1, Hq=64, Hkv=8, D=128, P_min=512, P_max=16384),
        # 16 ragged trees (the ragged verify workload)
        dict(name="attn_tree_ragged", op="attn", B=16, N=31, n_min=16, Hq=32, Hkv=8, D=128, P_min=512, P_max=8192),
        # 127-node trees behind 32768 tokens (the long-context verify workload): bound by the tensor cores
        dict(name="attn_tree_long", op="attn", B=4, N=127, n_min=127, Hq=64, Hkv=8, D=128, P_min=32768, P_max=32768),
        # commit of 16 ragged trees in one layer
        dict(name="commit_trees", op="commit", layers=1, B=16, N=31, Hkv=8, D=128, D_max=5, P_min=64, P_max=512),
        # commit of four requests in 32 stacked layers
        dict(name="commit_layers", op="commit", layers=32, B=4, N=63, Hkv=8, D=128, D_max=6, P_min=512, P_max=512),
        # log probabilities along the accepted path of one 8B-shaped tree, five alternatives each
        dict(name="logprobs_path", op="path_logprobs", B=1, N=63, V=128256, D_max=6, k=5),
        # log probabilities of every node of four 127-node trees, twenty alternatives each
        dict(name="logprobs_rows", op="logprobs", R=508, V=128256, k=20, bf16=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["slots", "write", "attn", "attn", "attn", "commit", "path_logprobs", "logprobs"])
    if op == "slots":
        N = _log_int(rng, 1, 8192)
        P = _log_int(rng, 1, 8192)
        return dict(op=op, B=_log_int(rng, 1, 64), N=N, n_min=rng.randint(0, N), P_min=rng.randint(0, P), P_max=P)
    if op == "write":
        T = _log_int(rng, 1, 16384)
        return dict(op=op, T=T, Hkv=rng.choice([1, 2, 4, 5, 8]), D=rng.choice([64, 128]), spare=_log_int(rng, 1, 512))
    if op == "attn":
        Hkv, g, D = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8, 16]), rng.choice([64, 128, 128])
        N = rng.choice([1, _log_int(rng, 1, 256)])
        B = _log_int(rng, 1, 32)
        P = _log_int(rng, 1, 32768)
        while B * P > 131072 or B * P * N * g * Hkv * D > 4 * 32768 * 127 * 8 * 8 * 128:
            P = max(1, P // 2)
            B = max(1, B - 1)
        return dict(op=op, B=B, N=N, n_min=rng.randint(1, N), Hq=Hkv * g, Hkv=Hkv, D=D, P_min=rng.randint(0, P), P_max=P)
    if op == "commit":
        N = _log_int(rng, 2, 128)
        P = _log_int(rng, 1, 512)
        return dict(op=op, layers=_log_int(rng, 1, 32), B=_log_int(rng, 1, 4), N=N, Hkv=rng.choice([1, 4, 8]),
                    D=rng.choice([64, 128]), D_max=rng.randint(1, 12), P_min=rng.randint(0, P), P_max=P)
    V = _log_int(rng, 1000, 128256)
    if op == "path_logprobs":
        return dict(op=op, B=_log_int(rng, 1, 16), N=_log_int(rng, 2, 64), V=V, D_max=rng.randint(1, 8), k=rng.choice([0, 1, 5, 20, 32]))
    return dict(op=op, R=_log_int(rng, 1, 508), V=V, k=rng.choice([0, 1, 5, 20, 32]), bf16=rng.random() < 0.5)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _spread(lo, hi, n, rs):
    """n whole numbers from lo to hi, evenly spread, in random order (their sum does not depend on the seed)."""
    v = np.rint(np.linspace(lo, hi, n)).astype(np.int32) if n > 1 else np.asarray([hi], np.int32)
    return rs.permutation(v)


def _trees(rs, B, N, D_max):
    """Random trees in topological order: parents [B][N], depths, and ancestor rows (self included) [B][N][N]."""
    parent = np.full((B, N), -1, np.int32)
    depth = np.zeros((B, N), np.int32)
    anc = np.zeros((B, N, N), bool)
    rows = np.arange(B)
    anc[:, 0, 0] = True
    for i in range(1, N):
        p = (rs.random_sample(B) * i).astype(np.int32)
        p = np.where(depth[rows, p] < D_max, p, 0)
        parent[:, i] = p
        depth[:, i] = depth[rows, p] + 1
        anc[:, i] = anc[rows, p]
        anc[:, i, i] = True
    return parent, depth, anc


def _mask_words(anc):
    B, N, _ = anc.shape
    W = (N + 31) // 32
    bits = np.zeros((B, N, W * 32), np.uint64)
    bits[:, :, :N] = anc
    return (bits.reshape(B, N, W, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32).view(np.int32)


def _table(rs, lens, spare=0):
    need = (lens + PAGE - 1) // PAGE
    total = int(need.sum()) + spare
    ids = rs.permutation(total).astype(np.int32)
    table = np.zeros((len(lens), max(1, int(need.max()))), np.int32)
    pos = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[pos:pos + n]
        pos += n
    return table, max(1, total)


def _cache(gen, pages, Hkv, D):
    """A pool of quantised N(0, 1) values."""
    x = torch.randn((pages, Hkv, PAGE, D), generator=gen, device=gen.device, dtype=torch.float32).bfloat16().float()
    codes, scales = _quantise(x)
    return torch.cat([codes.reshape(pages, Hkv, -1), scales.reshape(pages, Hkv, -1)], -1)


def prepare(case, seed):
    dev = _device()
    rs = np.random.RandomState(seed % (1 << 32))
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def T(a):
        return torch.from_numpy(np.ascontiguousarray(a)).to(dev)

    op = case["op"]
    s = dict(case)
    if op == "slots":
        B, N = case["B"], case["N"]
        P = _spread(case["P_min"], case["P_max"], B, rs)
        n = _spread(case["n_min"], N, B, rs)
        held = (P + PAGE - 1) // PAGE
        most = int(((P + n + PAGE - 1) // PAGE).max())
        need = int(((P + n + PAGE - 1) // PAGE).sum())
        total = need + 32
        ids = rs.permutation(total).astype(np.int32)
        table = np.full((B, max(1, most)), -1, np.int32)
        pos = 0
        for b in range(B):
            table[b, :held[b]] = ids[pos:pos + held[b]]
            pos += held[b]
        free = np.zeros(total, np.int32)
        free[:total - pos] = ids[pos:]
        s.update(P=T(P), n=T(n), table=T(table), held=T(held.astype(np.int32)), free=T(free),
                 count=T(np.asarray([total - pos], np.int32)))
    elif op == "write":
        tokens, Hkv, D = case["T"], case["Hkv"], case["D"]
        pages = (tokens + case["spare"] + PAGE - 1) // PAGE
        k = torch.randn((tokens, Hkv, D), generator=gen, device=dev).bfloat16()
        v = torch.randn((tokens, Hkv, D), generator=gen, device=dev).bfloat16()
        s.update(k=k, v=v, slots=T(rs.permutation(pages * PAGE)[:tokens].astype(np.int32)),
                 every=torch.arange(pages * PAGE, dtype=torch.int32, device=dev),
                 kc=_cache(gen, pages, Hkv, D), vc=_cache(gen, pages, Hkv, D))
    elif op == "attn":
        B, N, Hq, Hkv, D = (case[x] for x in ("B", "N", "Hq", "Hkv", "D"))
        P = _spread(case["P_min"], case["P_max"], B, rs)
        n = _spread(case["n_min"], N, B, rs)
        _, _, anc = _trees(rs, B, N, 8)
        anc &= (np.arange(N)[None, :] < n[:, None])[:, :, None]
        table, pages = _table(rs, P + n)
        s.update(q=torch.randn((B, N, Hq, D), generator=gen, device=dev).bfloat16(), kc=_cache(gen, pages, Hkv, D),
                 vc=_cache(gen, pages, Hkv, D), table=T(table), P=T(P), n=T(n), mask=T(_mask_words(anc)),
                 err=T(np.zeros(B, np.int32)), max_slots=int((P + n).max()), scale=1.0 / math.sqrt(D))
    elif op == "commit":
        L, B, N, Hkv, D, Dm = (case[x] for x in ("layers", "B", "N", "Hkv", "D", "D_max"))
        P = _spread(case["P_min"], case["P_max"], B, rs)
        n = np.full(B, N, np.int32)
        parent, depth, _ = _trees(rs, B, N, Dm)
        table, pages = _table(rs, P + n, spare=2)
        A, path = _paths(rs, parent, depth, Dm)
        s.update(kc=_cache(gen, L * pages, Hkv, D).view(L, pages, Hkv, 9 * D), vc=_cache(gen, L * pages, Hkv, D).view(L, pages, Hkv, 9 * D),
                 table=T(table), P=T(P), n=T(n), A=T(A), path=T(path), err=T(np.zeros(B, np.int32)),
                 every=torch.arange(L * pages * PAGE, dtype=torch.int32, device=dev))
    elif op == "path_logprobs":
        B, N, V, Dm = case["B"], case["N"], case["V"], case["D_max"]
        parent, depth, _ = _trees(rs, B, N, Dm)
        A, path = _paths(rs, parent, depth, Dm)
        s.update(logits=torch.randn((B, N, V), generator=gen, device=dev) * math.sqrt(2.0), tokens=T(rs.randint(0, V, (B, N)).astype(np.int32)),
                 path=T(path), A=T(A), bonus=T(rs.randint(0, V, B).astype(np.int32)), err=T(np.zeros(B, np.int32)))
    else:
        R, V = case["R"], case["V"]
        x = torch.randn((R, V), generator=gen, device=dev) * math.sqrt(2.0)
        s.update(logits=x.bfloat16() if case["bf16"] else x, tokens=T(rs.randint(0, V, R).astype(np.int32)))
    return s


def _paths(rs, parent, depth, D_max):
    """An accepted path in each tree, to a node as deep as its tree goes: lengths, and safe node ids [B][D_max+1]."""
    B = len(parent)
    A = np.zeros(B, np.int32)
    path = np.zeros((B, D_max + 1), np.int32)
    for b in range(B):
        deep = np.flatnonzero(depth[b] == depth[b].max())
        i = int(deep[rs.randint(len(deep))])
        A[b] = depth[b, i]
        while i >= 0:
            path[b, depth[b, i]] = i + 1
            i = int(parent[b, i])
    return A, path


# ---------------------------------------------------------------------------
# the operators in their plain form
# ---------------------------------------------------------------------------


def _quantise(x):
    """fp32 [..., D] -> code bytes [..., D/2] and scale bytes [..., D/16]."""
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    mag = g.abs()
    r = (mag.amax(-1) / 6.0).clamp(max=10240.0)
    _, e = torch.frexp(r)
    quantum = torch.exp2((e - 1).clamp(min=-14).float() - 3.0)
    scale = torch.round(r / quantum) * quantum  # round half to even
    byte = scale.half().view(torch.int16) >> 7
    y = torch.where(scale[..., None] > 0, mag / scale[..., None], torch.zeros_like(mag))
    code = ((y > 0.25).to(torch.uint8) + (y >= 0.75).to(torch.uint8) + (y > 1.25).to(torch.uint8) + (y >= 1.75).to(torch.uint8)
            + (y > 2.5).to(torch.uint8) + (y >= 3.5).to(torch.uint8) + (y > 5.0).to(torch.uint8))
    code = code + torch.signbit(g).to(torch.uint8) * 8
    pair = code.reshape(*x.shape[:-1], -1, 2)
    return pair[..., 0] + pair[..., 1] * 16, byte.to(torch.uint8)


def _values(cache):
    """Cache bytes [..., Hkv, 9 D] -> fp32 [..., Hkv, 16, D]."""
    D = cache.shape[-1] // 9
    codes = cache[..., :8 * D].reshape(*cache.shape[:-1], PAGE, D // 2)
    scales = cache[..., 8 * D:].reshape(*cache.shape[:-1], PAGE, D // GROUP)
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=cache.device)
    both = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], D)
    scale = (scales.clamp(max=MAX_SCALE).to(torch.int16) << 7).view(torch.float16).float()
    return (table[both.int()].reshape(*scale.shape, GROUP) * scale[..., None]).reshape(both.shape)


def _rows(cache):
    """A pool's values by slot: fp32 [pages * 16, Hkv, D]."""
    v = _values(cache.reshape(-1, cache.shape[-2], cache.shape[-1]))
    return v.transpose(1, 2).reshape(-1, v.shape[1], v.shape[3])


def _plain_slots(s, trim):
    P, table, held, free, count = s["P"], s["table"], s["held"], s["free"], s["count"]
    n = s["n"]
    want = (P + (0 if trim else n) + PAGE - 1) // PAGE
    j = torch.arange(table.shape[1], device=table.device)[None, :]
    have = held[:, None].long()
    if trim:
        give = (held - want).clamp(min=0)
        first = give.cumsum(0) - give
        total = give.sum()
        back = (j >= want[:, None]) & (j < have)
        at = count.long() + total - 1 - (first[:, None] + j - want[:, None])
        free[at[back]] = table[back]
        table.masked_fill_(back, -1)
        count += total.int()
        held.copy_(torch.minimum(held, want))
        return None
    need = (want - held).clamp(min=0)
    start = need.cumsum(0) - need
    fits = start + need <= count
    take = (j >= held[:, None]) & (j < want[:, None]) & fits[:, None]
    at = (count.long() - 1 - (start[:, None] + j - held[:, None])).clamp(0, free.numel() - 1)
    table.copy_(torch.where(take, free[at], table))
    count -= (need * fits).sum().int()
    held.copy_(torch.where(fits, torch.maximum(held, want), held))
    i = torch.arange(s["N"], device=table.device)[None, :]
    pos = P[:, None] + i
    page = table.gather(1, (pos // PAGE).clamp(max=table.shape[1] - 1).long())
    return torch.where((i < n[:, None]) & fits[:, None], page * PAGE + pos % PAGE, -1).int()


def _plain_attention(s):
    q, table, P, n = s["q"].float(), s["table"], s["P"], s["n"]
    B, N, Hq, D = q.shape
    Hkv = s["kc"].shape[1]
    L = s["max_slots"]
    K = _values(s["kc"][table.long()].transpose(1, 2)).reshape(B, Hkv, -1, D)[:, :, :L]
    V = _values(s["vc"][table.long()].transpose(1, 2)).reshape(B, Hkv, -1, D)[:, :, :L]
    t = torch.arange(L, device=q.device)
    j = t[None, :] - P[:, None]  # the tree's node at each slot
    word = s["mask"].gather(2, (j.clamp(0, N - 1) // 32)[:, None, :].expand(B, N, L).long())
    sees = (word >> (j.clamp(0, N - 1) % 32)[:, None, :].int()) & 1
    inside = (j < n[:, None])[:, None, :]
    sees = ((j < 0)[:, None, :] | (sees != 0)) & inside & (torch.arange(N, device=q.device)[None, :] < n[:, None])[:, :, None]
    sees = sees[:, None, :, None, :]
    V = V.masked_fill(~inside[:, :, :, None], 0.0)
    rows = q.reshape(B, N, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    x = (rows @ K.transpose(2, 3) * s["scale"]).reshape(B, Hkv, N, -1, L).masked_fill(~sees, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m.clamp(min=-3e38)).masked_fill(~sees, 0.0)
    total = p.sum(-1, keepdim=True)
    out = (p.reshape(B, Hkv, -1, L) @ V).reshape(B, Hkv, N, -1, D) / total.clamp(min=1e-38)
    lse = (m + torch.log(total))[..., 0]
    return out.permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D).to(s["q"].dtype), lse.permute(0, 2, 1, 3).reshape(B, N, Hq)


def _plain_commit(s):
    table, P, A, path = s["table"], s["P"], s["A"], s["path"]
    k = torch.arange(path.shape[1], device=P.device)[None, :]
    src, dst = P[:, None] + path - 1, P[:, None] + k
    moved = (k <= A[:, None]) & (src != dst)
    b = torch.arange(len(P), device=P.device)[:, None].expand_as(moved)[moved]
    src, dst = src[moved].long(), dst[moved].long()
    D = s["D"]
    for c in (s["kc"], s["vc"]):
        codes = c[..., :8 * D].unflatten(-1, (PAGE, D // 2))
        scales = c[..., 8 * D:].unflatten(-1, (PAGE, D // GROUP))
        for part in (codes, scales):
            part[:, table[b, dst // PAGE].long(), :, dst % PAGE] = part[:, table[b, src // PAGE].long(), :, src % PAGE].clone()
    return P + A + 1, moved.sum(1).int()


def _ordered(x):
    """Integers that order as the floats do, both zeros alike."""
    i = (x + 0.0).view(torch.int32)
    return torch.where(i < 0, i ^ 0x7FFFFFFF, i).long()


def _plain_logprobs(x, token, k):
    x = x.float()
    V = x.shape[-1]
    m = x.amax(-1, keepdim=True)
    d = x - m
    e = torch.exp(d)
    total = e.sum(-1)
    log_total = torch.log(total)
    lp = d.gather(-1, token.long()[..., None])[..., 0] - log_total
    entropy = log_total - (e * d).sum(-1) / total
    key = (_ordered(x) << 32) + (V - 1 - torch.arange(V, device=x.device))
    best = torch.topk(key, k, dim=-1).values if k else key[..., :0]
    ids = V - 1 - (best & 0xFFFFFFFF)
    return lp, entropy, ids.int(), d.gather(-1, ids) - log_total[..., None]


def _plain(s):
    op = s["op"]
    if op == "slots":
        slots = _plain_slots(s, False)
        _plain_slots(s, True)
        return slots, s["table"], s["held"], s["free"], s["count"]
    if op == "write":
        page, row = s["slots"].long() // PAGE, s["slots"].long() % PAGE
        D = s["D"]
        for x, c in ((s["k"], s["kc"]), (s["v"], s["vc"])):
            codes, scales = _quantise(x.float())
            c[..., :8 * D].unflatten(-1, (PAGE, D // 2))[page, :, row] = codes
            c[..., 8 * D:].unflatten(-1, (PAGE, D // GROUP))[page, :, row] = scales
        return _rows(s["kc"]).bfloat16(), _rows(s["vc"]).bfloat16()
    if op == "attn":
        return _plain_attention(s)
    if op == "commit":
        length, moved = _plain_commit(s)
        return length, moved, _rows(s["kc"]).bfloat16(), _rows(s["vc"]).bfloat16()
    if op == "path_logprobs":
        path, A = s["path"].long(), s["A"]
        k = torch.arange(path.shape[1], device=path.device)[None, :]
        b = torch.arange(len(A), device=path.device)[:, None]
        here = (k <= A[:, None])
        node = (path - 1).clamp(min=0)
        ahead = torch.cat([node[:, 1:], node[:, :1]], 1)
        token = torch.where(k < A[:, None], s["tokens"][b, ahead], s["bonus"][:, None])
        lp, ent, ids, top = _plain_logprobs(s["logits"][b, node], token, s["k"])
        return (torch.where(here, token, -1), torch.where(here, lp, 0.0), torch.where(here, ent, 0.0),
                torch.where(here[..., None], ids, -1), torch.where(here[..., None], top, -math.inf))
    return _plain_logprobs(s["logits"], s["tokens"], s["k"])


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------


def run(s):
    if not own:
        return _plain(s)
    import tree_speculative_decoding_virtual_gb300 as tsd

    op = s["op"]
    if op == "slots":  # a step's two calls: room for its tokens, then what was not committed goes back
        slots = tsd.kv_slots_build(s["P"], s["n"], s["N"], s["table"], s["held"], s["free"], s["count"])
        tsd.kv_blocks_release(s["P"], s["table"], s["held"], s["free"], s["count"])
        return slots, s["table"], s["held"], s["free"], s["count"]
    if op == "write":
        tsd.kv_write_q4(s["k"], s["v"], s["slots"], s["kc"], s["vc"])
        return tsd.kv_read_q4(s["kc"], s["vc"], s["every"])
    if op == "attn":
        return tsd.tree_attn_fwd_q4(s["q"], s["kc"], s["vc"], s["table"], s["P"], s["n"], s["mask"], s["err"], s["max_slots"],
                                    scale=s["scale"])
    if op == "commit":
        length, moved = tsd.kv_commit_path_q4(s["kc"], s["vc"], s["table"], s["P"], s["n"], s["A"], s["path"], s["err"], s["N"], s["D_max"])
        k, v = tsd.kv_read_q4(s["kc"], s["vc"], s["every"])
        return length, moved, k, v
    if op == "path_logprobs":
        return tsd.tree_path_logprobs(s["logits"], s["tokens"], s["path"], s["A"], s["bonus"], s["err"], s["D_max"], k=s["k"])
    return tsd.token_logprobs(s["logits"], s["tokens"], k=s["k"])


def work(case):
    op = case["op"]
    if op == "slots":
        B, N = case["B"], case["N"]
        new = B * (case["n_min"] + N) / 2 if B > 1 else N
        taken = new / PAGE
        # lengths and held counts both ways, slots, and each new block read and written as it is taken and given back
        return {"bytes": 4.0 * (6 * B + B * N + 2 * new / PAGE + 6 * taken), "flops": 0}
    if op == "write":
        row = case["Hkv"] * case["D"]
        slots = (case["T"] + case["spare"] + PAGE - 1) // PAGE * PAGE
        # rows in (2 bytes) and out (9/16 byte); then the pool in and its values out
        return {"bytes": 2.0 * row * (case["T"] + slots) * (2 + 9 / 16) + 4.0 * (case["T"] + slots), "flops": 0}
    if op == "attn":
        B, N, Hq, Hkv, D = (case[x] for x in ("B", "N", "Hq", "Hkv", "D"))
        P = (case["P_min"] + case["P_max"]) / 2 if B > 1 else case["P_max"]
        n = (case["n_min"] + N) / 2 if B > 1 else N
        return {"bytes": B * ((P + n) * 2 * Hkv * D * 9 / 16 + 2.0 * N * Hq * D * 2 + 4.0 * N * Hq), "flops": 4.0 * B * n * Hq * D * (P + n)}
    if op == "commit":
        B, Hkv, D, L = (case[x] for x in ("B", "Hkv", "D", "layers"))
        P = (case["P_min"] + case["P_max"]) / 2 if B > 1 else case["P_max"]
        slots = (math.ceil((P + case["N"]) / PAGE) * B + 2) * PAGE * L
        moves = B * min(case["D_max"], case["N"] - 1) * L
        return {"bytes": 2.0 * Hkv * D * (slots * (2 + 9 / 16) + moves * 2 * 9 / 16), "flops": 0}
    if op == "path_logprobs":
        return {"bytes": 4.0 * case["B"] * (min(case["D_max"], case["N"] - 1) + 1) * (case["V"] + 2 + 2 * case["k"]), "flops": 0}
    return {"bytes": case["R"] * (case["V"] * (2.0 if case["bf16"] else 4.0) + 4.0 * (3 + 2 * case["k"])), "flops": 0}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------


def _scale_values():
    b = np.arange(MAX_SCALE + 1)
    e, f = b >> 3, b & 7
    return np.where(e == 0, f * 2.0 ** -17, (8 + f) * 2.0 ** (e - 18.0))


def _nearest_even(y, grid):
    """Index of the value of `grid` (ascending) nearest to y >= 0, ties to the even index, at most the last one."""
    mid = (grid[1:] + grid[:-1]) / 2
    below, above = torch.searchsorted(mid, y, right=False), torch.searchsorted(mid, y, right=True)
    return torch.where(below == above, below, below + (below & 1))


def _exact_stored(x):
    """What a row of values reads back as."""
    grid = torch.from_numpy(_scale_values()).to(x.device)
    e2m1 = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    g = x.double().reshape(*x.shape[:-1], -1, GROUP)
    scale = grid[_nearest_even((g.abs().amax(-1) / 6).contiguous(), grid)][..., None]
    code = _nearest_even((g.abs() / torch.where(scale > 0, scale, torch.ones_like(scale))).contiguous(), e2m1)
    return (torch.sign(g) * e2m1[code] * scale).reshape(x.shape)


def _exact_pool(cache):
    """fp64 [pages * 16, Hkv, D] of a pool [pages, Hkv, 9 D]."""
    D = cache.shape[-1] // 9
    pages, Hkv = cache.shape[:2]
    grid = torch.from_numpy(_scale_values()).to(cache.device)
    e2m1 = torch.tensor([(-1.0) ** (c >> 3) * E2M1[c & 7] for c in range(16)], dtype=torch.float64, device=cache.device)
    out = torch.empty((pages * PAGE, Hkv, D), dtype=torch.float64, device=cache.device)
    for r in range(PAGE):
        byte = cache[:, :, r * (D // 2):(r + 1) * (D // 2)].int()
        scale = grid[cache[:, :, 8 * D + r * (D // GROUP):8 * D + (r + 1) * (D // GROUP)].int().clamp(max=MAX_SCALE)]
        scale = scale.repeat_interleave(GROUP, -1)
        out[r::PAGE, :, 0::2] = e2m1[byte % 16] * scale[..., 0::2]
        out[r::PAGE, :, 1::2] = e2m1[byte // 16] * scale[..., 1::2]
    return out


def _exact_row_stats(x, token, k):
    x = x.double()
    lse = torch.logsumexp(x, -1)
    lp = x - lse[..., None]
    entropy = -(torch.exp(lp) * lp).sum(-1)
    top = torch.sort(lp, dim=-1, descending=True, stable=True)
    return lp.gather(-1, token.long()[..., None])[..., 0], entropy, top.values[..., :k]


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "slots":
        return None
    if op == "write":
        got = []
        for x, c in ((s["k"], s["kc"]), (s["v"], s["vc"])):
            pool = _exact_pool(c)
            pool[s["slots"].long()] = _exact_stored(x)
            got.append(pool)
        return tuple(got)
    if op == "commit":
        P, A, path, table = (s[x].cpu().numpy() for x in ("P", "A", "path", "table"))
        L, pages = s["kc"].shape[:2]
        got = []
        for c in (s["kc"], s["vc"]):
            pool = _exact_pool(c.reshape(L * pages, *c.shape[2:])).view(L, pages * PAGE, c.shape[2], -1)
            for b in range(len(P)):
                at = [int(table[b, t // PAGE]) * PAGE + int(t % PAGE) for t in P[b] + path[b, :A[b] + 1] - 1]
                to = [int(table[b, t // PAGE]) * PAGE + int(t % PAGE) for t in P[b] + np.arange(A[b] + 1)]
                pool[:, to] = pool[:, at].clone()
            got.append(pool.view(L * pages * PAGE, *pool.shape[2:]))
        return None, None, got[0], got[1]
    if op == "attn":
        q = s["q"].double()
        B, N, Hq, D = q.shape
        Hkv = s["kc"].shape[1]
        k, v = _exact_pool(s["kc"]), _exact_pool(s["vc"])
        out = torch.zeros((B, N, Hq, D), dtype=torch.float64, device=q.device)
        lse = torch.full((B, N, Hq), -math.inf, dtype=torch.float64, device=q.device)
        for b in range(B):
            P, n = int(s["P"][b]), int(s["n"][b])
            t = torch.arange(P + n, device=q.device)
            slot = s["table"][b].long()[t // PAGE] * PAGE + t % PAGE
            words = s["mask"][b, :n].cpu().numpy().view(np.uint32)
            bits = np.unpackbits(words.view(np.uint8), axis=-1, bitorder="little")[:, :n].astype(bool)
            sees = torch.cat([torch.ones((n, P), dtype=torch.bool, device=q.device), torch.from_numpy(bits).to(q.device)], 1)
            rows = q[b, :n].reshape(n, Hkv, Hq // Hkv, D)
            x = torch.einsum("ihgd,thd->hgit", rows, k[slot]) * s["scale"]
            x = x.masked_fill(~sees, -math.inf)
            z = torch.logsumexp(x, -1)
            out[b, :n] = torch.einsum("hgit,thd->ihgd", torch.exp(x - z[..., None]), v[slot]).reshape(n, Hq, D)
            lse[b, :n] = z.permute(2, 0, 1).reshape(n, Hq)
        return out, lse
    if op == "path_logprobs":
        B, Dm, k = case["B"], case["D_max"], case["k"]
        f64 = dict(dtype=torch.float64, device=s["logits"].device)
        lp, ent, top = torch.zeros((B, Dm + 1), **f64), torch.zeros((B, Dm + 1), **f64), torch.full((B, Dm + 1, k), -math.inf, **f64)
        for b in range(B):
            a = int(s["A"][b])
            node = s["path"][b, :a + 1].long() - 1
            token = torch.cat([s["tokens"][b, node[1:]], s["bonus"][b:b + 1]])
            lp[b, :a + 1], ent[b, :a + 1], top[b, :a + 1] = _exact_row_stats(s["logits"][b, node], token, k)
        return None, lp, ent, None, top
    lp, ent, top = _exact_row_stats(s["logits"], s["tokens"], case["k"])
    return lp, ent, None, top
