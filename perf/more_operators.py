"""Cases of a verify step of requests that share a prompt: per-head norms, rotation and the
append of K and V to the paged cache, tree attention with the shared prefix computed once,
and sampling with temperature, top-k, top-p and min-p (tokens from given random numbers, and
the filtered distribution that stochastic verification takes).

``own`` false: the operators in elementary torch operations; true: the library's entry points.
"""

import math

import numpy as np
import torch

own = False

PAGE = 16
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
THETA = 500000.0
EPS = 1e-6


def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------


def listed():
    return [
        # one request, one token: the latency end of the append
        dict(name="append_token", op="append", B=1, N=1, n_min=1, Hq=32, Hkv=8, D=128, R=128, axes=1, norm=False, pairs=False, q4=False, P_max=4096, spare=64),
        # 16 ragged trees of up to 31 nodes into a 4-bit cache: one layer of every verify step
        dict(name="append_trees_q4", op="append", B=16, N=31, n_min=16, Hq=32, Hkv=8, D=128, R=128, axes=1, norm=True, pairs=False, q4=True, P_max=8192, spare=64),
        # a prompt of 32768 tokens of text and pictures: positions of three axes, norms of queries and keys
        dict(name="append_prompt", op="append", B=1, N=32768, n_min=32768, Hq=64, Hkv=8, D=128, R=128, axes=3, norm=True, pairs=False, q4=False, P_max=0, spare=512),
        # one token for each of 4 requests behind a prompt of 2048 tokens: the latency end of the attention
        dict(name="shared_few", op="attn", B=4, N=1, n_min=1, G=1, Hq=32, Hkv=8, D=128, S_min=2048, S_max=2048, own_min=16, own_max=256),
        # plain decoding of 64 requests behind one system prompt: the cache's bytes, once for all
        dict(name="shared_tokens", op="attn", B=64, N=1, n_min=1, G=1, Hq=64, Hkv=8, D=128, S_min=16384, S_max=16384, own_min=64, own_max=1024),
        # several continuations of each of 4 prompts of different lengths, verified as ragged trees
        dict(name="shared_trees", op="attn", B=16, N=31, n_min=16, G=4, Hq=32, Hkv=8, D=128, S_min=512, S_max=8192, own_min=64, own_max=512),
        # 127-node trees of 8 requests over one document of 32768 tokens: bound by the tensor cores
        dict(name="shared_long", op="attn", B=8, N=127, n_min=127, G=1, Hq=64, Hkv=8, D=128, S_min=32768, S_max=32768, own_min=500, own_max=500),
        # the next token of one request
        dict(name="sample_token", op="sample", B=1, N=1, draws=1, V=128256, bf16=False, top_k=50, top_p=0.95, min_p=0.0),
        # the next tokens of 64 requests, each with settings of its own
        dict(name="sample_batch", op="sample", B=64, N=1, draws=1, V=128256, bf16=True, top_k=-1, top_p=-1.0, min_p=-1.0),
        # a drafter draws four children for every node of four 127-node trees
        dict(name="sample_nodes", op="sample", B=4, N=127, draws=4, V=128256, bf16=False, top_k=0, top_p=0.9, min_p=0.0),
        # one 63-node tree's logits before stochastic verification
        dict(name="filter_tree", op="filter", B=1, N=63, V=128256, bf16=False, probs=False, top_k=50, top_p=0.95, min_p=0.0),
        # the draft probabilities of four 127-node trees
        dict(name="filter_nodes", op="filter", B=4, N=127, V=128256, bf16=False, probs=True, top_k=0, top_p=0.9, min_p=0.01),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "sample", "filter"])
    if op == "append":
        Hkv = rng.choice([1, 2, 4, 5, 8])
        D = rng.choice([64, 128])
        q4 = rng.random() < 0.3
        tokens = _log_int(rng, 1, 1024 if q4 else 24576)
        B = min(tokens, _log_int(rng, 1, 64))
        N = max(1, tokens // B)
        return dict(op=op, B=B, N=N, n_min=rng.randint(1, N), Hq=Hkv * rng.choice([1, 2, 4, 7, 8]), Hkv=Hkv, D=D, R=rng.choice([D, D, D // 2]),
                    axes=rng.choice([1, 1, 2, 3]), norm=rng.random() < 0.5, pairs=rng.random() < 0.3, q4=q4, P_max=_log_int(rng, 1, 200000),
                    spare=_log_int(rng, 1, 512))
    if op == "attn":
        Hkv, g, D = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8, 16]), rng.choice([64, 128, 128])
        N = rng.choice([1, _log_int(rng, 1, 256)])
        B = _log_int(rng, 1, 128)
        S, extra = _log_int(rng, 1, 32768), _log_int(rng, 1, 2048)
        while B * (S + extra) * N * g * Hkv * D > 8 * 33000 * 127 * 64 * 128 or B * (S + extra) * Hkv * D > 64 * 17000 * 8 * 128:
            S = max(1, S // 2)
            B = max(1, B - 1)
        return dict(op=op, B=B, N=N, n_min=rng.randint(1, N), G=rng.randint(1, min(B, 5)), Hq=Hkv * g, Hkv=Hkv, D=D, S_min=rng.randint(0, S), S_max=S,
                    own_min=rng.randint(0, extra), own_max=extra)
    N = _log_int(rng, 1, 128)
    s = dict(op=op, B=_log_int(rng, 1, max(1, 508 // N)), N=N, V=_log_int(rng, 1000, 128256), bf16=rng.random() < 0.5,
             top_k=rng.choice([0, 0, 1, _log_int(rng, 1, 2000), -1]), top_p=rng.choice([1.0, rng.uniform(0.05, 0.999), -1.0]),
             min_p=rng.choice([0.0, 0.0, rng.uniform(0.001, 0.3), -1.0]))
    return dict(s, draws=rng.choice([1, 1, 2, 8])) if op == "sample" else dict(s, probs=rng.random() < 0.5)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _spread(lo, hi, n, rs):
    """n whole numbers from lo to hi, evenly spread, in random order (their sum does not depend on the seed)."""
    v = np.rint(np.linspace(lo, hi, n)).astype(np.int32) if n > 1 else np.asarray([hi], np.int32)
    return rs.permutation(v)


def _trees(rs, B, N, D_max):
    """Random trees in topological order: depths [B][N], and ancestor rows (self included) [B][N][N]."""
    depth = np.zeros((B, N), np.int32)
    anc = np.zeros((B, N, N), bool)
    rows = np.arange(B)
    anc[:, 0, 0] = True
    for i in range(1, N):
        p = (rs.random_sample(B) * i).astype(np.int32)
        p = np.where(depth[rows, p] < D_max, p, 0)
        depth[:, i] = depth[rows, p] + 1
        anc[:, i] = anc[rows, p]
        anc[:, i, i] = True
    return depth, anc


def _mask_words(anc):
    B, N, _ = anc.shape
    W = (N + 31) // 32
    bits = np.zeros((B, N, W * 32), np.uint64)
    bits[:, :, :N] = anc
    return (bits.reshape(B, N, W, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32).view(np.int32)


def _settings(rs, case):
    """Per request: temperature, top-k, top-p and min-p (-1 in a case: they differ from request to request)."""
    B = case["B"]
    t = rs.choice([0.6, 0.8, 1.0, 1.0, 1.3], B)
    k = rs.choice([0, 1, 20, 50, 1000], B) if case["top_k"] < 0 else np.full(B, case["top_k"])
    p = rs.choice([0.5, 0.8, 0.9, 0.95, 0.99, 1.0], B) if case["top_p"] < 0 else np.full(B, case["top_p"])
    m = rs.choice([0.0, 0.0, 0.02, 0.1], B) if case["min_p"] < 0 else np.full(B, case["min_p"])
    if case["top_k"] < 0:
        t[rs.randint(0, B)] = 0.0  # one of them wants the most probable token
    return t.astype(np.float32), k.astype(np.int32), p.astype(np.float32), m.astype(np.float32)


def prepare(case, seed):
    dev = _device()
    rs = np.random.RandomState(seed % (1 << 32))
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def T(a):
        return torch.from_numpy(np.ascontiguousarray(a)).to(dev)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    op = case["op"]
    s = dict(case)
    if op == "append":
        B, N, Hq, Hkv, D, R = (case[x] for x in ("B", "N", "Hq", "Hkv", "D", "R"))
        n = _spread(case["n_min"], N, B, rs)
        pages = (B * N + case["spare"] + PAGE - 1) // PAGE
        slots = rs.permutation(pages * PAGE)[:B * N].astype(np.int32).reshape(B, N)
        slots[np.arange(N)[None, :] >= n[:, None]] = -1
        qkv = normal(B, N, Hq + 2 * Hkv, D).bfloat16()  # rows of a fused projection
        if case["axes"] == 1:
            pos = _trees(rs, B, N, 8)[0] if N <= 256 else np.tile(np.arange(N, dtype=np.int32), (B, 1))
        else:  # time, height, width of patches of pictures, in reading order
            i = np.tile(np.arange(N, dtype=np.int32), (B, 1))
            pos = np.stack([i // 256 * 16, i // 256 * 16 + i // 16 % 16, i // 256 * 16 + i % 16][:case["axes"]])
        s.update(q=qkv[:, :, :Hq], k=qkv[:, :, Hq:Hq + Hkv], v=qkv[:, :, Hq + Hkv:], slots=T(slots), pos=T(pos.astype(np.int32)),
                 base=T(_spread(0, case["P_max"], B, rs)), inv_freq=T((THETA ** (-np.arange(R // 2) * 2.0 / R)).astype(np.float32)),
                 axis=T((np.arange(R // 2) * case["axes"] // (R // 2)).astype(np.int32)) if case["axes"] > 1 else None,
                 qw=(1 + 0.2 * normal(D)).bfloat16() if case["norm"] else None, kw=(1 + 0.2 * normal(D)).bfloat16() if case["norm"] else None,
                 every=torch.arange(pages * PAGE, dtype=torch.int32, device=dev))
        if case["q4"]:  # any bytes will do as codes; scales between 2^-4 and 2^2
            pool = torch.randint(0, 256, (2, pages, Hkv, 9 * D), generator=gen, device=dev, dtype=torch.uint8)
            pool[..., 8 * D:] = pool[..., 8 * D:] % 48 + 88
            s.update(kc=pool[0], vc=pool[1])
        else:
            s.update(kc=normal(pages, Hkv, PAGE, D).bfloat16(), vc=normal(pages, Hkv, PAGE, D).bfloat16())
    elif op == "attn":
        B, N, G, Hq, Hkv, D = (case[x] for x in ("B", "N", "G", "Hq", "Hkv", "D"))
        S = _spread(case["S_min"], case["S_max"], G, rs)
        first = np.concatenate([[0], np.sort(rs.permutation(B - 1)[:G - 1]) + 1, [B]]).astype(np.int32)
        group = np.repeat(np.arange(G), np.diff(first))
        n = _spread(case["n_min"], N, B, rs)
        P = (S[group] + _spread(case["own_min"], case["own_max"], B, rs)).astype(np.int32)
        _, anc = _trees(rs, B, N, 8)
        anc &= (np.arange(N)[None, :] < n[:, None])[:, :, None]
        # whole blocks of the shared prefix are the same blocks; its last, partly filled one is each request's own copy
        whole = S // PAGE
        need = (P + n + PAGE - 1) // PAGE - whole[group]
        ids = rs.permutation(int(whole.sum() + need.sum())).astype(np.int32)
        table = np.zeros((B, int(((P + n + PAGE - 1) // PAGE).max())), np.int32)
        at = int(whole.sum())
        start = np.concatenate([[0], np.cumsum(whole)])
        for b in range(B):
            g = group[b]
            table[b, :whole[g]] = ids[start[g]:start[g + 1]]
            table[b, whole[g]:whole[g] + need[b]] = ids[at:at + need[b]]
            at += need[b]
        kc, vc = normal(len(ids), Hkv, PAGE, D).bfloat16(), normal(len(ids), Hkv, PAGE, D).bfloat16()
        for g in np.flatnonzero(S % PAGE):
            r, one, others = S[g] % PAGE, table[first[g], whole[g]], table[first[g]:first[g + 1], whole[g]].astype(np.int64)
            for c in (kc, vc):
                c[T(others), :, :r] = c[int(one), :, :r].clone()
        s.update(q=normal(B, N, Hq, D).bfloat16(), kc=kc, vc=vc, table=T(table), P=T(P), n=T(n), mask=T(_mask_words(anc)), err=T(np.zeros(B, np.int32)),
                 first=T(first), S=T(S.astype(np.int32)), scale=1.0 / math.sqrt(D), slots=int((P + n).max()))
    else:
        B, N, V = case["B"], case["N"], case["V"]
        # most of a vocabulary is noise; some hundred tokens stand out, a few of them far
        x = 2.0 * normal(B, N, V)
        few = min(V, 256)
        up = (torch.randint(0, V, (B, N, 1), generator=gen, device=dev) + torch.arange(few, device=dev) * (V // few)) % V
        x.scatter_(2, up, 3.0 * torch.empty(up.shape, device=dev).exponential_(generator=gen) + 2.0 * normal(*up.shape))
        t, k, p, m = _settings(rs, case)
        s.update(logits=x.bfloat16() if case["bf16"] else x, t=T(t), k=T(k), p=T(p), m=T(m))
        if op == "sample":
            s.update(u=torch.rand((B, N, case["draws"]), generator=gen, device=dev))
    return s


# ---------------------------------------------------------------------------
# the operators in their plain form
# ---------------------------------------------------------------------------


def _turned(x, weight, cos, sin, s):
    """Rows [B, N, H, D] normed and rotated, in fp32; cos and sin [B, N, R/2]."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    R = s["R"]
    head, rest = x[..., :R], x[..., R:]
    a, b = (head[..., 0::2], head[..., 1::2]) if s["pairs"] else (head[..., :R // 2], head[..., R // 2:])
    c, d = cos[:, :, None], sin[:, :, None]
    a, b = a * c - b * d, b * c + a * d
    head = torch.stack([a, b], -1).flatten(-2) if s["pairs"] else torch.cat([a, b], -1)
    return torch.cat([head, rest], -1)


def _quantise(x):
    """bf16 values as fp32 [..., D] -> code bytes [..., D/2] and scale bytes [..., D/16] of the 4-bit cache."""
    g = x.reshape(*x.shape[:-1], -1, 16)
    mag = g.abs()
    r = (mag.amax(-1) / 6.0).clamp(max=10240.0)
    quantum = torch.exp2((torch.frexp(r)[1] - 1).clamp(min=-14).float() - 3.0)
    scale = torch.round(r / quantum) * quantum
    y = torch.where(scale[..., None] > 0, mag / scale[..., None], torch.zeros_like(mag))
    code = ((y > 0.25).to(torch.uint8) + (y >= 0.75).to(torch.uint8) + (y > 1.25).to(torch.uint8) + (y >= 1.75).to(torch.uint8)
            + (y > 2.5).to(torch.uint8) + (y >= 3.5).to(torch.uint8) + (y > 5.0).to(torch.uint8)) + torch.signbit(g).to(torch.uint8) * 8
    pair = code.reshape(*x.shape[:-1], -1, 2)
    return pair[..., 0] + pair[..., 1] * 16, (scale.half().view(torch.int16) >> 7).to(torch.uint8)


def _stored(cache):
    """A 4-bit pool's values by slot: bf16 [pages * 16, Hkv, D]."""
    pages, Hkv, D = cache.shape[0], cache.shape[1], cache.shape[2] // 9
    codes = cache[..., :8 * D].reshape(pages, Hkv, PAGE, D // 2)
    scales = (cache[..., 8 * D:].reshape(pages, Hkv, PAGE, D // 16).to(torch.int16) << 7).view(torch.float16).float()
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=cache.device)
    both = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    v = table[both.int()] * scales.repeat_interleave(16, -1)
    return v.transpose(1, 2).reshape(-1, Hkv, D).bfloat16()


def _plain_append(s):
    B, N = s["B"], s["N"]
    pos = s["pos"][None] if s["axis"] is None else s["pos"]
    pos = pos + s["base"][None, :, None]
    axis = torch.zeros(s["R"] // 2, dtype=torch.long, device=pos.device) if s["axis"] is None else s["axis"].long()
    angle = pos.double().permute(1, 2, 0)[..., axis] * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    q = _turned(s["q"], s["qw"], cos, sin, s).bfloat16()
    k = _turned(s["k"], s["kw"], cos, sin, s).bfloat16()
    here = s["slots"] >= 0
    page, row = s["slots"][here].long() // PAGE, s["slots"][here].long() % PAGE
    if not s["q4"]:
        s["kc"][page, :, row] = k[here]
        s["vc"][page, :, row] = s["v"][here]
        return q, s["kc"], s["vc"]
    D = s["D"]
    for x, c in ((k[here], s["kc"]), (s["v"][here], s["vc"])):
        codes, scales = _quantise(x.float())
        c[..., :8 * D].unflatten(-1, (PAGE, D // 2))[page, :, row] = codes
        c[..., 8 * D:].unflatten(-1, (PAGE, D // 16))[page, :, row] = scales
    return q, _stored(s["kc"]), _stored(s["vc"])


def _plain_attention(s):
    q, table, P, n = s["q"].float(), s["table"], s["P"], s["n"]
    B, N, Hq, D = q.shape
    Hkv, L = s["kc"].shape[1], s["slots"]
    K = s["kc"][table.long()].transpose(1, 2).reshape(B, Hkv, -1, D)[:, :, :L].float()
    V = s["vc"][table.long()].transpose(1, 2).reshape(B, Hkv, -1, D)[:, :, :L].float()
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


def _plain_kept(s):
    """Scaled logits d = (x - max x) / T [R, V] (fp32), weights e^d (fp32 values in 64 bits), and what the filters keep."""
    x = s["logits"].float().flatten(0, 1)
    N, V = s["N"], x.shape[1]
    t, k, p, m = (s[a].repeat_interleave(N)[:, None] for a in ("t", "k", "p", "m"))
    d = (x - x.amax(-1, keepdim=True)) * torch.where(t > 0, 1.0 / t.clamp(min=1e-30), torch.ones_like(t))
    w = torch.exp(d)
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices  # ties to the lowest index
    rank = torch.arange(V, device=x.device)[None, :]
    keep = (rank < torch.where(k > 0, k, V)) & ((t > 0) | (rank == 0))
    sorted_w = w.gather(-1, order).double() * keep  # (sums of 128256 weights, compared with each other: 64 bits)
    total = sorted_w.sum(-1, keepdim=True)
    before = sorted_w.cumsum(-1) - sorted_w
    keep &= (before < p.double() * total) | (p >= 1) | (rank == 0)
    kept = torch.zeros_like(keep).scatter_(-1, order, keep) & (w >= m)
    return d, w.double() * kept, kept


def _plain(s):
    op = s["op"]
    if op == "append":
        return _plain_append(s)
    if op == "attn":
        return _plain_attention(s)
    d, w, kept = _plain_kept(s)
    B, N = s["B"], s["N"]
    if op == "filter":
        out = w / w.sum(-1, keepdim=True) if s["probs"] else d.masked_fill(~kept, -math.inf)
        return out.float().view(B, N, -1)
    cum = w.cumsum(-1)
    total = cum[:, -1:].contiguous()
    at = torch.searchsorted(cum, s["u"].flatten(0, 1).double() * total, right=True)
    at = torch.minimum(at, torch.searchsorted(cum, total))  # (rounding left none: the last of any weight)
    logprob = d.gather(-1, at).double() - torch.log(total)
    return at.int().view(B, N, -1), logprob.float().view(B, N, -1)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------


def run(s):
    if not own:
        return _plain(s)
    import tree_speculative_decoding_virtual_gb300 as tsd

    op = s["op"]
    if op == "append":
        append = tsd.kv_append_rope_q4 if s["q4"] else tsd.kv_append_rope
        q = append(s["q"], s["k"], s["v"], s["slots"], s["kc"], s["vc"], s["inv_freq"], s["pos"], base=s["base"], freq_axis=s["axis"],
                   q_weight=s["qw"], k_weight=s["kw"], eps=EPS, interleaved=s["pairs"])
        if not s["q4"]:
            return q, s["kc"], s["vc"]
        return (q,) + tuple(tsd.kv_read_q4(s["kc"], s["vc"], s["every"]))
    if op == "attn":
        return tsd.tree_attn_fwd_shared(s["q"], s["kc"], s["vc"], s["table"], s["P"], s["n"], s["mask"], s["err"], s["first"], s["S"], scale=s["scale"])
    if op == "sample":
        return tsd.token_sample(s["logits"], s["u"], temperature=s["t"], top_k=s["k"], top_p=s["p"], min_p=s["m"])
    return tsd.logits_filter(s["logits"], temperature=s["t"], top_k=s["k"], top_p=s["p"], min_p=s["m"], probs=s["probs"])


def work(case):
    op = case["op"]
    if op == "append":
        B, N, Hq, Hkv, D = (case[x] for x in ("B", "N", "Hq", "Hkv", "D"))
        n = (case["n_min"] + N) / 2 if B > 1 else N
        slots = (B * N + case["spare"] + PAGE - 1) // PAGE * PAGE
        b = 2.0 * 2 * B * N * Hq * D + 2 * 2.0 * B * n * Hkv * D + 4.0 * B * N * (1 + case["axes"])
        b += 2 * (B * n * Hkv * D * 9 / 16 + slots * Hkv * D * (9 / 16 + 2)) if case["q4"] else 2 * 2.0 * B * n * Hkv * D
        return {"bytes": b, "flops": 0}
    if op == "attn":
        B, N, G, Hq, Hkv, D = (case[x] for x in ("B", "N", "G", "Hq", "Hkv", "D"))
        S = (case["S_min"] + case["S_max"]) / 2 if G > 1 else case["S_max"]
        extra = (case["own_min"] + case["own_max"]) / 2 if B > 1 else case["own_max"]
        n = (case["n_min"] + N) / 2 if B > 1 else N
        keys = G * S + B * (extra + n)
        return {"bytes": keys * 2 * Hkv * D * 2 + B * N * Hq * (2.0 * D * 2 + 4.0), "flops": 4.0 * B * n * Hq * D * (S + extra + n)}
    R, V = case["B"] * case["N"], case["V"]
    read = R * V * (2.0 if case["bf16"] else 4.0)
    return {"bytes": read + (12.0 * R * case["draws"] if op == "sample" else 4.0 * R * V), "flops": 0}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------


def _nearest_even(y, grid):
    """Index of the value of `grid` (ascending) nearest to y >= 0, ties to the even index, at most the last one."""
    mid = (grid[1:] + grid[:-1]) / 2
    below, above = torch.searchsorted(mid, y, right=False), torch.searchsorted(mid, y, right=True)
    return torch.where(below == above, below, below + (below & 1))


def _scales(device):
    b = np.arange(0xE3)
    return torch.from_numpy(np.where(b >> 3 == 0, (b & 7) * 2.0 ** -17, (8 + (b & 7)) * 2.0 ** ((b >> 3) - 18.0))).to(device)


def _exact_append(s):
    B, N, R, D = s["B"], s["N"], s["R"], s["D"]
    f64 = dict(dtype=torch.float64, device=s["q"].device)
    inv, where = s["inv_freq"].double(), (s["axis"] if s["axis"] is not None else torch.zeros(R // 2, device=s["q"].device)).long()
    pos = s["pos"].view(-1, B, N)

    def rotated(x, weight):
        y = x.double()
        if weight is not None:
            y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / D + EPS) * weight.double()
        out = y.clone()
        for f in range(R // 2):
            angle = (pos[where[f]] + s["base"][:, None]).double() * inv[f]
            i, j = (2 * f, 2 * f + 1) if s["pairs"] else (f, f + R // 2)
            z = torch.complex(y[..., i], y[..., j]) * torch.polar(torch.ones_like(angle), angle)[..., None]
            out[..., i], out[..., j] = z.real, z.imag
        return out

    q, k, v = rotated(s["q"], s["qw"]), rotated(s["k"], s["kw"]), s["v"].double()
    pools = []
    for x, c in ((k, s["kc"]), (v, s["vc"])):
        if s["q4"]:
            grid, e2m1 = _scales(c.device), torch.tensor(E2M1, **f64)
            both = torch.stack([c[..., :8 * D] & 15, c[..., :8 * D] >> 4], -1).flatten(-2).int()
            sign = 1.0 - 2.0 * (both >> 3)
            pool = (sign * e2m1[both & 7]).view(*c.shape[:2], PAGE, D // 16, 16) * grid[c[..., 8 * D:].int()].view(*c.shape[:2], PAGE, D // 16, 1)
            pool = pool.reshape(*c.shape[:2], PAGE, D).transpose(1, 2).reshape(-1, c.shape[1], D)
            g = x.bfloat16().double().reshape(*x.shape[:-1], -1, 16)  # (the cache's writer takes bf16)
            scale = grid[_nearest_even((g.abs().amax(-1) / 6).contiguous(), grid)][..., None]
            code = _nearest_even((g.abs() / torch.where(scale > 0, scale, torch.ones_like(scale))).contiguous(), e2m1)
            x = (torch.sign(g) * e2m1[code] * scale).reshape(x.shape)
        else:
            pool = c.double().transpose(1, 2).reshape(-1, c.shape[1], D).clone()
        here = s["slots"] >= 0
        pool[s["slots"][here].long()] = x[here]
        pools.append(pool if s["q4"] else pool.view(c.shape[0], PAGE, c.shape[1], D).transpose(1, 2))
    return q, pools[0], pools[1]


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "append":
        return _exact_append(s)
    if op == "attn":
        q = s["q"].double()
        B, N, Hq, D = q.shape
        Hkv = s["kc"].shape[1]
        out = torch.zeros((B, N, Hq, D), dtype=torch.float64, device=q.device)
        lse = torch.full((B, N, Hq), -math.inf, dtype=torch.float64, device=q.device)
        for b in range(B):
            P, n = int(s["P"][b]), int(s["n"][b])
            t = torch.arange(P + n, device=q.device)
            page = s["table"][b].long()[t // PAGE]
            words = s["mask"][b, :n].cpu().numpy().view(np.uint32)
            bits = np.unpackbits(words.view(np.uint8), axis=-1, bitorder="little")[:, :n].astype(bool)
            sees = torch.cat([torch.ones((n, P), dtype=torch.bool, device=q.device), torch.from_numpy(bits).to(q.device)], 1)
            for h in range(Hkv):
                k, v = s["kc"][page, h, t % PAGE].double(), s["vc"][page, h, t % PAGE].double()
                g = Hq // Hkv
                x = (q[b, :n, h * g:(h + 1) * g] @ k.T * s["scale"]).masked_fill(~sees[:, None], -math.inf)
                z = torch.logsumexp(x, -1)
                out[b, :n, h * g:(h + 1) * g] = torch.exp(x - z[..., None]) @ v
                lse[b, :n, h * g:(h + 1) * g] = z
        return out, lse
    B, N, V = case["B"], case["N"], case["V"]
    answers = []
    for b in range(B):
        t, k, p, m = (float(s[a][b]) for a in ("t", "k", "p", "m"))
        for i in range(N):
            x = s["logits"][b, i].double()
            d = (x - x.max()) / (t if t > 0 else 1.0)
            best, ids = torch.sort(d, descending=True, stable=True)
            some = 1 if t <= 0 else int(k) if k > 0 else V
            w = torch.exp(best[:some])
            if p < 1:
                w = w[:max(1, int(torch.searchsorted(w.cumsum(0) - w, p * w.sum())))]
            w = w[:max(1, int((w >= m).sum()))]
            ids, best = ids[:len(w)], best[:len(w)]
            if op == "sample":
                ids, up = torch.sort(ids)
                cum = w[up].cumsum(0)
                at = torch.searchsorted(cum, s["u"][b, i].double() * cum[-1], right=True).clamp(max=len(w) - 1)
                answers.append(d[ids[at]] - torch.log(w.sum()))
            else:
                row = torch.full((V,), 0.0 if case["probs"] else -math.inf, dtype=torch.float64, device=x.device)
                row[ids] = w / w.sum() if case["probs"] else best
                answers.append(row)
    got = torch.stack(answers).view(B, N, -1)
    return (None, got) if op == "sample" else got
