"""Speculative decoding and token eviction over the paged cache: the cases
these operators are measured on, their plain forms and their exact results.

Four operators over the cache [num_blocks, num_kv_heads, 16, head_size]:

- ``tree``: attention of a tree of drafted tokens over the cached context
  (pa_tree_attention);
- ``commit``: moving the K/V of the accepted path of that tree to the
  positions right after the context (pa_tree_commit);
- ``scored``: decode attention that adds every cached token's attention
  weight to an accumulator (pa_decode_scored);
- ``evict``: keeping the tokens of largest accumulated weight, with the
  first and the newest ones protected, and compacting K/V into fresh blocks
  (pa_evict).

``own`` selects the library's calls; otherwise ``run`` computes the plain
form with elementary torch operations in 32 bits.
"""

import math
import random

import numpy as np
import torch

own = False

BS = 16  # tokens per cache block

_DT = {"bf16": torch.bfloat16, "f32": torch.float32, "fp8": torch.float8_e4m3fn}
_ESIZE = {"bf16": 2, "f32": 4, "fp8": 1}


def listed():
    return [
        # one user's chat turn, 8 drafted tokens: the smallest call, where latency counts
        dict(name="tree-one-user", op="tree", dtype="bf16", B=1, H=32, Hkv=8, D=128, n=8, median=500, lo=500, hi=500,
             ragged=False, lens_seed=1),
        # the multi-head serving batch with a 16-token tree per sequence
        dict(name="tree-mha-batch", op="tree", dtype="bf16", B=64, H=32, Hkv=32, D=128, n=16, median=512, lo=16,
             hi=2048, ragged=True, lens_seed=2),
        # the grouped-query serving batch, trees of up to 32 tokens, some sequences without a draft
        dict(name="tree-gqa-batch", op="tree", dtype="bf16", B=256, H=32, Hkv=8, D=128, n=32, median=1024, lo=32,
             hi=8192, ragged=True, lens_seed=3),
        # few long documents with wide trees (64 tokens x 4 heads a group): near the ridge of bandwidth and tensor rate
        dict(name="tree-long-context", op="tree", dtype="bf16", B=8, H=32, Hkv=8, D=128, n=64, median=80 * 1024,
             lo=32 * 1024, hi=128 * 1024, ragged=False, lens_seed=4),
        # the accepted path of one small fp8 cache, and of the whole grouped-query batch
        dict(name="commit-one-user", op="commit", dtype="fp8", B=1, H=32, Hkv=8, D=128, n=8, median=500, lo=500,
             hi=500, ragged=False, lens_seed=5),
        dict(name="commit-batch", op="commit", dtype="bf16", B=256, H=32, Hkv=32, D=128, n=64, median=200, lo=1,
             hi=400, ragged=True, lens_seed=6),
        # scored decode: the tiny fp32 check, the grouped-query batch, and the multi-head batch over an fp8 cache
        dict(name="scored-tiny", op="scored", dtype="f32", B=4, H=8, Hkv=8, D=64, n=1, median=33, lo=1, hi=100,
             ragged=False, lens_seed=7),
        dict(name="scored-gqa-batch", op="scored", dtype="bf16", B=256, H=32, Hkv=8, D=128, n=1, median=1024, lo=32,
             hi=8192, ragged=False, lens_seed=8),
        dict(name="scored-mha-fp8", op="scored", dtype="fp8", B=64, H=32, Hkv=32, D=128, n=1, median=512, lo=16,
             hi=2048, ragged=False, lens_seed=9),
        # eviction: one user over budget by a few tokens, a batch cut to half, few long documents cut to an eighth
        dict(name="evict-one-user", op="evict", dtype="bf16", B=1, H=32, Hkv=8, D=128, n=1, median=300, lo=300,
             hi=300, ragged=False, keep=0.85, sink=4, recent=64, lens_seed=10),
        dict(name="evict-batch", op="evict", dtype="bf16", B=64, H=32, Hkv=32, D=128, n=1, median=512, lo=16,
             hi=2048, ragged=True, keep=0.5, sink=4, recent=32, lens_seed=11),
        dict(name="evict-long-context", op="evict", dtype="bf16", B=8, H=32, Hkv=8, D=128, n=1, median=80 * 1024,
             lo=32 * 1024, hi=128 * 1024, ragged=False, keep=0.125, sink=4, recent=128, lens_seed=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: any operator, over the whole range of its sizes."""
    op = rng.choice(["tree", "tree", "commit", "scored", "evict"])
    dtype, D = rng.choice({
        "tree": [("bf16", 128)] * 4 + [("bf16", 64)] * 2 + [("f32", 64), ("f32", 128)],
        "scored": [("bf16", 128)] * 3 + [("bf16", 64), ("f32", 64), ("f32", 128), ("fp8", 128)],
        "commit": [("bf16", 128), ("bf16", 64), ("f32", 64), ("f32", 128), ("fp8", 128)],
        "evict": [("bf16", 128), ("bf16", 64), ("f32", 64), ("f32", 128), ("fp8", 128)],
    }[op])
    G = rng.choice([1, 2, 4, 8])
    Hkv = rng.choice([1, 2, 3, 4, 5, 8, 12, 16, 32])
    while G * Hkv > 64:
        Hkv = rng.choice([1, 2, 3, 4, 5, 8])
    while True:
        B = _log_int(rng, 1, 256)
        median = _log_int(rng, 1, 100_000)
        n = _log_int(rng, 1, 96) if op in ("tree", "commit") else 1
        c = dict(op=op, dtype=dtype, B=B, H=G * Hkv, Hkv=Hkv, D=D, n=n, median=median, lo=max(1, median // 8),
                 hi=min(128 * 1024, median * 4), ragged=rng.random() < 0.5, lens_seed=rng.randrange(1 << 30))
        if op == "evict":
            c.update(keep=rng.choice([0.1, 0.25, 0.5, 0.8, 0.95]), sink=rng.choice([0, 1, 4]),
                     recent=rng.choice([0, 1, 16, 100]))
        tokens = sum(a + b for a, b in zip(_ctx(c), _drafts(c)))
        w = work(c)
        room = tokens * Hkv * D * 2 * _ESIZE[dtype]
        f_cap = 20e9 if dtype == "f32" else 500e9
        if room <= 1.5e9 and w["bytes"] <= 1.5e9 and w["flops"] <= f_cap:
            return c


# -- the parts of a case that its numbers alone decide --------------------------

def _rng(case, tag):
    return np.random.default_rng([case["lens_seed"], tag])


def _ctx(case):
    """Committed tokens of each sequence (before the drafted ones)."""
    x = case["median"] * np.exp(0.75 * _rng(case, 1).standard_normal(case["B"]))
    return [int(v) for v in np.clip(np.rint(x), case["lo"], case["hi"])]


def _drafts(case):
    """Drafted tokens of each sequence; a ragged batch has shorter trees and sequences without any."""
    if case["op"] not in ("tree", "commit"):
        return [0] * case["B"]
    if not case["ragged"]:
        return [case["n"]] * case["B"]
    r = _rng(case, 2).integers(0, case["n"] + 1, case["B"])
    r[0] = case["n"]
    return [int(v) for v in r]


def _trees(case):
    """Parent of every drafted token (-1: the context's last token); children follow their parents."""
    g = _rng(case, 3)
    out = []
    for n in _drafts(case):
        # a token extends one of the newest eight, so that trees are neither chains nor stars
        out.append([-1 if j == 0 else max(-1, j - 1 - int(g.integers(0, 8))) for j in range(n)])
    return out


def _ancestors(parents):
    """Bits of the drafted tokens that each one sees: its ancestors and itself."""
    m = []
    for j, p in enumerate(parents):
        m.append((m[p] if p >= 0 else 0) | (1 << j))
    return m


def _path(parents):
    """An accepted path: root to deepest token (the first of them)."""
    depth, best = [], -1
    for j, p in enumerate(parents):
        depth.append(1 + (depth[p] if p >= 0 else 0))
        if best < 0 or depth[j] > depth[best]:
            best = j
    path = []
    while best >= 0:
        path.append(best)
        best = parents[best]
    return path[::-1]


def _keeps(case):
    """Tokens that each sequence keeps; a ragged batch has sequences within their budget already."""
    c = _ctx(case)
    k = [max(1, int(v * case["keep"])) for v in c]
    if case["ragged"]:
        k = [v if i % 5 == 4 else x for i, (v, x) in enumerate(zip(c, k))]
    return k


def work(case):
    ctx, e, D, H, Hkv, B = _ctx(case), _ESIZE[case["dtype"]], case["D"], case["H"], case["Hkv"], case["B"]
    row = Hkv * D * e  # K (or V) of one token
    if case["op"] == "tree":
        nd = _drafts(case)
        tokens = sum(c + n for c, n in zip(ctx, nd) if n > 0)  # a sequence without a draft reads nothing
        T = sum(nd)
        pairs = sum(n * c + sum(bin(m).count("1") for m in _ancestors(p))
                    for c, n, p in zip(ctx, nd, _trees(case)))
        return {"bytes": tokens * 2 * row + T * H * D * e * 2 + tokens / 4 + T * 4 * ((case["n"] + 31) // 32),
                "flops": 4 * D * H * pairs}
    if case["op"] == "commit":
        moved = sum(sum(1 for k, u in enumerate(_path(p)) if u != k) for p in _trees(case))
        return {"bytes": moved * 2 * row * 2 + B * 8 + moved * 4, "flops": 0}
    if case["op"] == "scored":
        t = sum(ctx)
        qe = 2 if case["dtype"] == "fp8" else e
        return {"bytes": t * 2 * row + B * H * D * qe * 2 + t * Hkv * 8 + t / 4, "flops": 4 * D * H * t}
    t, k = sum(ctx), sum(_keeps(case))
    # scores read, kept K/V read and written, kept scores and positions written
    return {"bytes": t * Hkv * 4 + k * 4 * row + k * Hkv * 8, "flops": 0}


# -- inputs ---------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, B, H, Hkv, D = case["op"], case["B"], case["H"], case["Hkv"], case["D"]
    dt = _DT[case["dtype"]]
    ctx, nd = _ctx(case), _drafts(case)
    total = [c + n for c, n in zip(ctx, nd)]
    blocks = [(t + BS - 1) // BS for t in total]
    keeps = _keeps(case) if op == "evict" else [0] * B
    dst_blocks = [(k + BS - 1) // BS for k in keeps]
    nb = sum(blocks) + sum(dst_blocks) + 3
    order = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)

    def pool(std):
        if case["dtype"] == "fp8":
            x = torch.empty(nb, Hkv, BS, D, device="cuda", dtype=dt)
            for lo in range(0, nb, 4096):  # codes of values / scale, in pieces
                hi = min(nb, lo + 4096)
                x[lo:hi] = (torch.randn(hi - lo, Hkv, BS, D, generator=g, device="cuda") * 60).to(dt)
            return x
        return torch.empty(nb, Hkv, BS, D, device="cuda", dtype=dt).normal_(0.0, std, generator=g)

    def tables(counts, at):
        t = torch.full((B, max(max(counts), 1)), -1, dtype=torch.int32, device="cuda")
        col = torch.arange(t.shape[1], device="cuda")[None, :]
        cnt = torch.tensor(counts, device="cuda")[:, None]
        t[col < cnt] = order[at:at + sum(counts)]
        return t

    s = {"case": dict(case), "ctx": ctx, "nd": nd, "total": total, "kc": pool(1.0), "vc": pool(1.0),
         "scale": 1.0 / math.sqrt(D), "bt": tables(blocks, 0),
         "cl": torch.tensor(total, dtype=torch.int32, device="cuda")}
    i32 = dict(dtype=torch.int32, device="cuda")
    if op in ("tree", "commit"):
        trees = _trees(case)
        start = np.concatenate([[0], np.cumsum(nd)]).astype(np.int32)
        s["qs_host"], s["trees"] = [int(v) for v in start], trees
        s["qs"] = torch.tensor(start, device="cuda")
    if op == "tree":
        T, W = sum(nd), (case["n"] + 31) // 32
        words = np.zeros((T, W), np.uint32)
        r = 0
        for p in trees:
            for m in _ancestors(p):
                for w in range(W):
                    words[r, w] = (m >> (32 * w)) & 0xFFFFFFFF
                r += 1
        s["mask"] = torch.tensor(words.view(np.int32), device="cuda")
        s["q"] = torch.empty(T, H, D, device="cuda", dtype=dt).normal_(0.0, 2.0, generator=g)
        s["out"] = torch.empty_like(s["q"])
    elif op == "commit":
        paths = [_path(p) for p in trees]
        s["paths"] = paths
        P = max(max(len(p) for p in paths), 1)
        s["acc"] = torch.tensor([p + [0] * (P - len(p)) for p in paths], **i32)
        s["nacc"] = torch.tensor([len(p) for p in paths], **i32)
    elif op == "scored":
        qdt = torch.bfloat16 if case["dtype"] == "fp8" else dt
        s["q"] = torch.empty(B, H, D, device="cuda", dtype=qdt).normal_(0.0, 2.0, generator=g)
        s["out"] = torch.empty_like(s["q"])
        s["scores"] = torch.rand(B, Hkv, s["bt"].shape[1] * BS, generator=g, device="cuda")
        s["ks"] = s["vs"] = None
        if case["dtype"] == "fp8":
            s["ks"] = torch.rand(Hkv, generator=g, device="cuda") * 0.01 + 0.012
            s["vs"] = torch.rand(Hkv, generator=g, device="cuda") * 0.01 + 0.012
    elif op == "evict":
        s["keeps"] = keeps
        s["keep"] = torch.tensor(keeps, **i32)
        s["dst"] = tables(dst_blocks, sum(blocks))
        S = s["bt"].shape[1] * BS
        # accumulated weights have a heavy tail, and tokens that nothing attended tie at zero
        u = torch.rand(B, Hkv, S, generator=g, device="cuda")
        s["scores"] = torch.where(u < 0.1, torch.zeros_like(u), torch.exp(6 * u - 6))
        s["scores_out"] = torch.empty(B, Hkv, s["dst"].shape[1] * BS, device="cuda")
        s["kept"] = torch.empty(B, Hkv, max(keeps), **i32)
    if own:
        s["call"] = _own_call(s)
    return s


def _own_call(s):
    import paged_kv_cache_351_b200 as pa

    c = s["case"]
    op, H, Hkv, D, B = c["op"], c["H"], c["Hkv"], c["D"], c["B"]
    if op == "tree":
        n = pa.pa_tree_attention_workspace_bytes(H, Hkv, D, c["n"])
        ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
        return pa.prepare_tree_attention(s["out"], s["q"], s["kc"], s["vc"], s["bt"], s["cl"], s["qs"], s["mask"],
                                         c["n"], s["scale"], Hkv, workspace=ws)
    if op == "commit":
        return pa.prepare_tree_commit(s["kc"], s["vc"], s["bt"], s["cl"], s["qs"], s["acc"], s["nacc"])
    if op == "scored":
        n = pa.pa_decode_scored_workspace_bytes(B, H, Hkv, D, s["bt"].shape[1])
        ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
        return pa.prepare_decode_scored(s["out"], s["scores"], s["q"], s["kc"], s["vc"], s["bt"], s["cl"],
                                        s["scale"], Hkv, ws, k_scale=s["ks"], v_scale=s["vs"])
    return pa.prepare_evict(s["kc"], s["vc"], s["bt"], s["cl"], s["scores"], s["dst"], s["keep"], c["sink"],
                            c["recent"], s["scores_out"], s["kept"])


def run(state):
    op = state["case"]["op"]
    if own:
        state["call"]()
    else:
        {"tree": _plain_tree, "commit": _plain_commit, "scored": _plain_scored, "evict": _plain_evict}[op](state)
    if op == "tree":
        return state["out"]
    if op == "commit":
        return _values(state["kc"]), _values(state["vc"])
    if op == "scored":
        return state["out"], state["scores"]
    return _values(state["kc"]), _values(state["vc"]), state["scores_out"], state["kept"]


def _values(cache):
    """The cache as it is (8-bit codes as their bytes: they are only moved)."""
    return cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache


def _rows(cache, table, n):
    """The first n tokens that a table row names: [Hkv, n, D]."""
    x = cache[table[:(n + BS - 1) // BS].long()]
    return x.permute(1, 0, 2, 3).reshape(x.shape[1], -1, x.shape[3])[:, :n]


# -- plain forms ------------------------------------------------------------------

def _attend(q, k, v, scale, visible=None):
    """q [Hkv, R, D] over k, v [Hkv, n, D] in 32 bits: (output, weights)."""
    x = torch.matmul(q * scale, k.transpose(1, 2))
    if visible is not None:
        x = x.masked_fill(~visible, float("-inf"))
    m = x.amax(dim=-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    l = p.sum(dim=-1, keepdim=True)
    p = p / torch.where(l > 0, l, torch.ones_like(l))
    return torch.matmul(p, v), p


def _plain_tree(s):
    c = s["case"]
    Hkv, D, G = c["Hkv"], c["D"], c["H"] // c["Hkv"]
    bits = torch.arange(32, device="cuda", dtype=torch.int32)
    for i in range(c["B"]):
        n, r0 = s["nd"][i], s["qs_host"][i]
        if n == 0:
            continue
        k = _rows(s["kc"], s["bt"][i], s["total"][i]).float()
        v = _rows(s["vc"], s["bt"][i], s["total"][i]).float()
        q = s["q"][r0:r0 + n].float().view(n, Hkv, G, D).permute(1, 0, 2, 3).reshape(Hkv, n * G, D)
        tree = ((s["mask"][r0:r0 + n, :, None] >> bits) & 1).bool().reshape(n, -1)[:, :n]
        seen = torch.cat([torch.ones(n, s["ctx"][i], dtype=torch.bool, device="cuda"), tree], 1)
        o, _ = _attend(q, k, v, s["scale"], seen.repeat_interleave(G, 0)[None])
        s["out"][r0:r0 + n] = o.view(Hkv, n, G, D).permute(1, 0, 2, 3).reshape(n, c["H"], D).to(s["out"].dtype)


def _plain_commit(s):
    kc, vc = _values(s["kc"]), _values(s["vc"])
    c = s["case"]
    B, P = s["acc"].shape
    base = (s["cl"] - (s["qs"][1:] - s["qs"][:-1])).long()[:, None]
    step = torch.arange(P, device="cuda")[None, :]
    live = step < s["nacc"][:, None]
    src = torch.where(live, base + s["acc"].long(), torch.zeros_like(base))
    dst = torch.where(live, base + step, torch.zeros_like(base))
    row = torch.arange(B, device="cuda")[:, None]
    sb, db = s["bt"][row, src // BS].long(), s["bt"][row, dst // BS].long()
    live = live.reshape(-1)
    # which entries are live is known from the paths on the host
    keep = [i * P + k for i, p in enumerate(s["paths"]) for k in range(len(p))]
    keep = torch.tensor(keep, device="cuda", dtype=torch.long)
    sb, db, so, do = (x.reshape(-1)[keep] for x in (sb, db, src % BS, dst % BS))
    for cache in (kc, vc):
        cache[db, :, do] = cache[sb, :, so]


def _plain_scored(s):
    c = s["case"]
    Hkv, D, G = c["Hkv"], c["D"], c["H"] // c["Hkv"]
    for i in range(c["B"]):
        n = s["ctx"][i]
        k, v = _rows(s["kc"], s["bt"][i], n).float(), _rows(s["vc"], s["bt"][i], n).float()
        if s["ks"] is not None:
            k, v = k * s["ks"][:, None, None], v * s["vs"][:, None, None]
        o, p = _attend(s["q"][i].float().view(Hkv, G, D), k, v, s["scale"])
        s["out"][i] = o.reshape(c["H"], D).to(s["out"].dtype)
        s["scores"][i, :, :n] += p.sum(dim=1)


def _chosen(score, n, keep, sink, recent):
    """Ascending positions [Hkv, keep] that stay of n tokens with scores [Hkv, n]."""
    if keep >= n:
        return torch.arange(n, device=score.device).expand(score.shape[0], n)
    recent = min(recent, keep)
    sink = min(sink, keep - recent)
    mid = score[:, sink:n - recent]
    mid = torch.where(torch.isnan(mid), torch.full_like(mid, float("-inf")), mid)
    top = torch.sort(mid, dim=1, descending=True, stable=True).indices[:, :keep - sink - recent] + sink
    ends = torch.cat([torch.arange(sink, device=score.device), torch.arange(n - recent, n, device=score.device)])
    return torch.sort(torch.cat([top, ends.expand(score.shape[0], -1)], 1), dim=1).values


def _plain_evict(s):
    c = s["case"]
    Hkv = c["Hkv"]
    kc, vc = _values(s["kc"]), _values(s["vc"])
    s["scores_out"].zero_()
    s["kept"].fill_(-1)
    head = torch.arange(Hkv, device="cuda")[:, None]
    for i in range(c["B"]):
        n, keep = s["ctx"][i], min(s["keeps"][i], s["ctx"][i])
        at = _chosen(s["scores"][i, :, :n], n, keep, c["sink"], c["recent"])
        s["kept"][i, :, :keep] = at
        s["scores_out"][i, :, :keep] = s["scores"][i].gather(1, at)
        to = torch.arange(keep, device="cuda")
        db, do = s["dst"][i, to // BS].long(), to % BS
        sb, so = s["bt"][i][at // BS].long(), at % BS
        for cache in (kc, vc):
            cache[db[None, :], head, do[None, :]] = cache[sb, head, so]


# -- exact results, from the definitions, in 64 bits --------------------------------

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op in ("commit", "evict"):
        return _exact_moves(s)
    Hkv, D, G = case["Hkv"], case["D"], case["H"] // case["Hkv"]

    def token_rows(cache, i, h, n):
        pos = torch.arange(n, device="cuda")
        return cache[s["bt"][i][pos // BS].long(), h, pos % BS].double()

    if op == "tree":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        for i, tree in enumerate(s["trees"]):
            n, c = len(tree), s["ctx"][i]
            if n == 0:
                continue
            # -inf where a drafted token is not an ancestor
            bias = torch.full((n, n), -math.inf, dtype=torch.float64)
            for j in range(n):
                a = j
                while a >= 0:
                    bias[j, a] = 0.0
                    a = tree[a]
            bias = bias.cuda()
            r = slice(s["qs_host"][i], s["qs_host"][i] + n)
            for h in range(Hkv):
                k, v = token_rows(s["kc"], i, h, c + n), token_rows(s["vc"], i, h, c + n)
                for j in range(h * G, h * G + G):
                    z = s["q"][r, j].double() @ k.T * s["scale"]
                    z[:, c:] += bias
                    out[r, j] = torch.softmax(z, dim=1) @ v
        return out
    if op == "scored":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        acc = s["scores"].double()
        for i, n in enumerate(s["ctx"]):
            for h in range(Hkv):
                k, v = token_rows(s["kc"], i, h, n), token_rows(s["vc"], i, h, n)
                if s["ks"] is not None:
                    k, v = k * s["ks"][h].double(), v * s["vs"][h].double()
                w = torch.softmax(s["q"][i, h * G:h * G + G].double() @ k.T * s["scale"], dim=1)
                out[i, h * G:h * G + G] = w @ v
                acc[i, h, :n] += w.sum(0)
        return out, acc


def _exact_moves(s):
    """The caches after a commit or an eviction, one copied row at a time; positions and 8-bit codes, which have no
    64-bit value, are None."""
    c, op = s["case"], s["case"]["op"]
    bt = s["bt"].cpu().numpy()
    src, dst = [], []  # (block, head, offset) of every moved row
    scores_out = torch.zeros(s["scores_out"].shape, dtype=torch.float64) if op == "evict" else None
    for i, n in enumerate(s["ctx"]):
        if op == "commit":
            for k, u in enumerate(s["paths"][i]):
                for h in range(c["Hkv"]):
                    src.append((bt[i, (n + u) // BS], h, (n + u) % BS))
                    dst.append((bt[i, (n + k) // BS], h, (n + k) % BS))
            continue
        keep, to = min(s["keeps"][i], n), s["dst"][i].cpu().numpy()
        newest = min(c["recent"], keep)
        first = min(c["sink"], keep - newest)
        for h in range(c["Hkv"]):
            w = s["scores"][i, h, :n].cpu().numpy().astype(np.float64)
            rank = w.copy()
            if keep < n:
                rank[:first] = rank[n - newest:] = np.inf
            pos = np.sort(np.lexsort((np.arange(n), -rank))[:keep])
            scores_out[i, h, :keep] = torch.from_numpy(w[pos])
            j = np.arange(keep)
            src.append(np.stack([bt[i][pos // BS], np.full(keep, h), pos % BS], 1))
            dst.append(np.stack([to[j // BS], np.full(keep, h), j % BS], 1))
    a, b = (torch.from_numpy(np.concatenate([np.atleast_2d(x) for x in m]).astype(np.int64)).cuda() for m in (src, dst))
    caches = []
    for cache in (s["kc"], s["vc"]):
        if c["dtype"] == "fp8":
            caches.append(None)
            continue
        x = cache.double()
        x[b[:, 0], b[:, 1], b[:, 2]] = cache[a[:, 0], a[:, 1], a[:, 2]].double()
        caches.append(x)
    if op == "commit":
        return None if caches[0] is None else tuple(caches)
    return caches[0], caches[1], scores_out, None
