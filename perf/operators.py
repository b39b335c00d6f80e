"""The operators of a decoding loop over a paged KV cache, and what is measured of them.

Four operators: ``rope`` (rotary positions of new tokens, appended to the
pages), ``chunk`` (causal attention of a chunk of new tokens over the pages),
``sample`` (tokens from filtered logits and given uniforms, with the
distribution they were drawn from) and ``commit`` (the accepted path's rows
moved behind the prefix, in pages).

``own`` chooses what :func:`run` computes: False, the plain form written in
elementary torch operations; True, the package's kernels.
"""

import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "bf16": 2}


# ----------------------------------------------------------------- the cases

def listed():
    return [
        # One user's next token: a single query against about a thousand cached
        # keys. Nothing but latency.
        dict(name="chunk_one_token", op="chunk", dtype="bf16", B=1, T=1, Hq=32, Hkv=8, D=128,
             page=16, P=1024, ragged=False, lens=1),
        # A serving batch's next tokens, prefixes of every length up to 4096.
        dict(name="chunk_decode_batch", op="chunk", dtype="bf16", B=32, T=1, Hq=64, Hkv=8, D=128,
             page=64, P=4096, ragged=True, lens=2),
        # Two prompts' chunks on top of what is cached already: the tensor cores' case.
        dict(name="chunk_prefill", op="chunk", dtype="bf16", B=2, T=2048, Hq=64, Hkv=8, D=128,
             page=128, P=4096, ragged=True, lens=3),
        # A small model kept in fp32, ragged chunks of odd lengths.
        dict(name="chunk_f32", op="chunk", dtype="f32", B=3, T=201, Hq=8, Hkv=4, D=64, page=32,
             P=509, ragged=True, lens=4),
        # Eight sequences' next tokens.
        dict(name="rope_one_token", op="rope", dtype="bf16", B=8, T=1, Hq=32, Hkv=8, D=128, rot=128,
             interleaved=False, tree=False, fused=False, page=16, P=2048, ragged=False, lens=5),
        # Token trees of 64 nodes at prefixes of 4096, q, k and v as columns of one projection.
        dict(name="rope_tree", op="rope", dtype="bf16", B=32, T=64, Hq=64, Hkv=8, D=128, rot=128,
             interleaved=False, tree=True, fused=True, page=64, P=4096, ragged=True, lens=6),
        # A prompt's chunk far into a long context, half of each head rotated in
        # interleaved pairs.
        dict(name="rope_chunk_far", op="rope", dtype="bf16", B=1, T=4096, Hq=64, Hkv=8, D=128, rot=64,
             interleaved=True, tree=False, fused=False, page=128, P=100003, ragged=False, lens=7),
        # Four users' next tokens.
        dict(name="sample_decode", op="sample", dtype="f32", R=4, V=32000, S=1, probs=True, lens=8),
        # A serving batch over a large vocabulary, every row with its own settings.
        dict(name="sample_batch", op="sample", dtype="bf16", R=128, V=128256, S=1, probs=True,
             lens=9),
        # Proposals of a whole tree level: several draws a row, and the rows kept for the verifier.
        dict(name="sample_proposals", op="sample", dtype="f32", R=1024, V=32000, S=4, probs=True,
             lens=10),
        # The commit after a verification step of 32 trees.
        dict(name="commit_trees", op="commit", dtype="bf16", B=32, T=64, Hkv=8, D=128, page=64,
             P=1500, n=8, lens=11),
        # A large batch with one KV head per query head and long accepted paths.
        dict(name="commit_batch", op="commit", dtype="bf16", B=128, T=64, Hkv=32, D=128, page=16,
             P=700, n=16, lens=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw(rng):
    op = rng.choice(["chunk", "chunk", "rope", "sample", "commit"])
    lens = rng.randrange(1 << 30)
    if op == "sample":
        return dict(op=op, dtype=rng.choice(["f32", "bf16"]), R=_log_int(rng, 1, 1024),
                    V=_log_int(rng, 200, 150000), S=rng.choice([1, 1, 2, 4, 7]),
                    probs=rng.random() < 0.7, lens=lens)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    G = rng.choice([1, 2, 4, 7, 8])
    page = rng.choice([16, 32, 64, 128, 256])
    D = rng.choice([64, 128])
    if op == "commit":
        T = rng.choice([8, 20, 24, 64, 128])
        return dict(op=op, dtype=dtype, B=_log_int(rng, 1, 128), T=T, Hkv=Hkv, D=D, page=page,
                    P=_log_int(rng, 1, 2000), n=rng.randint(1, min(T, 16)), lens=lens)
    if op == "rope":
        tree = rng.random() < 0.4
        T = rng.choice([6, 20, 64, 128]) if tree else _log_int(rng, 1, 4096)
        rot = rng.choice([D, D, D // 2, D // 4, 24])
        return dict(op=op, dtype=dtype, B=_log_int(rng, 1, 32), T=T, Hq=G * Hkv, Hkv=Hkv, D=D,
                    rot=rot, interleaved=rng.random() < 0.5, tree=tree, fused=rng.random() < 0.5,
                    page=page, P=_log_int(rng, 1, 100000), ragged=rng.random() < 0.6, lens=lens)
    T = 1 if rng.random() < 0.4 else _log_int(rng, 2, 2048)
    P = _log_int(rng, 1, 8192)
    if dtype == "f32":
        T, P = min(T, 256), min(P, 1024)
    return dict(op=op, dtype=dtype, B=_log_int(rng, 1, 32), T=T, Hq=G * Hkv, Hkv=Hkv, D=D, page=page,
                P=P, ragged=rng.random() < 0.7, lens=lens)


def draw(rng):
    limits = {}
    for case in listed():
        key = (case["op"], case["dtype"] if case["op"] == "chunk" else "")
        w = work(case)
        old = limits.get(key, {"bytes": 0, "flops": 0})
        limits[key] = {k: max(w[k], old[k]) for k in w}
    while True:
        case = _draw(rng)
        limit = limits[(case["op"], case["dtype"] if case["op"] == "chunk" else "")]
        w = work(case)
        if 0 < w["bytes"] <= limit["bytes"] and w["flops"] <= limit["flops"]:
            return case


def _lengths(case):
    """Prefix and new-token counts of each sequence: fixed by the case, so that its work is."""
    rng = random.Random(case["lens"])
    B, T, P = case["B"], case["T"], case["P"]
    if not case.get("ragged"):
        return [P] * B, [T] * B
    prefix = [P] + [rng.randint(P // 8, P) for _ in range(B - 1)]
    new = [T] + [rng.randint((T + 1) // 2, T) for _ in range(B - 1)]
    return prefix, new


def _paths(case):
    """Prefix lengths and accepted paths: first children as far as they go (already in
    place), then nodes of a later branch."""
    rng = random.Random(case["lens"])
    T, n = case["T"], case["n"]
    prefix, paths = [], []
    for _ in range(case["B"]):
        prefix.append(rng.randint(max(case["P"] // 2, 1), case["P"]))
        k = rng.randint((n + 1) // 2, n)
        stay = rng.randint(0, k)
        rest = list(range(k, T))
        move = sorted(rng.sample(rest, min(k - stay, len(rest))))
        paths.append((list(range(stay)) + move) or [0])
    return prefix, paths


def work(case):
    op, es = case["op"], SIZES[case["dtype"]]
    if op == "sample":
        R, V = case["R"], case["V"]
        return {"bytes": R * V * (es + (4 if case["probs"] else 0)) + R * (16 + 12 * case["S"]),
                "flops": 4 * R * V}
    if op == "commit":
        _, paths = _paths(case)
        moved = sum(1 for path in paths for i, u in enumerate(path) if u != i)
        return {"bytes": 4 * moved * case["Hkv"] * case["D"] * es, "flops": 0}
    prefix, new = _lengths(case)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if op == "rope":
        return {"bytes": 2 * sum(new) * (Hq + 2 * Hkv) * D * es,
                "flops": 3 * sum(new) * (Hq + Hkv) * case["rot"]}
    keys = sum(t * p + t * (t + 1) // 2 for p, t in zip(prefix, new))
    return {"bytes": (2 * sum(new) * Hq + 2 * Hkv * (sum(prefix) + sum(new))) * D * es,
            "flops": 4 * D * Hq * keys}


# ---------------------------------------------------------------- the inputs

def _pages(case, prefix, new, g, dev, fill=True):
    """Block tables over a shuffled pool. Positions before the first page that the call
    touches are a prompt that all sequences share where `fill` is false."""
    page = case["page"]
    first = [0 if fill else p // page for p in prefix]
    blocks = [(p + t - 1) // page + 1 for p, t in zip(prefix, new)]
    shared = 0 if fill else 1
    num = shared + sum(n - f for n, f in zip(blocks, first)) + 2
    order = [shared + int(i) for i in torch.randperm(num - shared, generator=g, device=dev).tolist()]
    table = torch.zeros(case["B"], max(blocks) + 1, dtype=torch.int32)
    for b, (f, n) in enumerate(zip(first, blocks)):
        for i in range(f, n):
            table[b, i] = order.pop()
    return table.to(dev), num


def _randn(shape, dtype, g, dev):
    return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dtype)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    state = {"case": case}
    if case["op"] == "sample":
        R, V, S = case["R"], case["V"], case["S"]
        rng = random.Random(seed)
        # logits of a trained head: a broad body and a handful of likely tokens
        logits = 2.0 * torch.randn(R, V, generator=g, device=dev)
        hot = torch.randint(0, V, (R, 16), generator=g, device=dev)
        logits.scatter_add_(1, hot, 6.0 * torch.rand(R, 16, generator=g, device=dev))
        rows = [(rng.choice([0.6, 0.8, 1.0, 1.3]), rng.choice([0, 0, 20, 50, 1000]),
                 rng.choice([1.0, 0.8, 0.9, 0.95]), rng.choice([0.0, 0.0, 0.05]))
                for _ in range(R)]
        state.update(
            logits=logits.to(dt),
            temperature=torch.tensor([r[0] for r in rows], dtype=torch.float32, device=dev),
            top_k=torch.tensor([min(r[1], V) for r in rows], dtype=torch.int32, device=dev),
            top_p=torch.tensor([r[2] for r in rows], dtype=torch.float32, device=dev),
            min_p=torch.tensor([r[3] for r in rows], dtype=torch.float32, device=dev),
            u=torch.rand(R, S, generator=g, device=dev, dtype=torch.float64),
            tokens=torch.empty(R, S, dtype=torch.int32, device=dev),
            probs=torch.empty(R, V, dtype=torch.float32, device=dev) if case["probs"] else None)
        return state
    B, T, Hkv, D = case["B"], case["T"], case["Hkv"], case["D"]
    if case["op"] == "commit":
        prefix, paths = _paths(case)
        table, num = _pages(case, prefix, [T] * B, g, dev, fill=False)
        path = torch.full((B, T), -1, dtype=torch.int32)
        for b, p in enumerate(paths):
            path[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
        state.update(path=path.to(dev), paths=paths,
                     tokens=torch.zeros(B, T + 1, dtype=torch.int32, device=dev),
                     n_accepted=torch.tensor([len(p) for p in paths], dtype=torch.int32, device=dev))
    else:
        prefix, new = _lengths(case)
        table, num = _pages(case, prefix, new, g, dev, fill=case["op"] == "chunk")
        Hq = case["Hq"]
        state.update(new=new, n_new=torch.tensor(new, dtype=torch.int32, device=dev))
        if case["op"] == "chunk":
            state["q"] = _randn((B, T, Hq, D), dt, g, dev)
            state["out"] = torch.zeros_like(state["q"])
        elif case["fused"]:
            qkv = _randn((B, T, Hq + 2 * Hkv, D), dt, g, dev)
            state.update(q=qkv[:, :, :Hq], k=qkv[:, :, Hq:Hq + Hkv], v=qkv[:, :, Hq + Hkv:])
        else:
            state.update(q=_randn((B, T, Hq, D), dt, g, dev), k=_randn((B, T, Hkv, D), dt, g, dev),
                         v=_randn((B, T, Hkv, D), dt, g, dev))
        if case["op"] == "rope":
            state["out"] = torch.zeros(B, T, Hq, D, dtype=dt, device=dev)
            i = torch.arange(case["rot"] // 2, dtype=torch.float64, device=dev)
            state["inv_freq"] = 10000.0 ** (-2.0 * i / case["rot"])
            state["depth"] = None
            if case["tree"]:
                rng = random.Random(seed)
                depth = torch.zeros(B, T, dtype=torch.int32)
                for b in range(B):
                    d = []
                    for u in range(new[b]):
                        d.append(1 + (d[rng.randrange(u)] if u and rng.random() < 0.8 else 0))
                    depth[b, :new[b]] = torch.tensor(d, dtype=torch.int32)
                state["depth"] = depth.to(dev)
    state.update(prefix=prefix, prefix_len=torch.tensor(prefix, dtype=torch.int32, device=dev),
                 table=table, k_pages=_randn((num, Hkv, case["page"], D), dt, g, dev),
                 v_pages=_randn((num, Hkv, case["page"], D), dt, g, dev))
    return state


# ----------------------------------------------------------- the plain forms

def _logical(pages, table, n):
    """The first n logical positions of one sequence as [Hkv][n][D]."""
    page = pages.shape[2]
    rows = pages[table[:(n + page - 1) // page].long()]
    return rows.transpose(0, 1).reshape(pages.shape[1], -1, pages.shape[3])[:, :n]


def _plain_chunk(s):
    q, case = s["q"], s["case"]
    Hkv, D = case["Hkv"], case["D"]
    G = case["Hq"] // Hkv
    out = torch.zeros_like(q)
    for b, (P, T) in enumerate(zip(s["prefix"], s["new"])):
        n = P + T
        k = _logical(s["k_pages"], s["table"][b], n).float()
        v = _logical(s["v_pages"], s["table"][b], n).float()
        step = max(1, (1 << 28) // (Hkv * G * n))
        for t0 in range(0, T, step):
            t1 = min(T, t0 + step)
            m = P + t1
            qs = q[b, t0:t1].float().reshape(t1 - t0, Hkv, G, D).permute(1, 2, 0, 3)
            x = torch.matmul(qs.reshape(Hkv, -1, D), k[:, :m].transpose(1, 2)) * D ** -0.5
            x = x.reshape(Hkv, G, t1 - t0, m)
            if t1 - t0 > 1:
                pos = torch.arange(P + t0, P + t1, device=q.device)[:, None]
                key = torch.arange(m, device=q.device)[None, :]
                x = x.masked_fill(key > pos, float("-inf"))
            p = torch.exp(x - x.amax(-1, keepdim=True))
            o = torch.matmul(p.reshape(Hkv, -1, m), v[:, :m]).reshape(Hkv, G, t1 - t0, D)
            o = o / p.sum(-1, keepdim=True)
            out[b, t0:t1] = o.permute(2, 0, 1, 3).reshape(t1 - t0, -1, D).to(q.dtype)
    return {"out": out}


def _rotate(x, cos, sin, rot, interleaved):
    """x [n][H][D], cos and sin [n][rot/2]; computed and returned in cos' type."""
    y = x.to(cos.dtype)
    c, s = cos[:, None], sin[:, None]
    z = y.clone()
    if interleaved:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        z[..., 0:rot:2], z[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        z[..., :rot // 2], z[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    return z


def _plain_rope(s):
    case = s["case"]
    B, T, page = case["B"], case["T"], case["page"]
    dev = s["q"].device
    # slots behind a sequence's last token repeat it
    u = torch.arange(T, device=dev)[None].expand(B, T)
    t = torch.minimum(u, s["n_new"][:, None] - 1)
    offset = t if s["depth"] is None else torch.gather(s["depth"], 1, t) - 1
    angle = (s["prefix_len"][:, None] + offset).double().reshape(-1)[:, None] * s["inv_freq"][None]
    cos, sin = angle.cos().float(), angle.sin().float()
    seq = torch.arange(B, device=dev)[:, None].expand(B, T)
    q, k, v = (s[name][seq, t].flatten(0, 1) for name in ("q", "k", "v"))
    q = _rotate(q, cos, sin, case["rot"], case["interleaved"]).to(k.dtype)
    k = _rotate(k, cos, sin, case["rot"], case["interleaved"]).to(v.dtype)
    live = (u < s["n_new"][:, None]).reshape(-1, 1, 1)
    out = torch.where(live, q, torch.zeros_like(q)).view(B, T, -1, case["D"])
    slot = (s["prefix_len"][:, None] + t).reshape(-1).long()
    where = s["table"][seq.reshape(-1), slot // page].long()
    s["k_pages"][where, :, slot % page] = k
    s["v_pages"][where, :, slot % page] = v
    return {"q": out, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_sample(s):
    logits = s["logits"].float()
    R, V = logits.shape
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    x = order.values.double()
    w = torch.exp((x - x[:, :1]) / s["temperature"].double()[:, None])
    rank = torch.arange(V, device=logits.device)[None]
    top_k = torch.where(s["top_k"] > 0, s["top_k"], torch.full_like(s["top_k"], V))
    w = torch.where(rank < top_k[:, None], w, torch.zeros_like(w))
    before = w.cumsum(1) - w
    nucleus = before < s["top_p"].double()[:, None] * w.sum(1, keepdim=True)
    keep = (nucleus | (s["top_p"] >= 1)[:, None]) & (w >= s["min_p"].double()[:, None])
    w = torch.where(keep, w, torch.zeros_like(w))
    w = torch.zeros_like(w).scatter_(1, order.indices, w)
    cdf = w.cumsum(1)
    total = cdf[:, -1:]
    token = torch.searchsorted(cdf, s["u"] * total, right=True)
    last = (w > 0).long().mul(torch.arange(V, device=w.device)).amax(1, keepdim=True)
    out = {"tokens": torch.minimum(token, last).int()}
    if s["probs"] is not None:
        out["probs"] = (w / total).float()
    return out


def _plain_commit(s):
    case = s["case"]
    page = case["page"]
    path, n, P = s["path"].long(), s["n_accepted"], s["prefix_len"]
    B, T = path.shape
    # entries behind a path's last node repeat it
    i = torch.minimum(torch.arange(T, device=path.device)[None], n[:, None].long() - 1)
    seq = torch.arange(B, device=path.device)[:, None].expand(B, T).reshape(-1)
    start = P[:, None].long()
    src = (start + torch.gather(path, 1, i)).reshape(-1)
    dst = (start + i).reshape(-1)
    a, b = s["table"][seq, src // page].long(), s["table"][seq, dst // page].long()
    for pages in (s["k_pages"], s["v_pages"]):
        pages[b, :, dst % page] = pages[a, :, src % page]
    return {"prefix_len": P + n, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


# ------------------------------------------------------------------ the calls

def _own(s):
    import tree_speculative_decoding_ancestor_b200 as tsd

    op = s["case"]["op"]
    if op == "chunk":
        return {"out": tsd.chunk_attention_paged(s["q"], s["k_pages"], s["v_pages"], s["table"],
                                                 s["prefix_len"], s["n_new"], out=s["out"])}
    if op == "rope":
        q = tsd.rope_append_paged(s["q"], s["k"], s["v"], s["inv_freq"], s["k_pages"], s["v_pages"],
                                  s["table"], s["prefix_len"], s["n_new"], depth=s["depth"],
                                  interleaved=s["case"]["interleaved"], out=s["out"])
        return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if op == "sample":
        r = tsd.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"],
                       top_p=s["top_p"], min_p=s["min_p"], tokens=s["tokens"], probs=s["probs"])
        return {"tokens": r.tokens} if r.probs is None else {"tokens": r.tokens, "probs": r.probs}
    result = tsd.VerifyResult(s["tokens"], s["path"], s["n_accepted"])
    n = tsd.kv_commit_paged(s["k_pages"], s["v_pages"], s["table"], s["prefix_len"], result)
    return {"prefix_len": n, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def run(state):
    if own:
        return _own(state)
    return {"chunk": _plain_chunk, "rope": _plain_rope, "sample": _plain_sample,
            "commit": _plain_commit}[state["case"]["op"]](state)


# ------------------------------------------------- the definitions in 64 bits

def _exact_chunk(s):
    case = s["case"]
    Hkv, D, page = case["Hkv"], case["D"], case["page"]
    G = case["Hq"] // Hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    for b in range(case["B"]):
        P, T = s["prefix"][b], s["new"][b]
        pos = torch.arange(P + T, device=out.device)
        where = s["table"][b].long()[pos // page]
        for h in range(Hkv):
            k = s["k_pages"][where, h, pos % page].double()
            v = s["v_pages"][where, h, pos % page].double()
            rows = max(1, (1 << 27) // (P + T))
            for g in range(G):
                for t0 in range(0, T, rows):
                    t = torch.arange(t0, min(T, t0 + rows), device=out.device)
                    x = (s["q"][b, t, h * G + g].double() @ k.T) / math.sqrt(D)
                    x[pos[None] > (P + t)[:, None]] = float("-inf")
                    out[b, t, h * G + g] = torch.softmax(x, dim=1) @ v
    return {"out": out}


def _exact_rope(s):
    case = s["case"]
    rot, page, D = case["rot"], case["page"], case["D"]
    half = rot // 2
    i = torch.arange(rot, device=s["q"].device)
    pair = i // 2 if case["interleaved"] else i % half
    if case["interleaved"]:
        partner, sign = i ^ 1, torch.where(i % 2 == 0, -1.0, 1.0).double()
    else:
        partner, sign = (i + half) % rot, torch.where(i < half, -1.0, 1.0).double()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=s["out"].device)
    k_pages, v_pages = s["k_pages"].double(), s["v_pages"].double()
    for b in range(case["B"]):
        P, T = s["prefix"][b], s["new"][b]
        t = torch.arange(T, device=out.device)
        pos = P + (t if s["depth"] is None else s["depth"][b, :T].long() - 1)
        angle = (pos.double()[:, None] * s["inv_freq"][None])[:, pair]
        c, si = torch.cos(angle)[:, None], (torch.sin(angle) * sign)[:, None]
        where, row = s["table"][b].long()[(P + t) // page], (P + t) % page
        for x, put in ((s["q"][b, :T].double(), None), (s["k"][b, :T].double(), k_pages)):
            y = torch.cat([x[..., :rot] * c + x[..., partner] * si, x[..., rot:D]], dim=-1)
            if put is None:
                out[b, :T] = y
            else:
                put[where, :, row] = y
        v_pages[where, :, row] = s["v"][b, :T].double()
    return {"q": out, "k_pages": k_pages, "v_pages": v_pages}


def _exact_sample(s):
    logits = s["logits"].float().cpu().numpy()
    get = {k: s[k].cpu().numpy() for k in ("temperature", "top_k", "top_p", "min_p", "u")}
    R, V = logits.shape
    tokens = np.zeros(get["u"].shape, dtype=np.int32)
    probs = np.zeros((R, V), dtype=np.float64) if s["probs"] is not None else None
    for r in range(R):
        x = logits[r].astype(np.float64)
        p = np.exp((x - x.max()) / float(get["temperature"][r]))
        keep = np.lexsort((np.arange(V), -x))
        if get["top_k"][r] > 0:
            keep = keep[:get["top_k"][r]]
        if get["top_p"][r] < 1:
            c = np.cumsum(p[keep])
            keep = keep[:1 + int(np.sum(c < float(get["top_p"][r]) * c[-1]))]
        keep = np.sort(keep[p[keep] >= float(get["min_p"][r])])
        c = np.cumsum(p[keep])
        for j, u in enumerate(get["u"][r]):
            tokens[r, j] = keep[min(int(np.sum(c <= u * c[-1])), len(keep) - 1)]
        if probs is not None:
            probs[r, keep] = p[keep] / c[-1]
    out = {"tokens": torch.from_numpy(tokens)}
    if probs is not None:
        out["probs"] = torch.from_numpy(probs)
    return out


def _exact_commit(s):
    case, page = s["case"], s["case"]["page"]
    table = s["table"].cpu()
    out = {"prefix_len": torch.tensor([P + len(p) for P, p in zip(s["prefix"], s["paths"])],
                                      dtype=torch.int32)}
    for name in ("k_pages", "v_pages"):
        old = s[name].cpu()
        new = old.double()
        for b, (P, path) in enumerate(zip(s["prefix"], s["paths"])):
            for i, u in enumerate(path):
                new[table[b, (P + i) // page], :, (P + i) % page] = \
                    old[table[b, (P + u) // page], :, (P + u) % page].double()
        out[name] = new
    return out


def exact(case, seed):
    state = prepare(case, seed)
    return {"chunk": _exact_chunk, "rope": _exact_rope, "sample": _exact_sample,
            "commit": _exact_commit}[case["op"]](state)
