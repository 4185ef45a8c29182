"""Cases and plain forms of the operators around the paged pool: per-head norm + rotation of queries
and keys, forking and copying pooled sequences, and ragged pre-fill attention over the pool.

Shapes are those of the workloads of this repository (32 query and 8 KV heads of 128, half of them
retrieval heads, 16 sinks, window 512, contexts to 128K) and generic odd ones.
"""
import math
import random

import torch

own = False

PAGE = 128
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases

def _rope(name, n, hq, hkv, d, dtype, norm, axes, rot, interleaved):
    return dict(name=name, op="rope", n=n, hq=hq, hkv=hkv, d=d, dtype=dtype, norm=norm, axes=axes, rot=rot,
                interleaved=interleaved)


def _pool(name, op, layers, hq, hkv, hr, S, W, prefix, **more):
    return dict(name=name, op=op, layers=layers, hq=hq, hkv=hkv, hr=hr, S=S, W=W, prefix=prefix, **more)


def listed():
    return [
        # one decoded token of one sequence: nothing but latency
        _rope("rope_token", 1, 32, 8, 128, "bf16", False, 1, 128, False),
        # a decode step of a ragged batch, normed queries and keys, half of each head rotated
        _rope("norm_rope_batch", 97, 32, 8, 128, "bf16", True, 1, 64, False),
        # image and video tokens: three position axes, small heads in 32 bits, neighbours paired
        _rope("norm_rope_axes3", 10007, 16, 16, 64, "fp32", True, 3, 64, True),
        # a long pre-fill chunk as it comes from the projection
        _rope("norm_rope_chunk", 32768, 32, 8, 128, "bf16", True, 1, 128, False),
        # one branch of a short conversation (a draft that may be dropped again)
        _pool("fork_one", "fork", 4, 32, 8, 4, 16, 512, "333", n=1),
        # eight samples of one prompt
        _pool("fork_eight", "fork", 8, 32, 8, 4, 16, 512, "4200", n=8),
        # a short sequence to another pool
        _pool("copy_short", "copy", 2, 32, 8, 4, 16, 512, "1000"),
        # a long sequence to a larger pool
        _pool("copy_long", "copy", 8, 32, 8, 4, 16, 512, "32900"),
        # draft tokens of four sequences, checked together
        _pool("prefill_drafts", "prefill", 1, 32, 8, 4, 16, 512, "700,1500,128,2049", new="5,5,5,5"),
        # a question on a long shared document
        _pool("prefill_question", "prefill", 1, 32, 8, 4, 16, 512, "131000", new="64"),
        # a batch of sequences at all stages: first prompts, continued chunks, single tokens
        _pool("prefill_ragged", "prefill", 1, 32, 8, 4, 16, 512, "2048,4096,0,16384,32768,999,65536,1",
              new="130,1,1111,500,64,2000,257,300"),
        # one chunk of a long prompt
        _pool("prefill_chunk", "prefill", 1, 32, 8, 4, 16, 512, "24576", new="8192"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "fork", "copy", "prefill", "prefill"])
    if op == "rope":
        d = rng.choice([64, 128])
        hkv = rng.choice([1, 2, 4, 8, 16])
        hq = hkv * rng.choice([1, 2, 3, 4, 7, 8])
        elems = _log(rng, 1, 10 ** 8)
        n = max(1, min(32768, elems // ((hq + 2 * hkv) * d)))
        rot = rng.choice([d, d, d // 2, d // 2 + 16])
        c = _rope("", n, hq, hkv, d, rng.choice(["bf16", "bf16", "fp32"]), rng.random() < 0.7, rng.choice([1, 1, 2, 3]),
                  rot, rng.random() < 0.4)
    else:
        hkv = rng.choice([1, 2, 4, 8])
        hr = rng.randint(0, hkv)
        G = rng.choice([1, 2, 4, 4, 5, 7, 8, 16]) if hkv <= 4 else rng.choice([1, 2, 4, 4, 5])
        S, W = rng.choice([0, 1, 4, 16, 64, 130]), rng.choice([1, 17, 64, 128, 256, 512, 700])
        if op == "prefill":
            nseq = rng.choice([1, 1, 2, 3, 5, 8])
            prefix = [rng.choice([0, _log(rng, 1, 30000)]) if rng.random() < 0.2 else _log(rng, 1, 30000)
                      for _ in range(nseq)]
            new = [_log(rng, 1, 1500) for _ in range(nseq)]
            c = _pool("", op, 1, hkv * G, hkv, hr, S, W, ",".join(map(str, prefix)), new=",".join(map(str, new)))
        else:
            layers = rng.randint(1, 8)
            c = _pool("", op, layers, hkv * G, hkv, hr, S, W, str(_log(rng, 1, 32000)))
            if op == "fork":
                c["n"] = _log(rng, 1, 8)
        while work(c)["flops"] > 2.5e12 or work(c)["bytes"] > 1.2e9:  # no more than the largest listed ones
            c["prefix"] = ",".join(str(p // 2) for p in _ints(c["prefix"]))
    del c["name"]
    return c


def _ints(text):
    return [int(x) for x in text.split(",")]


def _filled(S, W, length):
    """Rows that a streaming head keeps of `length` tokens."""
    return min(length, S + W) if length <= S else S + min(length - S, W)


def work(case):
    c = case
    if c["op"] == "rope":
        rows = c["n"] * (c["hq"] + 2 * c["hkv"])
        e = 2 if c["dtype"] == "bf16" else 4
        moved = 2 * rows * c["d"] * e + 4 * c["n"] * c["axes"] + (2 * c["d"] * e if c["norm"] else 0)
        per = (4 if c["norm"] else 0) * c["d"] + 3 * c["rot"]
        return {"bytes": moved, "flops": c["n"] * (c["hq"] + c["hkv"]) * per}
    hr, hs, S, W = c["hr"], c["hkv"] - c["hr"], c["S"], c["W"]
    prefix = _ints(c["prefix"])
    row = 2 * 128 * 2  # a K and a V row
    if c["op"] == "copy":
        return {"bytes": 2 * row * c["layers"] * (hr * prefix[0] + hs * _filled(S, W, prefix[0])), "flops": 0}
    one = [c["layers"] * (hr * (p % PAGE) + hs * _filled(S, W, p)) for p in prefix]  # rows a fork copies
    if c["op"] == "fork":
        return {"bytes": row * one[0] * (1 + c["n"]), "flops": 0}
    G, hq, nbytes, flops = c["hq"] // c["hkv"], c["hq"], 0, 0
    for p, n, f in zip(prefix, _ints(c["new"]), one):
        full = n * p + n * (n + 1) // 2
        seen = sum(min(i + 1, W) + min(max(i + 1 - W, 0), S) for i in range(p, p + n))
        flops += 4 * 128 * G * (hr * full + hs * seen)
        nbytes += 2 * row * f                                   # the branch
        nbytes += row * (hr * p + hs * _filled(S, W, p))        # history
        nbytes += 2 * n * hq * 256 + 4 * n * hq                 # q, out, lse
        nbytes += row * n * c["hkv"] + row * (hr * n + hs * min(n, S + W))  # k, v, and the appended rows
    return {"bytes": nbytes, "flops": flops}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _rope_inputs(case, seed):
    c, g = case, _gen(seed)
    dt = DTYPES[c["dtype"]]
    n, pairs = c["n"], c["rot"] // 2
    s = {"qkv": _randn(g, n, c["hq"] + 2 * c["hkv"], c["d"], dtype=dt)}
    if c["norm"]:
        s["wq"] = (1 + 0.2 * torch.randn(c["d"], generator=g, device="cuda")).to(dt)
        s["wk"] = (1 + 0.2 * torch.randn(c["d"], generator=g, device="cuda")).to(dt)
    if c["axes"] == 1:  # sequences of a batch at positions of their own, or a chunk far in a prompt
        at = torch.randint(0, 1 << 20, (1, 1 if n > 256 else n), generator=g, device="cuda")
        pos = at + torch.arange(n, device="cuda") if n > 256 else at
    else:  # frames of a video, 40 patches wide and 30 high, after some text
        i = torch.arange(n, device="cuda")
        start = torch.randint(0, 4096, (1,), generator=g, device="cuda")
        pos = start + torch.stack([i // 1200, i % 1200 // 40, i % 40])[: c["axes"]]
    s["pos"] = pos.to(torch.int32).contiguous()
    s["inv_freq"] = [10000.0 ** (-i / pairs) for i in range(pairs)]
    first = pairs // 4 if c["axes"] == 3 else pairs // 2
    s["pair_axis"] = [0 if c["axes"] == 1 or i < first else 1 + (i - first) * (c["axes"] - 1) // (pairs - first)
                      for i in range(pairs)]
    return s


def _heads(case, seed):
    """Retrieval and streaming KV heads, chosen by the seed."""
    order = list(range(case["hkv"]))
    random.Random(int(seed) * 7919 + 1).shuffle(order)
    return sorted(order[: case["hr"]]), sorted(order[case["hr"]:])


def _tokens(case, seed):
    """K and V of the prefixes ([layers][2][len][hkv][128]), and q, k, v of the new tokens."""
    c, g = case, _gen(seed)
    s = {"past": [_randn(g, c["layers"], 2, p, c["hkv"], 128) for p in _ints(c["prefix"])]}
    if c["op"] == "prefill":
        total = sum(_ints(c["new"]))
        s["q"] = _randn(g, total, c["hq"], 128)
        s["k"] = _randn(g, total, c["hkv"], 128)
        s["v"] = _randn(g, total, c["hkv"], 128)
    return s


def _slots(S, W, length):
    """(positions kept by a streaming head after `length` tokens, their rows)."""
    p = torch.arange(length, device="cuda")
    p = p[(p < S) | (p >= length - W)]
    return p, torch.where(p < S, p, S + p % W)


def _pages_of(tokens, heads):
    """[layers][2][len][hkv][128] as whole pages of the retrieval heads [layers][2][pages][hr][128][128]."""
    L, two, n = tokens.shape[:3]
    np_ = -(-n // PAGE)
    out = torch.zeros(L, two, np_ * PAGE, len(heads), 128, dtype=tokens.dtype, device="cuda")
    out[:, :, :n] = tokens[:, :, :, heads]
    return out.view(L, two, np_, PAGE, len(heads), 128).transpose(3, 4).contiguous()


def _ring_of(case, tokens, heads):
    """The sink and ring rows of the streaming heads, [layers][2][hs][S+W][128]."""
    S, W = case["S"], case["W"]
    p, at = _slots(S, W, tokens.shape[2])
    out = torch.zeros(tokens.shape[0], 2, len(heads), S + W, 128, dtype=tokens.dtype, device="cuda")
    out[:, :, :, at] = tokens[:, :, p][:, :, :, heads].transpose(2, 3)
    return out


def prepare(case, seed):
    c = case
    if c["op"] == "rope":
        s = _rope_inputs(c, seed)
        if own:
            from head_split_kv_duo_b200.duo import DuoRope
            s["rope"] = DuoRope(c["d"], s["inv_freq"], pair_axis=s["pair_axis"], interleaved=c["interleaved"])
        s["inv_freq"] = torch.tensor(s["inv_freq"], dtype=torch.float64, device="cuda")
        s["pair_axis"] = torch.tensor(s["pair_axis"], device="cuda")
    else:
        t = _tokens(c, seed)
        ret, stm = _heads(c, seed)
        prefix, new = _ints(c["prefix"]), _ints(c.get("new", "0"))
        # pages that the prefixes take, the first page that a pass takes, and how many it takes
        held = [-(-p // PAGE) for p in prefix]
        first = sum(held)
        if c["op"] == "copy":
            taken = held[0]
        elif c["op"] == "fork":
            taken = c["n"] * (prefix[0] % PAGE > 0)
        else:
            taken = sum(-(-(p + n) // PAGE) - p // PAGE for p, n in zip(prefix, new))
        children = 1 if c["op"] == "copy" else c.get("n", len(prefix))
        s = {"ret": ret, "stm": stm, "prefix": prefix, "new": new, "first": first, "taken": taken,
             "children": children}
        if c["op"] == "prefill":
            s.update(q=t["q"], k=t["k"], v=t["v"])
        if own:
            from head_split_kv_duo_b200.duo import DuoPool
            mask = torch.zeros(c["layers"], c["hkv"], dtype=torch.uint8)
            mask[:, ret] = 1
            longest = max(p + n for p, n in zip(prefix, new)) + 1
            make = lambda seqs, pages: DuoPool(c["layers"], c["hkv"], mask, c["S"], c["W"], seqs, longest,  # noqa: E731
                                               max(1, pages), q_heads=c["hq"])
            s["pool"] = pool = make(len(prefix) + (0 if c["op"] == "copy" else children),
                                    first + (0 if c["op"] == "copy" else taken))
            s["seqs"] = [pool.open() for _ in prefix]
            for i, past in zip(s["seqs"], t["past"]):
                for layer in range(c["layers"] if past.shape[2] else 0):
                    pool.append_kv(layer, i, past[layer, 0].contiguous(), past[layer, 1].contiguous())
            to, slot, page = pool, len(prefix), first
            if c["op"] == "copy":
                s["to"] = to = make(1, taken + 5)
                s["to"].close_seq(s["to"].open())
                slot = page = 0
            s["out"] = _views(c, to, slot, children, page, taken, len(ret), len(stm))
        else:
            s["past_pages"] = [_pages_of(x, ret) for x in t["past"]]
            s["past_rings"] = torch.stack([_ring_of(c, x, stm) for x in t["past"]], 2)
            shape = (c["layers"], 2, taken, len(ret), PAGE, 128)
            s["pages"] = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
            s["rings"] = torch.zeros(c["layers"], 2, children, len(stm), c["S"] + c["W"], 128, dtype=torch.bfloat16,
                                     device="cuda")
    s["case"] = c
    return s


def _views(c, pool, slot, children, page, taken, hr, hs):
    """What a pass writes into a pool: sinks + rings of its sequences and the pages they take, per layer."""
    from head_split_kv_duo_b200 import duo
    rings, pages = [], []
    for layer in range(c["layers"]):
        for which in (duo.DUO_REGION_STRM_K, duo.DUO_REGION_STRM_V):
            r = pool.region(layer, which).view(torch.bfloat16).view(-1, hs, c["S"] + c["W"], 128) if hs else None
            rings.append(r[slot:slot + children] if hs else torch.zeros(0, device="cuda"))
        for which in (duo.DUO_REGION_RETR_K, duo.DUO_REGION_RETR_V):
            r = pool.region(layer, which).view(torch.bfloat16).view(-1, hr, PAGE, 128) if hr else None
            pages.append(r[page:page + taken] if hr else torch.zeros(0, device="cuda"))
    return {"rings": rings, "pages": pages}


# ------------------------------------------------------------------ one pass

def run(s):
    c = s["case"]
    if own:
        return _run_own(s)
    if c["op"] == "rope":
        return _plain_rope(s)
    if c["op"] == "prefill":
        return _plain_prefill(s)
    pages, rings = s["pages"], s["rings"]
    rings.copy_(s["past_rings"])  # one row per child, each the parent's
    if c["op"] == "copy":
        pages.copy_(s["past_pages"][0])
    else:
        pages.copy_(s["past_pages"][0][:, :, -1:])
    return _outputs(c, rings, pages)


def _outputs(c, rings, pages):
    none = torch.zeros(0, device=rings.device)
    both = [(layer, kv) for layer in range(c["layers"]) for kv in range(2)]
    return {"rings": [rings[i, j] if rings.shape[3] else none for i, j in both],
            "pages": [pages[i, j] if pages.shape[3] else none for i, j in both]}


def _run_own(s):
    c = s["case"]
    if c["op"] == "rope":
        q, k, v = s["qkv"].split((c["hq"], c["hkv"], c["hkv"]), 1)
        return s["rope"].norm_rope(q, k, s["pos"], v=v, q_weight=s.get("wq"), k_weight=s.get("wk"), eps=1e-6)
    pool = s["pool"]
    if c["op"] == "copy":
        s["to"].close_seq(pool.copy(s["seqs"][0], s["to"]))
        return s["out"]
    if c["op"] == "fork":
        children = pool.fork(s["seqs"][0], c["n"])
        for i in children:
            pool.close_seq(i)
        return s["out"]
    children = [pool.fork(i)[0] for i in s["seqs"]]
    out, lse = pool.prefill(0, children, s["new"], s["q"], s["k"], s["v"])
    for i in children:
        pool.close_seq(i)
    return {"out": out, "lse": lse, **s["out"]}


# ------------------------------------------------------------------ plain forms

def _plain_rope(s):
    c = s["case"]
    dt, rot = DTYPES[c["dtype"]], c["rot"]
    q, k, v = s["qkv"].split((c["hq"], c["hkv"], c["hkv"]), 1)
    turns = s["pos"].double()[s["pair_axis"]].t() * s["inv_freq"] / (2 * math.pi)  # [n][pairs], far positions in 64 bits
    a = (2 * math.pi * (turns - turns.floor()))
    cos, sin = a.cos().float()[:, None], a.sin().float()[:, None]

    def one(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
        r = x[..., :rot]
        u, w2 = (r[..., 0::2], r[..., 1::2]) if c["interleaved"] else (r[..., : rot // 2], r[..., rot // 2:])
        u, w2 = u * cos - w2 * sin, u * sin + w2 * cos
        r = torch.stack((u, w2), -1).flatten(-2) if c["interleaved"] else torch.cat((u, w2), -1)
        return torch.cat((r, x[..., rot:]), -1).to(dt)

    return one(q, s.get("wq")), one(k, s.get("wk")), v.contiguous()


def _softmax_attend(q, k, v, seen, scale):
    """q [h][G][n][128], k, v [h][L][128] in 32 bits, seen [n][L]: (out [h][G][n][128], lse [h][G][n])."""
    h, G, n, _ = q.shape
    x = torch.bmm(q.reshape(h, G * n, 128), k.transpose(1, 2)).view(h, G, n, -1) * scale
    x = x.masked_fill_(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    x = x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    o = torch.bmm(x.view(h, G * n, -1), v).view(h, G, n, 128) / l
    return o, (m + l.log())[..., 0]


def _plain_prefill(s):
    c = s["case"]
    S, W, G = c["S"], c["W"], c["hq"] // c["hkv"]
    ret, stm, scale = s["ret"], s["stm"], 1 / math.sqrt(128)
    out = torch.empty(s["q"].shape, dtype=torch.float32, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
    pages, rings = s["pages"], s["rings"]
    pages.zero_()
    tok, branch, fresh = 0, 0, sum(p % PAGE > 0 for p in s["prefix"])
    # sequence by sequence: their histories have different lengths
    for i, (p, n) in enumerate(zip(s["prefix"], s["new"])):
        at = slice(tok, tok + n)
        tok += n
        kv = torch.stack((s["k"][at], s["v"][at]))
        q = s["q"][at].float().view(n, c["hkv"], G, 128).permute(1, 2, 0, 3)  # [hkv][G][n][128]
        pos = torch.arange(p, p + n, device="cuda")
        o_at, l_at = out[at].view(n, c["hkv"], G, 128), lse[at].view(n, c["hkv"], G)
        if ret:
            # past rows as they lie in the pages, then the chunk's
            past = s["past_pages"][i][0].transpose(2, 3).flatten(1, 2)[:, :p]
            full = torch.cat((past, kv[:, :, ret]), 1).float().transpose(1, 2)  # [2][hr][p+n][128]
            keys = torch.arange(p + n, device="cuda")
            step = max(1, (1 << 28) // (len(ret) * G * (p + n)))  # queries whose logits fit a gigabyte
            for a in range(0, n, step):
                b = min(n, a + step)
                o, l = _softmax_attend(q[ret][:, :, a:b], full[0], full[1], keys <= pos[a:b, None], scale)
                o_at[a:b, ret] = o.permute(2, 0, 1, 3)
                l_at[a:b, ret] = l.permute(2, 0, 1)
            # the chunk's rows behind the branch's, in the pages that the pass takes
            lead = p % PAGE
            count = -(-(p + n) // PAGE) - p // PAGE
            tail = torch.zeros(2, count * PAGE, len(ret), 128, dtype=kv.dtype, device="cuda")
            tail[:, :lead] = past[:, p - lead:]
            tail[:, lead:lead + n] = kv[:, :, ret]
            tail = tail.view(2, count, PAGE, len(ret), 128).transpose(2, 3)
            if lead:
                pages[0, :, branch] = tail[:, 0]
            pages[0, :, fresh:fresh + count - (lead > 0)] = tail[:, int(lead > 0):]
        branch += p % PAGE > 0
        fresh += -(-(p + n) // PAGE) - -(-p // PAGE)
        if stm:
            kept, rows = _slots(S, W, p)
            full = torch.cat((s["past_rings"][0, :, i][:, :, rows].transpose(1, 2), kv[:, :, stm]), 1)
            full = full.float().transpose(1, 2)
            keys = torch.cat((kept, pos))
            step = max(1, (1 << 28) // (len(stm) * G * len(keys)))
            for a in range(0, n, step):
                b = min(n, a + step)
                x = pos[a:b, None]
                o, l = _softmax_attend(q[stm][:, :, a:b], full[0], full[1],
                                       (keys <= x) & ((keys < S) | (x - keys < W)), scale)
                o_at[a:b, stm] = o.permute(2, 0, 1, 3)
                l_at[a:b, stm] = l.permute(2, 0, 1)
            rings[0, :, i] = s["past_rings"][0, :, i]
            to, rows = _slots(S, W, p + n)
            to, rows = to[to >= p] - p, rows[to >= p]
            rings[0, :, i][:, :, rows] = kv[:, to][:, :, stm].transpose(1, 2)
    return {"out": out.to(torch.bfloat16), "lse": lse, **_outputs(c, rings, pages)}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    c = case
    if c["op"] == "rope":
        return _exact_rope(c, _rope_inputs(c, seed))
    t = _tokens(c, seed)
    ret, stm = _heads(c, seed)
    prefix, new = _ints(c["prefix"]), _ints(c.get("new", "0"))
    res, at = {}, 0
    after = []  # every token of each sequence after the pass
    if c["op"] == "prefill":
        res = {"out": torch.zeros(t["q"].shape, dtype=torch.float64, device="cuda"),
               "lse": torch.zeros(t["q"].shape[:2], dtype=torch.float64, device="cuda")}
        for past, p, n in zip(t["past"], prefix, new):
            k = torch.cat((past[0, 0], t["k"][at:at + n]))
            v = torch.cat((past[0, 1], t["v"][at:at + n]))
            after.append(torch.stack((k, v))[None])
            _exact_attend(c, ret, t["q"][at:at + n], k, v, p, res["out"][at:at + n], res["lse"][at:at + n])
            at += n
    else:
        after = [t["past"][0]] * (c.get("n", 1))
    L = c["layers"]
    rings = torch.zeros(L, 2, len(after), len(stm), c["S"] + c["W"], 128, dtype=torch.float64, device="cuda")
    branch, fresh = [], []
    for i, x in enumerate(after):
        for p in range(x.shape[2]) if x.shape[2] < 64 else _kept(c, x.shape[2]):
            row = p if p < c["S"] else c["S"] + p % c["W"]
            rings[:, :, i, :, row] = x[:, :, p, stm].double()
        np_ = -(-x.shape[2] // PAGE)
        full = torch.cat((x[:, :, :, ret].double(), torch.zeros(L, 2, np_ * PAGE - x.shape[2], len(ret), 128,
                                                                dtype=torch.float64, device="cuda")), 2)
        cut = [full[:, :, j * PAGE:(j + 1) * PAGE].transpose(2, 3) for j in range(np_)]
        if c["op"] == "copy":
            fresh += cut
        elif c["op"] == "fork":
            fresh += cut[-1:] if prefix[0] % PAGE else []
        else:
            cut = cut[prefix[i] // PAGE:]
            branch += cut[:1] if prefix[i] % PAGE else []
            fresh += cut[1:] if prefix[i] % PAGE else cut
    pages = torch.stack(branch + fresh, 2) if branch + fresh else torch.zeros(L, 2, 0, len(ret), PAGE, 128,
                                                                              device="cuda", dtype=torch.float64)
    return {**res, **_outputs(c, rings, pages)}


def _kept(c, length):
    """Positions that a streaming head keeps of a long sequence."""
    return list(range(min(c["S"], length))) + list(range(max(c["S"], length - c["W"]), length))


def _exact_attend(c, ret, q, k, v, p, out, lse):
    """The definition over the whole history, head by head."""
    G, n = c["hq"] // c["hkv"], q.shape[0]
    j = torch.arange(p + n, device="cuda")
    for g in range(c["hkv"]):
        kd, vd = k[:, g].double(), v[:, g].double()
        step = max(1, (1 << 27) // (G * (p + n)))
        for a in range(0, n, step):
            b = min(n, a + step)
            i = torch.arange(p + a, p + b, device="cuda")[:, None]
            ok = j <= i if g in ret else (j <= i) & ((j < c["S"]) | (j > i - c["W"]))
            qd = q[a:b, g * G:(g + 1) * G].double()
            x = torch.einsum("ngd,ld->ngl", qd, kd) / math.sqrt(128.0)
            x = torch.where(ok[:, None], x, -math.inf)
            z = torch.logsumexp(x, -1)
            lse[a:b, g * G:(g + 1) * G] = z
            out[a:b, g * G:(g + 1) * G] = torch.exp(x - z[..., None]) @ vd


def _exact_rope(c, s):
    q, k, v = s["qkv"].double().split((c["hq"], c["hkv"], c["hkv"]), 1)
    pairs = c["rot"] // 2
    angle = torch.zeros(c["n"], pairs, dtype=torch.float64, device="cuda")
    for i in range(pairs):
        angle[:, i] = s["pos"][s["pair_axis"][i]].double() * s["inv_freq"][i]
    z = torch.polar(torch.ones_like(angle), angle)[:, None]
    res = []
    for x, w in ((q, s.get("wq")), (k, s.get("wk"))):
        if w is not None:
            x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / c["d"] + 1e-6) * w.double()
        y = x.clone()
        i = torch.arange(pairs, device="cuda")
        first, second = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + pairs)
        turned = torch.complex(x[..., first], x[..., second]) * z
        y[..., first], y[..., second] = turned.real, turned.imag
        res.append(y)
    return res[0], res[1], v
