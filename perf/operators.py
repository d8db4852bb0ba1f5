"""Cases of the attention side of a decode or prefill step.

The token indexer of this package hands every query the tokens it selected.
Four operators turn that into attention: rotary positions on the rows that
need them, the attention cache written (and quantised) as tokens arrive, that
cache read back at listed tokens, and attention over the selected tokens or a
whole prefix, with a tree of drafted tokens behind it.

``run`` is one pass: with ``own`` false in elementary torch operations, with
``own`` true through the package's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0


# ----------------------------------------------------------------- the cases

def listed():
    return [
        # rotary positions of one decode step: the index queries of 8 sequences near position 131071 and their 8 new
        # index keys, half of each head rotated, positions scaled for the long context
        dict(name="rope_decode", op="rope", n=8, heads=64, keys=8, d=128, rot=64, first=0, layout="interleaved",
             scaling="yarn", factor=32.0, orig=4096, far=131072),
        # the same of a prefill chunk of 2048 queries, whole heads rotated in halves
        dict(name="rope_prefill", op="rope", n=2048, heads=64, keys=2048, d=128, rot=128, first=0, layout="half",
             scaling="none", factor=1.0, orig=4096, far=65536),
        # the new token of 8 sequences written to an e4m3 attention cache, its key rotated on the way
        dict(name="append_decode", op="append", n_seq=8, count=1, L=4096, h_kv=8, d=128, fp8=True, rot=64,
             layout="half"),
        # a prefill chunk of 2 sequences written to an e4m3 cache
        dict(name="append_prefill", op="append", n_seq=2, count=8192, L=16384, h_kv=8, d=128, fp8=True, rot=128,
             layout="interleaved"),
        # an odd number of tokens written to a bf16 cache
        dict(name="append_bf16", op="append", n_seq=5, count=333, L=1024, h_kv=4, d=128, fp8=False, rot=64,
             layout="half"),
        # the 2048 selected tokens of 8 sequences read back from an e4m3 cache
        dict(name="read_selected", op="read", n_seq=8, n=8, sel=2048, L=32768, h_kv=8, d=128, fp8=True),
        # a short odd list read back from a bf16 cache
        dict(name="read_short", op="read", n_seq=3, n=3, sel=77, L=1000, h_kv=2, d=64, fp8=False),
        # one short sequence, 256 selected tokens: latency
        dict(name="attend_tiny", op="attend", n_seq=1, per=1, L=4096, sel=256, h_kv=8, group=4, d=128, fp8=False,
             tree=False),
        # a decode batch at 128K: 8 sequences, 2048 selected tokens each, e4m3 cache
        dict(name="attend_decode", op="attend", n_seq=8, per=1, L=131072, sel=2048, h_kv=8, group=8, d=128, fp8=True,
             tree=False),
        # a prefill chunk: 512 queries of one sequence, each with its own 2048 selected tokens
        dict(name="attend_prefill", op="attend", n_seq=1, per=512, L=65536, sel=2048, h_kv=4, group=16, d=128, fp8=True,
             tree=False),
        # drafted trees of up to 16 tokens verified for 8 sequences, each node with its own selection
        dict(name="tree_selected", op="attend", n_seq=8, per=16, L=32768, sel=2048, h_kv=8, group=8, d=128, fp8=True,
             tree=True),
        # drafted trees of up to 24 tokens over the whole prefixes (no selection) of 4 ragged sequences
        dict(name="tree_prefix", op="attend", n_seq=4, per=24, L=32768, sel=0, h_kv=8, group=4, d=128, fp8=False,
             tree=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "read", "attend", "attend", "attend"])
    if op == "rope":
        n, d = _log(rng, 1, 2048), rng.choice([64, 128, 128, 256])
        rot = rng.choice([d, d // 2, 2 * rng.randint(1, d // 2)])
        return dict(op=op, n=n, heads=_log(rng, 1, 64 * 128 // d), keys=rng.choice([0, n, _log(rng, 1, 2048)]), d=d, rot=rot,
                    first=rng.choice([0, d - rot]), layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]), factor=rng.choice([2.0, 8.0, 32.0]),
                    orig=4096, far=rng.choice([4096, 65536, 262144]))
    if op == "append":
        n_seq, h_kv, d = _log(rng, 1, 32), rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
        count = _log(rng, 1, max(2, 16384 // n_seq))
        return dict(op=op, n_seq=n_seq, count=count, L=count + rng.randint(0, 2048), h_kv=h_kv, d=d,
                    fp8=rng.random() < 0.6, rot=rng.choice([0, d, d // 2]), layout=rng.choice(["half", "interleaved"]))
    if op == "read":
        n_seq, L = _log(rng, 1, 16), _log(rng, 64, 32768)
        return dict(op=op, n_seq=n_seq, n=_log(rng, 1, 32), sel=min(L, _log(rng, 1, 2048)), L=L,
                    h_kv=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 128]), fp8=rng.random() < 0.6)
    d, fp8 = rng.choice([64, 128, 128]), rng.random() < 0.6
    h_kv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 7, 8, 16])
    tree = rng.random() < 0.5
    if rng.random() < 0.3:  # whole prefixes
        n_seq, per, L, sel = _log(rng, 1, 8), _log(rng, 1, 24), _log(rng, 16, 16384), 0
        per = max(1, min(per, int(4e10 / (4 * n_seq * L * h_kv * group * d))))
    else:
        n_seq, L = _log(rng, 1, 16), _log(rng, 64, 65536)
        per, sel = _log(rng, 1, max(2, 128 // n_seq)), min(L, _log(rng, 16, 2048))
    return dict(op="attend", n_seq=n_seq, per=min(per, 64) if tree else per, L=L, sel=sel, h_kv=h_kv, group=group, d=d,
                fp8=fp8, tree=tree)


# ------------------------------------------------------------- made from both

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _lens(c):
    """Ragged prefix lengths: a quarter of the longest at the most is missing."""
    return [max(1, c["L"] - (131 * s) % (c["L"] // 4 + 1)) for s in range(c["n_seq"])]


def _nodes(c):
    """Queries of each sequence: ragged when they are the nodes of drafted trees."""
    if not c["tree"]:
        return [c["per"]] * c["n_seq"]
    return [c["per"] - (7 * s) % max(1, c["per"] // 3) for s in range(c["n_seq"])]


def _frequencies(rot, base, scaling, factor, orig):
    """Angle per position of each rotated pair (64 bits), and the amplitude of the rotated elements."""
    i = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
    amplitude = 1.0
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2)) if rot > 2 else base
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        def pair_of(turns):
            return rot * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(pair_of(32.0)), 0), min(math.ceil(pair_of(1.0)), rot - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f * (1 - ramp) + f / factor * ramp
        amplitude = 0.1 * math.log(factor) + 1.0
    return f, amplitude


def _quantised(x):
    """Rows of x (last axis) as e4m3 codes with one scale each."""
    amax = x.abs().amax(-1)
    scale = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
    return (x / scale[..., None]).to(torch.float8_e4m3fn), scale


def _cache(c, g, tokens, cap):
    """An attention cache of n_seq x cap tokens of which the first `tokens` hold keys and values, the others zero."""
    shape = (c["n_seq"], cap, c["h_kv"], c["d"])
    out = {}
    for name in ("k", "v"):
        # keys with a few strong channels, as trained keys have
        x = torch.randn(shape, generator=g, device=DEV)
        if name == "k":
            x *= 1 + 3 * (torch.arange(c["d"], device=DEV) % 16 == 5)
        x[:, tokens:] = 0
        if c["fp8"]:
            out[name], out[name + "_scale"] = _quantised(x)
        else:
            out[name], out[name + "_scale"] = x.to(torch.bfloat16), None
        del x
    return out


def _tree(nodes, per, seed):
    """Words of 32 visible drafted tokens for each node (itself and its ancestors), trees drawn from the seed."""
    g = torch.Generator().manual_seed(seed)
    words, rows = (per + 31) // 32, []
    for t in nodes:
        seen = []
        for j in range(t):
            parent = int(torch.randint(-1, j, (1,), generator=g)) if j else -1
            seen.append((seen[parent] if parent >= 0 else 0) | (1 << j))
        rows += [[(m >> (32 * w)) & 0xFFFFFFFF for w in range(words)] for m in seen]
    return torch.tensor(rows, dtype=torch.int64).to(torch.int32).to(DEV)


# ------------------------------------------------------------------- prepare

def prepare(case, seed):
    c, g = case, _gen(seed)
    st = dict(c)
    if c["op"] == "rope":
        st["freq"], st["amplitude"] = _frequencies(c["rot"], 10000.0, c["scaling"], c["factor"], c["orig"])
        st["rows"] = []
        for n, heads in ((c["n"], c["heads"]), (c["keys"], 1)):
            if n:
                x = torch.randn(n, heads, c["d"], generator=g, device=DEV).to(torch.bfloat16)
                pos = torch.randint(max(0, c["far"] - 2 * n), c["far"], (n,), generator=g, device=DEV).to(torch.int32)
                st["rows"].append((x, pos, torch.empty_like(x)))
    elif c["op"] == "append":
        st["freq"], st["amplitude"] = _frequencies(c["rot"], 500000.0, "none", 1.0, 4096) if c["rot"] else (None, 1.0)
        start = [(37 * s) % (c["L"] - c["count"] + 1) for s in range(c["n_seq"])]
        st["pos"] = torch.tensor(start, dtype=torch.int32, device=DEV)
        shape = (c["n_seq"], c["count"], c["h_kv"], c["d"])
        st["new_k"] = torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)
        st["new_v"] = torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)
        st |= _cache(c, g, max(start), c["L"])
        st["seq_len"] = st["pos"].clone()
    elif c["op"] == "read":
        st |= _cache(c, g, c["L"], c["L"])
        st["seq_len"] = torch.full((c["n_seq"],), c["L"], dtype=torch.int32, device=DEV)
        st["seq"] = torch.randint(0, c["n_seq"], (c["n"],), generator=g, device=DEV).to(torch.int32)
        score = torch.rand(c["n"], c["L"], generator=g, device=DEV)
        st["tok"] = score.topk(c["sel"], dim=1).indices.sort(dim=1).values.to(torch.int32)
    else:
        nodes, lens = _nodes(c), _lens(c)
        drafts = c["per"] if c["tree"] else 0
        st |= _cache(c, g, c["L"] + drafts, c["L"] + drafts)
        st["seq_len"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        counts = torch.tensor(nodes, device=DEV)
        st["q_seq"] = torch.repeat_interleave(torch.arange(c["n_seq"], device=DEV), counts).to(torch.int32)
        first = counts.cumsum(0) - counts
        back = 0 if c["tree"] else (counts[st["q_seq"].long()] - 1 - (torch.arange(int(sum(nodes)), device=DEV) -
                                                                     first[st["q_seq"].long()]))
        # a node sees the committed prefix; a prefill query sees the prefix that ends at itself
        st["q_pos"] = (st["seq_len"][st["q_seq"].long()] - 1 - back).clamp_min(0).to(torch.int32)
        st["q"] = torch.randn(sum(nodes), c["h_kv"] * c["group"], c["d"], generator=g, device=DEV).to(torch.bfloat16)
        st["topk"] = st["start"] = st["mask"] = None
        if c["sel"]:
            # queries of one sequence select mostly the same tokens
            score = torch.rand(c["n_seq"], c["L"], generator=g, device=DEV)[st["q_seq"].long()]
            score = score + 0.2 * torch.rand(score.shape, generator=g, device=DEV)
            at = torch.arange(c["L"], device=DEV)
            score = torch.where(at <= st["q_pos"][:, None], score, -1.0)
            best = score.topk(c["sel"], dim=1)
            tok = torch.where(best.values >= 0, best.indices, c["L"]).sort(dim=1).values
            st["topk"] = torch.where(tok < c["L"], tok, -1).to(torch.int32)
        if drafts:
            st["start"] = st["seq_len"].clone()
            st["mask"] = _tree(nodes, c["per"], seed)
    if own:
        st["handle"] = _handles(st)
    return st


def _handles(st):
    """What a program of the package's user keeps from call to call."""
    from long_context_misa_b200 import attention as A
    from long_context_misa_b200 import misa as M
    h = {}
    if st["op"] == "rope":
        h["rope"] = A.Rope(st["rot"], base=10000.0, layout=st["layout"], first=st["first"], scaling=st["scaling"],
                           factor=st["factor"], orig_len=st["orig"], device=DEV)
        return h
    h["kv"] = A.KVCache(st["k"], st["v"], st["k_scale"], st["v_scale"], st["seq_len"])
    if st["op"] == "append":
        h["rope"] = A.Rope(st["rot"], base=500000.0, layout=st["layout"], device=DEV) if st["rot"] else None
    elif st["op"] == "attend":
        h["q"] = A.AttentionQueries(st["q"], st["q_seq"], st["q_pos"])
        h["draft"] = A.Draft(st["start"], st["mask"], st["per"]) if st["tree"] else None
        h["ws"] = M.Workspace(DEV)
    return h


# ----------------------------------------------------------------------- run

def run(state):
    return (_run_own if own else {"rope": _rope, "append": _append, "read": _read, "attend": _attend}[state["op"]])(state)


def _run_own(st):
    from long_context_misa_b200 import attention as A
    h = st["handle"]
    if st["op"] == "rope":
        A.apply_rope(h["rope"], st["rows"])
        return [out for _, _, out in st["rows"]]
    if st["op"] == "append":
        A.append_kv(h["kv"], st["new_k"], st["new_v"], st["pos"], rope=h["rope"])
        return _written(st)
    if st["op"] == "read":
        return A.read_kv(h["kv"], st["seq"], st["tok"])
    out, lse = A.attend(h["kv"], h["q"], topk=st["topk"], draft=h["draft"], ws=h["ws"], with_lse=True)
    return {"out": out, "lse": lse}


def _written(st):
    r = {"k": st["k"], "v": st["v"], "seq_len": st["seq_len"]}
    return r | ({"k_scale": st["k_scale"], "v_scale": st["v_scale"]} if st["fp8"] else {})


def _rotated(x, pos, freq, amplitude, first, layout):
    """Rows x (..., heads, d) rotated by their positions (...), in 32 bits; the angles in 64."""
    x = x.float()
    rot = 2 * freq.numel()
    turn = torch.remainder(pos.double()[..., None] * freq, 2 * math.pi)
    cos = (torch.cos(turn) * amplitude).float()[..., None, :]
    sin = (torch.sin(turn) * amplitude).float()[..., None, :]
    part = x[..., first:first + rot]
    if layout == "half":
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        part = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    return torch.cat([x[..., :first], part, x[..., first + rot:]], dim=-1)


def _rope(st):
    return [_rotated(x, pos, st["freq"], st["amplitude"], st["first"], st["layout"]).to(torch.bfloat16)
            for x, pos, _ in st["rows"]]


def _append(st):
    at = st["pos"].long()[:, None] + torch.arange(st["count"], device=DEV)
    seq = torch.arange(st["n_seq"], device=DEV)[:, None]
    k, v = st["new_k"].float(), st["new_v"].float()
    if st["rot"]:
        k = _rotated(k, at, st["freq"], st["amplitude"], 0, st["layout"])
    for name, x in (("k", k), ("v", v)):
        if st["fp8"]:
            codes, st[name + "_scale"][seq, at] = _quantised(x)
            st[name].view(torch.uint8)[seq, at] = codes.view(torch.uint8)
        else:
            st[name][seq, at] = x.to(torch.bfloat16)
    st["seq_len"].copy_(st["pos"] + st["count"])
    return _written(st)


def _rows(st, name, seq, tok):
    """The cache's rows at (seq, tok), dequantised in 32 bits."""
    x = st[name]
    if not st["fp8"]:
        return x[seq, tok].float()
    return x.view(torch.uint8)[seq, tok].view(torch.float8_e4m3fn).float() * st[name + "_scale"][seq, tok][..., None]


def _read(st):
    seq, tok = st["seq"].long()[:, None], st["tok"].long()
    there = (tok >= 0)[..., None, None]
    return tuple(torch.where(there, _rows(st, n, seq, tok.clamp_min(0)), 0.0).to(torch.bfloat16) for n in ("k", "v"))


def _bits(st):
    """Visible drafted tokens of each query, as truth values."""
    j = torch.arange(st["per"], device=DEV)
    return (st["mask"][:, j // 32] >> (j % 32)) & 1 != 0


def _softmax_sum(s, seen, v, eq):
    """Weighted values and the logarithm of the weights' sum; nothing visible gives zeros and -inf."""
    s = torch.where(seen, s, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m > -math.inf, m, 0.0))
    total = p.sum(-1)
    o = torch.einsum(eq, p, v) / torch.where(total > 0, total, 1.0)[..., None]
    return o, m[..., 0] + torch.log(total)


def _attend(st):
    seq, d = st["q_seq"].long(), st["d"]
    q = st["q"].float().view(-1, st["h_kv"], st["group"], d)
    if st["sel"]:
        # a list of tokens for each query, the drafted ones behind it
        tok, seen = st["topk"].long().clamp_min(0), st["topk"] >= 0
        if st["tree"]:
            tok = torch.cat([tok, st["start"].long()[seq][:, None] + torch.arange(st["per"], device=DEV)], dim=1)
            seen = torch.cat([seen, _bits(st)], dim=1)
        k, v = (_rows(st, n, seq[:, None], tok) for n in ("k", "v"))
        s = torch.einsum("nhgd,nthd->nhgt", q, k) / math.sqrt(d)
        o, lse = _softmax_sum(s, seen[:, None, None, :], v, "nhgt,nthd->nhgd")
    else:
        # queries of one sequence side by side in a padded batch
        counts = torch.bincount(seq, minlength=st["n_seq"])
        place = torch.arange(seq.numel(), device=DEV) - (counts.cumsum(0) - counts)[seq]
        every = torch.arange(st["n_seq"], device=DEV)[:, None]
        cap = st["k"].shape[1]
        at = torch.arange(cap, device=DEV)
        k, v = (_rows(st, n, every, at[None, :]) for n in ("k", "v"))
        pad = torch.zeros(st["n_seq"], st["per"], *q.shape[1:], device=DEV)
        pad[seq, place] = q
        see = torch.zeros(st["n_seq"], st["per"], cap, dtype=torch.bool, device=DEV)
        row = at <= st["q_pos"][:, None]
        if st["tree"]:
            j = at[None, :] - st["start"].long()[seq][:, None]
            row = row | ((j >= 0) & (j < st["per"]) & torch.gather(_bits(st), 1, j.clamp(0, st["per"] - 1)))
        see[seq, place] = row
        s = torch.einsum("bnhgd,bthd->bnhgt", pad, k) / math.sqrt(d)
        o, lse = _softmax_sum(s, see[:, :, None, None, :], v, "bnhgt,bthd->bnhgd")
        o, lse = o[seq, place], lse[seq, place]
    return {"out": o.reshape(st["q"].shape).to(torch.bfloat16), "lse": lse.reshape(st["q"].shape[:2])}


# ---------------------------------------------------------------------- work

def work(case):
    c = case
    if c["op"] == "rope":
        elements = (c["n"] * c["heads"] + c["keys"]) * c["d"]
        return {"bytes": 4 * elements + 4 * (c["n"] + c["keys"]), "flops": 6 * elements * c["rot"] / c["d"] / 2}
    cell = c["d"] * (1 if c["fp8"] else 2) + (4 if c["fp8"] else 0)  # one head's key or value of a token
    if c["op"] == "append":
        rows = 2 * c["n_seq"] * c["count"] * c["h_kv"]
        return {"bytes": rows * (2 * c["d"] + cell), "flops": rows * c["d"] * 4}
    if c["op"] == "read":
        rows = 2 * c["n"] * c["sel"] * c["h_kv"]
        return {"bytes": rows * (2 * c["d"] + cell) + 4 * c["n"] * c["sel"], "flops": rows * c["d"]}
    nodes, lens = _nodes(c), _lens(c)
    drafts = c["per"] if c["tree"] else 0
    heads = c["h_kv"] * c["group"]
    # each sequence's tokens once (its queries may all select the same), the queries, their lists and the outputs
    tokens = sum(min(n, c["sel"]) if c["sel"] else n for n in lens) + c["n_seq"] * drafts
    pairs = sum(t * ((min(n, c["sel"]) if c["sel"] else n) + (drafts + 1) // 2) for t, n in zip(nodes, lens))
    return {"bytes": 2 * tokens * c["h_kv"] * cell + sum(nodes) * (heads * (4 * c["d"] + 4) + 4 * c["sel"]),
            "flops": 4 * pairs * heads * c["d"]}


# --------------------------------------------------------------------- exact

def exact(case, seed):
    """The operators' definitions in 64 bits."""
    st = prepare(case, seed)
    if st["op"] == "rope":
        return [_exact_rows(st, x.double(), pos.long(), st["first"]) for x, pos, _ in st["rows"]]
    if st["op"] == "append":
        return _exact_append(st)
    if st["op"] == "read":
        r = []
        for n in ("k", "v"):
            x = st[n].double() * (st[n + "_scale"].double()[..., None] if st["fp8"] else 1.0)
            r.append(torch.stack([x[s, t.long()] for s, t in zip(st["seq"].tolist(), st["tok"])]))
        return tuple(r)
    return _exact_attend(st)


def _exact_rows(st, x, pos, first):
    """Each pair (a, b) as a complex number times amplitude * e^(i angle)."""
    rot = 2 * st["freq"].numel()
    z = torch.polar(torch.full((), st["amplitude"], dtype=torch.float64, device=DEV).expand(pos.shape + (rot // 2,)).contiguous(),
                    pos.double()[..., None] * st["freq"])[..., None, :]
    i = torch.arange(rot // 2, device=DEV)
    ia, ib = (first + i, first + rot // 2 + i) if st["layout"] == "half" else (first + 2 * i, first + 2 * i + 1)
    w = torch.complex(x[..., ia], x[..., ib]) * z
    y = x.clone()
    y[..., ia], y[..., ib] = w.real, w.imag
    return y


def _exact_append(st):
    n = st["count"]
    for s, p in enumerate(st["pos"].tolist()):
        k, v = st["new_k"][s].double(), st["new_v"][s].double()
        if st["rot"]:
            k = _exact_rows(st, k, torch.arange(p, p + n, device=DEV), 0)
        for name, x in (("k", k), ("v", v)):
            if st["fp8"]:
                top = x.abs().amax(-1)
                scale = torch.where(top > 0, top / E4M3_MAX, 1.0)
                st[name + "_scale"][s, p:p + n] = scale.float()
                # to the nearest e4m3 value: 3 bits behind the leading one, steps of 2^-9 below 2^-6
                y = x / scale[..., None]
                step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
                st[name][s, p:p + n] = (torch.round(y / step) * step).float().to(torch.float8_e4m3fn)
            else:
                st[name][s, p:p + n] = x.to(torch.bfloat16)
        st["seq_len"][s] = p + n
    r = _written(st)
    return {n: x if n == "seq_len" else x.double() for n, x in r.items()}


def _exact_attend(st):
    """Query by query, over the tokens that it sees."""
    outs, lses = [], []
    seqs, ends = st["q_seq"].tolist(), st["q_pos"].tolist()
    if st["sel"]:
        # only the rows that some query of the sequence lists are needed, and each query's are few
        def rows(n, s, t):
            x = st[n][s].view(torch.uint8)[t].view(torch.float8_e4m3fn).double() if st["fp8"] else st[n][s][t].double()
            return x * st[n + "_scale"][s][t].double()[..., None] if st["fp8"] else x
    else:
        whole = {}

        def rows(n, s, t):
            if (n, s) not in whole:
                whole.clear() if len(whole) > 1 else None
                x = st[n][s].double()
                whole[n, s] = x * st[n + "_scale"][s].double()[..., None] if st["fp8"] else x
            return whole[n, s][t]
    for i, (s, p) in enumerate(zip(seqs, ends)):
        if st["sel"]:
            t = st["topk"][i].long()
            t = t[t >= 0]
        else:
            t = torch.arange(p + 1, device=DEV)
        if st["tree"]:
            words = st["mask"][i].tolist()
            mine = [j for j in range(st["per"]) if words[j // 32] >> (j % 32) & 1]
            t = torch.cat([t, torch.tensor(mine, dtype=torch.long, device=DEV) + st["start"][s].long()])
        k, v = rows("k", s, t), rows("v", s, t)
        q = st["q"][i].double().view(st["h_kv"], st["group"], st["d"])
        a = torch.matmul(q, k.permute(1, 2, 0)) * st["d"] ** -0.5
        outs.append(torch.matmul(torch.softmax(a, -1), v.transpose(0, 1)).reshape(-1, st["d"]))
        lses.append(torch.logsumexp(a, -1).reshape(-1))
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}
