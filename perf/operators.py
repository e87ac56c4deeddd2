"""Cases of the attention operators: query/key norms with the position rotation, attention with a sliding window
and visible first tokens (forward and backward), and attention of one new token over a paged cache.

`run` computes a case in plain torch operations, or, where `own` is true, through the library's entry points.
"""
import math
import random

import numpy as np
import torch

own = False

DT = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
EPS = 1e-6


# ---- cases -------------------------------------------------------------------------------------------------------

def listed():
    return [
        # one sequence's new token on its way into the cache: latency
        {"name": "append one token", "op": "append", "tokens": 1, "heads": 20, "kv_heads": 5, "dim": 128, "rot": 128,
         "interleaved": False, "dtype": "bfloat16", "page": 16, "far": 30000},
        # a prompt's projection rows
        {"name": "norm rope prompt", "op": "rope", "tokens": 8192, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 128,
         "interleaved": False, "dtype": "bfloat16", "far": 8192},
        # the small ternary GPT (4 heads of 32), an odd number of tokens, half of each head rotated, float32 throughout
        {"name": "norm rope backward odd", "op": "rope_backward", "tokens": 1025, "heads": 4, "kv_heads": 4, "dim": 32,
         "rot": 16, "interleaved": True, "dtype": "float32", "far": 2000},
        # a training step's rows
        {"name": "norm rope backward train", "op": "rope_backward", "tokens": 4096, "heads": 32, "kv_heads": 8,
         "dim": 128, "rot": 128, "interleaved": False, "dtype": "bfloat16", "far": 4096},
        # the small ternary GPT: 8 sequences of up to 256 tokens, 4 heads of 32
        {"name": "attention small ragged", "op": "attention", "seqs": 8, "longest": 256, "ragged": True, "extra": 0,
         "heads": 4, "kv_heads": 4, "dim": 32, "window": 0, "sinks": 0, "dtype": "float16", "lens": 1},
        # one long prompt, every earlier token visible
        {"name": "attention prompt", "op": "attention", "seqs": 1, "longest": 8192, "ragged": False, "extra": 0,
         "heads": 32, "kv_heads": 8, "dim": 128, "window": 0, "sinks": 0, "dtype": "bfloat16", "lens": 2},
        # several prompts behind cached tokens, a window and four first tokens
        {"name": "attention window sinks", "op": "attention", "seqs": 4, "longest": 4001, "ragged": True, "extra": 500,
         "heads": 20, "kv_heads": 5, "dim": 64, "window": 1024, "sinks": 4, "dtype": "bfloat16", "lens": 3},
        # odd everything: ragged, a head size between tiles, a window that ends inside tiles
        {"name": "attention backward odd", "op": "attention_backward", "seqs": 5, "longest": 777, "ragged": True,
         "extra": 0, "heads": 6, "kv_heads": 2, "dim": 80, "window": 200, "sinks": 3, "dtype": "float16", "lens": 4},
        # a training step
        {"name": "attention backward train", "op": "attention_backward", "seqs": 2, "longest": 4096, "ragged": False,
         "extra": 0, "heads": 20, "kv_heads": 5, "dim": 128, "window": 0, "sinks": 0, "dtype": "bfloat16", "lens": 5},
        # one sequence's new token: latency
        {"name": "paged one sequence", "op": "paged", "seqs": 1, "longest": 301, "ragged": False, "heads": 20,
         "kv_heads": 5, "dim": 128, "page": 16, "window": 0, "sinks": 0, "dtype": "bfloat16", "out": "float32",
         "lens": 6},
        # a serving batch of ragged lengths
        {"name": "paged batch", "op": "paged", "seqs": 64, "longest": 8192, "ragged": True, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 16, "window": 0, "sinks": 0, "dtype": "bfloat16", "out": "float32", "lens": 7},
        # two very long sequences, an odd last page
        {"name": "paged long", "op": "paged", "seqs": 2, "longest": 131071, "ragged": False, "heads": 20, "kv_heads": 5,
         "dim": 64, "page": 64, "window": 0, "sinks": 0, "dtype": "float16", "out": "float16", "lens": 8},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "rope", "rope_backward", "attention", "attention", "attention_backward",
                     "attention_backward", "paged", "paged"])
    kv_heads = rng.choice([1, 2, 3, 4, 5, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 8])
    dim = rng.choice([32, 64, 80, 96, 128])
    dtype = rng.choice(["float16", "bfloat16"])
    c = {"op": op, "heads": heads, "kv_heads": kv_heads, "dim": dim, "dtype": dtype}
    if op in ("append", "rope", "rope_backward"):
        most = 256 if op == "append" else min(8192, (8192 * 48 * 128) // ((heads + 2 * kv_heads) * dim))
        if op != "append":
            c["dtype"] = rng.choice(["float16", "bfloat16", "float32"])
        c.update(tokens=_log_int(rng, 1, most), rot=rng.choice([dim, dim, dim // 2]), interleaved=rng.random() < 0.4,
                 far=_log_int(rng, 1000, 100000))
        if op == "append":
            c["page"] = rng.choice([1, 16, 24, 64])
        return c
    # a query that sees one key only has no gradient through its softmax: the backward cases see several
    least = 8 if op == "attention_backward" else 1
    window = rng.choice([0, 0, 1]) * _log_int(rng, least, 2000)
    c.update(window=window, sinks=rng.choice([0, 1, 4, 70]) if window else 0, lens=rng.randrange(1 << 20))
    if op == "paged":
        longest = _log_int(rng, 1, 60000)
        seqs = _log_int(rng, 1, max(1, min(128, 500000 // longest)))
        c.update(seqs=seqs, longest=longest, ragged=rng.random() < 0.7, page=rng.choice([1, 16, 24, 64, 128]),
                 out=rng.choice(["float32", dtype]))
        return c
    longest = _log_int(rng, least, 3500)
    extra = rng.choice([0, 0, rng.randrange(1, 700)])
    pairs = longest * (longest + extra) * heads
    c.update(seqs=_log_int(rng, 1, max(1, min(16, 400_000_000 // pairs))), longest=longest, ragged=rng.random() < 0.7,
             extra=extra)
    return c


# ---- inputs ------------------------------------------------------------------------------------------------------

def _lengths(c):
    """Tokens of each sequence, by the case alone."""
    r = random.Random(c["lens"])
    n, top = c["seqs"], c["longest"]
    got = [r.randint(max(1, top // 8), top) if c["ragged"] else top for _ in range(n)]
    got[r.randrange(n)] = top
    return got


def _table(positions, rot):
    """cos | sin of position * 10000^(-2i/rot), float32, the angles in 64 bits."""
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * (10000.0 ** (-2.0 * i / rot))
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def _cu(lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    h, hk, d, t = c["heads"], c["kv_heads"], c["dim"], DT[c["dtype"]]

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)

    s = {"case": c}
    if c["op"] in ("append", "rope", "rope_backward"):
        m = c["tokens"]
        scale = torch.rand(m, 1, generator=g, device="cuda") * 2 + 0.1
        s.update(qkv=normal(m, (h + 2 * hk) * d) * scale,
                 gq=1 + 0.2 * normal(d), gk=1 + 0.2 * normal(d), table=_table(c["far"], c["rot"]),
                 pos=torch.randint(0, c["far"], (m,), generator=g, device="cuda", dtype=torch.int32))
        if c["op"] == "append":
            pages = 2 * (-(-m // c["page"])) + 3
            s["kcache"] = normal(pages, hk, c["page"], d, dtype=t)
            s["vcache"] = normal(pages, hk, c["page"], d, dtype=t)
            s["slots"] = torch.randperm(pages * c["page"], generator=g, device="cuda")[:m].contiguous()
        if c["op"] == "rope_backward":
            s.update(dq=normal(m, h, d, dtype=t), dk=normal(m, hk, d, dtype=t), dv=normal(m, hk, d, dtype=t))
        return s
    lens = _lengths(c)
    if c["op"] == "paged":
        width = -(-max(lens) // c["page"])
        need = [-(-n // c["page"]) for n in lens]
        total = sum(need) + 5
        at = np.random.RandomState(seed % (1 << 31)).permutation(total)
        pages = np.zeros((len(lens), width), np.int32)
        used = 0
        for b, n in enumerate(need):
            pages[b, :n] = at[used:used + n]
            used += n
        s.update(q=normal(len(lens), h, d, dtype=t), kcache=normal(total, hk, c["page"], d, dtype=t),
                 vcache=normal(total, hk, c["page"], d, dtype=t), pages=torch.from_numpy(pages).cuda(),
                 lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                 ws=torch.zeros(16 << 20, dtype=torch.uint8, device="cuda"))
        return s
    klens = [n + c["extra"] for n in lens]
    s.update(q=normal(sum(lens), h, d, dtype=t), k=normal(sum(klens), hk, d, dtype=t),
             v=normal(sum(klens), hk, d, dtype=t), cu_q=_cu(lens), cu_k=_cu(klens), max_q=max(lens), max_k=max(klens))
    if c["op"] == "attention_backward":
        s["out"], s["lse"] = _attention(s)
        s["dout"] = normal(sum(lens), h, d, dtype=t)
    return s


# ---- plain forms -------------------------------------------------------------------------------------------------

def _split(qkv, c):
    h, hk, d = c["heads"], c["kv_heads"], c["dim"]
    m = qkv.shape[0]
    q, k, v = qkv.split([h * d, hk * d, hk * d], 1)
    return q.reshape(m, h, d), k.reshape(m, hk, d), v.reshape(m, hk, d)


def _pairs(x, c):
    r = c["rot"]
    if c["interleaved"]:
        return x[..., 0:r:2], x[..., 1:r:2]
    return x[..., :r // 2], x[..., r // 2:r]


def _join(a, b, rest, c):
    both = torch.stack([a, b], -1).flatten(-2) if c["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([both, rest], -1)


def _cos_sin(s):
    t = s["table"][s["pos"].long()][:, None]
    half = t.shape[-1] // 2
    return t[..., :half], t[..., half:]


def _norm_rope(s, x, g):
    y = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * g
    a, b = _pairs(y, s["case"])
    cos, sin = _cos_sin(s)
    return _join(a * cos - b * sin, a * sin + b * cos, y[..., s["case"]["rot"]:], s["case"])


def _norm_rope_grad(s, x, g, dz):
    a, b = _pairs(dz, s["case"])
    cos, sin = _cos_sin(s)
    dy = _join(a * cos + b * sin, b * cos - a * sin, dz[..., s["case"]["rot"]:], s["case"])
    r = 1 / (x.square().mean(-1, keepdim=True) + EPS).sqrt()
    xr = x * r
    gy = g * dy
    return r * (gy - xr * (xr * gy).mean(-1, keepdim=True)), (dy * xr).sum((0, 1))


def _padded(x, cu, longest):
    """[tokens, heads, dim] -> [sequences, heads, longest, dim] in float32, and each row's index."""
    at = cu[:-1, None].long() + torch.arange(longest, device=x.device)
    return x[at.clamp(max=x.shape[0] - 1)].float().transpose(1, 2)


def _packed(x, cu, tokens):
    """[sequences, heads, longest, ...] -> [tokens, heads, ...]."""
    row = torch.arange(tokens, device=x.device)
    b = torch.searchsorted(cu[1:].long(), row, right=True)
    return x[b, :, row - cu[b]]


def _visible(s):
    c = s["case"]
    i = torch.arange(s["max_q"], device="cuda")[:, None]
    j = torch.arange(s["max_k"], device="cuda")
    nq, nk = s["cu_q"].diff()[:, None, None], s["cu_k"].diff()[:, None, None]
    p = i + nk - nq
    see = (i < nq) & (j < nk) & (j <= p)
    if c["window"]:
        see &= (j > p - c["window"]) | (j < c["sinks"])
    return see[:, None, None]


def _scores(s):
    c = s["case"]
    q, k = _padded(s["q"], s["cu_q"], s["max_q"]), _padded(s["k"], s["cu_k"], s["max_k"])
    q = q.unflatten(1, (c["kv_heads"], -1))
    x = q @ k[:, :, None].transpose(-1, -2)
    return q, k, x.mul_(1 / math.sqrt(c["dim"])).masked_fill_(~_visible(s), -math.inf)


def _attention(s):
    c = s["case"]
    _, _, x = _scores(s)
    top = x.amax(-1, keepdim=True).clamp_(min=-1e30)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    v = _padded(s["v"], s["cu_k"], s["max_k"])
    o = (p @ v[:, :, None]) / total.clamp(min=1e-30)
    lse = top + total.log()
    tokens = s["q"].shape[0]
    out = _packed(o.flatten(1, 2), s["cu_q"], tokens).to(s["q"].dtype)
    return out, _packed(lse.flatten(1, 2)[..., 0], s["cu_q"], tokens).transpose(0, 1).contiguous()


def _attention_grad(s):
    c = s["case"]
    t, hk = s["q"].dtype, c["kv_heads"]
    q, k, x = _scores(s)
    scale = 1 / math.sqrt(c["dim"])
    nq = s["max_q"]
    lse = _padded(s["lse"].transpose(0, 1)[..., None], s["cu_q"], nq).unflatten(1, (hk, -1))
    do = _padded(s["dout"], s["cu_q"], nq).unflatten(1, (hk, -1))
    o = _padded(s["out"], s["cu_q"], nq).unflatten(1, (hk, -1))
    v = _padded(s["v"], s["cu_k"], s["max_k"])
    p = x.sub_(lse.clamp(min=-1e30)).exp_()
    dv = (p.transpose(-1, -2) @ do).sum(2)
    ds = do @ v[:, :, None].transpose(-1, -2)
    ds = ds.sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    dq = (ds @ k[:, :, None]).flatten(1, 2)
    dk = (ds.transpose(-1, -2) @ q).sum(2)
    return (_packed(dq, s["cu_q"], s["q"].shape[0]).to(t), _packed(dk, s["cu_k"], s["k"].shape[0]).to(t),
            _packed(dv, s["cu_k"], s["k"].shape[0]).to(t))


def _paged(s):
    c = s["case"]
    n, width = s["pages"].shape
    hk, d = c["kv_heads"], c["dim"]

    def rows(cache):
        x = cache[s["pages"].long()]                                 # [sequences, width, kv_heads, page, dim]
        return x.transpose(1, 2).reshape(n, hk, width * c["page"], d).float()

    q = s["q"].float().reshape(n, hk, -1, d)
    x = (q @ rows(s["kcache"]).transpose(-1, -2)) * (1 / math.sqrt(d))
    j = torch.arange(width * c["page"], device="cuda")
    last = s["lens"][:, None, None, None] - 1
    see = j <= last
    if c["window"]:
        see = see & ((j > last - c["window"]) | (j < c["sinks"]))
    x = x.masked_fill_(~see, -math.inf)
    p = (x - x.amax(-1, keepdim=True).clamp(min=-1e30)).exp()
    o = (p @ rows(s["vcache"])) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return o.reshape(n, c["heads"], d).to(DT[c["out"]])


def _plain(s):
    c = s["case"]
    t = DT[c["dtype"]]
    if c["op"] in ("append", "rope", "rope_backward"):
        q, k, v = _split(s["qkv"], c)
    if c["op"] == "append":
        slot, page = s["slots"], c["page"]
        s["kcache"][slot // page, :, slot % page] = _norm_rope(s, k, s["gk"]).to(t)
        s["vcache"][slot // page, :, slot % page] = v.to(t)
        return _norm_rope(s, q, s["gq"]).to(t), s["kcache"], s["vcache"]
    if c["op"] == "rope":
        return _norm_rope(s, q, s["gq"]).to(t), _norm_rope(s, k, s["gk"]).to(t), v.to(t)
    if c["op"] == "rope_backward":
        dq, dgq = _norm_rope_grad(s, q, s["gq"], s["dq"].float())
        dk, dgk = _norm_rope_grad(s, k, s["gk"], s["dk"].float())
        return torch.cat([dq.flatten(1), dk.flatten(1), s["dv"].float().flatten(1)], 1), dgq, dgk
    if c["op"] == "attention":
        return _attention(s)
    if c["op"] == "attention_backward":
        return _attention_grad(s)
    return _paged(s)


# ---- the library -------------------------------------------------------------------------------------------------

def _library(s):
    import int8_row_absmax_b200 as bl
    c = s["case"]
    h, hk, d, t = c["heads"], c["kv_heads"], c["dim"], DT[c["dtype"]]
    if c["op"] == "append":
        q = bl.qk_norm_rope_append(s["qkv"], h, hk, d, s["pos"], s["table"], s["gq"], s["gk"], s["kcache"], s["vcache"],
                                   s["slots"], eps=EPS, interleaved=c["interleaved"])
        return q, s["kcache"], s["vcache"]
    if c["op"] == "rope":
        return bl.qk_norm_rope(s["qkv"], h, hk, d, s["pos"], s["table"], s["gq"], s["gk"], eps=EPS, dtype=t,
                               interleaved=c["interleaved"])
    if c["op"] == "rope_backward":
        return bl.qk_norm_rope_backward(s["dq"], s["dk"], s["dv"], s["qkv"], h, hk, d, s["pos"], s["table"], s["gq"],
                                        s["gk"], eps=EPS, interleaved=c["interleaved"])
    if c["op"] == "attention":
        return bl.attention(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["max_q"], window=c["window"],
                            sinks=c["sinks"])
    if c["op"] == "attention_backward":
        return bl.attention_backward(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"], s["cu_q"], s["cu_k"],
                                     s["max_q"], s["max_k"], window=c["window"], sinks=c["sinks"])
    return bl.paged_attention(s["q"], s["kcache"], s["vcache"], s["pages"], s["lens"], window=c["window"],
                              sinks=c["sinks"], out_dtype=DT[c["out"]], ws=s["ws"])


def run(state):
    return _library(state) if own else _plain(state)


# ---- 64 bits -----------------------------------------------------------------------------------------------------

def _turn(y, s, back):
    """The rotation (or its transpose) of rows y [tokens, heads, dim] in 64 bits, pair by pair of columns."""
    c = s["case"]
    half = c["rot"] // 2
    t = s["table"].double()[s["pos"].long()]
    i = torch.arange(half, device="cuda")
    a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
    z = y.clone()
    cos, sin = t[:, None, :half], t[:, None, half:] * (-1 if back else 1)
    z[..., a] = y[..., a] * cos - y[..., b] * sin
    z[..., b] = y[..., b] * cos + y[..., a] * sin
    return z


def _exact_rows(s):
    c = s["case"]
    x = s["qkv"].double().reshape(c["tokens"], -1, c["dim"])
    h, hk = c["heads"], c["kv_heads"]
    parts = {"q": (x[:, :h], s["gq"].double()), "k": (x[:, h:h + hk], s["gk"].double())}
    done = {}
    for name, (u, g) in parts.items():
        n = (u.pow(2).sum(-1, keepdim=True) / c["dim"] + EPS).pow(-0.5)
        if c["op"] != "rope_backward":
            done[name] = _turn(u * n * g, s, False)
            continue
        e = _turn(s["d" + name].double(), s, True)
        w = (u * g * e).sum(-1, keepdim=True) / c["dim"]
        done[name] = (n * g * e - u * n.pow(3) * w, (e * u * n).sum(1).sum(0))
    return done, x[:, h + hk:]


def _seen(p, nk, c):
    """Keys that a query at each position p sees: truth values [len(p), nk]."""
    j = torch.arange(nk, device="cuda")[None]
    p = p[:, None]
    see = j <= p
    return see & ((p - j < c["window"]) | (j < c["sinks"])) if c["window"] else see


def exact(case, seed):
    c = dict(case)
    s = prepare(case, seed)
    if c["op"] in ("append", "rope", "rope_backward"):
        done, v = _exact_rows(s)
        if c["op"] == "rope":
            return done["q"], done["k"], v
        if c["op"] == "rope_backward":
            rows = torch.cat([done["q"][0], done["k"][0], s["dv"].double()], 1)
            return rows.flatten(1), done["q"][1], done["k"][1]
        kc, vc = s["kcache"].double(), s["vcache"].double()
        for m, slot in enumerate(s["slots"].tolist()):
            kc[slot // c["page"], :, slot % c["page"]] = done["k"][m]
            vc[slot // c["page"], :, slot % c["page"]] = v[m]
        return done["q"], kc, vc
    scale = 1 / math.sqrt(c["dim"])
    group = c["heads"] // c["kv_heads"]
    if c["op"] == "paged":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        for b, n in enumerate(s["lens"].tolist()):
            at = s["pages"][b, :-(-n // c["page"])].long()
            for u in range(c["kv_heads"]):
                k = s["kcache"][at, u].reshape(-1, c["dim"])[:n].double()
                v = s["vcache"][at, u].reshape(-1, c["dim"])[:n].double()
                see = _seen(torch.tensor([n - 1], device="cuda"), n, c)[0]
                k, v = k[see], v[see]
                heads = slice(u * group, (u + 1) * group)
                out[b, heads] = torch.softmax(s["q"][b, heads].double() @ k.T * scale, -1) @ v
        return out
    cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
    back = c["op"] == "attention_backward"
    like = torch.zeros_like
    f8 = dict(dtype=torch.float64)
    out, lse = like(s["q"], **f8), torch.zeros(c["heads"], s["q"].shape[0], device="cuda", **f8)
    dq, dk, dv = like(s["q"], **f8), like(s["k"], **f8), like(s["v"], **f8)
    for b in range(c["seqs"]):
        iq, ik = slice(cq[b], cq[b + 1]), slice(ck[b], ck[b + 1])
        nq, nk = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
        see = _seen(torch.arange(nq, device="cuda") + nk - nq, nk, c)
        for h in range(c["heads"]):
            u = h // group
            q, k, v = s["q"][iq, h].double(), s["k"][ik, u].double(), s["v"][ik, u].double()
            x = torch.where(see, q @ k.T * scale, torch.tensor(-math.inf, device="cuda", **f8))
            if not back:
                lse[h, iq] = torch.logsumexp(x, -1)
                out[iq, h] = torch.softmax(x, -1).nan_to_num() @ v
                continue
            p = torch.where(see, torch.exp(x - s["lse"][h, iq].double()[:, None]), 0.0)
            do = s["dout"][iq, h].double()
            dx = p * (do @ v.T - (do * s["out"][iq, h].double()).sum(-1, keepdim=True)) * scale
            dq[iq, h] = dx @ k
            dk[ik, u] += dx.T @ q
            dv[ik, u] += p.T @ do
    return (dq, dk, dv) if back else (out, lse)


# ---- what a case cannot do without -------------------------------------------------------------------------------

def _pair_count(nq, nk, c):
    p = np.arange(nq, dtype=np.int64) + nk - nq
    n = np.maximum(p + 1, 0)
    if c["window"]:
        first = np.maximum(p - c["window"] + 1, 0)                   # first key of the window
        n = np.maximum(p + 1 - first, 0) + np.minimum(np.minimum(first, c["sinks"]), np.maximum(p + 1, 0))
    return int(n.sum())


def work(case):
    c = case
    h, hk, d = c["heads"], c["kv_heads"], c["dim"]
    e = torch.finfo(DT[c["dtype"]]).bits // 8
    if c["op"] in ("append", "rope", "rope_backward"):
        m, wide = c["tokens"], (h + 2 * hk) * d
        rows = min(m, c["far"]) * c["rot"] * 4 + m * 4 + 2 * d * 4
        if c["op"] == "rope_backward":
            return {"bytes": m * wide * (4 + e + 4) - m * hk * d * 4 + rows + 2 * d * 4, "flops": 20 * m * wide}
        return {"bytes": m * wide * (4 + e) + rows + (8 * m if c["op"] == "append" else 0), "flops": 8 * m * wide}
    lens = _lengths(c)
    if c["op"] == "paged":
        seen = sum(_pair_count(1, n, c) for n in lens)
        out = torch.finfo(DT[c["out"]]).bits // 8
        return {"bytes": 2 * seen * hk * d * e + len(lens) * h * d * (e + out) + 4 * sum(-(-n // c["page"]) for n in lens),
                "flops": 4 * seen * h * d}
    nq, nk = sum(lens), sum(lens) + c["extra"] * len(lens)
    pairs = sum(_pair_count(n, n + c["extra"], c) for n in lens)
    if c["op"] == "attention":
        return {"bytes": (2 * nq * h + 2 * nk * hk) * d * e + nq * h * 4, "flops": 4 * pairs * h * d}
    return {"bytes": (4 * nq * h + 4 * nk * hk) * d * e + nq * h * 4, "flops": 10 * pairs * h * d}
