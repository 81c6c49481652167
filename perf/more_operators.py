"""The measured cases of the decoder operators: root-mean-square norm with the residual's addition (forward, training,
and with an output in 8 bits), the token cache in 8 bits (quantised as it is written, and read back), and attention of
drafted tokens, a tree of them among others, over that cache.

``run`` computes an operator in its plain form (elementary torch operations, rounded once at the end) while ``own`` is
False and calls the library's entry points when it is True; ``exact`` gives the same outputs from the definitions in
64 bits.

The cache is paged, 64 tokens a page: k [pages, Hk, 64, Dp] and v [pages, Hk, Dp, 64] codes (int8 or e4m3, Dp the next
multiple of 16 from D, zeros behind D), k_scale and v_scale [pages, Hk, 64] fp32; table [B, W] names a sequence's pages.
A row of D values x has scale = max(max |x| / 127 (or 448), 2^-126) in fp32, and its codes are the nearest to x / scale.
"""
import math

import torch

own = False

_T = {"f32": torch.float32, "bf16": torch.bfloat16}
_CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
_MOST = {"int8": 127.0, "e4m3": 448.0}
_TINY = 2.0 ** -126
_EPS = 1e-6
_PAGE = 64


# ------------------------------------------------------------------ cases

def listed():
    return [
        # sixteen planning tokens before a projection in 8 bits: latency
        dict(name="norm_few_codes", op="norm", rows=16, heads=1, c=256, dtype="bf16", residual=True, packed=False,
             codes="e4m3", block=128, train=False),
        # a large batch of wide tokens, residual added, 8 bits out with a scale for each 128 channels
        dict(name="norm_wide_codes", op="norm", rows=8192, heads=1, c=4096, dtype="bf16", residual=True, packed=False,
             codes="e4m3", block=128, train=False),
        # queries and keys of the 200 x 200 BEV cells normalised head by head, out of a packed projection
        dict(name="norm_heads", op="norm", rows=40000, heads=8, c=32, dtype="bf16", residual=False, packed=True,
             codes="", block=0, train=False),
        # training: the image tokens of four six-camera rigs (32 x 88), 256 channels
        dict(name="norm_train", op="norm", rows=67584, heads=1, c=256, dtype="bf16", residual=True, packed=False,
             codes="", block=0, train=True),
        # training at an odd width and count
        dict(name="norm_odd_train", op="norm", rows=10007, heads=1, c=1001, dtype="f32", residual=True, packed=False,
             codes="", block=0, train=True),
        # a step of serving: one new token of each of 64 sequences goes into the cache, and comes back
        dict(name="cache_tokens", op="cache", b=64, t=1, longest=4096, hk=8, d=128, dtype="bf16", codes="e4m3",
             ragged=False),
        # a frame of a 100 x 100 map for each of four rigs, ragged, put behind what is there
        dict(name="cache_frames", op="cache", b=4, t=10000, longest=2500, hk=8, d=32, dtype="bf16", codes="int8",
             ragged=True),
        # one ego token looks at the memory of four frames of 900 queries: latency
        dict(name="attn_ego_token", op="attn", b=1, t=1, longest=3600, hq=8, hk=8, d=32, dtype="bf16", codes="int8",
             form="memory", cap=0.0),
        # serving: 32 sequences of ragged length, one token each, grouped heads
        dict(name="attn_tokens", op="attn", b=32, t=1, longest=8192, hq=32, hk=8, d=128, dtype="bf16", codes="e4m3",
             form="chain", cap=0.0),
        # a tree of 15 drafted waypoints over five maps of 200 x 200 cells
        dict(name="attn_tree_cells", op="attn", b=1, t=15, longest=200000, hq=8, hk=2, d=64, dtype="bf16",
             codes="int8", form="tree", cap=0.0),
        # trees of 64 drafted waypoints for 16 scenes, fp32, capped scores
        dict(name="attn_trees", op="attn", b=16, t=64, longest=4096, hq=16, hk=4, d=128, dtype="f32", codes="e4m3",
             form="tree", cap=30.0),
        # a chunk of a prompt behind what the cache holds
        dict(name="attn_prompt", op="attn", b=2, t=1000, longest=6000, hq=16, hk=4, d=128, dtype="bf16", codes="int8",
             form="chain", cap=0.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["norm", "cache", "attn", "attn"])
    dtype = rng.choice(["f32", "bf16"])
    if op == "norm":
        kind = rng.choice(["plain", "codes", "train"])
        heads = rng.choice([1, 1, 1, 4, 8])
        c = _log_int(rng, 16, 256 if heads > 1 else 8192)
        if rng.random() < 0.5:
            c = max(32, c // 32 * 32)
        block = 0
        if kind == "codes":     # codes are values next to a border: their type carries the comparison
            dtype, block = "bf16", rng.choice([0, 32, 64, 128])
        most = (8 if dtype == "f32" else 16) * 1000 * 1000 // (c * heads)
        return dict(op="norm", rows=_log_int(rng, 1, min(most, 100000)), heads=heads, c=c, dtype=dtype,
                    residual=rng.random() < 0.6, packed=heads > 1 and rng.random() < 0.5,
                    codes=rng.choice(["int8", "e4m3"]) if kind == "codes" else "", block=block, train=kind == "train")
    d = rng.choice([16, 32, 40, 64, 80, 96, 128, 128])
    codes = rng.choice(["int8", "e4m3"])
    if op == "cache":
        hk = rng.choice([1, 2, 3, 4, 8])
        b = _log_int(rng, 1, 64)
        return dict(op="cache", b=b, t=_log_int(rng, 1, max(1, 5000 * 1000 // (b * hk * d))),
                    longest=_log_int(rng, 1, 5000), hk=hk, d=d, dtype=dtype, codes=codes, ragged=rng.random() < 0.5)
    hk = rng.choice([1, 2, 4, 8])
    hq = hk * rng.choice([1, 1, 2, 4, 8])
    form = rng.choice(["chain", "chain", "tree", "tree", "memory"])
    b = _log_int(rng, 1, 32)
    one = form != "tree" and rng.random() < 0.4
    t = 1 if one else _log_int(rng, 2, {"chain": 500, "tree": 130, "memory": 900}[form])
    most = min(200000, 150 * 1000 * 1000 // (b * hk * d), 10 ** 10 // (b * hq * t * d))
    return dict(op="attn", b=b, t=t, longest=_log_int(rng, 1, max(1, most)), hq=hq, hk=hk, d=d, dtype=dtype,
                codes=codes, form=form, cap=rng.choice([0.0, 0.0, 20.0, 50.0]))


def _starts(case):
    """Tokens of each sequence that the cache holds: from the longest down to half of it."""
    n = case["longest"]
    return [n - i * n // (2 * case["b"]) for i in range(case["b"])]


def _counts(case):
    """New tokens of each sequence (a padded batch where ragged)."""
    t = case["t"]
    return [t - (i * t // (2 * case["b"]) if case["ragged"] else 0) for i in range(case["b"])]


# ------------------------------------------------------------------ work

def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "norm":
        n = case["rows"] * case["heads"] * case["c"]
        ins, outs = (2, 1) if case["residual"] else (1, 0)      # x (and the residual); their sum
        if case["train"]:       # gy (and the sum's gradient) read; y and gx written
            moved = (ins + outs + 2 + (2 if case["residual"] else 1)) * n * es + 8 * case["c"]
            return {"bytes": moved, "flops": 14 * n}
        if case["codes"]:
            blocks = -(-case["c"] // case["block"]) if case["block"] else 1
            return {"bytes": (ins + outs) * n * es + n + 4 * blocks * case["rows"] * case["heads"] + 4 * case["c"],
                    "flops": 6 * n}
        return {"bytes": (ins + outs + 1) * n * es + 4 * case["c"], "flops": 5 * n}
    if case["op"] == "cache":
        rows = sum(_counts(case)) * case["hk"] * 2              # read, written as codes, read back, written
        back = case["b"] * case["t"] * case["hk"] * 2 * case["d"] * es
        return {"bytes": rows * (case["d"] * (es + 2) + 8) + back, "flops": 4 * rows * case["d"]}
    own_keys = 0 if case["form"] == "memory" else case["t"]
    keys = sum(_starts(case)) + case["b"] * own_keys
    moved = keys * case["hk"] * 2 * (case["d"] + 4) + 2 * case["b"] * case["t"] * case["hq"] * case["d"] * es
    seen = sum(_starts(case)) * case["t"]
    if case["form"] == "chain":
        seen += case["b"] * case["t"] * (case["t"] + 1) // 2
    elif case["form"] == "tree":
        seen += case["b"] * case["t"]                           # at least itself
    return {"bytes": moved, "flops": 4 * case["d"] * case["hq"] * seen}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = _T[case["dtype"]]

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)

    def uniform(lo, hi, *shape):
        return torch.rand(shape, generator=gen, device=dev, dtype=torch.float32) * (hi - lo) + lo

    st = dict(case)
    if case["op"] == "norm":
        rows, heads, c = case["rows"], case["heads"], case["c"]
        # tokens differ in size, and a few channels stand out
        size = uniform(0.3, 3.0, rows, 1, 1) * torch.where(uniform(0, 1, c) < 0.01, 8.0, 1.0)
        shape = (rows, 3, heads, c) if case["packed"] else (rows, 1, heads, c)
        st["x"] = (normal(*shape) * size.unsqueeze(1)).to(dt)[:, 0]
        st["res"] = normal(rows, heads, c, dtype=dt) if case["residual"] else None
        st["weight"] = uniform(0.5, 1.5, c)
        if case["train"]:
            st["gy"] = normal(rows, heads, c, dtype=dt)
            st["gh"] = normal(rows, heads, c, dtype=dt) if case["residual"] else None
        return st
    # a cache in use: pages handed out in any order, one more page that no sequence has
    b, t, hk, d = case["b"], case["t"], case["hk"], case["d"]
    st["dp"] = dp = -(-d // 16) * 16
    starts = _starts(case)
    pages = -(-(case["longest"] + t) // _PAGE)
    order = torch.randperm(b * pages, generator=gen, device=dev)
    st["table"] = order.to(torch.int32).reshape(b, pages)
    st["start"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    n = b * pages + 1
    kind = _CODES[case["codes"]]

    def side(*shape):
        """Codes and scales as rows of normal values leave them (a row's largest value is near 3)."""
        values = torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16)
        values = (values * (_MOST[case["codes"]] / 3.5)).clamp_(-_MOST[case["codes"]], _MOST[case["codes"]])
        return values.round_().to(torch.int8) if kind == torch.int8 else values.to(kind)

    st["k"], st["v"] = side(n, hk, _PAGE, dp), side(n, hk, dp, _PAGE)
    if dp > d:
        st["k"].view(torch.uint8)[..., d:] = 0
        st["v"].view(torch.uint8)[:, :, d:] = 0
    st["k_scale"] = uniform(2.0, 4.0, n, hk, _PAGE) / _MOST[case["codes"]]
    st["v_scale"] = uniform(2.0, 4.0, n, hk, _PAGE) / _MOST[case["codes"]]
    if case["op"] == "cache":
        size = uniform(0.2, 4.0, b, t, 1, 1)
        st["new_k"] = (normal(b, t, hk, d) * size).to(dt)
        st["new_v"] = normal(b, t, hk, d, dtype=dt)
        st["count"] = torch.tensor(_counts(case), dtype=torch.int32, device=dev) if case["ragged"] else None
        return st
    st["q"] = normal(b, t, case["hq"], d, dtype=dt)
    st["ancestors"] = None
    if case["form"] == "tree":
        # a drafted token hangs on one of the eight before it, or on the cache itself
        words = -(-t // 64)
        back = torch.randint(1, 9, (b, t), generator=gen, device=dev).tolist()
        rows = []
        for i in range(b):
            masks = []
            for j in range(t):
                parent = j - back[i][j]
                masks.append((masks[parent] if parent >= 0 else 0) | 1 << j)
            signed = [[(m >> 64 * w) & (1 << 64) - 1 for w in range(words)] for m in masks]
            rows.append([[x - (1 << 64) if x >> 63 else x for x in m] for m in signed])
        st["ancestors"] = torch.tensor(rows, dtype=torch.int64, device=dev)
    return st


# ------------------------------------------------------------------ plain forms

def _nearest(values, scale, kind):
    """The codes nearest to values / scale as numbers, ties to the even one."""
    q = (values.double() / scale.double()).clamp(-_MOST[kind], _MOST[kind])
    if kind == "int8":
        return torch.round(q)
    exponent = torch.frexp(q).exponent - 1
    step = torch.ldexp(torch.ones_like(q), exponent.clamp(min=-6) - 3)
    return torch.round(q / step) * step


def _scale_plain(values, kind):
    top = values.abs().amax(dim=-1, keepdim=True)
    return torch.div(top, torch.full_like(top, _MOST[kind])).clamp(min=_TINY)     # a quotient, not a product


def _norm_plain(st):
    x, dt, w = st["x"], st["x"].dtype, st["weight"]
    h = x if st["res"] is None else (x.float() + st["res"].float()).to(dt)
    hf = h.float()
    rstd = 1 / torch.sqrt((hf * hf).mean(dim=-1, keepdim=True) + _EPS)
    y = hf * rstd * w
    if st["codes"]:
        c, kind = st["c"], st["codes"]
        block = min(st["block"] or c, c)
        blocks = -(-c // block)
        padded = torch.nn.functional.pad(y, (0, blocks * block - c)).unflatten(-1, (blocks, block))
        scale = _scale_plain(padded, kind)
        codes = _nearest(padded, scale, kind).flatten(-2)[..., :c]
        codes = codes.to(_CODES[kind]) if kind == "e4m3" else codes.to(torch.bfloat16)
        return [codes, scale.squeeze(-1)] + ([] if st["res"] is None else [h])
    y = y.to(dt)
    if not st["train"]:
        return y if st["res"] is None else (y, h)
    gy = st["gy"].float()
    u = gy * w
    gx = rstd * (u - hf * (rstd * rstd) * (u * hf).mean(dim=-1, keepdim=True))
    if st["gh"] is not None:
        gx = gx + st["gh"].float()
    gw = (gy * hf * rstd).sum(dim=(0, 1))
    return y, h, gx.to(dt), gw


def _cache_plain(st):
    b, t, d, kind, dt = st["b"], st["t"], st["d"], st["codes"], _T[st["dtype"]]
    dev = st["k"].device
    at = st["start"].long()[:, None] + torch.arange(t, device=dev)
    kept = torch.ones((b, t), dtype=torch.bool, device=dev)
    if st["count"] is not None:
        kept = torch.arange(t, device=dev) < st["count"][:, None]
    page = torch.gather(st["table"].long(), 1, at // _PAGE)
    page = torch.where(kept, page, torch.full_like(page, st["k"].shape[0] - 1))     # the page that no sequence has
    slot = at % _PAGE

    def write(x, codes, scales, transposed):
        x = x.float()
        s = _scale_plain(x, kind)
        new = _nearest(x, s, kind).to(_CODES[kind]).view(torch.uint8)
        raw = codes.view(torch.uint8)
        if transposed:
            raw[page, :, :d, slot] = new
        else:
            raw[page, :, slot, :d] = new
        scales[page, :, slot] = s.squeeze(-1)

    def read(codes, scales, transposed):
        raw = codes.view(torch.uint8)
        got = raw[page, :, :d, slot] if transposed else raw[page, :, slot, :d]
        values = got.view(_CODES[kind]).float() * scales[page, :, slot].unsqueeze(-1)
        return torch.where(kept[:, :, None, None], values, torch.zeros_like(values)).to(dt)

    write(st["new_k"], st["k"], st["k_scale"], False)
    write(st["new_v"], st["v"], st["v_scale"], True)
    return read(st["k"], st["k_scale"], False), read(st["v"], st["v_scale"], True)


def _attn_plain(st):
    b, t, hq, hk, d = (st[n] for n in ("b", "t", "hq", "hk", "d"))
    dev, dt, g = st["q"].device, st["q"].dtype, hq // hk
    table = st["table"].long()
    n = table.shape[1] * _PAGE
    # [B, W, Hk, ...] pages side by side
    k = (st["k"].view(torch.uint8)[table].view(st["k"].dtype).float() * st["k_scale"][table].unsqueeze(-1))[..., :d]
    v = (st["v"].view(torch.uint8)[table].view(st["v"].dtype).float() * st["v_scale"][table].unsqueeze(-2))[..., :d, :]
    k = k.permute(0, 2, 4, 1, 3).reshape(b, hk, d, n).contiguous()
    v = v.permute(0, 2, 1, 4, 3).reshape(b, hk, n, d).contiguous()
    q = st["q"].float().reshape(b, t, hk, g, d).permute(0, 2, 1, 3, 4).reshape(b, hk, t * g, d).contiguous()
    s = torch.matmul(q, k) / math.sqrt(d)
    if st["cap"]:
        s = st["cap"] * torch.tanh(s / st["cap"])
    at = torch.arange(n, device=dev)
    start = st["start"].long()[:, None, None]
    seen = (at < start).expand(b, t, n)
    drafted = at - start                                        # a key's place among the new tokens
    if st["form"] == "chain":
        seen = drafted <= torch.arange(t, device=dev)[:, None]
    elif st["form"] == "tree":
        place = drafted.clamp(0, t - 1).expand(b, t, n)
        word = torch.gather(st["ancestors"], 2, place // 64)
        seen = seen | ((word >> (place % 64) & 1).bool() & (drafted >= 0) & (drafted < t))
    s = s.reshape(b, hk, t, g, n).masked_fill(~seen[:, None, :, None], float("-inf")).reshape(b, hk, t * g, n)
    m = s.amax(dim=-1, keepdim=True)
    p = torch.exp(s - torch.where(m == float("-inf"), torch.zeros_like(m), m))
    total = p.sum(dim=-1, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    o = torch.matmul(p, v)
    return o.reshape(b, hk, t, g, d).permute(0, 2, 1, 3, 4).reshape(b, t, hq, d).to(dt)


# ------------------------------------------------------------------ the library's calls

def _norm_own(st):
    from camera_bev_view_amd import ops
    if st["codes"]:
        codes, scales, h = ops.rms_norm_codes(st["x"], st["weight"], residual=st["res"], eps=_EPS,
                                              codes=_CODES[st["codes"]], block=st["block"])
        codes = codes if st["codes"] == "e4m3" else codes.to(torch.bfloat16)
        return [codes, scales] + ([] if st["res"] is None else [h])
    y, h, rstd = ops.rms_norm_forward(st["x"], st["weight"], residual=st["res"], eps=_EPS)
    if not st["train"]:
        return y if st["res"] is None else (y, h)
    gx, gw = ops.rms_norm_backward(st["gy"], h, rstd, st["weight"], grad_h=st["gh"])
    return y, h, gx, gw


def _cache_own(st):
    from camera_bev_view_amd import ops
    cache = ops.TokenCache(st["k"], st["v"], st["k_scale"], st["v_scale"], st["d"])
    ops.cache_write(cache, st["new_k"], st["new_v"], st["table"], st["start"], count=st["count"])
    return ops.cache_read(cache, st["table"], st["start"], st["t"], count=st["count"], dtype=_T[st["dtype"]])


def _attn_own(st):
    from camera_bev_view_amd import ops
    cache = ops.TokenCache(st["k"], st["v"], st["k_scale"], st["v_scale"], st["d"])
    return ops.cache_attention(st["q"], cache, st["table"], st["start"], ancestors=st["ancestors"],
                               drafted=st["form"] != "memory", cap=st["cap"])


_PLAIN = {"norm": _norm_plain, "cache": _cache_plain, "attn": _attn_plain}
_OWN = {"norm": _norm_own, "cache": _cache_own, "attn": _attn_own}


def run(state):
    return (_OWN if own else _PLAIN)[state["op"]](state)


# ------------------------------------------------------------------ the definitions in 64 bits

def _grid(kind):
    """All values that a code stands for, ascending."""
    if kind == "int8":
        return [float(i) for i in range(-127, 128)]
    up = [m / 8 * 2.0 ** -6 for m in range(1, 8)] + [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)]
    up = [x for x in up if x <= 448]
    return [-x for x in reversed(up)] + [0.0] + up


def _snap(q, kind):
    """The nearest value of the grid, ties to the one with the even last bit."""
    grid = torch.tensor(_grid(kind), dtype=torch.float64, device=q.device)
    zero = (len(grid) - 1) // 2
    hi = torch.searchsorted(grid, q.contiguous()).clamp(1, len(grid) - 1)
    lo = hi - 1
    down, up = q - grid[lo], grid[hi] - q
    take = (up < down) | ((up == down) & ((hi - zero) % 2 == 0))
    return torch.where(take, grid[hi], grid[lo])


def _rows_scale(values, kind):
    """The scale, a number of 32 bits by its definition."""
    top = torch.linalg.vector_norm(values, ord=float("inf"), dim=-1, keepdim=True).float()
    return torch.div(top, torch.tensor(_MOST[kind], device=top.device)).clamp(min=_TINY).double()


def _norm_exact(st):
    train = st["train"]
    x = st["x"].double()
    h = x if st["res"] is None else (x + st["res"].double()).to(st["x"].dtype).double()
    h.requires_grad_(train)
    w = st["weight"].double().requires_grad_(train)
    y = h * torch.rsqrt(h.square().mean(dim=-1, keepdim=True) + _EPS) * w
    if st["codes"]:
        kind, codes, scales = st["codes"], [], []
        for part in y.split(st["block"] or st["c"], dim=-1):
            s = part.abs().amax(dim=-1, keepdim=True) / _MOST[kind]
            scales.append(s.clamp(min=_TINY))
            codes.append(_snap((part / scales[-1]).clamp(-_MOST[kind], _MOST[kind]), kind))
        out = [torch.cat(codes, dim=-1), torch.cat(scales, dim=-1)]
        return out + ([] if st["res"] is None else [h])
    if not train:
        return y if st["res"] is None else (y, h)
    torch.autograd.backward([y] + ([h] if st["gh"] is not None else []),
                            [st["gy"].double()] + ([st["gh"].double()] if st["gh"] is not None else []))
    return y.detach(), h.detach(), h.grad, w.grad


def _cache_exact(st):
    out = []
    for x in (st["new_k"], st["new_v"]):
        x = x.double()
        s = _rows_scale(x, st["codes"])
        back = _snap((x / s).clamp(-_MOST[st["codes"]], _MOST[st["codes"]]), st["codes"]) * s
        if st["ragged"]:
            for i, n in enumerate(_counts(st)):
                back[i, n:] = 0
        out.append(back)
    return tuple(out)


def _attn_exact(st):
    b, t, hq, hk, d = (st[n] for n in ("b", "t", "hq", "hk", "d"))
    dev, g = st["q"].device, hq // hk
    out = torch.empty((b, t, hq, d), dtype=torch.float64, device=dev)
    for i, n in enumerate(_starts(st)):
        total = n if st["form"] == "memory" else n + t
        pages = st["table"][i].long()
        own_part = torch.zeros((t, total - n), dtype=torch.bool, device=dev)
        if st["form"] == "chain":
            own_part = torch.ones((t, t), dtype=torch.bool, device=dev).tril()
        elif st["form"] == "tree":
            bits = st["ancestors"][i]
            own_part = torch.cat([(bits[:, w, None] >> torch.arange(64, device=dev)) % 2 != 0
                                  for w in range(bits.shape[1])], dim=1)[:, :t]
        hidden = torch.cat((torch.zeros((t, n), dtype=torch.bool, device=dev), ~own_part), dim=1)
        for a in range(hk):
            k = st["k"].view(torch.uint8)[pages, a].view(st["k"].dtype).double() * st["k_scale"][pages, a].double()[..., None]
            v = st["v"].view(torch.uint8)[pages, a].view(st["v"].dtype).double() * st["v_scale"][pages, a].double()[:, None]
            k, v = k.flatten(0, 1)[:total, :d], v.transpose(1, 2).flatten(0, 1)[:total, :d]
            for h in range(a * g, a * g + g):
                s = st["q"][i, :, h].double() @ k.T * d ** -0.5
                if st["cap"]:
                    s = torch.tanh(s / st["cap"]) * st["cap"]
                s = s.masked_fill(hidden, float("-inf"))
                none = hidden.all(dim=-1, keepdim=True)
                out[i, :, h] = torch.softmax(s.masked_fill(none, 0.0), dim=-1).masked_fill(none, 0.0) @ v
    return out


_EXACT = {"norm": _norm_exact, "cache": _cache_exact, "attn": _attn_exact}


def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed))
