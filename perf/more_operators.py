"""Measured cases of the operators around the FP4 attention projections: norms
of queries and keys for each head with the position rotation in the same pass
(and their gradient), products of a few tokens with FP4 weights, the paged FP4
cache of keys and values that new tokens are appended to, and the attention
that reads it.

``own`` selects the side that ``run`` computes: False, the plain form in
elementary torch operations (fp32, the rotation of stored keys in fp64, rounded
once at the end); True, the framework's calls. ``listed`` and ``draw`` give the
cases, ``prepare`` their inputs, ``work`` the bytes and operations a pass cannot
do without and ``exact`` the outputs in fp64 from the definitions.

FP4 storage: E2M1 elements in blocks along a row, of 32 with one power of two
each (mxfp4) or of 16 with one E4M3 scale each and one fp32 scale per tensor
(nvfp4). A cache holds keys and values as two such matrices, one row per page,
head and place in the page, in that order. A rotation's table has one row per
position: the cosines of its angles, then the sines.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}
_BLOCK = {"mxfp4": 32, "nvfp4": 16}
_EPS = 1e-6


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one new token's queries and keys between the projection and the cache of an 8B model (latency)
        {"name": "qk-token", "op": "qk_fwd", "tokens": 1, "heads": 32, "kv": 8, "dim": 128, "rot": 128,
         "pairs": "halves", "x": "bf16", "y": "bf16", "kind": "rms", "w": "bf16", "far": 131072},
        # a training batch of an 8B model behind the fp32 output of one fused FP4 projection
        {"name": "qk-fwd-batch", "op": "qk_fwd", "tokens": 8192, "heads": 32, "kv": 8, "dim": 128, "rot": 128,
         "pairs": "halves", "x": "f32", "y": "bf16", "kind": "rms", "w": "bf16", "far": 8192},
        # a gradient with heads of an odd size, a rotation of a part of each and neighbouring elements as its pairs
        {"name": "qk-bwd-odd", "op": "qk_bwd", "tokens": 517, "heads": 15, "kv": 5, "dim": 90, "rot": 30,
         "pairs": "neighbours", "x": "f32", "y": "f32", "kind": "layer", "w": "f32", "far": 4096},
        # a training step of a 1.1B-class model: forward, then the gradient
        {"name": "qk-step", "op": "qk_step", "tokens": 8192, "heads": 32, "kv": 4, "dim": 64, "rot": 64,
         "pairs": "halves", "x": "bf16", "y": "bf16", "kind": "rms", "w": "f32", "far": 4096},
        # one token through the attention projection of an 8B model, its weight split (latency)
        {"name": "gemv-token", "op": "gemv", "tokens": 1, "in": 4096, "out": 4096, "rank": 64, "fmt": "mxfp4",
         "x": "bf16", "y": "bf16"},
        # a decoding batch through the up projection of an 8B model's FFN
        {"name": "gemv-batch", "op": "gemv", "tokens": 16, "in": 4096, "out": 14336, "rank": 64, "fmt": "mxfp4",
         "x": "bf16", "y": "f32"},
        # a few drafted tokens through its down projection in the other format, unsplit, from fp32 activations
        {"name": "gemv-draft", "op": "gemv", "tokens": 5, "in": 14336, "out": 4096, "rank": 0, "fmt": "nvfp4",
         "x": "f32", "y": "f32"},
        # one new token of each of 32 sequences
        {"name": "append-tokens", "op": "append", "seqs": 32, "new": 1, "ragged": False, "longest": 40, "kv": 8,
         "dim": 128, "rot": 128, "pairs": "halves", "page": 16, "fmt": "mxfp4", "x": "bf16", "spare": 3},
        # prompts of unequal length, from the fp32 output of the projection
        {"name": "append-prompts", "op": "append", "seqs": 7, "new": 2048, "ragged": True, "longest": 2048, "kv": 8,
         "dim": 128, "rot": 64, "pairs": "neighbours", "page": 48, "fmt": "nvfp4", "x": "f32", "spare": 0},
        # the next token of one sequence of ordinary length (latency)
        {"name": "attend-token", "op": "attend", "seqs": 1, "new": 1, "ragged": False, "longest": 1023, "least": 1023,
         "empty": 0, "heads": 32, "kv": 8, "dim": 128, "page": 16, "window": 0, "fmt": "mxfp4", "x": "bf16",
         "y": "bf16"},
        # a serving batch of unequal lengths, some places of the batch unused
        {"name": "attend-batch", "op": "attend", "seqs": 64, "new": 1, "ragged": False, "longest": 8192, "least": 64,
         "empty": 3, "heads": 32, "kv": 8, "dim": 128, "page": 64, "window": 0, "fmt": "mxfp4", "x": "bf16",
         "y": "bf16"},
        # drafted tokens of a few long sequences, counts unequal, looking back over a window
        {"name": "attend-draft", "op": "attend", "seqs": 5, "new": 6, "ragged": True, "longest": 32768, "least": 20000,
         "empty": 0, "heads": 12, "kv": 4, "dim": 64, "page": 16, "window": 30000, "fmt": "nvfp4", "x": "f32",
         "y": "f32"},
    ]


def _spread(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["qk_fwd", "qk_bwd", "qk_step", "gemv", "gemv", "append", "append", "attend", "attend", "attend"])
    t = lambda: rng.choice(["bf16", "bf16", "f32"])  # noqa: E731
    if op.startswith("qk"):
        dim = rng.choice([64, 96, 128, 192, 256, 2 * rng.randint(8, 128)])
        rot = rng.choice([dim, dim, 2 * rng.randint(1, dim // 2)])
        heads, kv = rng.randint(1, 32), rng.randint(1, 8)
        return {"op": op, "tokens": _spread(rng, 1, 10000000 // ((heads + kv) * dim)), "heads": heads, "kv": kv,
                "dim": dim, "rot": rot, "pairs": rng.choice(["halves", "neighbours"]), "x": t(), "y": t(),
                "kind": rng.choice(["rms", "rms", "layer", "none"]), "w": rng.choice(["bf16", "f32"]),
                "far": _spread(rng, 16, 131072)}
    fmt = rng.choice(["mxfp4", "nvfp4"])
    if op == "gemv":
        rank = rng.choice([0, rng.randint(1, 96), 64])
        unit = 32 if rank or fmt == "mxfp4" else 16
        out, inner = _spread(rng, 32, 14336), unit * _spread(rng, 1, 14336 // unit)
        out = max(32, out // 32 * 32) if rank else out
        return {"op": op, "tokens": _spread(rng, 1, min(64, 6000000000 // (out * inner))), "in": inner, "out": out,
                "rank": rank, "fmt": fmt, "x": t(), "y": t()}
    case = {"op": op, "kv": rng.randint(1, 8), "dim": 32 * rng.randint(1, 8),
            "page": rng.choice([16, 32, 64, rng.randint(1, 100)]), "fmt": fmt, "x": t()}
    if op == "append":
        seqs = _spread(rng, 1, 64)
        new = _spread(rng, 1, 4096 // seqs)
        case.update(seqs=seqs, new=new, ragged=new > 1 and rng.random() < 0.7,
                    longest=new + _spread(rng, 1, 4096 // seqs),
                    rot=rng.choice([0, case["dim"], 2 * rng.randint(1, case["dim"] // 2)]),
                    pairs=rng.choice(["halves", "neighbours"]), spare=rng.randint(0, 4))
        return case
    new = rng.choice([1, 1, rng.randint(2, 24)])
    group = rng.choice([1, 2, 3, 4, 5, 8, 16])
    room = min(1 << 28, (1 << 31) // (new * group)) // (case["kv"] * case["dim"])  # tokens of all sequences
    longest = _spread(rng, new, max(new, min(16384, room)))
    seqs = _spread(rng, 1, max(1, min(64, room // longest)))
    case.update(seqs=seqs, new=new, ragged=new > 1 and rng.random() < 0.6, longest=longest,
                least=_spread(rng, new, longest), empty=rng.randint(0, 2) if seqs > 3 else 0,
                heads=case["kv"] * group,
                window=rng.choice([0, 0, 0, _spread(rng, 1, longest)]), y=t())
    return case


def _steps(count, least, most):
    """`count` whole numbers between `least` and `most`, the first of them `most`, the others over the whole range."""
    return [most if i == 0 else least + int((most - least) * (i * 0.6180339887498949 % 1.0)) for i in range(count)]


def _counts(case):
    """New tokens of each sequence."""
    if not case["ragged"]:
        return [case["new"]] * case["seqs"]
    return _steps(case["seqs"], 1, case["new"])


def _lengths(case):
    """Tokens that each sequence has, its new ones among them."""
    counts = _counts(case)
    if case["op"] == "append":
        return [max(n, m) for n, m in zip(counts, _steps(case["seqs"], case["new"], case["longest"]))]
    got = [max(n, m) for n, m in zip(counts, _steps(case["seqs"], case["least"], case["longest"]))]
    for i in range(case["empty"]):
        got[1 + i] = 0
    return got


# ------------------------------------------------------------------ inputs
def _rand(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _table(positions, rot):
    """Cosines and sines of every position's angles, formed in fp64: one row per position, `rot` values."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / max(1, rot))
    angle = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * freq
    return torch.cat([torch.cos(angle), torch.sin(angle)], dim=1).float().contiguous()


def _heads(gen, tokens, heads, dim):
    """Projected queries or keys: channels of unequal size, a few of them large, heads of unequal norm."""
    x = _rand(gen, tokens, heads, dim)
    x *= torch.exp(0.4 * _rand(gen, 1, heads, dim)) * torch.exp(0.3 * _rand(gen, tokens, heads, 1))
    big = torch.randint(0, dim, (max(1, dim // 32),), generator=gen, device="cuda")
    x[:, :, big] *= 5.0
    return x + 0.1 * _rand(gen, 1, heads, 1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    by_op = {"gemv": _prepare_gemv, "append": _prepare_append, "attend": _prepare_attend}
    by_op.get(case["op"], _prepare_qk)(gen, case, s)
    return s


def _prepare_qk(gen, case, s):
    T, D, nq, nk = case["tokens"], case["dim"], case["heads"] * case["dim"], case["kv"] * case["dim"]
    # queries, keys and values lie side by side in the one output of their projection
    both = torch.cat([_heads(gen, T, case["heads"] + case["kv"], D).view(T, nq + nk), _rand(gen, T, nk)], dim=1)
    both = both.to(_TYPES[case["x"]])
    s["q"], s["k"] = both[:, :nq], both[:, nq:nq + nk]
    s["table"] = _table(case["far"], case["rot"])
    if T <= case["far"]:
        first = torch.randint(0, case["far"] - T + 1, (1,), generator=gen, device="cuda")
        s["positions"] = (first + torch.arange(T, device="cuda")).to(torch.int32)
    else:
        s["positions"] = (torch.arange(T, device="cuda") % case["far"]).to(torch.int32)
    w = lambda: (1.0 + 0.1 * _rand(gen, D)).to(_TYPES[case["w"]]) if case["kind"] != "none" else None  # noqa: E731
    s["wq"], s["wk"] = w(), w()
    if case["op"] != "qk_fwd":
        dy = lambda n: (1e-3 * torch.exp(0.5 * _rand(gen, T, 1)) * _rand(gen, T, n)).to(_TYPES[case["y"]])  # noqa: E731
        s["dq"], s["dk"] = dy(nq), dy(nk)


def _prepare_gemv(gen, case, s):
    T, K, N, r = case["tokens"], case["in"], case["out"], case["rank"]
    x = _rand(gen, T, K)
    x[:, torch.randint(0, K, (max(1, K // 512),), generator=gen, device="cuda")] *= 20.0
    s["x"] = x.to(_TYPES[case["x"]])
    s["R"] = _plain_codes(0.02 * _rand(gen, N, K), case["fmt"])
    if r:
        s["U"] = _plain_codes(_rand(gen, r, N) / math.sqrt(N), case["fmt"])
        s["V"] = _plain_codes(_rand(gen, r, K) / math.sqrt(K), case["fmt"])
        s["S"] = 50.0 / torch.arange(1, r + 1, device="cuda", dtype=torch.float32) * torch.exp(0.1 * _rand(gen, 1))
    if own:
        import fp4_spectral_split_amd as M

        fmt = M.MXFP4 if case["fmt"] == "mxfp4" else M.NVFP4
        fp4 = lambda c, rows, cols: M.Fp4Tensor(fmt, rows, cols, *c)  # noqa: E731
        s["W"] = M.SplitRecord(N, K, r, fmt, S=s["S"] if r else None, R_q=fp4(s["R"], N, K),
                               Ut_q=fp4(s["U"], r, N) if r else None, Vt_q=fp4(s["V"], r, K) if r else None)


def _prepare_cache(gen, case, s, spare):
    """Pages in an order of their own, each sequence's in its row of the table, and the lengths."""
    P, S = case["page"], case["seqs"]
    order = torch.randperm(S, generator=gen, device="cuda")
    lengths = torch.tensor(_lengths(case), device="cuda")[order]
    counts = torch.tensor(_counts(case), device="cuda")[order]
    most = max(1, -(-max(_lengths(case)) // P))
    held = (lengths + P - 1) // P  # pages of each sequence
    pages = int(sum(-(-n // P) for n in _lengths(case))) + spare
    s["pages"] = max(1, pages)
    free = torch.randperm(s["pages"], generator=gen, device="cuda")
    at = torch.cumsum(held, 0) - held
    place = torch.arange(most, device="cuda")
    used = place[None, :] < held[:, None]
    page = free[(at[:, None] + place).clamp(max=s["pages"] - 1)]
    s["table"] = torch.where(used, page, -1).to(torch.int32).contiguous()
    s["lengths"] = lengths.to(torch.int32)
    starts = torch.zeros(S + 1, dtype=torch.int32, device="cuda")
    starts[1:] = torch.cumsum(counts, 0)
    s["starts"], s["rows"] = starts, sum(_counts(case))
    rows, D = s["pages"] * case["kv"] * P, case["dim"]
    scale = torch.exp(0.3 * _rand(gen, case["kv"], 1, D)).expand(s["pages"], case["kv"], P, D)
    # a cache's tensor scales are chosen before anything is in it: here for magnitudes up to 64 and 8
    keys, values = _rand(gen, s["pages"], case["kv"], P, D) * scale, _rand(gen, rows, D)
    s["K"], s["V"] = (_plain_codes(x.view(rows, D), case["fmt"], torch.full((1,), top / 2688.0, device="cuda"))
                      for x, top in ((keys, 64.0), (values, 8.0)))
    if own:
        import fp4_spectral_split_amd as M

        s["cache"] = M.KvCache.from_codes(case["fmt"], s["pages"], P, case["kv"], D, s["K"], s["V"])
        one = case["new"] == 1 and not case["ragged"]
        s["batch"] = M.KvBatch(s["table"], s["lengths"], None if one else starts, case["new"])


def _prepare_append(gen, case, s):
    _prepare_cache(gen, case, s, case["spare"])
    D, t = case["dim"], _TYPES[case["x"]]
    n = case["kv"] * D
    both = torch.cat([_heads(gen, s["rows"], case["kv"], D).view(-1, n), _rand(gen, s["rows"], n)], dim=1).to(t)
    s["k"], s["v"] = both[:, :n], both[:, n:]
    s["angles"] = _table(case["longest"], case["rot"]) if case["rot"] else None


def _prepare_attend(gen, case, s):
    _prepare_cache(gen, case, s, 0)
    s["q"] = (1.5 * _rand(gen, s["rows"], case["heads"] * case["dim"])).to(_TYPES[case["x"]])


# -------------------------------------------------------------- plain form
def _pow2(e):
    """2^e, exact: e is put into the exponent field of an fp64."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _nearest(x, least, bits, top):
    """x rounded to nearest even, to `bits` bits behind the first one, in steps of 2^(least - bits) below 2^least,
    held at `top`."""
    _, e = torch.frexp(x)
    step = _pow2(torch.clamp(e - 1, min=least) - bits).to(x.dtype)
    return (torch.round(x / step) * step).clamp(-top, top)


def _plain_parts(x, fmt, tensor_scale=None):
    """FP4 form of the rows of x: E2M1 elements (rows x blocks x block), scales (rows x blocks) and, in nvfp4, the
    scale of the whole (that of x where none is given)."""
    rows, cols = x.shape
    v = x.float().view(rows, cols // _BLOCK[fmt], _BLOCK[fmt])
    top = v.abs().amax(dim=2)
    if fmt == "mxfp4":
        _, e = torch.frexp(top.double())
        e = torch.where(top > 0, e - 3, -127).clamp(-127, 127)
        scale = _pow2(e).float()
        return _nearest(v * _pow2(-e).float()[:, :, None], 0, 1, 6.0), scale, None
    if tensor_scale is None:
        tensor_scale = (top.amax() / 2688.0).clamp(min=2.0 ** -126).view(1)
    scale = _nearest(top / (6.0 * tensor_scale), -6, 3, 448.0)
    by = scale * tensor_scale
    q = torch.where(scale[:, :, None] > 0, v / torch.where(scale > 0, by, 1.0)[:, :, None], v * 0.0)
    return _nearest(q, 0, 1, 6.0), scale, tensor_scale


def _plain_codes(x, fmt, tensor_scale=None):
    """What is kept of x: codes, scale bytes and the tensor's scale (None in mxfp4)."""
    q, scale, whole = _plain_parts(x, fmt, tensor_scale)
    mag = q.abs()
    code = (mag > 0).to(torch.uint8)
    for lower in (0.5, 1.0, 1.5, 2.0, 3.0, 4.0):
        code += mag > lower
    code = code | torch.where(torch.signbit(q), 8, 0).to(torch.uint8)
    code = code.view(x.shape[0], -1)
    packed = (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous()
    _, e = torch.frexp(scale.double())
    if fmt == "mxfp4":
        byte = e - 1 + 127
    else:
        field = torch.where(scale > 0, torch.clamp(e - 1, min=-6), -6)
        byte = (field + 6) * 8 + (scale.double() / _pow2(field - 3)).to(torch.int64)
    return packed, byte.to(torch.uint8).contiguous(), whole


def _plain_values(kept, fmt):
    """fp32 values of codes (rows x cols / 2) and scale bytes."""
    packed, byte, whole = kept
    code = torch.stack([packed & 15, packed >> 4], dim=-1).view(*packed.shape[:-1], -1)
    level = (code & 7).float()
    mag = torch.where(level < 5, level * 0.5, torch.where(level < 6, 3.0, torch.where(level < 7, 4.0, 6.0)))
    v = torch.where(code > 7, -mag, mag)
    if fmt == "mxfp4":
        scale = _pow2(byte.to(torch.int64) - 127).float()
    else:
        b = byte.to(torch.int64)
        field, mant = (b >> 3) & 15, b & 7
        scale = torch.where(field > 0, mant + 8, mant).float() * _pow2(torch.clamp(field, min=1) - 10).float()
    v = v.view(*byte.shape, -1) * scale[..., None]
    if whole is not None:
        v = v * whole
    return v.flatten(-2)


def _rotated(x, table, pairs, back=False):
    """The last axis of x (tokens x heads x dim) with its first elements rotated by the tokens' rows of angles."""
    rot = table.shape[1]
    if not rot:
        return x
    c, s = table[:, None, :rot // 2].to(x.dtype), table[:, None, rot // 2:].to(x.dtype)
    if back:
        s = -s
    if pairs == "halves":
        a, b = x[:, :, :rot // 2], x[:, :, rot // 2:rot]
        return torch.cat([a * c - b * s, b * c + a * s, x[:, :, rot:]], dim=2)
    a, b = x[:, :, 0:rot:2], x[:, :, 1:rot:2]
    return torch.cat([torch.stack([a * c - b * s, b * c + a * s], dim=3).flatten(2), x[:, :, rot:]], dim=2)


def _statistics(x, kind):
    """Deviation from the mean (x itself in rms) and reciprocal deviation of every head."""
    d = x - x.mean(dim=2, keepdim=True) if kind == "layer" else x
    return d, 1.0 / torch.sqrt((d * d).mean(dim=2, keepdim=True) + _EPS)


def _plain_qk_fwd(x, w, table, case):
    x = x.float().reshape(x.shape[0], -1, case["dim"])
    if case["kind"] != "none":
        d, rstd = _statistics(x, case["kind"])
        x = d * rstd * w.float()
    return _rotated(x, table, case["pairs"]).flatten(1)


def _plain_qk_bwd(dy, x, w, table, case):
    D = case["dim"]
    g = _rotated(dy.float().reshape(dy.shape[0], -1, D), table, case["pairs"], back=True)
    if case["kind"] == "none":
        return g.flatten(1), None
    d, rstd = _statistics(x.float().reshape(x.shape[0], -1, D), case["kind"])
    xh = d * rstd
    u = g * w.float()
    dx = u - xh * (u * xh).mean(dim=2, keepdim=True)
    if case["kind"] == "layer":
        dx = dx - u.mean(dim=2, keepdim=True)
    return (dx * rstd).flatten(1), (g.double() * xh).sum(dim=(0, 1)).float()


def _places(s):
    """Of every new token: its sequence and its position."""
    row = torch.arange(s["rows"], device="cuda")
    seq = torch.searchsorted(s["starts"][1:].long(), row, right=True)
    count = (s["starts"][1:] - s["starts"][:-1]).long()
    return seq, s["lengths"].long()[seq] - count[seq] + row - s["starts"].long()[seq]


def _cache_rows(s, seq, position):
    """Rows of the cache that hold the heads of the given positions (last axis: heads)."""
    case = s["case"]
    page = s["table"].long()[seq, position // case["page"]]
    head = torch.arange(case["kv"], device="cuda")
    return (page[..., None] * case["kv"] + head) * case["page"] + (position % case["page"])[..., None]


def _plain_append(s):
    case = s["case"]
    D = case["dim"]
    seq, position = _places(s)
    k = s["k"].double().view(s["rows"], case["kv"], D)
    if case["rot"]:
        k = _rotated(k, s["angles"][position], case["pairs"])
    v = s["v"].float().reshape(-1, D)
    rows = _cache_rows(s, seq, position).view(-1)
    out = {}
    for name, kept, new in (("keys", s["K"], k.float().reshape(-1, D)), ("values", s["V"], v)):
        q, scale, whole = _plain_parts(new, case["fmt"], kept[2])
        got = q * scale[:, :, None]
        held = _plain_values(kept, case["fmt"])
        held[rows] = (got if whole is None else got * whole).view(-1, D)
        out[name] = held
    return out


def _plain_attend(s):
    case = s["case"]
    D, H, S, n = case["dim"], case["kv"], case["seqs"], case["new"]
    G = case["heads"] // H
    longest = s["table"].shape[1] * case["page"]
    lengths = s["lengths"].long()
    place = torch.arange(longest, device="cuda")
    rows = _cache_rows(s, torch.arange(S, device="cuda")[:, None], place[None, :].expand(S, longest))
    rows = rows.clamp(min=0).transpose(1, 2)  # sequences x heads x places; unused places are masked below
    k, v = (_plain_values((kept[0][rows], kept[1][rows], kept[2]), case["fmt"]) for kept in (s["K"], s["V"]))
    count = (s["starts"][1:] - s["starts"][:-1]).long()
    new = torch.arange(n, device="cuda")
    row = (s["starts"][:-1].long()[:, None] + new).clamp(max=s["rows"] - 1)  # sequences x new tokens
    there = new[None, :] < count[:, None]
    q = s["q"].float().view(s["rows"], H, G, D)[row].permute(0, 2, 1, 3, 4).reshape(S, H, n * G, D)
    scores = torch.matmul(q, k.transpose(2, 3).contiguous()) / math.sqrt(D)
    end = lengths[:, None] - count[:, None] + new + 1  # places below it are seen
    seen = place[None, None, :] < end[:, :, None]
    if case["window"]:
        seen = seen & (place[None, None, :] >= end[:, :, None] - case["window"])
    seen = seen.repeat_interleave(G, dim=1)[:, None].expand(S, H, n * G, longest)
    scores = torch.where(seen, scores, -math.inf)
    top = scores.amax(dim=3, keepdim=True)
    e = torch.where(seen, torch.exp(scores - torch.where(top > -math.inf, top, 0.0)), 0.0)
    total = e.sum(dim=3, keepdim=True)
    o = torch.matmul(e, v) / torch.where(total > 0, total, 1.0)
    o = o.view(S, H, n, G, D).permute(0, 2, 1, 3, 4).reshape(S, n, -1)
    return o[there].to(_TYPES[case["y"]])


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "gemv":
        x = s["x"].float()
        y = x @ _plain_values(s["R"], case["fmt"]).t()
        if case["rank"]:
            z = (x @ _plain_values(s["V"], case["fmt"]).t()) * s["S"]
            y = y + z @ _plain_values(s["U"], case["fmt"])
        return y.to(_TYPES[case["y"]])
    if op == "append":
        return _plain_append(s)
    if op == "attend":
        return _plain_attend(s)
    out, t = {}, _TYPES[case["y"]]
    table = s["table"][s["positions"].long()]
    if op != "qk_bwd":
        out["q"] = _plain_qk_fwd(s["q"], s["wq"], table, case).to(t)
        out["k"] = _plain_qk_fwd(s["k"], s["wk"], table, case).to(t)
    if op != "qk_fwd":
        dq, out["dwq"] = _plain_qk_bwd(s["dq"], s["q"], s["wq"], table, case)
        dk, out["dwk"] = _plain_qk_bwd(s["dk"], s["k"], s["wk"], table, case)
        out["dq"], out["dk"] = dq.to(_TYPES[case["x"]]), dk.to(_TYPES[case["x"]])
    return out


# --------------------------------------------------------- framework calls
def _run_own(s):
    import fp4_spectral_split_amd as M

    case = s["case"]
    op = case["op"]
    if op == "gemv":
        return M.metis_fp4_gemv(s["x"], s["W"], dtype=_TYPES[case["y"]])
    if op == "append":
        M.metis_kv_append(s["k"], s["v"], s["batch"], s["cache"], rope=s["angles"], pairs=case["pairs"])
        return {"keys": M.fp4_block_dequant(s["cache"].k), "values": M.fp4_block_dequant(s["cache"].v)}
    if op == "attend":
        return M.metis_kv_attention(s["q"], s["batch"], s["cache"], window=case["window"], dtype=_TYPES[case["y"]])[0]
    how = dict(kind=None if case["kind"] == "none" else case["kind"], eps=_EPS, pairs=case["pairs"])
    out = {}
    if op != "qk_bwd":
        out["q"], out["k"] = M.metis_qk_norm_rope_fwd(s["q"], s["k"], s["positions"], s["table"], case["dim"], s["wq"],
                                                      s["wk"], dtype=_TYPES[case["y"]], **how)
    if op != "qk_fwd":
        out["dq"], out["dk"], out["dwq"], out["dwk"] = M.metis_qk_norm_rope_bwd(
            s["dq"], s["dk"], s["q"], s["k"], s["positions"], s["table"], case["dim"], s["wq"], s["wk"],
            dtype=_TYPES[case["x"]], **how)
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# -------------------------------------------------------------------- work
def _held(rows, cols, fmt):
    return rows * (cols // 2 + cols // _BLOCK[fmt])


def work(case):
    op = case["op"]
    if op.startswith("qk"):
        n = case["tokens"] * (case["heads"] + case["kv"]) * case["dim"]
        x, y, table = n * _BYTES[case["x"]], n * _BYTES[case["y"]], case["tokens"] * (4 * case["rot"] + 4)
        w = 0 if case["kind"] == "none" else 2 * case["dim"]
        total, flops = table + w * _BYTES[case["w"]], 0
        if op != "qk_bwd":
            total += x + y
            flops += 8 * n
        if op != "qk_fwd":
            total += (2 * x if w else x) + y + 4 * w
            flops += 16 * n
        return {"bytes": total, "flops": flops}
    if op == "gemv":
        T, K, N, r = case["tokens"], case["in"], case["out"], case["rank"]
        total = _held(N, K, case["fmt"]) + T * (K * _BYTES[case["x"]] + N * _BYTES[case["y"]])
        if r:
            total += _held(r, K, case["fmt"]) + _held(r, N, case["fmt"]) + 4 * r
        return {"bytes": total, "flops": 2 * T * N * K + 2 * T * r * (N + K)}
    D, H, counts = case["dim"], case["kv"], _counts(case)
    if op == "append":
        n = sum(counts) * H
        rows = (sum(-(-m // case["page"]) for m in _lengths(case)) + case["spare"]) * case["page"] * H
        total = 2 * n * D * _BYTES[case["x"]] + 2 * _held(n, D, case["fmt"]) + sum(counts) * 4 * case["rot"]
        # the cache is read back whole, as fp32
        return {"bytes": total + 2 * _held(rows, D, case["fmt"]) + 8 * rows * D, "flops": 12 * n * D}
    G = case["heads"] // H
    read = seen = 0
    for length, count in zip(_lengths(case), counts):
        ends = [max(0, length - count + 1 + i) for i in range(count)]
        back = case["window"] or length
        read += max(0, length - max(0, (ends[0] if ends else 0) - back)) if length else 0
        seen += sum(min(e, back) for e in ends)
    total = 2 * _held(read * H, D, case["fmt"])
    total += sum(counts) * case["heads"] * D * (_BYTES[case["x"]] + _BYTES[case["y"]])
    return {"bytes": total, "flops": 4 * seen * H * G * D}


# ------------------------------------------------------------------- exact
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _exact_scales(fmt):
    """Value of every scale byte that is a number."""
    if fmt == "mxfp4":
        return [2.0 ** (b - 127) for b in range(255)]
    return [(b & 7) * 2.0 ** -9 if b < 8 else (8 + (b & 7)) * 2.0 ** ((b >> 3) - 10) for b in range(127)]


def _exact_values(kept, fmt):
    packed, byte, whole = kept
    grid = torch.tensor(_E2M1, device="cuda", dtype=torch.float64)
    v = torch.empty(*packed.shape, 2, device="cuda", dtype=torch.float64)
    v[..., 0] = grid[(packed % 16).long()]
    v[..., 1] = grid[(packed // 16).long()]
    scale = torch.tensor(_exact_scales(fmt), device="cuda", dtype=torch.float64)[byte.long()]
    v = v.reshape(*packed.shape[:-1], -1) * scale.repeat_interleave(_BLOCK[fmt], dim=-1)
    return v if whole is None else v * whole.double()


def _exact_nearest(x, grid):
    """Index of the entry of the ascending `grid` nearest to each x >= 0, a tie at the even one."""
    middle = (grid[1:] + grid[:-1]) / 2.0
    low = torch.searchsorted(middle, x.contiguous())
    tie = x == middle[low.clamp(max=middle.numel() - 1)]
    return torch.where(tie & (low % 2 == 1), low + 1, low).clamp(max=grid.numel() - 1)


def _exact_stored(x, fmt, whole):
    """The fp32 rows of x as their FP4 form holds them. In nvfp4 the form is defined by fp32 divisions."""
    rows, cols = x.shape
    v = x.view(rows, -1, _BLOCK[fmt])
    top = v.abs().amax(dim=2)
    grid = torch.tensor(_E2M1[:8], device="cuda", dtype=torch.float64)
    scales = torch.tensor(_exact_scales(fmt), device="cuda", dtype=torch.float64)
    if fmt == "mxfp4":
        # the largest power of two not above a quarter of the block's largest magnitude
        at = (torch.searchsorted(scales, top.double() / 4.0, right=True) - 1).clamp(min=0)
        scale = scales[at]
        mag = v.double().abs() / scale[:, :, None]
        return (torch.copysign(grid[_exact_nearest(mag, grid)], v.double()) * scale[:, :, None]).view(rows, cols)
    scale = scales[_exact_nearest((top / (whole * 6.0)).double(), scales)]
    by = scale.float() * whole
    mag = torch.where(by[:, :, None] > 0, v.abs() / by[:, :, None], 0.0).double()
    value = torch.copysign(grid[_exact_nearest(mag, grid)], v.double()) * scale[:, :, None]
    return (value * whole.double()).view(rows, cols)


def _exact_angles(x, cos, sin, pairs):
    """x (tokens x heads x dim) turned by complex factors, in fp64."""
    half = cos.shape[1]
    turn = torch.complex(cos, sin)[:, None]
    y = x.clone()
    if pairs == "halves":
        z = torch.complex(x[..., :half], x[..., half:2 * half]) * turn
        y[..., :half], y[..., half:2 * half] = z.real, z.imag
    else:
        z = torch.view_as_complex(x[..., :2 * half].reshape(*x.shape[:-1], half, 2).contiguous()) * turn
        y[..., :2 * half] = torch.view_as_real(z).flatten(-2)
    return y


def _exact_qk(case, s):
    D, rot, T = case["dim"], case["rot"], case["tokens"]
    table = s["table"].double().index_select(0, s["positions"].long())
    cos, sin = table[:, :rot // 2], table[:, rot // 2:]
    out = {}
    for name, x, w, dy in (("q", s["q"], s["wq"], s.get("dq")), ("k", s["k"], s["wk"], s.get("dk"))):
        x = x.double().reshape(T, -1, D)
        if case["kind"] == "none":
            xh, rstd, w = x, torch.ones_like(x[..., :1]), torch.ones(D, device="cuda", dtype=torch.float64)
        else:
            if case["kind"] == "layer":
                x = x - x.sum(2, keepdim=True) / D
            rstd = ((x ** 2).sum(2, keepdim=True) / D + _EPS) ** -0.5
            xh, w = x * rstd, w.double()
        if case["op"] != "qk_bwd":
            out[name] = _exact_angles(xh * w, cos, sin, case["pairs"]).reshape(T, -1)
        if case["op"] != "qk_fwd":
            g = _exact_angles(dy.double().reshape(T, -1, D), cos, -sin, case["pairs"])
            u = g * w
            if case["kind"] == "none":
                out["d" + name] = u.reshape(T, -1)
                continue
            level = u.sum(2, keepdim=True) / D if case["kind"] == "layer" else 0.0
            out["d" + name] = (rstd * (u - level - xh * ((u * xh).sum(2, keepdim=True) / D))).reshape(T, -1)
            out["dw" + name] = (g * xh).sum(0).sum(0)
    return out


def _exact_append(case, s):
    D, H, P = case["dim"], case["kv"], case["page"]
    keys, values = _exact_values(s["K"], case["fmt"]), _exact_values(s["V"], case["fmt"])
    k, v = s["k"].double().view(-1, H, D), s["v"].float().reshape(-1, H, D)
    starts, lengths = s["starts"].tolist(), s["lengths"].tolist()
    for i in range(case["seqs"]):
        a, b = starts[i], starts[i + 1]
        position = torch.arange(lengths[i] - (b - a), lengths[i], device="cuda")
        new = k[a:b]
        if case["rot"]:
            angle = s["angles"].double()[position]
            new = _exact_angles(new, angle[:, :case["rot"] // 2], angle[:, case["rot"] // 2:], case["pairs"])
        page = s["table"][i].long()[torch.div(position, P, rounding_mode="floor")]
        for h in range(H):
            rows = (page * H + h) * P + position.remainder(P)
            keys[rows] = _exact_stored(new[:, h].float().contiguous(), case["fmt"], s["K"][2])
            values[rows] = _exact_stored(v[a:b, h].contiguous(), case["fmt"], s["V"][2])
    return {"keys": keys, "values": values}


def _exact_attend(case, s):
    D, H, P = case["dim"], case["kv"], case["page"]
    G = case["heads"] // H
    starts, lengths = s["starts"].tolist(), s["lengths"].tolist()
    out = torch.zeros(s["rows"], H, G, D, device="cuda", dtype=torch.float64)
    q = s["q"].double().view(-1, H, G, D)
    for i in range(case["seqs"]):
        a, b, length = starts[i], starts[i + 1], lengths[i]
        if not length:
            continue
        place = torch.arange(length, device="cuda")
        page = s["table"][i].long()[torch.div(place, P, rounding_mode="floor")]
        for h in range(H):
            rows = (page * H + h) * P + place.remainder(P)
            k, v = (_exact_values((kept[0][rows], kept[1][rows], kept[2]), case["fmt"]) for kept in (s["K"], s["V"]))
            score = (q[a:b, h].reshape(-1, D) @ k.t()).view(b - a, G, length) * D ** -0.5
            end = length - (b - a) + 1 + torch.arange(b - a, device="cuda")
            hidden = place[None, :] >= end[:, None]
            if case["window"]:
                hidden |= place[None, :] < end[:, None] - case["window"]
            p = torch.softmax(score.masked_fill(hidden[:, None, :], -math.inf), dim=2)
            out[a:b, h] = (p.reshape(-1, length) @ v).view(b - a, G, D)
    return out.view(s["rows"], -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gemv":
        x = s["x"].double()
        y = x @ _exact_values(s["R"], case["fmt"]).t()
        if case["rank"]:
            low = (_exact_values(s["V"], case["fmt"]) @ x.t()) * s["S"].double()[:, None]
            y += (_exact_values(s["U"], case["fmt"]).t() @ low).t()
        return y
    if case["op"] == "append":
        return _exact_append(case, s)
    if case["op"] == "attend":
        return _exact_attend(case, s)
    return _exact_qk(case, s)
