"""Cases, plain forms and exact values of the token operators: query/key norm with
multi-axis rotary positions (forward and backward), the append to a paged cache, and
attention over that cache.

A token is one cell of a pooled BEV grid, one pixel of a camera feature map, or one
word; its position is a point (frame, row, column) or a single index.  The sizes are the
camera maps (16 x 44 pixels, six cameras), BEV grids (128 x 128 cells) and channel widths
(64, 80, 128) of this repository's workloads, and generic serving sizes.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16,
          "e4m3": torch.float8_e4m3fn}
BYTES = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1}
EPS = 1e-6
K_SCALE, V_SCALE = 0.0175, 0.0125     # of e4m3 caches: normed keys reach 7.8, values 5.6


# ---------------------------------------------------------------------------------------
# cases
def _rope_case(name, tokens, q_heads, k_heads, dim, dtype, sections, layout, grid, frame0, norm,
               backward, packed):
    return {"name": name, "op": "norm_rope", "tokens": tokens, "q_heads": q_heads,
            "k_heads": k_heads, "dim": dim, "dtype": dtype, "sections": sections,
            "layout": layout, "grid": grid, "frame0": frame0, "norm": norm,
            "backward": backward, "packed": packed}


def _append_case(name, seqs, new, ctx, kind, mix, q_heads, k_heads, dim, dtype, cache, page,
                 sections, layout, norm):
    return {"name": name, "op": "append", "seqs": seqs, "new": new, "ctx": ctx, "kind": kind,
            "mix": mix, "q_heads": q_heads, "k_heads": k_heads, "dim": dim, "dtype": dtype,
            "cache": cache, "page": page, "sections": sections, "layout": layout, "norm": norm}


def _attend_case(name, seqs, new, ctx, kind, mix, q_heads, k_heads, dim, dtype, cache, page,
                 causal, window):
    return {"name": name, "op": "attend", "seqs": seqs, "new": new, "ctx": ctx, "kind": kind,
            "mix": mix, "q_heads": q_heads, "k_heads": k_heads, "dim": dim, "dtype": dtype,
            "cache": cache, "page": page, "causal": causal, "window": window}


def listed():
    return [
        # the tokens of a few small requests, forward only: latency
        _rope_case("rope_small_f16", 24, 8, 2, 64, "f16", "8,12,12", "halves", "16x44", 3, True,
                   False, False),
        # a training step over one 128 x 128 BEV grid, queries and keys inside one packed
        # projection, three axes, an old stream's frame number
        _rope_case("rope_train_bf16", 16384, 16, 4, 128, "bf16", "16,24,24", "halves", "128x128",
                   250000, True, True, True),
        # an odd number of tokens of two axes, partial rotation, 80 channels, 32-bit training
        _rope_case("rope_train_odd_f32", 4223, 5, 5, 80, "f32", "12,12", "adjacent", "32x88", 0,
                   True, True, False),
        # one new token for each of 64 requests: latency
        _append_case("append_step_bf16", 64, 1, 100, "ragged", 1, 32, 8, 128, "bf16", "bf16", 16,
                     "64", "halves", True),
        # one frame of 128 x 128 cells into an e4m3 cache
        _append_case("append_frame_e4m3", 1, 16384, 100, "even", 0, 16, 8, 128, "bf16", "e4m3",
                     64, "16,24,24", "halves", True),
        # prompts of every length, 80 channels, no norm
        _append_case("append_ragged_f16", 23, 1501, 64, "ragged", 2, 8, 8, 80, "f16", "f16", 32,
                     "8,16,16", "adjacent", False),
        # the smallest call: one token of one short request
        _attend_case("attend_step_small_f16", 1, 1, 510, "even", 0, 8, 2, 64, "f16", "f16", 16,
                     True, 0),
        # single tokens of 64 requests of every length up to 8,192
        _attend_case("attend_step_bf16", 64, 1, 8191, "ragged", 3, 32, 8, 128, "bf16", "bf16", 16,
                     True, 0),
        # single tokens of two very long requests over an e4m3 cache
        _attend_case("attend_step_long_e4m3", 2, 1, 131071, "even", 0, 32, 4, 128, "bf16", "e4m3",
                     64, True, 0),
        # a prompt's next chunk over what is cached
        _attend_case("attend_chunk_bf16", 1, 4096, 8192, "even", 0, 32, 8, 128, "bf16", "bf16",
                     64, True, 0),
        # six cameras' 16 x 44 pixels over four frames each, every pixel of the new frame sees
        # every other
        _attend_case("attend_frames_f16", 6, 704, 2112, "even", 0, 8, 8, 80, "f16", "f16", 32,
                     False, 0),
        # chunks and single tokens in one batch, a sliding window, an e4m3 cache
        _attend_case("attend_mixed_e4m3", 24, 333, 6000, "mixed", 5, 14, 2, 64, "f16", "e4m3", 16,
                     True, 4096),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_heads(rng):
    k = rng.choice([1, 2, 4, 5, 8])
    return k * rng.choice([1, 2, 3, 4, 7, 8]), k


SECTIONS = {64: ["32", "8,12,12", "8,8", "16,16"], 80: ["40", "8,16,16", "12,12", "24"],
            96: ["48", "16,16,16", "24,24"], 128: ["64", "16,24,24", "32", "32,32"],
            256: ["128", "32,48,48", "32"]}


def draw(rng):
    op = rng.choice(["norm_rope", "append", "attend", "attend"])
    dim = rng.choice([64, 80, 96, 128, 128, 256])
    q_heads, k_heads = _draw_heads(rng)
    layout = rng.choice(["halves", "adjacent"])
    sections = rng.choice(SECTIONS[dim])
    norm = rng.random() < 0.75
    dtype = rng.choice(["f16", "bf16"])
    if op == "norm_rope":
        most = min(16384, 16384 * 20 * 128 // ((q_heads + k_heads) * dim))
        c = _rope_case("", _log_int(rng, 1, most), q_heads, k_heads, dim,
                       rng.choice(["f16", "bf16", "f32"]), sections, layout,
                       rng.choice(["16x44", "32x88", "128x128"]), _log_int(rng, 1, 1000000), norm,
                       rng.random() < 0.6, rng.random() < 0.5)
    elif op == "append":
        seqs = _log_int(rng, 1, 128)
        most = max(1, min(16384, 16384 * 32 * 128 // ((q_heads + 2 * k_heads) * dim)) // seqs)
        c = _append_case("", seqs, 1 if rng.random() < 0.4 else _log_int(rng, 1, most),
                         _log_int(rng, 1, 300), rng.choice(["even", "ragged"]), rng.randrange(10**6),
                         q_heads, k_heads, dim, dtype, rng.choice([dtype, "e4m3"]),
                         rng.choice([16, 32, 64, 128]), sections, layout, norm)
    else:
        cache = rng.choice([dtype, dtype, "e4m3"])
        page = rng.choice([16, 32, 64, 128])
        window = 0 if rng.random() < 0.75 else _log_int(rng, 32, 4096)
        causal = rng.random() < 0.75
        if rng.random() < 0.5:
            seqs = _log_int(rng, 1, 128)
            most = min(32768, (1 << 28) // (seqs * k_heads * dim))
            c = _attend_case("", seqs, 1, _log_int(rng, 1, most), rng.choice(["even", "ragged"]),
                             rng.randrange(10**6), q_heads, k_heads, dim, dtype, cache, page,
                             causal, window)
        else:
            seqs = _log_int(rng, 1, 16)
            new = _log_int(rng, 2, 4096)
            # scores of the padded batch: fewer than the largest listed case's
            most = (1 << 37) // (seqs * new * q_heads * max(dim, 128)) - new
            new, ctx = (new, _log_int(rng, 1, min(16384, most))) if most >= 64 else (64, 700)
            c = _attend_case("", seqs, new, ctx, rng.choice(["even", "ragged", "mixed"]),
                             rng.randrange(10**6), q_heads, k_heads, dim, dtype, cache, page,
                             causal, window)
    del c["name"]
    return c


def _lengths(c):
    """New and cached tokens of each sequence, by the case alone."""
    rng = random.Random(c["mix"])
    new, ctx = [], []
    for s in range(c["seqs"]):
        if c["kind"] == "even":
            new.append(c["new"])
            ctx.append(c["ctx"])
            continue
        ctx.append(rng.randint(c["ctx"] // 4, c["ctx"]))
        if c["kind"] == "ragged":
            new.append(c["new"] if s == 0 else rng.randint(1, c["new"]))
        else:
            new.append(c["new"] if s % 4 == 0 else 1)
    return new, ctx


# ---------------------------------------------------------------------------------------
# inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(DTYPES[dtype])


def _e4m3_or(g, shape, dtype, scale):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float16)
    if dtype == "e4m3":
        return (x / scale).clamp_(-448, 448).to(torch.float8_e4m3fn)
    return x.to(DTYPES[dtype])


def _rope_tables(c):
    sections = [int(v) for v in c["sections"].split(",")]
    half = sum(sections)
    i = torch.arange(half, dtype=torch.float64)
    inv_freq = (10000.0 ** (-i / half)).to(torch.float32).cuda()
    axis = torch.repeat_interleave(torch.arange(len(sections)), torch.tensor(sections)).cuda()
    return sections, inv_freq, axis


def _grid_positions(n, sections, rows, cols, frame0):
    i = torch.arange(n, device="cuda")
    point = [frame0 + i // (rows * cols), (i // cols) % rows, i % cols]
    point = {1: [frame0 + i], 2: point[1:], 3: point}[len(sections)]
    return torch.stack(point).to(torch.int32).contiguous()


def _weights(g, c):
    if not c["norm"]:
        return None, None
    return tuple((1.0 + 0.2 * torch.randn(c["dim"], generator=g, device="cuda")).to(DTYPES[c["dtype"]])
                 for _ in range(2))


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"c": c}
    hq, hk, d = c["q_heads"], c["k_heads"], c["dim"]
    if c["op"] == "norm_rope":
        n = c["tokens"]
        s["sections"], s["inv_freq"], s["axis"] = _rope_tables(c)
        rows, cols = (int(v) for v in c["grid"].split("x"))
        s["positions"] = _grid_positions(n, s["sections"], rows, cols, c["frame0"])
        s["qw"], s["kw"] = _weights(g, c)

        def pair():
            if c["packed"]:
                x = _randn(g, (n, hq + 2 * hk, d), c["dtype"])
                return x[:, :hq], x[:, hq:hq + hk]
            return _randn(g, (n, hq, d), c["dtype"]), _randn(g, (n, hk, d), c["dtype"])
        s["q"], s["k"] = pair()
        if c["backward"]:
            s["dq"], s["dk"] = pair()
    else:
        new, ctx = _lengths(c)
        page, seqs = c["page"], c["seqs"]
        kv = [a + b for a, b in zip(new, ctx)]
        n = sum(new)
        s["max_new"], s["max_kv"] = max(new), max(kv)
        s["q_offsets"] = torch.tensor([0] + torch.tensor(new).cumsum(0).tolist(),
                                      dtype=torch.int32, device="cuda")
        s["kv_lengths"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
        # every sequence's pages lie anywhere in the pool
        need = [-(-v // page) for v in kv]
        n_pages, width = sum(need) + 3, max(need)
        order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed),
                               dtype=torch.int32)
        table = torch.full((seqs, width), -1, dtype=torch.int32)
        at = 0
        for i, v in enumerate(need):
            table[i, :v] = order[at:at + v]
            at += v
        s["block_table"] = table.cuda()
        shape = (n_pages, hk, page, d)
        s["k_cache"] = _e4m3_or(g, shape, c["cache"], K_SCALE)
        s["v_cache"] = _e4m3_or(g, shape, c["cache"], V_SCALE)
        s["k_scale"], s["v_scale"] = (K_SCALE, V_SCALE) if c["cache"] == "e4m3" else (1.0, 1.0)
        if c["op"] == "append":
            s["sections"], s["inv_freq"], s["axis"] = _rope_tables(c)
            s["positions"] = _grid_positions(n, s["sections"], 128, 128, c["ctx"])
            s["qw"], s["kw"] = _weights(g, c)
            x = _randn(g, (n, hq + 2 * hk, d), c["dtype"])
            s["q"], s["k"], s["v"] = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
        else:
            s["q"] = _randn(g, (n, hq, d), c["dtype"], 2.0)
    if own:
        import depth_weighted_scatter_amd as dws
        if "sections" in s:
            s["rope"] = dws.Rope(s["inv_freq"], s["sections"],
                                 dws.ROPE_HALVES if c["layout"] == "halves" else dws.ROPE_ADJACENT)
        if "k_cache" in s:
            s["cache"] = dws.PagedCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
            s["batch"] = dws.PagedBatch(s["q_offsets"], s["kv_lengths"], s["block_table"])
    return s


# ---------------------------------------------------------------------------------------
# plain forms
def _angles(s):
    """cos and sin of position * inv_freq; the angle in 64 bits, far positions lose it in 32."""
    a = s["positions"].double()[s["axis"]] * s["inv_freq"].double()[:, None]     # [half, n]
    a = a.t()[:, None, :]
    return a.cos().float(), a.sin().float()


def _pairs(c, x, half):
    if c["layout"] == "halves":
        return x[..., :half], x[..., half:2 * half]
    return x[..., 0:2 * half:2], x[..., 1:2 * half:2]


def _joined(c, a, b, rest):
    if c["layout"] == "halves":
        return torch.cat([a, b, rest], -1)
    return torch.cat([torch.stack([a, b], -1).flatten(-2), rest], -1)


def _rotated(c, x, cos, sin):
    half = cos.shape[-1]
    a, b = _pairs(c, x, half)
    return _joined(c, a * cos - b * sin, b * cos + a * sin, x[..., 2 * half:])


def _normed(x, w):
    if w is None:
        return x.float()
    x = x.float()
    return x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * w.float()


def _plain_backward(c, x, w, dy, cos, sin):
    g = _rotated(c, dy.float(), cos, -sin)
    if w is None:
        return g.to(dy.dtype), None
    x = x.float()
    r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    xh = x * r
    dw = (g * xh).double().sum((0, 1)).float()
    g = g * w.float()
    dx = r * (g - xh * (g * xh).mean(-1, keepdim=True))
    return dx.to(dy.dtype), dw


def _plain_norm_rope(s):
    c = s["c"]
    cos, sin = _angles(s)
    got = {"q": _rotated(c, _normed(s["q"], s["qw"]), cos, sin).to(s["q"].dtype),
           "k": _rotated(c, _normed(s["k"], s["kw"]), cos, sin).to(s["k"].dtype)}
    if c["backward"]:
        got["dq"], got["dq_weight"] = _plain_backward(c, s["q"], s["qw"], s["dq"], cos, sin)
        got["dk"], got["dk_weight"] = _plain_backward(c, s["k"], s["kw"], s["dk"], cos, sin)
    return got


def _owners(s):
    """Sequence of each token, its index there and its place in the sequence."""
    off, kv = s["q_offsets"].long(), s["kv_lengths"].long()
    i = torch.arange(s["q"].shape[0], device="cuda")
    seq = torch.searchsorted(off, i, right=True) - 1
    at = i - off[seq]
    return seq, at, kv[seq] - (off[seq + 1] - off[seq]) + at


def _stored(x, cache, scale):
    if cache.dtype == torch.float8_e4m3fn:
        return (x.float() / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return x.to(cache.dtype)


def _plain_append(s):
    c, page = s["c"], s["c"]["page"]
    cos, sin = _angles(s)
    q = _rotated(c, _normed(s["q"], s["qw"]), cos, sin).to(s["q"].dtype)
    k = _rotated(c, _normed(s["k"], s["kw"]), cos, sin)
    seq, _, place = _owners(s)
    where = s["block_table"].long()[seq, place // page], slice(None), place % page
    for name, x, scale in (("k_cache", k, s["k_scale"]), ("v_cache", s["v"], s["v_scale"])):
        cache = s[name]
        raw = cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache
        raw[where] = _stored(x, cache, scale)
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attend(s):
    c = s["c"]
    d, hk, page = c["dim"], c["k_heads"], c["page"]
    grp = c["q_heads"] // hk
    seqs, new, kv = c["seqs"], s["max_new"], s["max_kv"]
    off, lens = s["q_offsets"].long(), s["kv_lengths"].long()
    n = s["q"].shape[0]
    at = torch.arange(new, device="cuda")
    rows = (off[:-1, None] + at).clamp(max=n - 1)                         # [seqs, new]
    q = s["q"][rows].float().view(seqs, new, hk, grp, d).permute(0, 2, 3, 1, 4)
    q = q.reshape(seqs * hk, grp * new, d)
    j = torch.arange(kv, device="cuda")
    pages = s["block_table"].long()[:, j // page].clamp(min=0)           # [seqs, kv]

    def rows_of(cache, scale):
        if cache.dtype == torch.float8_e4m3fn:
            x = cache.view(torch.uint8)[pages, :, j % page].view(torch.float8_e4m3fn).float() * scale
        else:
            x = cache[pages, :, j % page].float()
        return x.transpose(1, 2).reshape(seqs * hk, kv, d)                # [seqs * hk, kv, d]

    kt = rows_of(s["k_cache"], s["k_scale"]).transpose(1, 2).contiguous()
    scores = torch.matmul(q, kt).view(seqs, hk, grp, new, kv) * d ** -0.5
    place = (lens - (off[1:] - off[:-1]))[:, None] + at                    # [seqs, new]
    seen = (j < lens[:, None])[:, None, :].expand(seqs, new, kv)
    if c["causal"]:
        seen = seen & (j <= place[..., None])
    if c["window"]:
        seen = seen & (j > place[..., None] - c["window"])
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = (scores - torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(seqs * hk, grp * new, kv), rows_of(s["v_cache"], s["v_scale"]))
    o = o.view(seqs, hk, grp, new, d) / torch.where(total == 0, 1.0, total)
    seq, at, _ = _owners(s)
    return o[seq, :, :, at].reshape(n, hk * grp, d).to(s["q"].dtype)


def run(state):
    s, c = state, state["c"]
    if not own:
        return {"norm_rope": _plain_norm_rope, "append": _plain_append,
                "attend": _plain_attend}[c["op"]](s)
    import depth_weighted_scatter_amd as dws
    if c["op"] == "norm_rope":
        got = {}
        got["q"], got["k"] = dws.bevpool_qk_norm_rope(s["q"], s["k"], s["positions"], s["rope"],
                                                      s["qw"], s["kw"], EPS)
        if c["backward"]:
            got["dq"], got["dk"], got["dq_weight"], got["dk_weight"] = \
                dws.bevpool_qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["positions"],
                                                  s["rope"], s["qw"], s["kw"], EPS)
        return got
    if c["op"] == "append":
        q = dws.bevpool_kv_append(s["k"], s["v"], s["cache"], s["batch"], s["positions"],
                                  s["rope"], q=s["q"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS)
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    return dws.bevpool_paged_attention(s["q"], s["cache"], s["batch"], causal=c["causal"],
                                       window=c["window"])


# ---------------------------------------------------------------------------------------
# what a pass cannot do without
def work(case):
    c = case
    hq, hk, d, e = c["q_heads"], c["k_heads"], c["dim"], BYTES[c["dtype"]]
    if c["op"] == "norm_rope":
        n, elems = c["tokens"], c["tokens"] * (hq + hk) * d
        parts = 5 if c["backward"] else 2        # x, y; dy, dx and x again for the gradient
        return {"bytes": parts * elems * e + 4 * n * len(c["sections"].split(",")),
                "flops": (35 if c["backward"] else 10) * elems}
    new, ctx = _lengths(c)
    b = BYTES[c["cache"]]
    if c["op"] == "append":
        n = sum(new)
        return {"bytes": n * d * (2 * hq * e + 2 * hk * e + 2 * hk * b)
                + 4 * n * len(c["sections"].split(",")), "flops": 10 * n * (hq + hk) * d}
    pairs = read = 0
    for t, x in zip(new, ctx):
        first = x - c["window"] + 1 if c["window"] else 0     # of the first new token's keys
        read += t + x - max(0, first)
        for i in (range(t) if c["causal"] or c["window"] else ()):
            last = x + i if c["causal"] else x + t - 1
            pairs += last - max(0, x + i - c["window"] + 1 if c["window"] else 0) + 1
        if not (c["causal"] or c["window"]):
            pairs += t * (t + x)
    return {"bytes": 2 * sum(new) * hq * d * e + 2 * read * hk * d * b, "flops": 4 * d * hq * pairs}


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits
def _exact_turned(c, x, pos, inv_freq, axis):
    """x [n, heads, d] in float64, each pair turned as a complex number."""
    half = inv_freq.numel()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       pos.double()[axis].mul(inv_freq.double()[:, None])).t()[:, None]
    part = x[..., :2 * half]
    part = part.unflatten(-1, (2, half)).transpose(-1, -2) if c["layout"] == "halves" \
        else part.unflatten(-1, (half, 2))
    z = torch.view_as_real(torch.view_as_complex(part.contiguous()) * turn)
    z = z.transpose(-1, -2).flatten(-2) if c["layout"] == "halves" else z.flatten(-2)
    return torch.cat([z, x[..., 2 * half:]], -1)


def _exact_normed(x, w):
    if w is None:
        return x
    return w * x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS)


def _exact_norm_rope(s):
    c, got = s["c"], {}
    for name in "qk":
        x = s[name].double().requires_grad_(c["backward"])
        w = s[name + "w"]
        w = None if w is None else w.double().requires_grad_(c["backward"])
        y = _exact_turned(c, _exact_normed(x, w), s["positions"], s["inv_freq"], s["axis"])
        got[name] = y.detach()
        if c["backward"]:
            grads = torch.autograd.grad(y, [x] if w is None else [x, w], s["d" + name].double())
            got["d" + name] = grads[0]
            got["d%s_weight" % name] = None if w is None else grads[1]
    return got


def _exact_append(s):
    c = s["c"]
    got = {}
    for name in "qk":
        w = s[name + "w"]
        x = _exact_normed(s[name].double(), None if w is None else w.double())
        got[name] = _exact_turned(c, x, s["positions"], s["inv_freq"], s["axis"])
    caches = {"k_cache": s["k_cache"].double(), "v_cache": s["v_cache"].double()}
    new, ctx = _lengths(c)
    at = 0
    for i, (t, x) in enumerate(zip(new, ctx)):
        place = torch.arange(x, x + t, device="cuda")
        page, slot = s["block_table"][i].long()[place // c["page"]], place % c["page"]
        for name, rows, scale in (("k_cache", got["k"], s["k_scale"]),
                                  ("v_cache", s["v"].double(), s["v_scale"])):
            rows = rows[at:at + t] / scale
            caches[name][page, :, slot] = rows.clamp(-448, 448) if c["cache"] == "e4m3" else rows
        at += t
    return {"q": got["q"], **caches}


def _exact_attend(s):
    c = s["c"]
    hk, d, page = c["k_heads"], c["dim"], c["page"]
    grp = c["q_heads"] // hk
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    new, ctx = _lengths(c)
    pool = [(s[n].double() * s[m]).transpose(1, 2)                      # [pages, page, hk, d]
            for n, m in (("k_cache", "k_scale"), ("v_cache", "v_scale"))]
    at = 0
    for i, (t, x) in enumerate(zip(new, ctx)):
        pages = s["block_table"][i, :-(-(t + x) // page)].long()
        k, v = (x64[pages].flatten(0, 1)[:t + x] for x64 in pool)       # [kv, hk, d]
        j = torch.arange(t + x, device="cuda")[None]
        p = torch.arange(x, x + t, device="cuda")[:, None]
        hidden = torch.zeros((t, t + x), dtype=torch.bool, device="cuda")
        if c["causal"]:
            hidden |= j > p
        if c["window"]:
            hidden |= j <= p - c["window"]
        for h in range(hk):
            for g in range(h * grp, (h + 1) * grp):
                w = torch.mm(s["q"][at:at + t, g].double(), k[:, h].t().contiguous()) / math.sqrt(d)
                w = torch.softmax(w.masked_fill_(hidden, -math.inf), -1)
                out[at:at + t, g] = torch.mm(w, v[:, h].contiguous())
        at += t
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm_rope": _exact_norm_rope, "append": _exact_append,
            "attend": _exact_attend}[case["op"]](s)
