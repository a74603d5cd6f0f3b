"""Measured cases of the operators that stand between the rotated linears of a served model.

Four operators:
  norm       RMS norm with the residual's addition, output in e4m3 with a scale per row and 128 columns
  linear8    matrix product in e4m3: activations scaled per row and 128 columns, weights per 128 x 128 block
  rope       rotary positions of q and k, with the write of k and v into a paged cache
  attention  attention of one new token per sequence over the paged cache

`own` chooses between elementary torch operations and the framework's kernels. `exact` evaluates
each operator's definition in 64 bits.
"""
import math

import torch

own = False

BLOCK = 128  # columns that share one 8-bit scale
E4M3_MAX = 448.0
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the norm before a projection at batch-1 decode, 4096 wide: latency
        {"name": "norm decode 1", "op": "norm", "rows": 1, "n": 4096, "type": "bf16", "residual": True, "weight": True},
        # a ragged width from an fp32 stream without residual or weight
        {"name": "norm odd", "op": "norm", "rows": 515, "n": 5000, "type": "f32", "residual": False, "weight": False},
        # the norm over a long prompt, 8192 wide: bandwidth
        {"name": "norm prompt", "op": "norm", "rows": 8192, "n": 8192, "type": "bf16", "residual": True, "weight": True},
        # the output head (32000 tokens of vocabulary) at batch-1 decode: the weights' bandwidth
        {"name": "linear8 head 1", "op": "linear8", "rows": 1, "n_in": 4096, "n_out": 32000, "type": "bf16"},
        # the down projection (11008 -> 4096) of a small decode batch of odd size
        {"name": "linear8 down 19", "op": "linear8", "rows": 19, "n_in": 11008, "n_out": 4096, "type": "f16"},
        # the gate projection over a prompt: tensor-core rate
        {"name": "linear8 gate prompt", "op": "linear8", "rows": 4096, "n_in": 8192, "n_out": 28672, "type": "bf16"},
        # 64 query and 8 key heads, 8 sequences each appending one token: latency
        {"name": "rope decode 8", "op": "rope", "rows": 8, "per_seq": 1, "heads": 64, "kv": 8, "dim": 128, "rot": 128,
         "interleaved": False, "scaling": "none", "page": 16, "far": 4096, "type": "bf16"},
        # a long prompt of 4 sequences, half of each head rotated in adjacent pairs, stretched to far positions
        {"name": "rope prompt", "op": "rope", "rows": 8192, "per_seq": 2048, "heads": 32, "kv": 32, "dim": 128, "rot": 64,
         "interleaved": True, "scaling": "bands", "page": 64, "far": 131072, "type": "bf16"},
        # one short sequence with as many key heads as query heads: latency
        {"name": "attention short 1", "op": "attention", "seqs": 1, "longest": 500, "shortest": 500, "heads": 32, "kv": 32,
         "dim": 128, "page": 16, "type": "bf16"},
        # one very long sequence, 8 query heads to a key head: the split over the length
        {"name": "attention long 1", "op": "attention", "seqs": 1, "longest": 131072, "shortest": 131072, "heads": 64, "kv": 8,
         "dim": 128, "page": 64, "type": "bf16"},
        # a served batch of very different lengths
        {"name": "attention ragged 32", "op": "attention", "seqs": 32, "longest": 8191, "shortest": 1, "heads": 64, "kv": 8,
         "dim": 128, "page": 16, "type": "bf16"},
        # many short sequences, narrow heads, some rows of the batch empty
        {"name": "attention batch 128", "op": "attention", "seqs": 128, "longest": 1000, "shortest": 0, "heads": 32, "kv": 32,
         "dim": 64, "page": 32, "type": "f16"},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "linear8", "rope", "attention"])
    if op == "norm":
        n = _log(rng, 64, 16384)
        return {"op": op, "rows": _log(rng, 1, min(8192, (8192 * 8192) // n)), "n": n, "type": rng.choice(["f32", "bf16", "f16"]),
                "residual": rng.random() < 0.6, "weight": rng.random() < 0.7}
    if op == "linear8":
        return {"op": op, "rows": _log(rng, 1, 4096), "n_in": _log(rng, 128, 8192), "n_out": _log(rng, 64, 28672),
                "type": rng.choice(["bf16", "f16"])}
    if op == "rope":
        dim = rng.choice([64, 96, 128])
        kv = rng.choice([1, 2, 4, 8, 16, 32])
        per_seq = _log(rng, 1, 2048)
        return {"op": op, "rows": per_seq * rng.randint(1, max(1, min(32, 4096 // per_seq))), "per_seq": per_seq,
                "heads": kv * rng.choice([1, 2, 4, 8][: 4 if kv <= 4 else 2]), "kv": kv, "dim": dim, "rot": rng.choice([dim, dim // 2]),
                "interleaved": rng.random() < 0.5, "scaling": rng.choice(["none", "linear", "bands"]),
                "page": rng.choice([8, 16, 32, 64]), "far": _log(rng, 4096, 1000000), "type": rng.choice(["bf16", "f16"])}
    seqs, kv, dim = _log(rng, 1, 128), rng.choice([1, 2, 4, 8, 32]), rng.choice([64, 96, 128])
    longest = _log(rng, 32, max(33, min(131072, (1 << 27) // (seqs * kv * dim))))
    return {"op": op, "seqs": seqs, "longest": longest, "shortest": rng.choice([0, 1, longest // 2, longest]),
            "heads": kv * rng.choice([1, 3, 4, 8]), "kv": kv, "dim": dim, "page": rng.choice([8, 16, 32, 64]),
            "type": rng.choice(["bf16", "f16"])}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _e4m3_rows(x):
    """e4m3 of x with a scale per row and 128 columns; scales as [blocks][rows], seen transposed."""
    rows, n = x.shape
    blocks = -(-n // BLOCK)
    padded = torch.nn.functional.pad(x, (0, blocks * BLOCK - n)).view(rows, blocks, BLOCK)
    s = padded.abs().amax(-1) / E4M3_MAX
    s = torch.where(s == 0, torch.ones_like(s), s)
    q = (padded / s[..., None]).view(rows, -1)[:, :n].to(torch.float8_e4m3fn)
    return q, s


def _row_padded(q):
    """The same values in rows that start on 16-byte boundaries, as the 8-bit operands are held."""
    rows, n = q.shape
    wide = torch.zeros((rows, -(-n // 16) * 16), dtype=torch.uint8, device=q.device)
    wide[:, :n] = q.view(torch.uint8)
    return wide.view(torch.float8_e4m3fn)[:, :n]


def _column_major(s):
    """[rows, blocks] scales in memory as [blocks][rows], each block's rows on a 16-byte boundary."""
    rows, blocks = s.shape
    t = torch.zeros((blocks, -(-rows // 4) * 4), dtype=torch.float32, device=s.device)
    t[:, :rows] = s.t()
    return t[:, :rows].t()


def _lengths(case, g):
    low, high, seqs = case["shortest"], case["longest"], case["seqs"]
    n = torch.randint(low, high + 1, (seqs,), generator=g, device="cuda", dtype=torch.int32)
    n[0] = high
    if seqs > 1:
        n[-1] = low
    return n


def _pages(seqs, per_seq, g):
    """A table of distinct pages in shuffled order, with some pages of the pool unused."""
    total = seqs * per_seq + 3
    return torch.randperm(total, generator=g, device="cuda")[: seqs * per_seq].view(seqs, per_seq).to(torch.int32), total


def prepare(case, seed):
    g = _gen(seed)
    t = TYPES[case["type"]]

    def randn(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)

    if case["op"] == "norm":
        rows, n = case["rows"], case["n"]
        s = {"case": case, "x": randn(rows, n, dtype=t), "residual": None, "weight": None}
        s["x"][:, ::97] *= 8  # the few loud channels of a residual stream
        if case["residual"]:
            s["residual"] = (randn(rows, n) * 2).to(t)
        if case["weight"]:
            s["weight"] = (1 + 0.1 * randn(n)).to(t)
        return s
    if case["op"] == "linear8":
        rows, n_in, n_out = case["rows"], case["n_in"], case["n_out"]
        q, sx = _e4m3_rows(randn(rows, n_in))
        w = randn(n_out, n_in) / math.sqrt(n_in)
        kb, nb = -(-n_in // BLOCK), -(-n_out // BLOCK)
        tiles = torch.nn.functional.pad(w, (0, kb * BLOCK - n_in, 0, nb * BLOCK - n_out)).view(nb, BLOCK, kb, BLOCK)
        sw = (tiles.abs().amax((1, 3)) / E4M3_MAX).contiguous()
        codes = (tiles / sw[:, None, :, None]).view(nb * BLOCK, kb * BLOCK)[:n_out, :n_in].to(torch.float8_e4m3fn)
        s = {"case": case, "x": _row_padded(q), "sx": _column_major(sx), "w": _row_padded(codes), "sw": sw}
        if own:
            import rotated_bit_matmul_b200 as rb

            s["layer"] = rb.HarpLinear8(s["w"], s["sw"])
        return s
    page, dim, kv, heads = case["page"], case["dim"], case["kv"], case["heads"]
    if case["op"] == "rope":
        rows, per_seq = case["rows"], case["per_seq"]
        seqs = rows // per_seq
        start = torch.randint(0, case["far"] - per_seq + 1, (seqs,), generator=g, device="cuda")
        pos = (start[:, None] + torch.arange(per_seq, device="cuda")).view(-1)
        first = start // page
        used = int(per_seq // page + 2)
        live, total = _pages(seqs, used, g)
        # the table covers every position up to `far`; pages before the new tokens are a shared, unread one
        table = torch.zeros((seqs, -(-case["far"] // page) + 2), dtype=torch.int32, device="cuda")
        table.scatter_(1, first[:, None] + torch.arange(used, device="cuda"), live)
        qkv = randn(rows, heads + 2 * kv, dim, dtype=t)  # as one fused projection leaves them
        s = {"case": case, "q": qkv[:, :heads], "k": qkv[:, heads : heads + kv], "v": qkv[:, heads + kv :],
             "positions": pos.to(torch.int32), "table": table,
             "seq_ids": torch.arange(seqs, device="cuda", dtype=torch.int32).repeat_interleave(per_seq),
             "k_pages": randn(total, kv, page, dim, dtype=t), "v_pages": randn(total, kv, page, dim, dtype=t)}
        if own:
            import rotated_bit_matmul_b200 as rb

            s["rope"] = rb.HarpRope(dim, case["rot"], interleaved=case["interleaved"], **_scaling_arguments(case))
            s["cache"] = rb.HarpCache(s["k_pages"], s["v_pages"])
        return s
    lengths = _lengths(case, g)
    table, total = _pages(case["seqs"], max(1, -(-case["longest"] // page)), g)
    s = {"case": case, "q": randn(case["seqs"], heads, dim, dtype=t), "table": table, "lengths": lengths,
         "k_pages": randn(total, kv, page, dim, dtype=t), "v_pages": randn(total, kv, page, dim, dtype=t)}
    if own:
        import rotated_bit_matmul_b200 as rb

        s["cache"] = rb.HarpCache(s["k_pages"], s["v_pages"])
    return s


# ------------------------------------------------------------------ rotary frequencies
BASE, FACTOR, ORIGINAL, LOW, HIGH = 10000.0, 8.0, 4096, 1.0, 4.0


def _scaling_arguments(case):
    if case["scaling"] == "none":
        return {"base": BASE}
    if case["scaling"] == "linear":
        return {"base": BASE, "scaling": "linear", "factor": FACTOR}
    return {"base": BASE, "scaling": "bands", "factor": FACTOR, "original": ORIGINAL, "low": LOW, "high": HIGH}


def _frequencies(case):
    """Radians per position of each pair. bands: pairs that turn more than HIGH times in ORIGINAL
    positions stay, those that turn less than LOW times are slowed by FACTOR, linear between."""
    rot = case["rot"]
    f = BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    if case["scaling"] == "linear":
        f = f / FACTOR
    elif case["scaling"] == "bands":
        keep = ((ORIGINAL * f / (2 * math.pi) - LOW) / (HIGH - LOW)).clamp(0, 1)
        f = f * keep + f / FACTOR * (1 - keep)
    return f


# ------------------------------------------------------------------ plain forms
def _plain_norm(s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h * (h.square().mean(-1, keepdim=True) + 1e-5).rsqrt()
    if s["weight"] is not None:
        y = y * s["weight"].float()
    q, scale = _e4m3_rows(y)
    return (q, scale) if s["residual"] is None else (q, scale, h.to(s["x"].dtype))


def _plain_linear8(s):
    case = s["case"]
    x = s["x"].float() * s["sx"].repeat_interleave(BLOCK, 1)[:, : case["n_in"]]
    blocks = s["sw"].repeat_interleave(BLOCK, 0)[: case["n_out"]].repeat_interleave(BLOCK, 1)[:, : case["n_in"]]
    return (x @ (s["w"].float() * blocks).t()).to(TYPES[case["type"]])


def _turned(x, cos, sin, case):
    x, rot = x.float(), case["rot"]
    cos, sin = cos[:, None], sin[:, None]
    if case["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        r = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2 : rot]
        r = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((r, x[..., rot:]), -1)


def _plain_rope(s):
    case, pos = s["case"], s["positions"].long()
    angle = pos.double()[:, None] * _frequencies(case)  # far positions: 32 bits lose the angle
    cos, sin = angle.cos().float(), angle.sin().float()
    t = s["q"].dtype
    page = s["table"][s["seq_ids"].long(), pos // case["page"]].long()
    row = pos % case["page"]
    s["k_pages"][page, :, row] = _turned(s["k"], cos, sin, case).to(t)
    s["v_pages"][page, :, row] = s["v"]
    return _turned(s["q"], cos, sin, case).to(t), s["k_pages"], s["v_pages"]


def _plain_attention(s):
    case = s["case"]
    seqs, heads, dim = s["q"].shape
    kv = case["kv"]
    q = s["q"].float().view(seqs, kv, heads // kv, dim)
    gather = lambda pages: pages[s["table"].long()].transpose(1, 2).reshape(seqs, kv, -1, dim).float()  # noqa: E731
    scores = q @ gather(s["k_pages"]).transpose(-1, -2) / math.sqrt(dim)
    live = torch.arange(scores.shape[-1], device="cuda") < s["lengths"][:, None, None, None]
    scores = scores.masked_fill(~live, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.where(live, (scores - top).exp(), 0.0)  # a sequence without keys: all zero
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    return (p @ gather(s["v_pages"])).view(seqs, heads, dim).to(s["q"].dtype)


def run(state):
    op = state["case"]["op"]
    if own:
        import rotated_bit_matmul_b200 as rb

        if op == "norm":
            return rb.harp_rmsnorm_q8(state["x"], weight=state["weight"], residual=state["residual"], eps=1e-5)
        if op == "linear8":
            return state["layer"](state["x"], state["sx"], out_dtype=TYPES[state["case"]["type"]])
        if op == "rope":
            q = state["rope"].append(state["cache"], state["q"], state["k"], state["v"], state["positions"], state["table"],
                                     seq_ids=state["seq_ids"])
            return q, state["k_pages"], state["v_pages"]
        return rb.harp_paged_attention(state["q"], state["cache"], state["table"], state["lengths"])
    return {"norm": _plain_norm, "linear8": _plain_linear8, "rope": _plain_rope, "attention": _plain_attention}[op](state)


# ------------------------------------------------------------------ what cannot be done without
def work(case):
    size = SIZE[case["type"]]
    if case["op"] == "norm":
        cells = case["rows"] * case["n"]
        moved = cells * (size * (3 if case["residual"] else 1) + 1) + case["rows"] * -(-case["n"] // BLOCK) * 4
        return {"bytes": moved + (case["n"] * size if case["weight"] else 0), "flops": 6 * cells}
    if case["op"] == "linear8":
        rows, n_in, n_out = case["rows"], case["n_in"], case["n_out"]
        kb, nb = -(-n_in // BLOCK), -(-n_out // BLOCK)
        return {"bytes": rows * n_in + n_out * n_in + 4 * kb * (rows + nb) + size * rows * n_out, "flops": 2 * rows * n_in * n_out}
    if case["op"] == "rope":
        cells = case["rows"] * (case["heads"] + 2 * case["kv"]) * case["dim"]
        return {"bytes": 2 * size * cells + 12 * case["rows"], "flops": 3 * case["rows"] * (case["heads"] + case["kv"]) * case["rot"]}
    low, high, seqs = case["shortest"], case["longest"], case["seqs"]
    keys = high if seqs == 1 else high + low + (seqs - 2) * (low + high) / 2  # lengths are drawn evenly between the two
    q = seqs * case["heads"] * case["dim"]
    return {"bytes": 2 * size * keys * case["kv"] * case["dim"] + 2 * size * q + 4 * keys / case["page"] + 4 * seqs,
            "flops": 4 * keys * case["heads"] * case["dim"]}


# ------------------------------------------------------------------ definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        rows, n = s["x"].shape
        h = s["x"].double() + (0 if s["residual"] is None else s["residual"].double())
        y = h / torch.sqrt((h * h).sum(1, keepdim=True) / n + 1e-5)
        if s["weight"] is not None:
            y = y * s["weight"].double()
        q, scales = torch.empty_like(y), []
        for at in range(0, n, BLOCK):
            block = y[:, at : at + BLOCK]
            scale = block.abs().max(1, keepdim=True).values / E4M3_MAX
            scale[scale == 0] = 1
            v = block / scale
            # e4m3: 3 bits after the leading one, exponents from -6
            step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0**-6))) - 3)
            q[:, at : at + BLOCK] = torch.round(v / step) * step
            scales.append(scale)
        scales = torch.cat(scales, 1)
        return (q, scales) if s["residual"] is None else (q, scales, h)
    if case["op"] == "linear8":
        y = torch.zeros((case["rows"], case["n_out"]), dtype=torch.float64, device="cuda")
        row_of = torch.arange(case["n_out"], device="cuda") // BLOCK
        for b in range(s["sw"].shape[1]):
            at = slice(b * BLOCK, min((b + 1) * BLOCK, case["n_in"]))
            part = s["x"][:, at].double() @ s["w"][:, at].double().t()
            y += part * s["sx"][:, b : b + 1].double() * s["sw"][row_of, b].double()
        return y
    if case["op"] == "rope":
        # a rotation by the angle is the product of complex numbers
        angle = s["positions"].double()[:, None] * _exact_frequencies(case)
        phase = torch.polar(torch.ones_like(angle), angle)[:, None]
        rot, out = case["rot"], []
        for x in (s["q"].double(), s["k"].double()):
            y = x.clone()
            first, second = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
            z = torch.complex(x[..., first], x[..., second]) * phase
            y[..., first], y[..., second] = z.real, z.imag
            out.append(y)
        k, v = s["k_pages"].double(), s["v_pages"].double()
        where = s["positions"].long()
        page = torch.gather(s["table"][s["seq_ids"].long()].long(), 1, torch.div(where, case["page"], rounding_mode="floor")[:, None])[:, 0]
        slot = page * case["page"] + where % case["page"]
        for pages, rows in ((k, out[1]), (v, s["v"].double())):
            flat = pages.transpose(1, 2).reshape(-1, case["kv"], case["dim"])
            flat[slot] = rows
            pages.copy_(flat.view(pages.shape[0], case["page"], case["kv"], case["dim"]).transpose(1, 2))
        return out[0], k, v
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    group = case["heads"] // case["kv"]
    for b, n in enumerate(s["lengths"].tolist()):
        if not n:
            continue
        at = s["table"][b, : -(-n // case["page"])].long()
        k, v = (p[at].double().transpose(0, 1).reshape(case["kv"], -1, case["dim"])[:, :n] for p in (s["k_pages"], s["v_pages"]))
        q = s["q"][b].double().view(case["kv"], group, case["dim"])
        weights = torch.softmax(torch.einsum("hgd,hnd->hgn", q, k) * case["dim"] ** -0.5, -1)
        out[b] = torch.einsum("hgn,hnd->hgd", weights, v).view(case["heads"], case["dim"])
    return out


def _exact_frequencies(case):
    rot, f = case["rot"], []
    for i in range(rot // 2):
        w = math.exp(-2 * i / rot * math.log(BASE))
        if case["scaling"] == "linear":
            w /= FACTOR
        elif case["scaling"] == "bands":
            wavelength = 2 * math.pi / w
            keep = min(1.0, max(0.0, (ORIGINAL / wavelength - LOW) / (HIGH - LOW)))
            w = (1 - keep) * w / FACTOR + keep * w
        f.append(w)
    return torch.tensor(f, dtype=torch.float64, device="cuda")
