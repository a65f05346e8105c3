"""The operators of the 4-bit latent cache and the norm in front of it, as cases that can be timed.

Four operators, in the order in which a serving step meets them:

* "norm": residual addition, root-mean-square norm and an E4M3 output with scales, one launch for what
  precedes the projections;
* "append": new latent rows quantised to 4 bits as they are written to the cache, and read back;
* "gather": rows of the 4-bit cache read back as bfloat16;
* "attn": sparse attention over the 4-bit cache (whole prefill chunks, packed batches, decode, paged).

A row of the cache is 416 bytes: 512 latent values as 4-bit codes (256 bytes), their 32 scales (one byte for
16 values), and 64 rotary values in bfloat16 (128 bytes). The code c in 0..15 stands for c - 8, and the scale
byte b for (1 + (b & 7) / 8) * 2^((b >> 3) - 18): the smallest one that keeps the group's largest magnitude
within 7 steps. In each 32-bit word of eight values, value j sits in nibble j/2 (j even) or 4 + j/2 (j odd).
"""
import math

import torch

own = False

D_LATENT, D_ROPE, D_ROW = 512, 64, 576
GROUP, ROW_BYTES = 16, 416


def listed():
    return [
        # one token of a decode step in front of the projections: latency
        dict(name="norm_token", op="norm", n=1, d=7168, dtype="bf16", residual=True, group=0, normed=False),
        # the low-rank query of a ragged batch, scales of 128 values, the bfloat16 row kept for the other projections
        dict(name="norm_ragged", op="norm", n=509, d=1536, dtype="bf16", residual=False, group=128, normed=True),
        # a prefill chunk of the hidden size
        dict(name="norm_chunk", op="norm", n=16384, d=7168, dtype="bf16", residual=True, group=0, normed=False),
        # the new tokens of a decode batch, each to its own sequence's page
        dict(name="append_decode", op="append", n=64, rows=65536, dtype="bf16", pad=0),
        # a prefill chunk with a padded tail, scattered over pages
        dict(name="append_chunk", op="append", n=16384, rows=131072, dtype="bf16", pad=37),
        # one selection's rows
        dict(name="gather_selection", op="gather", n=2048, rows=65536),
        # a whole long sequence read back
        dict(name="gather_sequence", op="gather", n=131072, rows=131072),
        # one sequence decoding: latency, the selection split over the GPU
        dict(name="attn_decode_one", op="attn", form="decode", T=1, L=65536, heads=128, topk=2048, seqs=1),
        # a full decode batch with the heads of one of eight shards
        dict(name="attn_decode_shard", op="attn", form="paged", T=64, L=16384, heads=16, topk=2048, seqs=64),
        # a full decode batch with all heads
        dict(name="attn_decode_batch", op="attn", form="decode", T=64, L=65536, heads=128, topk=2048, seqs=64),
        # a packed batch of short sequences, odd heads, selections that are not full or empty
        dict(name="attn_packed_odd", op="attn", form="varlen", T=333, L=2900, heads=17, topk=501, seqs=3),
        # the last tokens of a long prefill
        dict(name="attn_prefill", op="attn", form="prefill", T=1024, L=131072, heads=128, topk=2048, seqs=1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "append", "gather", "attn", "attn"])
    if op == "norm":
        return dict(op=op, n=_log(rng, 1, 12000), d=rng.choice([64 * _log(rng, 1, 128), _log(rng, 33, 8192)]),
                    dtype=rng.choice(["bf16", "bf16", "f32", "f16"]), residual=rng.random() < 0.6,
                    group=rng.choice([0, 0, 128]), normed=rng.random() < 0.4)
    if op == "append":
        n = _log(rng, 1, 16384)
        return dict(op=op, n=n, rows=n + _log(rng, 64, 100000), dtype=rng.choice(["bf16", "bf16", "f32"]),
                    pad=rng.choice([0, n // 9]))
    if op == "gather":
        return dict(op=op, n=_log(rng, 1, 131072), rows=_log(rng, 64, 131072))
    form = rng.choice(["decode", "paged", "varlen", "prefill"])
    heads = rng.choice([128, 128, 64, 16, rng.randint(1, 127)])
    topk = rng.choice([2048, 2048, _log(rng, 1, 2047)])
    if form in ("decode", "paged"):
        t = _log(rng, 1, 96)
        return dict(op=op, form=form, T=t, L=64 * _log(rng, 2, 600), heads=heads, topk=topk, seqs=t)
    seqs = 1 if form == "prefill" else rng.randint(1, 6)
    return dict(op=op, form=form, T=_log(rng, seqs, 1000), L=_log(rng, 70, 60000), heads=heads, topk=topk, seqs=seqs)


_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def work(c):
    if c["op"] == "norm":
        e = 4 if c["dtype"] == "f32" else 2
        v = c["n"] * c["d"]
        groups = c["n"] if not c["group"] else c["n"] * -(-c["d"] // c["group"])
        return {"bytes": v * (e * (1 + 2 * c["residual"] + c["normed"]) + 1) + c["d"] * e + groups * 4, "flops": 8 * v}
    if c["op"] == "append":
        n = c["n"] - c["pad"]
        e = 4 if c["dtype"] == "f32" else 2
        return {"bytes": n * (D_ROW * e + 4 + 2 * ROW_BYTES) + c["n"] * D_ROW * 2, "flops": 4 * n * D_LATENT}
    if c["op"] == "gather":
        return {"bytes": c["n"] * (4 + D_ROW * 2) + min(c["n"], c["rows"]) * ROW_BYTES, "flops": c["n"] * D_LATENT}
    t, h, k = c["T"], c["heads"], min(c["topk"], c["L"])
    distinct = t * k if c["form"] in ("decode", "paged") else min(t * k, c["seqs"] * c["L"])
    return {"bytes": distinct * ROW_BYTES + t * h * (D_ROW + D_LATENT) * 2 + t * c["topk"] * 4 + t * h * 4,
            "flops": 2 * t * k * h * (D_ROW + D_LATENT)}


# ---------------------------------------------------------------- the cache's rows, in elementary operations


def _step(byte):
    """The value of a scale byte, put together from its bits (a power function need not be exact)."""
    return ((byte << 20) + ((127 - 18) << 23)).view(torch.float32)


def pack(x):
    """[n, 576] rows (latent, rotary) as [n, 416] bytes of the cache. In 64 bits, where no quotient lies
    between two codes by its rounding."""
    n = x.shape[0]
    g = torch.nan_to_num(x[:, :D_LATENT].double(), nan=0.0).reshape(n, -1, GROUP)
    m, e = torch.frexp(g.abs().amax(dim=2) / 7)
    byte = torch.where(m > 0, (e + 17) * 8 + torch.ceil(m * 16).to(torch.int32) - 8, 0).clamp(0, 255)
    step = _step(byte).double()
    codes = (torch.round(g / step[:, :, None]).clamp(-7, 7) + 8).to(torch.uint8).reshape(n, -1, 4, 2)
    nib = torch.cat([codes[..., 0], codes[..., 1]], dim=-1)  # values 0 2 4 6 1 3 5 7 of each word
    return torch.cat([(nib[..., 0::2] | (nib[..., 1::2] << 4)).reshape(n, -1), byte.to(torch.uint8),
                      x[:, D_LATENT:].to(torch.bfloat16).contiguous().view(torch.uint8)], dim=1)


def unpack(b):
    """[n, 416] bytes of the cache as [n, 576] values in 32 bits (every one of them exact)."""
    n = b.shape[0]
    w = b[:, :256].reshape(n, -1, 4)
    nib = torch.stack([w & 15, w >> 4], dim=-1).reshape(n, -1, 2, 4).transpose(2, 3)
    step = _step(b[:, 256:288].to(torch.int32))
    lat = (nib.reshape(n, -1, GROUP).float() - 8) * step[:, :, None]
    return torch.cat([lat.reshape(n, -1), b[:, 288:].contiguous().view(torch.bfloat16).float()], dim=1)


# ---------------------------------------------------------------- inputs


def _latents(n, g):
    """Rows as they leave the latent's norm and the rotary encoding: spreads that differ by dimension, a few
    dimensions far above the others."""
    spread = torch.exp(0.4 * torch.randn(D_ROW, device="cuda", generator=g))
    spread[:: 97] *= 6
    return torch.randn(n, D_ROW, device="cuda", generator=g) * spread


def _cache(rows, g):
    pool = torch.empty(rows, ROW_BYTES, dtype=torch.uint8, device="cuda")
    for r in range(0, rows, 1 << 18):
        pool[r:r + (1 << 18)] = pack(_latents(min(rows - r, 1 << 18), g))
    return pool


def _selections(lens, topk, g):
    """For each token as many distinct rows below its length as the selection holds, in a ranking's order, then -1."""
    t = lens.numel()
    want = torch.clamp(lens, max=topk)[:, None].double()
    j = torch.arange(topk, device="cuda", dtype=torch.float64)[None, :]
    u = torch.rand(t, topk, device="cuda", generator=g, dtype=torch.float64)
    pos = torch.floor((j + u) * lens[:, None].double() / want.clamp(min=1))
    pos = torch.minimum(pos, (lens[:, None] - 1).double())
    rank = torch.where(j < want, torch.rand(t, topk, device="cuda", generator=g, dtype=torch.float64), 2.0)
    order = torch.argsort(rank, dim=1)
    pos = torch.gather(torch.where(j < want, pos, -1.0), 1, order)
    return pos.to(torch.int32).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    c, s = case, {"case": dict(case)}
    if c["op"] == "norm":
        t = _TYPES[c["dtype"]]
        s["x"] = (2 * torch.randn(c["n"], c["d"], device="cuda", generator=g)).to(t)
        s["residual"] = (8 * torch.randn(c["n"], c["d"], device="cuda", generator=g)).to(t) if c["residual"] else None
        s["weight"] = (1 + 0.2 * torch.randn(c["d"], device="cuda", generator=g)).to(t)
        return s
    if c["op"] == "append":
        s["x"] = _latents(c["n"], g).to(_TYPES[c["dtype"]])
        s["pool"] = torch.full((c["rows"] + 1, ROW_BYTES), 0x88, dtype=torch.uint8, device="cuda")
        slots = torch.randperm(c["rows"], device="cuda", generator=g)[:c["n"]].to(torch.int32)
        slots[c["n"] - c["pad"]:] = -1
        s["slots"] = slots
        return s
    if c["op"] == "gather":
        s["pool"] = _cache(c["rows"], g)
        s["rows"] = torch.randint(0, c["rows"], (c["n"],), device="cuda", generator=g).to(torch.int32)
        return s
    t, rows, seqs = c["T"], c["L"], c["seqs"]
    s["q"] = torch.randn(t, c["heads"], D_ROW, device="cuda", generator=g).to(torch.bfloat16)
    s["scale"] = 1.0 / math.sqrt(D_ROW)
    if c["form"] in ("decode", "paged"):
        lens = torch.randint(max(1, rows // 2), rows + 1, (t,), device="cuda", generator=g)
        s["pool"] = _cache(t * rows, g)
        s["first"] = torch.arange(t, device="cuda") * rows
        if c["form"] == "paged":
            pages = rows // 64
            s["table"] = torch.randperm(t * pages, device="cuda", generator=g).to(torch.int32).reshape(t, pages)
    elif c["form"] == "varlen":
        cut = [t * i // seqs for i in range(seqs + 1)]
        size = [max(1, rows - rows * i // (2 * seqs)) for i in range(seqs)]
        s["cu_q"] = torch.tensor(cut, dtype=torch.int32, device="cuda")
        s["cu_k"] = torch.tensor([sum(size[:i]) for i in range(seqs + 1)], dtype=torch.int32, device="cuda")
        of = torch.tensor([i for i in range(seqs) for _ in range(cut[i + 1] - cut[i])], device="cuda")
        s["first"] = s["cu_k"][of].long()
        lens = (torch.rand(t, device="cuda", generator=g) * (torch.tensor(size, device="cuda")[of] + 1)).long()
        lens[t // 2] = 0  # a padded token: nothing selected
        s["pool"] = _cache(sum(size), g)
    else:
        lens = torch.clamp(rows - t + 1 + torch.arange(t, device="cuda"), min=1)
        s["first"] = torch.zeros(t, dtype=torch.long, device="cuda")
        s["pool"] = _cache(rows, g)
    s["idx"] = _selections(lens, c["topk"], g)
    return s


# ---------------------------------------------------------------- one pass


def run(s):
    c = s["case"]
    if own:
        return _run_own(c, s)
    if c["op"] == "norm":
        return _norm(s["x"], s["residual"], s["weight"], c["group"], c["normed"])
    if c["op"] == "append":
        keep = s["slots"] >= 0
        at = torch.where(keep, s["slots"], s["pool"].shape[0] - 1).long()  # the last row is nobody's
        s["pool"][at] = pack(s["x"])
        return (unpack(s["pool"][at]) * keep[:, None]).to(torch.bfloat16)
    if c["op"] == "gather":
        return unpack(s["pool"][s["rows"].long()]).to(torch.bfloat16)
    return _attn(s["q"], s["pool"], _pool_rows(s), s["idx"] >= 0, s["scale"])


def _run_own(c, s):
    import long_context_03_b200 as dsa
    if c["op"] == "norm":
        codes, scale, summed, normed = dsa.rms_norm_quantize_e4m3_rows(
            s["x"], s["weight"], residual=s["residual"], eps=1e-6, group=c["group"], want_normed=c["normed"])
        out = {"codes": codes.view(torch.float8_e4m3fn), "scale": scale}
        return out | ({"sum": summed} if c["residual"] else {}) | ({"normed": normed} if c["normed"] else {})
    if c["op"] == "append":
        pool = s["pool"][:-1]
        dsa.latent_q4_append(s["x"], s["slots"], pool)
        return dsa.latent_q4_gather(pool, s["slots"])
    if c["op"] == "gather":
        return dsa.latent_q4_gather(s["pool"], s["rows"])
    if c["form"] == "decode":
        return dsa.sparse_mla_attn_q4_decode(s["q"], s["pool"].view(c["T"], c["L"], ROW_BYTES), s["idx"], s["scale"],
                                             want_lse=True)
    if c["form"] == "paged":
        return dsa.sparse_mla_attn_q4_paged(s["q"], s["pool"], s["table"], s["idx"], c["L"], s["scale"], page_size=64,
                                            want_lse=True, split=True)
    if c["form"] == "varlen":
        return dsa.sparse_mla_attn_q4_varlen(s["q"], s["pool"], s["idx"], s["cu_q"], s["cu_k"], s["scale"],
                                             want_lse=True)
    return dsa.sparse_mla_attn_q4(s["q"], s["pool"], s["idx"], s["scale"], want_lse=True)


def _norm(x, residual, weight, group, want_normed):
    h = x.float() if residual is None else x.float() + residual.float()
    y = h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + 1e-6) * weight.float()
    n, d = y.shape
    size = group or d
    g = torch.nn.functional.pad(y, (0, -d % size)).reshape(n, -1, size)
    top = g.abs().amax(dim=2)
    scale = torch.where(top > 0, top / 448, 1.0)
    codes = (g / scale[:, :, None]).clamp(-448, 448).reshape(n, -1)[:, :d].to(torch.float8_e4m3fn)
    out = {"codes": codes.contiguous(), "scale": scale if group else scale.reshape(n)}
    if residual is not None:
        out["sum"] = h.to(x.dtype)
    return out | ({"normed": y.to(x.dtype)} if want_normed else {})


def _pool_rows(s):
    idx = s["idx"].clamp(min=0).long()
    if "table" in s:
        return torch.gather(s["table"].long(), 1, idx // 64) * 64 + idx % 64
    return s["first"][:, None] + idx


def _attn(q, pool, rows, keep, scale):
    t, k = rows.shape
    kv = unpack(pool[rows.reshape(-1)]).reshape(t, k, D_ROW)
    z = torch.matmul(q.float(), kv.transpose(1, 2)) * scale
    z = z.masked_fill(~keep[:, None, :], -math.inf)
    top = z.amax(dim=2, keepdim=True)
    p = torch.exp(z - torch.where(torch.isfinite(top), top, 0.0))
    total = p.sum(dim=2, keepdim=True)
    out = torch.matmul(p, kv[:, :, :D_LATENT]) / torch.where(total > 0, total, 1.0)
    return out.to(torch.bfloat16), (top + torch.log(total))[:, :, 0]


# ---------------------------------------------------------------- the definitions, in 64 bits


def _e4m3(v):
    """The nearest E4M3 values, ties to the even code."""
    e = torch.frexp(v.abs().clamp(min=2.0 ** -6))[1].long() - 1
    step = torch.tensor([2.0 ** (k - 3) for k in range(-6, 10)], dtype=torch.float64, device=v.device)[e + 6]
    return (torch.round(v / step) * step).clamp(-448, 448)


def _nearest_row(x):
    """A row after its way through the cache, from the definition: the first scale that fits, the nearest step."""
    steps = _table()[1].to(x.device)
    lat = x[:, :D_LATENT].double().reshape(x.shape[0], -1, GROUP)
    at = torch.searchsorted(7 * steps, lat.abs().amax(dim=2).contiguous()).clamp(max=255)
    step = steps[at][:, :, None]
    q = torch.round(lat / step).clamp(-7, 7) * step
    return torch.cat([q.reshape(x.shape[0], -1), x[:, D_LATENT:].to(torch.bfloat16).double()], dim=1)


def _table():
    """value - by nibble of a word - of each of the 16 codes, and each scale byte's value, in 64 bits."""
    return (torch.arange(16).double() - 8,
            torch.tensor([(8 + b % 8) / 8 * 2.0 ** (b // 8 - 18) for b in range(256)], dtype=torch.float64))


def _values(b):
    code, step = (t.to(b.device) for t in _table())
    word = b[:, :256].contiguous().view(torch.int32).long() & 0xFFFFFFFF
    v = [code[(word >> (4 * (j // 2 + 4 * (j % 2)))) & 15] for j in range(8)]
    lat = torch.stack(v, dim=2).reshape(b.shape[0], 32, 16) * step[b[:, 256:288].long()][:, :, None]
    return torch.cat([lat.reshape(b.shape[0], -1), b[:, 288:].contiguous().view(torch.bfloat16).double()], dim=1)


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "norm":
        h = s["x"].double()
        if c["residual"]:
            h = h + s["residual"].double()
        y = h / torch.sqrt(h.square().sum(dim=1, keepdim=True) / c["d"] + 1e-6) * s["weight"].double()
        cut = [y] if not c["group"] else list(torch.split(y, c["group"], dim=1))
        scale = torch.stack([p.abs().amax(dim=1) / 448 for p in cut], dim=1)
        scale = torch.where(scale > 0, scale, 1.0)
        codes = torch.cat([_e4m3(p / scale[:, i:i + 1]) for i, p in enumerate(cut)], dim=1)
        out = {"codes": codes, "scale": scale if c["group"] else scale[:, 0]}
        return out | ({"sum": h} if c["residual"] else {}) | ({"normed": y} if c["normed"] else {})
    if c["op"] == "append":
        return torch.where((s["slots"] >= 0)[:, None], _nearest_row(s["x"]), 0.0)
    if c["op"] == "gather":
        return _values(s["pool"][s["rows"].long()])
    rows, out, lse = _pool_rows(s), [], []
    for i in range(c["T"]):
        at = rows[i][s["idx"][i] >= 0]
        if not at.numel():
            out.append(torch.zeros(c["heads"], D_LATENT, dtype=torch.float64, device="cuda"))
            lse.append(torch.full((c["heads"],), -math.inf, dtype=torch.float64, device="cuda"))
            continue
        kv = _values(s["pool"][at])
        z = s["scale"] * (s["q"][i].double() @ kv.T)
        lse.append(torch.logsumexp(z, dim=1))
        out.append(torch.softmax(z, dim=1) @ kv[:, :D_LATENT])
    return torch.stack(out), torch.stack(lse)
