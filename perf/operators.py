"""The paged decode path's operators as measured cases: their plain forms and the library's calls.

Four operators that a serving loop runs around the sparse attention:

``norm``    RMS norm of a layer's input with the residual's addition, and its result in
            bf16 and / or e4m3 with one scale per 128 values
``append``  latent rows and indexer keys written to a paged cache (bf16, e4m3 or 4-bit
            microscaled), with the position rotation applied on the way
``index``   lightning-indexer scores of one query per sequence over paged keys
``attn``    absorbed-MLA sparse attention over a paged latent cache, 4-bit rows included

A case is a dict of plain values; ``prepare`` makes its inputs on the GPU from a seed,
``run`` makes one pass (the plain form in elementary torch operations, or the library's
call where ``own`` is true), ``work`` counts what a pass cannot do without, and ``exact``
computes the same outputs in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
LATENT, ROPE = 512, 64            # a latent row: 512 latent dims, then 64 rotated ones
KV_DIM = LATENT + ROPE
HEADS, KEY_DIM, IDX_HEADS = 16, 128, 64
ROW_BYTES = {"bf16": 1152, "e4m3": 656, "mxf4": 400}
E4M3_MAX = 448.0
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
E2M1_ALL = E2M1 + tuple(-v for v in E2M1)
MAX_POS = 262144


# --------------------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step's layer input, 64 sequences: the latency case
        dict(name="norm_decode", op="norm", rows=64, n=4096, residual=True, y=False, codes=True),
        # a prefill chunk's layer input, kept in bf16 for the residual path and in e4m3
        dict(name="norm_prefill", op="norm", rows=16384, n=7168, residual=True, y=True, codes=True),
        # one new token of 64 sequences: a few hundred kilobytes
        dict(name="append_decode", op="append", rows=64, kv="bf16", k="e4m3", page=64,
             halves=False),
        # a prefill chunk into the 4-bit cache
        dict(name="append_chunk", op="append", rows=8192, kv="mxf4", k="e4m3", page=64,
             halves=False),
        # a long prompt into the 8-bit cache, with the half-split rotation, odd row count
        dict(name="append_prompt", op="append", rows=65521, kv="e4m3", k="bf16", page=32,
             halves=True),
        # the indexer of a single stream, and of a full batch at the 200K context
        dict(name="index_one", op="index", batch=1, ctx=8192, ragged=False, k="bf16", page=64),
        dict(name="index_64x200k", op="index", batch=64, ctx=200000, ragged=False, k="e4m3",
             page=64),
        # a batch of requests of different lengths, one of them empty (a padded slot)
        dict(name="index_ragged", op="index", batch=37, ctx=60001, ragged=True, k="e4m3", page=32),
        # attention of a single stream, and of a full batch at the 200K context, 4-bit cache
        dict(name="attn_one", op="attn", batch=1, rows=1, ctx=8192, ragged=False, topk=2048,
             kv="mxf4", page=64),
        dict(name="attn_64x200k", op="attn", batch=64, rows=1, ctx=200000, ragged=False,
             topk=2048, kv="mxf4", page=64),
        # chunked prefill: 341 query rows of each of three sequences
        dict(name="attn_chunk", op="attn", batch=3, rows=341, ctx=40000, ragged=False, topk=2048,
             kv="mxf4", page=64),
        # ragged decode over the 8-bit cache, an odd top-k, small pages
        dict(name="attn_ragged", op="attn", batch=33, rows=1, ctx=32768, ragged=True, topk=1000,
             kv="e4m3", page=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "append", "index", "attn"))
    if op == "norm":
        n = 8 * _log(rng, 64, 1024)
        rows = min(_log(rng, 1, 16384), 16384 * 7168 // n)
        y = rng.random() < 0.5
        return dict(op=op, rows=rows, n=n, residual=rng.random() < 0.5, y=y,
                    codes=not y or rng.random() < 0.5)
    if op == "append":
        return dict(op=op, rows=_log(rng, 1, 60000), kv=rng.choice(("bf16", "e4m3", "mxf4")),
                    k=rng.choice(("bf16", "e4m3")), page=rng.choice((16, 32, 64, 128)),
                    halves=rng.random() < 0.5)
    ctx, batch = _log(rng, 100, 200000), _log(rng, 1, 64)
    ragged = rng.random() < 0.5 and batch > 1
    if op == "index":
        k = rng.choice(("bf16", "e4m3"))
        return dict(op=op, batch=batch // 2 + 1 if k == "bf16" else batch, ctx=ctx, ragged=ragged,
                    k=k, page=rng.choice((16, 32, 64, 128)))
    rows = 1 if rng.random() < 0.6 else max(1, min(ctx, _log(rng, 2, 1000) // batch))
    return dict(op=op, batch=batch, rows=rows, ctx=ctx, ragged=ragged,
                topk=_log(rng, 16, 2048), kv=rng.choice(("bf16", "e4m3", "mxf4", "mxf4")),
                page=rng.choice((16, 32, 64, 128)))


def _lengths(case):
    """Tokens of each sequence: the context, or (ragged) a spread from 0 up to it."""
    ctx, batch = case["ctx"], case["batch"]
    if not case["ragged"]:
        return [ctx] * batch
    return [int(ctx * ((b * 0.6180339887) % 1.0)) for b in range(batch)]


def work(case):
    op = case["op"]
    if op == "norm":
        e = case["rows"] * case["n"]
        b = 2 * e + 2 * case["n"]
        if case["residual"]:
            b += 4 * e                                 # the residual read, the sum written
        if case["y"]:
            b += 2 * e
        if case["codes"]:
            b += e + 4 * case["rows"] * -(-case["n"] // 128)
        return {"bytes": b, "flops": 6 * e}
    if op == "append":
        row = 2 * KV_DIM + ROW_BYTES[case["kv"]] + 2 * KEY_DIM + 4 + 8 + 4 * ROPE
        row += 2 * KEY_DIM if case["k"] == "bf16" else KEY_DIM + 4
        return {"bytes": row * case["rows"], "flops": 4 * KV_DIM * case["rows"]}
    lens = _lengths(case)
    tokens = sum(lens)
    if op == "index":
        key = 2 * KEY_DIM if case["k"] == "bf16" else KEY_DIM + 4
        q = IDX_HEADS * (2 * KEY_DIM + 4 if case["k"] == "bf16" else KEY_DIM + 8)
        return {"bytes": tokens * (key + 4) + case["batch"] * q + 4 * tokens // case["page"],
                "flops": 2 * IDX_HEADS * KEY_DIM * tokens}
    pairs = sum(min(case["topk"], max(0, n - case["rows"] + r + 1))
                for n in lens for r in range(case["rows"]))
    queries = case["batch"] * case["rows"]
    # each selected row of a query read once, except that no more rows can come from
    # memory than the cache holds
    rows = min(pairs, tokens)
    return {"bytes": rows * ROW_BYTES[case["kv"]] + queries * (HEADS * (KV_DIM + LATENT) * 2 +
                                                               HEADS * 4 + 4 * case["topk"]),
            "flops": 2 * HEADS * (KV_DIM + LATENT) * pairs}


# --------------------------------------------------------------------------- the inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device=DEV) * std


def _rope_table():
    """cos | sin of position * 10000^(-i / 32), i = 0..31: what a program keeps per model."""
    inv = 10000.0 ** (-torch.arange(ROPE // 2, device=DEV, dtype=torch.float64) / (ROPE // 2))
    ang = torch.arange(MAX_POS, device=DEV, dtype=torch.float64)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], dim=1).float()


def _latent_rows(g, rows):
    """Latent rows as a model's cache sees them: normalised dims with a per-channel gain."""
    gain = torch.rand(KV_DIM, generator=g, device=DEV) + 0.5
    return (_normal(g, rows, KV_DIM) * gain).bfloat16()


def _pages(g, lens, page):
    """A block table over a shuffled pool: pages of every sequence, and the pool's pages."""
    need = [-(-n // page) for n in lens]
    total = sum(need) + 3
    order = torch.randperm(total, generator=g, device=DEV).int()
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    return table, total


def _pool(g, total_rows, make):
    """A cache of total_rows rows drawn from up to 32768 distinct ones (rows are far apart)."""
    distinct = min(total_rows, 32768)
    rows = make(distinct)
    if total_rows == distinct:
        return rows
    pick = torch.randint(0, distinct, (total_rows,), generator=g, device=DEV)
    return tuple(r.index_select(0, pick) for r in rows)


def _prepare_norm(case, g):
    rows, n = case["rows"], case["n"]
    s = {"x": _normal(g, rows, n).bfloat16(),
         "weight": (1 + 0.1 * _normal(g, n)).bfloat16(), "eps": 1e-6}
    if case["residual"]:
        s["residual"] = _normal(g, rows, n, std=4.0).bfloat16()
        s["h"] = torch.zeros(rows, n, dtype=torch.bfloat16, device=DEV)
    if case["y"]:
        s["y"] = torch.zeros(rows, n, dtype=torch.bfloat16, device=DEV)
    if case["codes"]:
        s["codes"] = torch.zeros(rows, n, dtype=torch.uint8, device=DEV)
        s["scales"] = torch.zeros(rows, -(-n // 128), device=DEV)
    return s


def _prepare_append(case, g):
    rows, page = case["rows"], case["page"]
    pool = -(-(rows + rows // 4 + 1) // page) * page
    s = {"kv": _latent_rows(g, rows), "k": _normal(g, rows, KEY_DIM).bfloat16(),
         "rope": _rope_table(), "halves": case["halves"],
         "pos": torch.randint(0, MAX_POS, (rows,), generator=g, device=DEV, dtype=torch.int32),
         "slots": torch.randperm(pool, generator=g, device=DEV)[:rows]}
    if case["kv"] == "bf16":
        s["kv_cache"] = torch.zeros(pool, KV_DIM, dtype=torch.bfloat16, device=DEV)
    else:
        s["kv_cache"] = torch.zeros(pool, ROW_BYTES[case["kv"]], dtype=torch.uint8, device=DEV)
    if case["k"] == "bf16":
        s["k_cache"] = torch.zeros(pool, KEY_DIM, dtype=torch.bfloat16, device=DEV)
        s["k_scale"] = None
    else:
        s["k_cache"] = torch.zeros(pool, KEY_DIM, dtype=torch.uint8, device=DEV)
        s["k_scale"] = torch.zeros(pool, device=DEV)
    return s


def _prepare_index(case, g):
    lens, page, batch = _lengths(case), case["page"], case["batch"]
    table, pages = _pages(g, lens, page)
    std = KEY_DIM ** -0.5
    q = _normal(g, batch, 1, IDX_HEADS, KEY_DIM, std=std).bfloat16()
    s = {"w": torch.rand(batch, 1, IDX_HEADS, generator=g, device=DEV) / 8, "table": table,
         "lens": torch.tensor(lens, dtype=torch.int32, device=DEV), "page": page,
         "scores": torch.zeros(batch, case["ctx"], device=DEV), "q_scale": None, "k_scale": None}
    if case["k"] == "bf16":
        s["q"] = q
        (s["k_cache"],) = _pool(g, pages * page,
                                lambda m: (_normal(g, m, KEY_DIM, std=std).bfloat16(),))
    else:
        s["q"], s["q_scale"] = _to_e4m3(q.float(), KEY_DIM)
        s["q_scale"] = s["q_scale"][..., 0].contiguous()
        s["k_cache"], ks = _pool(g, pages * page,
                                 lambda m: _to_e4m3(_normal(g, m, KEY_DIM, std=std), KEY_DIM))
        s["k_scale"] = ks[:, 0].contiguous()
    return s


def _prepare_attn(case, g):
    lens, page, batch, rows = _lengths(case), case["page"], case["batch"], case["rows"]
    topk = case["topk"]
    table, pages = _pages(g, lens, page)
    pack = {"bf16": lambda x: x.bfloat16(), "e4m3": _pack_e4m3, "mxf4": _pack_mxf4}[case["kv"]]
    (cache,) = _pool(g, pages * page, lambda m: (pack(_latent_rows(g, m).float()),))
    # ascending index sets: one position out of each of k equal stretches of the
    # row's causal context; every position, then -1, where the context is shorter
    n = (torch.tensor(lens, device=DEV)[:, None] - rows + 1 +
         torch.arange(rows, device=DEV)).clamp(min=0)[..., None]
    j = torch.arange(topk, device=DEV)
    lo, hi = j * n // topk, (j + 1) * n // topk
    u = torch.rand(batch, rows, topk, generator=g, device=DEV)
    spread = lo + torch.minimum((u * (hi - lo)).long(), (hi - lo - 1).clamp(min=0))
    idx = torch.where(n > topk, spread, torch.where(j < n, j, -1)).int()
    return {"q": _normal(g, batch, rows, HEADS, KV_DIM).bfloat16(), "kv_cache": cache,
            "kv": case["kv"], "idx": idx, "table": table, "page": page,
            "lens": torch.tensor(lens, dtype=torch.int32, device=DEV),
            "scale": KV_DIM ** -0.5,
            "out": torch.zeros(batch, rows, HEADS, LATENT, dtype=torch.bfloat16, device=DEV),
            "lse": torch.zeros(batch, rows, HEADS, device=DEV),
            # the partial results of split queries; a program keeps one for its largest batch
            "workspace": torch.empty(64 << 20, dtype=torch.uint8, device=DEV)}


def prepare(case, seed):
    s = globals()["_prepare_" + case["op"]](case, _gen(seed))
    s["op"] = case["op"]
    return s


# --------------------------------------------------------------------------- plain forms
def _to_e4m3(x, group):
    """uint8 codes and fp32 scales (amax / 448, 1 for a zero group) of groups of x's last dim."""
    n = x.shape[-1]
    m = -(-n // group)
    g = torch.nn.functional.pad(x, (0, m * group - n)).unflatten(-1, (m, group))
    amax = g.abs().amax(-1)
    scale = torch.where(amax > 0, amax / E4M3_MAX, 1.0)
    codes = (g / scale[..., None]).to(torch.float8_e4m3fn).flatten(-2)[..., :n]
    return codes.view(torch.uint8).contiguous(), scale


def _bytes(x):
    return x.contiguous().view(torch.uint8)


def _pack_e4m3(x):
    """656-byte rows: 512 e4m3 codes, four fp32 scales, 64 rope dims in bf16."""
    codes, scale = _to_e4m3(x[:, :LATENT], 128)
    return torch.cat([codes, _bytes(scale), _bytes(x[:, LATENT:].bfloat16())], dim=1)


def _pack_mxf4(x):
    """400-byte rows: 512 e2m1 codes (two a byte, the even dim low), 16 e8m0 scales of 32
    dims each, 64 rope dims in bf16.  The scale is the smallest power of two that puts the
    block's largest magnitude at 6 or less."""
    g = x[:, :LATENT].unflatten(1, (16, 32))
    amax = g.abs().amax(-1)
    field = (amax.view(torch.int32) + 0x3FFFFF) >> 23
    e = (field - 2).clamp(min=0)
    a = torch.ldexp(g.abs(), (127 - e)[..., None])
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75).to(torch.uint8) + (a > 1.25).to(torch.uint8) +
            (a >= 1.75).to(torch.uint8) + (a > 2.5).to(torch.uint8) +
            (a >= 3.5).to(torch.uint8) + (a > 5.0).to(torch.uint8))
    code = (code + 8 * torch.signbit(g).to(torch.uint8)).flatten(1)
    return torch.cat([code[:, 0::2] + 16 * code[:, 1::2], e.to(torch.uint8),
                      _bytes(x[:, LATENT:].bfloat16())], dim=1)


def _unpack(cache, kind):
    """fp32 latent rows [..., 576] of cache rows (an e4m3 row stands for bf16 values)."""
    if kind == "bf16":
        return cache.float()
    if kind == "e4m3":
        codes = cache[..., :LATENT].contiguous().view(torch.float8_e4m3fn).float()
        scale = cache[..., LATENT:LATENT + 16].contiguous().view(torch.float32)
        lat = (codes.unflatten(-1, (4, 128)) * scale[..., None]).flatten(-2).bfloat16().float()
        return torch.cat([lat, cache[..., 528:656].contiguous().view(torch.bfloat16).float()], -1)
    lut = torch.tensor(E2M1_ALL, device=cache.device)
    b = cache[..., :256]
    codes = torch.stack([lut[(b & 15).int()], lut[(b >> 4).int()]], -1).flatten(-2)
    scale = torch.ldexp(torch.ones((), device=cache.device), cache[..., 256:272].int() - 127)
    lat = (codes.unflatten(-1, (16, 32)) * scale[..., None]).flatten(-2)
    return torch.cat([lat, cache[..., 272:400].contiguous().view(torch.bfloat16).float()], -1)


def _rotate(x, cs, halves):
    """x [rows, 64] rotated by the angles whose cos | sin are cs [rows, 64]."""
    c, s = cs[:, :ROPE // 2], cs[:, ROPE // 2:]
    if halves:
        a, b = x[:, :ROPE // 2], x[:, ROPE // 2:]
        return torch.cat([a * c - b * s, b * c + a * s], dim=1)
    a, b = x[:, 0::2], x[:, 1::2]
    return torch.stack([a * c - b * s, b * c + a * s], -1).flatten(1)


def _plain_norm(s):
    h = s["x"].float()
    if "residual" in s:
        h = h + s["residual"].float()
        s["h"].copy_(h)
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + s["eps"]) * s["weight"].float()
    if "y" in s:
        s["y"].copy_(y)
    if "codes" in s:
        s["codes"][:], s["scales"][:] = _to_e4m3(y, 128)


def _plain_append(s):
    cs = s["rope"][s["pos"]]
    kv, k = s["kv"].float(), s["k"].float()
    kv = torch.cat([kv[:, :LATENT], _rotate(kv[:, LATENT:], cs, s["halves"])], dim=1)
    k = torch.cat([_rotate(k[:, :ROPE], cs, s["halves"]), k[:, ROPE:]], dim=1)
    width = s["kv_cache"].shape[1]
    rows = (kv.bfloat16() if width == KV_DIM else
            _pack_e4m3(kv) if width == ROW_BYTES["e4m3"] else _pack_mxf4(kv))
    s["kv_cache"][s["slots"]] = rows
    if s["k_scale"] is None:
        s["k_cache"][s["slots"]] = k.bfloat16()
    else:
        codes, scale = _to_e4m3(k, KEY_DIM)
        s["k_cache"][s["slots"]] = codes
        s["k_scale"][s["slots"]] = scale[:, 0]


def _slots(table, pos, page):
    """Cache rows of positions pos [B, ...] (0 where the position has none)."""
    p = pos.clamp(min=0).long()
    got = table.gather(1, (p // page).clamp(max=table.shape[1] - 1).flatten(1)).view(p.shape)
    return (got.clamp(min=0).long() * page + p % page).clamp(min=0)


def _plain_index(s):
    q, k = s["q"], s["k_cache"]
    n = s["scores"].shape[1]
    pos = torch.arange(n, device=q.device).expand(q.shape[0], n)
    rows = _slots(s["table"], pos, s["page"])
    w = s["w"][:, 0]
    if s["k_scale"] is None:
        q, keys = q.float(), k[rows].float()
    else:
        q = q.view(torch.float8_e4m3fn).float()
        keys = k[rows].view(torch.float8_e4m3fn).float()
        w = w * s["q_scale"][:, 0]
    dots = torch.relu(torch.matmul(keys, q[:, 0].transpose(1, 2)))       # [B, n, heads]
    score = torch.matmul(dots, w[..., None])[..., 0]
    if s["k_scale"] is not None:
        score = score * s["k_scale"][rows]
    s["scores"].copy_(torch.where(pos < s["lens"][:, None], score, s["scores"]))


def _plain_attn(s):
    idx, lens = s["idx"], s["lens"][:, None, None]
    valid = (idx >= 0) & (idx < lens)
    kv = _unpack(s["kv_cache"][_slots(s["table"], idx, s["page"])], s["kv"])  # [B, R, k, 576]
    z = torch.matmul(s["q"].float(), kv.transpose(-1, -2)) * s["scale"]
    z = z.masked_fill(~valid[:, :, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    p = torch.exp(z - top.clamp(min=-3e38))
    total = p.sum(-1, keepdim=True)
    s["out"].copy_(torch.matmul(p / total.clamp(min=1e-30), kv[..., :LATENT]))
    s["lse"].copy_((top + torch.log(total))[..., 0])


# --------------------------------------------------------------------------- one pass
def _outputs(s):
    """Everything a pass writes.  8-bit codes and scales come as the values they stand for;
    4-bit codes as their bytes, which are compared bit for bit."""
    f8 = torch.float8_e4m3fn
    if s["op"] == "norm":
        out = {name: s[name] for name in ("h", "y", "scales") if name in s}
        if "codes" in s:
            out["codes"] = s["codes"].view(f8)
        return out
    if s["op"] == "append":
        c = s["kv_cache"]
        if c.shape[1] == KV_DIM:
            out = {"kv": c}
        elif c.shape[1] == ROW_BYTES["e4m3"]:
            out = {"codes": c[:, :512].view(f8), "scales": c[:, 512:528].view(torch.float32),
                   "rope": c[:, 528:].view(torch.bfloat16)}
        else:
            out = {"codes": c[:, :256], "scales": c[:, 256:272].view(torch.float8_e8m0fnu),
                   "rope": c[:, 272:].view(torch.bfloat16)}
        out["k"] = s["k_cache"] if s["k_scale"] is None else s["k_cache"].view(f8)
        if s["k_scale"] is not None:
            out["k_scale"] = s["k_scale"]
        return out
    if s["op"] == "index":
        return {"scores": s["scores"]}
    return {"out": s["out"], "lse": s["lse"]}


def _own_pass(s):
    from sparse_attention_indexer_sum_b200 import binding as ic
    kinds = {"bf16": ic.IC_BF16, "e4m3": ic.IC_E4M3, "mxf4": ic.IC_MXF4}
    if s["op"] == "norm":
        ic.ic_rms_norm(s["x"], s["weight"], s["eps"], residual=s.get("residual"), h=s.get("h"),
                       y=s.get("y"), codes=s.get("codes"), scales=s.get("scales"))
    elif s["op"] == "append":
        width = s["kv_cache"].shape[1]
        kind = next(k for k, b in ROW_BYTES.items()
                    if b == width * s["kv_cache"].element_size())
        ic.ic_cache_append(s["slots"], kv=s["kv"], kv_cache=s["kv_cache"], kv_dtype=kinds[kind],
                           k=s["k"], k_cache=s["k_cache"], k_scale=s["k_scale"], pos=s["pos"],
                           rope=s["rope"], kv_halves=s["halves"], k_halves=s["halves"])
    elif s["op"] == "index":
        ic.ic_indexer_scores_paged(s["q"], s["k_cache"], s["w"], s["table"], s["lens"],
                                   page_size=s["page"], q_scale=s["q_scale"],
                                   k_scale=s["k_scale"], scores=s["scores"])
    else:
        ic.ic_sparse_attn_paged(s["q"], s["kv_cache"], s["idx"], s["table"], s["lens"],
                                s["scale"], page_size=s["page"], kv_dtype=kinds[s["kv"]],
                                out=s["out"], lse=s["lse"], workspace=s["workspace"])


def run(state):
    if own:
        _own_pass(state)
    else:
        globals()["_plain_" + state["op"]](state)
    return _outputs(state)


# --------------------------------------------------------------------------- in 64 bits
def _grid_e4m3(v):
    """v (float64) at the nearest e4m3 value, ties to the even code."""
    exp = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -40))).clamp(min=-6)
    step = torch.exp2(exp - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_quant(v, group):
    n = v.shape[-1]
    m = -(-n // group)
    g = torch.nn.functional.pad(v, (0, m * group - n)).reshape(*v.shape[:-1], m, group)
    scale = g.abs().amax(-1) / E4M3_MAX
    scale[scale == 0] = 1.0
    return _grid_e4m3(g / scale[..., None]).reshape(*v.shape[:-1], m * group)[..., :n], scale


def _exact_norm(s):
    h = s["x"].double()
    out = {}
    if "residual" in s:
        h = h + s["residual"].double()
        out["h"] = h
    y = s["weight"].double() * h / (h.pow(2).sum(-1, keepdim=True) / h.shape[-1] +
                                    s["eps"]).sqrt()
    if "y" in s:
        out["y"] = y
    if "codes" in s:
        out["codes"], out["scales"] = _exact_quant(y, 128)
    return out


def _exact_append(s):
    half = ROPE // 2
    ang = s["pos"].double()[:, None] * 10000.0 ** (-torch.arange(half, device=DEV).double() / half)
    turn = torch.polar(torch.ones_like(ang), ang)       # rotation as complex numbers

    def rotated(x):
        x = x.double()
        z = (torch.complex(x[:, :half], x[:, half:]) if s["halves"] else
             torch.view_as_complex(x.reshape(-1, half, 2).contiguous())) * turn
        return torch.cat([z.real, z.imag], 1) if s["halves"] else torch.view_as_real(z).flatten(1)

    def placed(rows):
        full = torch.zeros(s["kv_cache"].shape[0], *rows.shape[1:], dtype=torch.float64,
                           device=DEV)
        full[s["slots"]] = rows.double()
        return full

    lat, rope = s["kv"][:, :LATENT].double(), rotated(s["kv"][:, LATENT:])
    key = torch.cat([rotated(s["k"][:, :ROPE]), s["k"][:, ROPE:].double()], 1)
    width = s["kv_cache"].shape[1]
    if width == KV_DIM:
        out = {"kv": placed(torch.cat([lat, rope], 1))}
    elif width == ROW_BYTES["e4m3"]:
        codes, scale = _exact_quant(lat, 128)
        out = {"codes": placed(codes), "scales": placed(scale), "rope": placed(rope)}
    else:
        peak = lat.reshape(-1, 16, 32).abs().amax(-1)
        scale = torch.exp2(torch.ceil(torch.log2(peak.clamp(min=1e-37) / 6)))
        full = placed(scale)
        full[full == 0] = 2.0 ** -127                    # a byte of 0, as the cache starts
        out = {"codes": None, "scales": full, "rope": placed(rope)}
    if s["k_scale"] is None:
        out["k"] = placed(key)
    else:
        codes, scale = _exact_quant(key, KEY_DIM)
        out["k"], out["k_scale"] = placed(codes), placed(scale[:, 0])
    return out


def _exact_index(s):
    scores = s["scores"].double()
    for b, n in enumerate(s["lens"].tolist()):
        t = torch.arange(n, device=DEV)
        at = s["table"][b, t // s["page"]].long() * s["page"] + t % s["page"]
        q, w, keys = s["q"][b, 0], s["w"][b, 0].double(), s["k_cache"][at]
        if s["k_scale"] is not None:
            f8 = torch.float8_e4m3fn
            q = q.view(f8).double() * s["q_scale"][b, 0].double()[:, None]
            keys = keys.view(f8).double() * s["k_scale"][at].double()[:, None]
        scores[b, :n] = w @ (q.double() @ keys.double().T).clamp(min=0)
    return {"scores": scores}


def _exact_rows(s, at):
    """The latent rows at cache rows `at` in 64 bits."""
    c = s["kv_cache"][at]
    if s["kv"] == "bf16":
        return c.double()
    if s["kv"] == "e4m3":
        v = c[:, :512].contiguous().view(torch.float8_e4m3fn).double()
        v = v * c[:, 512:528].contiguous().view(torch.float32).double().repeat_interleave(128, 1)
        lat, tail = v.bfloat16().double(), c[:, 528:656]
    else:
        b = torch.stack([c[:, :256] & 15, c[:, :256] >> 4], 2).reshape(-1, 512).long()
        lat = torch.tensor(E2M1_ALL, dtype=torch.float64, device=DEV)[b]
        lat = lat * torch.exp2(c[:, 256:272].double() - 127).repeat_interleave(32, 1)
        tail = c[:, 272:400]
    return torch.cat([lat, tail.contiguous().view(torch.bfloat16).double()], 1)


def _exact_attn(s):
    out, lse = s["out"].double(), s["lse"].double()
    for b, n in enumerate(s["lens"].tolist()):
        for r in range(s["idx"].shape[1]):
            t = s["idx"][b, r].long()
            t = t[(t >= 0) & (t < n)]
            if t.numel() == 0:
                out[b, r], lse[b, r] = 0.0, -math.inf
                continue
            rows = _exact_rows(s, s["table"][b, t // s["page"]].long() * s["page"] + t % s["page"])
            z = s["q"][b, r].double() @ rows.T * s["scale"]
            lse[b, r] = torch.logsumexp(z, 1)
            out[b, r] = torch.softmax(z, 1) @ rows[:, :LATENT]
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    return globals()["_exact_" + case["op"]](s)
