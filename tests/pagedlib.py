"""Plain 64-bit forms of the paged operators, for the tests (no code of the library)."""
import math

import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E2M1_ALL = np.concatenate([E2M1, -E2M1])


def e4m3_half_step(v):
    """Half the distance of e4m3 neighbours at |v| <= 448 (float64 tensor): 2^-4 of the
    power of two below, and that of the subnormals under 2^-6."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    return torch.exp2(e - 4)


def pack_mxf4(rows):
    """[n, 400] uint8 of latent rows [n, 576] (float64 numpy holding bf16 values): 512 e2m1
    codes, the even dim low, 16 e8m0 scales (the smallest power of two with the block's
    largest magnitude at 6 or less), and the 64 last dims as bf16."""
    n = rows.shape[0]
    out = np.zeros((n, 400), np.uint8)
    for r in range(n):
        for b in range(16):
            x = rows[r, 32 * b:32 * b + 32]
            if not np.isfinite(x).all():
                out[r, 256 + b] = 255
                continue
            amax = np.abs(x).max()
            e = -127
            if amax > 0:
                e = max(-127, int(math.floor(math.log2(amax / 6.0))) - 1)
                while amax > 6.0 * 2.0 ** e:
                    e += 1
            out[r, 256 + b] = e + 127
            for i, v in enumerate(x / 2.0 ** e):
                d = np.abs(E2M1 - abs(v))
                best = np.flatnonzero(d == d.min())
                c = int(best[0] if len(best) == 1 or best[0] % 2 == 0 else best[1])
                if math.copysign(1.0, v) < 0:
                    c += 8
                out[r, 16 * b + i // 2] |= c << (4 * (i % 2))
    tail = torch.from_numpy(rows[:, 512:].copy()).bfloat16().view(torch.uint8).numpy()
    out[:, 272:] = tail
    return out


def unpack(cache, kind):
    """float64 latent rows [..., 576] of cache rows (torch, any device)."""
    if kind == "bf16":
        return cache.double()
    if kind == "e4m3":
        codes = cache[..., :512].contiguous().view(torch.float8_e4m3fn).float().double()
        scale = cache[..., 512:528].contiguous().view(torch.float32).double()
        # an fp8 row stands for its values rounded to bf16
        lat = (codes.unflatten(-1, (4, 128)) * scale[..., None]).flatten(-2).bfloat16().double()
        return torch.cat([lat, cache[..., 528:656].contiguous().view(torch.bfloat16).double()], -1)
    b = cache[..., :256]
    lut = torch.tensor(E2M1_ALL, dtype=torch.float64, device=cache.device)
    codes = lut[torch.stack([b & 15, b >> 4], -1).flatten(-2).long()]
    e = cache[..., 256:272].double()
    scale = torch.where(e == 255, math.nan, torch.exp2(e - 127))
    lat = (codes.unflatten(-1, (16, 32)) * scale[..., None]).flatten(-2)
    return torch.cat([lat, cache[..., 272:400].contiguous().view(torch.bfloat16).double()], -1)


def rotate(x, cos, sin, halves):
    """x [n, 64] (float64) turned by the angles of cos, sin [n, 32]."""
    y = x.clone()
    for i in range(32):
        p, q = (i, i + 32) if halves else (2 * i, 2 * i + 1)
        y[:, p] = x[:, p] * cos[:, i] - x[:, q] * sin[:, i]
        y[:, q] = x[:, q] * cos[:, i] + x[:, p] * sin[:, i]
    return y


def paged_rows(table, b, tokens, page):
    """Pool rows of token numbers (1-d long tensor) of sequence b."""
    return table[b, tokens // page].long() * page + tokens % page


def attention(q, kv, scale):
    """(out [H, 512], lse [H], spread [H, 512], zerr [H]) of one query q [H, 576] over
    latent rows kv [n, 576], float64.  spread = sum p |v|, the size that a relative error
    of the probabilities acts on; zerr = max_j scale sum_d |q_d k_jd|, that of the logits."""
    if kv.shape[0] == 0:
        z = q.new_zeros(q.shape[0], 512)
        return z, q.new_full((q.shape[0],), -math.inf), z, q.new_zeros(q.shape[0])
    z = q @ kv.T * scale
    p = torch.softmax(z, -1)
    v = kv[:, :512]
    return p @ v, torch.logsumexp(z, -1), p @ v.abs(), (q.abs() @ kv.abs().T * scale).amax(-1)


def shuffled_table(lens, page, spare, gen, fill=-1):
    """(block table [B, max_pages] int32, pages of the pool): shuffled pages, `spare` of
    them unused; entries past a sequence's pages hold `fill`."""
    need = [-(-n // page) for n in lens]
    order = torch.randperm(sum(need) + spare, generator=gen)
    table = torch.full((len(lens), max(1, max(need))), fill, dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    return table, sum(need) + spare
