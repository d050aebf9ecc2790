"""Plain 64-bit definitions of the 8-bit operators for their tests (numpy, one loop per item)."""
import numpy as np
import torch


def e4m3(y):
    """The e4m3 number nearest to y (float64), ties to the even code, saturating at 448."""
    a = np.abs(y)
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.where(a > 0, a, 1.0))), -6.0) - 3.0)
    return np.clip(np.rint(y / step) * step, -448.0, 448.0)


def scale_of(amax):
    """The smallest 2^e, e in -40 .. 40, with amax <= 448 * 2^e."""
    for e in range(-40, 41):
        if amax <= 448.0 * 2.0 ** e:
            return 2.0 ** e
    return 2.0 ** 40


def quantize(x, block):
    """x float64 [R, C] -> (codes as values [R, C], scale [ceil(C/128), ceil(R/block)])."""
    R, C = x.shape
    q, s = np.zeros_like(x), np.zeros((-(-C // 128), -(-R // block)))
    for t in range(s.shape[0]):
        for r in range(s.shape[1]):
            at = (slice(r * block, (r + 1) * block), slice(128 * t, 128 * t + 128))
            part = x[at]
            if not np.isfinite(part).all():
                part = np.zeros_like(part)
            s[t, r] = scale_of(np.abs(part).max())
            q[at] = e4m3(part / s[t, r])
    return q, s


def append(codes, scale, x, table, lens, n_new):
    """In place on codes (values) [pages, H, page, D] and scale [pages, H]; x [B, H, S, D] float64."""
    pages, H, page, D = codes.shape
    for b in range(x.shape[0]):
        for h in range(H):
            for p in range(table.shape[1]):
                lo, hi = max(lens[b], p * page), min(lens[b] + n_new[b], (p + 1) * page)
                if lens[b] < 0 or lo >= hi or not 0 <= table[b, p] < pages:
                    continue
                new = x[b, h, lo - lens[b]:hi - lens[b]].copy()
                new[~np.isfinite(new).all(1)] = 0.0
                at, held = table[b, p], lo - p * page
                s = scale_of(np.abs(new).max())
                if held:
                    s = max(s, scale[at, h])
                    codes[at, h, :held] = e4m3(codes[at, h, :held] * (scale[at, h] / s))
                codes[at, h, held:hi - p * page] = e4m3(new / s)
                scale[at, h] = s


def attend(q, k, v, ks, vs, table, lens, q_lens, scale, causal):
    """float64 (out, lse, weights [B, H, slots]) and bounds of what bf16 / binary16 / binary32 may be off.

    Bounds, per output: a score is off by at most ds = (D + 4) 2^-23 sum |q k| scale (binary32 sum of
    exact products, one factor); a probability by e^(2 ds) and the 2^-21 of the exponential; its
    binary16 form by 2^-11 more; the sum and product over n tokens by n 2^-24; the bf16 result by
    2^-8 of itself."""
    B, Hq, Sq, D = q.shape
    pages, H, page, _ = k.shape
    G, slots = Hq // H, table.shape[1] * page
    out, lse = np.zeros(q.shape), np.full(q.shape[:3], -np.inf)
    dout, dlse = np.zeros(q.shape), np.zeros(q.shape[:3])
    w, dw = np.zeros((B, H, slots)), np.zeros((B, H, slots))
    for b in range(B):
        n, m = int(np.clip(lens[b], 0, slots)), int(np.clip(q_lens[b], 0, Sq))
        ids = table[b, :-(-n // page)]
        good = np.repeat((ids >= 0) & (ids < pages), page)[:n]
        ids = np.where((ids >= 0) & (ids < pages), ids, 0)
        for h in range(H):
            kk = (k[ids, h] * ks[ids, h][:, None, None]).reshape(-1, D)[:n]
            vv = (v[ids, h] * vs[ids, h][:, None, None]).reshape(-1, D)[:n]
            vv = np.where(good[:, None], vv, 0.0)
            for i in range(m):
                see = good & (np.arange(n) < (n - m + i + 1 if causal else n))
                if not see.any():
                    continue
                for g in range(h * G, h * G + G):
                    s = np.where(see, kk @ q[b, g, i] * scale, -np.inf)
                    ds = (D + 4) * 2.0 ** -23 * (np.abs(kk) @ np.abs(q[b, g, i]))[see].max() * abs(scale)
                    top = s.max()
                    p = np.exp(s - top)
                    tot = p.sum()
                    p /= tot
                    out[b, g, i], lse[b, g, i] = p @ vv, top + np.log(tot)
                    rel = 2 * ds + 2.0 ** -20 + n * 2.0 ** -24 + 2.0 ** -22 * (np.abs(s[see]).max() + abs(lse[b, g, i]))
                    dout[b, g, i] = 2.0 ** -8 * np.abs(out[b, g, i]) + (2.0 ** -11 + 2 * rel) * (p @ np.abs(vv)) \
                        + n * 2.0 ** -35 * np.abs(vv).max()
                    dlse[b, g, i] = rel
                    w[b, h, :n] += p
                    dw[b, h, :n] += p * 2 * rel
    return out, lse, w, dout, dlse, dw


def evict(k, v, ks, vs, table, lens, weights, budget, recent, to):
    """In place on the caches; returns (out_lens, kept weights as a list of arrays per (b, h))."""
    page = k.shape[2]
    kept_w = {}
    for b in range(len(lens)):
        for h in range(k.shape[1]):
            n = int(lens[b])
            kept = list(range(n))
            if n > budget:
                last = min(recent, budget)
                key = [-np.inf if np.isnan(x) else x for x in weights[b, h, :n - last]]
                order = sorted(range(n - last), key=lambda j: (np.isnan(weights[b, h, j]), -key[j], j))
                kept = sorted(order[:budget - last]) + list(range(n - last, n))
            kept_w[b, h] = weights[b, h, kept]
            for codes, scale in ((k, ks), (v, vs)):
                src = [(table[b, j // page], j % page) for j in kept]
                rows = [codes[a, h, r].copy() for a, r in src]
                sc = [scale[a, h] for a, _ in src]
                for p in range(-(-len(kept) // page)):
                    part = range(p * page, min((p + 1) * page, len(kept)))
                    top = max(sc[i] for i in part)
                    for i in part:
                        codes[to[b, p], h, i - p * page] = e4m3(rows[i] * (sc[i] / top))
                    scale[to[b, p], h] = top
    return np.minimum(lens, budget), kept_w


def values(t):
    """A float8 (or any) tensor's values, float64 numpy."""
    return t.detach().float().cpu().numpy().astype(np.float64)


def random_cache(gen, pages, H, page, D, stale_nan=False):
    """float8 codes and power-of-two scales of a filled pool, on the CPU."""
    out = []
    for kind in range(2):
        x = torch.randn(pages, H, page, D, generator=gen) * torch.exp(torch.randn(pages, H, 1, 1, generator=gen))
        if kind == 0:
            x[..., :3] *= 10.0
        s = torch.tensor([scale_of(float(a)) for a in x.abs().amax((2, 3)).reshape(-1)]).view(pages, H)
        out.append(((x / s[:, :, None, None]).to(torch.float8_e4m3fn), s))
    return out[0][0], out[1][0], out[0][1], out[1][1]
