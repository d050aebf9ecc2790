"""Attention over the e4m3 KV cache where the pages' scales are far apart, tiny or no powers of two, for
few rows (up to 32 a key head) and many: the bounds hold for every row on the slots that this row
sees, so a loud page may cost a row that does not look at it nothing."""
import numpy as np
import pytest
import torch

import kv8_oracle as K

pytestmark = pytest.mark.gpu

ROWS = [8, 32, 33, 200, 300]  # a key head's rows: units of 8, of 16, and of 256 (one tile, two, two units)


@pytest.fixture(scope="module")
def hq():
    import post_quantization_tile_b200 as m
    m.lib()
    return m


def make(hq, seed, pages, page, D, k_exp=None, v_exp=None):
    """(cache, its parts in 64 bits, the table) of one sequence and head; page i has scales 2^k_exp[i], 2^v_exp[i]
    and codes over e4m3's whole range."""
    g = torch.Generator().manual_seed(seed)
    order = torch.randperm(pages, generator=g)
    parts = []
    for exp in (k_exp, v_exp):
        mant = torch.randint(0, 2, (pages, 1, page, D), generator=g) * 0x80 + torch.randint(0, 0x7F, (pages, 1, page, D), generator=g)
        s = torch.ones(pages, 1) * 2.0 ** -8
        if exp is not None:
            s[order, 0] = torch.tensor(exp, dtype=torch.float64).exp2().float()
        parts.append((mant.to(torch.uint8), s))
    (k, ks), (v, vs) = parts
    cache = hq.Kv8Cache(k.cuda().view(hq.FP8), v.cuda().view(hq.FP8), ks.cuda(), vs.cuda())
    return cache, order.to(torch.int32).view(1, pages)


def check(hq, cache, table, n, q, scale=None, causal=True, weights=False):
    """Attention of q [1, G, m, D] against the formula in 64 bits.  Bounds: a score is off by (D + 4) roundings of its
    sum of magnitudes, a probability by that and its exponential, its binary16 form by half a step: 2^-11
    of itself, or 2^-32 of the row's largest where that is more (binary16 ends at 2^-24 and the largest stands
    at 2^7 or above) but never more than itself; the result by half a step of bf16."""
    G, m, D = q.shape[1:]
    page = cache.k.shape[2]
    sc = D ** -0.5 if scale is None else scale
    out, lse = torch.empty_like(q, memory_format=torch.contiguous_format), torch.empty(1, G, m, device="cuda")
    w = torch.empty(1, 1, table.shape[1] * page, device="cuda") if weights else None
    hq.kv8_attend(q, cache, table.cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"), scale=scale, causal=causal, out=out, lse=lse,
                  weights=w)
    ids = table[0].long().numpy()
    k, v = ((K.values(c)[ids, 0] * K.values(s)[ids, 0][:, None, None]).reshape(-1, D)[:n]
            for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
    got, got_lse, total, dtotal = K.values(out)[0], K.values(lse)[0], np.zeros(n), np.zeros(n)
    for h in range(G):
        for i in range(m):
            see = min(n, max(0, n - m + i + 1)) if causal else n
            if see == 0:
                assert np.all(got[h, i] == 0.0) and got_lse[h, i] == -np.inf
                continue
            x = K.values(q)[0, h, i]
            s = k[:see] @ x * sc
            p = np.exp(s - s.max())
            l = s.max() + np.log(p.sum())
            step = np.minimum(p, 2.0 ** -32) / p.sum()
            p /= p.sum()
            rel = 2 * (D + 4) * 2.0 ** -23 * (np.abs(k[:see]) @ np.abs(x)).max() * abs(sc) + 2.0 ** -20 + n * 2.0 ** -24 \
                + 2.0 ** -22 * (np.abs(s).max() + abs(l))
            ref = p @ v[:see]
            tol = 2.0 ** -8 * np.abs(ref) + ((2.0 ** -11 + 2 * rel) * p + step) @ np.abs(v[:see])
            err = np.abs(got[h, i] - ref)
            assert np.all(err <= tol), (h, i, float((err / tol).max()))
            assert abs(got_lse[h, i] - l) <= rel
            total[:see] += p
            dtotal[:see] += 2 * rel * p
    if weights:
        assert np.all(np.abs(K.values(w)[0, 0, :n] - total) <= dtotal + 2.0 ** -22 * total)


def queries(seed, G, m, D):
    return torch.randn(1, G, m, D, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("far", [15, 16, 20, 22, 23, 25, 30, 50, 80])
@pytest.mark.parametrize("rows", ROWS)
def test_quiet_pages_before_a_loud_one(hq, rows, far, D):
    """Early rows of a causal chunk see quiet pages of small codes only, late rows a loud one too."""
    low = max(-40, -20 - far // 2)
    cache, table = make(hq, far, 8, 64, D, k_exp=[-9] * 8, v_exp=[low] * 7 + [low + far])
    cache.v.view(torch.uint8)[table[0, :7].long().cuda()] &= 0x83
    n = 448 + min(16, rows - 1)
    check(hq, cache, table, n, queries(rows, 1, rows, D))
    check(hq, cache, table, n, queries(rows, 1, rows, D), causal=False)


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("rows", ROWS)
def test_loud_pages_that_nobody_looks_at(hq, rows, page):
    """Pages of every loudness by turns; only the quiet ones' keys meet the queries, the others get
    probabilities far below binary16."""
    exps = [(-40, -3, 33, -22, 10)[i % 5] for i in range(640 // page)]
    cache, table = make(hq, page, len(exps), page, 64, k_exp=[-12] * len(exps), v_exp=exps)
    q = queries(rows, 1, rows, 64)
    q[..., 0] = 64.0
    keys = cache.k.view(torch.uint8)
    for quiet in (-40, -22, 10):
        for i, e in enumerate(exps):
            keys[int(table[0, i]), :, :, 0] = 0x00 if e == quiet else 0xFE  # 0 or -448: 64 * -448 * 2^-12 / 8 is 0.9
        check(hq, cache, table, 620, q, scale=20.0)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("rows", ROWS)
def test_scales_that_are_no_powers_of_two(hq, rows, causal):
    cache, table = make(hq, 5, 10, 32, 128, k_exp=np.linspace(-9.7, -8.1, 10), v_exp=np.linspace(-11.3, 9.9, 10))
    check(hq, cache, table, 310, queries(rows, 1, rows, 128), causal=causal)
    check(hq, cache, table, 1, queries(rows, 1, rows, 128), causal=causal)  # one slot: its values come back


@pytest.mark.parametrize("k_exp", [-40, -27, 0])
@pytest.mark.parametrize("rows", ROWS)
def test_scores_whose_factor_vanishes_in_binary32(hq, rows, k_exp):
    """scale 0, tiny scales and tiny queries against pages of tiny (or zero) keys that a causal row sees in part."""
    cache, table = make(hq, 7, 6, 64, 64, k_exp=[k_exp] * 6)
    for scale, up in ((0.0, 1.0), (-0.0, 1.0), (1e-38, 1.0), (0.125, 2.0 ** -100), (0.125, 0.0), (-0.125, 2.0 ** -126)):
        q = (queries(rows, 1, rows, 64).float() * up).to(torch.bfloat16)
        check(hq, cache, table, 333, q, scale=scale, weights=True)
        cache.k.view(torch.uint8)[int(table[0, 4])] = 0


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("rows,G", [(40, 1), (40, 4), (300, 1)])
def test_many_units_of_unlike_windows(hq, rows, G, causal, page):
    """More units than thread blocks, of one to three tiles, whose pages span one to four windows: a thread block goes
    through several, with and without a second row tile.  The formula in 64 bits on the GPU, the bounds of check()."""
    B, H, D, P = 60, 5, 64, 384 // page
    g = torch.Generator().manual_seed(rows + page)
    pages = B * P
    codes = [(torch.randint(0, 2, (pages, H, page, D), generator=g) * 0x80 + torch.randint(0, 0x7F, (pages, H, page, D), generator=g))
             .to(torch.uint8) for _ in range(2)]
    wide = torch.tensor([0.0, 11.0, 25.0, 40.0])[torch.randint(0, 4, (pages, H), generator=g)]  # octaves either way
    vs = torch.exp2(torch.round((2 * torch.rand(pages, H, generator=g) - 1) * wide))
    vs = torch.where(torch.rand(pages, H, generator=g) < 0.1, vs * 0.75, vs).clamp(2.0 ** -40, 2.0 ** 40)
    cache = hq.Kv8Cache(codes[0].cuda().view(hq.FP8), codes[1].cuda().view(hq.FP8), torch.full((pages, H), 2.0 ** -8).cuda(), vs.cuda())
    table = torch.randperm(pages, generator=g).to(torch.int32).view(B, P).cuda()
    lens = torch.randint(0, 385, (B,), generator=g, dtype=torch.int32).cuda()
    m = torch.randint(0, rows + 1, (B,), generator=g, dtype=torch.int32).cuda()
    q = torch.randn(B, H * G, rows, D, generator=g).to(torch.bfloat16).cuda()
    out, lse = torch.full_like(q, 7.0), torch.full((B, H * G, rows), 7.0, device="cuda")
    hq.kv8_attend(q, cache, table, lens, q_lens=m, causal=causal, out=out, lse=lse)
    ids = table.long()
    k, v = ((c.double() * s.double()[:, :, None, None])[ids].transpose(1, 2).reshape(B, H, 384, D)
            for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
    i, j = torch.arange(rows, device="cuda"), torch.arange(384, device="cuda")
    n, mm = lens[:, None, None].long(), m[:, None, None].long()
    sees = (j < n) & (j <= i[None, :, None] + (n - mm)) if causal else (j < n).expand(B, rows, 384)
    for h in range(H * G):
        x, kk, vv = q[:, h].double(), k[:, h // G], v[:, h // G]
        s = torch.where(sees, x @ kk.transpose(1, 2) * D ** -0.5, -torch.inf)
        top = s.amax(2, keepdim=True)
        some = torch.isfinite(top)
        p = torch.exp(s - torch.where(some, top, 0.0))
        total = p.sum(2, keepdim=True)
        step = torch.where(p > 0, p.clamp(max=2.0 ** -32), 0.0) / total.clamp(min=1e-300)
        p = p / total.clamp(min=1e-300)
        size = torch.where(sees, x.abs() @ kk.abs().transpose(1, 2), 0.0).amax(2, keepdim=True)
        ref_lse = torch.where(some, top + torch.log(total.clamp(min=1e-300)), -torch.inf)[:, :, 0]
        big = torch.where(sees, s.abs(), 0.0).amax(2, keepdim=True) + torch.where(some, ref_lse[:, :, None].abs(), 0.0)
        rel = 2 * (D + 4) * 2.0 ** -23 * size * D ** -0.5 + 2.0 ** -20 + 384 * 2.0 ** -24 + 2.0 ** -22 * big
        ref = p @ vv
        tol = 2.0 ** -8 * ref.abs() + ((2.0 ** -11 + 2 * rel) * p + step) @ vv.abs()
        asked = (i < mm[:, 0])
        err = (out[:, h].double() - ref).abs()
        assert torch.all((err <= tol) | ~asked[:, :, None]), float(((err / tol.clamp(min=1e-300)) * asked[:, :, None]).max())
        assert torch.all((out[:, h] == 7.0) | asked[:, :, None]) and torch.all((lse[:, h] == 7.0) | asked)
        got = lse[:, h].double()
        assert torch.all((got == ref_lse) | ((got - ref_lse).abs() <= rel[:, :, 0]) | ~asked)
