"""The e4m3 KV cache on the GPU against plain 64-bit definitions: append and evict code for code,
attention within bounds derived from its roundings (kv8_oracle.attend), at the lengths, masks,
page sizes, strides and head layouts where it can go wrong; then a run of all operators together."""
import numpy as np
import pytest
import torch

import kv8_oracle as K

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hq():
    import post_quantization_tile_b200 as m
    m.lib()
    return m


def gen(seed):
    return torch.Generator().manual_seed(seed)


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def setup_cache(hq, g, B, P, H, page, D, spare=2):
    """(cache on the GPU, its parts as float64 numpy, table numpy)"""
    pages = B * P + spare
    k, v, ks, vs = K.random_cache(g, pages, H, page, D)
    table = torch.randperm(pages, generator=g)[:B * P].view(B, P).to(torch.int32)
    cache = hq.Kv8Cache(k.cuda(), v.cuda(), ks.cuda(), vs.cuda())
    return cache, [K.values(t) for t in (k, v, ks, vs)], table.numpy()


def check_attend(hq, B, H, G, Sq, D, page, lens, q_lens=None, causal=True, scale=None, seed=0, weights=True, P=None,
                 change=None, strided=True):
    g = gen(seed)
    P = P or max(1, -(-max(max(lens), 1) // page))
    cache, (k, v, ks, vs), table = setup_cache(hq, g, B, P, H, page, D)
    ql = [Sq] * B if q_lens is None else q_lens
    q = torch.randn(B, Sq, H * G, D, generator=g).to(torch.bfloat16).cuda().transpose(1, 2)
    if not strided:
        q = q.contiguous()
    if change:
        table = change(cache, k, v, table)
    L = P * page
    out = torch.full((B, Sq, H * G, D), 7.0, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    lse = torch.full((B, H * G, Sq), 7.0, device="cuda")
    win = torch.rand(B, H, L, generator=g).cuda()
    w = torch.full((B, H, L), 7.0, device="cuda") if weights else None
    sc = D ** -0.5 if scale is None else scale
    hq.kv8_attend(q, cache, i32(table), i32(lens), q_lens=None if q_lens is None else i32(q_lens), scale=scale, causal=causal,
                  out=out, lse=lse, weights=w, weights_in=win if weights else None)
    ref, rl, rw, do, dl, dw = K.attend(K.values(q), k, v, ks, vs, table, np.asarray(lens), np.asarray(ql), sc, causal)
    got, gl = K.values(out), K.values(lse)
    for b in range(B):
        m, n = ql[b], max(0, min(lens[b], L))
        assert np.all(got[b, :, m:] == 7.0) and np.all(gl[b, :, m:] == 7.0)  # rows behind: as they were
        err = np.abs(got[b, :, :m] - ref[b, :, :m])
        assert np.all(err <= do[b, :, :m] + 1e-30), (b, float((err / (do[b, :, :m] + 1e-30)).max()))
        fin = np.isfinite(rl[b, :, :m])
        assert np.array_equal(gl[b, :, :m] == -np.inf, ~fin)
        assert np.all(np.abs(gl[b, :, :m][fin] - rl[b, :, :m][fin]) <= dl[b, :, :m][fin] + 2.0 ** -22)
        if weights:
            gw, wi = K.values(w)[b], K.values(win)[b]
            assert np.all(gw[:, n:] == 7.0)
            assert np.all(np.abs(gw[:, :n] - wi[:, :n] - rw[b, :, :n]) <= dw[b, :, :n] + 2.0 ** -23 * (wi[:, :n] + rw[b, :, :n]))
    return got


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_attend_one_token(hq, D, page):
    check_attend(hq, 3, 2, 4, 1, D, page, [1, 200, 77])


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 300, 1025])
def test_attend_lengths(hq, n):
    check_attend(hq, 1, 1, 1, 1, 128, 64, [n], seed=n)


@pytest.mark.parametrize("G,Sq", [(1, 1), (3, 1), (5, 2), (16, 1), (17, 1), (4, 5), (8, 7), (2, 40), (5, 13), (1, 33)])
@pytest.mark.parametrize("D", [64, 128])
def test_attend_rows_of_a_group(hq, G, Sq, D):
    check_attend(hq, 2, 2, G, Sq, D, 16, [150, Sq], seed=G * 100 + Sq)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,Sq,lens,page", [(1, 128, [128], 64), (1, 129, [130], 16), (2, 128, [300], 128), (4, 70, [500, 70], 32),
                                            (8, 40, [257, 1000, 40], 64), (3, 200, [200, 333], 16), (1, 17, [2000], 64),
                                            (1, 300, [300], 64)])
def test_attend_many_rows(hq, D, G, Sq, lens, page):
    check_attend(hq, len(lens), 1, G, Sq, D, page, lens, seed=Sq + D, weights=False)


def test_attend_many_rows_masks_and_ragged_queries(hq):
    """No slots, fewer slots than queries, no queries, row tiles without rows, and all slots visible."""
    for causal in (True, False):
        check_attend(hq, 6, 2, 2, 150, 64, 32, [0, 30, 400, 64, 150, 257], q_lens=[150, 150, 70, 0, 150, 1], causal=causal, seed=50)
    check_attend(hq, 2, 1, 5, 30, 128, 64, [90, 650], scale=-0.05, seed=51, strided=False)
    check_attend(hq, 2, 1, 5, 30, 128, 64, [90, 65], scale=0.0, seed=52)
    check_attend(hq, 3, 1, 4, 33, 64, 16, [0, 0, 0], seed=53, P=3)


def test_attend_many_rows_stale_bytes_and_bad_pages(hq):
    def stale(cache, k, v, table):
        page = k.shape[2]
        used = np.zeros(k.shape[:1] + k.shape[2:3], bool)
        for b, n in enumerate([170, 116]):
            for j in range(n):
                used[table[b, j // page], j % page] = True
        bad = torch.from_numpy(~used).cuda()[:, None, :, None].expand(*k.shape)
        for t in (cache.k, cache.v):
            t.view(torch.uint8).masked_fill_(bad, 0x7F)
        return table
    check_attend(hq, 2, 2, 3, 50, 128, 32, [170, 116], seed=54, change=stale, P=8)

    def outside(cache, k, v, table):
        table = table.copy()
        table[0, 1], table[1, 0] = -1, 1 << 30
        return table
    check_attend(hq, 2, 1, 2, 100, 64, 16, [160, 140], seed=55, change=outside)


def test_attend_many_rows_value_scales_far_apart(hq):
    g = gen(56)
    cache, (k, v, ks, vs), table = setup_cache(hq, g, 1, 5, 1, 64, 64)
    for i, e in enumerate([0, -12, 6, -9, 3]):
        cache.v_scale[int(table[0, i]), :] = 2.0 ** e
        vs[int(table[0, i]), :] = 2.0 ** e
        cache.k_scale[int(table[0, i]), :] *= 2.0 ** (i - 2)
        ks[int(table[0, i]), :] *= 2.0 ** (i - 2)
    q = torch.randn(1, 2, 40, 64, generator=g).to(torch.bfloat16).cuda()
    out = hq.kv8_attend(q, cache, i32(table), i32([300]))
    ref, rl, _, do, dl, _ = K.attend(K.values(q), k, v, ks, vs, table, [300], [40], 0.125, True)
    assert np.all(np.abs(K.values(out) - ref) <= do + 2.0 ** -24 * np.abs(v).max() * vs.max())


@pytest.mark.parametrize("causal", [True, False])
def test_attend_ragged_with_empty_rows(hq, causal):
    """No slots, fewer slots than queries (rows that see nothing), no queries, padded queries."""
    check_attend(hq, 6, 2, 2, 6, 64, 32, [0, 3, 100, 64, 6, 1], q_lens=[6, 6, 4, 0, 6, 1], causal=causal, seed=3)


def test_attend_all_sequences_empty(hq):
    check_attend(hq, 2, 2, 2, 3, 128, 32, [0, 0], seed=4, P=2)


def test_attend_ragged_batch_larger_than_the_grid(hq):
    lens = [int(x) for x in np.random.default_rng(5).integers(0, 90, 400)]
    check_attend(hq, 400, 1, 2, 1, 64, 16, lens, seed=5)


def test_attend_other_scales_and_strides(hq):
    check_attend(hq, 2, 2, 2, 2, 128, 64, [90, 65], scale=0.03, strided=False, seed=6)
    check_attend(hq, 2, 2, 2, 2, 128, 64, [90, 65], scale=0.0, seed=6)
    check_attend(hq, 2, 2, 2, 2, 128, 64, [90, 65], scale=-0.1, seed=6)


def test_attend_stale_bytes_are_never_used(hq):
    """Slots behind the sequences and pages outside them hold NaN codes."""
    def change(cache, k, v, table):
        page = k.shape[2]
        used = np.zeros(k.shape[:1] + k.shape[2:3], bool)
        for b, n in enumerate([70, 16]):
            for j in range(n):
                used[table[b, j // page], j % page] = True
        bad = torch.from_numpy(~used).cuda()[:, None, :, None].expand(*k.shape)
        for t in (cache.k, cache.v):
            t.view(torch.uint8).masked_fill_(bad, 0x7F)
        return table
    check_attend(hq, 2, 2, 3, 2, 128, 32, [70, 16], seed=7, change=change, P=4)


def test_attend_pages_outside_the_pool_are_unseen(hq):
    def change(cache, k, v, table):
        table = table.copy()
        table[0, 1], table[1, 0] = -1, 1 << 30
        return table
    check_attend(hq, 2, 1, 2, 2, 64, 16, [60, 40], seed=8, change=change)


def test_attend_value_scales_far_apart(hq):
    """Pages whose scales differ by many octaves, one of zeros (scale 2^-40)."""
    def change(cache, k, v, table):
        for i, e in enumerate([0, -40, 12, -9, 25]):
            cache.v_scale[int(table[0, i]), :] = 2.0 ** e
            vs[int(table[0, i]), :] = 2.0 ** e
        return table
    g = gen(9)
    cache, (k, v, ks, vs), table = setup_cache(hq, g, 1, 5, 1, 16, 64)
    change(cache, k, v, table)
    q = torch.randn(1, 2, 1, 64, generator=g).to(torch.bfloat16).cuda()
    lse = torch.empty(1, 2, 1, device="cuda")
    out = hq.kv8_attend(q, cache, i32(table), i32([80]), lse=lse)
    ref, rl, _, do, dl, _ = K.attend(K.values(q), k, v, ks, vs, table, [80], [1], 0.125, True)
    assert np.all(np.abs(K.values(out) - ref) <= do)


def test_attend_nan_query_spoils_its_row_only(hq):
    g = gen(10)
    cache, parts, table = setup_cache(hq, g, 1, 2, 1, 32, 128)
    q = torch.randn(1, 4, 1, 128, generator=g).to(torch.bfloat16).cuda()
    ref = hq.kv8_attend(q, cache, i32(table), i32([50]))
    q[0, 2, 0, 5] = float("nan")
    out = hq.kv8_attend(q, cache, i32(table), i32([50]))
    assert out[0, 2].isnan().all()
    assert torch.equal(out[0, [0, 1, 3]], ref[0, [0, 1, 3]])


def test_attend_is_deterministic_and_replays_from_graphs(hq):
    g = gen(11)
    cache, parts, table = setup_cache(hq, g, 3, 9, 2, 64, 128)
    t, lens = i32(table), i32([500, 3, 130])
    q = torch.randn(3, 8, 2, 128, generator=g).to(torch.bfloat16).cuda()
    w = [torch.zeros(3, 2, 576, device="cuda") for _ in range(3)]
    direct = hq.kv8_attend(q, cache, t, lens, weights=w[0])
    outs, graphs = [], []
    for i in (1, 2):  # two graphs, each with scratch of its own
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(hq.kv8_attend(q, cache, t, lens, weights=w[i]))
    for _ in range(2):
        for gr in graphs:
            gr.replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i], direct) and torch.equal(w[i + 1], w[0])
    lens.fill_(40)  # a replay reads the lengths of its moment
    graphs[0].replay()
    assert torch.equal(outs[0], hq.kv8_attend(q, cache, t, lens))


def test_attend_many_rows_is_deterministic_and_replays_from_a_graph(hq):
    g = gen(13)
    cache, parts, table = setup_cache(hq, g, 2, 9, 2, 64, 128)
    t, lens = i32(table), i32([560, 131])
    q = torch.randn(2, 8, 90, 128, generator=g).to(torch.bfloat16).cuda()
    w = [torch.zeros(2, 2, 576, device="cuda") for _ in range(2)]
    direct = hq.kv8_attend(q, cache, t, lens, weights=w[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = hq.kv8_attend(q, cache, t, lens, weights=w[1])
    for _ in range(3):
        graph.replay()
    assert torch.equal(out, direct) and torch.equal(w[1], w[0])
    lens.fill_(100)
    graph.replay()
    assert torch.equal(out, hq.kv8_attend(q, cache, t, lens))


@pytest.mark.parametrize("Sq", [1, 40])
def test_attend_shared_pages_and_short_weights(hq, Sq):
    """Two sequences over the same first pages; weights for fewer slots than the sequences have."""
    g = gen(14)
    cache, (k, v, ks, vs), table = setup_cache(hq, g, 2, 6, 2, 16, 64)
    table[1, :4] = table[0, :4]
    q = torch.randn(2, 4, Sq, 64, generator=g).to(torch.bfloat16).cuda()
    w = torch.full((2, 2, 50), 7.0, device="cuda")
    ws = hq.Workspace(hq.lib().hq_kv8_attend_workspace_bytes(2, 2, 4, Sq, 64, 1))
    out = hq.kv8_attend(q, cache, i32(table), i32([90, 77]), weights=w, ws=ws)
    ref, _, rw, do, _, dw = K.attend(K.values(q), k, v, ks, vs, table, [90, 77], [Sq, Sq], 0.125, True)
    assert np.all(np.abs(K.values(out) - ref) <= do)
    assert np.all(np.abs(K.values(w) - rw[:, :, :50]) <= dw[:, :, :50] + 2.0 ** -23 * rw[:, :, :50])
    assert hq.status(ws)[0] == 7


def test_attend_on_another_stream_with_a_workspace(hq):
    g = gen(15)
    cache, parts, table = setup_cache(hq, g, 2, 20, 2, 64, 128)
    t, lens = i32(table), i32([1200, 40])
    q = torch.randn(2, 4, 2, 128, generator=g).to(torch.bfloat16).cuda()
    ref = hq.kv8_attend(q, cache, t, lens)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    ws = hq.Workspace(hq.lib().hq_kv8_attend_workspace_bytes(2, 2, 4, 2, 128, 0))
    with torch.cuda.stream(stream):
        for _ in range(5):
            out = hq.kv8_attend(q, cache, t, lens, ws=ws)
        assert hq.status(ws) == (0, 0)
    assert torch.equal(out, ref)


def test_calls_on_two_streams_do_not_share_scratch(hq):
    g = gen(12)
    cache, parts, table = setup_cache(hq, g, 4, 32, 4, 64, 128)
    t, lens = i32(table), i32([2000, 1500, 2048, 9])
    q = [torch.randn(4, 16, 1, 128, generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
    ref = [hq.kv8_attend(x, cache, t, lens) for x in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(hq.kv8_attend(q[i], cache, t, lens))
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref[i]) for i in range(2) for o in got[i])


# ------------------------------------------------------------------------------------------------
# append
# ------------------------------------------------------------------------------------------------
def check_append(hq, B, H, S, D, page, lens, n_new=None, dtype=torch.bfloat16, seed=0, P=None, edit=None, status=0):
    g = gen(seed)
    P = P or max(1, -(-max(a + S for a in lens) // page))
    cache, (k, v, ks, vs), table = setup_cache(hq, g, B, P, H, page, D)
    kv = torch.randn(B, S, 2 * H, D, generator=g) * torch.exp(2 * torch.randn(B, S, 1, 1, generator=g))
    if edit:
        table = edit(kv, table)
    kv = kv.to(dtype).cuda()
    xk, xv = kv[:, :, :H].transpose(1, 2), kv[:, :, H:].transpose(1, 2)
    ws = hq.fp8_workspace()
    hq.kv8_append(cache, xk, xv, i32(table), i32(lens), n_new=None if n_new is None else i32(n_new), ws=ws)
    new = [S] * B if n_new is None else n_new
    K.append(k, ks, K.values(xk), table, lens, new)
    K.append(v, vs, K.values(xv), table, lens, new)
    for got, ref in ((cache.k, k), (cache.v, v), (cache.k_scale, ks), (cache.v_scale, vs)):
        assert np.array_equal(K.values(got), ref)
    st = hq.status(ws)
    assert st[0] == status
    return st


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_append_one_token(hq, D, page, dtype):
    check_append(hq, 5, 3, 1, D, page, [0, 1, page - 1, page, 2 * page + 5], dtype=dtype, seed=page)


@pytest.mark.parametrize("S", [2, 15, 16, 17, 64, 65, 200])
def test_append_many_tokens(hq, S):
    check_append(hq, 3, 2, S, 128, 64, [0, 60, 129], seed=S)
    check_append(hq, 3, 2, S, 64, 16, [0, 60, 129], n_new=[S, 0, S // 2], seed=S, dtype=torch.float32)


def test_append_growing_scales_move_old_codes(hq):
    def edit(kv, table):
        kv *= 1e4
        return table
    check_append(hq, 3, 2, 1, 128, 64, [1, 63, 30], edit=edit, seed=20)


def test_append_zero_and_tiny_and_huge_values(hq):
    def edit(kv, table):
        kv[0] = 0.0
        kv[1] *= 1e-30
        kv[2, 0, 0, 3] = 3e38
        return table
    check_append(hq, 3, 1, 2, 64, 16, [0, 16, 5], edit=edit, seed=21, dtype=torch.float32, status=7)


def test_append_non_finite_vectors_become_zeros(hq):
    def edit(kv, table):
        kv[0, 1, 0, 5], kv[1, 0, 3, 0] = float("inf"), float("nan")
        return table
    st = check_append(hq, 2, 2, 3, 128, 32, [3, 31], edit=edit, seed=22, status=4)
    assert st[1] == 2


def test_append_bad_pages_and_full_tables(hq):
    def edit(kv, table):
        table = table.copy()
        table[0, 1] = 1 << 20
        return table
    check_append(hq, 2, 2, 40, 64, 16, [10, 0], edit=edit, seed=23, status=7)
    check_append(hq, 2, 2, 40, 64, 16, [10, 0], P=2, seed=24, status=7)   # tokens past the table are dropped
    check_append(hq, 2, 2, 4, 64, 16, [-3, 0], P=2, seed=24, status=7)


def test_attend_repeats_bit_for_bit_on_a_long_cache(hq):
    """A cache far larger than L2, so that loads land late and close together: every call the same bits."""
    B, H, D, page, n = 8, 32, 128, 64, 4096
    P = n // page
    cache = hq.alloc_kv8(B * P, H, D, page)
    g = torch.Generator(device="cuda").manual_seed(7)
    for part in (cache.k, cache.v):
        part.view(torch.uint8).copy_(torch.randint(0, 0x60, part.shape, generator=g, device="cuda", dtype=torch.uint8))
    for scale in (cache.k_scale, cache.v_scale):
        scale.fill_(2.0 ** -4)
    table = torch.randperm(B * P, generator=g, device="cuda").to(torch.int32).view(B, P)
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    q = torch.randn(B, H, 1, D, generator=g, device="cuda").to(torch.bfloat16)
    outs = []
    for _ in range(60):
        out, lse = torch.empty_like(q), torch.empty(B, H, 1, device="cuda")
        hq.kv8_attend(q, cache, table, lens, out=out, lse=lse)
        outs.append((out, lse))
    assert all(torch.equal(o, outs[0][0]) and torch.equal(l, outs[0][1]) for o, l in outs[1:])


# ------------------------------------------------------------------------------------------------
# evict
# ------------------------------------------------------------------------------------------------
def check_evict(hq, B, H, D, page, lens, budget, recent, seed=0, edit=None, strided=False):
    g = gen(seed)
    P, TP = max(1, -(-max(lens) // page)), -(-budget // page)
    cache, (k, v, ks, vs), both = setup_cache(hq, g, B, P + TP, H, page, D)
    table, to = both[:, :P], both[:, P:]
    L = max(max(lens), 1)
    w = torch.rand(B, H, L, generator=g)
    w = torch.where(torch.rand(B, H, L, generator=g) < 0.3, torch.full_like(w, 0.25), w)
    if edit:
        edit(w)
    big = torch.zeros(B, H, 2 * L, device="cuda")
    big[:, :, :L] = w.cuda()
    w_dev = big[:, :, :L] if strided else w.cuda()
    ws = hq.Workspace(hq.lib().hq_kv8_evict_workspace_bytes(B, H, budget))
    full = i32(both)
    n, ow = hq.kv8_evict(cache, full[:, :P] if strided else i32(table), i32(lens), w_dev, budget, recent,
                         full[:, P:] if strided else i32(to), ws=ws)
    rn, rw = K.evict(k, v, ks, vs, table, np.asarray(lens), K.values(w), budget, recent, to)
    assert n.cpu().tolist() == rn.tolist()
    for (b, h), ref in rw.items():
        got = K.values(ow)[b, h]
        assert np.array_equal(got[:len(ref)], ref, equal_nan=True) and np.all(got[len(ref):] == 0.0)
    for got, ref in ((cache.k, k), (cache.v, v), (cache.k_scale, ks), (cache.v_scale, vs)):
        assert np.array_equal(K.values(got), ref)
    assert hq.status(ws)[0] == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_evict_pages(hq, D, page):
    check_evict(hq, 3, 2, D, page, [300, 0, 129], 100, 20, seed=page)


@pytest.mark.parametrize("n,budget,recent", [(1, 1, 0), (2, 1, 0), (2, 1, 1), (50, 50, 3), (50, 49, 0), (50, 49, 49), (50, 20, 30),
                                             (1500, 700, 0), (1500, 1, 0), (1025, 1024, 5), (3000, 33, 32)])
def test_evict_budgets(hq, n, budget, recent):
    check_evict(hq, 1, 2, 64, 16, [n], budget, recent, seed=n + budget)


@pytest.mark.parametrize("n,budget", [(1024, 500), (4096, 100), (4097, 2000), (8192, 8000), (8300, 4000), (45000, 300)])
def test_evict_long_sequences(hq, n, budget):
    """Weights in registers (runs of 2, 4, 8), in shared memory, and more than it holds."""
    check_evict(hq, 1, 1, 64, 128, [n], budget, 7, seed=n)


@pytest.mark.parametrize("n,budget", [(600, 599), (4000, 1000), (4097, 40)])
@pytest.mark.parametrize("strided", [False, True])
def test_evict_many_heads(hq, n, budget, strided):
    """More heads than multiprocessors; rows of weights on and off 16 bytes."""
    check_evict(hq, 5, 40, 64, 128, [n, n - 1, 0, 17, n // 2 + 1], budget, min(13, budget), strided=strided, seed=n + 1)


def test_evict_ties_zeros_signs_and_nan(hq):
    def edit(w):
        w[:] = 0.0
        w[:, :, ::3] = -0.0
        w[:, :, 5] = float("nan")
        w[:, :, 7] = -1.0
        w[:, :, 11] = float("inf")
        w[:, :, 13] = -float("inf")
        w[:, :, 17] = 1e-45
    check_evict(hq, 2, 2, 64, 16, [90, 40], 30, 4, edit=edit, seed=30)
    check_evict(hq, 2, 2, 64, 16, [40, 38], 39, 0, edit=edit, seed=31)
    check_evict(hq, 2, 2, 64, 16, [40, 40], 37, 0, edit=edit, seed=31)


def test_evict_strided_tables_and_weights(hq):
    check_evict(hq, 2, 3, 128, 32, [200, 150], 64, 8, strided=True, seed=32)


def test_evict_pages_outside_the_pool_leave_the_target(hq):
    g = gen(33)
    cache, (k, v, ks, vs), both = setup_cache(hq, g, 1, 6, 1, 16, 64)
    table, to = both[:, :4].copy(), both[:, 4:].copy()
    table[0, 2], to[0, 0] = 1 << 29, -5
    ws = hq.Workspace(hq.lib().hq_kv8_evict_workspace_bytes(1, 1, 20))
    w = torch.rand(1, 1, 64, generator=g).cuda()
    before = [t.clone() for t in (cache.k.view(torch.uint8), cache.v.view(torch.uint8))]
    hq.kv8_evict(cache, i32(table), i32([64]), w, 20, 20, i32(to), ws=ws)
    assert hq.status(ws)[0] == 7
    for t, b in zip((cache.k, cache.v), before):
        keep = torch.ones(t.shape[0], dtype=torch.bool)
        keep[int(to[0, 1])] = False
        assert torch.equal(t.view(torch.uint8)[keep.cuda()], b[keep.cuda()])


def test_evict_lengths_in_place(hq):
    g = gen(34)
    cache, parts, both = setup_cache(hq, g, 3, 12, 4, 16, 64)
    lens = i32([128, 5, 100])
    w = torch.rand(3, 4, 128, generator=g).cuda()
    n, _ = hq.kv8_evict(cache, i32(both[:, :8]), lens, w, 50, 10, i32(both[:, 8:]), out_lens=lens)
    assert n.data_ptr() == lens.data_ptr() and lens.cpu().tolist() == [50, 5, 50]


def test_append_and_evict_replay_from_graphs(hq):
    g = gen(35)
    (a, _, both), (b, _, _) = (setup_cache(hq, gen(36), 2, 12, 2, 16, 64) for _ in range(2))
    table, to = i32(both[:, :8]), i32(both[:, 8:])
    x = torch.randn(2, 2, 3, 64, generator=g).to(torch.bfloat16).cuda()
    w = torch.rand(2, 2, 128, generator=g).cuda()
    lens = i32([70, 20])

    def step(cache):
        hq.kv8_append(cache, x, 2 * x, table, lens)
        return hq.kv8_evict(cache, table, lens, w, 30, 5, to)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n, ow = step(a)
    for l in ([70, 20], [101, 64], [3, 0]):
        lens.copy_(i32(l))
        x *= 1.5
        graph.replay()
        rn, rw = step(b)
        assert torch.equal(n, rn) and torch.equal(ow[:, :, :3], rw[:, :, :3])
        for t, r in ((a.k, b.k), (a.v, b.v)):
            assert torch.equal(t.view(torch.uint8), r.view(torch.uint8))
        assert torch.equal(a.k_scale, b.k_scale) and torch.equal(a.v_scale, b.v_scale)


# ------------------------------------------------------------------------------------------------
# together
# ------------------------------------------------------------------------------------------------
def test_a_layer_decodes_with_eviction(hq):
    """A layer's steps: block-scaled projections of the hidden state, append, attention with weights, the
    output projection, and an eviction in between; each step against the definitions, on the caches
    that the run itself left."""
    g = gen(40)
    B, H, G, D, page, hidden = 2, 2, 2, 64, 16, 200
    Hq = H * G
    w_qkv = hq.fp8_quantize((0.1 * torch.randn((Hq + 2 * H) * D, hidden, generator=g)).to(torch.bfloat16).cuda(), block=128)
    w_out = hq.fp8_quantize((0.1 * torch.randn(hidden, Hq * D, generator=g)).to(torch.bfloat16).cuda(), block=128)
    cache = hq.alloc_kv8(40, H, D, page)
    order = torch.randperm(40, generator=g).to(torch.int32)
    table, other = order[:16].view(2, 8).cuda(), order[16:32].view(2, 8).cuda()
    lens, score = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, H, 128, device="cuda")
    x = torch.randn(B, 30, hidden, generator=g).to(torch.bfloat16).cuda()
    for step in range(12):
        S = x.shape[1]
        before = [K.values(t) for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
        n0 = lens.cpu().numpy().copy()
        a = hq.fp8_quantize(x.reshape(B * S, hidden))
        qkv = hq.gemm_fp8(a, w_qkv)
        want = K.values(a.dequantize()) @ K.values(w_qkv.dequantize()).T
        size = np.abs(K.values(a.dequantize())) @ np.abs(K.values(w_qkv.dequantize())).T
        assert np.all(np.abs(K.values(qkv) - want) <= 2.0 ** -8 * np.abs(want) + hidden * 2.0 ** -23 * size)
        qkv = qkv.view(B, S, Hq + 2 * H, D)
        q, k, v = (t.transpose(1, 2) for t in qkv.split([Hq, H, H], 2))
        hq.kv8_append(cache, k, v, table, lens)
        tab = table.cpu().numpy()
        K.append(before[0], before[2], K.values(k), tab, n0, [S] * B)
        K.append(before[1], before[3], K.values(v), tab, n0, [S] * B)
        for t, ref in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), before):
            assert np.array_equal(K.values(t), ref)
        lens += S
        old = K.values(score)
        out = hq.kv8_attend(q, cache, table, lens, weights=score, weights_in=score)
        n = n0 + S
        ref, _, rw, do, _, dw = K.attend(K.values(q), *before, tab, n, [S] * B, D ** -0.5, True)
        assert np.all(np.abs(K.values(out) - ref) <= do)
        for b in range(B):
            d = np.abs(K.values(score)[b, :, :n[b]] - old[b, :, :n[b]] - rw[b, :, :n[b]])
            assert np.all(d <= dw[b, :, :n[b]] + 2.0 ** -22 * (old[b, :, :n[b]] + rw[b, :, :n[b]]))
        y = hq.gemm_fp8(hq.fp8_quantize(out.transpose(1, 2).reshape(B * S, Hq * D)), w_out)
        x = torch.tanh(y.view(B, S, hidden)[:, -1:].float()).to(torch.bfloat16).contiguous()
        if step % 4 == 3:
            w_old, n_old = K.values(score), lens.cpu().numpy().copy()
            new = torch.zeros_like(score)
            hq.kv8_evict(cache, table, lens, score, 24, 8, other, out_lens=lens, out_weights=new)
            _, kept = K.evict(*before, tab, n_old, w_old, 24, 8, other.cpu().numpy())
            for t, ref in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), before):
                assert np.array_equal(K.values(t), ref)
            for (b, h), ref in kept.items():
                assert np.array_equal(K.values(new)[b, h, :len(ref)], ref)
            table, other, score = other, table, new
            assert lens.cpu().tolist() == [24, 24]
