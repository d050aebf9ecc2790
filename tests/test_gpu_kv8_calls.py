"""Calls of the e4m3 cache's operators as a program makes them: scratch, outputs and arguments."""
import ctypes

import pytest
import torch

from test_gpu_kv8 import gen, i32, setup_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hq():
    import post_quantization_tile_b200 as m
    m.lib()
    return m


def attend_struct(hq, q, cache, table, lens, out, weights):
    from test_fp8_arguments import ATTEND
    B, Hq, Sq, D = q.shape
    pages, heads, page, _ = cache.k.shape
    L = weights.shape[2] if weights is not None else 0
    return ATTEND.pack(*(t.data_ptr() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)), pages, heads, page, D, q.data_ptr(),
                       out.data_ptr(), B, Hq, Sq, *q.stride()[:3], *out.stride()[:3], table.data_ptr(), table.shape[1], table.shape[1],
                       lens.data_ptr(), 0, D ** -0.5, 1, 0, 0, 0, 0, weights.data_ptr() if weights is not None else 0, 0, 0, heads * L, L, L)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows,lens,H", [(1, [50], 1), (8, [3000, 1], 2), (9, [64, 700], 1), (32, [5000], 1), (33, [50], 1), (33, [129], 2),
                                         (200, [300, 200], 2), (257, [257], 1), (600, [4000], 1), (40, [70] * 200, 2)])
def test_a_workspace_of_the_needed_size_is_enough(hq, rows, lens, H, D):
    """Nothing is written behind it, and the result is the one of a larger workspace."""
    B, page = len(lens), 16
    cache, _, table = setup_cache(hq, gen(rows), B, -(-max(lens) // page), H, page, D)
    q = torch.randn(B, H, rows, D, generator=gen(1)).to(torch.bfloat16).cuda()
    w = [torch.zeros(B, H, max(lens), device="cuda") for _ in range(2)]
    t, n, out = i32(table), i32(lens), torch.empty_like(q)
    lib = hq.lib()
    need = lib.hq_kv8_attend_workspace_need(attend_struct(hq, q, cache, t, n, out, w[0]))
    most = lib.hq_kv8_attend_workspace_bytes(B, H, H, rows, D, 1)
    assert 0 < need <= most
    buf = torch.full((need + 65536,), 0x5A, dtype=torch.uint8, device="cuda")
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    args = attend_struct(hq, q, cache, t, n, out, w[0])
    assert lib.hq_kv8_attend(args, buf.data_ptr(), need, stream) == 0
    assert lib.hq_kv8_attend(args, buf.data_ptr(), need - 1, stream) == 1
    ref = hq.kv8_attend(q, cache, t, n, weights=w[1], ws=hq.Workspace(most))
    assert torch.equal(out, ref) and torch.equal(w[0], w[1])
    assert torch.all(buf[need:] == 0x5A)


def test_a_short_call_of_many_rows_takes_little_scratch(hq):
    cache, _, table = setup_cache(hq, gen(2), 1, 1, 1, 64, 128)
    q = torch.randn(1, 1, 33, 128, generator=gen(3)).to(torch.bfloat16).cuda()
    t, n, out = i32(table), i32([50]), torch.empty_like(q)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    hq.kv8_attend(q, cache, t, n, out=out)
    assert torch.cuda.max_memory_allocated() - before < 1 << 20


def views(n, rows, dim, dtype):
    """(output, input) pairs of views of one buffer: rows that meet, and rows that do not."""
    def buf(*shape):
        return torch.zeros(*shape, dtype=dtype, device="cuda")
    a, b, c = buf(2 * n * rows * dim + 64), buf(n, rows, 2, dim), buf(n, 2 * rows, dim)
    whole = a[:n * rows * dim].view(n, rows, dim)
    meet = [(a[8:8 + n * rows * dim].view(n, rows, dim), whole), (whole, a[dim:dim + n * rows * dim].view(n, rows, dim)),
            (whole, a[(n * rows - 1) * dim:(2 * n * rows - 1) * dim].view(n, rows, dim)), (c[:, :rows], c[:, rows - 1:-1])]
    apart = [(b[:, :, 0], b[:, :, 1]), (b[:, :, 1], b[:, :, 0]), (c[:, :rows], c[:, rows:]), (c[:, rows:], c[:, :rows]),
             (whole, a[n * rows * dim:2 * n * rows * dim].view(n, rows, dim))]
    return meet, apart


def test_attend_refuses_outputs_that_meet_their_inputs(hq):
    """out and q, weights and weights_in of one buffer: refused where rows meet, computed where they do not."""
    cache, _, table = setup_cache(hq, gen(4), 3, 2, 4, 16, 64)
    t, n = i32(table), i32([20, 3, 32])
    x = torch.randn(3, 4, 64, generator=gen(5)).to(torch.bfloat16).cuda()
    ref = hq.kv8_attend(x.view(3, 4, 1, 64), cache, t, n)
    meet, apart = views(3, 4, 64, torch.bfloat16)
    for out, q in meet:
        with pytest.raises(ValueError):
            hq.kv8_attend(q.unsqueeze(2), cache, t, n, out=out.unsqueeze(2))
    for out, q in apart:
        q.copy_(x)
        assert torch.equal(hq.kv8_attend(q.unsqueeze(2), cache, t, n, out=out.unsqueeze(2)), ref)
    q, win = x.view(3, 4, 1, 64), torch.rand(3, 4, 32, generator=gen(6)).cuda()
    want = win.clone()
    hq.kv8_attend(q, cache, t, n, weights=want, weights_in=want)
    meet, apart = views(3, 4, 32, torch.float32)
    for w, w_in in meet:
        with pytest.raises(ValueError):
            hq.kv8_attend(q, cache, t, n, weights=w, weights_in=w_in)
    for w, w_in in apart:
        w_in.copy_(win)
        w.copy_(win)
        hq.kv8_attend(q, cache, t, n, weights=w, weights_in=w_in)
        assert torch.equal(w, want)


def test_evict_refuses_outputs_that_meet_their_inputs(hq):
    cache, _, both = setup_cache(hq, gen(7), 3, 4, 4, 16, 64)
    table, to, lens = i32(both[:, :2]), i32(both[:, 2:]), i32([32, 9, 20])
    x = torch.rand(3, 4, 32, generator=gen(8)).cuda()
    _, ref = hq.kv8_evict(cache, table, lens, x, 32, 4, to)
    meet, apart = views(3, 4, 32, torch.float32)
    for ow, w in meet + [(x[:, :, 3:], x)]:
        with pytest.raises(ValueError):
            hq.kv8_evict(cache, table, lens, w, 29 if ow.shape[2] == 29 else 32, 4, to, out_weights=ow)
    for ow, w in apart:
        w.copy_(x)
        ow.zero_()
        assert torch.equal(hq.kv8_evict(cache, table, lens, w, 32, 4, to, out_weights=ow)[1], ref)
    ints = torch.zeros(8, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        hq.kv8_evict(cache, table, ints[:3], x, 8, 4, to, out_lens=ints[1:4])


def test_expanded_outputs_are_refused(hq):
    cache, _, table = setup_cache(hq, gen(9), 2, 2, 2, 16, 64)
    t, n, q = i32(table), i32([20, 3]), torch.zeros(2, 4, 3, 64, dtype=torch.bfloat16, device="cuda")
    for shape in ((1, 4, 3, 64), (2, 1, 3, 64), (2, 4, 1, 64)):
        with pytest.raises(ValueError):
            hq.kv8_attend(q, cache, t, n, out=torch.zeros(shape, dtype=torch.bfloat16, device="cuda").expand(2, 4, 3, 64))
    w = torch.zeros(1, 2, 32, device="cuda").expand(2, 2, 32)
    with pytest.raises(ValueError):
        hq.kv8_attend(q, cache, t, n, lse=torch.zeros(2, 1, 3, device="cuda").expand(2, 4, 3))
    with pytest.raises(ValueError):
        hq.kv8_attend(q, cache, t, n, weights=w)
    with pytest.raises(ValueError):
        hq.kv8_evict(cache, t, n, w.contiguous(), 16, 2, t, out_weights=torch.zeros(2, 1, 16, device="cuda").expand(2, 2, 16))
    # inputs may be: every row of q and of the weights is the same
    one = torch.randn(1, 1, 1, 64, generator=gen(10)).to(torch.bfloat16).cuda()
    assert torch.equal(hq.kv8_attend(one.expand(2, 4, 3, 64), cache, t, n), hq.kv8_attend(one.expand(2, 4, 3, 64).contiguous(), cache, t, n))


def test_expanded_outputs_are_refused_at_the_c_entry_points(hq):
    from test_fp8_arguments import EVICT
    cache, _, table = setup_cache(hq, gen(9), 2, 2, 2, 16, 64)
    t, n, q = i32(table), i32([20, 3]), torch.zeros(2, 4, 3, 64, dtype=torch.bfloat16, device="cuda")
    lib, ws, stream = hq.lib(), hq.Workspace(1 << 26), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    out = torch.zeros_like(q)
    assert lib.hq_kv8_attend(attend_struct(hq, q, cache, t, n, out, None), ws.ptr(), ws.nbytes, stream) == 0
    for i in range(3):
        bad = out.narrow(i, 0, 1).expand_as(out)
        assert lib.hq_kv8_attend(attend_struct(hq, q, cache, t, n, bad, None), ws.ptr(), ws.nbytes, stream) == 1
    w = torch.zeros(2, 2, 32, device="cuda")
    head = [x.data_ptr() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale)] + [cache.k.shape[0], 2, 16, 64]
    to, ow = i32([[4], [5]]), torch.zeros(2, 2, 16, device="cuda")
    for strides, code in (((32, 16), 0), ((0, 16), 1), ((32, 0), 1)):
        args = EVICT.pack(*head, 2, t.data_ptr(), 2, 2, n.data_ptr(), w.data_ptr(), 64, 32, 32, 16, 2, to.data_ptr(), 1, 1, i32([0, 0]).data_ptr(),
                          ow.data_ptr(), *strides)
        assert lib.hq_kv8_evict(args, ws.ptr(), ws.nbytes, stream) == code


def test_causal_without_a_truth_value_raises_its_own_error(hq):
    cache, _, table = setup_cache(hq, gen(11), 1, 2, 1, 16, 64)
    q, t, n = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16, device="cuda"), i32(table), i32([20])

    class Unsure:
        def __bool__(self):
            raise ZeroDivisionError
    with pytest.raises(ZeroDivisionError):
        hq.kv8_attend(q, cache, t, n, causal=Unsure())
    with pytest.raises(TypeError):
        hq.kv8_attend(q, cache, t, n, scale="wide")
    assert hq.kv8_attend(q, cache, t, n, causal=0).shape == q.shape


@pytest.mark.parametrize("rows", [1, 33])
def test_the_largest_batch(hq, rows):
    """2048 sequences, most of them short, with few rows and with many."""
    import numpy as np
    from test_gpu_kv8 import check_attend
    rng = np.random.default_rng(rows)
    lens, asked = rng.integers(0, 20, 2048).tolist(), np.minimum(rng.integers(0, 3, 2048), rows)
    asked[[0, 1000, 2047]] = rows
    check_attend(hq, 2048, 1, 1, rows, 64, 16, lens, q_lens=asked.tolist(), seed=rows, P=2)


def test_a_pool_of_more_than_32_bits_of_bytes(hq):
    """Keys of 5.4 GB, values too: sequences on the pool's first and last pages give what they give in a small pool."""
    H, page, D, far = 4, 64, 128, 164000
    big, small = hq.alloc_kv8(far + 8, H, D, page), hq.alloc_kv8(16, H, D, page)
    assert big.k.numel() > 5 << 30
    high, low = i32([[far + 3, 1, far + 7], [far, far + 5, 0]]), i32([[3, 9, 7], [0, 5, 8]])
    high_to, low_to = i32([[far + 1], [far + 6]]), i32([[1], [6]])
    x = torch.randn(2, 2 * H, 150, D, generator=gen(12)).to(torch.bfloat16).cuda()
    q = torch.randn(2, 2 * H, 40, D, generator=gen(13)).to(torch.bfloat16).cuda()
    got = []
    for cache, table, to in ((big, high, high_to), (small, low, low_to)):
        lens, w = i32([0, 0]), torch.zeros(2, H, 192, device="cuda")
        hq.kv8_append(cache, x[:, :H, :149], x[:, H:, :149], table, lens)
        lens += 149
        hq.kv8_append(cache, x[:, :H, 149:], x[:, H:, 149:], table, lens)
        lens += 1
        outs = [hq.kv8_attend(q, cache, table, lens, weights=w, weights_in=w), hq.kv8_attend(q[:, :, :2], cache, table, lens)]
        n, ow = hq.kv8_evict(cache, table, lens, w, 50, 10, to)
        got.append(outs + [w, n, ow, hq.kv8_attend(q, cache, to, n)])
    assert all(torch.equal(a, b) for a, b in zip(*got)) and got[0][0].abs().amax() > 0.1
