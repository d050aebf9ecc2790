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
