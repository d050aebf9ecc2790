"""e4m3 quantization and the block-scaled e4m3 GEMM on the GPU against plain 64-bit definitions:
quantization code for code, the product within the roundings of binary32 sums."""
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


def check_quantize(hq, x, block, status=0):
    ws = hq.fp8_workspace()
    code = hq.fp8_quantize(x, block=block, ws=ws)
    q, s = K.quantize(K.values(x), block)
    got = K.values(code.data)
    assert np.array_equal(got[:, :x.shape[1]], q) and np.all(got[:, x.shape[1]:] == 0.0)
    assert np.array_equal(K.values(code.scale), s)
    st = hq.status(ws)
    assert st[0] == status
    return st


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (3, 7), (31, 129), (33, 256), (128, 128), (129, 260), (300, 1000)])
def test_quantize(hq, rows, cols, block, dtype):
    g = torch.Generator().manual_seed(rows + cols)
    x = torch.randn(rows, cols, generator=g) * torch.exp(3 * torch.randn(1, cols, generator=g))
    check_quantize(hq, x.to(dtype).cuda(), block)


@pytest.mark.parametrize("block", [1, 128])
def test_quantize_strided_and_unaligned_rows(hq, block):
    x = torch.randn(50, 401, generator=torch.Generator().manual_seed(1)).cuda()
    check_quantize(hq, x[:, 1:300], block)
    check_quantize(hq, x.to(torch.bfloat16)[:, 8:264], block)
    check_quantize(hq, x[3:4, :130], block)


def test_quantize_every_boundary(hq):
    """Halfway points between codes, the borders of the scale's octave, subnormal and extreme magnitudes."""
    mids = [(1 + (i + 0.5) / 8) * 2.0 ** e for e in range(-6, 8) for i in range(8)] + [448.0] * 8
    mids += [(i + 0.5) * 2.0 ** -9 for i in range(8)]
    x = torch.zeros(6, 128)
    x[0, :len(mids)] = torch.tensor(mids, dtype=torch.float32)
    x[1, 0] = 448.0
    x[2, 0] = float(np.nextafter(np.float32(448.0), np.float32(1e9)))
    x[3, :3] = torch.tensor([1e-45, -1e-38, 3e-40])
    x[4, :2] = torch.tensor([2.0 ** -50, -2.0 ** -49])
    check_quantize(hq, x.cuda(), 1)
    x[5, 0] = 3e38
    check_quantize(hq, x.cuda(), 1, status=7)


@pytest.mark.parametrize("block,bad", [(1, 2), (128, 1)])
def test_quantize_non_finite_blocks_become_zeros(hq, block, bad):
    x = torch.randn(20, 200, generator=torch.Generator().manual_seed(2))
    x[3, 5], x[7, 100] = float("nan"), -float("inf")
    st = check_quantize(hq, x.cuda(), block, status=4)
    assert st[1] == bad


def codes(hq, g, rows, cols, block):
    x = torch.randn(rows, cols, generator=g) * torch.exp(torch.randn(1, cols, generator=g))
    return hq.fp8_quantize(x.cuda(), block=block)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K_", [(1, 1, 1), (1, 128, 128), (7, 33, 200), (128, 128, 128), (129, 130, 131), (16, 1000, 48),
                                    (300, 257, 1000), (1, 4096, 4096), (130, 5000, 640), (2000, 1300, 300), (2300, 2100, 300), (2300, 2304, 200), (130, 19001, 200)])
def test_gemm(hq, M, N, K_, dtype):
    check_gemm(hq, M, N, K_, dtype)


def check_gemm(hq, M, N, K_, dtype):
    g = torch.Generator().manual_seed(M + N + K_)
    a, w = codes(hq, g, M, K_, 1), codes(hq, g, N, K_, 128)
    a.scale *= torch.rand(a.scale.shape, generator=g).cuda() + 0.5   # scales need not be powers of two
    w.scale *= torch.rand(w.scale.shape, generator=g).cuda() + 0.5
    y = hq.gemm_fp8(a, w, dtype=dtype)
    av, wv = K.values(a.data)[:, :K_], K.values(w.data)[:, :K_]
    ref, size = np.zeros((M, N)), np.zeros((M, N))
    for t in range(-(-K_ // 128)):
        at = slice(128 * t, 128 * t + 128)
        f = K.values(a.scale)[t][:, None] * np.repeat(K.values(w.scale)[t], 128)[:N]
        ref += av[:, at] @ wv[:, at].T * f
        size += np.abs(av[:, at]) @ np.abs(wv[:, at]).T * f
    # 128 products and the blocks' sums in binary32, two roundings of the factor, one of the result
    tol = (128 + -(-K_ // 128) + 3) * 2.0 ** -23 * size + (2.0 ** -8 * np.abs(ref) if dtype == torch.bfloat16 else 0.0)
    assert np.all(np.abs(K.values(y) - ref) <= tol)


def test_gemm_ignores_the_padding_and_writes_in_place(hq):
    g = torch.Generator().manual_seed(3)
    a, w = codes(hq, g, 40, 100, 1), codes(hq, g, 50, 100, 128)
    ref = hq.gemm_fp8(a, w)
    for t in (a, w):
        t.data.view(torch.uint8)[:, 100:] = 0x7F   # NaN codes behind the columns
    out = torch.empty(40, 50, dtype=torch.bfloat16, device="cuda")
    ws = hq.fp8_workspace()
    assert hq.gemm_fp8(a, w, out=out, ws=ws) is out
    assert torch.equal(out, ref) and hq.status(ws)[0] == 0


def test_gemm_rows_do_not_depend_on_the_batch(hq):
    """Above sixteen rows (where K is not divided) a row's result is the same whichever rows stand beside it."""
    g = torch.Generator().manual_seed(4)
    w = codes(hq, g, 700, 900, 128)
    a = codes(hq, g, 600, 900, 1)
    whole = hq.gemm_fp8(a, w, dtype=torch.float32)
    for r in (0, 5, 500):
        some = hq.Fp8Code(100, 900, 1, a.data[r:r + 100].contiguous(), a.scale[:, r:r + 100].contiguous())
        assert torch.equal(hq.gemm_fp8(some, w, dtype=torch.float32), whole[r:r + 100])


@pytest.mark.parametrize("M", [1, 15, 16, 17, 32, 33, 63, 64, 65])
@pytest.mark.parametrize("N,K_", [(128, 128), (200, 300), (1000, 2000), (20000, 256), (130, 20000), (4096, 4096), (1024, 4096), (11008, 2100)])
def test_gemm_few_rows(hq, M, N, K_):
    """Both sides of the rules for few rows: K undivided and divided, more blocks than a ring holds."""
    check_gemm(hq, M, N, K_, torch.float32)


def test_graph_replay(hq):
    g = torch.Generator().manual_seed(5)
    w = codes(hq, g, 384, 512, 128)
    x = torch.randn(20, 512, generator=g).cuda()
    ref = hq.gemm_fp8(hq.fp8_quantize(x), w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = hq.gemm_fp8(hq.fp8_quantize(x), w)
    graph.replay()
    assert torch.equal(y, ref)
    x *= 2
    graph.replay()
    assert torch.equal(y, 2 * ref)
