"""Failure detection of the e4m3 product without a GPU fault: where a bounded wait runs out, the kernel
reports HQ_ERR_TIMEOUT, leaves nothing under way behind it, and the context stays usable."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu
# sizes of the three kernels (few rows divided over clusters, tiles of one CTA, pairs of CTAs), a withheld block and the
# stages of the ring
CASES = [(16, 130, 20000, 3, 8), (333, 1000, 1460, 2, 8), (300, 2000, 1460, 0, 8), (2560, 2560, 2000, 4, 5)]


@pytest.fixture(scope="module")
def hq():
    import post_quantization_tile_b200 as m
    m.lib()
    return m


@pytest.fixture(scope="module")
def silent(hq):
    """The test library's product whose tensor-core work stops at a block."""
    from post_quantization_tile_b200 import build
    T = ctypes.CDLL(build.TEST_LIB)
    f = T.hq_test_gemm_fp8_silent_block
    P, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    f.argtypes = [P, i64, P, i64, P, i64, P, i64, i64, P, i32, P, ctypes.c_size_t, i32, P, P]
    f.restype = i32
    return f


def run(hq, silent, M, N, K_, block):
    g = torch.Generator().manual_seed(M)
    a = hq.fp8_quantize(torch.randn(M, K_, generator=g).cuda())
    w = hq.fp8_quantize(torch.randn(N, K_, generator=g).cuda(), block=128)
    ref = hq.gemm_fp8(a, w)
    y, ws, log = torch.empty_like(ref), hq.fp8_workspace(), torch.zeros(4096, 3, dtype=torch.int32, device="cuda")
    ld = a.data.shape[1]
    assert silent(a.data.data_ptr(), ld, a.scale.data_ptr(), M, w.data.data_ptr(), ld, w.scale.data_ptr(), N, K_, y.data_ptr(), 0,
                  ws.ptr(), ws.nbytes, block, log.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    assert hq.status(ws)[0] == 6
    assert torch.equal(hq.gemm_fp8(a, w, ws=ws), ref) and hq.status(ws)[0] == 0
    log = log.cpu()
    return log[log[:, 0] > 0]


@pytest.mark.parametrize("M,N,K_,block,stages", CASES)
def test_no_box_is_under_way_after_a_timeout(hq, silent, M, N, K_, block, stages):
    log = run(hq, silent, M, N, K_, block)
    assert len(log)
    for issued, landed, _ in log.tolist():
        assert issued == block + stages and landed == stages


@pytest.mark.parametrize("M,N,K_,block,stages", CASES)
def test_no_tensor_core_work_is_under_way_after_a_timeout(hq, silent, M, N, K_, block, stages):
    log = run(hq, silent, M, N, K_, block)
    assert len(log) and torch.all(log[:, 2] == 1)


@pytest.mark.parametrize("M,N,K_,block,stages", CASES)
def test_the_test_librarys_own_product_withholds_nothing(hq, M, N, K_, block, stages):
    from post_quantization_tile_b200 import build
    P, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    f = ctypes.CDLL(build.TEST_LIB).hq_gemm_fp8
    f.argtypes, f.restype = [P, i64, P, i64, P, i64, P, i64, i64, P, i32, P, ctypes.c_size_t, P], i32
    g = torch.Generator().manual_seed(M)
    a = hq.fp8_quantize(torch.randn(M, K_, generator=g).cuda())
    w = hq.fp8_quantize(torch.randn(N, K_, generator=g).cuda(), block=128)
    y, ws, ld = torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), hq.fp8_workspace(), a.data.shape[1]
    assert f(a.data.data_ptr(), ld, a.scale.data_ptr(), M, w.data.data_ptr(), ld, w.scale.data_ptr(), N, K_, y.data_ptr(), 0, ws.ptr(), ws.nbytes,
             torch.cuda.current_stream().cuda_stream) == 0
    assert hq.status(ws)[0] == 0 and torch.equal(y, hq.gemm_fp8(a, w))
