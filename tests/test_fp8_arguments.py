"""The 8-bit operators' argument checks (no GPU needed: refused before anything is launched), their
argument structs, and the 64-bit definitions that the GPU tests compare with."""

import os
import struct
import subprocess

import numpy as np
import pytest
import torch

import kv8_oracle as K
import post_quantization_tile_b200 as hq

ARG, UNSUPPORTED = 1, 2
# hq_kv8_append_t, hq_kv8_attend_t and hq_kv8_evict_t as packed bytes
_HEAD = "<4Qq3i4x"
APPEND = struct.Struct(_HEAD + "2Qi4x2q6qQ2q2Q")
ATTEND = struct.Struct(_HEAD + "2Q3q6qQ2q2QfiQ2q2Q4qq")
EVICT = struct.Struct(_HEAD + "qQ2qQQ2qq2qQ2q2Q2q")
PTR = 4096  # an aligned address that is never read


@pytest.fixture(scope="module")
def L():
    from post_quantization_tile_b200 import build
    build.build()
    return hq.lib()


def test_e4m3_definition_is_torchs():
    x = torch.cat([torch.linspace(-448, 448, 20001), torch.randn(20000, generator=torch.Generator().manual_seed(0)) * 0.02])
    assert np.array_equal(K.e4m3(x.double().numpy()), x.to(torch.float8_e4m3fn).double().numpy())
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    every = every[~every.isnan()].numpy()
    assert np.array_equal(K.e4m3(every), every)


def test_scale_definition():
    assert K.scale_of(0.0) == 2.0 ** -40 and K.scale_of(448.0) == 1.0 and K.scale_of(np.nextafter(448.0, 1e9)) == 2.0
    assert K.scale_of(1e30) == 2.0 ** 40 and K.scale_of(224.0) == 0.5


def test_attention_definition_is_a_softmax():
    g = torch.Generator().manual_seed(1)
    k, v, ks, vs = (K.values(t) for t in K.random_cache(g, 3, 1, 16, 64))
    q = torch.randn(1, 2, 3, 64, generator=g).double()
    out, lse, w, *_ = K.attend(q.numpy(), k, v, ks, vs, np.array([[2, 0]]), [20], [3], 0.125, True)
    kk = torch.from_numpy(np.concatenate([k[2, 0] * ks[2, 0], k[0, 0] * ks[0, 0]])[:20])
    vv = torch.from_numpy(np.concatenate([v[2, 0] * vs[2, 0], v[0, 0] * vs[0, 0]])[:20])
    mask = torch.ones(3, 20).tril(17).bool()
    s = (q[0] @ kk.t() * 0.125).masked_fill(~mask, -np.inf)
    assert np.allclose(out[0], (torch.softmax(s, 2) @ vv).numpy(), rtol=1e-12, atol=1e-12)
    assert np.allclose(lse[0], torch.logsumexp(s, 2).numpy()) and np.allclose(w[0, 0, :20], torch.softmax(s, 2).sum((0, 1)).numpy())


def quantize(L, x=PTR, dtype=0, rows=4, cols=100, ldx=100, block=1, q=PTR, ldq=112, scale=PTR, ws=None, wn=0):
    return L.hq_fp8_quantize(x, dtype, rows, cols, ldx, block, q, ldq, scale, ws, wn, None)


@pytest.mark.parametrize("bad,code", [(dict(x=None), ARG), (dict(q=None), ARG), (dict(scale=None), ARG), (dict(dtype=2), ARG),
                                      (dict(rows=0), ARG), (dict(cols=0), ARG), (dict(ldx=99), ARG), (dict(ldq=100), ARG),
                                      (dict(ldq=128), ARG), (dict(block=64), UNSUPPORTED), (dict(x=PTR + 1), ARG),
                                      (dict(q=PTR + 8), ARG), (dict(scale=PTR + 2), ARG), (dict(ws=PTR, wn=64), ARG),
                                      (dict(ws=PTR + 8, wn=1 << 20), ARG), (dict(rows=(1 << 31) + 1), ARG)])
def test_quantize_refuses(L, bad, code):
    assert quantize(L, **bad) == code


def gemm(L, A=PTR, lda=112, sa=PTR, M=4, W=PTR, ldw=112, sw=PTR, N=8, K_=100, Y=PTR, dtype=0, ws=None, wn=0):
    return L.hq_gemm_fp8(A, lda, sa, M, W, ldw, sw, N, K_, Y, dtype, ws, wn, None)


@pytest.mark.parametrize("bad,code", [(dict(A=None), ARG), (dict(W=None), ARG), (dict(sa=None), ARG), (dict(sw=None), ARG),
                                      (dict(Y=None), ARG), (dict(M=0), ARG), (dict(N=0), ARG), (dict(K_=0), ARG),
                                      (dict(lda=96), ARG), (dict(ldw=104), ARG), (dict(dtype=3), ARG), (dict(A=PTR + 8), ARG),
                                      (dict(W=PTR + 4), ARG), (dict(Y=PTR + 1), ARG), (dict(sa=PTR + 1), ARG),
                                      (dict(M=1 << 31), UNSUPPORTED), (dict(K_=(1 << 20) + 1, lda=1 << 21, ldw=1 << 21), UNSUPPORTED),
                                      (dict(ws=PTR, wn=8), ARG)])
def test_gemm_refuses(L, bad, code):
    assert gemm(L, **bad) == code


HEAD = dict(k=PTR, v=PTR, ks=PTR, vs=PTR, pages=8, heads=2, page=16, dim=64)


def head(d):
    h = {**HEAD, **{x: d.pop(x) for x in list(d) if x in HEAD}}
    return [h[x] for x in ("k", "v", "ks", "vs", "pages", "heads", "page", "dim")]


def append(L, ws=None, wn=0, **d):
    h = head(d)
    a = {**dict(xk=PTR, xv=PTR, dtype=0, B=2, S=3, st=[384, 192, 64] * 2, table=PTR, ts=4, P=4, lens=PTR, new=0), **d}
    return L.hq_kv8_append(APPEND.pack(*h, a["xk"], a["xv"], a["dtype"], a["B"], a["S"], *a["st"], a["table"], a["ts"],
                                               a["P"], a["lens"], a["new"]), ws, wn, None)


HEAD_BAD = [(dict(k=0), ARG), (dict(v=0), ARG), (dict(ks=0), ARG), (dict(vs=0), ARG), (dict(pages=0), ARG), (dict(heads=0), ARG),
            (dict(k=PTR + 8), ARG), (dict(vs=PTR + 2), ARG), (dict(page=48), UNSUPPORTED), (dict(page=256), UNSUPPORTED),
            (dict(dim=96), UNSUPPORTED), (dict(dim=256), UNSUPPORTED), (dict(table=0), ARG), (dict(lens=0), ARG), (dict(B=0), ARG),
            (dict(P=0), ARG), (dict(ts=3), ARG), (dict(table=PTR + 1), ARG)]


@pytest.mark.parametrize("bad,code", HEAD_BAD + [(dict(xk=0), ARG), (dict(xv=0), ARG), (dict(dtype=5), ARG), (dict(S=0), ARG),
                                                 (dict(st=[384, 192, 60] * 2), ARG), (dict(xk=PTR + 2), ARG),
                                                 (dict(new=PTR + 1), ARG), (dict(ws=PTR, wn=64), ARG)])
def test_append_refuses(L, bad, code):
    assert append(L, **bad) == code


def attend(L, ws=PTR, wn=1 << 40, **d):
    h = head(d)
    a = {**dict(q=PTR, out=2 * PTR, B=2, Hq=4, Sq=3, st=[768, 192, 64] * 2, table=PTR, ts=4, P=4, lens=PTR, ql=0, scale=0.125, causal=1,
                lse=0, win=0, w=0, most=64), **d}
    return L.hq_kv8_attend(ATTEND.pack(*h, a["q"], a["out"], a["B"], a["Hq"], a["Sq"], *a["st"], a["table"], a["ts"], a["P"],
                                               a["lens"], a["ql"], a["scale"], a["causal"], a["lse"], 12, 3, a["win"], a["w"], 128, 64,
                                               128, 64, a["most"]), ws, wn, None)


@pytest.mark.parametrize("bad,code", HEAD_BAD + [(dict(q=0), ARG), (dict(out=0), ARG), (dict(out=PTR), ARG), (dict(Sq=0), ARG), (dict(Hq=5), ARG),
                                                 (dict(Hq=1), ARG), (dict(st=[768, 192, 60] * 2), ARG), (dict(q=PTR + 8), ARG),
                                                 (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG),
                                                 (dict(win=PTR), ARG), (dict(w=PTR, most=0), ARG), (dict(B=5000), UNSUPPORTED),
                                                 (dict(ws=None), ARG), (dict(ws=PTR + 64), ARG), (dict(wn=100), ARG),
                                                 (dict(lse=PTR + 2), ARG), (dict(Sq=1 << 25), UNSUPPORTED)])
def test_attend_refuses(L, bad, code):
    assert attend(L, **bad) == code


def evict(L, ws=PTR, wn=1 << 40, **d):
    h = head(d)
    a = {**dict(B=2, table=PTR, ts=4, P=4, lens=PTR, w=PTR, most=64, budget=20, recent=4, to=PTR, tos=2, top=2, ol=PTR, ow=0), **d}
    return L.hq_kv8_evict(EVICT.pack(*h, a["B"], a["table"], a["ts"], a["P"], a["lens"], a["w"], 128, 64, a["most"], a["budget"],
                                             a["recent"], a["to"], a["tos"], a["top"], a["ol"], a["ow"], 40, 20), ws, wn, None)


@pytest.mark.parametrize("bad,code", HEAD_BAD + [(dict(w=0), ARG), (dict(most=0), ARG), (dict(budget=0), ARG), (dict(recent=-1), ARG),
                                                 (dict(budget=33), ARG), (dict(to=0), ARG), (dict(tos=1), ARG), (dict(ol=0), ARG),
                                                 (dict(ow=PTR), ARG), (dict(ws=None), ARG), (dict(wn=100), ARG)])
def test_evict_refuses(L, bad, code):
    assert evict(L, **bad) == code


def test_packed_structs_have_the_headers_sizes(tmp_path):
    src = tmp_path / "size.c"
    header = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "hq.h")
    src.write_text(f'#include <stdio.h>\n#include "{header}"\nint main(void) {{ printf("%zu %zu %zu", sizeof(hq_kv8_append_t), '
                   "sizeof(hq_kv8_attend_t), sizeof(hq_kv8_evict_t)); return 0; }\n")
    subprocess.run(["gcc", "-o", str(tmp_path / "size"), str(src)], check=True)
    sizes = subprocess.run([str(tmp_path / "size")], check=True, capture_output=True, text=True).stdout.split()
    assert sizes == [str(s.size) for s in (APPEND, ATTEND, EVICT)]


def test_workspace_sizes(L):
    assert L.hq_fp8_workspace_bytes() >= 64 + 8 * 4096
    one = L.hq_kv8_attend_workspace_bytes(2, 4, 8, 3, 128, 0)
    assert one > L.hq_fp8_workspace_bytes() and L.hq_kv8_attend_workspace_bytes(2, 4, 8, 3, 128, 1) >= one + 2 * 8 * 3 * 4
    assert L.hq_kv8_attend_workspace_bytes(0, 4, 8, 3, 128, 0) == 0 and L.hq_kv8_attend_workspace_bytes(2, 4, 8, 3, 96, 0) == 0
    assert L.hq_kv8_evict_workspace_bytes(2, 3, 10) >= 2 * 3 * 10 * 4 and L.hq_kv8_evict_workspace_bytes(2, 3, 0) == 0


def test_python_refuses_cpu_tensors_and_wrong_shapes(L):
    f8 = torch.zeros(4, 2, 16, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    cache = hq.Kv8Cache(f8, f8, torch.ones(4, 2), torch.ones(4, 2))
    i = torch.zeros(1, dtype=torch.int32)
    t = torch.zeros(1, 2, dtype=torch.int32)
    q = torch.zeros(1, 4, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        hq.fp8_quantize(torch.zeros(2, 3))
    a = hq.Fp8Code(1, 16, 1, f8[0, 0, :1, :16], torch.ones(1, 1))
    w = hq.Fp8Code(1, 16, 128, f8[0, 0, :1, :16], torch.ones(1, 1))
    for pair in ((a, w), (w, a), (a, a), (a, hq.Fp8Code(1, 32, 128, w.data, w.scale))):
        with pytest.raises(ValueError):
            hq.gemm_fp8(*pair)
    with pytest.raises(ValueError):
        hq.kv8_attend(q, cache, t, i)
    with pytest.raises(ValueError):
        hq.kv8_append(cache, q, q, t, i)
    with pytest.raises(ValueError):
        hq.kv8_evict(cache, t, i, torch.zeros(1, 2, 32), 4, 1, t)
    for bad in (None, 3, "x", [1.0]):
        with pytest.raises(ValueError):
            hq._native().fp8_quantize(bad, 1, None, None, None)
    with pytest.raises(TypeError):
        hq._native().kv8_append(1, 2)


def test_dequantize_is_code_times_scale():
    x = torch.randn(5, 140, generator=torch.Generator().manual_seed(2))
    q, s = K.quantize(x.double().numpy(), 1)
    data = torch.zeros(5, 144)
    data[:, :140] = torch.from_numpy(q)
    code = hq.Fp8Code(5, 140, 1, data.to(torch.float8_e4m3fn), torch.from_numpy(s).float())
    want = q * np.repeat(s.T, 128, axis=1)[:, :140]
    assert np.array_equal(code.dequantize().double().numpy(), want) and np.abs(want - x.numpy()).max() < 2.0 ** -4 * np.abs(x.numpy()).max()
