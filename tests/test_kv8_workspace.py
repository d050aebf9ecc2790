"""The attention's workspace follows the call: what its queries and tables need, at most what
hq_kv8_attend_workspace_bytes says for the longest tables (no GPU needed)."""
import pytest

from test_fp8_arguments import ATTEND, L, PTR, head  # noqa: F401


def need(L, **d):  # noqa: F811
    h = head(d)
    a = {**dict(B=1, Hq=2, Sq=1, P=4, w=0), **d}
    return L.hq_kv8_attend_workspace_need(ATTEND.pack(*h, PTR, 2 * PTR, a["B"], a["Hq"], a["Sq"], *[768, 192, 64] * 2, PTR, a["P"], a["P"],
                                                      PTR, 0, 0.125, 1, 0, 12, 3, 0, a["w"], 128, 64, 128, 64, 64))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rows", [1, 8, 9, 32, 33, 300, 4096])
def test_need_grows_with_the_table_up_to_the_bound(L, rows, dim):  # noqa: F811
    most = L.hq_kv8_attend_workspace_bytes(3, 2, 4, rows, dim, 0)
    sizes = [need(L, B=3, Hq=4, Sq=rows, dim=dim, P=P) for P in (1, 4, 30, 1000, 1 << 24)]
    assert sizes == sorted(sizes) and 0 < sizes[0] and sizes[-1] == most
    assert need(L, B=3, Hq=4, Sq=rows, dim=dim, P=1, w=PTR) >= sizes[0] + 4 * 3 * 4 * rows


def test_short_calls_need_little(L):  # noqa: F811
    """One unit of 256 rows over one tile: a share's two parts of 256 rows, and the status slots."""
    parts = 2 * 256 * (128 * 4 + 8)
    assert need(L, dim=128, Sq=33, P=4, heads=2, Hq=2) <= 2 * parts + 40000       # two heads, 64 slots
    assert need(L, dim=128, Sq=33, P=4, heads=1, Hq=1) <= parts + 40000
    assert L.hq_kv8_attend_workspace_bytes(1, 1, 1, 33, 128, 0) <= 148 * parts + 40000


@pytest.mark.parametrize("bad", [dict(B=0), dict(Hq=3), dict(Sq=0), dict(P=0), dict(dim=96), dict(page=48), dict(B=5000)])
def test_need_of_a_call_that_is_refused_is_zero(L, bad):  # noqa: F811
    assert need(L, **bad) == 0
