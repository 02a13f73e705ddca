"""Which groups attend their pages together, seen from outside: shared pages are read from the page-table row of a
group's first sequence alone, so that with -1 in the other members' rows a group that attends together gives the result
and status 0, and one whose members attend by themselves reports BAD_PAGE."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from bit_kv_cache_evict_gb300 import build as B  # noqa: E402
from bit_kv_cache_evict_gb300 import oscar as O  # noqa: E402
from history_scene import SCALE, Scene, out_tolerance  # noqa: E402

D = 128
F32, BF16 = torch.float32, torch.bfloat16
BOTH = pytest.mark.parametrize("bits", [2, 4])
TYPES = pytest.mark.parametrize("dtype", [F32, BF16])


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    O.lib()


def blind(c):
    """The table with the groups' pages in the rows of their first sequences only (histories reach behind the pages)."""
    table, seen = c.table.copy(), set()
    for b in range(c.B):
        g = int(c.group[b])
        if g >= 0 and g in seen:
            table[b, :c.group_pages[g]] = -1
        seen.add(g)
    return table


def run(c, dtype, table, min_members):
    d = dict(getattr(c, "d", None) or c.device(), table=torch.from_numpy(table).cuda())
    out = torch.full((c.B, c.hq, D), float("nan"), dtype=dtype, device="cuda")
    ws = torch.empty(O.oscar_decode_workspace_bytes_shared(c.sh, c.bits, c.B, c.max_pages, c.n_groups), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    O.oscar_decode_attn_shared(c.sh, c.bits, d["q"], d["kv"], d["len"], d["pool"], d["table"], c.max_pages, c.num_pages, d["hist"], d["group"],
                               d["group_pages"], d["U"], SCALE, out, ws, min_members=min_members, dev_status=status)
    return out.float().cpu().numpy().astype(np.float64), int(status)


def check(c, got, want, dtype):
    assert (np.abs(got - want[0]) <= out_tolerance(want[0], want[3], c.bits, dtype == BF16, fp16_shared=dtype == BF16)).all()


@BOTH
@TYPES
@pytest.mark.parametrize("members,hq,hk", [(2, 1, 1), (5, 8, 1), (40, 8, 2)])
def test_min_members(bits, dtype, members, hq, hk):
    c = Scene(50 + members, bits, [64 * 6 + 3 * i for i in range(members)], hq, hk, 64, groups=[0] * members, shared=6)
    want, table = c.want(), blind(c)
    for least in (1, 2, members):
        got, status = run(c, dtype, table, least)
        assert status == 0, least
        check(c, got, want, dtype)
    assert run(c, dtype, table, members + 1)[1] == O.OSCAR_STATUS_BAD_PAGE
    got, status = run(c, dtype, c.table, members + 1)
    assert status == 0
    check(c, got, want, dtype)


@BOTH
@TYPES
def test_each_group_by_its_own_members(bits, dtype):
    """Three groups of two, three and four behind one minimum: those below it attend by themselves."""
    c = Scene(60, bits, [64 * 4 + 5] * 9, 4, 1, 32, groups=[0, 1, 2, 2, 1, 0, 2, 1, 2], shared=4)
    want, whole = c.want(), c.table
    for least, together in ((2, (0, 1, 2)), (3, (1, 2)), (4, (2,))):
        table = np.where(np.isin(c.group, together)[:, None], blind(c), whole)
        got, status = run(c, dtype, table, least)
        assert status == 0
        check(c, got, want, dtype)
        for g in set((0, 1, 2)) - set(together):
            assert run(c, dtype, np.where((c.group == g)[:, None], blind(c), table), least)[1] == O.OSCAR_STATUS_BAD_PAGE


@BOTH
@TYPES
def test_the_librarys_rule(bits, dtype):
    """min_members 0: pairs never, nine sequences behind many pages of 64 KV heads, not behind few."""
    for members, pages, together in ((2, 40, False), (9, 3, False), (9, 60, True)):
        c = Scene(61, bits, [64 * pages + i for i in range(members)], 64, 64, 128, groups=[0] * members, shared=pages)
        c.len[:] = 4
        table = blind(c)
        got, status = run(c, dtype, table, 0)
        assert status == (0 if together else O.OSCAR_STATUS_BAD_PAGE), (members, pages)
        if not together:
            got, status = run(c, dtype, c.table, 0)
            assert status == 0
        check(c, got, c.want(), dtype)
