"""The choice of history tokens by their scores on the GPU against a plain sort (exact)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from bit_kv_cache_evict_gb300 import build as B  # noqa: E402
from bit_kv_cache_evict_gb300 import oscar as O  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    O.lib()


def ref_select(w, n, m, protect):
    """Kept positions of one row, in increasing order."""
    m = min(m, n)
    newest = min(protect, m)
    x = w[:n - newest].astype(np.float64)
    x = np.where(np.isnan(x), np.inf, x)
    nan = np.isnan(w[:n - newest])
    order = np.lexsort((np.arange(n - newest), -x, ~nan))   # NaN first, then by score, then by position
    return np.sort(np.concatenate([order[:m - newest], np.arange(n - newest, n)])).astype(np.int64)


def run(w, hist, budget, protect, keep_stride=None, kept=True, status=None):
    w = torch.from_numpy(np.ascontiguousarray(w, np.float32)).cuda()
    i32 = lambda a: torch.from_numpy(np.array(a, np.int32)).cuda()  # noqa: E731
    keep = torch.full((w.shape[0], keep_stride if keep_stride is not None else max(1, w.shape[1])), -7, dtype=torch.int32, device="cuda")
    n = torch.full((w.shape[0],), -7, dtype=torch.int32, device="cuda")
    kw = torch.full(keep.shape, -7.0, device="cuda") if kept else None
    O.oscar_history_select(w, i32(hist), i32(budget), keep, n, protect=protect, kept_weight=kw, dev_status=status)
    return keep.cpu().numpy(), n.cpu().numpy(), None if kw is None else kw.cpu().numpy()


def check(w, hist, budget, protect, **k):
    keep, n, kw = run(w, hist, budget, protect, **k)
    for b in range(len(hist)):
        want = ref_select(w[b], hist[b], budget[b], protect)
        assert n[b] == len(want), (b, n[b], len(want))
        assert np.array_equal(keep[b, :n[b]], want), (b, hist[b], budget[b], protect)
        assert (keep[b, n[b]:] == -7).all()
        if kw is not None:
            assert np.array_equal(kw[b, :n[b]].view(np.uint32), np.float32(w[b])[want].view(np.uint32))
            assert (kw[b, n[b]:] == -7).all()


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 64, 705, 1023, 1025, 4097, 16385, 32449])
@pytest.mark.parametrize("protect", [0, 1, 64])
def test_lengths(n, protect):
    rng = np.random.default_rng(n + protect)
    w = rng.lognormal(0, 2, (5, n + 3)).astype(np.float32)
    hist = [n, n, max(0, n - 1), n // 2, 0]
    budget = [n // 2, n, 1, n // 3 + 1, 5]
    check(w, hist, budget, protect)


@pytest.mark.parametrize("values", ["few", "equal", "signs", "bits"])
def test_ties_signs_and_neighbours(values):
    rng = np.random.default_rng(1)
    shape = (6, 9001)
    if values == "few":
        w = rng.integers(0, 5, shape).astype(np.float32) / 4
    elif values == "equal":
        w = np.full(shape, 0.125, np.float32)
    elif values == "signs":
        w = rng.standard_normal(shape).astype(np.float32)
        w[:, ::7] = 0.0
        w[:, 3::7] = -0.0                                  # counts as 0: the lower position goes first
    else:                                                  # neighbours: only the last bits differ
        w = (np.uint32(0x3F800000) + rng.integers(0, 3000, shape).astype(np.uint32)).view(np.float32)
    hist = [9001, 9000, 8192, 4097, 100, 9001]
    for budget in ([4500] * 6, [1, 8999, 8191, 17, 99, 9000], [0, 9001, 20000, 2, 50, 3]):
        check(w, hist, budget, 16)


def test_infinities_and_nan():
    rng = np.random.default_rng(2)
    w = rng.standard_normal((3, 3000)).astype(np.float32)
    w[:, ::50] = np.inf
    w[:, 1::50] = -np.inf
    w[:, 2::50] = np.nan
    w[:, 3::200] = -np.nan
    for m in (10, 70, 130, 1500, 2950):
        check(w, [3000, 2999, 1500], [m, m, min(m, 1490)], 5)
    w[1, 2000:] = np.nan                                   # behind the history: not looked at
    check(w, [3000, 2000, 100], [500, 500, 50], 0)


@pytest.mark.parametrize("protect", [0, 10, 300, 5000])
def test_protected_tokens_and_budgets(protect):
    rng = np.random.default_rng(3)
    w = rng.random((8, 1000)).astype(np.float32)
    check(w, [1000, 1000, 1000, 300, 299, 10, 1, 0], [500, 10, 1000, 300, 400, 11, 1, 3], protect)
    check(w, [1000, 1000, 1000, 300, 299, 10, 1, 0], [0, 1, 9, 299, 1, 9, 0, 0], protect, kept=False)


def test_longer_than_the_blocks_keep():
    rng = np.random.default_rng(4)
    n = 8 * 32768 + 777
    w = rng.random((2, n)).astype(np.float32)
    w[1] = (w[1] * 100).round()
    check(w, [n, n - 5], [n // 2, 1000], 100)


@pytest.mark.parametrize("batch", [1, 37, 400])
def test_batches(batch):
    rng = np.random.default_rng(batch)
    w = rng.lognormal(0, 1, (batch, 2500)).astype(np.float32)
    hist = rng.integers(0, 2501, batch)
    check(w, hist, rng.integers(0, 2501, batch), 32)


def test_bad_lengths_are_clamped_and_reported():
    rng = np.random.default_rng(5)
    w = rng.random((4, 500)).astype(np.float32)
    for hist, budget, stride in (([501, 500, 500, 500], [10] * 4, 500), ([500] * 4, [10, -1, 10, 10], 500), ([-3, 500, 500, 500], [10] * 4, 500),
                                 ([500] * 4, [10, 10, 101, 10], 100)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        keep, n, _ = run(w, hist, budget, 4, keep_stride=stride, status=status)
        assert int(status) == O.OSCAR_STATUS_BAD_POS
        for b in range(4):
            m = min(max(budget[b], 0), stride)
            assert np.array_equal(keep[b, :n[b]], ref_select(w[b], min(max(hist[b], 0), 500), m, 4))


def test_a_captured_call_follows_its_inputs():
    rng = np.random.default_rng(6)
    w = torch.from_numpy(rng.random((3, 5000)).astype(np.float32)).cuda()
    hist, budget = (torch.tensor(a, dtype=torch.int32, device="cuda") for a in ([5000, 100, 3000], [1000, 50, 10]))
    keep, n = torch.zeros(3, 5000, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    O.oscar_history_select(w, hist, budget, keep, n, protect=8)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        O.oscar_history_select(w, hist, budget, keep, n, protect=8)
    for step in range(3):
        w.copy_(torch.from_numpy(rng.random((3, 5000)).astype(np.float32)))
        hist -= 7
        budget += 3
        graph.replay()
        for b in range(3):
            want = ref_select(w[b].cpu().numpy(), int(hist[b]), int(budget[b]), 8)
            assert int(n[b]) == len(want) and np.array_equal(keep[b, :len(want)].cpu().numpy(), want)


@pytest.mark.parametrize("n", [700, 20000])
def test_the_new_lengths_over_the_old(n):
    """n_keep may be hist_len or budget itself: one thread block per sequence, and several."""
    rng = np.random.default_rng(n)
    w = rng.random((3, n)).astype(np.float32)
    old = {"hist": [n, n // 2, 9], "budget": [n // 3, n, 0]}
    for place in old:
        t = {k: torch.tensor(v, dtype=torch.int32, device="cuda") for k, v in old.items()}
        keep = torch.zeros(3, n, dtype=torch.int32, device="cuda")
        O.oscar_history_select(torch.from_numpy(w).cuda(), t["hist"], t["budget"], keep, t[place], protect=5)
        for b in range(3):
            want = ref_select(w[b], old["hist"][b], old["budget"][b], 5)
            assert int(t[place][b]) == len(want) and np.array_equal(keep[b, :len(want)].cpu().numpy(), want)
