"""A token of nearly all the weight before a long tail of equal ones in one run of shared pages, on the GPU: the
tail's weights reach the products of values as they reach the sum of weights."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from bit_kv_cache_evict_gb300 import build as B  # noqa: E402
from bit_kv_cache_evict_gb300 import oscar as O  # noqa: E402
from bit_kv_cache_evict_gb300 import synth as S  # noqa: E402
from history_scene import SCALE, Scene, f64, unpack  # noqa: E402

D = 128
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    O.lib()


def tail_scene(bits, pages, at, peak):
    """160 sequences in 80 pairs, so that a pair's pages are one item; all of them see the same `pages` pages: the token
    `at` of page 1 has the key (1.5, 1.5, ...) in the rotated domain and every other the key 0.  Queries are
    multiples of R (1, 1, ...), whose logits pass the tail's by peak[0] to peak[1] in base 2."""
    c = Scene(40, bits, [64 * 8] * 2, 1, 1, 128, groups=[0, 0], shared=8, wide=0)
    n = 160
    own = c.table[0, :8]                                   # page 1: the token; pages 0, 2 .. 7: the tail's
    blk = c.pool.reshape(c.num_pages, 1, -1)
    for page in own:
        for t in range(64):
            c.set_pairs(page, 0, 0, t, np.float16([[0, 1.5 if page == own[1] and t == at else 0]]))
            c.set_pairs(page, 0, 1, t, np.float16([[1.0 / (2 ** bits - 1), 0.5]]))   # values in [0.5, 1.5]
    assert blk.shape[0] == c.num_pages
    rng = np.random.default_rng(41)
    order = np.concatenate([[0, 1], 2 + rng.integers(0, 6, pages - 2)])
    c.B, c.max_pages, c.table = n, pages, np.repeat(own[order][None], n, 0).astype(np.int32)
    c.hist, c.len = np.full(n, 64 * pages, np.int32), np.zeros(n, np.int32)
    c.group, c.n_groups, c.group_pages = np.repeat(np.arange(n // 2), 2).astype(np.int32), n // 2, np.full(n // 2, pages, np.int32)
    ones = c.R[0][0] @ np.ones(D)
    want = np.linspace(peak[0], peak[1], n)                # base-2 logits: 1.5 c D SCALE / ln 2
    c.q = S.bf16_bits((want * np.log(2) / (1.5 * D * SCALE))[:, None, None] * ones)
    c.kv = np.zeros((n, O.make_shape(1, 1).sink + O.make_shape(1, 1).recent, 1, 2, D), np.uint16)
    # float64: the token's weight is 1, every other's 2^-gap (a query's gap from its bf16 bits)
    gap = f64(c.q)[:, 0] @ ones * 1.5 * SCALE / np.log(2)
    v = unpack(c.pool, 1, bits, 128)[:, 0, 1]              # [page][64][128]
    count = np.bincount(order, minlength=8)
    total = sum(count[i] * v[own[i]].sum(0) for i in range(8)) - v[own[1], at]
    tail = 2.0 ** -gap[:, None]
    ref = ((v[own[1], at] + tail * total) / (1 + tail * (64 * pages - 1))) @ c.R[0][1].T
    out = v[own].reshape(-1, D) @ c.R[0][1].T
    return c, ref, gap, np.minimum(tail * 64 * pages, 1), max(np.abs(v).max(), np.abs(out).max()), np.abs(out).mean(0)


def run(c, dtype):
    d = c.device()
    out = torch.full((c.B, 1, D), float("nan"), dtype=dtype, device="cuda")
    ws = torch.empty(O.oscar_decode_workspace_bytes_shared(c.sh, c.bits, c.B, c.max_pages, c.n_groups), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    O.oscar_decode_attn_shared(c.sh, c.bits, d["q"], d["kv"], d["len"], d["pool"], d["table"], c.max_pages, c.num_pages, d["hist"], d["group"],
                               d["group_pages"], d["U"], SCALE, out, ws, min_members=2, dev_status=status)
    assert int(status) == 0
    return out[:, 0].float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("at,peak", [(0, (20.3, 29.7)), (63, (20.3, 29.7)), (17, (10.1, 24.9))])
def test_fp32(bits, at, peak):
    """512 pages in a run.  Bound: a logit of size A = gap is off by A 2^-19, so a tail weight by 2 ln 2 A 2^-19, relatively
    (history_scene.out_tolerance), of the tail's part (mean |value| of an output); weights and values to 22 bits, 2^-20 together; the
    fp32 sums over the pages, 2^-24 each."""
    c, ref, gap, share, big, mean = tail_scene(bits, 512, at, peak)
    got = run(c, F32)
    tol = share * mean * 2 * gap[:, None] * 2.0 ** -19 + big * (2.0 ** -20 + 512 * 2.0 ** -24)
    err = np.abs(got - ref)
    assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("at,peak", [(0, (25.3, 27.7)), (63, (25.3, 27.7)), (0, (0.0, 0.5))])
def test_bf16(bits, at, peak):
    """16384 shared pages: a long tail (up to 2.5 % of the weight), and a flat softmax.  Bound: q' and k rounded to fp16 move a logit
    by A 2^-10 and a tail weight by 2 ln 2 times that; weights and values rounded to fp16, 2^-10 of the largest value; the
    products, truncated to 2^-24 of a sum over 256 pages at most: half of 2^14 2^-24 on the average of a flat softmax, and of a tail no more than its
    share in 256 pages is lost, 2^-11: 2^-11 of the largest; 2^-8 for the output."""
    c, ref, gap, share, big, mean = tail_scene(bits, 16384, at, peak)
    got = run(c, BF16)
    tol = share * mean * 2 * gap[:, None] * 2.0 ** -10 + big * (2.0 ** -10 + 2.0 ** -11) + np.abs(ref) * 2.0 ** -8
    err = np.abs(got - ref)
    assert (err <= tol).all(), (err / tol).max()
