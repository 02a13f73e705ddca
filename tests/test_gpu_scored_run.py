"""The scored decode, the choice of tokens and the compaction together, as a decode loop
under a budget uses them, and the decode of a prefix that the radix cache found."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import gpu_harness as H  # noqa: E402
from bit_kv_cache_evict_gb300 import build as B  # noqa: E402
from bit_kv_cache_evict_gb300 import oscar as O  # noqa: E402
from bit_kv_cache_evict_gb300 import synth as S  # noqa: E402
from history_scene import NSLOT, SCALE, Scene, out_tolerance, weight_tolerance  # noqa: E402

D = 128


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    O.lib()


def block(c):
    return (O.block_bytes if c.bits == 2 else O.block_bytes_int4)(c.sh)


@pytest.mark.parametrize("bits", [2, 4])
def test_a_decode_loop_under_a_budget(bits):
    """Three steps (the oldest window token evicted with its score, the new one in its slot, the scored decode), then
    half of the history dropped by score, then one more step over what was kept."""
    hq, hk, g, lens = 8, 2, 32, [500, 130]
    c = Scene(30, bits, lens, hq, hk, g, std=2.0)
    n_seq, steps, rng = 2, 3, np.random.default_rng(5)
    # room for the steps' tokens and for the compacted histories
    total = [n + steps + 1 for n in lens]
    need = [(t + 63) // 64 for t in total]
    c.max_pages = max(need)
    spare = iter(range(c.num_pages, c.num_pages + 40))
    table = np.full((n_seq, c.max_pages), -1, np.int32)
    for b in range(n_seq):
        old = c.table[b][c.table[b] >= 0][:need[b]]
        table[b, :len(old)] = old
        for i in range(len(old), need[b]):
            table[b, i] = next(spare)
    c.table = table
    fresh = np.array([[next(spare) for _ in range(c.max_pages)] for _ in range(n_seq)], np.int32)
    c.num_pages += 40
    c.pool = np.concatenate([c.pool, np.zeros(40 * hk * block(c), np.uint8)])
    d = c.device()
    evict = O.oscar_evict_quantize if bits == 2 else O.oscar_evict_quantize_int4
    clip = torch.full((hk, 2), 0.95, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    weight, slot_weight = torch.zeros(n_seq, 64 * c.max_pages, device="cuda"), torch.zeros(n_seq, NSLOT, device="cuda")
    ws = torch.empty(O.oscar_decode_workspace_bytes_weights(c.sh, bits, n_seq, c.max_pages), dtype=torch.uint8, device="cuda")
    out = torch.empty(n_seq, hq, D, device="cuda")
    seq = torch.arange(n_seq, dtype=torch.int32, device="cuda")
    for step in range(steps):
        slot = 64 + step
        row = seq * NSLOT + slot
        new = H.bf16_t(S.bf16_bits(2 * rng.standard_normal((n_seq, hk, 2, D))))
        evict(c.sh, d["kv"].view(n_seq * NSLOT, hk, 2, D), seq, d["hist"], d["U"], clip, d["pool"], d["table"], n_seq, c.max_pages, c.num_pages,
              src_row=row, new_kv=new, dev_status=status)
        weight[torch.arange(n_seq), d["hist"].long()] = slot_weight[:, slot]   # the token's score goes with it
        slot_weight[:, slot] = 0
        d["hist"] += 1
        before, before_slots = weight.clone(), slot_weight.clone()
        d["q"] = H.bf16_t(S.bf16_bits(rng.standard_normal((n_seq, hq, D))))
        O.oscar_decode_attn_weights(c.sh, bits, d["q"], d["kv"], d["len"], d["pool"], d["table"], c.max_pages, c.num_pages, d["hist"], d["U"],
                                    SCALE, out, weight, ws, slot_weight=slot_weight, dev_status=status)
        # the state as it is now, in 64 bits
        c.pool, c.hist = d["pool"].cpu().numpy(), d["hist"].cpu().numpy()
        c.kv, c.q = (d[k].view(torch.int16).cpu().numpy().view(np.uint16) for k in ("kv", "q"))
        ref, rw, rsw, mag, we, swe = c.want()
        assert (np.abs(out.cpu().numpy() - ref) <= out_tolerance(ref, mag, bits, False)).all()
        was, was_slots = before.cpu().numpy().astype(np.float64), before_slots.cpu().numpy().astype(np.float64)
        inside = np.arange(rw.shape[1]) < c.hist[:, None]
        assert (np.abs(weight.cpu().numpy() - was - rw)[inside] <= weight_tolerance(rw, we, was, hq, bits)[inside]).all()
        assert (np.abs(slot_weight.cpu().numpy() - was_slots - rsw) <= weight_tolerance(rsw, swe, was_slots, hq, bits)).all()
    # half of each history stays; the newest 16 whatever their score
    budget = (d["hist"] // 2).int()
    keep = torch.full((n_seq, 64 * c.max_pages), -1, dtype=torch.int32, device="cuda")
    n_keep, kept = torch.zeros_like(budget), torch.zeros_like(weight)
    O.oscar_history_select(weight, d["hist"], budget, keep, n_keep, protect=16, kept_weight=kept, dev_status=status)
    fresh_dev = H.i32_t(fresh)
    O.oscar_history_gather(c.sh, bits, d["pool"], d["table"], fresh_dev, keep, n_keep, c.num_pages, dev_status=status)
    w, n = weight.cpu().numpy(), n_keep.cpu().numpy()
    for b in range(n_seq):
        h = int(c.hist[b])
        assert n[b] == h // 2
        order = np.concatenate([np.arange(h - 16, h), np.lexsort((np.arange(h - 16), -w[b, :h - 16]))])[:n[b]]
        assert np.array_equal(keep[b, :n[b]].cpu().numpy(), np.sort(order))
        assert np.array_equal(kept[b, :n[b]].cpu().numpy(), w[b][np.sort(order)])
    O.oscar_decode_attn_weights(c.sh, bits, d["q"], d["kv"], d["len"], d["pool"], fresh_dev, c.max_pages, c.num_pages, n_keep, d["U"], SCALE, out,
                                kept, ws, dev_status=status)
    c.pool, c.table, c.hist = d["pool"].cpu().numpy(), fresh, n
    ref, rw, _, mag, we, _ = c.want()
    assert (np.abs(out.cpu().numpy() - ref) <= out_tolerance(ref, mag, bits, False)).all()
    assert int(status) == 0


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_prefix_that_the_radix_cache_found(bits, dtype):
    """The pages of a cached prompt are adopted by five sequences, which decode them together; two others have their own."""
    shared, tails = 8, [70, 1, 0, 130, 64]
    c = Scene(31, bits, [64 * shared + t for t in tails] + [200, 700], 16, 4, 64, groups=[0] * 5 + [-1, -1], shared=shared, std=2.0)
    pages = O.Pages(c.num_pages)
    pages.alloc(c.num_pages)                               # (the scene has laid them all out)
    radix = O.Radix(pages)
    tokens = np.random.default_rng(0).integers(0, 1000, 64 * (1 + shared) + 20).astype(np.int32)
    radix.insert(tokens, c.table[0, :shared])
    for b in range(1, 5):                                  # each finds the same pages behind the same tokens
        found = radix.match(np.concatenate([tokens[:64 * (1 + shared)], [b]]).astype(np.int32), 100)
        assert np.array_equal(found, c.table[b, :shared])
        pages.release(found)
    d = c.device()
    want = c.want()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.empty(c.B, c.hq, D, dtype=dtype, device="cuda")
    ws = torch.empty(O.oscar_decode_workspace_bytes_shared(c.sh, bits, c.B, c.max_pages, 1), dtype=torch.uint8, device="cuda")
    for least in (2, 0):
        O.oscar_decode_attn_shared(c.sh, bits, d["q"], d["kv"], d["len"], d["pool"], d["table"], c.max_pages, c.num_pages, d["hist"], d["group"],
                                   H.i32_t([len(found)]), d["U"], SCALE, out, ws, min_members=least, dev_status=status)
        got = out.float().cpu().numpy()
        assert (np.abs(got - want[0]) <= out_tolerance(want[0], want[3], bits, dtype == torch.bfloat16, dtype == torch.bfloat16)).all()
    assert int(status) == 0
    radix.close()
    pages.close()
