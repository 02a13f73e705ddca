"""The split of one long sequence's pages by the decode that accumulates attention weight, as the call leaves it in its
workspace: the offsets of the long items int32 [batch + 1] 256 bytes in, those of the short ones on the next 256 bytes."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from bit_kv_cache_evict_gb300 import build as B  # noqa: E402
from bit_kv_cache_evict_gb300 import oscar as O  # noqa: E402


@pytest.mark.parametrize("hq,dtype,per_sm", [(64, torch.float32, 2), (64, torch.bfloat16, 3), (32, torch.float32, 3)])
def test_one_long_sequence_in_one_wave(hq, dtype, per_sm):
    """A sequence of fewer pages than two waves of the shortest items is split into one wave of the blocks that run side by
    side: two per SM with eight heads per KV head and an fp32 output, else three."""
    B.build()
    hk, sms = 8, torch.cuda.get_device_properties(0).multi_processor_count
    pages = 29 * sms * per_sm // hk                        # 29 for each block
    sh = O.make_shape(hq, hk, quant_group=128)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    pool = torch.zeros(2 * hk * O.block_bytes(sh), dtype=torch.uint8, device="cuda")
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None] % 2
    ws = torch.zeros(O.oscar_decode_workspace_bytes_weights(sh, 2, 1, pages), dtype=torch.uint8, device="cuda")
    out = torch.full((1, hq, 128), float("nan"), dtype=dtype, device="cuda")
    weight = torch.zeros(1, 64 * pages, device="cuda")
    q, kv = torch.zeros(1, hq, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 320, hk, 2, 128, dtype=torch.bfloat16, device="cuda")
    U = torch.eye(128, device="cuda").expand(hk, 2, 128, 128).contiguous()
    O.oscar_decode_attn_weights(sh, 2, q, kv, i32(0), pool, table, pages, 2, i32(64 * pages), U, 128 ** -0.5, out, weight, ws)
    items = int(ws[256:264].view(torch.int32)[1]) + int(ws[512:520].view(torch.int32)[1])
    assert sms * per_sm // 2 < items <= sms * per_sm, items
    # pools of zeros: every token has the same weight
    assert (weight * 64 * pages / hq - 1).abs().max() < 1e-5 and (out == 0).all()
