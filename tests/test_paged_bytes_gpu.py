"""The bytes of 8-bit rows' powers, all 256 of them, as the operators of pages read them."""
import pytest
import torch

from decode_megakernel_llama_gb300 import _lib
from decode_megakernel_llama_gb300.build import build
from tests import paged_reference as ref
from tests.test_paged_gpu import Paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def test_every_byte_reads_as_the_header_says():
    """Up to 134 the value, rounded to bf16 where its last bit, 2^(s - 136), is below bf16's 2^-133; above not a number."""
    dev = torch.device("cuda")
    codes = torch.arange(256, dtype=torch.uint8).view(1, 1, 1, 4, 64).repeat(1, 256, 1, 2, 1)
    codes[(codes & 127) == 127] = 0
    scales = torch.arange(256, dtype=torch.uint8).view(1, 256, 1, 1, 1).expand(1, 256, 1, 8, 2).contiguous().to(dev)
    k, v = (torch.zeros(1, 256, 1, 8, 64, dtype=torch.bfloat16, device=dev) for _ in range(2))
    kp = codes.to(dev).view(ref.E4M3)
    _lib.kv_read_pages(kp, kp.clone(), k, v, torch.arange(256, dtype=torch.int32, device=dev)[:, None],
                       torch.full((256,), 8, dtype=torch.int32, device=dev), k_scales=scales, v_scales=scales.clone())
    want = ref.values(kp, scales)[0]
    assert torch.equal(k[0, :135], want[:135].bfloat16()) and torch.equal(k[0, 3:135].double(), want[3:135])
    assert bool(k[0, 135:].isnan().all()) and torch.equal(k.nan_to_num(9.0), v.nan_to_num(9.0))


@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("byte", [134, 135, 254])
@pytest.mark.parametrize("hd,new", [(64, 3), (128, 3), (64, 150), (128, 150)])
def test_attention_over_large_bytes(byte, hd, new, type):
    """A value's block with the byte, in the last row but one: the tokens that see it are no numbers above 134, the others
    are not touched."""
    p = Paged([300], [new], 4, 2, hd, 16, type, "e4m3", seed=byte)
    page, row = int(p.table[0, 298 // 16]), 298 % 16
    p.vs[page, 1, row, 1] = byte
    values = ref.values(p.v, torch.where(p.vs > 134, 255, p.vs))
    p.v64 = values
    p.run()
    p.check()
    assert bool(p.out[:new - 2].isfinite().all())
    last = p.out[new - 2:new, 2:, 32:64]
    assert bool(last.isfinite().all()) == (byte == 134)
