"""Embedding rows of every short width and phase, at a scale of 1 bit for bit: NaN payloads
included, nothing written beside the rows."""
import pytest
import torch

from row_wise_normalization_gb300 import capi
from token_util import CODE, DT, Framed

pytestmark = pytest.mark.gpu
BITS = {"f32": torch.int32, "bf16": torch.int16, "f16": torch.int16}


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("off_o", [0, 1, 2, 5, 7])
def test_rows_of_every_short_width_and_phase(dtype, off_o):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(off_o)
    n, vocab = 9, 7
    tok = torch.tensor([3, 0, -1, 6, 6, 2, 7, 5, 1], device="cuda")
    there = (tok >= 0) & (tok < vocab)
    lim = 1 << (31 if dtype == "f32" else 15)
    for d in range(1, 45):
        for off_t in range(4 if dtype == "f32" else 8):
            bits = torch.randint(-lim, lim, (vocab, d), device="cuda", generator=gen)
            bits = bits.to(BITS[dtype])
            ldt, ldo = d + off_t % 3, d + d % 2
            table = Framed(vocab, d, DT[dtype], ldt, off_t, fill=bits.view(DT[dtype]))
            out = Framed(n, d, DT[dtype], ldo, off_o)
            capi.check(capi.embed_fwd(CODE[dtype], 1, tok.data_ptr(), table.view.data_ptr(), ldt,
                                      out.view.data_ptr(), ldo, n, vocab, d, 1.0,
                                      torch.cuda.current_stream().cuda_stream))
            want = torch.where(there[:, None], bits[tok.clamp(0, vocab - 1)], 0)
            got = out.view.contiguous().view(BITS[dtype])
            assert torch.equal(got, want), (d, off_t)
            out.check((d, off_t))
