"""Arguments of the beam step that its C ABI cannot hold (on a host without a GPU)."""
import pytest

import fp32_gemm_f32_amd as g


@pytest.mark.parametrize("pad", [2 ** 63, -2 ** 63 - 1, 2 ** 64 + 2, 10 ** 30])
def test_a_pad_token_past_64_bits_is_refused(pad):
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError, match="pad_token"):
        g.beam_step(torch.zeros(2, 4), torch.zeros(1, 2), pad_token=pad)
    for fits in (2 ** 63 - 1, -2 ** 63):
        with pytest.raises(ValueError, match="GPU"):
            g.beam_step(torch.zeros(2, 4), torch.zeros(1, 2), pad_token=fits)
