"""The example that runs the operators and the layer together: one
mixture-of-experts block, against its plain FP32 form.

Bounds.  The routed experts keep BF16 activations (decode band) and the
shared expert's two quantisations are each within half an E4M3 step (1/16 of
a value, about 1/40 root mean square), so the block's output, a sum of both,
stays within a cosine of 0.995; past the decode band the routed experts'
activations are NVFP4 (cosine 0.987 on their own).  The residual is FP32
arithmetic rounded to BF16."""
import pytest

from tests.gpu_util import ensure_built

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,cos", [(1, 0.995), (8, 0.995), (24, 0.98)])
def test_block_matches_its_plain_form(tokens, cos):
    ensure_built()
    from examples import moe_block
    got = moe_block.main(["--tokens", str(tokens), "--experts", "24", "--hidden", "1024", "--intermediate", "192",
                          "--top-k", "4"])
    assert got["cos_residual"] > 0.99999 and got["cos_block"] > cos and got["cos_graph"] > 0.9999
