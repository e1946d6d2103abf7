"""Which workspace a call of the log probabilities asks for, before any device call (CPU only)."""
import pytest

torch = pytest.importorskip("torch")

import moe_expert_offload_gemv_amd as moe  # noqa: E402
from tests.test_dense_refusals import P, _refused  # noqa: E402
from tests.test_head_refusals import LOGP  # noqa: E402


@pytest.mark.parametrize("T,V,needed", [
    (1, 20000, False), (1, 100000, True), (100, 131072, True), (300, 40000, False), (600, 70000, False), (4096, 1 << 22, False),
])
def test_only_a_call_that_cuts_its_rows_needs_one(T, V, needed):
    # the checks of the arguments come before that of the device, of which there is none of this number
    a = {**LOGP, "device": -1, "n_tokens": T, "n_vocab": V, "z_stride": V}
    size = moe.moe_token_logprobs_workspace_bytes(T, V, a["top_n"])
    _refused("moe_token_logprobs", {**a, "workspace_bytes": size}, "device")
    _refused("moe_token_logprobs", {**a, "workspace": None, "workspace_bytes": 0}, "workspace" if needed else "device")
    if needed:
        _refused("moe_token_logprobs", {**a, "workspace": 8 * P + 64}, "workspace")
