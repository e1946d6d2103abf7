"""The binding of the operators beside the experts (CPU only): sizes and
flags that do not fit the library's 32-bit parameters are refused, not cut."""
import pytest

torch = pytest.importorskip("torch")

import moe_expert_offload_gemv_amd as moe  # noqa: E402


class Rows:
    """A tensor of the sizes asked for, in nobody's memory: no call here may get as far as touching it."""

    def __init__(self, *shape, dtype=torch.float32):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device("cuda", 0)

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return 0

    def stride(self):
        n = [1]
        for d in reversed(self.shape[1:]):
            n.insert(0, n[0] * d)
        return tuple(n)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x10000

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return torch.empty((), dtype=self.dtype).element_size()


def planes(n, k):
    return Rows(n, k // 32, 16, dtype=torch.uint8), Rows(n, k // 32, dtype=torch.float16)


MANY = (1 << 32) + 2  # 2 in 32 bits


def test_sizes_past_32_bits_are_refused():
    with pytest.raises(ValueError, match="x: shape"):
        moe.moe_add_rmsnorm(Rows(MANY, 64), None, Rows(MANY, 64))
    with pytest.raises(ValueError, match="x: shape"):
        moe.moe_add_rmsnorm(Rows(2, MANY), None, Rows(2, MANY))
    with pytest.raises(ValueError, match="x: shape"):
        moe.moe_q4_matmul(Rows(MANY, 64), *planes(8, 64), Rows(MANY, 8))
    with pytest.raises(ValueError, match="nibbles: shape"):
        moe.moe_q4_matmul(Rows(2, 64), *planes(MANY, 64), Rows(2, MANY))
    for ws in (moe.moe_q4_workspace, lambda x, nib: moe.moe_q4_matmul(x, nib, None, None)):
        with pytest.raises(ValueError, match="x: shape"):
            ws(Rows(MANY, 64), planes(8, 64)[0])
    E = 8
    outs = [Rows(E, dtype=torch.int32), Rows(E), Rows(4)]
    with pytest.raises(ValueError, match="logits: shape"):
        moe.moe_router_balance(Rows(MANY, E), 2, *outs, Rows(MANY))
    with pytest.raises(ValueError, match="logits: shape"):
        moe.moe_router_balance_grad(Rows(MANY, E), outs[1], outs[2], Rows(MANY), Rows(MANY, E))
    with pytest.raises(ValueError, match="logits: shape"):
        moe.moe_router_balance_workspace(Rows(MANY, E))


def test_workspace_sizes_of_sizes_past_32_bits():
    for bad in ((MANY, 8, 64, 0), (2, MANY, 64, 0), (2, 8, (1 << 32) + 64, 0), (2, 8, 64, 1 << 32), (2 - (1 << 33), 8, 64, 0)):
        assert moe.moe_q4_workspace_bytes(*bad) == -1
    assert moe.moe_router_balance_workspace_bytes(MANY, 8) == -1
    assert moe.moe_router_balance_workspace_bytes(2, (1 << 32) + 8) == -1


def test_flags_and_picks_past_32_bits_are_refused(monkeypatch):
    monkeypatch.setattr(moe, "_stream_of", lambda stream, dev: None)
    ws = Rows(1 << 20, dtype=torch.uint8)
    E = 8
    outs = [Rows(E, dtype=torch.int32), Rows(E), Rows(4), Rows(2)]
    for top_k, flags, what in (((1 << 32) + 2, 0, "top_k"), (2, 1 << 32, "flags"), (2, -(1 << 40), "flags")):
        with pytest.raises(ValueError, match=what):
            moe.moe_router_balance(Rows(2, E), top_k, *outs, workspace=ws, flags=flags)
    with pytest.raises(ValueError, match="flags"):
        moe.moe_router_balance_grad(Rows(2, E), outs[1], outs[2], outs[3], Rows(2, E), flags=1 << 32)
    with pytest.raises(ValueError, match="flags"):
        moe.moe_q4_matmul(Rows(2, 64), *planes(8, 64), Rows(2, 8), workspace=ws, flags=1 << 32)


def test_tensors_of_other_dimensions_are_refused():
    one = Rows(64)
    with pytest.raises(ValueError, match="nibbles: shape"):
        moe.moe_q4_matmul(Rows(2, 64), Rows(), Rows(8, 2, dtype=torch.float16), Rows(2, 8))
    with pytest.raises(ValueError, match="x: shape"):
        moe.moe_q4_workspace(one, planes(8, 64)[0])
    with pytest.raises(ValueError, match="nibbles: shape"):
        moe.moe_q4_workspace(Rows(2, 64), one)
    with pytest.raises(ValueError, match="logits: shape"):
        moe.moe_router_balance_workspace(one)


def test_refusals_of_the_library_come_with_their_message(monkeypatch):
    monkeypatch.setattr(moe, "_stream_of", lambda stream, dev: None)
    with pytest.raises(moe.MoeError, match="moe_add_rmsnorm: eps -1"):
        moe.moe_add_rmsnorm(Rows(2, 64), None, Rows(2, 64, dtype=torch.bfloat16), eps=-1.0)
    with pytest.raises(moe.MoeError, match="moe_q4_matmul: x_scales go with 8-bit x"):
        moe.moe_q4_matmul(Rows(2, 64, dtype=torch.int8), *planes(8, 64), Rows(2, 8))
    E = 8
    outs, ws = [Rows(E, dtype=torch.int32), Rows(E), Rows(4), Rows(2)], Rows(1 << 20, dtype=torch.uint8)
    with pytest.raises(moe.MoeError, match="moe_router_balance: n_tokens 2, n_experts 8 or top_k 9 out of range"):
        moe.moe_router_balance(Rows(2, E), 9, *outs, workspace=ws)
    with pytest.raises(moe.MoeError, match="moe_router_balance_grad: unknown flags"):
        moe.moe_router_balance_grad(Rows(2, E), *outs[1:], Rows(2, E), flags=4)
    with pytest.raises(moe.MoeError, match="moe_q4_split: rows 5 or k 0 out of range") as e:
        moe.moe_q4_split(torch.zeros((5, 0, 18), dtype=torch.uint8).numpy())
    assert e.value.code == moe.MOE_E_INVAL


def test_a_workspace_serves_every_smaller_batch():
    tokens = sorted({1, 16, 31, 32, 33, 64, 65, 127, 128, 129, 200, 256, 257, 300, 512, 513, 1000, 1024, 2047, 2048, 2049, 2064,
                     4096, 4097, 8192, 16383, 16384, 16385, 40000, 1 << 20, (1 << 20) + 1, 1 << 24})
    for n_experts in (1, 8, 64, 65, 128, 129, 200, 256, 257, 512, 513, 1024, 2048, 4096):
        need = [moe.moe_router_balance_workspace_bytes(t, n_experts) for t in [0] + tokens]
        assert need == sorted(need), n_experts
    for x_type in (moe.MOE_F32, moe.MOE_F16, moe.MOE_BF16, moe.MOE_Q8_32):
        for n_out in (1, 64, 255, 256, 257, 1000, 4096, 5120, 65537, 1 << 22):
            for k in (32, 96, 256, 2048, 4096, 14336, 65536, 1 << 20):
                need = [moe.moe_q4_workspace_bytes(t, n_out, k, x_type) for t in tokens]
                assert need == sorted(need), (x_type, n_out, k)
