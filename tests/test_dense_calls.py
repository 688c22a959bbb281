"""What the binding of the dense half lets through to the library: a stub takes the calls (CPU)."""
import pytest
import torch

from ragged_grouped_gemm_device_amd import moe as M

BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


class Stub:
    """Records the entry points that a call reaches, and answers that all is well."""

    def __init__(self):
        self.reached = []

    def __getattr__(self, name):
        return lambda *a: self.reached.append(name) or 0


@pytest.fixture
def lib(monkeypatch):
    stub = Stub()
    monkeypatch.setattr(M, "_lib", lambda: stub)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    return stub


def _z(*shape, t=BF, dev="cpu"):
    return torch.zeros(*shape, dtype=t, device=dev)


def _calls(dev):
    z = lambda *s, t=BF: _z(*s, t=t, dev=dev)  # noqa: E731
    ws = z(4096, t=U8)
    losses = (z(3, t=F32), z(1, 8, t=I32), z(1, 8, t=F32), z(3, t=I32))
    return {
        "moe_linear_fwd": lambda: M.moe_linear_fwd(z(4, 64), z(64, 128), z(4, 128), workspace=ws),
        "moe_act_bwd": lambda: M.moe_act_bwd(z(4, 128), z(4, 128), M.MOE_ACT_SILU, z=z(4, 128)),
        "moe_linear_dgrad": lambda: M.moe_linear_dgrad(z(4, 128), z(64, 128), z(4, 64), workspace=ws),
        "moe_linear_wgrad": lambda: M.moe_linear_wgrad(z(4, 64), z(4, 128), z(64, 128, t=F32), workspace=ws),
        "moe_dequant_mxfp8": lambda: M.moe_dequant_mxfp8(z(4, 64, t=U8), z(4, 2, t=U8), z(4, 64)),
        "moe_balance_loss": lambda: M.moe_balance_loss(z(6, 8, t=F32), z(6, 2, t=I32), *losses, ws, 1.0, 1.0),
        "moe_balance_loss_bwd": lambda: M.moe_balance_loss_bwd(z(6, 8, t=F32), losses[1], losses[3], z(6, 8, t=F32), 2,
                                                               1.0, 1.0),
    }


@pytest.mark.parametrize("dev", ["cpu", "meta"])
@pytest.mark.parametrize("name", list(_calls("meta")))
def test_operands_that_are_all_off_the_gpu_are_refused(lib, name, dev):
    """The library gets addresses: a host one must not reach a kernel, even where every operand agrees."""
    with pytest.raises(ValueError, match="GPU"):
        _calls(dev)[name]()
    assert lib.reached == []


def test_router_losses_refuse_another_k(lib):
    """The forward would count topk_idx's k experts a token, and the backward divide by the Router's k."""
    router = M.Router(6, 64, 8, 1, device="cpu")
    with pytest.raises(ValueError, match="k = 1"):
        router.losses(_z(6, 2, t=I32))
    assert "moe_balance_loss" not in lib.reached


@pytest.mark.parametrize("which", ["router", "shared", "both"])
def test_backward_without_the_input_that_it_needs_starts_nothing(lib, which):
    """The weight gradients of the router and the shared expert read x: refused before any launch, not
    after the routed experts' backward and a half-done dx."""
    buf = M.Buffers(8, 2, 8, 64, 64, device="cpu")
    kw = {}
    if which != "shared":
        kw["router"] = (M.Router(8, 64, 8, 2, device="cpu"), _z(64, 8))
    if which != "router":
        kw["shared"] = (M.SharedExpert(8, 64, 32, device="cpu"), _z(64, 64), _z(32, 64))
    lib.reached.clear()
    with pytest.raises(ValueError, match="x_tokens"):
        M.backward(buf, _z(8, 64), _z(8, 64, 128), _z(8, 64, 64), **kw)
    assert lib.reached == []


def test_backward_of_a_shared_expert_with_its_own_copy_of_x_needs_none(lib):
    buf = M.Buffers(8, 2, 8, 64, 64, device="cpu")
    shared = M.SharedExpert(8, 64, 32, x8=True, device="cpu")
    with pytest.raises(ValueError, match="GPU"):        # as far as the first product, on host tensors here
        M.backward(buf, _z(8, 64), _z(8, 64, 128), _z(8, 64, 64), shared=(shared, _z(64, 64), _z(32, 64)))


BIG = 1 << 32


@pytest.mark.parametrize("name, call", [
    ("moe_linear_fwd", lambda z: M.moe_linear_fwd(z(1, BIG + 64), z(BIG + 64, 8), z(1, 8))),
    ("moe_linear_fwd", lambda z: M.moe_linear_fwd(z(1, 64), z(64, BIG + 8), z(1, BIG + 8))),
    ("moe_act_bwd", lambda z: M.moe_act_bwd(z(1, BIG + 8), z(1, BIG + 8))),
    ("moe_linear_dgrad", lambda z: M.moe_linear_dgrad(z(1, BIG + 8), z(8, BIG + 8), z(1, 8))),
    ("moe_linear_dgrad", lambda z: M.moe_linear_dgrad(z(1, 8), z(BIG + 8, 8), z(1, BIG + 8))),
    ("moe_linear_wgrad", lambda z: M.moe_linear_wgrad(z(1, BIG + 8), z(1, 8), z(BIG + 8, 8))),
    ("moe_linear_wgrad", lambda z: M.moe_linear_wgrad(z(1, 8), z(1, BIG + 8), z(8, BIG + 8))),
    ("moe_dequant_mxfp8", lambda z: M.moe_dequant_mxfp8(z(1, BIG + 32, t=U8), z(1, BIG // 32 + 1, t=U8), z(1, BIG + 32))),
    ("moe_balance_loss", lambda z: M.moe_balance_loss(z(4, BIG + 8, t=F32), z(4, 2, t=I32), z(3, t=F32), z(1, BIG + 8, t=I32),
                                                      z(1, BIG + 8, t=F32), z(3, t=I32), z(64, t=U8), 1.0, 1.0)),
    ("moe_balance_loss", lambda z: M.moe_balance_loss(z(4, 8, t=F32), z(4, BIG + 2, t=I32), z(3, t=F32), z(1, 8, t=I32),
                                                      z(1, 8, t=F32), z(3, t=I32), z(64, t=U8), 1.0, 1.0)),
    ("moe_balance_loss", lambda z: M.moe_balance_loss(z(4, 8, t=F32), z(4, 2, t=I32), z(3, t=F32), z(BIG + 1, 8, t=I32),
                                                      z(BIG + 1, 8, t=F32), z(BIG + 3, t=I32), z(64, t=U8), 1.0, 1.0)),
    ("moe_balance_loss_bwd", lambda z: M.moe_balance_loss_bwd(z(4, 8, t=F32), z(1, 8, t=I32), z(3, t=I32), z(4, 8, t=F32), BIG + 2,
                                                              1.0, 1.0)),
])
def test_sizes_past_32_bits_are_refused(lib, monkeypatch, name, call):
    """They would wrap to another, valid size, as the row counts would (meta tensors: nothing is allocated;
    taken for the first GPU's, as tensors of this size would be there)."""
    monkeypatch.setattr(M, "_device", lambda t: 0)
    monkeypatch.setattr(M, "_operand", lambda *a: None)
    monkeypatch.setattr(M, "_space", lambda *a: (None, 0))
    with pytest.raises(ValueError, match="32 bits"):
        call(lambda *s, t=BF: torch.empty(*s, dtype=t, device="meta"))
    assert lib.reached == []


def test_a_trained_weight_leaves_no_history_in_the_routers_copy(lib):
    """12 experts: the padded copy must not join the weight's autograd graph, which would grow by a step a call."""
    router = M.Router(6, 64, 12, 2, device="cpu")
    wg = torch.nn.Parameter(torch.ones(64, 12, dtype=BF))
    with pytest.raises(ValueError, match="GPU"):        # after the copy, on host tensors here
        router.project(_z(6, 64), wg)
    wide = router.wide[0]
    assert (wide[:, :12] == 1).all() and (wide[:, 12:] == 0).all()
    assert not wide.requires_grad and wide.grad_fn is None
