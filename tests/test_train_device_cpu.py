"""The training calls refuse tensors and streams of a device that is not the
current one, before anything is queued.  No GPU: tensors that say they are on
one, and a library that only counts its calls."""
import pytest
import torch

import expert_routing_ffn_gb300 as moe
from expert_routing_ffn_gb300 import train


class On(torch.Tensor):
    """A host tensor that answers for a tensor of device `dev`."""
    __torch_function__ = torch._C._disabled_torch_function_impl
    dev = 0
    is_cuda = True

    def get_device(self):
        return self.dev


def on(dev, *shape, dtype=torch.bfloat16):
    t = torch.zeros(shape, dtype=dtype).as_subclass(On)
    t.dev = dev
    return t


T, d, N, k, I = 4, 40, 8, 2, 24
M, F32, I32 = T * k, torch.float32, torch.int32


def calls(D, dev):
    """Every call: function, positional arguments by name; dev(name) is the device of that tensor."""
    def t(name, *shape, dtype=torch.bfloat16):
        return name, on(dev(name), *shape, dtype=dtype)

    ws = t("ws", 64, dtype=torch.uint8)
    off, inv = t("expert_offsets", N + 1, dtype=I32), t("inv_perm", M, dtype=I32)
    w = lambda n, dt=torch.bfloat16: t(n, N, I, d, dtype=dt)  # noqa: E731
    return {
        "moe_dispatch_rows": [t("x", T, d), t("expert_idx", T, k, dtype=I32), 0, t("x_perm", M, d), off,
                              t("perm", M, dtype=I32), inv, ws],
        "moe_dispatch_rows_grad": [t("dx_perm", M, d), inv, t("add", T, d), t("dx", T, d)],
        "moe_combine_rows": [t("y_perm", M, d), t("gate", T, k, dtype=F32), inv, t("add", T, d), t("out", T, d)],
        "moe_combine_rows_grad": [t("dout", T, d), t("y_perm", M, d), t("gate", T, k, dtype=F32), inv, t("dy_perm", M, d),
                                  t("dgate", T, k, dtype=F32)],
        "moe_gate_grad": [t("router_prob", T, N, dtype=F32), t("topk_idx", T, k, dtype=I32), t("dgate", T, k, dtype=F32),
                          0.1, t("dlogits", T, N, dtype=F32), t("balance_loss", 1, dtype=F32), ws],
        "moe_experts_up": [t("x_perm", M, d), off, w("w_gate"), w("w_up"), t("g", M, I), t("u", M, I), t("h", M, I), ws],
        "moe_experts_up_grad": [t("dg", M, I), t("du", M, I), t("x_perm", M, d), off, w("w_gate"), w("w_up"),
                                t("dx_perm", M, d), w("dw_gate", F32), w("dw_up", F32), True, ws],
        "moe_experts_down": [t("h", M, I), off, w("w_down"), t("y_perm", M, d), ws],
        "moe_experts_down_grad": [t("dy_perm", M, d), t("h", M, I), t("g", M, I), t("u", M, I), off, w("w_down"),
                                  t("dg", M, I), t("du", M, I), w("dw_down"), False, ws],
    }


NAMES = [(c, a[0]) for c, args in calls(None, lambda n: 0).items() for a in args if isinstance(a, tuple)]


@pytest.fixture
def queued(monkeypatch):
    """The C calls made, on a machine whose current device is 0."""
    made = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: made.append(name) or moe.MOE_OK

    monkeypatch.setattr(train, "lib", Lib)
    monkeypatch.setattr(train, "_here", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0)
    return made


def run(call, dev):
    D = moe.make_dims(T, d, N, k, I)
    getattr(moe, call)(D, *(a[1] if isinstance(a, tuple) else a for a in calls(D, dev)[call]))


@pytest.mark.parametrize("call", sorted({c for c, _ in NAMES}))
def test_tensors_of_the_current_device_are_taken(call, queued):
    run(call, lambda n: 0)
    assert queued == [call]


@pytest.mark.parametrize("call,name", NAMES)
def test_a_tensor_of_another_device_is_refused(call, name, queued):
    with pytest.raises(ValueError, match=f"{name} is on cuda:1"):
        run(call, lambda n: 1 if n == name else 0)
    assert not queued


@pytest.mark.parametrize("call", sorted({c for c, _ in NAMES}))
def test_a_call_whose_tensors_are_all_elsewhere_is_refused(call, queued):
    with pytest.raises(ValueError, match="current device"):
        run(call, lambda n: 1)
    assert not queued


def test_a_stream_of_another_device_is_refused(queued, monkeypatch):
    class Stream:
        def __init__(self, device_index):
            self.device_index, self.cuda_stream = device_index, 0x1000

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    D = moe.make_dims(T, d, N, k, I)
    args = [a[1] for a in calls(D, lambda n: 0)["moe_combine_rows"]]
    moe.moe_combine_rows(D, *args, stream=Stream(0))
    with pytest.raises(ValueError, match="the stream is of cuda:1"):
        moe.moe_combine_rows(D, *args, stream=Stream(1))
    assert queued == ["moe_combine_rows"]
