"""The router, the expert layer and the adapters take CUDA tensors: any one of
the others' arguments in host memory is refused before the library is called.

On a machine without a GPU only the all-host calls can be made; the rest runs on
one, still without a launch."""

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def fl():
    import precision_linear_algebra_gb300 as fl
    from precision_linear_algebra_gb300 import build
    build.build()
    fl.load()
    return fl


def arguments(name):
    i32 = torch.int32
    if name == "moe_route":
        return dict(logits=torch.zeros(200, 8), ids=torch.zeros(200, 2, dtype=i32),
                    weights=torch.zeros(200, 2), m_offsets=torch.zeros(9, dtype=i32),
                    order=torch.zeros(400, dtype=i32),
                    workspace=torch.zeros(1 << 16, dtype=torch.uint8))
    if name == "moe_layer":
        u8 = torch.uint8
        return dict(x=torch.zeros(2, 32), ids=torch.zeros(2, 2, dtype=i32),
                    weights=torch.zeros(2, 2), w13=torch.zeros(4, 32, 32, dtype=u8),
                    scale13=torch.zeros(4), w2=torch.zeros(4, 32, 16, dtype=u8),
                    scale2=torch.zeros(4), y=torch.zeros(2, 32, dtype=torch.bfloat16),
                    workspace=torch.zeros(1 << 25, dtype=u8))
    bf = torch.bfloat16
    c = dict(x=torch.zeros(6, 16), A=torch.zeros(2, 4, 16, dtype=bf),
             B=torch.zeros(2, 4, 24, dtype=bf), alpha=torch.zeros(2),
             m_offsets=torch.tensor([0, 2, 6], dtype=i32),
             adapter_ids=torch.tensor([0, 1], dtype=i32))
    if name == "lora_apply":
        return dict(c, base=torch.zeros(6, 24, dtype=bf), out=torch.zeros(6, 24, dtype=bf),
                    v=torch.zeros(6, 4))
    return dict(c, dy=torch.zeros(6, 24), v=torch.zeros(6, 4),
                dx_base=torch.zeros(6, 16, dtype=bf), dx=torch.zeros(6, 16, dtype=bf),
                dA=torch.zeros(2, 4, 16), dB=torch.zeros(2, 4, 24),
                workspace=torch.zeros(1 << 12, dtype=torch.uint8))


def call(fl, name, args):
    args = dict(args)
    if name == "moe_route":
        return fl.moe_route(args.pop("logits"), 2, **args)
    return getattr(fl, name)(**args)


NAMES = ("moe_route", "moe_layer", "lora_apply", "lora_backward")


@pytest.mark.parametrize("name", NAMES)
def test_host_tensors(fl, name):
    with pytest.raises(AssertionError):
        call(fl, name, arguments(name))


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_one_host_tensor(fl, name):
    host = arguments(name)
    device = {k: t.cuda() for k, t in host.items()}
    call(fl, name, device)
    torch.cuda.synchronize()
    assert fl.device_status() == 0
    for k in host:
        with pytest.raises(AssertionError):
            call(fl, name, dict(device, **{k: host[k]}))
