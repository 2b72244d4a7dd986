"""The calls that check their tensors refuse any that is on another device than the
current one, whose memory a launch there cannot be trusted to reach.  Nothing is launched:
the tensors say of themselves which device they are on."""

import pytest

torch = pytest.importorskip("torch")


class On:
    """A tensor that says that it is on a device."""

    def __init__(self, t, device=0):
        self._t, self._device = t, device

    def get_device(self):
        return self._device

    is_cuda = True

    def __getattr__(self, name):
        return getattr(self._t, name)


@pytest.fixture
def fl(monkeypatch):
    import precision_linear_algebra_gb300 as fl
    from precision_linear_algebra_gb300 import build
    build.build()
    fl.load()
    calls = []
    monkeypatch.setattr(fl, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(fl, "_stream", lambda: None)
    monkeypatch.setattr(fl, "_call", lambda name, *args: calls.append(name))
    fl.calls = calls
    yield fl
    del fl.calls


def _arguments(name):
    i32, bf, u8 = torch.int32, torch.bfloat16, torch.uint8
    if name == "moe_route":
        return dict(logits=torch.zeros(200, 8), ids=torch.zeros(200, 2, dtype=i32),
                    weights=torch.zeros(200, 2), m_offsets=torch.zeros(9, dtype=i32),
                    order=torch.zeros(400, dtype=i32), workspace=torch.zeros(1 << 16, dtype=u8))
    if name == "moe_layer":
        return dict(x=torch.zeros(2, 32), ids=torch.zeros(2, 2, dtype=i32),
                    weights=torch.zeros(2, 2), w13=torch.zeros(4, 32, 32, dtype=u8),
                    scale13=torch.zeros(4), w2=torch.zeros(4, 32, 16, dtype=u8),
                    scale2=torch.zeros(4), y=torch.zeros(2, 32, dtype=bf),
                    workspace=torch.zeros(1 << 25, dtype=u8))
    if name.startswith("lora"):
        c = dict(x=torch.zeros(6, 16), A=torch.zeros(2, 4, 16, dtype=bf),
                 B=torch.zeros(2, 4, 24, dtype=bf), alpha=torch.zeros(2),
                 m_offsets=torch.zeros(3, dtype=i32), adapter_ids=torch.zeros(2, dtype=i32),
                 v=torch.zeros(6, 4))
        if name == "lora_apply":
            return dict(c, base=torch.zeros(6, 24, dtype=bf), out=torch.zeros(6, 24, dtype=bf))
        return dict(c, dy=torch.zeros(6, 24), dx_base=torch.zeros(6, 16, dtype=bf),
                    dx=torch.zeros(6, 16, dtype=bf), dA=torch.zeros(2, 4, 16),
                    dB=torch.zeros(2, 4, 24), workspace=torch.zeros(1 << 12, dtype=u8))
    c = dict(m_offsets=torch.zeros(3, dtype=i32), kv_lens=torch.zeros(2, dtype=i32),
             page_table=torch.zeros(2, 4, dtype=i32))
    if name == "kv_attention":
        return dict(c, q=torch.zeros(5, 4, 64), out=torch.zeros(5, 4, 64, dtype=bf),
                    lse=torch.zeros(5, 4), prefix_table=torch.zeros(2, dtype=i32),
                    prefix_len=torch.zeros(1, dtype=i32),
                    workspace=torch.zeros(1 << 25, dtype=u8))
    return dict(c, k=torch.zeros(5, 2, 64), v=torch.zeros(5, 2, 64))


def _cache(fl, devices=(0, 0, 0, 0)):
    codes = [On(torch.zeros(6, 2, 16, 64, dtype=torch.uint8), d) for d in devices[:2]]
    scales = [On(torch.ones(6, 2, 16), d) for d in devices[2:]]
    return fl.KVCache(*codes, *scales)


def _run(fl, name, args, cache=None):
    args = dict(args)
    if name.startswith("kv"):
        args["cache"] = cache or _cache(fl)
    if name == "kv_read":
        args["rows"] = 5
    if name == "moe_route":
        args["top_k"] = 2
    getattr(fl, name)(**args)


NAMES = ("moe_route", "moe_layer", "lora_apply", "lora_backward", "kv_append", "kv_read",
         "kv_attention")


@pytest.mark.parametrize("name", NAMES)
def test_a_tensor_of_another_device_is_refused(fl, name):
    args = {k: On(t) for k, t in _arguments(name).items()}
    _run(fl, name, args)
    assert len(fl.calls) == 1
    for k, t in _arguments(name).items():
        with pytest.raises(AssertionError):
            _run(fl, name, dict(args, **{k: On(t, 1)}))
    with pytest.raises(AssertionError):  # all of them elsewhere, and the launch here
        _run(fl, name, {k: On(t, 1) for k, t in _arguments(name).items()},
             _cache(fl, (1, 1, 1, 1)) if name.startswith("kv") else None)
    if name.startswith("kv"):
        with pytest.raises(AssertionError):
            _run(fl, name, args, _cache(fl, (1, 1, 1, 1)))
    assert len(fl.calls) == 1


@pytest.mark.parametrize("at", range(4))
def test_a_cache_is_on_one_device(fl, at):
    devices = [0, 0, 0, 0]
    devices[at] = 1
    with pytest.raises(AssertionError):
        _cache(fl, devices)
