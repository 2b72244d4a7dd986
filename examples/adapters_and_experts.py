"""One decoding step and one adapter training step through the library.

Decoding: the tokens of several requests go through a shared FP8 projection,
each request's low-rank adapter is added beside it, and the sum goes through a
mixture-of-experts layer.  Training: the gradient at the projection's output
goes back through the adapters and the shared projection.

    python examples/adapters_and_experts.py            # needs a GB300

Prints what each step computed against the same step in 64 bits, and its time.
"""

import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def make_model(fl, width, inner, experts, adapters, rank, seed=0):
    """Random weights of a projection [width][width], experts (width, inner)
    and adapters, quantised as a user would once after loading them."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, sigma):
        return torch.randn(*shape, generator=g, device="cuda") * sigma

    m = {"width": width, "experts": experts}
    w = normal(width, width, sigma=0.02)
    m["w"] = w
    m["qw"], _, m["sw"] = fl.quantize_pertensor(w)
    m["qwt"], _, m["swt"] = fl.quantize_pertensor(w.t().contiguous())
    m["router"] = normal(experts, width, sigma=width ** -0.5)
    for name, rows, cols in (("w13", 2 * inner, width), ("w2", width, inner)):
        stack = normal(experts * rows, cols, sigma=0.02)
        offs = torch.arange(experts + 1, dtype=torch.int32, device="cuda") * rows
        codes, _, scales = fl.quantize_pertensor_grouped(stack, offs)
        m[name], m["s" + name] = codes.view(experts, rows, cols), scales
    m["A"] = normal(adapters, rank, width, sigma=width ** -0.5).to(torch.bfloat16)
    m["B"] = normal(adapters, rank, width, sigma=0.02).to(torch.bfloat16)
    m["alpha"] = torch.full((adapters,), 2.0, device="cuda")
    return m


def decode_step(fl, m, x, m_offsets, adapter_ids, top_k=2):
    """x fp32 [T][width] -> (hidden bf16, experts' output bf16, v, ids, weights)."""
    qx, _, sx = fl.quantize_pertensor(x)
    base = fl.gemm(qx, m["qw"], sx, m["sw"])
    hidden, v = fl.lora_apply(base, x, m["A"], m["B"], m["alpha"], m_offsets, adapter_ids,
                              out=base)
    ids, weights, _, _ = fl.moe_route(hidden.float() @ m["router"].t(), top_k, sort=False)
    out = fl.moe_layer(hidden, ids, weights, m["w13"], m["sw13"], m["w2"], m["sw2"])
    return hidden, out, v, ids, weights


def train_step(fl, m, x, v, dy, m_offsets, adapter_ids, rate=1e-3):
    """Gradients of the adapters and of x for dy bf16 [T][width], and one step
    of plain gradient descent on the adapters.  The shared projection's part of
    dx takes E5M2 gradients, whose range is wider."""
    import torch
    qd, _, sd = fl.quantize_pertensor(dy.float(), fmt="e5m2")
    dx_base = fl.gemm(qd, m["qwt"], sd, m["swt"], a_fmt="e5m2")
    dx, dA, dB = fl.lora_backward(dy, x, v, m["A"], m["B"], m["alpha"], m_offsets,
                                  adapter_ids, dx_base, dx=dx_base)
    m["A"] = (m["A"].float() - rate * dA).to(torch.bfloat16)
    m["B"] = (m["B"].float() - rate * dB).to(torch.bfloat16)
    return dx, dA, dB


def check(fl, m, x, m_offsets, adapter_ids, step):
    """Relative distances of the decoding step's outputs from 64 bits, each
    from the inputs that its own operator had."""
    import torch
    hidden, out, v, ids, weights = step
    offs, who = m_offsets.tolist(), adapter_ids.tolist()
    want = x.double() @ m["w"].double().t()
    for lo, hi, i in zip(offs, offs[1:], who):
        if i >= 0:
            want[lo:hi] += m["alpha"][i].double() * (
                x[lo:hi].double() @ m["A"][i].double().t() @ m["B"][i].double())
    y = torch.zeros_like(want)
    h = hidden.double()
    inner = m["w2"].shape[2]
    for t in range(x.shape[0]):
        for j, e in enumerate(ids[t].tolist()):
            w13 = m["w13"][e].view(torch.float8_e4m3fn).double() * m["sw13"][e].double()
            w2 = m["w2"][e].view(torch.float8_e4m3fn).double() * m["sw2"][e].double()
            gu = w13 @ h[t]
            y[t] += weights[t, j].double() * (
                w2 @ (torch.nn.functional.silu(gu[:inner]) * gu[inner:]))

    def rel(a, b):
        return ((a.double() - b).norm() / b.norm()).item()

    return rel(hidden, want), rel(out, y)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--requests", type=int, default=16)
    ap.add_argument("--width", type=int, default=2048)
    ap.add_argument("--inner", type=int, default=1408)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--adapters", type=int, default=4)
    ap.add_argument("--rank", type=int, default=16)
    ap.add_argument("--train-tokens", type=int, default=1024)
    a = ap.parse_args(argv)
    import torch
    import precision_linear_algebra_gb300 as fl
    from precision_linear_algebra_gb300 import build
    build.build()
    m = make_model(fl, a.width, a.inner, a.experts, a.adapters, a.rank)

    # one token for each request; the last request has no adapter
    x = torch.randn(a.requests, a.width, device="cuda")
    offs = torch.arange(a.requests + 1, dtype=torch.int32, device="cuda")
    who = torch.arange(a.requests, dtype=torch.int32, device="cuda") % a.adapters
    who[-1] = -1
    step = decode_step(fl, m, x, offs, who)
    err = check(fl, m, x, offs, who, step)

    # a training batch: one long segment for each adapter
    T = a.train_tokens
    tx = torch.randn(T, a.width, device="cuda").to(torch.bfloat16)
    toffs = torch.tensor([T * i // a.adapters for i in range(a.adapters + 1)],
                         dtype=torch.int32, device="cuda")
    twho = torch.arange(a.adapters, dtype=torch.int32, device="cuda")
    qx, _, sx = fl.quantize_pertensor(tx.float())
    base = fl.gemm(qx, m["qw"], sx, m["sw"])
    _, v = fl.lora_apply(base, tx, m["A"], m["B"], m["alpha"], toffs, twho)
    dy = (torch.randn(T, a.width, device="cuda") * 0.01).to(torch.bfloat16)

    def timed(f, n=20):
        f()
        start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        for _ in range(n):
            f()
        stop.record()
        stop.synchronize()
        return start.elapsed_time(stop) / n * 1e3

    t_dec = timed(lambda: decode_step(fl, m, x, offs, who))
    t_train = timed(lambda: train_step(fl, m, tx, v, dy, toffs, twho))
    status = fl.device_status()
    print("decode %d tokens: projection + adapters off by %.2e, experts off by %.2e; "
          "%.0f us a step" % (a.requests, err[0], err[1], t_dec))
    print("train %d tokens, %d adapters of rank %d: %.0f us a step"
          % (T, a.adapters, a.rank, t_train))
    return err, status


if __name__ == "__main__":
    main()
