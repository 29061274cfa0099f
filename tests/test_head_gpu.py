"""The attribute head: its layers together against the same network in 64 bits, and its example."""
import math
import os
import sys

import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a CUDA device", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from gaussian_splatting_gb300.head import AttributeHead, train_colours  # noqa: E402

pytestmark = pytest.mark.gpu


def _norm(h, g, s, eps):
    m = h.mean(1, keepdim=True)
    return (h - m) * ((h - m).square().mean(1, keepdim=True) + eps) ** -0.5 * g + s


def _reference(head, features, base):
    """The head's forward in 64 bits with autograd, on leaf copies of its parameters."""
    p = {k: v.double().requires_grad_() for k, v in head.p.items()}
    f = features.double().requires_grad_()
    h = f @ p["w_in"].T + p["b_in"]
    for k in range(head.blocks):
        n = _norm(h, p[f"g{k}"], p[f"s{k}"], head.eps)
        z = n @ p[f"w1_{k}"].T + p[f"b1_{k}"]
        h = h + (z * 0.5 * torch.erfc(-z / math.sqrt(2.0))) @ p[f"w2_{k}"].T + p[f"b2_{k}"]
    y = base.double() + _norm(h, p["g_out"], p["s_out"], head.eps) @ p["w_out"].T + p["b_out"]
    return p, f, y


@pytest.mark.parametrize("n,n_in,hidden,n_out", [(1, 8, 16, 3), (37, 24, 64, 3), (2048, 24, 64, 3), (40_000, 40, 96, 59)])
def test_head_against_64_bits(n, n_in, hidden, n_out):
    """Each layer is good to about 1e-6 of its terms; through seven of them 2e-5 of the result's norm covers it."""
    head = AttributeHead(n_in, hidden, n_out, blocks=2, seed=3)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    for v in head.p.values():
        v.add_(torch.randn(v.shape, generator=gen, device="cuda") * 0.05)
    features = torch.randn((n, n_in), generator=gen, device="cuda")
    plane = torch.randn((n, n_out + 1), generator=gen, device="cuda")
    base, last = plane[:, :n_out], plane[:, n_out].clone()
    dy = torch.randn((n, n_out), generator=gen, device="cuda") * 1e-3
    p, f, want = _reference(head, features, base)
    want.backward(dy.double())
    y = head.forward(features, base, out=base)
    assert y.data_ptr() == plane.data_ptr() and torch.equal(plane[:, n_out], last)

    def close(got, ref, what):
        off = (got.double() - ref).norm() / max(ref.norm().item(), 1e-300)
        assert off <= 2e-5, (what, off.item())

    close(y, want.detach(), "y")
    df = head.backward(dy, need_dfeatures=True)
    close(df, f.grad, "dfeatures")
    for k, v in head.g.items():
        close(v, p[k].grad, k)
    again = head.forward(features, plane[:, :n_out].clone(), train=False)
    assert torch.isfinite(again).all()
    with pytest.raises(RuntimeError):
        head.backward(dy)


def test_adam_updates_every_parameter_and_nothing_else():
    head = AttributeHead(5, 16, 3, blocks=1, seed=1)
    before = head.flat.clone()
    for v in head.g.values():
        v.fill_(0.5)
    head.step(1e-2)
    used = torch.zeros_like(head.flat, dtype=torch.bool)
    for v in head.p.values():
        start = (v.data_ptr() - head.flat.data_ptr()) // 4
        used[start:start + v.numel()] = True
        assert v.data_ptr() % 16 == 0
    # the first step of Adam with equal gradients moves every parameter by the learning rate
    assert torch.allclose(before - head.flat, torch.where(used, 1e-2, 0.0), atol=1e-6)
    assert not head.flat_grad.any()


def test_example_learns_the_colours():
    losses = train_colours(steps=60)
    assert all(math.isfinite(v) for v in losses)
    assert losses[-1] < 0.5 * losses[0], losses[::10]


def _trained_step(head, features, base, dy, lr=1e-2):
    head.forward(features, base)
    head.backward(dy)
    head.step(lr)


@pytest.mark.parametrize("when", ["forward", "backward"])
def test_a_wait_that_gives_up_leaves_the_parameters(when):
    """A layer whose operands never arrive (the library's test hook): the head's record is set, the update and all
    after it are skipped on the device until the head has been asked, and then go on."""
    from gaussian_splatting_gb300 import _native as N
    head = AttributeHead(24, 96, 3, blocks=1, seed=2)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    features, base = (torch.randn((20_000, n), generator=gen, device="cuda") for n in (24, 3))
    dy = torch.randn((20_000, 3), generator=gen, device="cuda") * 1e-3
    _trained_step(head, features, base, dy)
    assert head.ok()
    before = [t.clone() for t in (head.flat, head.exp_avg, head.exp_avg_sq)]
    lib = N.load()
    try:
        lib.gs_debug_set_wait_limit(2000)
        if when == "forward":
            lib.gs_debug_drop_publish(3)
        head.forward(features, base)
        if when == "backward":
            lib.gs_debug_drop_publish(3)
        head.backward(dy)
        torch.cuda.synchronize()
    finally:
        lib.gs_debug_set_wait_limit(0)
        lib.gs_debug_drop_publish(0)
    head.step(1e-2)
    assert head.status[0, 1].item() == 2
    _trained_step(head, features, base, dy)  # skipped too: nobody has asked
    for a, b in zip(before, (head.flat, head.exp_avg, head.exp_avg_sq)):
        assert torch.equal(a, b)
    assert not head.ok() and head.ok()
    _trained_step(head, features, base, dy)
    assert head.ok() and torch.isfinite(head.flat).all() and not torch.equal(before[0], head.flat)


def test_a_step_of_a_batch_that_overflowed_leaves_the_parameters():
    head = AttributeHead(5, 16, 3, blocks=1, seed=1)
    before = head.flat.clone()
    for v in head.g.values():
        v.fill_(0.5)
    counts = torch.zeros((4, 2), dtype=torch.int64, device="cuda")
    counts[2, 1] = 1
    head.step(1e-2, counts=counts)
    assert torch.equal(before, head.flat)
    counts.zero_()
    head.step(1e-2, counts=counts)
    assert not torch.equal(before, head.flat) and head.ok()


def test_a_forward_without_training_keeps_no_block():
    """Its memory does not grow with the number of blocks."""
    features, base = torch.randn((100_000, 16), device="cuda"), torch.randn((100_000, 3), device="cuda")
    peaks = []
    for blocks in (2, 8):
        head = AttributeHead(16, 64, 3, blocks=blocks)
        head.forward(features, base, train=False)
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        start = torch.cuda.memory_allocated()
        head.forward(features, base, train=False)
        torch.cuda.synchronize()
        peaks.append(torch.cuda.max_memory_allocated() - start)
    assert peaks[1] <= peaks[0], peaks
    assert peaks[0] <= 4 * 100_000 * 64 * 4  # h, its norm, the activations and the output
