"""A per-Gaussian attribute head: a residual MLP that corrects columns of the Gaussians' records.

``AttributeHead`` maps a row of features per Gaussian (an embedding, a view or time code) to corrections of
some columns of its record, before gs_project reads it, and takes the record's gradient back through itself
after gs_project_bwd:

    h = features W_in^T + b_in
    h = h + gelu(norm(h) W_1^T + b_1) W_2^T + b_2      (once per block)
    record = base + norm(h) W_out^T + b_out

Every layer is one call of gs_linear_fwd / gs_layernorm_fwd forward and one of gs_linear_bwd / gs_layernorm_bwd
backward: the residual connections ride in the linear layers' epilogues forward and in the norms' ``skip``
backward, and the base record is the last layer's residual, read and written in place in the record's own
layout (a plane of [N][4] floats, of which the head may own three).  The parameters are one float32 buffer laid
out as 60-float records, so that gs_sparse_adam updates them.

Every linear layer is given the head's status record, which ``step`` hands to gs_sparse_adam: after a device-side
wait that gave up the update skips itself, as the trainer's does after a view that overflowed, and goes on skipping
until ``ok`` has been asked.

``python -m gaussian_splatting_gb300.head`` trains a head on the smallest scene: the base colours are set grey
and the head learns to restore them from the images.
"""
from __future__ import annotations

import math

import torch

from . import _native as N
from . import dense

_RECORD = 60  # floats that gs_sparse_adam updates per index


class AttributeHead:
    """features [N, ``n_in``] -> corrections [N, ``n_out``], width ``hidden``, ``blocks`` residual blocks."""

    def __init__(self, n_in: int, hidden: int, n_out: int, blocks: int = 2, device="cuda", seed: int = 0, eps: float = 1e-5):
        self.blocks, self.eps = blocks, eps
        shapes = {"w_in": (hidden, n_in), "b_in": (hidden,)}
        for k in range(blocks):
            shapes |= {f"g{k}": (hidden,), f"s{k}": (hidden,), f"w1_{k}": (hidden, hidden), f"b1_{k}": (hidden,),
                       f"w2_{k}": (hidden, hidden), f"b2_{k}": (hidden,)}
        shapes |= {"g_out": (hidden,), "s_out": (hidden,), "w_out": (n_out, hidden), "b_out": (n_out,)}
        # every tensor starts on a 16-byte boundary of the one buffer
        at, total = {}, 0
        for name, shape in shapes.items():
            at[name] = total
            total += (math.prod(shape) + 3) // 4 * 4
        self.records = (total + _RECORD - 1) // _RECORD
        dev = torch.device(device)

        def buffer():
            flat = torch.zeros(self.records * _RECORD, dtype=torch.float32, device=dev)
            return flat, {n: flat[at[n]:at[n] + math.prod(s)].view(s) for n, s in shapes.items()}

        self.flat, self.p = buffer()
        self.flat_grad, self.g = buffer()
        self.exp_avg, self.exp_avg_sq = torch.zeros_like(self.flat), torch.zeros_like(self.flat)
        self.all = torch.arange(self.records, dtype=torch.int32, device=dev)
        self.n_all = torch.full((1,), self.records, dtype=torch.int64, device=dev)
        self.t = 0
        # a record as gs_bin_sort's counts (count, status): the layers set the low word of the second entry
        self.status = torch.zeros((1, 2), dtype=torch.int64, device=dev)
        self._status_word = self.status.view(torch.int32)[0, 2:3]
        gen = torch.Generator(device=dev)
        gen.manual_seed(seed)
        for name, shape in shapes.items():
            if name[0] == "w" and name != "w_out":  # w_out starts at zero: the record starts as the base
                self.p[name].normal_(std=1.0 / math.sqrt(shape[1]), generator=gen)
            elif name[0] == "g":
                self.p[name].fill_(1.0)
        self.kept = None

    def forward(self, features: torch.Tensor, base: torch.Tensor, out: torch.Tensor | None = None, train: bool = True):
        """base + corrections, into ``out`` (which may be a strided view of a record plane, or ``base`` itself).
        ``train`` keeps what ``backward`` reads."""
        p, kept, st = self.p, [], self._status_word
        h, _ = dense.linear_fwd(features, p["w_in"], p["b_in"], status=st)
        for k in range(self.blocks):
            n, mean, rstd = dense.layernorm_fwd(h, p[f"g{k}"], p[f"s{k}"], self.eps, stats=train)
            a, z = dense.linear_fwd(n, p[f"w1_{k}"], p[f"b1_{k}"], act="gelu", keep_z=train, status=st)
            after, _ = dense.linear_fwd(a, p[f"w2_{k}"], p[f"b2_{k}"], residual=h, out=None if train else h, status=st)
            if train:
                kept.append((h, mean, rstd, n, z, a))
            h = after
        n, mean, rstd = dense.layernorm_fwd(h, p["g_out"], p["s_out"], self.eps, stats=train)
        y, _ = dense.linear_fwd(n, p["w_out"], p["b_out"], residual=base, out=out, status=st)
        self.kept = (features, kept, (h, mean, rstd, n)) if train else None
        return y

    def backward(self, dy: torch.Tensor, need_dfeatures: bool = False):
        """The gradient of the last ``forward``, given that of its output: into ``self.g`` (overwritten); returns
        the features' gradient if asked for.  The base's gradient is dy itself."""
        if self.kept is None:
            raise RuntimeError("backward needs a forward with train=True before it")
        p, g, st = self.p, self.g, self._status_word
        features, kept, (h, mean, rstd, n) = self.kept
        self.kept = None
        dn, _, _ = dense.linear_bwd(dy, n, p["w_out"], dw=g["w_out"], dbias=g["b_out"], status=st)
        dh, _, _ = dense.layernorm_bwd(dn, h, p["g_out"], mean, rstd, dgamma=g["g_out"], dbeta=g["s_out"])
        for k in reversed(range(self.blocks)):
            h, mean, rstd, n, z, a = kept[k]
            da, _, _ = dense.linear_bwd(dh, a, p[f"w2_{k}"], dw=g[f"w2_{k}"], dbias=g[f"b2_{k}"], status=st)
            dn, _, _ = dense.linear_bwd(da, n, p[f"w1_{k}"], z, act="gelu", dw=g[f"w1_{k}"], dbias=g[f"b1_{k}"], status=st)
            dh, _, _ = dense.layernorm_bwd(dn, h, p[f"g{k}"], mean, rstd, skip=dh, dx=dn, dgamma=g[f"g{k}"], dbeta=g[f"s{k}"])
        df, _, _ = dense.linear_bwd(dh, features, p["w_in"], dw=g["w_in"], dbias=g["b_in"], need_dx=need_dfeatures, status=st)
        return df

    def step(self, lr: float, betas=(0.9, 0.999), eps: float = 1e-8, counts: torch.Tensor | None = None):
        """Adam on all parameters (gs_sparse_adam with every record listed); the gradients are zero afterwards.
        Leaves everything as it is where a layer's wait gave up, or where one of ``counts``, the status records of the
        trainer's step that the gradient came from (``StepResult.status``), is set."""
        self.t += 1
        records = self.status if counts is None else torch.cat([self.status, counts])
        N.gs_sparse_adam(self.flat, self.flat_grad, self.exp_avg, self.exp_avg_sq, self.records, self.all, self.n_all,
                         self.records, lr, betas[0], betas[1], eps, 1, self.t, records, records.shape[0])

    def ok(self) -> bool:
        """Whether no layer's wait has given up since the last time this was asked (synchronises)."""
        set_ = bool(self.status[0, 1].item())
        self.status.zero_()
        return not set_


def train_colours(steps: int = 60, lr: float = 3e-3, hidden: int = 64, seed: int = 0, report=None):
    """The module's example: the smallest scene with its base colours set grey, a head over a code per Gaussian
    that learns them back through render, loss and both backward passes.  Returns the losses."""
    import numpy as np

    import scenes
    from .trainer import Trainer

    cfg = scenes.CONFIGS[0]
    params = torch.from_numpy(scenes.make_params(0)).cuda()
    cam = scenes.make_cameras(0)[0]
    trainer = Trainer(params.clone(), cfg.width, cfg.height, 1)
    target = trainer.render(cam).clone()[None]
    base = trainer.params[3, :, :3].clone().zero_()  # the colours' degree-0 coefficients
    gen = np.random.Generator(np.random.PCG64(seed))
    features = torch.from_numpy(gen.standard_normal((trainer.n, 24)).astype(np.float32)).cuda()
    head = AttributeHead(24, hidden, 3, seed=seed)
    losses = []
    for k in range(steps):
        head.forward(features, base, out=trainer.params[3, :, :3])
        trainer.grads.zero_()
        result = trainer.step_async([cam], target, adam=False)
        head.backward(trainer.grads[3, :, :3])
        head.step(lr, counts=result.status)
        losses.append(result.loss.clone())
        if report and k % 10 == 0:
            report(f"step {k}: loss {losses[-1].item():.5f}")
    if not head.ok():
        raise RuntimeError("a device-side wait of the head's layers gave up")
    return [float(v.item()) for v in losses]


if __name__ == "__main__":
    import os
    import sys
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    done = train_colours(report=print)
    print(f"loss {done[0]:.5f} -> {done[-1]:.5f} in {len(done)} steps")
