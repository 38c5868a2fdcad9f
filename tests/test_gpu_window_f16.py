"""Sliding-window attention on fp16 tensors where weights are far from
1: fp16 has a narrow range, normal from 2^-14 to 2^16, and what the kernels round to
it for a product is brought into it by powers of two.

Tolerances as in test_gpu_window.py, but for the relative error of a weight, which
is taken for the head size: err = (d 2^-23 + 2^-21) (1 + L).  What falls below
fp16's normal range is rounded to steps of 2^-24, so by 2^-25 of
  the weights of O, which are 2^7 at a row's maximum (as it was when it last moved): 2^-32.
Nothing else is added for the types' range but half a step of the fp16 results, 2^-25."""
import math

import pytest
import torch

import test_gpu_window as base
from test_gpu_window import F16, _forward, _logits, _near, _seen

pytestmark = pytest.mark.gpu
pkg = base.pkg
U = torch.finfo(F16).eps / 2
STEP = 2.0 ** -25


def _err(q, k, seen, scale):
    """Relative error of a weight, by rows."""
    rep = k.repeat_interleave(q.shape[1] // k.shape[1], 1)
    big = (abs(scale) * (q.abs() @ rep.abs().mT)).masked_fill(~seen, 0).amax(-1, keepdim=True)
    return (q.shape[-1] * 2.0 ** -23 + 2.0 ** -21) * (1 + big)


def _check_forward(pkg, q, k, v, window, sinks, scale):
    o, lse = pkg.attn_fwd_window(q, k, v, window, sinks, scale=scale)
    assert pkg.sync_status() == 0
    q, k, v = q.double(), k.double(), v.double()
    ro, rl = _forward(q, k, v, window, sinks, scale)
    seen = _seen(q.shape[2], k.shape[2], window, sinks, q.device)
    err, n = _err(q, k, seen, scale), seen.sum(-1).max().item() * 2.0 ** -24
    p = torch.softmax(_logits(q, k, scale).masked_fill(~seen, -math.inf), -1)
    vv = v.abs().repeat_interleave(q.shape[1] // k.shape[1], 1)
    _near("o", o, ro, U * ro.abs() + ((2 * U + 2 * err + n) * p + 2.0 ** -32 * seen) @ vv + STEP)
    _near("lse", lse, rl, err[..., 0] + 2.0 ** -22 * rl.abs())
    return o, lse


def _randn(seed, *shapes):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(s, generator=g) for s in shapes]


def _half(*x):
    return [t.to(F16).cuda() for t in x]


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("gap", [8.0, 13.0, 15.25, 17.5, 21.0])
@pytest.mark.parametrize("nq,nk,window,sinks", [(700, 700, 200, 1), (4, 3000, 2500, 1), (300, 300, 300, 0)])
def test_a_sink_that_holds_the_weight(pkg, d, gap, nq, nk, window, sinks):
    """A first key with nearly all of the weight and a value of zero, as models make of sinks: O is what the other keys' small weights make of it."""
    q, k, v = _randn(nq + d, (1, 4, nq, d), (1, 2, nk, d), (1, 2, nk, d))
    q, k, v = q * 0.05, k * 0.5, v * 4000
    q[..., 0], k[..., 0], k[:, :, 0] = 1.0, 0.0, 0.0
    k[:, :, 0, 0], v[:, :, 0] = gap, 0.0
    _check_forward(pkg, *_half(q, k, v.clamp(-6e4, 6e4)), window, sinks, 1.0)
