"""The weights of the paged attention: within 2^-17 of their fp32 values, with any number of query rows to a key head.

Tolerance, from the arithmetic (u = 2^-24).  Queries have one channel that is not 0, so that scores are exact products and
  exponent  x = s c - m with c = fl(scale log2 e), m = fl(s0 c): |error| <= 4 u X for |s| log2 e <= X.
  weight    relative E1 = ln 2 * 4 u X + 2^-22 (the power, 2 ulp), and 2^-17 as two bf16 numbers.
  o         numerator and sum both: sum p |v| (2^-17 + 2 E1 + 2 n u) over n keys (2 u a step of either's sum), then one
            rounding of o to bf16, 2^-8 of its value.
Values cancel in one channel for each query row, so that the rounding of o does not hide the weights' error.
"""
import math

import pytest
import torch

import haar_wavelet_patching_b200 as hwp
from test_gpu_paged_attention import RB, U, both, cache, check, dev, reference

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
ROWS = [(1, 4), (5, 3), (5, 4), (8, 4), (11, 3), (5, 8), (16, 4), (20, 8), (64, 2)]  # Nq, Hq of one key head


@pytest.mark.parametrize("Nq,Hq", ROWS)
@pytest.mark.parametrize("D", [64, 40, 128, 72])
@pytest.mark.parametrize("half,page", [(40, 16), (100, 3)])
def test_weights_where_values_cancel(Nq, Hq, D, half, page):
    n, rows = 2 * half + Nq, Nq * Hq
    kp, vp, table = cache([n], page, 1, D)
    a = (0.3 + 1.4 * torch.arange(rows, device="cuda") / rows).to(BF16)     # a row's score of the second half's keys
    q = torch.zeros(1, Nq, Hq, D, dtype=BF16, device="cuda")
    q[..., 0] = a.view(1, Nq, Hq)
    minus = -torch.exp(-a.double()).to(BF16)                                # the value that takes 1 away again, nearly
    k = torch.zeros(n, D, dtype=BF16, device="cuda")
    v = torch.zeros(n, D, dtype=BF16, device="cuda")                        # the last Nq tokens: seen by some, of no value
    k[half: 2 * half, 0] = 1
    v[:half] = 1
    v[half: 2 * half] = minus[torch.arange(D, device="cuda") % rows]
    at = table[0, torch.arange(n, device="cuda") // page].long(), torch.arange(n, device="cuda") % page
    kp[(*at, 0)], vp[(*at, 0)] = k, v
    o = hwp.paged_attention(q, kp, vp, table, dev([n]), scale=1.0)[0].double().reshape(rows, D)

    see = n - Nq + 1 + torch.arange(rows, device="cuda") // Hq
    w = torch.exp(a.double()[:, None] * k[:, 0].double())                   # [rows, n], relative to the first key's
    w = torch.where(torch.arange(n, device="cuda") < see[:, None], w, 0)
    total = w.sum(1, keepdim=True)
    want = w / total @ v.double()
    X = 1.7 * 1.4426950408889634
    E1 = math.log(2) * 4 * U * X + 2.0 ** -22
    tol = w / total @ v.double().abs() * (2.0 ** -17 + 2 * E1 + 2 * n * U) + RB * want.abs()
    check(o, want, tol, "o")
    # One rounding of the weights to bf16 would show.
    once = w.to(BF16).double() / total @ v.double()
    mine = torch.arange(min(rows, D), device="cuda")
    beyond = ((once - want).abs() > 4 * tol)[mine, mine]
    assert beyond.double().mean() > 0.5


@pytest.mark.parametrize("Nq,Hq", [(1, 4), (5, 4), (5, 8)])
@pytest.mark.parametrize("D", [64, 128])
def test_weights_rescaled_with_what_their_rounding_left(Nq, Hq, D):
    """Tens of thousands of keys, then one far above them: all streams alike, one to an SM, so that one CTA has it all."""
    n, page, B = 40000, 16, 148
    kp, vp, table = cache([n], page, 1, D)
    a = (0.5 + 0.06 * torch.arange(Nq * Hq, device="cuda") / (Nq * Hq)).to(BF16)
    q = torch.zeros(1, Nq, Hq, D, dtype=BF16, device="cuda")
    q[..., 0] = a.view(1, Nq, Hq)
    kp.zero_()
    kp[..., 0] = 1
    vp[:] = 1
    kp[int(table[0, 0]), 0] = 0                                             # what weights are relative to at first
    far = n - Nq - 1
    kp[int(table[0, far // page]), far % page, 0, 0] = 26
    vp[int(table[0, far // page]), far % page, 0, ::2] = 0.5
    both(q, kp, vp, table, dev([n]), None, 1.0)
    o = hwp.paged_attention(q.expand(B, -1, -1, -1), kp, vp, table.expand(B, -1).contiguous(), dev([n] * B), scale=1.0)
    assert torch.equal(o, o[:1].expand_as(o))
    want = reference(q, kp, vp, table, [n], None, 1.0)
    check(o[:1], want[0], want[1], "o")
