"""Attention over the 8-bit K/V cache where a row's scores are far apart: one key
(a sink) stands high above the others and its value is zero, so that the output
is made of the small probabilities alone.

The bounds are those of test_gpu_fp8_kv.py, relative to the softmax's mean of
|v|, which here is the small probabilities' own: a kernel that rounds them
relative to the sink's fails, however small they are.
"""
import numpy as np
import pytest
import torch

from . import test_gpu_fp8_kv as T

msa = T.msa
pytestmark = pytest.mark.gpu

ROWS = {
    "one block": dict(ctx=[100, 128, 77], nq=[1, 1, 2], kv=2, topk=1),
    "16 blocks, one row": dict(ctx=[2100], nq=[1], kv=4, topk=16),
    "64 blocks, one row": dict(ctx=[8200], nq=[1], kv=1, topk=64),
    "16 blocks, a batch": dict(ctx=[2100 + 31 * i for i in range(30)], nq=[1] * 30, kv=1, topk=16),
    "64 blocks, verify rows": dict(ctx=[8200, 9000], nq=[4, 4], kv=1, topk=64),
}


def sink_case(seed, gap, equal, which, **shape):
    """Key 0 of every sequence scores `gap` nats, the others N(0, 0.9) or all 0; block 0 is in every selection.
    Dims 0 .. 15 carry the sink's score alone: 16 * 448 * 2^-6 / sqrt(128) = 9.9 nats for queries of 1 there."""
    c = T.Case(seed, which=which, **shape)
    c.k[..., :16] = 0
    if equal:
        c.k[:] = 0
        c.v[:] = 0x79                                  # 288
    c.ks[:] = 2.0 ** -6
    for s in range(len(c.ctx)):
        page = c.table[s, 0]
        c.k[page, :, 0, :16], c.k[page, :, 0, 16:] = 0x7E, 0
        c.v[page, :, 0] = 0
    c.q[..., :16] = gap / (16 * 448 * 2.0 ** -6 / 128 ** 0.5)
    for t in range(c.rows):
        for g in range(c.kv):
            own = c.sel[t, g][c.sel[t, g] > 0]
            if len(own) < c.topk:
                c.sel[t, g] = -1
                c.sel[t, g, 0], c.sel[t, g, 1:len(own) + 1] = 0, own
            elif c.topk > 1:
                c.sel[t, g, 0] = 0
    return c


@pytest.mark.parametrize("which", T.FORMS)
@pytest.mark.parametrize("equal", [False, True], ids=["spread", "equal"])
@pytest.mark.parametrize("gap", [12, 15, 19])
@pytest.mark.parametrize("shape", ROWS)
def test_small_probabilities_under_a_sink(cuda_ok, shape, gap, equal, which):
    c = sink_case(61, gap, equal, which, **ROWS[shape])
    out, lse = c.run()
    assert msa.device_status() == msa.MSA_OK
    c.check(out, lse, range(c.main))


@pytest.mark.parametrize("which", T.FORMS)
def test_a_row_is_as_exact_in_a_batch_as_alone(cuda_ok, which):
    """The same row with its sink, alone and as the last one of a batch (other borders between the CTAs): both within the
    bound of the definition."""
    shape = dict(ctx=[2100 + 31 * i for i in range(40)], nq=[1] * 40, kv=2, topk=16)
    c = sink_case(62, 16, False, which, **shape)
    out, lse = c.run()
    assert msa.device_status() == msa.MSA_OK
    c.check(out, lse, [c.main - 1])
    one = sink_case(62, 16, False, which, ctx=[shape["ctx"][-1]], nq=[1], kv=2, topk=16)
    out, lse = one.run()
    assert msa.device_status() == msa.MSA_OK
    one.check(out, lse, [0])


@pytest.mark.parametrize("which", T.FORMS)
def test_queries_with_one_large_element(cuda_ok, which):
    """An element 2^10 times the others, which meets keys that are 0 there: the scores are the others' own, and their bits
    count.  Those above 2^-14 of the largest (2^-4 here) are held exactly; the few below (one in 20) are off by up to 2^-22 of
    it, 2^-12, which moves a score by about sqrt(128 / 20) * 2^-12 / sqrt(3) * 60 * 2^-6.5 / sqrt(128) = 2e-5."""
    c = T.Case(63, ctx=[1, 2, 130, 900, 2100], nq=[1, 1, 2, 3, 1], which=which, kv=2, topk=6)
    c.q[..., 3] = 1024.0
    c.k[..., 3] = 0
    out, lse = c.run()
    assert msa.device_status() == msa.MSA_OK
    c.check(out, lse, range(c.main))


@pytest.mark.parametrize("which", T.FORMS)
@pytest.mark.parametrize("q_size", [3e6, 1e9, 1e20, -1e9, -1e30])
def test_huge_scores(cuda_ok, which, q_size):
    """Every key of a row the same, scores up to 2^86 and down to -2^106: equal probabilities, whatever the scores' last bits.  The output is
    448 v_scale, moved by less than 2^-6 of itself (test_largest_values_under_equal_scores)."""
    c = T.Case(64, ctx=[400, 257], nq=[3, 2], which=which)
    c.k[:] = 0x7E
    c.v[:] = 0x7E
    c.ks[:] = 2.0 ** -6
    c.vs[:] = 2.0 ** -7
    c.q = torch.full_like(c.q, q_size)
    out, lse = c.run()
    assert msa.device_status() == msa.MSA_OK
    assert ((out[:c.rows].float() - 3.5).abs() <= 3.5 * 2.0 ** -6).all(), (float(out.min()), float(out.max()))
    want = float(c.q[0, 0, 0]) * 448 * 2.0 ** -6 * 128 ** 0.5
    assert ((lse[:c.rows].double() - want).abs() <= 1e-5 * abs(want)).all()
