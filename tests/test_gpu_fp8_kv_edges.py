"""The 8-bit K/V cache's calls at the edges of what their documentation allows."""
import threading

import numpy as np
import pytest
import torch

from . import test_gpu_fp8_kv as T

msa = T.msa
pytestmark = pytest.mark.gpu


def _together(work, args):
    """work(a) for every a, in threads of their own that begin together; what they raise is raised here."""
    wrong, start = [], threading.Barrier(len(args))

    def run(a):
        try:
            start.wait()
            side = torch.cuda.Stream()
            with torch.cuda.stream(side):
                work(a)
            side.synchronize()
        except Exception as e:  # noqa: BLE001
            wrong.append(e)
    threads = [threading.Thread(target=run, args=(a,)) for a in args]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if wrong:
        raise wrong[0]


def test_advances_of_many_and_of_more_sequences_at_once(cuda_ok):
    """Both want more shared memory than a kernel has without asking, and not the same amount."""
    dev = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    calls = [dict(delta=dev(n), ctx=dev(n), table=dev(n, 1), ring=dev(4), pool=dev(4), qs=dev(n + 1)) for n in (3000, 8192, 5000)]
    torch.cuda.synchronize()

    def work(c):
        for _ in range(1500):
            msa.advance_batch(c["delta"], c["ctx"], c["table"], c["ring"], c["pool"], c["ctx"], c["pool"], c["qs"])
    _together(work, calls)
    assert msa.device_status() == msa.MSA_OK


def test_inserts_of_different_head_counts_at_once(cuda_ok):
    cases = [T._insert_case(71 + kv, ctx=[40], nq=[1], kv=kv) for kv in (13, 16)]
    for c in cases:
        c["dev"] = [c[n].cuda() for n in ("q", "k_new", "v_new", "qw", "kw")] + \
            [torch.from_numpy(x).cuda() for x in (*c["codes"], *c["scales"])]
    torch.cuda.synchronize()

    def work(c):
        q, kn, vn, qw, kw, k, v, ks, vs = c["dev"]
        for _ in range(1000):
            msa.qknorm_rope_insert_fp8(c["cfg"], c["batch"], q, kn, vn, qw, kw, q, k, v, ks, vs)
    _together(work, cases)
    assert msa.device_status() == msa.MSA_OK


@pytest.mark.parametrize("which", T.FORMS)
def test_a_nan_value_reaches_its_own_dim_only(cuda_ok, which):
    """Single NaN codes in values: rows that see one have NaN in its dim, for every head, and what the others hold
    elsewhere; lse does not notice."""
    c = T.Case(72, ctx=[100, 700], nq=[100, 40], which=which, kv=2, topk=6)
    for s, at, g, dim, code in ((0, 60, 0, 5, 0x7F), (0, 0, 1, 127, 0xFF), (0, 99, 1, 0, 0x7F), (1, 130, 1, 64, 0x7F),
                                (1, 130, 1, 79, 0xFF), (1, 690, 0, 33, 0xFF)):
        c.v[c.table[s, at // 128], g, at % 128, dim] = code
    rows = np.arange(c.main)
    ref, ref_lse, mag = T.K.attention(c.q[rows].double().numpy(), T.K.values(c.k, c.ks), T.K.values(c.v, c.vs), c.seq[rows],
                                      c.pos[rows], c.sel[rows], c.table)
    out, lse = c.run()
    assert msa.device_status() == msa.MSA_OK
    got = out[:c.main].double().cpu().numpy()
    nan = np.isnan(ref)
    assert 0 < nan.sum() < nan.size // 16 and np.array_equal(np.isnan(got), nan)
    assert (np.abs(got - ref)[~nan] <= (2.0 ** -8 * np.abs(ref) + (2.0 ** -7 + 2.0 ** -12) * mag)[~nan]).all()
    assert np.abs(lse[:c.main].cpu().numpy() - ref_lse).max() <= T.LSE_ABS


def test_insert_of_more_rows_than_the_context_holds_writes_nothing(cuda_ok):
    """ctx_len 200 with 400 new rows: the positions would begin at -200.  Recorded, the caches stay, the other sequence's
    rows are inserted."""
    c = T._insert_case(73, ctx=[400, 130], nq=[400, 3], kv=2)
    whole = T._insert(c)
    c["batch"].ctx_len = torch.tensor([200, 130], dtype=torch.int32, device="cuda")
    got = T._insert(c)
    assert msa.device_status() == msa.MSA_ERR_DEVICE_BOUNDS
    kept = c["table"][0][c["table"][0] >= 0]
    other = c["table"][1][c["table"][1] >= 0]
    for x, before, all_in in zip(got[1:], (*c["codes"], *c["scales"]), whole[1:]):
        assert np.array_equal(x[torch.from_numpy(kept).long().cuda()].cpu().numpy(), before[kept])
        assert torch.equal(x[torch.from_numpy(other).long().cuda()], all_in[torch.from_numpy(other).long().cuda()])


@pytest.mark.parametrize("power", [125, 126, 127])
def test_insert_under_the_largest_scales(cuda_ok, power):
    """A page that goes on under an old scale of 2^126 and more: a code is value / scale there too.  (Values of 2^120 need
    no such scale, but the page keeps the one that it has.)"""
    c = T._insert_case(74, ctx=[40, 77], nq=[4, 12], kv=1)
    c["v_new"] = (c["v_new"].double().sign() * 2.0 ** torch.from_numpy(np.random.default_rng(0).uniform(118, 123, (16, 1, 128)))).to(torch.bfloat16)
    for s in range(2):
        c["scales"][1][c["table"][s, 0]] = 2.0 ** power
    got = T._insert(c)
    assert msa.device_status() == msa.MSA_OK
    T._check_insert(c, got)
    assert (got[2][int(c["table"][0, 0]), 0, 36:40] & 0x7F).any()


def test_calls_without_the_native_module_give_the_same_bits(cuda_ok, monkeypatch):
    """The checks of _bind.so and those of Python stand side by side: the same calls pass either."""
    def results():
        got = []
        for which in T.FORMS:
            c = T.Case(75, ctx=[300, 129], nq=[2, 1], which=which)
            got += [*c.run(), c.run(lse=False)[0]]
        got += T._insert(T._insert_case(76, ctx=[300, 129], nq=[20, 1], kv=2))
        table, ring, pool = T._pool_case(9, [127, 300], [2, -45])
        got += [torch.tensor(x) for x in T._advance([2, -45], [127, 300], table, ring, pool, 3)]
        return got
    native = results()
    assert msa._calls is not msa._NotNative
    monkeypatch.setattr(msa, "_calls", msa._NotNative)
    for a, b in zip(native, results()):
        assert torch.equal(a, b)
    assert msa.device_status() == msa.MSA_OK


@pytest.mark.parametrize("which", T.FORMS)
def test_a_nan_scale_makes_its_block_nan(cuda_ok, which):
    c = T.Case(77, ctx=[300, 300, 300], nq=[2, 2, 2], which=which, kv=2, topk=3)
    c.ks[c.table[0, 1], 1] = float("nan")
    c.vs[c.table[1, 0], 0] = float("nan")
    out, lse = c.run()
    assert msa.device_status() == msa.MSA_OK
    assert out[0:2, 16:].isnan().all() and lse[0:2, 16:].isnan().all() and not out[0:2, :16].isnan().any()
    assert out[2:4, :16].isnan().all() and not lse[2:4].isnan().any() and not out[2:4, 16:].isnan().any()
    c.check(out, lse, [4, 5])
