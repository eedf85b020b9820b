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
