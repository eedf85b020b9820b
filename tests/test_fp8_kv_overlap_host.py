"""Inserts whose buffers lie over one another are refused before anything is
launched (made-up addresses; no GPU needed)."""
import ctypes

import pytest
import torch

import block_sparse_long_13_b200 as msa
from block_sparse_long_13_b200 import build

# addresses that nothing holds: only where no kernel could take them
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses")
NAMES = ["q", "k_new", "v_new", "q_norm_w", "k_norm_w", "q_out", "k_cache", "v_cache", "k_scale", "v_scale"]
WRITTEN = NAMES[5:]
ROWS, PAGES = 100, 3
SIZES = dict(q=ROWS * 64 * 256, k_new=ROWS * 4 * 256, v_new=ROWS * 4 * 256, q_norm_w=256, k_norm_w=256, q_out=ROWS * 64 * 256,
             k_cache=PAGES * 4 * 16384, v_cache=PAGES * 4 * 16384, k_scale=PAGES * 16, v_scale=PAGES * 16)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return msa.load_library()


def _call(lib, at, batch=None):
    batch = batch or msa.Batch.make([0, ROWS], [256], [[0, 1]], PAGES, device="cpu")
    return lib.msa_qknorm_rope_insert_fp8(ctypes.byref(msa.Config()._c()), ctypes.byref(batch._c(host_only=True)),
                                          *[ctypes.c_void_p(at[n]) for n in NAMES], 64, 1e4, 1e-6, None)


def _apart():
    return {n: (i + 1) << 28 for i, n in enumerate(NAMES)}


@pytest.mark.parametrize("written", WRITTEN)
def test_what_is_written_must_not_lie_over_anything(lib, written):
    for other in NAMES:
        if other == written:
            continue
        align = 4 if "scale" in written else 16
        # the last bytes of the other buffer, its first ones, and all of it
        for to in (_apart()[other] + SIZES[other] - align, _apart()[other] - SIZES[written] + align, _apart()[other]):
            if {written, other} == {"q", "q_out"} and to == _apart()[other]:
                continue                                    # in place: allowed
            if to % 16 and "scale" not in written:
                continue
            at = {**_apart(), written: to}
            assert _call(lib, at) == msa.MSA_ERR_INVALID_ARG, (written, other, to)
            message = lib.msa_last_error().decode()
            assert "overlap" in message and written in message and other in message


def test_queries_in_place_and_keys_there_too(lib):
    at = {**_apart(), "q_out": _apart()["q"], "k_new": _apart()["q"]}
    assert _call(lib, at) == msa.MSA_ERR_INVALID_ARG and "k_new" in lib.msa_last_error().decode()


def test_written_over_the_batch_arrays(lib):
    batch = msa.Batch.make([0, ROWS], [256], [[0, 1]], PAGES, device="cpu")
    for name in ("q_start", "ctx_len", "page_table"):
        at = {**_apart(), "k_scale": getattr(batch, name).data_ptr()}
        assert _call(lib, at, batch) == msa.MSA_ERR_INVALID_ARG
        assert name in lib.msa_last_error().decode()
    assert torch.equal(batch.q_start, torch.tensor([0, ROWS], dtype=torch.int32))
