"""The 8-bit K/V cache without a GPU: the calls' checks of their arguments, and
the oracle of its arithmetic against hand-worked values."""
import ctypes
import sys

import numpy as np
import pytest
import torch

import block_sparse_long_13_b200 as msa
from block_sparse_long_13_b200 import build
from oracle import fp8_cache as F
from oracle import fp8_kv as K


@pytest.fixture(scope="module")
def lib():
    build.build()
    return msa.load_library()


def _cfg(**kw):
    c = msa.Config()
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _batch(rows=128, device="cpu"):
    return msa.Batch.make([0, rows], [256], [[0, 1]], 2, device=device)


P = ctypes.c_void_p(16)       # never dereferenced: the checks fail first


def _attn(lib, which, cfg=None, batch=None, ptrs=None, ws=P, nbytes=1 << 40):
    cfg, batch = cfg or msa.Config(), batch or _batch()
    fn = lib.msa_attn_decode_fp8 if which == "decode" else lib.msa_attn_prefill_fp8
    q, k, v, ks, vs, sel, out, lse = ptrs or [P] * 8
    return fn(ctypes.byref(cfg._c()), ctypes.byref(batch._c(host_only=True)), q, k, v, ks, vs, sel, out, lse, ws, nbytes, None)


@pytest.mark.parametrize("which", ["decode", "prefill"])
def test_attention_refusals(lib, which):
    for i in range(7):                                              # lse alone may be NULL
        ptrs = [P] * 8
        ptrs[i] = None
        assert _attn(lib, which, ptrs=ptrs) == msa.MSA_ERR_INVALID_ARG, i
        assert b"NULL" in lib.msa_last_error()
    for i in (0, 1, 2, 6):
        ptrs = [P] * 8
        ptrs[i] = ctypes.c_void_p(24)
        assert _attn(lib, which, ptrs=ptrs) == msa.MSA_ERR_INVALID_ARG, i
    for i in (3, 4, 5, 7):
        ptrs = [P] * 8
        ptrs[i] = ctypes.c_void_p(18)
        assert _attn(lib, which, ptrs=ptrs) == msa.MSA_ERR_INVALID_ARG, i
        assert b"4-byte" in lib.msa_last_error()
    size = (msa.decode_fp8_workspace_bytes if which == "decode" else msa.prefill_fp8_workspace_bytes)(msa.Config(), _batch())
    assert size > 0
    assert _attn(lib, which, nbytes=size - 1) == msa.MSA_ERR_INVALID_ARG and b"workspace" in lib.msa_last_error()
    assert _attn(lib, which, ws=None) == msa.MSA_ERR_INVALID_ARG
    assert _attn(lib, which, cfg=_cfg(head_dim=64)) == msa.MSA_ERR_UNSUPPORTED
    assert _attn(lib, which, cfg=_cfg(topk=65)) == msa.MSA_ERR_UNSUPPORTED
    big = _batch()
    big.num_pages = 1 << 23                                         # 2^23 pages x 4 heads x 128 rows = 2^32
    assert _attn(lib, which, batch=big) == msa.MSA_ERR_UNSUPPORTED
    big = _batch()
    big.total_q = 1 << 24                                           # 2^24 rows x 4 groups x 64 slots = 2^32
    assert _attn(lib, which, cfg=_cfg(topk=64), batch=big) == msa.MSA_ERR_UNSUPPORTED
    # no rows: checked, nothing launched
    assert _attn(lib, which, batch=_batch(0)) == msa.MSA_OK


def test_workspace_sizes_of_invalid_arguments_are_zero(lib):
    for fn in (lib.msa_decode_fp8_workspace_bytes, lib.msa_prefill_fp8_workspace_bytes):
        assert fn(ctypes.byref(_cfg(head_dim=64)._c()), ctypes.byref(_batch()._c(host_only=True))) == 0


def test_insert_refusals(lib):
    def call(ptrs=None, rd=64, theta=10000.0, eps=1e-6, cfg=None, rows=128):
        a = ptrs or [P] * 10
        return lib.msa_qknorm_rope_insert_fp8(ctypes.byref((cfg or msa.Config())._c()),
                                              ctypes.byref(_batch(rows)._c(host_only=True)), *a, rd, theta, eps, None)
    for i in range(10):
        ptrs = [P] * 10
        ptrs[i] = None
        assert call(ptrs) == msa.MSA_ERR_INVALID_ARG, i
        ptrs[i] = ctypes.c_void_p(18 if i >= 8 else 24)
        assert call(ptrs) == msa.MSA_ERR_INVALID_ARG, i
        assert b"aligned" in lib.msa_last_error()
    for rd in (0, -8, 60, 136):
        assert call(rd=rd) == msa.MSA_ERR_INVALID_ARG, rd
    for bad in (dict(theta=0.0), dict(theta=float("inf")), dict(eps=-1.0), dict(eps=float("nan"))):
        assert call(**bad) == msa.MSA_ERR_INVALID_ARG, bad
    assert call(cfg=_cfg(block_size=64)) == msa.MSA_ERR_UNSUPPORTED
    assert call(rows=0) == msa.MSA_OK


def test_advance_refusals(lib):
    def call(n=2, width=4, pages=8, block=128, ptrs=None, rows=4):
        return lib.msa_advance_batch(n, width, pages, block, *(ptrs or [P] * 9), rows, None)
    for bad in (dict(n=0), dict(width=0), dict(pages=0), dict(rows=-1)):
        assert call(**bad) == msa.MSA_ERR_INVALID_ARG, bad
    for bad in (dict(n=8193), dict(width=16385), dict(pages=1 << 24), dict(block=64),
                dict(rows=(1 << 30) + 1)):
        assert call(**bad) == msa.MSA_ERR_UNSUPPORTED, bad
    for i in range(8):
        ptrs = [P] * 9
        ptrs[i] = None
        assert call(ptrs=ptrs) == msa.MSA_ERR_INVALID_ARG, i
    for i in range(9):
        ptrs = [P] * 9
        ptrs[i] = ctypes.c_void_p(18)
        assert call(ptrs=ptrs) == msa.MSA_ERR_INVALID_ARG, i
    assert call(ptrs=[P] * 8 + [None], rows=3) == msa.MSA_ERR_INVALID_ARG


def _refused(fn, *args, **kw):
    with pytest.raises(msa.MsaError) as e:
        fn(*args, **kw)
    assert e.value.status == msa.MSA_ERR_INVALID_ARG
    return str(e.value)


def test_binding_refuses_wrong_shapes_and_cpu_tensors(lib):
    cfg, b = msa.Config(), _batch(4)
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)  # noqa: E731
    good = dict(q=z(4, 64, 128), k=z(2, 4, 128, 128, dtype=torch.uint8), v=z(2, 4, 128, 128, dtype=torch.uint8),
                ks=z(2, 4, dtype=torch.float32), vs=z(2, 4, dtype=torch.float32), sel=z(4, 4, 16, dtype=torch.int32),
                out=z(4, 64, 128), lse=z(4, 64, dtype=torch.float32), ws=z(1 << 20, dtype=torch.uint8))
    wrong = dict(q=z(3, 64, 128), k=z(3, 4, 128, 128, dtype=torch.uint8), v=z(2, 4, 64, 128, dtype=torch.uint8),
                 ks=z(2, dtype=torch.float32), vs=z(4, 2, dtype=torch.float32), sel=z(4, 4, 15, dtype=torch.int32),
                 out=z(4, 64, 64), lse=z(4, 4, dtype=torch.float32))
    for fn in (msa.attn_decode_fp8, msa.attn_prefill_fp8):
        for name, t in wrong.items():
            assert "shape" in _refused(fn, cfg, b, *{**good, name: t}.values()), name
        assert "CUDA tensor" in _refused(fn, cfg, b, *good.values())
    ins = dict(q=z(4, 64, 128), kn=z(4, 4, 128), vn=z(4, 4, 128), qw=z(128), kw=z(128), qo=z(4, 64, 128), k=good["k"],
               v=good["v"], ks=good["ks"], vs=good["vs"])
    wrong = dict(q=z(5, 64, 128), kn=z(4, 2, 128), vn=z(3, 4, 128), qw=z(64), kw=z(129), qo=z(4, 64, 64))
    for name, t in wrong.items():
        assert "shape" in _refused(msa.qknorm_rope_insert_fp8, cfg, b, *{**ins, name: t}.values()), name
    assert "CUDA tensor" in _refused(msa.qknorm_rope_insert_fp8, cfg, b, *ins.values())
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    adv = dict(delta=i32(2), ctx=i32(2), table=i32(2, 4), ring=i32(8), pool=i32(4), ctx2=i32(2), pool2=i32(4), qs=i32(3), sl=i32(5))
    for name, t in dict(delta=i32(3), ctx=i32(1), table=i32(8), pool=i32(2), ctx2=i32(4), pool2=i32(3), qs=i32(2)).items():
        _refused(msa.advance_batch, *{**adv, name: t}.values())
    assert "CUDA tensor" in _refused(msa.advance_batch, *adv.values())


def test_native_calls_leave_what_does_not_fit_to_python(lib):
    """None for whatever is not exactly right, no Python error left behind and no reference lost or kept."""
    cfg, b = msa.Config(), _batch(4)
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)  # noqa: E731
    args = [z(4, 64, 128), z(2, 4, 128, 128, dtype=torch.uint8), z(2, 4, 128, 128, dtype=torch.uint8),
            z(2, 4, dtype=torch.float32), z(2, 4, dtype=torch.float32), z(4, 4, 16, dtype=torch.int32), z(4, 64, 128), None,
            None, None]
    held = [cfg, b, b.q_start, b.ctx_len, b.page_table, *args[:7], cfg.num_q_heads]
    before = [sys.getrefcount(x) for x in held[:-1]]
    ints = [torch.zeros(n, dtype=torch.int32) for n in (2, 2, 8, 4, 2, 4, 3)]
    for _ in range(50):
        assert msa._native().attn(False, cfg, b, *args) is None
        assert msa._native().attn(True, cfg, b, *args) is None
        assert msa._native().attn(False, None, b, *args) is None
        assert msa._native().attn(False, cfg, "batch", *args) is None
        assert msa._native().attn(False, cfg, b) is None
        for i in range(len(args)):
            assert msa._native().attn(False, cfg, b, *args[:i], object(), *args[i + 1:]) is None
        assert msa._native().attn(False, msa.Config(num_q_heads=1 << 40), b, *args) is None
        assert msa._native().attn(False, msa.Config(softmax_scale="1"), b, *args) is None
        assert msa._native().insert(cfg, b, *args[:4], args[3], args[3], args[0], *args[1:5], 64, 1e4, 1e-6, None) is None
        assert msa._native().advance(*ints[:2], torch.zeros(2, 4, dtype=torch.int32), *ints[2:], None, 128, None) is None
        assert msa._native().advance(*ints[:2], ints[2], *ints[2:], None, 128, None) is None
        assert msa._native().advance() is None
    assert [sys.getrefcount(x) for x in held[:-1]] == before
    with pytest.raises(TypeError):
        msa._native().setup(1, 2)
    with pytest.raises((TypeError, ValueError)):
        msa._native().setup(0, 0, 0, 0)


def test_binding_refuses_another_device(lib, monkeypatch):
    """A tensor that is not on the current device is named, whatever else is right."""
    class On:
        shape, dtype, is_cuda = torch.Size([4]), torch.int32, True

        def __init__(self, device):
            self.device = device

        def get_device(self):
            return self.device

        def is_contiguous(self):
            return True

        def data_ptr(self):
            return 16
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    assert msa._pointers((On(0), torch.int32, (4,), "a"), (None, torch.int32, (4,), "b")) == [16, 0]
    assert "b is on device 1, but device 0 is current" in _refused(msa._pointers, (On(0), torch.int32, (4,), "a"),
                                                                  (On(1), torch.int32, (4,), "b"))


# ----------------------------------------------------------------- the oracle
def test_block_scale_is_the_least_power_of_two_that_holds_the_value():
    assert K.block_scale(448.0) == 1.0 and K.block_scale(np.nextafter(448.0, 500.0)) == 2.0
    assert K.block_scale(3.5) == 2.0 ** -7 and K.block_scale(0.0) == 2.0 ** -126
    for a in (1e-3, 0.1, 1.0, 7.0, 1000.0):
        s = K.block_scale(a)
        assert 448 * s >= a > 224 * s


def test_oracle_insert_keeps_and_grows_scales():
    codes = np.full((2, 1, 128, 128), 0x38, dtype=np.uint8)          # 1.0
    scale = np.array([[0.5], [0.5]])
    v = np.zeros((2, 1, 128))
    v[0, 0, 0], v[1, 0, 0] = 100.0, 1000.0
    one = np.ones(128)
    for row, want, old in ((0, 0.5, 1.0), (1, 4.0, 0.125)):
        _, _, (target, s, kind) = K.insert(np.zeros((1, 16, 128)), np.zeros((1, 1, 128)), v[row:row + 1], one, one, [0],
                                           [3], [[1]], codes, codes, scale, scale)
        assert s[1, 0] == want and s[0, 0] == 0.5
        assert target[1, 0, 3, 0] == v[row, 0, 0] / want and (target[1, 0, :3] == old).all() and (target[1, 0, 4:] == 1).all()
        assert list(kind[1, 0, :5]) == ([0, 0, 0, 2, 0] if row == 0 else [1, 1, 1, 2, 0]) and not kind[0].any()


def test_oracle_attention_of_equal_keys_is_the_mean():
    codes = np.zeros((1, 1, 128, 128), dtype=np.uint8)
    rng = np.random.default_rng(0)
    vcodes = rng.integers(0, 0x7F, size=codes.shape).astype(np.uint8)
    one = np.ones((1, 1))
    out, lse, _ = K.attention(np.ones((1, 16, 128)), K.values(codes, one), K.values(vcodes, 2 * one), [0], [9], [[[0]]], [[0]])
    assert np.allclose(out, 2 * F.decode_bits(vcodes)[0, 0, :10].mean(axis=0)) and np.allclose(lse, np.log(10))


def test_oracle_advance_by_hand():
    # two pages free (5 then 2); sequence 0 crosses into a new page, 1 ends, 2 sits out
    ctx, table, ring, pool, q_start, slots = K.advance([3, -200, 0], [127, 200, 1], [[7, -1], [3, 4], [6, -1]],
                                                       [0, 5, 2, 0, 0, 0, 0, 0], [1, 2, 0, 0], 4)
    assert ctx == [130, 0, 1] and table[0] == [7, 5] and q_start == [0, 3, 3, 3]
    assert pool == [2, 3, 0, 3] and [ring[i] for i in (2, 3, 4)] == [2, 3, 4]
    assert slots == [7 * 128 + 127, 5 * 128, 5 * 128 + 1, -1]
    assert K.advance([500, 0], [0, 0], [[-1] * 8] * 2, [4, 5], [0, 2], 500)[3] == [0, 2, 2, 0]
    assert K.advance([-1, 0], [0, 0], [[-1] * 8] * 2, [4, 5], [0, 2], 500)[3] == [0, 2, -1, 0]
