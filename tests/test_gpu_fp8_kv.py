"""The 8-bit K/V cache on the GPU against its float64 oracle (oracle/fp8_kv.py):
attention over it, the insert into it, the batch's index arrays, and a run of
them together.

Tolerances, from the roundings on the way (a rounding is off by at most half a
step: bf16 2^-8, e4m3 2^-4, relative to the value):
* an attention output is rounded to bf16 at the end, 2^-8 |out|; its
  probabilities may be held with 8 significant bits, 2^-8 each, and partial
  results over a block in bf16, 2^-8 of the partial, which move the output by at
  most 2^-8 of the softmax's mean of |v| (`mag`) each; fp32 sums, exponentials and
  the scaling add under 2^-12 mag.  Together 2^-8 |out| + (2^-7 + 2^-12) mag.
* a logit is an fp32 sum of 128 exact products: at most 128 2^-24 of the sum of
  their sizes, at most 128 2^-24 * 30 = 2.3e-4 for these inputs, which is what an
  lse moves by at most (the exponentials' and the logarithm's errors are 2^-22).
* a code is off by half a step, 2^-4 of the value or 2^-10 of the scale (below
  the codes' normal range), on top of fp32 arithmetic (1e-5).
"""
import threading

import numpy as np
import pytest
import torch

import block_sparse_long_13_b200 as msa
from oracle import fp8_cache as F
from oracle import fp8_kv as K

pytestmark = pytest.mark.gpu

LSE_ABS = 2.5e-4
ATTN = {"decode": msa.attn_decode_fp8, "prefill": msa.attn_prefill_fp8}
WORKSPACE = {"decode": msa.decode_fp8_workspace_bytes, "prefill": msa.prefill_fp8_workspace_bytes}
# a prefill call of few rows takes the decode form: "tiles" are prefill calls with a long sequence more
FORMS = ["decode", "prefill", "tiles"]
BALLAST = 2600


# ----------------------------------------------------------------- attention
class Case:
    def __init__(self, seed, ctx, nq, which="decode", kv=4, topk=16, pad=0, extra_width=0, empty=(), q_size=1.0):
        rng = np.random.default_rng(seed)
        self.fn, self.size = ATTN.get(which, msa.attn_prefill_fp8), WORKSPACE.get(which, msa.prefill_fp8_workspace_bytes)
        self.main = sum(nq)                        # rows of the sequences that the test is about
        if which == "tiles":
            ctx, nq = list(ctx) + [BALLAST], list(nq) + [BALLAST]
        self.kv, self.topk, self.ctx, self.nq = kv, topk, ctx, nq
        starts = np.concatenate([[0], np.cumsum(nq)])
        self.rows, self.starts = int(starts[-1]), starts
        width = max(-(-c // 128) for c in ctx) + extra_width
        need = sum(-(-c // 128) for c in ctx)
        self.pages = need + 2
        perm = rng.permutation(self.pages)
        self.table = np.full((len(ctx), width), -1, dtype=np.int32)
        at = 0
        for s, c in enumerate(ctx):
            n = -(-c // 128)
            self.table[s, :n] = perm[at:at + n]
            at += n
        # every byte is legal outside the tokens: NaN codes there must not matter
        self.k = rng.integers(0, 256, size=(self.pages, kv, 128, 128)).astype(np.uint8)
        self.v = rng.integers(0, 256, size=(self.pages, kv, 128, 128)).astype(np.uint8)
        for s, c in enumerate(ctx):
            for b in range(-(-c // 128)):
                n = min(128, c - b * 128)
                for x in (self.k, self.v):
                    y = torch.from_numpy(rng.normal(size=(kv, n, 128)) * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
                    x[self.table[s, b], :, :n] = y.view(torch.uint8).numpy()
        self.ks = (2.0 ** rng.uniform(-7.5, -5.5, size=(self.pages, kv))).astype(np.float32)
        self.vs = (2.0 ** rng.uniform(-7.5, -5.5, size=(self.pages, kv))).astype(np.float32)
        self.q = torch.from_numpy(rng.normal(size=(self.rows, 16 * kv, 128)) * q_size).to(torch.bfloat16)
        self.seq = np.concatenate([np.full(n, s) for s, n in enumerate(nq)] + [[]]).astype(np.int64)
        self.pos = np.concatenate([np.arange(c - n, c) for c, n in zip(ctx, nq)] + [[]]).astype(np.int64)
        self.sel = np.full((self.rows, kv, topk), -1, dtype=np.int32)
        for t in range(self.rows):
            cur = int(self.pos[t]) // 128
            for g in range(kv):
                if (t, g) in empty:
                    continue
                ids = rng.permutation(cur)[:topk - 1]
                self.sel[t, g, :len(ids) + 1] = np.sort(np.append(ids, cur))
        self.pad = pad
        self.cfg = msa.Config(num_q_heads=16 * kv, num_kv_heads=kv, idx_heads=kv, topk=topk)
        self.batch = msa.Batch.make(starts.tolist(), ctx, self.table, self.pages)
        self.batch.total_q += pad

    def device(self):
        if not hasattr(self, "_d"):
            grow = lambda x: torch.cat([x, x[:1].expand(self.pad, *x.shape[1:])]) if self.pad else x  # noqa: E731
            self._d = [grow(self.q).cuda(), *[torch.from_numpy(x).cuda() for x in (self.k, self.v, self.ks, self.vs)],
                       grow(torch.from_numpy(self.sel)).contiguous().cuda()]
        return self._d

    def run(self, lse=True, stream=None):
        d = self.device()
        out = torch.full_like(d[0], 7.0)
        l = torch.full(d[0].shape[:2], 7.0, device="cuda") if lse else None
        ws = torch.full((self.size(self.cfg, self.batch),), 0xFF, dtype=torch.uint8, device="cuda")
        self.fn(self.cfg, self.batch, *d, out, l, ws, stream=stream)
        return out, l

    def check(self, out, lse, rows=None):
        if rows is None:
            rows = [*range(0, self.main, max(1, self.main // 200)), *range(self.main, self.rows, 97)]
        rows = np.asarray(list(rows))
        ref, ref_lse, mag = K.attention(self.q[rows].double().numpy(), K.values(self.k, self.ks), K.values(self.v, self.vs),
                                        self.seq[rows], self.pos[rows], self.sel[rows], self.table)
        got = out[torch.from_numpy(rows).cuda()].double().cpu().numpy()
        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -7 + 2.0 ** -12) * mag
        err = np.abs(got - ref)
        assert (err <= tol).all(), (float((err - tol).max()), np.argwhere(~(err <= tol))[:4].tolist())
        if lse is not None:
            gl = lse[torch.from_numpy(rows).cuda()].double().cpu().numpy()
            empty = np.isinf(ref_lse)
            assert (gl[empty] == -np.inf).all() and (got[empty] == 0).all()
            off = np.abs(gl[~empty] - ref_lse[~empty])
            assert (off <= LSE_ABS).all(), float(off.max())


SHAPES = {
    "one token": dict(ctx=[1], nq=[1]),
    "lengths around a block": dict(ctx=[1, 2, 127, 128, 129, 255, 256, 257], nq=[1, 2, 1, 1, 2, 3, 1, 2]),
    "many blocks a row": dict(ctx=[9000, 300], nq=[3, 1], topk=64),
    "one block a row": dict(ctx=[700, 129, 128], nq=[2, 2, 8], topk=1),
    "odd topk, one group": dict(ctx=[3000, 1111], nq=[4, 8], kv=1, topk=7),
    "two groups": dict(ctx=[2500, 100, 5000], nq=[1, 3, 2], kv=2, topk=15),
    "sequences without rows": dict(ctx=[400, 500, 300, 50, 600], nq=[0, 2, 0, 1, 0], extra_width=3),
    "rows of one sequence": dict(ctx=[1500], nq=[150], kv=2, topk=4),
    "more rows than one wave": dict(ctx=[300] * 60, nq=[3] * 60, topk=3),
    "many tiles a block": dict(ctx=[1700, 300], nq=[1600, 260], kv=1, topk=4),
    "blocks shared by few rows": dict(ctx=[6000, 3000], nq=[300, 200], kv=2, topk=16),
}


@pytest.mark.parametrize("which", FORMS)
@pytest.mark.parametrize("shape", SHAPES)
def test_attention_matches_oracle(cuda_ok, shape, which):
    c = Case(3, which=which, **SHAPES[shape])
    out, lse = c.run()
    assert msa.device_status() == msa.MSA_OK
    c.check(out, lse)


def test_more_rows_than_a_window(cuda_ok):
    """Rows of several scheduling windows, tiles in several rounds over the CTAs."""
    c = Case(15, ctx=[9000, 12000, 100], nq=[8000, 9500, 50], which="prefill", kv=1, topk=12)
    out, lse = c.run()
    assert msa.device_status() == msa.MSA_OK
    c.check(out, lse, [*range(0, c.rows, 251), 7999, 8000, 8191, 8192, 16383, 16384, 17499, 17500, 17549])


@pytest.mark.parametrize("which", FORMS)
def test_rows_without_keys_and_padded_rows(cuda_ok, which):
    """A selection of -1 only gives out 0 and lse -inf; rows behind the last sequence stay as they were."""
    c = Case(4, ctx=[1000, 40, 2000], nq=[4, 2, 3], which=which, pad=5, empty=[(0, 0), (0, 1), (0, 2), (0, 3), (4, 2), (8, 3), (5, 0)])
    out, lse = c.run()
    assert msa.device_status() == msa.MSA_OK
    c.check(out[:c.rows], lse[:c.rows])
    assert (out[c.rows:] == 7.0).all() and (lse[c.rows:] == 7.0).all()


@pytest.mark.parametrize("which", FORMS)
def test_holes_and_order_of_the_selection_do_not_matter(cuda_ok, which):
    """-1 anywhere in a row and ids in any order; without lse."""
    c = Case(5, ctx=[3000, 700], nq=[3, 2], which=which, topk=16)
    rng = np.random.default_rng(0)
    for t in range(c.rows):
        for g in range(c.kv):
            c.sel[t, g] = rng.permutation(c.sel[t, g])
            c.sel[t, g, rng.integers(0, 16, size=3)] = -1
    out, _ = c.run(lse=False)
    assert msa.device_status() == msa.MSA_OK
    c.check(out, None)


@pytest.mark.parametrize("which", FORMS)
def test_a_block_selected_twice_counts_twice(cuda_ok, which):
    c = Case(16, ctx=[700, 500], nq=[2, 3], which=which, kv=2, topk=5)
    c.sel[:c.main, :, 0] = c.sel[:c.main, :, 1]
    out, lse = c.run()
    assert msa.device_status() == msa.MSA_OK
    c.check(out, lse)


@pytest.mark.parametrize("which", FORMS)
@pytest.mark.parametrize("q_size", [0.0, 1.0, 300.0, 3e4])
def test_largest_values_under_equal_scores(cuda_ok, which, q_size):
    """Every code is the largest one and every key of a row the same: 128 equal probabilities a block, and logits up to
    2^21.  The output is 448 v_scale for any weights; the weights' roundings (8 bits, 2^-8), a partial's (2^-8) and the output's
    (2^-8) move it by less than 2^-6 of itself."""
    c = Case(41, ctx=[400, 257], nq=[3, 2], which=which)
    c.k[:] = 0x7E
    c.v[:] = 0x7E
    c.ks[:] = 2.0 ** -6
    c.vs[:] = 2.0 ** -7
    c.q = torch.full_like(c.q, q_size)
    out, lse = c.run()
    assert msa.device_status() == msa.MSA_OK
    assert ((out[:c.rows].float() - 3.5).abs() <= 3.5 * 2.0 ** -6).all(), (float(out.min()), float(out.max()))
    assert torch.isfinite(lse[:c.rows]).all()


@pytest.mark.parametrize("which", FORMS)
@pytest.mark.parametrize("q_size", [1e-30, 1e-3, 4.0])
def test_query_sizes(cuda_ok, which, q_size):
    """Queries from tiny to large, a head of zeros, elements 2^-12 below their head's largest."""
    c = Case(6, ctx=[900, 130], nq=[2, 2], which=which, kv=2, topk=4, q_size=q_size)
    c.q[0, 3] = 0
    c.q[1, 5, ::2] *= 2.0 ** -12
    if q_size > 1:                      # logits in the hundreds: an fp32 sum's bound grows with them
        c.ks *= 0.25
    out, lse = c.run()
    assert msa.device_status() == msa.MSA_OK
    c.check(out, lse)


@pytest.mark.parametrize("which", FORMS)
def test_block_scales_far_apart(cuda_ok, which):
    """Scales of 0, tiny, large, negative and a block whose V alone is large: each block's own scale acts on it."""
    c = Case(7, ctx=[1300], nq=[2], which=which, kv=1, topk=11)
    for b, (ks, vs) in enumerate([(0.0, 1.0), (1e-20, 1e-20), (2.0 ** -6, 0.0), (2.0 ** -6, 2.0 ** 20), (2.0 ** -5, 2.0 ** -126),
                                  (-2.0 ** -6, -2.0 ** -6)]):
        c.ks[c.table[0, b], 0], c.vs[c.table[0, b], 0] = ks, vs
    out, lse = c.run()
    assert msa.device_status() == msa.MSA_OK
    c.check(out, lse)


@pytest.mark.parametrize("which", FORMS)
def test_nan_reaches_its_own_row_only(cuda_ok, which):
    """A NaN code among a row's keys or values, or in its query, makes that row's heads NaN and no other's."""
    c = Case(8, ctx=[300, 300, 300, 300], nq=[1] * 4, which=which, kv=1, topk=3)
    c.k[c.table[0, 1], 0, 5, 7] = 0x7F
    c.v[c.table[1, 0], 0, 9, :] = 0xFF
    c.q[2, 4, 100] = float("nan")
    out, lse = c.run()
    assert msa.device_status() == msa.MSA_OK
    assert out[0].isnan().all() and lse[0].isnan().all() and out[1].isnan().all() and not lse[1].isnan().any()
    assert out[2, 4].isnan().all() and lse[2, 4].isnan() and int(out[2].isnan().sum()) == 128
    c.check(out, lse, [3])
    ref = Case(8, ctx=[300, 300, 300, 300], nq=[1] * 4, which=which, kv=1, topk=3)
    ro, rl = ref.run()
    keep = [h for h in range(16) if h != 4]
    assert torch.equal(out[2, keep], ro[2, keep]) and torch.equal(lse[2, keep], rl[2, keep])


@pytest.mark.parametrize("which", FORMS)
def test_nan_value_behind_a_row_does_not_reach_it(cuda_ok, which):
    """Rows of one block on both sides of a NaN value: only those that see it are NaN."""
    c = Case(13, ctx=[100], nq=[100], which=which, kv=1, topk=1)
    c.v[c.table[0, 0], 0, 60] = 0x7F
    out, lse = c.run()
    assert msa.device_status() == msa.MSA_OK
    assert out[60:100].isnan().all() and not out[:60].isnan().any() and not lse[:100].isnan().any()
    c.check(out, lse, [*range(0, 60, 7), 59])


@pytest.mark.parametrize("which", FORMS)
def test_every_code_is_read_as_its_value(cuda_ok, which):
    """One key a row: the output is the value itself, and a one-hot query's lse the key's element."""
    c = Case(14, ctx=[1] * 16, nq=[1] * 16, which=which, kv=1, topk=1)
    for s in range(16):
        codes = (np.arange(128) + 128 * (s // 8)).astype(np.uint8)
        codes[127] = 0
        page = c.table[s, 0]
        c.k[page, 0, 0], c.v[page, 0, 0] = codes, codes
        c.ks[page, 0], c.vs[page, 0] = 0.5, 0.25
        c.q[s] = 0
        for h in range(16):
            c.q[s, h, 16 * (s % 8) + h] = 1.0
    out, lse = c.run()
    assert msa.device_status() == msa.MSA_OK
    for s in range(16):
        value = torch.from_numpy(F.decode_bits(c.k[c.table[s, 0], 0, 0]))
        assert torch.equal(out[s].double().cpu(), (0.25 * value).expand(16, 128))
        want = 0.5 * value[16 * (s % 8):16 * (s % 8) + 16] / 128 ** 0.5
        assert torch.allclose(lse[s].double().cpu(), want, rtol=2e-6, atol=1e-6)


@pytest.mark.parametrize("which", FORMS)
def test_bad_pages_and_blocks_are_recorded_and_left_out(cuda_ok, which):
    c = Case(9, ctx=[2000, 900], nq=[2, 1], which=which, kv=2, topk=5, extra_width=1)
    want = c.sel.copy()
    bad_b = int(c.sel[0, 0, 0])
    c.table = c.table.copy()
    good = c.table.copy()
    c.table[0, bad_b] = c.pages                        # a page past the pool
    want[:2][want[:2] == bad_b] = -1                   # sequence 0's rows lose that block
    c.sel[2, 1, 1] = 16                                # a block id past the table
    want[2, 1, 1] = -1
    c.sel[2, 0, 0] = 12                                # a block after the query's
    want[2, 0, 0] = -1
    c.batch = msa.Batch.make(c.starts.tolist(), c.ctx, c.table, c.pages)
    out, lse = c.run()
    assert msa.device_status() == msa.MSA_ERR_DEVICE_BOUNDS
    assert msa.device_status() == msa.MSA_OK
    c.sel, c.table = want, good
    c.check(out, lse)


@pytest.mark.parametrize("which", FORMS)
def test_same_bits_again_on_other_pages_and_another_stream(cuda_ok, which):
    c = Case(10, ctx=[5000, 260, 3000], nq=[5, 40, 7], which=which, topk=16)
    a = c.run()
    b = c.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        e = c.run()
    torch.cuda.current_stream().wait_stream(side)
    perm = np.random.default_rng(1).permutation(c.pages)        # page p moves to inv[p]
    inv = np.argsort(perm)
    c.k, c.v, c.ks, c.vs = c.k[perm], c.v[perm], c.ks[perm], c.vs[perm]
    c.table = np.where(c.table >= 0, inv[c.table], -1).astype(np.int32)
    c.batch = msa.Batch.make(c.starts.tolist(), c.ctx, c.table, c.pages)
    del c._d
    f = c.run()
    assert msa.device_status() == msa.MSA_OK
    for x in (b, e, f):
        assert torch.equal(a[0], x[0]) and torch.equal(a[1], x[1])


@pytest.mark.parametrize("which", FORMS)
def test_two_threads_call_at_once(cuda_ok, which):
    """Each on a stream and with a workspace of its own; the interpreter's lock is not held inside the call."""
    cases = [Case(51 + i, ctx=[700, 40], nq=[3, 1], which=which) for i in range(2)]
    want = [c.run() for c in cases]
    torch.cuda.synchronize()
    got, wrong = [[], []], []

    def work(i):
        try:
            side = torch.cuda.Stream()
            with torch.cuda.stream(side):
                got[i] = [cases[i].run() for _ in range(10)]
            side.synchronize()
        except Exception as e:  # noqa: BLE001
            wrong.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    assert msa.device_status() == msa.MSA_OK
    for i in range(2):
        for out, lse in got[i]:
            assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])


def test_forms_of_the_arguments(cuda_ok):
    """Streams as objects and numbers, weights as parameters and numbers of other types give the same bits; what is of
    the wrong type, layout or shape is refused by name."""
    c = Case(31, ctx=[300, 129], nq=[2, 1])
    d = c.device()
    ref, _ = c.run()
    ws = torch.zeros(c.size(c.cfg, c.batch), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    scale = float(c.cfg.head_dim) ** -0.5
    for cfg, q, stream in ((c.cfg, d[0], side), (c.cfg, d[0], side.cuda_stream), (c.cfg, d[0], 0),
                           (c.cfg, torch.nn.Parameter(d[0]), None),
                           (msa.Config(64, 4, idx_heads=4, topk=np.int64(16), softmax_scale=np.float64(scale)), d[0], None),
                           (msa.Config(64, 4, idx_heads=4, topk=16, softmax_scale=0), d[0], None)):
        out = torch.full_like(d[0], 7.0)
        side.wait_stream(torch.cuda.current_stream())
        c.fn(cfg, c.batch, q, *d[1:], out, None, ws, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
    good = [*d, torch.empty_like(d[0]), None, ws]
    for i, bad, what in ((0, d[0].float(), "q must be torch.bfloat16"), (0, d[0].transpose(0, 1).contiguous().transpose(0, 1), "contiguous"),
                         (1, d[1].view(torch.int8), "k_cache_e4m3 must be"), (3, d[3].double(), "k_scale must be"),
                         (5, d[5].long(), "block_idx must be"), (6, good[6][:-1], "out has shape"), (7, ref, "lse has shape"),
                         (8, ws.view(1, -1), "workspace has shape"), (8, ws.cpu(), "CUDA tensor")):
        with pytest.raises(msa.MsaError) as e:
            c.fn(c.cfg, c.batch, *good[:i], bad, *good[i + 1:])
        assert e.value.status == msa.MSA_ERR_INVALID_ARG and what in str(e.value)


@pytest.mark.parametrize("which", FORMS)
def test_graphs_with_their_own_workspaces(cuda_ok, which):
    """Two captured calls, replayed in turn and with new inputs in place, give what the eager calls give."""
    cases = [Case(11, ctx=[2000, 500], nq=[3, 1], which=which), Case(12, ctx=[129, 4000], nq=[9, 30], which=which)]
    graphs, results = [], []
    for c in cases:
        c.run()                                             # the first call is not captured
        d = c.device()
        out, lse = torch.zeros_like(d[0]), torch.zeros(d[0].shape[:2], device="cuda")
        ws = torch.zeros(c.size(c.cfg, c.batch), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.fn(c.cfg, c.batch, *d, out, lse, ws)
        graphs.append(g)
        results.append((out, lse, ws))
    for turn in range(3):
        for c, g, (out, lse, _) in zip(cases, graphs, results):
            c.device()[0].mul_(0.5 if turn else 1.0)
            g.replay()
            want = c.run()
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert msa.device_status() == msa.MSA_OK


# ----------------------------------------------------------------- insert
def _insert_case(seed, ctx, nq, kv=4, pad=0, magnitude=None, theta=10000.0, rotary_dim=64):
    rng = np.random.default_rng(seed)
    starts = np.concatenate([[0], np.cumsum(nq)])
    T = int(starts[-1])
    width = max(-(-c // 128) for c in ctx)
    touched = [(s, b) for s, (c, n) in enumerate(zip(ctx, nq)) if n for b in range((c - n) // 128, (c - 1) // 128 + 1)]
    pages = len(touched) + 3
    perm = rng.permutation(pages)
    table = np.full((len(ctx), width), -1, dtype=np.int32)
    for (s, b), page in zip(touched, perm):
        table[s, b] = page
    bf = lambda *shape: torch.from_numpy(rng.normal(size=shape)).to(torch.bfloat16)  # noqa: E731
    size = torch.from_numpy(2.0 ** rng.uniform(-3, 3, size=(T, kv, 1))) if magnitude is None else magnitude
    c = dict(q=bf(T, 16 * kv, 128), k_new=(bf(T, kv, 128).double() * size).to(torch.bfloat16),
             v_new=(bf(T, kv, 128).double() * size).to(torch.bfloat16), qw=(1 + 0.3 * bf(128).float()).to(torch.bfloat16),
             kw=(1 + 0.3 * bf(128).float()).to(torch.bfloat16))
    codes = [rng.integers(0, 255, size=(pages, kv, 128, 128)).astype(np.uint8) for _ in range(2)]
    for x in codes:
        x[(x & 0x7F) == 0x7F] = 0                        # NaN codes have a test of their own
    scales = [(2.0 ** rng.integers(-10, -4, size=(pages, kv))).astype(np.float32) for _ in range(2)]
    batch = msa.Batch.make(starts.tolist(), ctx, table, pages)
    batch.total_q += pad
    seq = np.concatenate([np.full(n, s) for s, n in enumerate(nq)]).astype(np.int64)
    pos = np.concatenate([np.arange(x - n, x) for x, n in zip(ctx, nq)]).astype(np.int64)
    c.update(cfg=msa.Config(num_q_heads=16 * kv, num_kv_heads=kv, idx_heads=kv), batch=batch, table=table, codes=codes,
             scales=scales, seq=seq, pos=pos, theta=theta, rotary_dim=rotary_dim, pad=pad, T=T)
    return c


def _insert(c, in_place=False, stream=None):
    grow = lambda x: torch.cat([x, x[:1].expand(c["pad"], *x.shape[1:])]).contiguous().cuda() if c["pad"] else x.cuda()  # noqa: E731
    q = grow(c["q"])
    q_out = q if in_place else torch.full_like(q, 7.0)
    k, v = (torch.from_numpy(x).cuda() for x in c["codes"])
    ks, vs = (torch.from_numpy(x).cuda() for x in c["scales"])
    msa.qknorm_rope_insert_fp8(c["cfg"], c["batch"], q, grow(c["k_new"]), grow(c["v_new"]), c["qw"].cuda(), c["kw"].cuda(), q_out,
                               k, v, ks, vs, rotary_dim=c["rotary_dim"], rope_theta=c["theta"], eps=1e-6, stream=stream)
    return q_out, k, v, ks, vs


def _check_insert(c, got):
    q_out, k, v, ks, vs = got
    q_ref, rk, rv = K.insert(c["q"], c["k_new"], c["v_new"], c["qw"], c["kw"], c["seq"], c["pos"], c["table"], *c["codes"],
                             *c["scales"], rotary_dim=c["rotary_dim"], theta=c["theta"])
    q = q_out[:c["T"]].double().cpu().numpy()
    assert (np.abs(q - q_ref) <= (2.0 ** -8 + 1e-5) * np.abs(q_ref) + 1e-5).all(), float(np.abs(q - q_ref).max())
    for codes, scale, before, old, (target, want, kind) in ((k, ks, c["codes"][0], c["scales"][0], rk),
                                                            (v, vs, c["codes"][1], c["scales"][1], rv)):
        codes, scale = codes.cpu().numpy(), scale.double().cpu().numpy()
        assert np.array_equal(scale, want), np.argwhere(scale != want)[:4]
        value = F.decode_bits(codes)
        assert np.array_equal(codes[kind == 0], before[kind == 0])           # nothing else is written
        for which in (1, 2):
            a, b = value[kind == which], np.clip(target[kind == which], -448, 448)
            assert (np.abs(a - b) <= (2.0 ** -4 + 1e-5) * np.abs(b) + 2.0 ** -10 + 1e-5).all(), (which, float(np.abs(a - b).max()))
        # older codes that stay normal lose nothing when a power of two grows to another (code * old / new is then the code
        # with another exponent; from any other old scale the product has more bits and is rounded, which the bound allows)
        power = np.frexp(old)[0] == 0.5
        normal = (kind == 1)[..., None] & (np.abs(target) >= 2.0 ** -6) & power[:, :, None, None]
        assert np.array_equal(value[normal], target[normal])


INSERTS = {
    "decode rows": dict(ctx=[1, 128, 129, 1000, 77777, 1 << 20], nq=[1] * 6),
    "verify rows over page borders": dict(ctx=[130, 4, 258, 1027], nq=[4, 4, 4, 4], kv=2),
    "a prefill and decode rows": dict(ctx=[700, 300, 65], nq=[700, 1, 65], kv=1),
    "chunks begun and continued": dict(ctx=[500, 383, 129, 400], nq=[300, 128, 129, 17]),
    "sequences without rows": dict(ctx=[300, 500, 20, 7], nq=[0, 130, 0, 7], kv=2, pad=3),
}


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("shape", INSERTS)
def test_insert_matches_oracle(cuda_ok, shape, in_place):
    c = _insert_case(21, **INSERTS[shape])
    got = _insert(c, in_place)
    assert msa.device_status() == msa.MSA_OK
    _check_insert(c, got)
    if c["pad"]:
        tail = c["q"][:1].expand(c["pad"], -1, -1) if in_place else torch.full((c["pad"], *c["q"].shape[1:]), 7.0, dtype=torch.bfloat16)
        assert torch.equal(got[0][c["T"]:].cpu(), tail)


@pytest.mark.parametrize("shape", [dict(ctx=[8, 135, 500, 132], nq=[8, 8, 8, 8]), dict(ctx=[9, 135, 500, 132], nq=[9, 8, 3, 8]),
                                   dict(ctx=[*range(1, 701)], nq=[1] * 700, kv=1), dict(ctx=[1300, 40], nq=[1100, 3], kv=1)],
                         ids=["8 rows", "9 rows", "more pieces than CTAs", "rows of several waves"])
def test_insert_at_the_borders_of_its_forms(cuda_ok, shape):
    """Old scales are any numbers here: those that stay divide the new rows."""
    c = _insert_case(23, **shape)
    rng = np.random.default_rng(24)
    for x in c["scales"]:
        x[:] = rng.uniform(0.004, 0.05, size=x.shape)
    got = _insert(c)
    assert msa.device_status() == msa.MSA_OK
    _check_insert(c, got)


def test_insert_refuses_more_rows_than_the_batch_says(cuda_ok):
    """A sequence longer than max_q_per_seq is recorded, and the caches keep what they held for it."""
    for most in (2, 100):
        c = _insert_case(26, ctx=[300, 50], nq=[200, 1], kv=2)
        c["batch"].max_q_per_seq = most
        got = _insert(c)
        assert msa.device_status() == msa.MSA_ERR_DEVICE_BOUNDS
        kept = c["table"][0][c["table"][0] >= 0]
        for x, before in zip(got[1:], (*c["codes"], *c["scales"])):
            assert np.array_equal(x[torch.from_numpy(kept).long().cuda()].cpu().numpy(), before[kept])


@pytest.mark.parametrize("rotary_dim,theta", [(8, 1e4), (56, 5e6), (128, 10.0), (64, 1.0)])
def test_insert_rotations(cuda_ok, rotary_dim, theta):
    c = _insert_case(22, ctx=[1 << 21, 200], nq=[3, 20], kv=1, rotary_dim=rotary_dim, theta=theta)
    _check_insert(c, _insert(c))
    assert msa.device_status() == msa.MSA_OK


def test_insert_scales_at_their_borders(cuda_ok):
    """Values of exactly 448 * 2^k keep the smaller scale; zeros take the least scale, or keep the page's."""
    T = 6
    c = _insert_case(23, ctx=[1, 1, 1, 60, 60, 60], nq=[1] * T, kv=1)
    c["v_new"] = torch.zeros(T, 1, 128, dtype=torch.bfloat16)
    c["v_new"][0, 0, 3], c["v_new"][1, 0, 3], c["v_new"][4, 0, 0], c["v_new"][5, 0, 0] = -3.5, 3.515625, 448 * 2.0 ** -4, -0.5
    pages = [int(c["table"][s, 0]) for s in range(T)]
    for s in (3, 4, 5):
        c["scales"][1][pages[s]] = 2.0 ** -4
    c["scales"][1][pages[5]] = 0.0                                            # not positive: counts as an empty page
    got = _insert(c)
    assert [float(got[4][p, 0]) for p in pages] == [2.0 ** -7, 2.0 ** -6, 2.0 ** -126, 2.0 ** -4, 2.0 ** -4, 2.0 ** -9]
    assert not (got[2][pages[5], 0, :59] & 0x7F).any() and got[2][pages[2], 0, 0].eq(0).all()
    _check_insert(c, got)
    assert msa.device_status() == msa.MSA_OK


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -1.0, 1e-42])
def test_insert_where_the_old_scale_holds_nothing(cuda_ok, scale):
    """A scale that is no positive number (a denormal one counts as 0): the page's earlier codes become 0."""
    c = _insert_case(27, ctx=[40, 77], nq=[4, 2], kv=1)
    page = int(c["table"][0, 0])
    for s in c["scales"]:
        s[page] = scale
    got = _insert(c)
    assert msa.device_status() == msa.MSA_OK
    for codes, scales, new in ((got[1], got[3], c["k_new"]), (got[2], got[4], c["v_new"])):
        assert not (codes[page, 0, :36] & 0x7F).any() and (codes[page, 0, 36:40] & 0x7F).any()
        assert 448 * float(scales[page, 0]) >= 1e-3 and np.isfinite(float(scales[page, 0]))
    assert float(got[4][page, 0]) == K.block_scale(float(c["v_new"][:4].abs().max()))


def test_insert_of_infinities_and_nan(cuda_ok):
    """An infinity saturates and a NaN stays NaN; neither moves the page's scale."""
    c = _insert_case(24, ctx=[40], nq=[4], kv=1)
    plain = _insert(c)
    c["v_new"][1, 0, 5], c["v_new"][2, 0, 6], c["v_new"][3, 0, 7] = float("inf"), float("-inf"), float("nan")
    got = _insert(c)
    assert msa.device_status() == msa.MSA_OK
    assert torch.equal(got[4], plain[4])
    page = int(c["table"][0, 0])
    assert [int(got[2][page, 0, 36 + i, 4 + i]) for i in (1, 2)] == [0x7E, 0xFE] and int(got[2][page, 0, 39, 7]) & 0x7F == 0x7F
    same = got[2] == plain[2]
    assert int((~same).sum()) <= 3


def test_insert_records_bad_pages(cuda_ok):
    c = _insert_case(25, ctx=[300, 50], nq=[200, 1], kv=2)
    table = c["table"].copy()
    lost = int(table[0, 1])
    table[0, 1] = c["batch"].num_pages
    c["batch"].page_table = torch.from_numpy(table).cuda()
    got = _insert(c)
    assert msa.device_status() == msa.MSA_ERR_DEVICE_BOUNDS
    for x, before in zip(got[1:], (*c["codes"], *c["scales"])):
        assert np.array_equal(x[lost].cpu().numpy(), before[lost])
    assert (got[0] != 7.0).any(dim=-1).all()                                   # the queries are written all the same


def test_insert_step_by_step_stays_near_inserting_at_once(cuda_ok):
    """128 single-token inserts into one page: the scale grows with the largest token so far, every code stays within
    one rounding of its value (two below the normal range), and the scale ends where inserting at once puts it."""
    rng = np.random.default_rng(5)
    size = torch.from_numpy(2.0 ** np.linspace(-4, 4, 128)[rng.permutation(128)]).view(128, 1, 1)
    whole = _insert_case(26, ctx=[128], nq=[128], kv=1, magnitude=size)
    k, v = (torch.from_numpy(x).cuda() for x in whole["codes"])
    ks, vs = (torch.from_numpy(x).cuda() for x in whole["scales"])
    q_out = torch.empty(1, 16, 128, dtype=torch.bfloat16, device="cuda")
    for t in range(128):
        b = msa.Batch.make([0, 1], [t + 1], whole["table"], whole["batch"].num_pages)
        msa.qknorm_rope_insert_fp8(whole["cfg"], b, whole["q"][t:t + 1].cuda(), whole["k_new"][t:t + 1].cuda(),
                                   whole["v_new"][t:t + 1].cuda(), whole["qw"].cuda(), whole["kw"].cuda(), q_out, k, v, ks, vs)
    at_once = _insert(whole)
    assert msa.device_status() == msa.MSA_OK
    page = int(whole["table"][0, 0])
    assert torch.equal(ks[page], at_once[3][page]) and torch.equal(vs[page], at_once[4][page])
    y = whole["v_new"][:, 0].double().numpy()
    got = F.decode_bits(v[page, 0].cpu().numpy()) * float(vs[page, 0])
    # a first rounding by 2^-4 |y|, or 2^-10 of a scale no larger than the last; at most one more of 2^-10 of each larger scale
    assert (np.abs(got - y) <= 2.0 ** -4 * np.abs(y) + 2 * 2.0 ** -10 * float(vs[page, 0])).all()


# ----------------------------------------------------------------- advance
def _advance(delta, ctx, table, ring, pool, max_rows, in_place=False, stream=None):
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    n = len(ctx)
    ctx_d, table_d, ring_d, pool_d = dev(ctx), dev(table), dev(ring), dev(pool)
    ctx_o = ctx_d if in_place else torch.full((n,), -5, dtype=torch.int32, device="cuda")
    pool_o = pool_d if in_place else torch.full((4,), -5, dtype=torch.int32, device="cuda")
    q_start = torch.full((n + 1,), -5, dtype=torch.int32, device="cuda")
    slots = torch.full((max_rows,), -5, dtype=torch.int32, device="cuda") if max_rows else None
    msa.advance_batch(dev(delta), ctx_d, table_d, ring_d, pool_d, ctx_o, pool_o, q_start, slots, stream=stream)
    torch.cuda.synchronize()
    return [x.tolist() if x is not None else [] for x in (ctx_o, table_d, ring_d, pool_o, q_start, slots)]


def _pool_case(seed, ctx, delta, spare=4):
    rng = np.random.default_rng(seed)
    have = [-(-c // 128) for c in ctx]
    want = [-(-max(0, c + d) // 128) for c, d in zip(ctx, delta)]
    width = max(1, *have, *want)
    need = sum(max(0, w - h) for h, w in zip(have, want))
    pages = sum(have) + need + spare
    perm = rng.permutation(pages).tolist()
    table, at = [], 0
    for h in have:
        table.append(perm[at:at + h] + [-1] * (width - h))
        at += h
    free = perm[at:]
    head = int(rng.integers(0, pages))
    ring = [-1] * pages
    for i, p in enumerate(free):
        ring[(head + i) % pages] = p
    return table, ring, [head, len(free), 0, 0]


def _mixed(seed, n, hi, new):
    rng = np.random.default_rng(seed)
    ctx = [int(x) for x in np.exp(rng.uniform(0, np.log(hi), size=n))]
    delta = [int(rng.integers(-c, 0)) if r < 0.15 else -c if r < 0.25 else 0 if r < 0.35 else int(rng.integers(1, new + 1))
             for c, r in zip(ctx, rng.uniform(size=n))]
    return ctx, delta


ADVANCES = {
    "one token": ([5000], [1]),
    "first tokens": ([0, 0, 0], [1, 128, 129]),
    "page borders": ([127, 128, 129, 255, 256, 1], [1, 1, -1, 2, -1, -1]),
    "all end": ([500, 1, 128], [-500, -1, -128]),
    "nothing": ([7, 0], [0, 0]),
    "mixed 40": _mixed(1, 40, 5000, 5),
    "mixed 1025": _mixed(2, 1025, 3000, 40),
    "mixed 8192": _mixed(3, 8192, 500, 3),
    "a long prompt": ([0, 300], [100001, 1]),
}


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("shape", ADVANCES)
def test_advance_matches_oracle(cuda_ok, shape, in_place):
    ctx, delta = ADVANCES[shape]
    table, ring, pool = _pool_case(9, ctx, delta)
    rows = sum(d for d in delta if d > 0) + 3
    got = _advance(delta, ctx, table, ring, pool, rows, in_place)
    assert msa.device_status() == msa.MSA_OK
    for name, a, b in zip(("ctx", "table", "ring", "pool", "q_start", "slots"), got, K.advance(delta, ctx, table, ring, pool, rows)):
        assert a == b, name
    assert _advance(delta, ctx, table, ring, pool, 0)[:5] == got[:5]          # without a slot map


@pytest.mark.parametrize("what", ["short of pages", "negative length", "too long", "too many rows", "bad head", "overfull"])
def test_advance_that_does_not_fit_changes_nothing(cuda_ok, what):
    ctx, delta = _mixed(4, 30, 4000, 200)
    table, ring, pool = _pool_case(10, ctx, delta, spare=0)
    rows = sum(d for d in delta if d > 0)
    if what == "short of pages":
        pool[1] -= 2
    elif what == "negative length":
        delta[3] = -ctx[3] - 1
    elif what == "too long":
        delta[5] = len(table[0]) * 128 - ctx[5] + 1
        rows += delta[5]
    elif what == "too many rows":
        rows -= 1
    elif what == "bad head":
        pool[0] = len(ring)
    else:
        pool[1] = len(ring)
    got = _advance(delta, ctx, table, ring, pool, rows)
    want = K.advance(delta, ctx, table, ring, pool, rows)
    for name, a, b in zip(("ctx", "table", "ring", "pool", "q_start", "slots"), got, want):
        assert a == b, name
    assert got[3][2] == (2 if what == "short of pages" else -1)
    assert msa.device_status() == (msa.MSA_OK if what == "short of pages" else msa.MSA_ERR_DEVICE_BOUNDS)


def test_advance_steps_conserve_the_pages(cuda_ok):
    """Many steps in place: no page is lost or held twice, and the lengths are the sums of the deltas."""
    rng = np.random.default_rng(6)
    n, width, pages = 20, 12, 100
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    ctx, pool, ring = dev([0] * n), dev([0, pages, 0, 0]), dev(list(range(pages)))
    table, q_start = torch.full((n, width), -1, dtype=torch.int32, device="cuda"), dev([0] * (n + 1))
    host = [0] * n
    for step in range(60):
        delta = [int(rng.integers(-c, 1)) if c and rng.uniform() < 0.3 else int(rng.integers(0, min(300, width * 128 - c) + 1)) for c in host]
        msa.advance_batch(dev(delta), ctx, table, ring, pool, ctx, pool, q_start)
        head, count, missing, rows = pool.tolist()
        if missing == 0:
            host = [c + d for c, d in zip(host, delta)]
        assert missing >= 0 and ctx.tolist() == host
        held = [p for r, c in zip(table.tolist(), host) for p in r[:-(-c // 128)]]
        free = [ring.tolist()[(head + i) % pages] for i in range(count)]
        assert sorted(held + free) == list(range(pages))
    assert msa.device_status() == msa.MSA_OK


# ----------------------------------------------------------------- together
def test_a_captured_decode_step(cuda_ok):
    """advance, insert and attention of a decode step as one graph, replayed over page borders: what the calls one by one
    give, bit for bit."""
    rng = np.random.default_rng(8)
    kv, topk, width, n = 2, 4, 4, 5
    pages = n * width
    cfg = msa.Config(num_q_heads=16 * kv, num_kv_heads=kv, idx_heads=kv, topk=topk)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    host = [126, 127, 128, 255, 1]
    table = np.full((n, width), -1)
    perm, at = rng.permutation(pages), 0
    for s, c in enumerate(host):
        for b in range(-(-c // 128)):
            table[s, b] = perm[at]
            at += 1

    def state():
        ring = [-1] * pages
        for i, p in enumerate(perm[at:].tolist()):
            ring[(pages - 2 + i) % pages] = p
        st = dict(ctx=dev(host), pool=dev([pages - 2, pages - at, 0, 0]), ring=dev(ring), table=dev(table.tolist()),
                  q_start=dev([0] * (n + 1)), slots=dev([0] * n), delta=dev([1] * n))
        g = torch.Generator(device="cuda").manual_seed(3)
        st["kc"], st["vc"] = (torch.randint(0, 127, (pages, kv, 128, 128), dtype=torch.uint8, device="cuda", generator=g) for _ in range(2))
        st["ks"], st["vs"] = (torch.full((pages, kv), 2.0 ** -8, device="cuda") for _ in range(2))
        st["q"], st["kn"], st["vn"] = (torch.zeros(n, h, 128, dtype=torch.bfloat16, device="cuda") for h in (16 * kv, kv, kv))
        st["qo"], st["out"] = torch.empty_like(st["q"]), torch.empty_like(st["q"])
        st["lse"] = torch.empty(n, 16 * kv, device="cuda")
        st["sel"] = torch.full((n, kv, topk), -1, dtype=torch.int32, device="cuda")
        st["batch"] = msa.Batch(q_start=st["q_start"], ctx_len=st["ctx"], page_table=st["table"], total_q=n, max_q_per_seq=1,
                                num_pages=pages)
        st["ws"] = torch.empty(msa.decode_fp8_workspace_bytes(cfg, st["batch"]), dtype=torch.uint8, device="cuda")
        return st

    weight = torch.ones(128, dtype=torch.bfloat16, device="cuda")

    def step(st):
        msa.advance_batch(st["delta"], st["ctx"], st["table"], st["ring"], st["pool"], st["ctx"], st["pool"], st["q_start"], st["slots"])
        msa.qknorm_rope_insert_fp8(cfg, st["batch"], st["q"], st["kn"], st["vn"], weight, weight, st["qo"], st["kc"], st["vc"], st["ks"], st["vs"])
        msa.attn_decode_fp8(cfg, st["batch"], st["qo"], st["kc"], st["vc"], st["ks"], st["vs"], st["sel"], st["out"], st["lse"], st["ws"])

    def feed(st, turn):
        g = torch.Generator(device="cuda").manual_seed(100 + turn)
        for name in ("q", "kn", "vn"):
            st[name].copy_(torch.randn(st[name].shape, generator=g, device="cuda"))
        for s, c in enumerate(host):
            cur = (c + turn) // 128
            st["sel"][s, :, :cur + 1] = torch.arange(cur + 1, dtype=torch.int32, device="cuda")

    a, b = state(), state()
    warm = state()
    feed(warm, 0)
    step(warm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a)
    for turn in range(5):
        feed(a, turn)
        feed(b, turn)
        graph.replay()
        step(b)
        for name in ("out", "lse", "kc", "vc", "ks", "vs", "ctx", "pool", "table", "ring", "slots"):
            assert torch.equal(a[name], b[name]), (turn, name)
    assert msa.device_status() == msa.MSA_OK and a["pool"].tolist()[2] == 0
    assert a["ctx"].tolist() == [c + 5 for c in host]


def test_a_served_batch_step_by_step(cuda_ok):
    """advance -> insert -> attention over a prefill, a mixed chunk, decode steps and a rollback, with every block
    selected: the attention is the dense causal one over the tokens that the cache holds."""
    rng = np.random.default_rng(7)
    kv, topk, width, pages, n = 2, 6, 6, 20, 3
    cfg = msa.Config(num_q_heads=16 * kv, num_kv_heads=kv, idx_heads=kv, topk=topk)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    ctx, pool, ring = dev([0] * n), dev([3, pages, 0, 0]), dev(rng.permutation(pages).tolist())
    table, q_start = torch.full((n, width), -1, dtype=torch.int32, device="cuda"), dev([0] * (n + 1))
    k, v = (torch.randint(0, 256, (pages, kv, 128, 128), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((pages, kv), float("nan"), device="cuda") for _ in range(2))
    bf = lambda *s: torch.from_numpy(rng.normal(size=s)).to(torch.bfloat16).cuda()  # noqa: E731
    wq, wk = (1 + 0.1 * bf(128).float()).to(torch.bfloat16), (1 + 0.1 * bf(128).float()).to(torch.bfloat16)
    host = [0] * n
    for delta in ([200, 0, 130], [1, 57, 127], [1, 1, 1], [4, 4, 4], [-3, 4, -261], [1, 100, 300], [1, 1, 1]):
        host = [c + d for c, d in zip(host, delta)]
        new = [max(0, d) for d in delta]
        rows = sum(new)
        slots = dev([0] * rows)
        msa.advance_batch(dev(delta), ctx, table, ring, pool, ctx, pool, q_start, slots)
        batch = msa.Batch(q_start=q_start, ctx_len=ctx, page_table=table, total_q=rows, max_q_per_seq=max(new), num_pages=pages)
        q, kn, vn = bf(rows, 16 * kv, 128), bf(rows, kv, 128), bf(rows, kv, 128)
        msa.qknorm_rope_insert_fp8(cfg, batch, q, kn, vn, wq, wk, q, k, v, ks, vs)
        seq = np.repeat(np.arange(n), new)
        pos = np.concatenate([np.arange(c - d, c) for c, d in zip(host, new)])
        assert slots.tolist() == [int(table[s, p // 128]) * 128 + int(p % 128) for s, p in zip(seq, pos)]
        sel = np.full((rows, kv, topk), -1, dtype=np.int32)
        for t, p in enumerate(pos):
            sel[t, :, :p // 128 + 1] = np.arange(p // 128 + 1)
        which = "decode" if max(new) <= 8 else "prefill"
        out, lse = torch.empty_like(q), torch.empty(rows, 16 * kv, device="cuda")
        ws = torch.empty(WORKSPACE[which](cfg, batch), dtype=torch.uint8, device="cuda")
        ATTN[which](cfg, batch, q, k, v, ks, vs, torch.from_numpy(sel).cuda(), out, lse, ws)
        assert msa.device_status() == msa.MSA_OK and pool.tolist()[2] == 0
        kc, vc = (K.values(x.cpu().numpy(), y.cpu().numpy()) for x, y in ((k, ks), (v, vs)))
        ref, ref_lse, mag = K.attention(q.double().cpu().numpy(), kc, vc, seq, pos, sel, table.cpu().numpy())
        err = np.abs(out.double().cpu().numpy() - ref)
        assert (err <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -7 + 2.0 ** -12) * mag).all(), delta
        assert np.abs(lse.cpu().numpy() - ref_lse).max() <= LSE_ABS
        # the new values are in the cache, one rounding away
        page, slot = np.array(slots.tolist()) // 128, np.array(slots.tolist()) % 128
        got = vc[page, :, slot]
        want = vn.double().cpu().numpy()
        assert (np.abs(got - want) <= 2.0 ** -4 * np.abs(want) + 2.0 ** -10 * vs.cpu().numpy()[page][..., None]).all()
