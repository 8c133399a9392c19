"""qknorm_paged_attend on the GPU against the float64 oracle: decode and
prompts, head widths and groups, splits, windows, empty and masked rows, pages
that end inside a tile, NaN in masked places, strides and stale rows.

Tolerance, per output: the result's rounding to bf16, 2^-8 |o|; the
probabilities' rounding to bf16, 2^-8 sum p |v|; float32 scores of up to 256
products within (256 + 8) 2^-24 of sum |q k| scale (at most ~60 here, so
2 * 60 * 264 * 2^-24 < 2^-9 relative in p, counted with the sums' own
rounding as another 2^-8 sum p |v|).
"""

import numpy as np
import pytest
import torch

import layerwise_qk_norm_qknorm_amd as qk
import operator_cases as C
from oracle import operators as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qk.load_library()
    yield
    torch.cuda.synchronize()


class Case:
    """lens and n_q per sequence; pages handed out in random order; what no sequence
    holds is random bytes, NaN scales among them."""

    def __init__(self, seed, d, heads_q, heads_k, lens, n_q, ps=16, spare=3, extra_rows=0):
        r = C.rng(seed)
        self.d, self.hq, self.hk, self.lens, self.n_q, self.ps = d, heads_q, heads_k, lens, n_q, ps
        need = [-(-n // ps) for n in lens]
        pages = sum(need) + spare
        ids = r.permutation(pages)
        width = max(need + [1]) + 1
        self.table = r.integers(-5, pages + 5, (len(lens), width)).astype(np.int32)    # unused entries: anything
        self.codes = [r.integers(0, 256, (pages, heads_k, ps, d // 2), dtype=np.uint8) for _ in range(2)]
        self.scales = [r.integers(0, 256, (pages, heads_k, ps, d // 32), dtype=np.uint8) for _ in range(2)]
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            for j in range(n):
                tokens = min(ps, lens[b] - j * ps)
                for i in range(2):
                    c, s, _ = O.mxfp4_quantize(r.normal(size=(heads_k, tokens, d)))
                    self.codes[i][ids[at + j], :, :tokens], self.scales[i][ids[at + j], :, :tokens] = c, s
            at += n
        rows = sum(n_q)
        self.q = C.to_type(r.normal(size=(rows + extra_rows, heads_q * d)) * 1.5, "bf16")
        self.cu = np.concatenate(([0], np.cumsum(n_q))).astype(np.int32)

    def cached(self, b):
        out = []
        for i in range(2):
            x = O.mxfp4_values(self.codes[i][self.table[b, :-(-self.lens[b] // self.ps)]],
                               self.scales[i][self.table[b, :-(-self.lens[b] // self.ps)]])
            out.append(x.transpose(0, 2, 1, 3).reshape(-1, self.hk, self.d)[:self.lens[b]])
        return out

    def run(self, cu=True, **kw):
        out = torch.full((self.q.shape[0], self.hq * self.d), 3.0, dtype=torch.bfloat16, device="cuda")
        t = [torch.from_numpy(x).cuda() for x in self.codes + self.scales]
        qk.qknorm_paged_attend(C.dev(self.q), *t, C.dev(self.table), C.dev(np.array(self.lens, np.int32)), self.d,
                               cu_q=C.dev(self.cu) if cu else None, out=out, **kw)
        torch.cuda.synchronize()
        return out

    def check(self, out, causal=True, window=0, scale=None, skip=()):
        got = C.host_values(out).reshape(-1, self.hq, self.d)
        q = C.values(self.q).reshape(-1, self.hq, self.d)
        for b in range(len(self.lens)):
            if b in skip:
                continue
            rows = slice(self.cu[b], self.cu[b + 1])
            K, V = self.cached(b)
            want, mag, some = O.attend(q[rows], K, V, self.n_q[b], scale or self.d ** -0.5, causal, window)
            assert not got[rows][~some].any()
            C.close(got[rows], want, 2.0 ** -8 * np.abs(want) + 2.0 ** -7 * mag + 2.0 ** -134, f"sequence {b}")
        assert (got[self.cu[-1]:] == 3.0).all()      # rows behind the last sequence


# head_dim, query heads, key heads, lengths, query counts, page size
CASES = [
    (128, 5, 1, [1], [1], 16),
    (128, 40, 8, [333, 16, 17, 0, 4097], [1] * 5, 16),
    (64, 8, 2, [100, 31, 32, 33, 64], [1] * 5, 32),
    (256, 8, 4, [50, 700], [1, 1], 64),
    (128, 32, 32, [129, 255], [1, 1], 128),
    (128, 17, 1, [500], [1], 16),                 # 17 rows: two row tiles
    (64, 40, 1, [300, 700], [1, 1], 16),          # 40 rows: three of four
    (256, 20, 1, [300], [1], 16),
    (128, 64, 1, [40], [1], 16),
    (64, 100, 1, [40], [1], 16),                  # more rows than one block takes
    (128, 10, 2, [5, 60, 33], [5, 3, 7], 16),
    (128, 4, 2, [100, 3, 10, 70], [100, 3, 4, 0], 32),
    (64, 6, 3, [90, 257], [90, 130], 16),
    (256, 4, 2, [120, 50], [50, 50], 32),
    (128, 8, 8, [2, 0], [5, 2], 16),              # more queries than cached tokens
]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 13), (False, 0), (False, 40)])
def test_against_the_oracle(case, causal, window):
    print(f"[case] attend {case} causal={causal} window={window}", flush=True)
    d, hq, hk, lens, n_q, ps = case
    c = Case(41, d, hq, hk, lens, n_q, ps, extra_rows=3)
    c.check(c.run(causal=causal, window=window, max_q=max(max(n_q), 1), max_len=max(lens + [1])), causal, window)


def test_decode_without_row_offsets_and_with_another_scale():
    c = Case(43, 128, 16, 4, [77, 1, 300], [1, 1, 1])
    a = c.run(cu=False)
    b = c.run(cu=True)
    assert C.same_bits(a, b)
    c.check(c.run(cu=False, scale=0.31), scale=0.31)


@pytest.mark.parametrize("d,hq,hk", [(128, 5, 1), (64, 8, 1), (256, 2, 1), (128, 24, 1)])
def test_one_long_sequence_is_split(d, hq, hk):
    print(f"[case] attend split {d} {hq} {hk}", flush=True)
    c = Case(47, d, hq, hk, [9000], [1], 64)
    assert qk.load_library().qknorm_paged_attend_workspace(1, hq, hk, d, 1, 1, 9000) > 0
    c.check(c.run())
    c.check(c.run(window=2500), window=2500)
    c.check(c.run(window=100), window=100)       # one chunk of it is left


def test_bounds_below_the_truth_stay_correct():
    """max_q and max_len shape the launch; longer sequences only take longer."""
    c = Case(53, 128, 8, 2, [2000, 700], [70, 9], 16)
    c.check(c.run(max_q=1, max_len=64))
    c.check(c.run(max_q=3, max_len=600))
    c.check(c.run(max_q=4000, max_len=1 << 29))
    c = Case(53, 128, 8, 2, [5000, 700, 3000], [1] * 3, 16)
    c.check(c.run(max_len=513))


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_nan_blocks_reach_only_the_rows_that_see_them(which, d):
    """A NaN block of K makes the rows that see its token NaN (every column: the whole score is
    NaN), one of V its 32 columns of those rows."""
    lens, n_q, tok = [70], [40], 50
    c = Case(59, d, 4, 2, lens, n_q, 16, spare=1)
    clean = c.run()
    c.scales[which][c.table[0, tok // 16], 1, tok % 16, d // 32 - 1] = 255
    out = c.run().float().cpu().numpy().reshape(-1, 4, d)
    want = clean.float().cpu().numpy().reshape(-1, 4, d).copy()
    first = tok - (lens[0] - n_q[0])                # queries from here on see the token
    want[first:, 2:, (0 if which == 0 else d - 32):] = np.nan
    assert np.array_equal(np.isnan(out), np.isnan(want))
    ok = ~np.isnan(want)
    assert np.array_equal(out[ok], want[ok])
    # a window that has left the token behind
    out = c.run(window=5).float().cpu().numpy().reshape(-1, 4, d)
    sees = np.zeros(out.shape, bool)
    sees[first:first + 5, 2:, (0 if which == 0 else d - 32):] = True
    assert np.array_equal(np.isnan(out), sees)


def test_a_page_that_does_not_exist_is_loud():
    c = Case(61, 128, 4, 2, [100, 60], [1, 1], 16)
    good = c.run()
    for bad in (-1, 1 << 20):
        keep = c.table[0, 2]
        c.table[0, 2] = bad
        out = c.run()
        c.table[0, 2] = keep
        assert torch.isnan(out[0]).all()
        assert C.same_bits(out[1], good[1])


def test_a_query_that_is_not_finite_stays_in_its_row():
    c = Case(67, 128, 8, 2, [100, 60], [4, 4], 16)
    good = c.run()
    q = C.dev(c.q)
    q[2, 130] = float("nan")
    c.q = C.torch_to_np(q)
    out = c.run()
    bad = torch.zeros(out.shape, dtype=torch.bool, device="cuda")
    bad[2, 128:256] = True
    assert torch.equal(torch.isnan(out), bad)
    assert torch.equal(out[~bad], good[~bad])


def test_strided_rows_and_page_strides():
    c = Case(71, 64, 6, 2, [90, 33], [3, 1], 32)
    want = c.run()
    q = C.dev(c.q)
    wide = torch.zeros((q.shape[0], 6 * 64 + 40), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + 384] = q
    out = torch.full((q.shape[0], 6 * 64 + 24), 3.0, dtype=torch.bfloat16, device="cuda")
    pages = c.codes[0].shape[0]
    both = torch.zeros((pages, 2, 2, 32, 32), dtype=torch.uint8, device="cuda")        # K and V share pages
    sc = torch.zeros((pages, 2, 2, 32, 2), dtype=torch.uint8, device="cuda")
    for i in range(2):
        both[:, i], sc[:, i] = torch.from_numpy(c.codes[i]).cuda(), torch.from_numpy(c.scales[i]).cuda()
    qk.qknorm_paged_attend(wide[:, 8:8 + 384], both[:, 0], both[:, 1], sc[:, 0], sc[:, 1], C.dev(c.table),
                           C.dev(np.array(c.lens, np.int32)), 64, cu_q=C.dev(c.cu), out=out[:, 16:400])
    torch.cuda.synchronize()
    assert C.same_bits(out[:, 16:400], want)
    assert (out[:, :16] == 3.0).all() and (out[:, 400:] == 3.0).all()


def test_lengths_out_of_range_are_held():
    """A length past the table's pages counts as what the table holds, a negative one as empty."""
    c = Case(73, 128, 4, 1, [64, 64], [1, 1], 16, spare=0)
    c.table = np.ascontiguousarray(c.table[:, :4])
    good = c.run()
    c.lens = [1 << 30, -7]
    out = c.run()
    assert C.same_bits(out[0], good[0]) and not out[1].any()


def test_offsets_that_are_not_increasing_write_nothing_outside():
    c = Case(79, 128, 4, 1, [64, 64], [1, 1], 16, extra_rows=2)
    c.cu = np.array([2, 0, 99], np.int32)       # an empty range, then [0, T)
    out = c.run(max_q=4)
    assert torch.isfinite(out.float()).all()


def test_marshalling_refusals():
    c = Case(83, 128, 4, 2, [40], [1])
    t = [torch.from_numpy(x).cuda() for x in c.codes + c.scales]
    q, table, lens = C.dev(c.q), C.dev(c.table), C.dev(np.array([40], np.int32))
    for a in ((q, t[0], t[1], None, None, table, lens), (q, *t, table.long(), lens), (q, *t, table, lens.long()),
              (q, *t, table, lens.repeat(2)), (q, *t, table.cpu(), lens), (q, t[0], t[1], t[2], t[3][:1], table, lens)):
        with pytest.raises(ValueError):
            qk.qknorm_paged_attend(*a, 128)
    with pytest.raises(qk.QKNormError):
        qk.qknorm_paged_attend(q.float(), *t, table, lens, 128)
    with pytest.raises(qk.QKNormError):
        qk.qknorm_paged_attend(q, *t, table, lens, 128, scale=-1.0)
    with pytest.raises(qk.QKNormError):
        qk.qknorm_paged_attend(q.repeat(9, 1), *t, table.repeat(9, 600), lens.repeat(9), 128,
                               workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
