"""qknorm_paged_attend_wide on the GPU against the float64 oracle, over bf16 rows and MXFP8: single
tokens and prompts, head widths and groups, splits, windows, empty and masked rows, pages that end
inside a tile, infinities and NaN in masked places, strides, layouts and stale rows.

Tolerance, per output: the result's rounding to bf16, 2^-8 |o|; the probabilities' rounding to
bf16, 2^-8 sum p |v|; float32 scores of up to 256 products within (256 + 8) 2^-24 of sum |q k|
scale (at most ~60 here, so 2 * 60 * 264 * 2^-24 < 2^-9 relative in p, counted with the sums' own
rounding as another 2^-8 sum p |v|).
"""

import numpy as np
import pytest
import torch

import layerwise_qk_norm_qknorm_amd as qk
import operator_cases as C
from oracle import operators as O

pytestmark = pytest.mark.gpu
FORMATS = ["rows", "mxfp8"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qk.load_library()
    yield
    torch.cuda.synchronize()


class Case:
    """lens and n_q per sequence; pages handed out in random order; what no sequence holds is
    random bits, infinities and NaN among them."""

    def __init__(self, fmt, seed, d, heads_q, heads_k, lens, n_q, ps=16, spare=3, extra_rows=0):
        r = C.rng(seed)
        self.fmt, self.d, self.hq, self.hk, self.lens, self.n_q, self.ps = fmt, d, heads_q, heads_k, lens, n_q, ps
        need = [-(-n // ps) for n in lens]
        pages = sum(need) + spare
        ids = r.permutation(pages)
        width = max(need + [1]) + 1
        self.table = r.integers(-5, pages + 5, (len(lens), width)).astype(np.int32)    # unused entries: anything
        shape = (pages, heads_k, ps)
        if fmt == "rows":
            self.data = [r.integers(0, 1 << 16, shape + (d,), dtype=np.uint16) for _ in range(2)]
            self.scales = []
        else:
            self.data = [r.integers(0, 256, shape + (d,), dtype=np.uint8) for _ in range(2)]
            self.scales = [r.integers(0, 256, shape + (d // 32,), dtype=np.uint8) for _ in range(2)]
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            for j in range(n):
                tokens = min(ps, lens[b] - j * ps)
                for i in range(2):
                    x = r.normal(size=(heads_k, tokens, d))
                    if fmt == "rows":
                        self.data[i][ids[at + j], :, :tokens] = C.to_type(x, "bf16")
                    else:
                        c, s, _ = O.mxfp8_quantize(x)
                        self.data[i][ids[at + j], :, :tokens], self.scales[i][ids[at + j], :, :tokens] = c, s
            at += n
        rows = sum(n_q)
        self.q = C.to_type(r.normal(size=(rows + extra_rows, heads_q * d)) * 1.5, "bf16")
        self.cu = np.concatenate(([0], np.cumsum(n_q))).astype(np.int32)

    def cached(self, b):
        out = []
        for i in range(2):
            at = self.table[b, :-(-self.lens[b] // self.ps)]
            x = C.values(self.data[i][at]) if self.fmt == "rows" else O.mxfp8_values(self.data[i][at], self.scales[i][at])
            out.append(x.transpose(0, 2, 1, 3).reshape(-1, self.hk, self.d)[:self.lens[b]])
        return out

    def tensors(self):
        if self.fmt == "rows":
            return [C.dev(x) for x in self.data], {}
        s = [torch.from_numpy(x).cuda() for x in self.scales]
        return [torch.from_numpy(x).cuda() for x in self.data], dict(k_scales=s[0], v_scales=s[1])

    def run(self, cu=True, **kw):
        out = torch.full((self.q.shape[0], self.hq * self.d), 3.0, dtype=torch.bfloat16, device="cuda")
        cache, scales = self.tensors()
        qk.qknorm_paged_attend_wide(C.dev(self.q), *cache, C.dev(self.table), C.dev(np.array(self.lens, np.int32)),
                                    self.d, cu_q=C.dev(self.cu) if cu else None, out=out, **scales, **kw)
        torch.cuda.synchronize()
        return out

    def check(self, out, causal=True, window=0, scale=None):
        got = C.host_values(out).reshape(-1, self.hq, self.d)
        q = C.values(self.q).reshape(-1, self.hq, self.d)
        for b in range(len(self.lens)):
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
    (256, 20, 1, [300], [1], 16),
    (64, 40, 1, [300, 700], [1, 1], 16),          # 40 rows: each wave takes its own
    (128, 64, 1, [40], [1], 16),
    (64, 160, 1, [40], [1], 16),                  # more rows than one block of 128
    (128, 10, 2, [5, 60, 33], [5, 3, 7], 16),
    (128, 4, 2, [100, 3, 10, 70], [100, 3, 4, 0], 32),
    (64, 6, 3, [90, 257], [90, 130], 16),
    (256, 4, 2, [120, 50], [50, 50], 32),
    (128, 8, 8, [2, 0], [5, 2], 16),              # more queries than cached tokens
    (128, 5, 1, [190, 65, 64, 63], [66, 65, 1, 63], 16),
    (64, 5, 1, [300, 129], [300, 129], 64),       # 64 rows a wave
    (128, 14, 2, [200, 128], [100, 128], 32),
    (256, 5, 1, [140], [140], 128),
]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 13), (False, 0), (False, 40)])
def test_against_the_oracle(case, causal, window, fmt):
    print(f"[case] attend wide {fmt} {case} causal={causal} window={window}", flush=True)
    d, hq, hk, lens, n_q, ps = case
    c = Case(fmt, 41, d, hq, hk, lens, n_q, ps, extra_rows=3)
    c.check(c.run(causal=causal, window=window, max_q=max(max(n_q), 1), max_len=max(lens + [1])), causal, window)


@pytest.mark.parametrize("fmt", FORMATS)
def test_decode_without_row_offsets_and_with_another_scale(fmt):
    c = Case(fmt, 43, 128, 16, 4, [77, 1, 300], [1, 1, 1])
    a, b = c.run(cu=False), c.run(cu=True)
    assert C.same_bits(a, b)
    c.check(c.run(cu=False, scale=0.31), scale=0.31)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("d,hq,hk,n_q", [(128, 5, 1, 1), (64, 8, 1, 1), (256, 2, 1, 1), (128, 24, 1, 1), (128, 5, 1, 9),
                                         (64, 4, 1, 70), (256, 2, 1, 30)])
def test_one_long_sequence_is_split(d, hq, hk, n_q, fmt):
    print(f"[case] attend wide split {fmt} {d} {hq} {hk} {n_q}", flush=True)
    c = Case(fmt, 47, d, hq, hk, [9000], [n_q], 64)
    assert qk.load_library().qknorm_paged_attend_wide_workspace(n_q, hq, hk, d, 1, n_q, 9000) > 0
    c.check(c.run())
    c.check(c.run(window=2500), window=2500)
    c.check(c.run(window=100), window=100)       # one chunk of it is left


@pytest.mark.parametrize("fmt", FORMATS)
def test_bounds_below_the_truth_stay_correct(fmt):
    """max_q and max_len shape the launch; longer sequences only take longer."""
    c = Case(fmt, 53, 128, 8, 2, [2000, 700], [70, 9], 16)
    for kw in (dict(max_q=1, max_len=64), dict(max_q=3, max_len=600), dict(max_q=9, max_len=64),
               dict(max_q=4000, max_len=1 << 29), {}):
        c.check(c.run(**kw))
    c = Case(fmt, 53, 128, 8, 2, [5000, 700, 3000], [1] * 3, 16)
    c.check(c.run(max_len=513))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("d,n_q", [(64, 3), (128, 3), (256, 3), (64, 70), (128, 40), (128, 100), (256, 40)])
def test_nan_reaches_only_the_rows_that_see_it(which, d, n_q, fmt):
    """NaN in K makes the rows that see its token NaN (every column: the whole score is NaN), in V
    the columns it stands in (a code's or a scale's whole block)."""
    n = n_q + 30
    tok = n - n_q + n_q // 2
    c = Case(fmt, 59, d, 4, 2, [n], [n_q], 16, spare=1)
    clean = c.run()
    at = (c.table[0, tok // 16], 1, tok % 16)
    if fmt == "rows":
        c.data[which][at][d - 3] = 0x7FC0
        cols = [d - 3]
    elif d == 128:
        c.data[which][at][d - 3] = 0xFF           # a NaN code
        cols = [d - 3]
    else:
        c.scales[which][at][d // 32 - 1] = 247    # a NaN block
        cols = list(range(d - 32, d))
    sees = np.zeros((n_q, 4, d), bool)
    first = tok - (n - n_q)                       # queries from here on see the token
    sees[first:, 2:, slice(None) if which == 0 else cols] = True
    out = c.run().float().cpu().numpy().reshape(-1, 4, d)
    assert np.array_equal(np.isnan(out), sees)
    assert np.array_equal(out[~sees], clean.float().cpu().numpy().reshape(-1, 4, d)[~sees])
    # a window that leaves the token behind
    out = c.run(window=5).float().cpu().numpy().reshape(-1, 4, d)
    sees[first + 5:] = False
    assert np.array_equal(np.isnan(out), sees)


@pytest.mark.parametrize("n_q", [4, 50])
def test_infinite_values_reach_only_the_rows_that_see_them(n_q):
    n = n_q + 40
    c = Case("rows", 61, 128, 4, 2, [n], [n_q], 16, spare=1)
    clean = C.host_values(c.run()).reshape(-1, 4, 128)
    for tok, col, bits in ((n - 2, 7, 0x7F80), (n - 3, 9, 0xFF80), (n - 1, 11, 0x7F80), (n - 2, 11, 0xFF80)):
        c.data[1][c.table[0, tok // 16], 0, tok % 16, col] = bits
    out = C.host_values(c.run()).reshape(-1, 4, 128)
    want = clean.copy()
    want[n_q - 2:, :2, 7] = np.inf
    want[n_q - 3:, :2, 9] = -np.inf
    want[n_q - 2, :2, 11] = -np.inf
    want[n_q - 1, :2, 11] = np.nan
    assert np.array_equal(out, want, equal_nan=True)


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_page_that_does_not_exist_is_loud(fmt):
    for n_q in (1, 45):
        c = Case(fmt, 61, 128, 4, 2, [100, 60], [n_q, n_q], 16)
        good = c.run()
        for bad in (-1, 1 << 20):
            keep = c.table[0, 2]
            c.table[0, 2] = bad
            out = c.run()
            c.table[0, 2] = keep
            assert torch.isnan(out[:n_q]).all()
            assert C.same_bits(out[n_q:], good[n_q:])


@pytest.mark.parametrize("n_q", [4, 60])
def test_a_query_that_is_not_finite_stays_in_its_row(n_q):
    c = Case("rows", 67, 128, 8, 2, [100, 60], [n_q, 4], 16)
    good = c.run()
    q = C.dev(c.q)
    q[2, 130] = float("nan")
    c.q = C.torch_to_np(q)
    out = c.run()
    bad = torch.zeros(out.shape, dtype=torch.bool, device="cuda")
    bad[2, 128:256] = True
    assert torch.equal(torch.isnan(out), bad)
    assert torch.equal(out[~bad], good[~bad])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n_q", [2, 40])
def test_strided_rows_and_layouts_of_the_cache(n_q, fmt):
    c = Case(fmt, 71, 64, 6, 2, [90, 33], [n_q, 1], 32)
    want = c.run()
    q = C.dev(c.q)
    wide = torch.zeros((q.shape[0], 6 * 64 + 40), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + 384] = q
    cache, scales = c.tensors()
    pages = cache[0].shape[0]
    one = torch.zeros((pages, 2, 2, 32, 64), dtype=cache[0].dtype, device="cuda")       # K and V share pages
    mixed = torch.zeros((pages, 32, 2, 64 + 16), dtype=cache[0].dtype, device="cuda")   # tokens first, padded
    for layout in ("one allocation", "tokens first"):
        views = []
        for i in range(2):
            if layout == "one allocation":
                one[:, i] = cache[i]
                views.append(one[:, i])
            else:
                own = mixed.clone()
                own[..., :64] = cache[i].transpose(1, 2)
                views.append(own[..., :64].transpose(1, 2))
        out = torch.full((q.shape[0], 6 * 64 + 24), 3.0, dtype=torch.bfloat16, device="cuda")
        qk.qknorm_paged_attend_wide(wide[:, 8:8 + 384], *views, C.dev(c.table), C.dev(np.array(c.lens, np.int32)), 64,
                                    cu_q=C.dev(c.cu), out=out[:, 16:400], **scales)
        torch.cuda.synchronize()
        assert C.same_bits(out[:, 16:400], want), layout
        assert (out[:, :16] == 3.0).all() and (out[:, 400:] == 3.0).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n_q", [1, 50])
def test_lengths_out_of_range_are_held(n_q, fmt):
    """A length past the table's pages counts as what the table holds, a negative one as empty."""
    c = Case(fmt, 73, 128, 4, 1, [64, 64], [n_q, n_q], 16, spare=0)
    c.table = np.ascontiguousarray(c.table[:, :4])
    good = c.run()
    c.lens = [1 << 30, -7]
    out = c.run()
    assert C.same_bits(out[:n_q], good[:n_q]) and not out[n_q:].any()


def test_offsets_that_are_not_increasing_write_nothing_outside():
    c = Case("rows", 79, 128, 4, 1, [64, 64], [1, 1], 16, extra_rows=2)
    c.cu = np.array([2, 0, 99], np.int32)       # an empty range, then [0, T)
    for max_q in (4, 40):
        assert torch.isfinite(c.run(max_q=max_q).float()).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n_q", [1, 60])
def test_scores_far_from_zero(n_q, fmt):
    """Scores around +-1e4: the running maximum follows them; a float32 score is off by up to 136
    2^-24 of its products' magnitudes, about 0.1 here, so only rows with a clear largest score are
    compared: those whose second score is 4 below weigh 1 : e^-4 at worst."""
    c = Case(fmt, 89, 128, 4, 2, [300], [n_q], 16)
    for sign in (1.0, -1.0):
        c.q = C.to_type(sign * 600 * C.values(c.q) / np.abs(C.values(c.q)).max(), "bf16")
        out = C.host_values(c.run(scale=1.0)).reshape(-1, 4, 128)
        K, V = c.cached(0)
        q = C.values(c.q).reshape(-1, 4, 128)
        seen = 0
        for i in range(n_q):
            for h in range(4):
                hi = 300 - n_q + i + 1
                s = K[:hi, h // 2] @ q[i, h]
                order = np.argsort(s)
                if s[order[-1]] - s[order[-2]] < 20:
                    continue
                seen += 1
                v = V[order[-1], h // 2]
                assert np.abs(out[i, h] - v).max() <= 2.0 ** -7 * np.abs(V[:hi, h // 2]).max()
        assert seen > 0


def test_marshalling_refusals():
    c = Case("mxfp8", 83, 128, 4, 2, [40], [1])
    cache, s = c.tensors()
    rows = [torch.zeros(x.shape, dtype=torch.bfloat16, device="cuda") for x in cache]
    q, table, lens = C.dev(c.q), C.dev(c.table), C.dev(np.array([40], np.int32))
    for a, kw in (((q, *cache, table, lens), {}), ((q, *cache, table, lens), dict(k_scales=s["k_scales"])),
                  ((q, *rows, table.long(), lens), {}), ((q, *rows, table, lens.long()), {}),
                  ((q, *rows, table, lens.repeat(2)), {}), ((q, *rows, table.cpu(), lens), {}),
                  ((q, rows[0].float(), rows[1].float(), table, lens), {}), ((q, *rows, table, lens), s),
                  ((q, rows[0], rows[1][:1], table, lens), {}), ((q.cpu(), *rows, table, lens), {})):
        with pytest.raises(ValueError):
            qk.qknorm_paged_attend_wide(*a, 128, **kw)
    four = [torch.zeros((*x.shape[:3], 64), dtype=torch.uint8, device="cuda") for x in cache]
    for a, kw in (((q.float(), *rows, table, lens), {}), ((q, *rows, table, lens), dict(scale=-1.0)),
                  ((q, *four, table, lens), s),
                  ((q.repeat(9, 1), *rows, table.repeat(9, 600), lens.repeat(9)),
                   dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")))):
        with pytest.raises(qk.QKNormError):
            qk.qknorm_paged_attend_wide(*a, 128, **kw)
