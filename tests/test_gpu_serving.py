"""The paged-cache step on the GPU: plan, append, attention over a shared prefix and own pages.

Plan and append move whole numbers and bits, so they have to equal the oracle's.  Attention is held,
element by element, to a bound derived before the first run.  With u = 2^-8, the largest relative
rounding of a bf16 number (half a step), w_j a row's exact weights and d the head size:

* O is rounded to bf16: half a step at |O|;
* the weights are rounded to bf16 before the product with V and O is divided by the sum of the rounded
  weights: at most u / (1 - u) * sum_j w_j |v_j - O|, which is at most u / (1 - u) times the row's
  spread sqrt(sum_j w_j (v_j - O)^2) (the weights sum to 1);
* a score is a sum of d exact products in fp32, each addition off by at most 2^-23 of the sum of the
  magnitudes (whether it rounds or truncates), so by ds = d * 2^-23 * size, size = the row's largest
  scale * sum_c |q_c k_jc|; it is then scaled and the reference maximum subtracted in one fused step
  (2^-23 of size): every weight is off by a factor e^(+-ds), the quotient by at most twice that;
* the exponentials, the sums over keys and the join of the parts in fp32: 2^-16 of the spread and of |O|.

LSE: ds as above, twice the exponential's 2^-22, and 2^-22 of the magnitudes of m and LSE for the
logarithm, the products with ln 2 and the join of the parts.
"""
import math

import numpy as np
import pytest

import fa_inputs as fi
from oracle import paged
from parity import bf16_to_f64, bf16_ulp, to_device

pytestmark = pytest.mark.gpu

NAN_BITS, INF_BITS = 0x7FC0, 0x7F80


@pytest.fixture(scope="module", autouse=True)
def _library():
    import torch

    import exact_io_aware_07_gb300 as fa

    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    fa.build()
    fa.load_library()
    fa.fa_device_status()


def bits(x):
    return fi.f32_to_bf16_bits(np.asarray(x, dtype=np.float32))


def pages_of(n):
    return (n + 127) // 128


class Batch:
    """Random pools, tables and rows of one attention call; page tails and unused pages hold NaN and infinities."""

    def __init__(self, d, H, Hkv, prefix, own, new, pad=0, seed=0, sigma=1.0, spare=2, extra_cols=1):
        rng = np.random.default_rng([seed, d, H, Hkv, prefix, len(own), sum(own)])
        self.d, self.H, self.Hkv, self.prefix, self.own, self.new = d, H, Hkv, prefix, list(own), list(new)
        B = len(own)
        count = pages_of(prefix) + sum(pages_of(n) for n in own) + spare
        order = rng.permutation(count)
        self.k = np.empty((count, Hkv, 128, d), dtype=np.uint16)
        self.v = np.empty_like(self.k)
        for x in (self.k, self.v):
            x[:] = np.where(rng.random((count, 1, 128, 1)) < 0.5, NAN_BITS, INF_BITS).astype(np.uint16)
        self.max_pages = max([1] + [pages_of(n) for n in own]) + extra_cols
        self.table = np.full((B, self.max_pages), -9, dtype=np.int32)
        self.prefix_table = np.full(pages_of(prefix) + 1, -3, dtype=np.int32)
        at = 0

        def fill(row, n):
            nonlocal at
            for i in range(pages_of(n)):
                pg = row[i] = order[at]
                at += 1
                m = min(128, n - 128 * i)
                self.k[pg, :, :m] = bits(sigma * rng.standard_normal((Hkv, m, d)))
                self.v[pg, :, :m] = bits(rng.standard_normal((Hkv, m, d)))

        fill(self.prefix_table, prefix)
        for b, n in enumerate(own):
            fill(self.table[b], n)
        self.seq = np.array(own, dtype=np.int32)
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.q = bits(sigma * rng.standard_normal((int(self.cu[-1]) + pad, H, d)))

    def device(self):
        import torch

        i = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
        q = to_device(None, self.q)
        o = torch.full_like(q, 7.0)
        lse = torch.full(q.shape[:2], 7.0, device="cuda")
        return dict(q=q, k_pages=to_device(None, self.k), v_pages=to_device(None, self.v),
                    prefix_table=i(self.prefix_table), prefix_len=self.prefix, block_table=i(self.table),
                    seq_lens=i(self.seq), cu_new=i(self.cu), max_new=max([1] + self.new), o=o, lse=lse)

    def run(self, causal=True, scale=None, **kw):
        import torch

        import exact_io_aware_07_gb300 as fa

        a = self.device()
        a.update(kw)
        fa.fa_fwd_prefix_paged(**a, causal=causal, scale=scale or 1 / math.sqrt(self.d))
        torch.cuda.synchronize()
        assert fa.fa_device_status() == 0
        return a["o"], a["lse"]

    def reference(self, causal=True, scale=None):
        f = fi.bf16_bits_to_f64
        return paged.attention_prefix_paged(f(self.q), f(self.k), f(self.v), self.prefix_table, self.prefix, self.table,
                                            self.seq, self.cu, causal, scale or 1 / math.sqrt(self.d))

    def check(self, o, lse, causal=True, scale=None, label=""):
        compare(o, lse, self.reference(causal, scale), int(self.cu[-1]), self.d, label)


def compare(o, lse, ref, live, d, label=""):
    O, L, spread, size = (x[:live] for x in ref)
    got, got_lse = bf16_to_f64(o), lse.cpu().numpy().astype(np.float64)
    assert (got[live:] == 7.0).all() and (got_lse[live:] == 7.0).all(), f"{label}: rows behind the last request written"
    got, got_lse = got[:live], got_lse[:live]
    assert np.isfinite(got).all(), f"{label}: O not finite"
    empty = np.isneginf(L)
    assert (np.isneginf(got_lse) == empty).all() and (got[empty] == 0).all(), f"{label}: rows without a key"
    u = 2.0 ** -8
    ds = (d + 1) * 2.0 ** -23 * size
    bound = (0.5 * bf16_ulp(np.maximum(np.abs(O), np.abs(got)))
             + (u / (1 - u) + 2 * ds[..., None] + 2.0 ** -16) * spread + 2.0 ** -16 * np.abs(O))
    err = np.abs(got - O)
    worst = float((err / bound.clip(1e-30)).max(initial=0))
    assert (err <= bound).all(), f"{label}: O off by {worst:.2f} of its bound at {np.argwhere(err > bound)[:3].tolist()}"
    lse_bound = ds + 2.0 ** -21 + 2.0 ** -22 * (size + 2 * np.abs(np.where(empty, 0, L)))
    lse_err = np.abs(np.where(empty, 0, got_lse) - np.where(empty, 0, L))
    assert (lse_err <= lse_bound).all(), f"{label}: LSE off by {float((lse_err / lse_bound).max()):.2f} of its bound"


# ---------------------------------------------------------------- attention

EDGES = [1, 2, 127, 128, 129, 255, 256, 257, 1000]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("prefix", [0, 1, 127, 128, 129, 700])
def test_single_tokens_at_page_edges(d, prefix):
    b = Batch(d, 8, 2, prefix, EDGES, [1] * len(EDGES), pad=2, seed=1)
    b.check(*b.run(), label=f"edges d{d} P{prefix}")


@pytest.mark.parametrize("H,Hkv,d", [(1, 1, 64), (3, 1, 128), (6, 2, 64), (5, 1, 128), (16, 16, 64), (8, 1, 128),
                                     (12, 12, 64), (64, 1, 64), (128, 1, 128), (33, 1, 64), (14, 2, 128)])
def test_head_layouts(H, Hkv, d):
    b = Batch(d, H, Hkv, 200, [5, 130, 300], [1, 3, 2], seed=2)
    b.check(*b.run(), label=f"heads {H}/{Hkv} d{d}")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_ragged_new_tokens(d, causal):
    """Requests that add nothing, one token, a few, and chunks over several row tiles; caches longer than the chunk."""
    b = Batch(d, 4, 1, 150, [3, 40, 64, 500, 33, 129, 700, 10], [3, 0, 64, 1, 33, 129, 150, 0], pad=5, seed=3)
    b.check(*b.run(causal), causal, label=f"ragged d{d} causal{int(causal)}")


@pytest.mark.parametrize("d,H,Hkv,prefix,rows", [(64, 4, 4, 300, 600), (128, 8, 2, 260, 100), (128, 16, 1, 513, 40)])
def test_many_rows_share_the_prefix(d, H, Hkv, prefix, rows):
    """More rows than a tile over the prefix, from requests of one or two tokens with short caches."""
    new = [1 + (i % 3 == 0) for i in range(rows * 3 // 4)]
    own = [n + (i * 7) % 30 for i, n in enumerate(new)]
    b = Batch(d, H, Hkv, prefix, own, new, pad=1, seed=4)
    b.check(*b.run(), label=f"rows {rows} d{d}")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("prefix,own", [(0, [20000]), (9000, [1]), (5000, [6000, 17])])
def test_long_sequences(d, prefix, own):
    b = Batch(d, 4, 2, prefix, own, [1] * len(own), seed=5)
    b.check(*b.run(), label=f"long P{prefix} {own} d{d}")


def test_chunk_without_earlier_keys_is_causal_attention():
    """A prompt worked in one chunk: bit for bit the same rows whatever request stands beside it is not asked for,
    but its values are those of plain causal attention."""
    b = Batch(128, 4, 2, 0, [777, 1], [777, 1], seed=6)
    b.check(*b.run(), label="prompt")


@pytest.mark.parametrize("d", [64, 128])
def test_rows_that_see_nothing(d):
    """No prefix and no own key (an empty cache, or places before the first key): O = 0, LSE = -infinity."""
    b = Batch(d, 4, 2, 0, [0, 2, 130, 1], [1, 5, 2, 1], seed=7)
    o, lse = b.run()
    b.check(o, lse, label="empty rows")
    assert np.isneginf(lse.cpu().numpy()[:4]).all()  # the empty cache's row and three places before the first key
    b = Batch(d, 4, 2, 140, [0, 2, 130, 1], [1, 5, 2, 1], seed=7)
    b.check(*b.run(), label="prefix only")
    b = Batch(d, 2, 2, 0, [0, 0, 0], [1, 2, 0], seed=7)
    b.check(*b.run(causal=False), causal=False, label="all empty")


@pytest.mark.parametrize("sigma", [0.01, 6.0])
def test_flat_and_sharp_rows(sigma):
    """Equal weights, and rows that one key dominates (scores of hundreds, the maximum moving along the row)."""
    for d in (64, 128):
        b = Batch(d, 4, 2, 600, [700, 1, 90], [2, 1, 1], seed=8, sigma=sigma)
        b.check(*b.run(), label=f"sigma {sigma} d{d}")


def test_any_scale():
    b = Batch(128, 4, 2, 300, [100, 260], [1, 2], seed=9)
    for scale in (1e-4, 3.0):
        b.check(*b.run(scale=scale), scale=scale, label=f"scale {scale}")


@pytest.mark.parametrize("max_new", [1, 7, 100000])
def test_max_new_is_a_hint(max_new):
    b = Batch(64, 4, 1, 130, [300, 5, 64], [80, 5, 1], seed=10)
    b.check(*b.run(max_new=max_new), label=f"max_new {max_new}")


def test_many_requests():
    """More requests than threads or SMs, most without a new token."""
    own = [(i * 37) % 300 for i in range(1500)]
    new = [min(n, 1) if i % 4 else 0 for i, n in enumerate(own)]
    b = Batch(64, 2, 1, 140, own, new, seed=11)
    b.check(*b.run(), label="many requests")


def test_infinite_and_nan_inputs_stay_in_their_rows():
    """A NaN query row and an infinite value row reach the rows that use them, and no other."""
    b = Batch(64, 4, 2, 140, [60, 70], [2, 1], seed=12)
    o0, lse0 = b.run()
    b.q[1, 2] = NAN_BITS
    b.v[b.table[1, 0], 0, 3] = INF_BITS
    import torch

    import exact_io_aware_07_gb300 as fa

    a = b.device()
    fa.fa_fwd_prefix_paged(**a, causal=True, scale=0.125)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == 0
    o, lse = a["o"], a["lse"]
    assert torch.isnan(o[1, 2]).all() and torch.isnan(lse[1, 2])
    assert (o[2, :2] == float("inf")).all()  # K/V head 0 of request 1
    same = torch.ones(3, 4, dtype=torch.bool)
    same[1, 2] = same[2, 0] = same[2, 1] = False
    assert torch.equal(o[same.cuda()], o0[same.cuda()]) and torch.equal(lse[same.cuda()], lse0[same.cuda()])


def test_equal_calls_give_equal_bits():
    import torch

    b = Batch(128, 8, 2, 1000, [900, 30, 257, 1], [1, 4, 2, 1], seed=13)
    o1, l1 = b.run()
    for _ in range(3):
        o2, l2 = b.run()
        assert torch.equal(o1, o2) and torch.equal(l1, l2)


def test_offsets_beyond_32_bits():
    """A pool of more than 2^31 elements: pages at both ends."""
    import torch

    import exact_io_aware_07_gb300 as fa

    d, Hkv, H = 128, 2, 4
    b = Batch(d, H, Hkv, 200, [150, 300], [1, 2], seed=14)
    count = 2 ** 31 // (Hkv * 128 * d) + 20
    a = b.device()
    for name in ("k_pages", "v_pages"):
        big = torch.empty(count, Hkv, 128, d, dtype=torch.bfloat16, device="cuda")
        small = a[name]
        big[:4] = small[:4]
        big[count - small.shape[0] + 4:] = small[4:]
        a[name] = big
    move = lambda t: torch.where(t >= 4, t + count - b.k.shape[0], t)  # noqa: E731
    a["block_table"], a["prefix_table"] = move(a["block_table"]), move(a["prefix_table"])
    fa.fa_fwd_prefix_paged(**a, causal=True, scale=d ** -0.5)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == 0
    b.check(a["o"], a["lse"], label="large pool")
    # append to the last page of the large pool
    new = torch.randn(1, Hkv, d, device="cuda").to(torch.bfloat16)
    slot = torch.tensor([(count - 1) * 128 + 127], dtype=torch.int32, device="cuda")
    fa.fa_kv_append(new, -new, slot, a["k_pages"], a["v_pages"])
    assert torch.equal(a["k_pages"][count - 1, :, 127], new[0]) and torch.equal(a["v_pages"][count - 1, :, 127], -new[0])
    assert fa.fa_device_status() == 0


def test_pages_outside_the_pool_are_reported_and_read_as_zeros():
    import torch

    import exact_io_aware_07_gb300 as fa

    for where in ("table", "prefix_table"):
        for page in (-1, 10 ** 6):
            b = Batch(64, 2, 2, 140, [140], [1], seed=15)
            row = b.table[0] if where == "table" else b.prefix_table
            old, row[1] = int(row[1]), page
            a = b.device()
            fa.fa_fwd_prefix_paged(**a, causal=True, scale=0.125)
            assert fa.fa_device_status() == 14 and fa.fa_device_status() == 0
            row[1] = old
            b.k[old], b.v[old] = 0, 0  # what the page reads as
            b.check(a["o"], a["lse"], label="bad page", scale=0.125)


def test_lengths_outside_the_batch_are_cut_and_reported():
    import exact_io_aware_07_gb300 as fa

    b = Batch(64, 2, 1, 0, [256, 20], [1, 1], seed=16, extra_cols=0)
    b.seq[0] = 10 ** 6  # more than its table holds: cut to 256
    a = b.device()
    fa.fa_fwd_prefix_paged(**a, causal=True, scale=0.125)
    assert fa.fa_device_status() == 15 and fa.fa_device_status() == 0
    b.seq[0] = 256
    b.check(a["o"], a["lse"], label="long length", scale=0.125)
    b.seq[1] = -4
    a = b.device()
    fa.fa_fwd_prefix_paged(**a, causal=True, scale=0.125)
    assert fa.fa_device_status() == 15
    b.seq[1] = 0
    b.check(a["o"], a["lse"], label="negative length", scale=0.125)
    b.seq[1] = 20
    a = b.device()
    a["cu_new"][2] = 99  # beyond the rows of the batch: cut to them, all behind the first request's
    fa.fa_fwd_prefix_paged(**a, causal=True, scale=0.125)
    assert fa.fa_device_status() == 15
    b.check(a["o"], a["lse"], label="rows", scale=0.125)


def test_refused_calls_write_nothing():
    import torch

    import exact_io_aware_07_gb300 as fa

    b = Batch(64, 2, 2, 140, [140], [1], seed=17)
    for kw in (dict(o=b.device()["q"]), dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
               dict(seq_lens=torch.tensor([140], dtype=torch.int32))):  # the last one is host memory
        a = b.device()
        a.update(kw)
        if "o" in kw:
            a["o"] = a["q"]
        with pytest.raises(fa.FAError):
            fa.fa_fwd_prefix_paged(**a, causal=True, scale=0.125)
        torch.cuda.synchronize()
        assert (a["lse"] == 7.0).all()


def test_on_another_stream_and_in_graphs_that_share_a_workspace():
    import torch

    import exact_io_aware_07_gb300 as fa

    x, y = (Batch(128, 8, 2, 500, [300, 40, 129], [1, 2, 1], seed=s) for s in (18, 19))
    ax, ay = x.device(), y.device()
    n, H, d = ax["q"].shape
    ws = torch.empty(fa.fa_fwd_prefix_paged_workspace_bytes(n, 3, H, 2, d), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    fa.fa_fwd_prefix_paged(**ax, causal=True, scale=d ** -0.5, workspace=ws, stream=s)
    s.synchronize()
    x.check(ax["o"], ax["lse"], label="stream")
    graphs = []
    for a in (ax, ay):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fa.fa_fwd_prefix_paged(**a, causal=True, scale=d ** -0.5, workspace=ws)
        graphs.append(g)
    for a in (ax, ay):
        a["o"].fill_(7.0), a["lse"].fill_(7.0)
    ws.fill_(0xFF)
    for _ in range(3):
        graphs[0].replay()
        graphs[1].replay()
    torch.cuda.synchronize()
    x.check(ax["o"], ax["lse"], label="graph x")
    y.check(ay["o"], ay["lse"], label="graph y")
    # shorter caches, read by the same captured launch
    x.seq[:] = [200, 3, 128]
    ax["seq_lens"].copy_(torch.from_numpy(x.seq))
    graphs[0].replay()
    torch.cuda.synchronize()
    x.check(ax["o"], ax["lse"], label="replayed with new lengths")
    assert fa.fa_device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tokens", [2, 3, 4, 7, 8, 15, 16, 17, 31])
@pytest.mark.parametrize("prefix", [0, 333])
def test_rows_per_request(d, tokens, prefix):
    """4 to 124 rows a request and K/V head: requests on warp-level products, and those that fill part of a row tile;
    beside them requests of fewer rows."""
    own = [tokens, 1500, tokens + 130, 1 + tokens // 2, 257]
    b = Batch(d, 8, 2, prefix, own, [tokens, tokens, tokens, 1 + tokens // 2, 1], pad=1, seed=30)
    b.check(*b.run(), label=f"{4 * tokens} rows P{prefix} d{d}")


@pytest.mark.parametrize("d,H,Hkv,tokens", [(64, 2, 2, 1), (128, 4, 1, 1), (128, 8, 1, 2), (64, 32, 1, 1), (128, 16, 1, 4)])
def test_few_rows_in_all(d, H, Hkv, tokens):
    """One request, whose rows work the prefix as few rows too: long and short, alone or with own keys."""
    for prefix, own in ((4000, tokens), (1, 3000), (129, 0), (2049, 515)):
        b = Batch(d, H, Hkv, prefix, [own], [tokens], seed=31)
        b.check(*b.run(), label=f"one request P{prefix} own{own}")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("prefix", [0, 400])
def test_every_kind_of_request_in_one_batch(d, prefix):
    """Decoding, drafted, middling and big requests in turn, so that row blocks hold rows of several kinds."""
    new = [1, 200, 5, 20, 1, 0, 64, 33, 2, 1, 130]
    own = [900, 200, 77, 520, 1, 300, 700, 33, 129, 256, 1]
    b = Batch(d, 8, 2, prefix, own, new, pad=3, seed=32)
    for causal in (True, False):
        b.check(*b.run(causal), causal, label=f"kinds P{prefix} d{d} causal{int(causal)}")


def test_more_row_blocks_than_are_flagged():
    """2 065 tokens of 128 rows each, two tokens a row block: 1 033 blocks.  Three heads of every token are compared."""
    new = [1] * 400 + [0] + [1] * 1465 + [200]
    own = [i % 3 for i in range(len(new) - 1)] + [260]
    b = Batch(64, 128, 1, 130, own, new, pad=1, seed=33)
    o, lse = b.run()
    heads = [0, 77, 127]
    b.q = np.ascontiguousarray(b.q[:, heads])
    b.check(o[:, heads], lse[:, heads], label="row blocks")


def test_the_prefix_may_be_a_request_of_the_batch():
    """The prefix's table is the first entries of a request's own row: big, middling and decoding rows read both."""
    for new in ([150, 1], [20, 1], [1, 1]):
        b = Batch(64, 8, 2, 0, [700, 40], new, seed=34)
        b.prefix, b.prefix_table = 200, b.table[0, :2].copy()
        a = b.device()
        a["prefix_table"] = a["block_table"][0, :2]
        b.check(*b.run(prefix_table=a["prefix_table"], block_table=a["block_table"]), label=f"own prefix {new}")


@pytest.mark.parametrize("requests", [1, 40])
def test_calls_one_behind_the_other(requests):
    """Each call's O is the next call's query, in one workspace: a call starts only when the one before it is through."""
    import torch

    import exact_io_aware_07_gb300 as fa

    d = 128
    b = Batch(d, 8, 2, 300, [(37 * i) % 200 + 1 for i in range(requests)], [1] * requests, seed=35)
    a = b.device()
    n = a["q"].shape[0]
    ws = torch.empty(fa.fa_fwd_prefix_paged_workspace_bytes(n, requests, 8, 2, d), dtype=torch.uint8, device="cuda")
    qs = [a.pop("q")] + [torch.full_like(a["o"], 7.0) for _ in range(6)]
    lses = [torch.full_like(a["lse"], 7.0) for _ in range(6)]
    a.pop("o"), a.pop("lse")

    def chain():
        for i in range(6):
            fa.fa_fwd_prefix_paged(q=qs[i], o=qs[i + 1], lse=lses[i], causal=True, scale=1.0, workspace=ws, **a)

    chain()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for replay in (False, True):
        if replay:
            for x in qs[1:]:
                x.fill_(7.0)
            graph.replay()
        torch.cuda.synchronize()
        for i in range(6):
            b.q = qs[i].view(torch.int16).cpu().numpy().view(np.uint16)
            b.check(qs[i + 1], lses[i], scale=1.0, label=f"call {i} replay{int(replay)}")
    assert fa.fa_device_status() == 0


def test_batches_of_all_sizes_in_turn_share_a_workspace():
    """One request, a decoding batch and prompt chunks one behind the other on a stream and in a graph, all in one
    workspace: each gives the bits that it gives alone."""
    import torch

    import exact_io_aware_07_gb300 as fa

    shapes = [(128, 8, 2, 300, [40], [1]), (64, 16, 16, 100, [200, 3, 70], [6, 1, 2]),
              (128, 8, 2, 1000, [(53 * i) % 400 + 1 for i in range(90)], [1] * 90), (128, 8, 2, 260, [600, 64], [400, 30])]
    batches = [Batch(*x, pad=1, seed=40) for x in shapes]
    args = [b.device() for b in batches]
    size = max(fa.fa_fwd_prefix_paged_workspace_bytes(a["q"].shape[0], len(b.own), b.H, b.Hkv, b.d)
               for a, b in zip(args, batches))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    alone = []
    for b, a in zip(batches, args):
        fa.fa_fwd_prefix_paged(**a, causal=True, scale=b.d ** -0.5)
        torch.cuda.synchronize()
        b.check(a["o"], a["lse"], label="alone")
        alone.append((a["o"].clone(), a["lse"].clone()))
    order = [0, 2, 0, 1, 3, 0, 0, 2, 1, 1, 3, 2, 0]

    def turns():
        outs = []
        for i in order:
            a = dict(args[i], o=torch.full_like(args[i]["o"], 7.0), lse=torch.full_like(args[i]["lse"], 7.0))
            fa.fa_fwd_prefix_paged(**a, causal=True, scale=batches[i].d ** -0.5, workspace=ws)
            outs.append((a["o"], a["lse"]))
        return outs

    graph = torch.cuda.CUDAGraph()
    first = turns()
    with torch.cuda.graph(graph):
        second = turns()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert fa.fa_device_status() == 0
    for outs in (first, second):
        for i, (o, lse) in zip(order, outs):
            assert torch.equal(o, alone[i][0]) and torch.equal(lse, alone[i][1]), i


def test_two_calls_at_once():
    """Two streams, each with a workspace of its own."""
    import torch

    import exact_io_aware_07_gb300 as fa

    pair = [Batch(d, 8, 2, 700, [900, 33, 260, 1] * 6, [1, 3, 40, 1] * 6, seed=36) for d in (64, 128)]
    args = [x.device() for x in pair]
    ws = [torch.empty(fa.fa_fwd_prefix_paged_workspace_bytes(a["q"].shape[0], 24, 8, 2, x.d), dtype=torch.uint8,
                      device="cuda") for x, a in zip(pair, args)]
    streams = [torch.cuda.Stream() for _ in pair]
    torch.cuda.synchronize()
    for _ in range(20):
        for x, a, w, s in zip(pair, args, ws, streams):
            fa.fa_fwd_prefix_paged(**a, causal=True, scale=x.d ** -0.5, workspace=w, stream=s)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == 0
    for x, a in zip(pair, args):
        x.check(a["o"], a["lse"], label=f"d{x.d} beside another")


def test_wrappers_on_a_given_stream():
    """The convenience calls allocate, fill and run on the stream they are given, while the current stream is busy."""
    import torch

    import exact_io_aware_07_gb300 as fa

    b = Batch(128, 8, 2, 500, [300, 40, 129], [1, 2, 1], pad=2, seed=37)
    a = b.device()
    a.pop("o"), a.pop("lse")
    i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    plan = (i([126, 0]), i([3, 1]), i([5, 4, 9]), i([0]), i([[8, -1], [-1, -1]]))
    side = torch.cuda.Stream()
    big = torch.randn(8192, 8192, device="cuda")
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        for _ in range(4):
            big @ big  # work on the current stream that the side stream's calls neither wait for nor follow
        o, lse = fa.attention_prefix_paged(**a, stream=stream)
        seq, cu, slots, head = fa.page_plan(*plan, 5, 10, stream=stream)
        junk = [torch.full_like(o, 9.0) for _ in range(4)]  # takes any memory given back too early
        side.synchronize()
        assert (o[4:] == 0).all() and torch.isneginf(lse[4:]).all()
        o[4:], lse[4:] = 7.0, 7.0
        b.check(o, lse, label="wrapper on a stream")
        assert seq.tolist() == [129, 1] and cu.tolist() == [0, 3, 4] and head.tolist() == [2]
        assert slots.tolist() == [8 * 128 + 126, 8 * 128 + 127, 5 * 128, 4 * 128, -1]
        del junk
    torch.cuda.synchronize()
    assert fa.fa_device_status() == 0


@pytest.mark.parametrize("d,H,Hkv,prefix,own,new", [
    (64, 4, 4, 300, [700, 5, 129], [1, 2, 1]),      # few rows only
    (64, 12, 1, 300, [700, 40], [1, 1]),            # few rows of two tiles of eight
    (128, 8, 2, 500, [900, 64, 300], [150, 20, 1]),  # every kind
    (128, 6, 2, 0, [2000, 1], [1, 1]),              # rows cut into many parts
])
def test_nothing_else_is_written(d, H, Hkv, prefix, own, new):
    """Outputs and a workspace of exactly the asked size inside larger buffers: what surrounds them and every input stay."""
    import torch

    import exact_io_aware_07_gb300 as fa

    b = Batch(d, H, Hkv, prefix, own, new, pad=2, seed=39)
    a = b.device()
    before = {k: v.clone() for k, v in a.items() if torch.is_tensor(v) and k not in ("o", "lse")}
    n = a["q"].shape[0]
    size = fa.fa_fwd_prefix_paged_workspace_bytes(n, len(own), H, Hkv, d)
    room = 4096

    def inside(numel, dtype, fill):
        buf = torch.full((numel + 2 * room,), fill, dtype=dtype, device="cuda")
        return buf, buf[room:room + numel]

    ws_buf, ws = inside(size, torch.uint8, 0xA5)
    o_buf, o = inside(n * H * d, torch.bfloat16, 7.0)
    lse_buf, lse = inside(n * H, torch.float32, 7.0)
    a.update(o=o.view(n, H, d), lse=lse.view(n, H))
    for _ in range(2):
        fa.fa_fwd_prefix_paged(**a, causal=True, scale=d ** -0.5, workspace=ws)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == 0
    b.check(a["o"], a["lse"], label="inside larger buffers")
    for buf, fill in ((ws_buf, 0xA5), (o_buf, 7.0), (lse_buf, 7.0)):
        assert (buf[:room] == fill).all() and (buf[-room:] == fill).all()
    for k, v in before.items():
        assert torch.equal(v.view(torch.uint8), a[k].view(torch.uint8)), k


def test_decreasing_cu_new_is_reported():
    import exact_io_aware_07_gb300 as fa

    b = Batch(64, 4, 1, 130, [20, 30, 300], [2, 1, 140], seed=38)
    a = b.device()
    a["cu_new"][1], a["cu_new"][2] = 3, 1
    fa.fa_fwd_prefix_paged(**a, causal=True, scale=0.125)
    assert fa.fa_device_status() == 15 and fa.fa_device_status() == 0


# ---------------------------------------------------------------- plan

def _plan_inputs(ctx, new, seed, slack=3, head=2, extra_cols=1):
    rng = np.random.default_rng(seed)
    ctx, new = np.array(ctx, dtype=np.int32), np.array(new, dtype=np.int32)
    held, total = pages_of(ctx), pages_of(ctx + new)
    table = np.full((len(ctx), int(total.max(initial=1)) + extra_cols), -5, dtype=np.int32)
    num_pages = int(total.sum()) + slack + head
    order = rng.permutation(num_pages).astype(np.int32)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = order[at:at + n]
        at += n
    return ctx, new, table, order[at:], head, num_pages


def _run_plan(ctx, new, table, free, head, num_pages, max_tokens):
    import torch

    import exact_io_aware_07_gb300 as fa

    i = lambda x: torch.from_numpy(np.ascontiguousarray(np.asarray(x, dtype=np.int32))).cuda()  # noqa: E731
    t = i(table)
    out = fa.page_plan(i(ctx), i(new), i(free), i([head]), t, max_tokens, num_pages)
    return [x.cpu().numpy() for x in (t, *out)]


@pytest.mark.parametrize("ctx,new,pad", [
    ([0], [1], 0), ([127], [1], 3), ([128], [1], 0), ([0, 0, 5], [0, 0, 0], 2), ([1, 127, 128, 129, 0], [300, 1, 128, 0, 1], 7),
    ([(i * 91) % 700 for i in range(1023)], [(i * 7) % 5 for i in range(1023)], 1),
    ([(i * 91) % 700 for i in range(1024)], [1] * 1024, 0),
    ([(i * 13) % 400 for i in range(2500)], [(i * 11) % 9 for i in range(2500)], 300),
    ([100, 0], [30000, 20000], 11),
])
def test_plan_equals_the_oracle(ctx, new, pad):
    import exact_io_aware_07_gb300 as fa

    ctx, new, table, free, head, num_pages = _plan_inputs(ctx, new, seed=20)
    max_tokens = max(1, int(new.sum()) + pad)
    got = _run_plan(ctx, new, table, free, head, num_pages, max_tokens)
    want = paged.page_plan(ctx, new, free, head, table, max_tokens)
    for name, g, w in zip(("table", "seq", "cu", "slots", "head"), got, want):
        assert np.array_equal(g.reshape(-1), np.reshape(w, -1)), name
    assert fa.fa_device_status() == 0


def test_plan_reports_a_list_that_runs_out():
    import exact_io_aware_07_gb300 as fa

    ctx, new, table, free, head, num_pages = _plan_inputs([120, 0, 0], [20, 200, 5], seed=21)
    got = _run_plan(ctx, new, table, free[:head + 2], head, num_pages, 225)  # four pages wanted, two there
    assert fa.fa_device_status() == 16 and fa.fa_device_status() == 0
    t, _, cu, slots, out = got
    assert t[0, 1] == free[head] and t[1, 0] == free[head + 1] and t[1, 1] == -1 and t[2, 0] == -1
    assert out[0] == head + 2 and cu.tolist() == [0, 20, 220, 225]
    assert (slots[:148] >= 0).all() and (slots[148:] == -1).all()
    got = _run_plan([0], [3], np.full((1, 2), 8), [], 0, num_pages, 3)
    assert fa.fa_device_status() == 16 and (got[3] == -1).all() and got[0].tolist() == [[-1, 8]] and got[4][0] == 0


def test_plan_reports_bad_lengths_and_pages():
    import exact_io_aware_07_gb300 as fa

    ctx, new, table, free, head, num_pages = _plan_inputs([10, 10, 10, 10], [5, 5, 5, 5], seed=22)
    ctx[1], new[2], new[3] = -1, -7, 10 ** 9  # these three requests add nothing
    _, seq, cu, slots, out = _run_plan(ctx, new, table, free, head, num_pages, 8)
    assert fa.fa_device_status() == 15
    assert cu.tolist() == [0, 5, 5, 5, 5] and out[0] == head and (slots[:5] >= 0).all() and (slots[5:] == -1).all()
    ctx, new, table, free, head, num_pages = _plan_inputs([10, 0], [5, 3], seed=23)
    table[0, 0], free[head] = -1, num_pages  # a held page and a free page that are not of the pool
    t, _, _, slots, _ = _run_plan(ctx, new, table, free, head, num_pages, 9)
    assert fa.fa_device_status() == 14
    assert (slots == -1).all() and t[1, 0] == -1 and t[0, 0] == -1
    ctx, new, table, free, head, num_pages = _plan_inputs([0, 3], [4, 4], seed=24)
    _, _, cu, slots, _ = _run_plan(ctx, new, table, free, head, num_pages, 6)  # eight tokens, room for six
    assert fa.fa_device_status() == 15
    assert cu.tolist() == [0, 4, 8] and np.array_equal(slots, paged.page_plan(ctx, new, free, head, table, 8)[3][:6])


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,Hkv,wide", [(1, 1, 0), (1, 8, 24), (5, 3, 8), (64, 8, 0), (700, 2, 64), (3000, 5, 0)])
def test_append_equals_the_oracle(d, N, Hkv, wide):
    """Keys and values as columns of one projection (``wide`` further columns), slots in any order, some skipped."""
    import torch

    import exact_io_aware_07_gb300 as fa

    rng = np.random.default_rng([25, d, N, Hkv])
    num_pages = pages_of(N) + 2
    slots = rng.permutation(num_pages * 128)[:N].astype(np.int32)
    slots[rng.random(N) < 0.2] = -1
    if N > 1:
        slots[-1], slots[0] = -2 ** 31, num_pages * 128 - 1 if num_pages * 128 - 1 not in slots else slots[0]
    proj = rng.integers(0, 2 ** 16, (N, 2 * Hkv * d + wide)).astype(np.uint16)  # any bits, NaN among them
    pools = rng.integers(0, 2 ** 16, (2, num_pages, Hkv, 128, d)).astype(np.uint16)
    t = to_device(None, proj)
    kp, vp = to_device(None, pools[0]), to_device(None, pools[1])
    k, v = t[:, :Hkv * d].unflatten(1, (Hkv, d)), t[:, Hkv * d:2 * Hkv * d].unflatten(1, (Hkv, d))
    fa.fa_kv_append(k, v, torch.from_numpy(slots).cuda(), kp, vp)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == 0
    for got, pool, new in ((kp, pools[0], proj[:, :Hkv * d]), (vp, pools[1], proj[:, Hkv * d:2 * Hkv * d])):
        want = paged.kv_append(new.reshape(N, Hkv, d), slots, pool)
        assert np.array_equal(got.view(torch.int16).cpu().numpy().view(np.uint16), want)


def test_append_reports_a_slot_outside_the_pool():
    import torch

    import exact_io_aware_07_gb300 as fa

    pool = torch.zeros(2, 3, 128, 64, dtype=torch.bfloat16, device="cuda")
    pools = pool.clone(), pool.clone()
    new = torch.ones(4, 3, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([255, 256, 2 ** 31 - 1, 0], dtype=torch.int32, device="cuda")
    fa.fa_kv_append(new, new, slots, *pools)
    assert fa.fa_device_status() == 14 and fa.fa_device_status() == 0
    pool[1, :, 127], pool[0, :, 0] = 1, 1
    assert torch.equal(pools[0], pool) and torch.equal(pools[1], pool)


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("d,H,Hkv", [(64, 4, 2), (128, 8, 1)])
def test_steps_together(d, H, Hkv):
    """A batch that starts from prompts and decodes, behind a shared prefix: plan, append and attention of every step,
    the decoding steps replayed from one captured graph, against attention on each request's gathered keys."""
    import torch

    import exact_io_aware_07_gb300 as fa

    rng = np.random.default_rng([26, d])
    prefix, B, num_pages, max_pages = 200, 5, 40, 6
    prompts, steps = [126, 1, 300, 0, 127], 4
    order = rng.permutation(num_pages).astype(np.int32)
    i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    free, prefix_table = i(order[2:]), i(order[:2])
    pools = [torch.full((num_pages, Hkv, 128, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    kv = rng.standard_normal((2, B + 1, 600, Hkv, d)).astype(np.float32)  # every key and value there will be
    kv_bits = bits(kv)
    head, table, ctx = i([0]), i(np.full((B, max_pages), -1)), i([0] * B)
    seq, cu, head2 = i([0] * B), i([0] * (B + 1)), i([0])
    slots = prefix_table.long().repeat_interleave(128)[:prefix] * 128 + torch.arange(prefix, device="cuda") % 128
    fa.fa_kv_append(*(to_device(None, x[B, :prefix]) for x in kv_bits), slots.int(), *pools)  # like any tokens

    def step(new, slots, k, v, q, o, lse, ws, max_new):
        fa.fa_page_plan(ctx, new, free, head, table, seq, cu, slots, head2, num_pages)
        fa.fa_kv_append(k, v, slots, *pools)
        fa.fa_fwd_prefix_paged(q, *pools, prefix_table, prefix, table, seq, cu, max_new, o, lse, True, d ** -0.5, ws)
        ctx.copy_(seq)
        head.copy_(head2)

    def buffers(rows):
        e = dict(dtype=torch.bfloat16, device="cuda")
        return (torch.empty(rows, dtype=torch.int32, device="cuda"), torch.empty(rows, Hkv, d, **e),
                torch.empty(rows, Hkv, d, **e), torch.empty(rows, H, d, **e), torch.full((rows, H, d), 7.0, **e),
                torch.full((rows, H), 7.0, device="cuda"),
                torch.empty(fa.fa_fwd_prefix_paged_workspace_bytes(rows, B, H, Hkv, d), dtype=torch.uint8, device="cuda"))

    have = [0] * B

    def load(new, buf):
        rows = [(b, have[b] + t) for b, n in enumerate(new) for t in range(n)]
        for dst, x in ((buf[1], kv_bits[0]), (buf[2], kv_bits[1])):
            if rows:
                dst[:len(rows)] = to_device(None, np.stack([x[b, t] for b, t in rows]))
        q = bits(rng.standard_normal((buf[3].shape[0], H, d)))
        buf[3].copy_(to_device(None, q))
        buf[4].fill_(7.0), buf[5].fill_(7.0)
        for b, n in enumerate(new):
            have[b] += n
        return q

    def check(q, new, buf, label):
        torch.cuda.synchronize()
        assert fa.fa_device_status() == 0
        f = fi.bf16_bits_to_f64
        scale, at = d ** -0.5, 0
        O, L, spread, size = (np.zeros((sum(new), H, *s)) for s in ((d,), (), (d,), ()))
        for b, n in enumerate(new):
            for t in range(n):
                for h in range(H):
                    g, seen = h // (H // Hkv), have[b] - n + t + 1
                    k, v = (np.concatenate([f(x[B, :prefix, g]), f(x[b, :seen, g])]) for x in kv_bits)
                    O[at, h], L[at, h], spread[at, h], size[at, h] = paged.row(f(q[at, h]), k, v, scale)
                at += 1
        compare(buf[4], buf[5], (O, L, spread, size), sum(new), d, label)
        assert seq.tolist() == have and int(head) == sum(pages_of(n) for n in have)

    buf = buffers(sum(prompts) + 3)
    q = load(prompts, buf)
    step(i(prompts), *buf, max(prompts))
    check(q, prompts, buf, "prompts")
    buf, new = buffers(B + 2), i([0] * B)
    q = load([0] * B, buf)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(new, *buf, 1)  # nothing new: a first call outside the capture
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(new, *buf, 1)
    for s in range(steps):
        want = [1 if (s + b) % 4 else 0 for b in range(B)]
        q = load(want, buf)
        new.copy_(i(want))
        graph.replay()
        check(q, want, buf, f"step {s}")


@pytest.mark.parametrize("op", ["plan", "append", "prefix", "step"])
def test_command_line(op, monkeypatch, capsys):
    import sys

    from exact_io_aware_07_gb300 import __main__ as cli

    monkeypatch.setattr(sys, "argv", ["x", "--op", op, "--B", "3", "--H", "4", "--hkv", "2", "--T", "200", "--d", "64",
                                      "--prefix", "300", "--new", "2"])
    assert cli.main() == 0
    assert "device status 0" in capsys.readouterr().out


# ---------------------------------------------------------------- values that are not finite

@pytest.mark.parametrize("prefix", [0, 200])
@pytest.mark.parametrize("d,H,Hkv,own,new", [
    (64, 8, 2, [40, 30, 150, 3000], [1, 2, 20, 2]),
    (64, 16, 16, [200, 64, 700], [8, 5, 1]),              # few-row items of 8 and 16 rows
    (128, 8, 2, [400, 33, 300, 5000], [150, 2, 20, 2]),   # big, few and middling requests, one cut into many parts
    (128, 4, 4, [2000], [7]),                             # one request
    (64, 8, 2, [1200, 9], [1100, 2]),                     # over 7 296 rows
    (128, 8, 2, [1000, 40], [1000, 1]),
])
def test_values_that_are_not_finite_reach_only_the_rows_that_see_them(d, H, Hkv, own, new, prefix):
    """New tokens whose values have a NaN and infinities in some columns: the rows before them, whose weights there are 0,
    keep every column; the rows from them on keep the other columns.  A NaN in the prefix beside them reaches all rows'
    column.  The clean call before and after gives the same bits."""
    import torch

    import exact_io_aware_07_gb300 as fa

    b = Batch(d, H, Hkv, prefix, own, new, pad=1, seed=41)
    ref = b.reference()
    a = b.device()
    n, group = a["q"].shape[0], H // Hkv
    ws = torch.full((fa.fa_fwd_prefix_paged_workspace_bytes(n, len(own), H, Hkv, d),), 0xFF, dtype=torch.uint8, device="cuda")

    def run():
        a["o"].fill_(7.0), a["lse"].fill_(7.0)
        fa.fa_fwd_prefix_paged(**a, causal=True, scale=d ** -0.5, workspace=ws)
        torch.cuda.synchronize()
        assert fa.fa_device_status() == 0
        return a["o"].clone(), a["lse"].clone()

    o0, lse0 = run()
    compare(o0, lse0, ref, int(b.cu[-1]), d, "clean")
    marks = {}  # (row, head, column) -> what it has to be
    v = b.v.copy()
    for r, (s, t) in enumerate(zip(own, new)):
        for i in sorted({1, t // 2, t - 1}) if t > 1 else []:
            key = s - t + i
            for g in {0, Hkv - 1}:
                at = v[b.table[r, key // 128], g, key % 128]
                for col, x in ((3 + i % 7, NAN_BITS), (20, INF_BITS), (d - 1, INF_BITS | 0x8000)):
                    at[col] = x
                    for row in range(int(b.cu[r]) + i, int(b.cu[r + 1])):
                        for h in range(g * group, (g + 1) * group):
                            marks[row, h, col] = x
    if prefix:
        v[b.prefix_table[0], Hkv - 1, 7, 40] = NAN_BITS
        for row in range(int(b.cu[-1])):
            for h in range((Hkv - 1) * group, H):
                marks[row, h, 40] = NAN_BITS
    a["v_pages"] = to_device(None, v)
    o, lse = run()
    assert torch.equal(lse, lse0)  # values do not reach the statistics
    got = bf16_to_f64(o)
    for (row, h, col), x in marks.items():
        y = got[row, h, col]
        assert np.isnan(y) if x == NAN_BITS else y == (np.inf if x == INF_BITS else -np.inf), (row, h, col, y)
    index = torch.tensor(list(marks), device="cuda").t()
    o[index[0], index[1], index[2]] = o0[index[0], index[1], index[2]]
    compare(o, lse, ref, int(b.cu[-1]), d, "beside marked values")
    a["v_pages"] = to_device(None, b.v)
    o, lse = run()
    assert torch.equal(o, o0) and torch.equal(lse, lse0)


def test_a_value_that_all_rows_see_changes_no_other_column():
    """Rows that all see a NaN value are left as they are: the column of each is NaN, the others are those of the clean call,
    bit for bit."""
    import torch

    import exact_io_aware_07_gb300 as fa

    b = Batch(128, 8, 2, 0, [500, 30], [500, 2], seed=42)
    a = b.device()
    fa.fa_fwd_prefix_paged(**a, causal=True, scale=128 ** -0.5)
    o0 = a["o"].clone()
    b.v[b.table[0, 0], 1, 0, 9] = NAN_BITS
    a["v_pages"] = to_device(None, b.v)
    fa.fa_fwd_prefix_paged(**a, causal=True, scale=128 ** -0.5)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == 0
    assert torch.isnan(a["o"][:500, 4:, 9]).all()
    a["o"][:500, 4:, 9] = o0[:500, 4:, 9]
    assert torch.equal(a["o"], o0)


# ---------------------------------------------------------------- large batches, host threads

def check_rows(b, o, lse, rows, heads, label):
    """Rows `rows` and heads `heads` against the oracle, one by one; every row is finite."""
    f = fi.bf16_bits_to_f64
    group = b.H // b.Hkv
    prefix = {}
    out = [[], [], [], []]
    for n in rows:
        r = int(np.searchsorted(b.cu, n, side="right")) - 1
        seen = int(b.seq[r]) - int(b.cu[r + 1] - b.cu[r]) + int(n - b.cu[r]) + 1
        own = {}
        for h in heads:
            g = h // group
            if g not in prefix:
                prefix[g] = [f(paged.gather(x, b.prefix_table, b.prefix)[:, g]) for x in (b.k, b.v)]
            if g not in own:
                own[g] = [f(x[b.table[r, :pages_of(seen)], g].reshape(-1, b.d)[:seen]) for x in (b.k, b.v)]
            k, v = (np.concatenate(x) for x in zip(prefix[g], own[g]))
            for dst, x in zip(out, paged.row(f(b.q[n, h]), k, v, b.d ** -0.5)):
                dst.append(x)
    shape = len(rows), len(heads)
    ref = [np.array(x).reshape(*shape, *np.shape(x[0])) for x in out]
    index = np.ix_(rows, heads)
    compare(o[index], lse[index], ref, len(rows), b.d, label)
    live = int(b.cu[-1])
    assert bool(o[:live].isfinite().all()) and bool(lse[:live].isfinite().all()) and bool((o[live:] == 7).all()), label


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv,prefix,own,new", [
    (32, 8, 300, [700, 64, 1300] + [40] * 60, [600, 20, 160] + [1] * 60),  # rows of one part, of two and of cut items
    (16, 16, 0, [900], [900]),
    (8, 1, 1000, [5000, 3], [1000, 1]),
])
def test_more_rows_than_a_warp_each(d, H, Hkv, prefix, own, new):
    """Over 48 rows per SM: rows are joined eight lanes each."""
    b = Batch(d, H, Hkv, prefix, own, new, pad=2, seed=43)
    assert b.q.shape[0] * H > 48 * 152
    o, lse = b.run()
    rows = sorted({0, 1, 127, 128, 599, sum(new) - 1, *range(5, sum(new), 61)} & set(range(sum(new))))
    check_rows(b, o, lse, rows, sorted({0, 5, H - 1}), f"many rows d{d}")


@pytest.mark.parametrize("d,H,Hkv,prefix,own,new", [
    (64, 4, 2, 0, [6000], [6000]),
    (128, 8, 2, 500, [2500, 9000, 1], [2500, 4100, 1]),
])
def test_prompts_of_thousands_of_tokens(d, H, Hkv, prefix, own, new):
    b = Batch(d, H, Hkv, prefix, own, new, pad=1, seed=44)
    o, lse = b.run()
    rows = sorted({*range(0, sum(new), 331), *range(sum(new) - 5, sum(new))})
    check_rows(b, o, lse, rows, [0, H - 1], f"prompts {new} d{d}")


def test_plan_of_more_tokens_than_threads():
    """Two prompts of 80 000 tokens and places behind them: every thread of the grid has a second place."""
    import exact_io_aware_07_gb300 as fa

    ctx, new, table, free, head, num_pages = _plan_inputs([100, 0, 0, 64], [80000, 0, 80001, 1], seed=45)
    places = int(new.sum()) + 20000
    assert places > 152 * 1024
    got = _run_plan(ctx, new, table, free, head, num_pages, places)
    want = paged.page_plan(ctx, new, free, head, table, places)
    for name, g, w in zip(("table", "seq", "cu", "slots", "head"), got, want):
        assert np.array_equal(g.reshape(-1), np.reshape(w, -1)), name
    assert fa.fa_device_status() == 0


def test_calls_from_two_host_threads():
    """Each thread plans, appends and attends on a stream and in a workspace of its own, a hundred times."""
    import threading

    import torch

    import exact_io_aware_07_gb300 as fa

    pair = [Batch(d, 8, 2, 300, [600, 33, 260, 1], [1, 3, 40, 1], seed=46) for d in (64, 128)]
    failures = []

    def work(b):
        try:
            a = b.device()
            n = a["q"].shape[0]
            stream = torch.cuda.Stream()
            ws = torch.empty(fa.fa_fwd_prefix_paged_workspace_bytes(n, 4, 8, 2, b.d), dtype=torch.uint8, device="cuda")
            i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
            ctx, new, head = i(b.seq - np.diff(b.cu)), i(np.diff(b.cu)), i([0])
            # the new tokens' keys and values are in their places: appending them again changes nothing
            slots = [int(b.table[r, t // 128]) * 128 + t % 128 for r, (s, m) in enumerate(zip(b.own, b.new)) for t in range(s - m, s)]
            k, v = (x.transpose(1, 2).reshape(-1, 2, b.d)[slots].clone() for x in (a["k_pages"], a["v_pages"]))
            held, outs = (b.seq - np.diff(b.cu) + 127) // 128, []
            free = i([int(x) for r in range(4) for x in b.table[r, held[r]:pages_of(b.own[r])]])
            torch.cuda.synchronize()
            with torch.cuda.stream(stream):
                for _ in range(100):
                    table = a["block_table"].clone()
                    for r in range(4):
                        table[r, int(held[r]):] = -1
                    seq, cu, slot_map, _ = fa.page_plan(ctx, new, free, head, table, n, a["k_pages"].shape[0])
                    fa.fa_kv_append(k, v, slot_map, a["k_pages"], a["v_pages"])
                    o, lse = torch.empty_like(a["o"]), torch.empty_like(a["lse"])
                    args = {**a, "block_table": table, "seq_lens": seq, "cu_new": cu, "o": o, "lse": lse}
                    fa.fa_fwd_prefix_paged(**args, causal=True, scale=b.d ** -0.5, workspace=ws)
                    outs.append((o, lse))
                stream.synchronize()
            assert slot_map.tolist() == slots
            b.check(*outs[0], label=f"thread d{b.d}")
            assert all(torch.equal(o, outs[0][0]) and torch.equal(lse, outs[0][1]) for o, lse in outs)
        except BaseException as e:  # noqa: BLE001
            failures.append(e)

    threads = [threading.Thread(target=work, args=(b,)) for b in pair]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if failures:
        raise failures[0]
    assert fa.fa_device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("requests", [18, 19, 37, 38, 128, 129])
def test_both_sides_of_the_joins_borders(d, requests):
    """Decoding batches whose rows are just few enough, and just too many, for the early start and for each join."""
    b = Batch(d, 32, 8, 400, [(37 * i) % 250 + 1 for i in range(requests)], [1] * requests, pad=1, seed=47)
    o, lse = b.run()
    check_rows(b, o, lse, sorted({*range(0, requests, 5), requests - 1}), [0, 13, 31], f"{requests} requests d{d}")


def test_values_that_are_all_nan():
    """Every row that sees a key is NaN, its statistics are those of the scores, and a row that sees none is still 0."""
    import torch

    import exact_io_aware_07_gb300 as fa

    b = Batch(64, 8, 2, 0, [300, 9, 2], [280, 2, 5], seed=48)
    o0, lse0 = b.run()
    a = b.device()
    a["v_pages"].fill_(float("nan"))
    fa.fa_fwd_prefix_paged(**a, causal=True, scale=0.125)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == 0
    empty = torch.isneginf(lse0)
    assert torch.equal(a["lse"], lse0) and int(empty.sum()) == 3 * 8
    assert bool((a["o"][empty] == 0).all()) and bool(a["o"][~empty].isnan().all())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("requests", [1, 100, 600])  # each of the joins
def test_a_nan_that_a_row_sees_reaches_it_however_small_its_weight(d, requests):
    """Own keys whose scores are 600 below the prefix's: their part's weight is 0 in 32 bits, its NaN is one all the same."""
    import torch

    import exact_io_aware_07_gb300 as fa

    b = Batch(d, 8, 2, 140, [3] * requests, [1] * requests, pad=1, seed=49)
    b.q[:] = bits(1.0)
    b.k[b.prefix_table[:2]] = bits(300.0 / d)
    b.k[b.table[:, 0]] = bits(-300.0 / d)
    o0, lse0 = b.run(scale=1.0)
    b.check(o0, lse0, scale=1.0, label="prefix alone matters")
    b.v[b.table[0, 0], 1, 0, 5] = NAN_BITS
    a = b.device()
    fa.fa_fwd_prefix_paged(**a, causal=True, scale=1.0)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == 0 and torch.equal(a["lse"], lse0)
    assert bool(a["o"][0, 4:, 5].isnan().all())
    a["o"][0, 4:, 5] = o0[0, 4:, 5]
    assert torch.equal(a["o"], o0)
