"""The paged-cache step without a GPU: argument checks of its entry points, and pins of its oracle."""
import ctypes

import numpy as np
import pytest

import exact_io_aware_07_gb300 as fa
import oracle
from oracle import paged

A = 0x100000  # fake, aligned addresses: every check below fails (or stops at the device) before one is touched


@pytest.fixture(scope="module")
def lib():
    fa.build()
    return fa.load_library()


def _plan(lib, **kw):
    a = dict(ctx=A, new=A + 0x1000, free=A + 0x2000, head=A + 0x3000, table=A + 0x4000, seq=A + 0x8000, cu=A + 0x9000,
             slots=A + 0xA000, head_out=A + 0xB000, B=4, max_pages=8, num_pages=64, num_free=16, max_tokens=32)
    a.update(kw)
    return lib.fa_page_plan(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    *[({n: 0}, 1) for n in ("ctx", "new", "free", "head", "table", "seq", "cu", "slots", "head_out")],
    *[({n: A + 0x1002}, 2) for n in ("ctx", "new", "free", "head", "table", "seq", "cu", "slots", "head_out")],
    (dict(B=0), 3), (dict(max_pages=0), 3), (dict(num_pages=0), 3), (dict(num_free=-1), 3), (dict(max_tokens=0), 3),
    (dict(B=1 << 14, max_pages=1 << 10), 3), (dict(num_pages=1 << 24), 3),
])
def test_page_plan_refusals(lib, kw, code):
    assert _plan(lib, **kw) == code


def test_page_plan_without_free_pages_needs_no_list(lib):
    assert _plan(lib, free=0, num_free=0) in (6, 10)


def _append(lib, **kw):
    a = dict(k=A, v=A + 0x10000, slots=A + 0x20000, kp=A + 0x30000, vp=A + 0x80000, N=3, Hkv=2, d=64, ks=128, vs=128,
             num_pages=4)
    a.update(kw)
    return lib.fa_kv_append(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    *[({n: 0}, 1) for n in ("k", "v", "slots", "kp", "vp")],
    *[({n: A + 8}, 2) for n in ("k", "v", "kp", "vp")], (dict(slots=A + 2), 2),
    (dict(N=0), 3), (dict(Hkv=0), 3), (dict(num_pages=0), 3), (dict(num_pages=1 << 24), 3),
    (dict(d=96), 4), (dict(ks=132), 2), (dict(vs=130), 2), (dict(ks=120), 3), (dict(vs=-128), 3), (dict(vs=0), 3),
])
def test_kv_append_refusals(lib, kw, code):
    assert _append(lib, **kw) == code


def test_kv_append_of_one_token_takes_any_stride(lib):
    assert _append(lib, N=1, ks=0, vs=-5) in (6, 10)


def _attend(lib, **kw):
    a = dict(q=A, kp=A + 0x10000, vp=A + 0x20000, pt=A + 0x30000, bt=A + 0x31000, seq=A + 0x32000, cu=A + 0x33000,
             o=A + 0x40000, lse=A + 0x50000, N=3, B=2, H=4, Hkv=2, d=64, prefix_len=300, max_new=2, causal=1,
             scale=0.125, num_pages=16, max_pages=4, ws=A + 0x1000000, ws_bytes=1 << 40)
    a.update(kw)
    a["scale"] = ctypes.c_float(a["scale"])
    return lib.fa_fwd_prefix_paged(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    *[({n: 0}, 1) for n in ("q", "kp", "vp", "pt", "bt", "seq", "cu", "o", "lse")],
    *[({n: A + 8}, 2) for n in ("q", "kp", "vp", "o", "lse", "ws")], *[({n: A + 2}, 2) for n in ("pt", "bt", "seq", "cu")],
    (dict(N=0), 3), (dict(B=0), 3), (dict(H=0), 3), (dict(Hkv=0), 3), (dict(H=5), 3), (dict(prefix_len=-1), 3),
    (dict(max_new=0), 3), (dict(num_pages=0), 3), (dict(max_pages=0), 3), (dict(H=258), 3), (dict(num_pages=1 << 24), 3),
    (dict(N=1 << 24, H=256), 3),
    (dict(d=96), 4), (dict(scale=0.0), 5), (dict(scale=float("nan")), 5), (dict(scale=float("inf")), 5), (dict(causal=2), 9),
    (dict(ws=0), 13), (dict(ws_bytes=0), 13),
])
def test_prefix_attention_refusals(lib, kw, code):
    assert _attend(lib, **kw) == code


def test_prefix_attention_without_prefix_needs_no_table(lib):
    assert _attend(lib, pt=0, prefix_len=0) in (6, 10)
    assert _attend(lib) in (6, 10)


def test_prefix_attention_workspace_size(lib):
    size = fa.fa_fwd_prefix_paged_workspace_bytes
    assert size(3, 2, 4, 2, 64) > 0 and size(3, 2, 4, 2, 64) % 256 == 0
    assert size(1000, 2, 32, 8, 128) >= size(3, 2, 32, 8, 128)
    for bad in ((0, 2, 4, 2, 64), (3, 0, 4, 2, 64), (3, 2, 0, 2, 64), (3, 2, 4, 0, 64), (3, 2, 5, 2, 64),
                (3, 2, 4, 2, 96)):
        assert size(*bad) == 0


def _tensors(**kw):
    import torch

    i32 = dict(dtype=torch.int32)
    a = dict(q=torch.zeros(3, 4, 64, dtype=torch.bfloat16), k_pages=torch.zeros(5, 2, 128, 64, dtype=torch.bfloat16),
             v_pages=torch.zeros(5, 2, 128, 64, dtype=torch.bfloat16), prefix_table=torch.zeros(2, **i32),
             prefix_len=200, block_table=torch.zeros(2, 3, **i32), seq_lens=torch.ones(2, **i32),
             cu_new=torch.zeros(3, **i32), max_new=1, o=torch.zeros(3, 4, 64, dtype=torch.bfloat16),
             lse=torch.zeros(3, 4), causal=True, scale=0.125)
    a.update(kw)
    return a


def test_binding_refuses_wrong_tensors(lib):
    import torch

    bad = [dict(q=torch.zeros(3, 4, 64)), dict(q=torch.zeros(3, 64, 4, dtype=torch.bfloat16).transpose(1, 2)),
           dict(k_pages=torch.zeros(5, 2, 64, 64, dtype=torch.bfloat16)), dict(v_pages=torch.zeros(5, 2, 128, 64)),
           dict(prefix_table=torch.zeros(1, dtype=torch.int32)), dict(prefix_table=torch.zeros(2, dtype=torch.int64)),
           dict(prefix_table=None), dict(block_table=torch.zeros(3, dtype=torch.int32)),
           dict(block_table=torch.zeros(3, 2, dtype=torch.int32).t()), dict(seq_lens=torch.ones(3, dtype=torch.int32)),
           dict(cu_new=torch.zeros(2, dtype=torch.int32)), dict(lse=torch.zeros(4, 3)),
           dict(o=torch.zeros(3, 4, 128, dtype=torch.bfloat16)),
           dict(workspace=torch.zeros(1, dtype=torch.uint8).expand(2 ** 30))]
    for kw in bad:
        with pytest.raises(ValueError):
            fa.fa_fwd_prefix_paged(**_tensors(**kw))
    pool = torch.zeros(5, 2, 128, 64, dtype=torch.bfloat16)
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int32)
    for args in ((k.float(), k, slots), (k[:2], k, slots), (k, k, slots.long()), (k, k, slots[:2]),
                 (k.transpose(1, 2).contiguous().transpose(1, 2), k, slots),
                 (torch.zeros(3, 4, 64, dtype=torch.bfloat16)[:, ::2], k, slots)):
        with pytest.raises(ValueError):
            fa.fa_kv_append(*args, pool, pool)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    good = dict(ctx_lens=i(2), new_lens=i(2), free_pages=i(4), free_head=i(1), block_table=i(2, 3), seq_lens=i(2),
                cu_new=i(3), slot_map=i(5), free_head_out=i(1), num_pages=8)
    for kw in (dict(ctx_lens=i(3)), dict(new_lens=i(2).long()), dict(free_head=i(2)), dict(block_table=i(6)),
               dict(cu_new=i(2)), dict(slot_map=i(5, 1)), dict(slot_map=i(10)[::2]), dict(seq_lens=i(2).float())):
        with pytest.raises(ValueError):
            fa.fa_page_plan(**{**good, **kw})


# ---------------------------------------------------------------- the oracle against other definitions

def test_oracle_plan_by_hand():
    # a request of 127 fills its page with one token and opens page 9; a new request opens page 4
    table, seq, cu, slots, head = paged.page_plan([127, 0], [2, 1], [7, 9, 4], 1, [[3, -1], [-1, -1]], 5)
    assert table.tolist() == [[3, 9], [4, -1]] and seq.tolist() == [129, 1] and cu.tolist() == [0, 2, 3]
    assert slots.tolist() == [3 * 128 + 127, 9 * 128, 4 * 128, -1, -1] and head == 3


def test_oracle_append_by_hand():
    pages = np.zeros((2, 1, 128, 2))
    out = paged.kv_append(np.array([[[1.0, 2.0]], [[3.0, 4.0]], [[5.0, 6.0]]]), [130, -1, 0], pages)
    assert out[1, 0, 2].tolist() == [1, 2] and out[0, 0, 0].tolist() == [5, 6] and np.abs(out).sum() == 14


@pytest.mark.parametrize("causal", [0, 1])
def test_oracle_attention_is_attention_on_the_joined_keys(causal):
    """Prefix and own keys side by side, all rows new: plain causal attention of the joined sequence's last rows."""
    rng = np.random.default_rng(0)
    P, T, H, Hkv, d, scale = 130, 5, 4, 2, 8, 0.3
    pages = rng.standard_normal((2, 4, Hkv, 128, d))
    q = rng.standard_normal((T, H, d))
    pt, bt = [2, 0], [[3]]
    O, lse, _, _ = paged.attention_prefix_paged(q, pages[0], pages[1], pt, P, bt, [T], [0, T], causal, scale)
    k, v = (np.concatenate([paged.gather(x, pt, P), paged.gather(x, bt[0], T)]).transpose(1, 0, 2) for x in pages)
    full = np.zeros((1, H, P + T, d))
    full[0, :, P:] = q.transpose(1, 0, 2)
    O2, lse2 = oracle.attention_fwd_gqa(full, k[None], v[None], causal, scale)
    assert np.abs(O - O2[0, :, P:].transpose(1, 0, 2)).max() < 1e-12
    assert np.abs(lse - lse2[0, :, P:].T).max() < 1e-12


def test_oracle_empty_row():
    o, lse, spread, _ = paged.row(np.ones(4), np.zeros((0, 4)), np.zeros((0, 4)), 1.0)
    assert not o.any() and lse == -np.inf and not spread.any()


@pytest.mark.parametrize("N,d,stride", [
    (2 ** 24 + 1, 64, 2 ** 40),      # (N - 1) * stride is 2^64: nothing in 64 bits
    (2 ** 24 + 1, 128, 2 ** 39),     # as many bytes
    (2 ** 25 + 1, 64, 2 ** 39),
    (2 ** 30 + 1, 64, 2 ** 34),
    (2 ** 20 + 1, 64, 2 ** 40),      # 2^60 elements: no such memory
])
@pytest.mark.parametrize("which", ["ks", "vs"])
def test_kv_append_refuses_rows_past_any_memory(lib, N, d, stride, which):
    """Rows so far apart that the extent of the new keys or values does not fit 64 bits must not pass for a short one."""
    far = A * 2 ** 20  # the pool and the slots are clear of the other arguments
    kw = dict(slots=far, kp=2 * far, vp=3 * far, N=N, Hkv=1, d=d, ks=d, vs=d)
    assert _append(lib, **{**kw, which: stride}) == 3
    assert _append(lib, **kw) in (6, 10)  # rows side by side: up to the device


@pytest.mark.parametrize("sizes", [
    (1, 1, 258, 2, 64),                    # 129 query heads of one K/V head
    (1 << 24, 1, 256, 128, 64),            # 2^32 rows
    (2 ** 31 - 1, 1, 2, 2, 128),
    (2 ** 31 - 1, 1, 2 ** 31 - 1, 2 ** 31 - 1, 128),  # a size that does not fit 64 bits
])
def test_prefix_attention_workspace_size_is_0_out_of_range(lib, sizes):
    """Sizes that the call refuses whatever its other arguments have no workspace."""
    N, B, H, Hkv, d = sizes
    assert _attend(lib, N=N, B=B, H=H, Hkv=Hkv, d=d) == 3
    assert fa.fa_fwd_prefix_paged_workspace_bytes(*sizes) == 0
