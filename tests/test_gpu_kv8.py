"""8-bit KV caches: bytes, exponents and values against the definition, bit for bit."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def _rows(seed, layers, slots, heads, dim):
    """Rows of many magnitudes, with the format's corners among them."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(layers, slots, heads, dim, generator=g)
    x = x * torch.exp(6 * torch.randn(layers, slots, heads, 1, generator=g))
    x = x.to(torch.bfloat16)
    flat = x.view(-1, dim)
    corners = [torch.zeros(dim), torch.full((dim,), -0.0), torch.full((dim,), 448.0), torch.full((dim,), 449.0),
               torch.full((dim,), 450.0), torch.full((dim,), 2.0 ** -133), torch.full((dim,), 3.3e38),
               torch.linspace(-448, 448, dim), torch.ldexp(torch.ones(dim), -torch.arange(dim) % 40),
               torch.full((dim,), 2.0 ** -117), torch.full((dim,), 1.75 * 2.0 ** -116)]
    corners[2][0], corners[3][1], corners[4][0] = 17.0, 2.0 ** -10, 2.0 ** -9
    odd = torch.randn(dim, generator=g)
    odd[3], odd[5], odd[7] = math.nan, math.inf, -math.inf
    corners.append(odd)
    corners.append(torch.full((dim,), math.nan))
    corners.append(torch.full((dim,), math.inf))
    for i, c in enumerate(corners):
        if i < flat.shape[0]:
            flat[(7 * i) % flat.shape[0]] = c.to(torch.bfloat16)
    return x


def _same(a, b):
    return np.array_equal(np.asarray(a, dtype=np.float64), np.asarray(b, dtype=np.float64), equal_nan=True)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [None, 64, 128])
@pytest.mark.parametrize("slot0,slots", [(0, 1), (0, 16), (0, 64), (3, 1), (5, 29), (15, 2), (60, 70), (0, 200)])
def test_import_and_export(dim, page, slot0, slots):
    from _attend_util import head_model, rows8
    from speculative_decoding_verify_04_gb300 import spec
    layers, heads = 3, 3
    m = head_model(heads, heads, dim, layers=layers, max_batch=2)
    kv = spec.KVCache(m, 2, 203, page=page, q8=True)
    before = [kv.export_rows(0, 0, layers, 0, 203)] if page is None else None
    k, v = _rows(1, layers - 1, slots, heads, dim), _rows(2, layers - 1, slots, heads, dim)
    kv.import_rows(1, 1, k.cuda(), v.cuda(), slot0=slot0)
    gk, gv = kv.export_rows(1, 1, layers - 1, slot0, slots)
    (ck, ek, wk), (cv, ev, wv) = rows8(k.double().numpy()), rows8(v.double().numpy())
    assert _same(gk.double().cpu(), wk) and _same(gv.double().cpu(), wv)
    # the bytes and exponents themselves, through the page table
    table = kv.page_table()
    size = page or 256
    for layer in (1, 2):
        for slot in {slot0, slot0 + slots // 2, slot0 + slots - 1}:
            pg = table[1][slot // size]
            for which, code in ((0, ck), (1, cv), (2, ek), (3, ev)):
                got = kv.read_page(which, layer, pg).numpy()[:, slot % size]
                assert np.array_equal(got, code[layer - 1, slot - slot0]), (which, layer, slot)
    if before is not None:
        after = kv.export_rows(0, 0, layers, 0, 203)          # the other sequence and layer 0 are untouched
        assert torch.equal(before[0][0], after[0]) and torch.equal(before[0][1], after[1])
    assert m.device_error() == 0


def test_rows_at_odd_addresses():
    """Buffers that start one element past a 16-byte boundary."""
    from _attend_util import head_model, rows8
    from speculative_decoding_verify_04_gb300 import spec
    m = head_model(2, 2, 64)
    kv = spec.KVCache(m, 1, 40, q8=True)
    x = _rows(3, 1, 33, 2, 64)
    flat = torch.empty(x.numel() + 1, dtype=torch.bfloat16, device="cuda")
    flat[1:] = x.flatten().cuda()
    kv.import_rows(0, 0, flat[1:].view(x.shape), flat[1:].view(x.shape))
    k, v = kv.export_rows(0, 0, 1, 0, 33)
    want = rows8(x.double().numpy())[2]
    assert _same(k.double().cpu(), want) and _same(v.double().cpu(), want)
    out = torch.zeros(x.numel() + 2, dtype=torch.bfloat16, device="cuda")
    lib = spec.load()
    view = out[1:-1]
    spec._check(lib.spec_kv_export(kv.handle, 0, 0, 1, 0, 33, spec._ptr(view), spec._ptr(view), spec._stream()))
    assert _same(view.double().cpu().view(x.shape), want) and out[0] == 0 and out[-1] == 0


def test_a_second_write_replaces_the_row():
    from _attend_util import head_model
    from speculative_decoding_verify_04_gb300 import spec
    m = head_model(1, 1, 128)
    kv = spec.KVCache(m, 1, 16, q8=True)
    big = torch.full((1, 16, 1, 128), 1e20, dtype=torch.bfloat16, device="cuda")
    kv.import_rows(0, 0, big, big)
    small = torch.full((1, 1, 1, 128), 1e-20, dtype=torch.bfloat16, device="cuda")
    kv.import_rows(0, 0, small, small, slot0=7)
    k, _ = kv.export_rows(0, 0, 1, 0, 16)
    k = k.float().cpu()[0, :, 0, 0]
    assert abs(k[7] / 1e-20 - 1) <= 2.0 ** -4 + 2.0 ** -8 and (k[:7] > 9e19).all() and (k[8:] > 9e19).all()


def test_exact_values_come_back_exactly():
    """Rows that already are e4m3 values times a power of two survive."""
    from _attend_util import head_model
    from speculative_decoding_verify_04_gb300 import spec
    m = head_model(2, 2, 64)
    kv = spec.KVCache(m, 1, 64, q8=True)
    g = torch.Generator().manual_seed(4)
    x = torch.randint(0, 127, (1, 64, 2, 64), generator=g).to(torch.uint8).view(torch.float8_e4m3fn).float()
    x[..., 0] = 448.0
    x = (x * torch.exp2(torch.randint(-60, 60, (1, 64, 2, 1), generator=g).float())).to(torch.bfloat16).cuda()
    kv.import_rows(0, 0, x, x)
    k, v = kv.export_rows(0, 0, 1, 0, 64)
    assert torch.equal(k, x) and torch.equal(v, x)


def test_tree_commit_moves_rows_with_their_exponents():
    from _attend_util import head_model, rows8
    from speculative_decoding_verify_04_gb300 import spec
    for page in (None, 64):
        m = head_model(2, 2, 64, layers=2, max_batch=2)
        kv = spec.KVCache(m, 2, 100, page=page, q8=True)
        x = _rows(5, 2, 70, 2, 64)
        kv.import_rows(1, 0, x.cuda(), x.cuda())
        kv.set_lengths([0, 60])
        kv.import_rows(1, 0, x[:, 60:].contiguous().cuda(), x[:, 60:].contiguous().cuda(), slot0=60)
        path = torch.zeros(2, 64, dtype=torch.int32, device="cuda")
        path[1, :4] = torch.tensor([0, 2, 5, 9])
        spec.kv_commit(kv, torch.tensor([0, 3], dtype=torch.int32, device="cuda"), path)
        assert kv.get_lengths() == [1, 64]
        k, v = kv.export_rows(1, 0, 2, 0, 64)
        want = rows8(x.double().numpy())[2]
        want = np.concatenate([want[:, :61], want[:, [62, 65, 69]]], 1)
        assert _same(k.double().cpu(), want) and _same(v.double().cpu(), want)


def test_pages_run_out():
    from _attend_util import head_model
    from speculative_decoding_verify_04_gb300 import spec
    m = head_model(2, 2, 64, max_batch=3)
    kv = spec.KVCache(m, 3, 256, page=64, n_pages=5, q8=True)
    kv.set_lengths([64, 65, 128])
    assert kv.free_pages() == 0 and m.device_error() == 0
    assert kv.page_table() == [[0, -1, -1, -1], [1, 2, -1, -1], [3, 4, -1, -1]]
    kv.set_lengths([65, 65, 128])
    assert m.device_error() == spec.DEVERR_CAPACITY
    kv.set_lengths([64, 0, 200])
    assert m.device_error() == 0 and kv.free_pages() == 0
    assert sorted(p for row in kv.page_table() for p in row if p >= 0) == [0, 1, 2, 3, 4]


def test_many_sequences_take_pages_in_order():
    """More (sequence, block) pairs than the allocating block looks at in one step."""
    from _attend_util import head_model
    from speculative_decoding_verify_04_gb300 import spec
    B, blocks = 200, 9
    m = head_model(1, 1, 64, max_batch=B)
    kv = spec.KVCache(m, B, blocks * 64, page=64, q8=True)
    lens = [(37 * b) % (blocks * 64 + 1) for b in range(B)]
    kv.set_lengths(lens)
    want, at = [], 0
    for n in lens:
        need = -(-n // 64)
        want.append(list(range(at, at + need)) + [-1] * (blocks - need))
        at += need
    assert kv.page_table() == want and m.device_error() == 0
    assert kv.free_pages() == B * blocks - at
    # nothing missing, then a few more blocks here and there: the next pages, in the sequences' order
    kv.set_lengths(lens)
    assert kv.page_table() == want
    more = [min(blocks * 64, n + 64) if b % 3 == 0 else n for b, n in enumerate(lens)]
    kv.set_lengths(more)
    for row, n in zip(want, more):
        for p in range(-(-n // 64)):
            if row[p] < 0:
                row[p], at = at, at + 1
    assert kv.page_table() == want and m.device_error() == 0


def test_refusals():
    from _attend_util import head_model
    from speculative_decoding_verify_04_gb300 import spec
    m = head_model(1, 1, 64)
    for kw, match in ((dict(page=63), "power of two"), (dict(page=96), "power of two"), (dict(page=32), "power of two"),
                      (dict(page=64, n_pages=-1), "n_pages")):
        with pytest.raises(spec.SpecError, match=match):
            spec.KVCache(m, 1, 100, q8=True, **kw)
    with pytest.raises(spec.SpecError, match="bad sizes"):
        spec.KVCache(m, 1, 0, q8=True)
    kv = spec.KVCache(m, 1, 100, q8=True)
    x = torch.zeros(1, 8, 1, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(spec.SpecError, match="outside the cache"):
        kv.import_rows(0, 0, x, x, slot0=93)
    with pytest.raises(spec.SpecError, match="need a contiguous"):
        kv.import_rows(0, 0, x.float(), x.float())
    with pytest.raises(spec.SpecError, match="out of range"):
        kv.read_page(4, 0, 0)
    with pytest.raises(spec.SpecError, match="out of range"):
        spec.KVCache(m, 1, 100).read_page(2, 0, 0)
