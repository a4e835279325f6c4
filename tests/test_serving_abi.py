"""Host-side checks of the calls on ragged batches of new tokens and on pages: bad arguments are
refused before any launch, and the prefill plan follows its cost rule (no GPU is touched)."""
import ctypes
import random

import pytest

from tests.test_abi import FAKE, Dims, _dims, _kv, lib  # noqa: F401

I64, SZ = ctypes.c_int64, ctypes.c_size_t
WS = (FAKE, SZ(256))
SLOTS = I64(16 * 64)


class Pool(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("seqlens", ctypes.c_void_p), ("page_refs", ctypes.c_void_p),
                ("batch", ctypes.c_int), ("max_pages_per_seq", ctypes.c_int), ("page_size", ctypes.c_int),
                ("num_pages", ctypes.c_int)]


def _pool(batch=2, page_size=64, num_pages=16, refs=FAKE):
    return Pool(FAKE, FAKE, refs, batch, 4, page_size, num_pages)


def off(n):
    return ctypes.c_void_p((1 << 20) + n)


def _prefill(lib, d=None, q=FAKE, total=8, starts=FAKE, kv=FAKE, kr=FAKE, slots=SLOTS, idx=None, splits=4, o=FAKE, l=FAKE,
             out=FAKE, ws=WS):
    d = _dims() if d is None else d
    return lib.gqla_prefill_gqa(d if d == 0 else ctypes.byref(d), q, I64(total), starts, kv, kr, slots,
                                ctypes.byref(_kv() if idx is None else idx), splits, o, l, out, None, *ws, None)


@pytest.mark.parametrize("change,expected", [
    (dict(q=None), -1), (dict(starts=None), -1), (dict(kv=None), -1), (dict(kr=None), -1), (dict(out=None), -1),
    (dict(o=None), -1), (dict(l=None), -1), (dict(splits=0), -1), (dict(splits=65536), -1), (dict(splits=-65536), -1),
    (dict(total=-1), -1), (dict(total=1 << 31), -2), (dict(slots=I64(17)), -1), (dict(q=off(8)), -1), (dict(o=off(4)), -1),
    (dict(l=off(8)), -1), (dict(out=off(2)), -1), (dict(ws=(None, SZ(256))), -3), (dict(ws=(FAKE, SZ(8))), -3),
    (dict(idx=_kv(batch=0)), -1), (dict(idx=_kv(page_size=32)), -2), (dict(idx=_kv(batch=65536)), -2),
    (dict(d=_dims(h=100)), -1), (dict(d=_dims(h=0)), -1), (dict(d=_dims(lat=256)), -2), (dict(d=_dims(scale=float("inf"))), -1),
    (dict(d=_dims(h=258, g=2)), -2), (dict(total=0), 0), (dict(total=0, splits=-3, o=None, l=None), 0),
    (dict(total=0, splits=1, o=None, l=None), 0), (dict(total=0, d=_dims(h=15, g=5)), 0),
])
def test_prefill_rejects_bad_arguments(lib, change, expected):
    assert _prefill(lib, **change) == expected


def _append(lib, d=None, rows=FAKE, total=8, starts=FAKE, wk=FAKE, wv=FAKE, lat=FAKE, kv=FAKE, kr=FAKE, slots=SLOTS,
            idx=None, ws=WS):
    return lib.gqla_append_cache(ctypes.byref(_dims() if d is None else d), rows, I64(total), starts, wk, wv, lat, kv,
                                 kr, slots, ctypes.byref(_kv() if idx is None else idx), *ws, None)


@pytest.mark.parametrize("change,expected", [
    (dict(rows=None), -1), (dict(starts=None), -1), (dict(wk=None), -1), (dict(wv=None), -1), (dict(kv=None), -1),
    (dict(kr=None), -1), (dict(lat=None, kv=None, kr=None), -1), (dict(total=-1), -1), (dict(total=1 << 31), -2),
    (dict(rows=off(8)), -1), (dict(lat=off(8)), -1), (dict(kr=off(8)), -1), (dict(slots=I64(5)), -1),
    (dict(ws=(FAKE, SZ(255))), -3), (dict(idx=_kv(page_size=16)), -2), (dict(total=0), 0), (dict(total=0, lat=None), 0),
    (dict(total=0, wk=None, wv=None, kv=None, kr=None), 0),
])
def test_append_rejects_bad_arguments(lib, change, expected):
    assert _append(lib, **change) == expected


def test_page_calls_reject_bad_arguments(lib):
    d, p = ctypes.byref(_dims()), _pool()
    copy = lambda pairs=FAKE, n=2, pages=16, lat=FAKE, kv=FAKE, kr=FAKE, ws=WS: lib.gqla_copy_pages(  # noqa: E731
        d, pairs, I64(n), pages, lat, kv, kr, *ws, None)
    assert copy(pairs=None) == copy(n=-1) == copy(pages=0) == copy(lat=None, kv=None, kr=None) == -1
    assert copy(pairs=off(4)) == copy(lat=off(8)) == copy(kv=off(8)) == copy(kr=off(8)) == -1
    assert copy(pages=(1 << 19) + 1) == copy(n=1 << 31) == -2
    assert copy(ws=(None, SZ(256))) == -3 and copy(n=0) == 0
    P = ctypes.byref(p)
    assert lib.gqla_fork_sequences(None, FAKE, 1, FAKE, *WS, None) == -1
    assert lib.gqla_fork_sequences(P, None, 1, FAKE, *WS, None) == -1
    assert lib.gqla_fork_sequences(P, FAKE, 1, None, *WS, None) == -1
    assert lib.gqla_fork_sequences(P, FAKE, -1, FAKE, *WS, None) == -1
    assert lib.gqla_fork_sequences(P, off(4), 1, FAKE, *WS, None) == -1
    assert lib.gqla_fork_sequences(P, FAKE, 65536, FAKE, *WS, None) == -2
    assert lib.gqla_fork_sequences(P, FAKE, 0, FAKE, *WS, None) == 0
    assert lib.gqla_extend_sequences(P, None, *WS, None) == -1
    assert lib.gqla_extend_sequences(P, FAKE, FAKE, SZ(4), None) == -3
    assert lib.gqla_free_sequences(P, None, 1, *WS, None) == -1
    assert lib.gqla_free_sequences(P, FAKE, -2, *WS, None) == -1
    assert lib.gqla_free_sequences(P, FAKE, 65536, *WS, None) == -2
    assert lib.gqla_free_sequences(P, FAKE, 0, *WS, None) == 0
    assert lib.gqla_compact_pages(P, None, FAKE, FAKE, FAKE, *WS, None) == -1
    assert lib.gqla_compact_pages(P, FAKE, FAKE, off(4), FAKE, *WS, None) == -1
    assert lib.gqla_compact_pages(P, FAKE, FAKE, FAKE, None, *WS, None) == -1
    for bad, st in ((_pool(batch=0), -1), (_pool(num_pages=0), -1), (_pool(refs=None), -1), (_pool(page_size=32), -2),
                    (_pool(batch=65536), -2)):
        B = ctypes.byref(bad)
        assert lib.gqla_fork_sequences(B, FAKE, 1, FAKE, *WS, None) == st
        assert lib.gqla_extend_sequences(B, FAKE, *WS, None) == st
        assert lib.gqla_free_sequences(B, FAKE, 1, *WS, None) == st
        assert lib.gqla_compact_pages(B, FAKE, FAKE, FAKE, FAKE, *WS, None) == st


# ------------------------------------------------------------------ the prefill plan

BLOCK_COST, MIN_CHUNK, MERGE_COST = 5, 8, 5


def _blocks(h, g, new, lens):
    """Cost units of every query block, in plan order."""
    T, out = 128 // (h // g), []
    for n, L in zip(new, lens):
        for _ in range(g):
            for first in range(0, n, 4 * T):
                tok = min(4 * T, n - first)
                out.append((2 if tok > 2 * T else 1) * -(-(L - n + first + tok) // 128) + BLOCK_COST)
    return out


def _plan_by_hand(h, g, new, lens, most):
    units = _blocks(h, g, new, lens)
    total = sum(units)
    if not total:
        return -1
    div = max(1, min(most, total // MIN_CHUNK))
    whole = min(most, len(units))
    k, loads, at = max(2, -(-total // whole)), {}, 0
    for u in units:
        loads[at // k] = loads.get(at // k, 0) + u
        at += u
    return -whole if div == 1 or max(loads.values()) <= max(2, -(-total // div)) + MERGE_COST else div


def _plan(lib, h, g, new, lens, most):
    arr = lambda v: (ctypes.c_int32 * len(v))(*v)  # noqa: E731
    n = ctypes.c_int(0)
    st = lib.gqla_plan_prefill(ctypes.byref(_dims(h, g)), arr(new), arr(lens), len(new), most, ctypes.byref(n))
    return n.value if st == 0 else ("error", st)


def test_plan_prefill_matches_the_rule(lib):
    rng = random.Random(3)
    for _ in range(150):
        h, g = rng.choice([(32, 8), (128, 8), (128, 4), (24, 2), (8, 8), (128, 1)])
        B = rng.randint(1, 12)
        new = [rng.choice([0, 1, rng.randint(1, 40), rng.randint(1, 300)]) for _ in range(B)]
        lens = [n + rng.choice([0, rng.randint(0, 3000)]) for n in new]
        most = rng.choice([1, 5, 74])
        if len(_blocks(h, g, new, lens)) <= 4096:
            assert _plan(lib, h, g, new, lens, most) == _plan_by_hand(h, g, new, lens, most), (h, g, new, lens, most)


def test_plan_prefill_edges(lib):
    assert _plan(lib, 128, 8, [0, 0], [5, 0], 74) == -1          # nothing to do: one (empty) chunk
    assert _plan(lib, 32, 8, [5], [256], 74) == -8               # one block to a group, none divided
    assert _plan(lib, 128, 8, [8192], [8192], 74) == 74          # many blocks: equal shares
    assert _plan(lib, 128, 8, [1], [100000], 74) == 74           # one long block to a group: divided
    assert _plan(lib, 128, 8, [1 << 20], [1 << 20], 74) == 74    # too many blocks to walk
    assert _plan(lib, 128, 8, [3], [2], 74) == ("error", -1)
    assert _plan(lib, 128, 8, [-1], [2], 74) == ("error", -1)
    assert _plan(lib, 128, 8, [1], [2], 0) == ("error", -1)
    assert _plan(lib, 258, 2, [1], [2], 74) == ("error", -2)
    n = ctypes.c_int(0)
    arr = (ctypes.c_int32 * 1)(1)
    assert lib.gqla_plan_prefill(ctypes.byref(_dims()), None, arr, 1, 4, ctypes.byref(n)) == -1
    assert lib.gqla_plan_prefill(ctypes.byref(_dims()), arr, arr, 1, 4, None) == -1
    assert lib.gqla_plan_prefill(None, arr, arr, 1, 4, ctypes.byref(n)) == -1


def test_prefill_slots(lib):
    assert lib.gqla_prefill_slots(74) == 2 * 74 + 1
    assert lib.gqla_prefill_slots(129) == 2 * 129 + 2
    assert lib.gqla_prefill_slots(1) == lib.gqla_prefill_slots(-7) == 0
    assert lib.gqla_prefill_slots(0) == lib.gqla_prefill_slots(65536) == lib.gqla_prefill_slots(-65536) == -1


def test_pools_beyond_32_bit_page_counts_are_refused(lib):
    """Scans step 8192 pages past the last, and a row past 2^25 pages cannot be filled: both in 32 bits."""
    def calls(pages, width):
        p = _pool(num_pages=pages)
        p.max_pages_per_seq = width
        P = ctypes.byref(p)
        # calls with nothing to do, so that an accepted pool launches nothing
        return (lib.gqla_fork_sequences(P, FAKE, 0, FAKE, *WS, None), lib.gqla_free_sequences(P, FAKE, 0, *WS, None))

    most = (1 << 25) - 1
    assert calls(most, 4) == calls(16, most + 1) == calls(most, most + 1) == (0, 0)
    for pages, width in ((most + 1, 4), ((1 << 31) - 1, 4), ((1 << 31) - 8000, 4), (16, most + 2), (16, (1 << 31) - 1)):
        assert calls(pages, width) == (-2, -2)
        p = _pool(num_pages=pages)
        p.max_pages_per_seq = width
        P = ctypes.byref(p)
        assert lib.gqla_extend_sequences(P, FAKE, *WS, None) == -2
        assert lib.gqla_compact_pages(P, FAKE, FAKE, FAKE, FAKE, *WS, None) == -2


def test_index_pointers_off_their_type_are_refused(lib):
    """An int32 or float address that is no multiple of 4 would fault in the kernel: refused first, by
    calls with nothing to do (which an accepted pointer lets through), too."""
    assert _prefill(lib, total=0) == _append(lib, total=0) == 0
    assert _prefill(lib, total=0, starts=off(2)) == _append(lib, total=0, starts=off(1)) == -1
    assert _prefill(lib, total=0, starts=off(4)) == _append(lib, total=0, starts=off(4)) == 0
    d = _dims()
    assert lib.gqla_prefill_gqa(ctypes.byref(d), FAKE, I64(0), FAKE, FAKE, FAKE, SLOTS, ctypes.byref(_kv()), -1, None, None,
                                FAKE, off(2), *WS, None) == -1
    for name in ("page_table", "seqlens"):
        idx = _kv()
        setattr(idx, name, off(3))
        assert _prefill(lib, total=0, idx=idx) == _append(lib, total=0, idx=idx) == -1
    for name in ("page_table", "seqlens", "page_refs"):
        p = _pool()
        setattr(p, name, off(2))
        P = ctypes.byref(p)
        assert lib.gqla_fork_sequences(P, FAKE, 0, FAKE, *WS, None) == -1
        assert lib.gqla_free_sequences(P, FAKE, 0, *WS, None) == -1
        assert lib.gqla_extend_sequences(P, FAKE, *WS, None) == -1
        assert lib.gqla_compact_pages(P, FAKE, FAKE, FAKE, FAKE, *WS, None) == -1
    P = ctypes.byref(_pool())
    assert lib.gqla_free_sequences(P, off(2), 0, *WS, None) == -1
    assert lib.gqla_extend_sequences(P, off(2), *WS, None) == -1
    for i in range(4):
        a = [FAKE] * 4
        a[i] = off(2)
        assert lib.gqla_compact_pages(P, *a, *WS, None) == -1


def test_more_groups_than_the_grids_hold_are_refused(lib):
    many = _dims(h=4097, g=4097)
    assert _append(lib, d=many) == -2
    assert lib.gqla_copy_pages(ctypes.byref(many), FAKE, I64(1), 16, FAKE, None, None, *WS, None) == -2
    assert lib.gqla_copy_pages(ctypes.byref(_dims(h=4096, g=4096)), FAKE, I64(0), 16, FAKE, None, None, *WS, None) == 0


def test_the_binding_refuses_an_index_of_another_device(monkeypatch):
    import torch

    from decode_attention_06_b200 import gqla
    t = torch.zeros(2, dtype=torch.int32)
    pool = gqla.gqla_page_pool(FAKE, FAKE, FAKE, 2, 4, 64, 16)
    pool._keep, pool._device = (t,), 1
    monkeypatch.setattr(gqla, "_current_device", lambda: 0)
    for call in (lambda: gqla.gqla_fork_sequences(pool, t.view(1, 2), t.view(1, 2), t),
                 lambda: gqla.gqla_extend_sequences(pool, t, t), lambda: gqla.gqla_free_sequences(pool, t, t),
                 lambda: gqla.gqla_compact_pages(pool, t, t, t, t, t)):
        with pytest.raises(ValueError, match="current device is cuda:0"):
            call()
    pool._device = -1  # tensors that share no device
    with pytest.raises(ValueError, match="current device"):
        gqla.gqla_free_sequences(pool, t, t)
