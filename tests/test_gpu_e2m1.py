"""GPU parity of the 4-bit cache and of the appends with rotary positions, against the plain references of tests/_e2m1.py:
bytes and queries bit for bit, attention within tolerances derived there."""
import math

import numpy as np
import pytest
import torch

from fp8_paged_kv_e4m3_gb300 import build, kvq
from tests import _e2m1 as E
from tests._gpu import to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    kvq.load()


def _rng(*key):
    return np.random.default_rng(list(key))


def _err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _kv(rng, T, H, D):
    x = rng.standard_normal((T, H, D))
    x[..., 3] *= 20                       # an outlier channel
    return x.astype(np.float16)


def _same_bytes(got, ref, D):
    """Equal codes and scales; a block whose scale is NaN may hold any codes."""
    (gc, gb), (rc, rb) = E.unpack(got, D), E.unpack(ref, D)
    assert np.array_equal(gb, rb)
    live = np.repeat((rb & 127) != 127, 16, -1)
    assert np.array_equal(gc[live], rc[live])


# --- append and read-back --------------------------------------------------

@pytest.mark.parametrize("D,Hkv,T", [(64, 1, 1), (64, 3, 7), (128, 2, 1), (128, 4, 67), (128, 1, 300), (64, 8, 130)])
def test_append_bytes_and_untouched_slots(D, Hkv, T):
    rng = _rng(1, D, Hkv, T)
    P = T // 3 + 3
    slots = rng.permutation(4 * P)[:T].astype(np.int32)
    slots[::5] = -1
    k, v = _kv(rng, T, Hkv, D), _kv(rng, T, Hkv, D)
    ks, vs = (kvq.calibrate_scale_e2m1(to_dev(x)) for x in (k, v))
    assert ks == float(np.float32(np.abs(k).max()) / np.float32(2688))
    start = rng.integers(0, 256, (P, Hkv, 9 * D // 4)).astype(np.uint8)
    kc, vc, err = to_dev(start), to_dev(start), _err()
    kvq.kv_append_e2m1(to_dev(k), to_dev(v), to_dev(slots), kc, vc, ks, vs, err)
    assert np.array_equal(kc.cpu().numpy(), E.append(start, k, slots, ks))
    assert np.array_equal(vc.cpu().numpy(), E.append(start, v, slots, vs))
    assert err.item() == 0


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -9, 0.0371, 1.0 / 2688])
def test_append_every_fp16_pattern(scale):
    """All 65,536 binary16 patterns in shuffled blocks, so that small and large values share blocks; NaN and infinities
    among them."""
    x = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    for order in (x, _rng(2).permutation(x)):
        rows = order.view(np.float16).reshape(512, 1, 128)
        slots = np.arange(512, dtype=np.int32)
        kc = kvq.alloc_e2m1_pool(128, 1, 128)
        vc = kvq.alloc_e2m1_pool(128, 1, 128)
        kvq.kv_append_e2m1(to_dev(rows), to_dev(-rows), to_dev(slots), kc, vc, scale, scale)
        zero = np.zeros((128, 1, 288), np.uint8)
        _same_bytes(kc.cpu().numpy(), E.append(zero, rows, slots, scale), 128)
        _same_bytes(vc.cpu().numpy(), E.append(zero, -rows, slots, scale), 128)


def test_append_slots_beyond_the_pool_are_skipped():
    rng = _rng(3)
    k = _kv(rng, 4, 2, 64)
    slots = np.array([0, 40, 2 ** 31 - 1, 7], np.int32)
    kc, vc, err = kvq.alloc_e2m1_pool(10, 2, 64), kvq.alloc_e2m1_pool(10, 2, 64), _err()
    kvq.kv_append_e2m1(to_dev(k), to_dev(k), to_dev(slots), kc, vc, 0.01, 0.01, err)
    assert err.item() == kvq.DEV_BAD_SLOT
    assert np.array_equal(kc.cpu().numpy(), E.append(np.zeros((10, 2, 144), np.uint8), k, slots, 0.01))


@pytest.mark.parametrize("D", [64, 128])
def test_gather_reads_every_code_back(D):
    """Random bytes: every code, every block scale (negative and NaN ones among them), rounded to fp16 from binary32."""
    rng = _rng(4, D)
    pool = rng.integers(0, 256, (50, 3, 9 * D // 4)).astype(np.uint8)
    slots = np.concatenate([rng.permutation(200), [-1, -7, 200, 5]]).astype(np.int32)
    err = _err()
    ks, vs = np.float32(0.0123), np.float32(3.7)
    k, v = kvq.kv_gather_e2m1(to_dev(pool), to_dev(pool), to_dev(slots), float(ks), float(vs), err_flag=err)
    held = E.pool_values(pool, D).astype(np.float32)          # exact
    for got, scale in ((k, ks), (v, vs)):
        got = got.cpu().numpy()
        with np.errstate(over="ignore"):
            ref = (held * scale).astype(np.float16)
        ok = np.r_[0:200, 203]
        assert np.array_equal(got[ok], ref[slots[ok] // 4, :, slots[ok] % 4], equal_nan=True)
        assert not got[200:203].any()
    assert err.item() == kvq.DEV_BAD_SLOT


# --- rotary positions ------------------------------------------------------

@pytest.mark.parametrize("kw", [
    dict(), dict(base=500000.0), dict(scaling="linear", factor=8.0),
    dict(scaling="yarn", factor=16.0, original_positions=4096),
    dict(scaling="yarn", factor=4.0, original_positions=8192, beta_fast=16.0, beta_slow=2.0, magnitude=1.25),
])
@pytest.mark.parametrize("n,rot", [(1, 16), (4099, 64), (262144, 128)])
def test_rope_table(n, rot, kw):
    """Angles up to 262144 rad in binary64: the power's and the product's roundings (a few 2^-53 of the angle) move an entry
    by under 1e-9, its rounding to binary32 by at most half a step."""
    got = kvq.rope_table(n, rot, **kw).cpu().numpy()
    ref = E.rope_table(n, rot, kw.get("base", 10000.0), kw.get("scaling"), kw.get("factor", 1.0),
                       kw.get("original_positions", 0), kw.get("beta_fast", 32.0), kw.get("beta_slow", 1.0),
                       kw.get("magnitude", 0.0))
    assert (np.abs(got - ref) <= np.abs(ref) * 2.0 ** -24 + 1e-9).all()


def _rope_case(rng, T, Hq, Hkv, D, rot, packed, n=500):
    table = E.rope_table(n, rot).astype(np.float32)
    pos = rng.integers(0, n, T).astype(np.int32)
    x = _kv(rng, T, Hq + 2 * Hkv, D)
    dev = to_dev(x)
    q, k, v = (dev[:, a:b] if packed else dev[:, a:b].contiguous() for a, b in
               ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    return table, pos, x, q, k, v


ROPE_SHAPES = [  # T, Hq, Hkv, D, rot
    (1, 8, 2, 64, 64), (3, 4, 4, 128, 128), (130, 32, 4, 128, 64), (257, 7, 1, 128, 96), (64, 8, 2, 64, 16), (5, 1, 1, 64, 48),
]


@pytest.mark.parametrize("shape", ROPE_SHAPES + [(33, 3, 2, 96, 32), (9, 2, 1, 256, 240), (6, 5, 3, 16, 16)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kind", ["e4m3", "fp16", "e2m1"])
@pytest.mark.parametrize("packed", [False, True])
def test_append_rope_bits(kind, interleaved, shape, packed):
    """Queries and pools bit for bit: the rotation is products and sums each rounded to binary32."""
    T, Hq, Hkv, D, rot = shape
    if kind == "e2m1" and D not in (64, 128):
        pytest.skip("E2M1 pools have head_dim 64 or 128")
    rng = _rng(5, *shape)
    table, pos, x, q, k, v = _rope_case(rng, T, Hq, Hkv, D, rot, packed)
    P = T // 3 + 2
    slots = rng.permutation(4 * P)[:T].astype(np.int32)
    slots[1::4] = -1
    err = _err()
    turned = E.rotate(x[:, :Hq + Hkv], table, pos, interleaved)
    kref, vref = turned[:, Hq:], x[:, Hq + Hkv:]
    args = (q, k, v, to_dev(pos), to_dev(table), to_dev(slots))
    live = slots >= 0
    page, at = slots[live] // 4, slots[live] % 4
    if kind == "e2m1":
        kc, vc = (kvq.alloc_e2m1_pool(P, Hkv, D) for _ in range(2))
        out = kvq.kv_append_rope_e2m1(*args, kc, vc, 0.011, 0.017, interleaved=interleaved, err_flag=err)
        zero = np.zeros((P, Hkv, 9 * D // 4), np.uint8)
        assert np.array_equal(kc.cpu().numpy(), E.append(zero, kref, slots, 0.011))
        assert np.array_equal(vc.cpu().numpy(), E.append(zero, vref, slots, 0.017))
    else:
        kind_t = torch.uint8 if kind == "e4m3" else torch.float16
        kc, vc = (torch.zeros(P, Hkv, 4, D, dtype=kind_t, device="cuda") for _ in range(2))
        if kind == "e4m3":
            out = kvq.kv_append_rope_e4m3(*args, kc, vc, 0.11, 0.17, interleaved=interleaved, err_flag=err)
        else:
            out = kvq.kv_append_rope_fp16(*args, kc, vc, interleaved=interleaved, err_flag=err)
        for pool, rows, scale in ((kc, kref, 0.11), (vc, vref, 0.17)):
            ref = np.zeros(pool.shape, pool.cpu().numpy().dtype)
            if kind == "e4m3":
                y = (rows.astype(np.float32) / np.float32(scale)).astype(np.float32)
                ref[page, :, at] = (E.e4m3_encode(np.abs(y)) | (np.signbit(y) << 7))[live]
            else:
                ref[page, :, at] = rows.astype(np.float16)[live]
            assert np.array_equal(pool.cpu().numpy(), ref)
    assert np.array_equal(out.cpu().numpy(), turned[:, :Hq].astype(np.float16))
    assert err.item() == 0


def test_append_rope_without_rotation_of_values_equals_the_plain_appends():
    """At position 0 the rotation is the identity: the pools equal kv_append_*'s bit for bit."""
    rng = _rng(6)
    T, Hkv, D = 50, 2, 128
    table = kvq.rope_table(4, 128)
    k, v = to_dev(_kv(rng, T, Hkv, D)), to_dev(_kv(rng, T, Hkv, D))
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    slots = to_dev(rng.permutation(80)[:T].astype(np.int32))
    for kind in ("e4m3", "fp16", "e2m1"):
        if kind == "e2m1":
            pools = [kvq.alloc_e2m1_pool(20, Hkv, D) for _ in range(4)]
        else:
            t = torch.uint8 if kind == "e4m3" else torch.float16
            pools = [torch.zeros(20, Hkv, 4, D, dtype=t, device="cuda") for _ in range(4)]
        scales = () if kind == "fp16" else (0.02, 0.03)
        assert getattr(kvq, "kv_append_rope_" + kind)(None, k, v, pos, table, slots, *pools[:2], *scales) is None
        getattr(kvq, "kv_append_" + kind)(k, v, slots, *pools[2:], *scales)
        assert torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])


@pytest.mark.parametrize("interleaved", [False, True])
def test_append_rope_in_place(interleaved):
    rng = _rng(7)
    table, pos, x, q, k, v = _rope_case(rng, 200, 16, 2, 128, 96, False)
    slots = to_dev(rng.permutation(240)[:200].astype(np.int32))
    kc, vc = (torch.zeros(60, 2, 4, 128, dtype=torch.uint8, device="cuda") for _ in range(2))
    got = kvq.kv_append_rope_e4m3(q, k, v, to_dev(pos), to_dev(table), slots, kc, vc, 0.1, 0.1, q_out=q, interleaved=interleaved)
    assert got is q
    assert np.array_equal(q.cpu().numpy(), E.rotate(x[:, :16], table, pos, interleaved).astype(np.float16))


def test_append_rope_bad_positions_and_slots():
    rng = _rng(8)
    table, pos, x, q, k, v = _rope_case(rng, 6, 4, 2, 64, 64, True)
    pos[1], pos[4] = -1, 500
    slots = np.array([0, 1, -1, 3, 4, 99], np.int32)
    kc, vc, err = kvq.alloc_e2m1_pool(3, 2, 64), kvq.alloc_e2m1_pool(3, 2, 64), _err()
    out = torch.full((6, 4, 64), 9.0, dtype=torch.float16, device="cuda")
    kvq.kv_append_rope_e2m1(q, k, v, to_dev(pos), to_dev(table), to_dev(slots), kc, vc, 0.01, 0.01, q_out=out, err_flag=err)
    assert err.item() == kvq.DEV_BAD_POS | kvq.DEV_BAD_SLOT
    safe = np.where((pos < 0) | (pos >= 500), 0, pos)
    ref = E.rotate(x[:, :6], table, safe, False)
    good = [0, 2, 3, 5]
    assert np.array_equal(out.cpu().numpy()[good], ref[good, :4].astype(np.float16)) and (out[[1, 4]] == 9.0).all()
    keep = np.where(np.isin(np.arange(6), [0, 3]), slots, -1)
    assert np.array_equal(kc.cpu().numpy(), E.append(np.zeros((3, 2, 144), np.uint8), ref[:, 4:], keep, 0.01))


def test_append_rope_refuses_what_it_cannot_address():
    t = lambda *s, d=torch.float16: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    i = t(4, d=torch.int32)
    kc = t(8, 2, 4, 64, d=torch.uint8)
    q, k, table = t(4, 8, 64), t(4, 2, 64), t(10, 64, d=torch.float32)
    call = lambda **kw: kvq.kv_append_rope_e4m3(**{**dict(q=q, k_new=k, v_new=k, positions=i, table=table, slot_mapping=i,  # noqa: E731
                                                          k_cache=kc, v_cache=kc.clone(), k_scale=1.0, v_scale=1.0), **kw})
    call()
    for bad in (dict(k_new=k.transpose(1, 2)), dict(q=t(4, 64, 8).transpose(1, 2)), dict(q=t(5, 8, 64)), dict(q=t(1, 8, 64).expand(4, 8, 64)),
                dict(q_out=t(4, 8, 72)[..., :64]), dict(positions=i[:3]), dict(table=t(10, 64, d=torch.float32).t()),
                dict(k_cache=t(8, 1, 4, 64, d=torch.uint8)), dict(q=None, q_out=q), dict(k_new=t(4, 2, 128), v_new=t(4, 2, 128))):
        with pytest.raises((ValueError, TypeError)):
            call(**bad)
    with pytest.raises(kvq.KvqError) as e:
        call(q=t(4, 8 * 64 + 4)[:, :512].unflatten(1, (8, 64)))               # stride not a multiple of 8
    assert e.value.status == -6
    with pytest.raises(TypeError):
        call(positions=i.long())


# --- attention -------------------------------------------------------------

def _problem(seed, B, n, Hq, Hkv, D, lens, spare=5, garbage=True, topk=None):
    """Random K and V quantised by the reference into pools whose other slots hold NaN scales."""
    rng = _rng(9, seed)
    lens = np.asarray(lens, np.int32)
    need = (lens + 3) // 4
    P = int(need.sum()) + spare
    width = int(need.max()) + 2
    order = rng.permutation(P).astype(np.int32)
    bt = np.full((B, width), 2 ** 30, np.int32)           # entries past a sequence's pages are not read
    at = 0
    pools = [np.full((P, Hkv, 9 * D // 4), 0xFF if garbage else 0, np.uint8) for _ in range(2)]
    scales = (0.013, 0.0031)
    for b in range(B):
        bt[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    slots = np.concatenate([bt[b, np.arange(lens[b]) // 4] * 4 + np.arange(lens[b]) % 4 for b in range(B)]) if lens.sum() else []
    for i in range(2):
        pools[i] = E.append(pools[i], _kv(rng, len(slots), Hkv, D), slots, scales[i])
    q = rng.standard_normal((B, n, Hq, D)).astype(np.float16)
    idx = counts = None
    if topk:
        idx = np.zeros((B, Hkv, topk), np.int32)
        counts = np.zeros(B, np.int32)
        for b in range(0, B, 2):
            counts[b] = min(topk, lens[b])
            for g in range(Hkv):
                idx[b, g, :counts[b]] = np.sort(rng.permutation(lens[b])[:counts[b]])
    return q, pools[0], pools[1], bt, lens, *scales, idx, counts


def _run(q, kc, vc, bt, lens, ks, vs, idx, counts, partial=False, **kw):
    args = [to_dev(a) for a in (q, kc, vc, bt, lens)]
    p = kvq.attn_params(args[0], kc.shape[1], bt.shape[1], kw.get("num_splits", 0), 0 if idx is None else idx.shape[2],
                        split_pages=kw.get("split_pages", 0))
    ws = kvq.alloc_workspace(p, "cuda").fill_(float("nan"))
    err = _err()
    lists = (None, None) if idx is None else (to_dev(idx), to_dev(counts))
    if partial:
        p = kvq.paged_decode_attn_e2m1_partial(*args, ks, vs, ws, *lists, err_flag=err, **kw)
        return p, ws, err.item()
    out = kvq.paged_decode_attn_e2m1(*args, ks, vs, ws, None, *lists, err_flag=err, **kw)
    return out.cpu().numpy(), err.item()


SHAPES = [  # B, q_len, Hq, Hkv, D, lens
    (2, 1, 8, 2, 64, [37, 100]), (2, 4, 8, 2, 64, [37, 100]), (1, 1, 1, 1, 128, [1]), (3, 1, 8, 1, 128, [1, 2, 3]),
    (4, 1, 32, 4, 128, [31, 32, 33, 129]), (2, 4, 32, 4, 128, [300, 77]), (1, 3, 7, 1, 128, [1000]), (2, 2, 16, 2, 64, [65, 4]),
    (3, 4, 16, 1, 128, [4, 5, 260]), (2, 4, 16, 1, 64, [513, 12]), (5, 1, 24, 8, 64, [128, 9, 64, 127, 16]), (1, 1, 12, 4, 128, [2049]),
    (2, 4, 6, 2, 128, [515, 258]), (2, 2, 40, 2, 128, [90, 300]),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("splits", [0, 1, 3, 8, 17])
def test_decode(shape, splits):
    pr = _problem(SHAPES.index(shape), *shape)
    out, err = _run(*pr, num_splits=splits)
    ref, tol, flags = E.decode(*pr)
    assert err == flags == 0
    E.close(out, ref, tol)


@pytest.mark.parametrize("shape", [SHAPES[0], SHAPES[5], SHAPES[7], SHAPES[8], (4, 1, 16, 2, 128, [200, 90, 333, 5])])
@pytest.mark.parametrize("topk,splits,split_pages", [(1, 1, 0), (40, 2, 0), (77, 0, 3), (300, 5, 0)])
def test_decode_over_lists(shape, topk, splits, split_pages):
    pr = _problem(7, *shape, topk=topk)
    out, err = _run(*pr, num_splits=splits, split_pages=split_pages)
    ref, tol, flags = E.decode(*pr)
    assert err == flags == 0
    E.close(out, ref, tol)


def test_decode_split_pages_and_empty_splits():
    pr = _problem(11, 3, 1, 8, 2, 128, [700, 3, 260])
    ref, tol, _ = E.decode(*pr)
    for sp in (1, 16, 50):
        out, err = _run(*pr, split_pages=sp)
        assert err == 0
        E.close(out, ref, tol, f"split_pages {sp}")


@pytest.mark.parametrize("D", [64, 128])
def test_decode_bad_pages_lists_and_lengths(D):
    """A bad page's tokens are left out; a list's bad entries too; an invalid length and a list of nothing give zero rows.
    Infinite queries stay in their own rows."""
    q, kc, vc, bt, lens, ks, vs, idx, counts = _problem(12, 6, 2, 8, 2, D, [50, 60, 70, 80, 90, 33], topk=20)
    bt[0, 3], bt[1, 5], bt[1, 14] = -1, kc.shape[0], 2 ** 31 - 1
    idx[2, 0, 3], idx[2, 1, 19] = -1, 70
    counts[4] = 21                                       # longer than the list: cut, and flagged
    lens[3] = 4 * bt.shape[1] + 1
    lens[5] = 1                                          # below q_len
    out, err = _run(q, kc, vc, bt, lens, ks, vs, idx, counts, num_splits=3)
    fixed = counts.copy()
    fixed[4] = 20
    ref, tol, flags = E.decode(q, kc, vc, bt, lens, ks, vs, idx, fixed)
    assert err == flags | kvq.DEV_BAD_TOPK and flags & (kvq.DEV_BAD_PAGE | kvq.DEV_BAD_LEN)
    assert not out[3].any() and not out[5].any()
    E.close(out, ref, tol)


def test_decode_rows_that_a_mask_leaves_empty():
    """A list of the window's last token alone: earlier rows of the window see nothing and are zero."""
    q, kc, vc, bt, lens, ks, vs, idx, counts = _problem(13, 2, 4, 8, 2, 128, [100, 9], topk=8)
    idx[0, :, 0], counts[0] = 99, 1
    for splits in (1, 4):
        out, err = _run(q, kc, vc, bt, lens, ks, vs, idx, counts, num_splits=splits)
        ref, tol, _ = E.decode(q, kc, vc, bt, lens, ks, vs, idx, counts)
        assert err == 0 and not out[0, :3].any() and out[0, 3].any()
        E.close(out, ref, tol)


@pytest.mark.parametrize("q_len,Hq", [(1, 8), (4, 16), (4, 32)])
def test_decode_nan_scale_inside_the_context_reaches_its_rows_alone(q_len, Hq):
    q, kc, vc, bt, lens, ks, vs, _, _ = _problem(14, 2, q_len, Hq, 2, 128, [150, 150])
    for pool in (kc, vc):
        bad = pool.copy()
        bad[bt[0, 20], 1, 256 + 4 * 3 + 2] = 0x7F        # sequence 0, kv head 1, token 82, block 3
        pools = (bad, vc) if pool is kc else (kc, bad)
        out, err = _run(q, *pools, bt, lens, ks, vs, None, None, num_splits=4)
        ref, tol, _ = E.decode(q, kc, vc, bt, lens, ks, vs)
        rows = np.isnan(out[0, :, Hq // 2:])
        assert rows.all() if pool is kc else (rows[..., 48:64].all() and not rows[..., :48].any())
        E.close(out[1], ref[1], tol[1])
        E.close(out[0, :, :Hq // 2], ref[0, :, :Hq // 2], tol[0, :, :Hq // 2])


@pytest.mark.parametrize("q_len,Hq,Hkv", [(1, 4, 1), (4, 4, 1), (4, 8, 1), (3, 8, 1), (4, 12, 1)])
def test_decode_large_scores_and_rising_maxima(q_len, Hq, Hkv):
    """Scores in ascending order over hundreds of units (the running maximum moves all the time), and a temperature."""
    q, kc, vc, bt, lens, ks, vs, _, _ = _problem(15, 1, q_len, Hq, Hkv, 128, [777])
    rows = np.linspace(0.01, 30, 777)[:, None, None] * np.ones((777, Hkv, 128))
    slots = bt[0, np.arange(777) // 4] * 4 + np.arange(777) % 4
    kc = E.append(kc, rows.astype(np.float32), slots, ks)
    q[:] = np.abs(q)
    for sm in (None, 0.5):
        out, _ = _run(q, kc, vc, bt, lens, ks, vs, None, None, num_splits=2, sm_scale=sm or 0.0)
        ref, tol, _ = E.decode(q, kc, vc, bt, lens, ks, vs, sm=sm)
        E.close(out, ref, tol)
    # and in descending order, negated queries: every score below the first ones by far more than fp16 reaches
    out, _ = _run(-q, kc, vc, bt, lens, ks, vs, None, None, num_splits=2)
    ref, tol, _ = E.decode(-q, kc, vc, bt, lens, ks, vs)
    E.close(out, ref, tol)


@pytest.mark.parametrize("q_len,Hq,Hkv", [(2, 8, 2), (4, 8, 1), (4, 16, 1), (3, 16, 2)])
@pytest.mark.parametrize("splits", [1, 4])
def test_decode_dense_bad_pages(q_len, Hq, Hkv, splits):
    q, kc, vc, bt, lens, ks, vs, _, _ = _problem(22, 3, q_len, Hq, Hkv, 128, [500, 140, 260])
    bt[0, 3], bt[0, 70], bt[0, 124], bt[1, 0], bt[2, 64] = -1, kc.shape[0], 2 ** 31 - 1, -5, -2 ** 31
    out, err = _run(q, kc, vc, bt, lens, ks, vs, None, None, num_splits=splits)
    ref, tol, flags = E.decode(q, kc, vc, bt, lens, ks, vs)
    assert err == flags == kvq.DEV_BAD_PAGE
    E.close(out, ref, tol)


@pytest.mark.parametrize("q_len,Hq,D,topk", [(1, 8, 128, None), (1, 8, 64, 30), (4, 16, 128, None), (4, 32, 128, None)])
def test_decode_longest_first_over_several_waves(q_len, Hq, D, topk):
    """More CTAs than the card holds at once, lengths from 4 to 300: the sequences are taken longest first."""
    lens = [4 + (97 * i) % 297 for i in range(300)]
    pr = _problem(23, 300, q_len, Hq, 2, D, lens, topk=topk)
    out, err = _run(*pr, num_splits=3)
    q, kc, vc, bt, lens, ks, vs, idx, counts = pr
    some = np.r_[0:300:37, 299]                          # the reference takes a few of them
    cut = lambda x: None if x is None else x[some]  # noqa: E731
    ref, tol, flags = E.decode(q[some], kc, vc, bt[some], lens[some], ks, vs, cut(idx), cut(counts))
    assert err == flags == 0
    E.close(out[some], ref, tol)
    assert np.isfinite(out).all() and (np.abs(out).max((1, 2, 3)) > 0).all()


def test_decode_is_deterministic_and_partials_combine_to_it():
    pr = _problem(16, 4, 2, 16, 2, 128, [900, 31, 444, 100])
    out, _ = _run(*pr, num_splits=6)
    for _ in range(3):
        assert np.array_equal(_run(*pr, num_splits=6)[0], out)
    assert np.array_equal(_run(*pr, num_splits=6, strict_order=True)[0], out)
    p, ws, err = _run(*pr, partial=True, num_splits=6)
    merged = kvq.lse_combine(ws, torch.empty(pr[0].shape, dtype=torch.float16, device="cuda"), p)
    assert err == 0 and np.array_equal(merged.cpu().numpy(), out)
    o, m, l = (x.cpu().numpy() for x in kvq.workspace_views(ws, p))
    empty = l == 0
    assert empty.any() and np.isneginf(m[empty]).all() and np.isfinite(m[~empty]).all() and np.isfinite(o[~empty]).all()


def test_decode_pages_beyond_4_gib():
    """Page offsets that pass 32 bits: 4.6 GB pools, the attended pages at their end."""
    P, Hkv, D = 4_000_000, 4, 128
    q, kc, vc, bt, lens, ks, vs, _, _ = _problem(17, 2, 1, 8, Hkv, D, [130, 61], spare=0)
    n = kc.shape[0]
    big = [torch.zeros(P, Hkv, 288, dtype=torch.uint8, device="cuda") for _ in range(2)]
    slots = np.concatenate([(bt[b, np.arange(x) // 4] + P - n) * 4 + np.arange(x) % 4 for b, x in enumerate(lens)]).astype(np.int32)
    rng = _rng(18)
    rows = [_kv(rng, len(slots), Hkv, D) for _ in range(2)]
    kvq.kv_append_e2m1(*[to_dev(r) for r in rows], to_dev(slots), *big, ks, vs)
    for pool, r, s in zip((kc, vc), rows, (ks, vs)):
        pool[:] = E.append(pool, r, slots - 4 * (P - n), s)
    for b, x in enumerate(lens):
        bt[b, :(x + 3) // 4] += P - n
    args = [to_dev(a) for a in (q, bt, lens)]
    ws = kvq.alloc_workspace(kvq.attn_params(args[0], Hkv, bt.shape[1]), "cuda")
    out = kvq.paged_decode_attn_e2m1(args[0], *big, *args[1:], ks, vs, ws).cpu().numpy()
    for b, x in enumerate(lens):
        bt[b, :(x + 3) // 4] -= P - n
    ref, tol, _ = E.decode(q, kc, vc, bt, lens, ks, vs)
    E.close(out, ref, tol)
    k, _ = kvq.kv_gather_e2m1(*big, to_dev(slots[-3:]), ks, vs)
    assert np.array_equal(k.cpu().numpy(), (E.values(*E.quantize(rows[0][-3:], ks)).astype(np.float32) * np.float32(ks)).astype(np.float16))


@pytest.mark.parametrize("Hq,splits", [(8, 1), (8, 3), (16, 2)])
def test_tensor_core_kernel_gives_up_cleanly(Hq, splits):
    """A wait that runs out (a test build whose softmax warps first wait, 20 us long, for a product of their own): the
    error bit, empty partials, nothing hung, and the context usable."""
    import ctypes
    lib = kvq.load(build.build_variant("stall_softmax", {"KVQ_TEST_STALL_SOFTMAX": "20000ull"}, ("kvq_attn_e2m1_tc.cu",)))
    pr = _problem(24, 2, 4, Hq, 1, 128, [3000, 517])
    q, kc, vc, bt, lens = (to_dev(a) for a in pr[:5])
    p = kvq.attn_params(q, 1, bt.shape[1], splits)
    ws = kvq.alloc_workspace(p, "cuda").fill_(float("nan"))
    err = _err()
    ptr = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    st = lib.paged_decode_attn_e2m1_partial(ptr(q), ptr(kc), ptr(vc), kc.shape[0], ptr(bt), ptr(lens), ctypes.c_float(pr[5]),
                                            ctypes.c_float(pr[6]), None, None, ptr(ws), ws.numel() * 4, ctypes.byref(p), ptr(err),
                                            ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert st == 0 and err.item() == kvq.DEV_TIMEOUT
    _, m, l = kvq.workspace_views(ws, p)
    assert torch.isneginf(m).all() and (l == 0).all()
    out, err = _run(*pr, num_splits=splits)                # the library's own build, right after
    ref, tol, flags = E.decode(*pr)
    assert err == flags == 0
    E.close(out, ref, tol)


# --- prefill ---------------------------------------------------------------

@pytest.mark.parametrize("chunks,history,Hq,Hkv", [([1], [0], 4, 1), ([37, 1, 200], [5, 300, 0], 8, 2), ([129, 256], [127, 1], 4, 4)])
def test_prefill(chunks, history, Hq, Hkv):
    lens = [n + h for n, h in zip(chunks, history)]
    _, kc, vc, bt, lens, ks, vs, _, _ = _problem(19, len(lens), 1, Hq, Hkv, 128, lens)
    start = np.concatenate([[0], np.cumsum(chunks)]).astype(np.int32)
    q = _rng(20).standard_normal((start[-1], Hq, 128)).astype(np.float16)
    args = [to_dev(a) for a in (q, kc, vc, bt, lens, start)]
    p = kvq.prefill_params(args[0], Hkv, len(lens), bt.shape[1], max(chunks))
    err = _err()
    out = kvq.paged_prefill_attn_e2m1(*args, ks, vs, kvq.alloc_prefill_workspace(p, "cuda"), max_q_len=max(chunks),
                                      err_flag=err).cpu().numpy()
    assert err.item() == 0
    K, V = E.pool_values(kc, 128) * float(np.float32(ks)), E.pool_values(vc, 128) * float(np.float32(vs))
    for b, n in enumerate(chunks):
        pos = np.arange(lens[b])
        k, v = K[bt[b, pos // 4], :, pos % 4], V[bt[b, pos // 4], :, pos % 4]
        for i in range(n):
            see = lens[b] - n + i + 1
            for h in range(Hq):
                # the reference of the running maximum may trail it by 2^8: P up to 256 in fp16, whose subnormal steps count less
                ref, tol = E.attend(q[start[b] + i, h], k[:see, h * Hkv // Hq], v[:see, h * Hkv // Hq], 1 / math.sqrt(128))
                E.close(out[start[b] + i, h], ref, tol, f"chunk {b} token {i} head {h}")


# --- together --------------------------------------------------------------

def test_serving_run_eager_captured_and_on_another_stream():
    """Prompt chunks appended with rotation and attended, then decode steps: rotate and append, attend.  The same bits eager,
    captured and replayed, and on a side stream; the last step against the reference."""
    rng = _rng(21)
    B, Hq, Hkv, D, rot, prompt, steps = 3, 8, 2, 128, 64, [70, 9, 131], 5
    width = (max(prompt) + steps + 3) // 4
    bt = rng.permutation(B * width).astype(np.int32).reshape(B, width)
    P = B * width
    table = kvq.rope_table(256, rot)
    ks, vs = 0.012, 0.011
    chunk = _kv(rng, sum(prompt), Hq + 2 * Hkv, D)
    pos = np.concatenate([np.arange(n) for n in prompt]).astype(np.int32)
    seq = np.repeat(np.arange(B), prompt)
    slots = (bt[seq, pos // 4] * 4 + pos % 4).astype(np.int32)
    start = np.concatenate([[0], np.cumsum(prompt)]).astype(np.int32)
    new = _kv(rng, steps * B, Hq + 2 * Hkv, D).reshape(steps, B, -1, D)
    dev = {k: to_dev(x) for k, x in dict(chunk=chunk, pos=pos, slots=slots, start=start, bt=bt, new=new,
                                         lens=np.array(prompt, np.int32)).items()}

    def program(kc, vc, qp, outs, prefill, ws, pws):
        c = dev["chunk"]
        kvq.kv_append_rope_e2m1(c[:, :Hq], c[:, Hq:Hq + Hkv], c[:, Hq + Hkv:], dev["pos"], table, dev["slots"], kc, vc, ks, vs, q_out=qp)
        kvq.paged_prefill_attn_e2m1(qp, kc, vc, dev["bt"], dev["lens"], dev["start"], ks, vs, pws, prefill, max_q_len=max(prompt))
        for s in range(steps):
            x = dev["new"][s]
            at = dev["lens"] + s
            slot = (dev["bt"].gather(1, (at // 4).long()[:, None])[:, 0] * 4 + at % 4).int()
            q = torch.empty(B, 1, Hq, D, dtype=torch.float16, device="cuda")
            kvq.kv_append_rope_e2m1(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], at.int(), table, slot, kc, vc, ks, vs, q_out=q[:, 0])
            kvq.paged_decode_attn_e2m1(q, kc, vc, dev["bt"], (at + 1).int(), ks, vs, ws, outs[s])

    def buffers():
        q = torch.empty(B, 1, Hq, D, dtype=torch.float16, device="cuda")
        qp = torch.empty(sum(prompt), Hq, D, dtype=torch.float16, device="cuda")
        p = kvq.prefill_params(qp, Hkv, B, width, max(prompt))
        return (kvq.alloc_e2m1_pool(P, Hkv, D), kvq.alloc_e2m1_pool(P, Hkv, D), qp,
                torch.zeros(steps, B, 1, Hq, D, dtype=torch.float16, device="cuda"), torch.zeros_like(qp),
                kvq.alloc_workspace(kvq.attn_params(q, Hkv, width), "cuda"), kvq.alloc_prefill_workspace(p, "cuda"))

    eager = buffers()
    program(*eager)
    side = buffers()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        program(*side)
    torch.cuda.current_stream().wait_stream(stream)
    captured = buffers()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        program(*captured)
    for _ in range(2):
        for t in captured[:5]:
            t.zero_()
        graph.replay()
    torch.cuda.synchronize()
    for got in (side, captured):
        for a, b in zip(eager[:5], got[:5]):
            assert torch.equal(a, b)
    # the last step, from the reference
    t = table.cpu().numpy()
    kc, vc = (np.zeros((P, Hkv, 288), np.uint8) for _ in range(2))
    rows, at, where = [chunk], [pos], [slots]
    for s in range(steps):
        p = np.array(prompt, np.int32) + s
        rows.append(new[s])
        at.append(p)
        where.append(bt[np.arange(B), p // 4] * 4 + p % 4)
    for x, p, w in zip(rows, at, where):
        turned = E.rotate(x[:, :Hq + Hkv], t, p, False)
        kc = E.append(kc, turned[:, Hq:], w, ks)
        vc = E.append(vc, x[:, Hq + Hkv:], w, vs)
    assert np.array_equal(eager[0].cpu().numpy(), kc) and np.array_equal(eager[1].cpu().numpy(), vc)
    q = turned[:, None, :Hq].astype(np.float16)
    ref, tol, _ = E.decode(q, kc, vc, bt, np.array(prompt) + steps, ks, vs)
    E.close(eager[3][-1].cpu().numpy(), ref, tol)
