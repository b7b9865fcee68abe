"""The 4-bit cache and the rotary appends on the CPU: the reference is pinned against closed forms, and the library's host
checks fail closed (nothing here launches a kernel)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from fp8_paged_kv_e4m3_gb300 import build, kvq
from tests import _e2m1 as E

FAKE = ctypes.c_void_p(0x10000)     # never dereferenced: every call below fails before a launch
F = ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    build.build()
    return kvq.load()


# --- the reference ---------------------------------------------------------

def test_reference_e4m3_matches_torch():
    torch = pytest.importorskip("torch")
    x = np.concatenate([np.linspace(0, 600, 20011), E.e4m3_values()[:127],
                        (E.e4m3_values()[:126] + E.e4m3_values()[1:127]) / 2]).astype(np.float32)
    ref = torch.from_numpy(x).clamp(max=448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(E.e4m3_encode(x), ref)


def test_reference_e2m1_ties_and_saturation():
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    assert E.E2M1[E._nearest_even(ties, E.E2M1)].tolist() == [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0]
    assert E.E2M1[E._nearest_even(np.array([5.001, 6.0, 100.0]), E.E2M1)].tolist() == [6.0, 6.0, 6.0]


def test_reference_round_trip_and_error_bound():
    """Values on the grid come back exactly; any other is off by at most half the largest step (1 of 6) of its block,
    plus what the block scale's rounding saturates (2^-4 of 6)."""
    rng = np.random.default_rng(0)
    code = rng.integers(0, 16, (5, 3, 32)).astype(np.uint8)
    code[..., ::16] = 7                                  # a 6 in every block fixes its scale
    b = rng.integers(16, 127, (5, 3, 2)).astype(np.uint8)
    x = E.values(code, b).astype(np.float32)
    c2, b2 = E.quantize(x, 1.0)
    assert np.array_equal(b2, b) and np.array_equal(E.values(c2, b2), x)
    y = rng.standard_normal((64, 2, 64)).astype(np.float32)
    s = np.float32(np.abs(y).max() / 2688)
    back = E.values(*E.quantize(y, s)) * float(s)
    amax = np.repeat(np.abs(y.reshape(64, 2, 4, 16)).max(-1), 16, -1)
    assert (np.abs(back - y) <= amax * (1 / 6 + 2.0 ** -4) + 6 * 2.0 ** -9 * s).all()


def test_reference_pool_layout():
    D = 64
    x = np.random.default_rng(1).standard_normal((3, 2, D)).astype(np.float32)
    pool = E.append(np.zeros((2, 2, 9 * D // 4), np.uint8), x, [5, -1, 2], 0.001)
    codes, b = E.quantize(x, 0.001)
    assert pool[1, 0, D // 2] == codes[0, 0, 0] | codes[0, 0, 1] << 4          # page 1, token 1, byte 0
    assert pool[0, 1, 2 * D + 4 * 3 + 2] == b[2, 1, 3]                          # page 0, block 3, token 2
    got = E.pool_values(pool, D)
    assert np.array_equal(got[1, :, 1], E.values(codes[0], b[0])) and not got[1, :, [0, 2, 3]].any()


# --- host checks -----------------------------------------------------------

def _rope(**kw):
    p = dict(num_tokens=4, num_q_heads=8, num_kv_heads=2, head_dim=128, rot_dim=64, max_positions=100, flags=0,
             q_stride=0, k_stride=0, v_stride=0)
    p.update(kw)
    return kvq.RopeParams(**p)


def _append_rope(lib, p, kind="e4m3", q=FAKE, k=FAKE, v=FAKE, pos=FAKE, table=FAKE, slots=FAKE, q_out=ctypes.c_void_p(0x20000),
                 pages=10, ks=0.1, vs=0.1):
    f = getattr(lib, "kv_append_rope_" + kind)
    scales = () if kind == "fp16" else (F(ks), F(vs))
    return f(q, k, v, pos, table, slots, q_out, FAKE, FAKE, pages, *scales, ctypes.byref(p), None, None)


@pytest.mark.parametrize("kind", ["e4m3", "fp16", "e2m1"])
@pytest.mark.parametrize("field,value,status", [
    ("num_tokens", -1, -1), ("num_q_heads", -1, -1), ("num_kv_heads", 0, -1), ("head_dim", 0, -1), ("rot_dim", 0, -1),
    ("rot_dim", 144, -1), ("rot_dim", 24, -4), ("head_dim", 72, -4), ("head_dim", 272, -4), ("max_positions", 0, -1),
    ("flags", 2, -1), ("q_stride", 1000, -1), ("k_stride", 255, -1), ("v_stride", -256, -1), ("k_stride", 260, -6),
    ("q_stride", 1028, -6), ("num_tokens", 0, 0),
])
def test_rope_params_are_checked(lib, kind, field, value, status):
    assert _append_rope(lib, _rope(**{field: value}), kind) == status


def test_rope_pointers_and_scales_are_checked(lib):
    odd = ctypes.c_void_p(0x10008)
    for kind in ("e4m3", "fp16", "e2m1"):
        for name in ("q", "k", "v", "pos", "table", "slots", "q_out"):
            assert _append_rope(lib, _rope(), kind, **{name: None}) == -1
        for name in ("q", "k", "v", "table", "q_out"):
            assert _append_rope(lib, _rope(), kind, **{name: odd}) == -6
        assert _append_rope(lib, _rope(), kind, pages=0) == -1
        assert _append_rope(lib, _rope(q_stride=2048), kind, q_out=FAKE) == -1     # in place, layouts differ
    for kind in ("e4m3", "e2m1"):
        for bad in (0.0, -1.0, math.nan, math.inf):
            assert _append_rope(lib, _rope(), kind, ks=bad) == -2
            assert _append_rope(lib, _rope(), kind, vs=bad) == -2
    assert _append_rope(lib, _rope(), "e2m1", ks=1e-35) == -2
    assert _append_rope(lib, _rope(head_dim=96, rot_dim=96), "e2m1") == -4
    assert _append_rope(lib, None or _rope(num_tokens=0), "e4m3", q=None, k=None) == 0


def test_rope_table_arguments_are_checked(lib):
    def f(table=FAKE, n=10, rot=64, base=1e4, kind=0, factor=1.0, orig=0, fast=32.0, slow=1.0, mag=0.0):
        return lib.kvq_rope_table(table, n, rot, base, kind, factor, orig, fast, slow, mag, None)
    assert f(table=None) == -1 and f(n=0) == -1 and f(rot=0) == -1 and f(rot=24) == -4
    assert f(base=1.0) == -1 and f(base=math.inf) == -1 and f(kind=3) == -1 and f(mag=-1.0) == -1
    assert f(kind=1, factor=0.5) == -1 and f(kind=2, factor=4.0) == -1          # no original_positions
    assert f(kind=2, factor=4.0, orig=4096, fast=1.0, slow=32.0) == -1
    assert f(kind=2, factor=math.nan, orig=4096) == -1


def test_e2m1_scale_from_amax(lib):
    assert kvq.scale_from_amax_e2m1(2688.0) == 1.0 and kvq.scale_from_amax_e2m1(84.0) == 0.03125
    for bad in (0.0, -3.0, math.inf, math.nan):
        assert kvq.scale_from_amax_e2m1(bad) == 0.0


def test_e2m1_append_and_gather_host_checks(lib):
    a = lambda T=4, D=128, ks=1.0, vs=1.0, k=FAKE, c=FAKE, pages=10: lib.kv_append_e2m1(  # noqa: E731
        k, FAKE, FAKE, T, 2, D, c, FAKE, pages, F(ks), F(vs), None, None)
    g = lambda T=4, D=128, ks=1.0, vs=1.0, k=FAKE, c=FAKE, pages=10: lib.kv_gather_e2m1(  # noqa: E731
        c, FAKE, pages, FAKE, T, 2, D, F(ks), F(vs), k, FAKE, None, None)
    for f in (a, g):
        assert f(T=-1) == -1 and f(pages=0) == -1 and f(D=96) == -4 and f(ks=0.0) == -2 and f(vs=1e32) == -2
        assert f(k=None) == -1 and f(k=ctypes.c_void_p(0x10004)) == -6 and f(c=ctypes.c_void_p(0x10008)) == -6
        assert f(T=0, k=None, c=None) == 0


def _attn(lib, ks=0.1, vs=0.1, ws_bytes=1 << 20, q=FAKE, topk=None, **kw):
    p = dict(batch=2, q_len=1, num_q_heads=8, num_kv_heads=2, head_dim=64, num_splits=2, max_pages_per_seq=25, max_topk=0,
             sm_scale=0.0, split_pages=0, flags=0)
    p.update(kw)
    return lib.paged_decode_attn_e2m1(q, FAKE, FAKE, 40, FAKE, FAKE, F(ks), F(vs), topk, None, FAKE, ws_bytes, FAKE,
                                      ctypes.byref(kvq.AttnParams(**p)), None, None)


def test_e2m1_attention_host_checks(lib):
    assert _attn(lib, ks=0.0) == -2 and _attn(lib, vs=1e-38) == -2 and _attn(lib, ks=math.inf) == -2
    assert _attn(lib, ws_bytes=16) == -3 and _attn(lib, q=ctypes.c_void_p(0x10008)) == -6
    assert _attn(lib, topk=FAKE) == -1 and _attn(lib, head_dim=80) == -4 and _attn(lib, q_len=5) == -4
    assert _attn(lib, batch=0) == 0
    for f in (kvq.ATTN_BITCAST_DECODE, kvq.ATTN_MMA_SYNC, kvq.ATTN_FP8_QK, kvq.ATTN_LONGEST_FIRST):
        assert _attn(lib, flags=f) == -4
    assert _attn(lib, flags=64) == -1


def test_e2m1_prefill_host_checks(lib):
    def f(ks=0.1, ws=1 << 24, **kw):
        p = dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, max_pages_per_seq=100, max_q_len=300, total_q=600,
                 sm_scale=0.0, flags=0)
        p.update(kw)
        return lib.paged_prefill_attn_e2m1(FAKE, FAKE, FAKE, 40, FAKE, FAKE, FAKE, F(ks), F(0.1), FAKE, ws, FAKE,
                                           ctypes.byref(kvq.PrefillParams(**p)), None, None)
    assert f(ks=0.0) == -2 and f(ks=1e-38) == -2 and f(ws=16) == -3 and f(head_dim=64) == -4 and f(batch=0) == 0


def test_python_binding_refuses_cpu_tensors_and_bad_tables():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 2, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        kvq._heads(x, "q")
    with pytest.raises(ValueError):
        kvq.rope_table(10, 24, device="cpu")
    with pytest.raises(ValueError):
        kvq.rope_table(10, 64, scaling="cubic", device="cpu")
    assert kvq.e2m1_page_bytes(128) == 288 and kvq.e2m1_page_bytes(64) == 144


def test_call_module_leaves_unusual_arguments_to_the_checks():
    """The module that marshals the calls answers None (its caller then names what is wrong) for anything that is not a
    strided CUDA tensor of the right type: no exception, nothing read."""
    kvq.load()

    class Sub(torch.Tensor):
        pass

    z = torch.zeros(2, 2, 64, dtype=torch.float16)
    odd = [z, z.to("meta"), z.as_subclass(Sub), torch.nn.Parameter(z), z.to_sparse(), torch.empty(0), None, 3, "x", object()]
    for x in odd:
        for y in (z, x):
            assert kvq._pycall.append(x, y, x, x, y, 1.0, 1.0, None) is None
            assert kvq._pycall.gather(x, x, x, 1.0, 1.0, y, y, None) is None
            assert kvq._pycall.rope(2, x, y, y, x, x, x, y, x, x, 1.0, 1.0, 0, None) is None
            assert kvq._pycall.prefill(x, y, y, x, x, x, 1.0, 1.0, x, y, 1, 0.0, None) is None
            assert kvq._pycall.decode(x, y, y, x, x, 1.0, 1.0, x, None, None, None, 0, 0.0, None, 0, 0) is None
    assert kvq._pycall.append(z, z) is None
