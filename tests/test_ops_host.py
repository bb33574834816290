"""The operators around the decode step on the CPU: host-side refusals of their C
entry points and of the binding, the prompt plan, and pins of their oracle."""
import ctypes

import numpy as np
import pytest

from mla_decode_attention_08_gb300 import binding
from oracle.ops import kv_row_ref, merge_ref, page_map_ref, prefill_ref, rotate_ref

INVALID, WS_SMALL = 1, 3


@pytest.fixture(scope="module")
def lib(built_library):
    return binding.load_library(built_library)


def ptr(offset=0):
    """A pointer that is never dereferenced: the checks fail first."""
    return ctypes.c_void_p((1 << 20) + offset)


MAP = dict(kv_lens=ptr(), new_lens=ptr(), batch=4, table=ptr(), stride=16, max_pages=16, page=64,
           num_pages=128, free=ptr(), num_free=8, qo=ptr(), kv=ptr(), indices=ptr(), indices_len=4096,
           slots=ptr(), positions=ptr(), slots_len=64, used=ptr(), ws=ptr(), ws_bytes=256)


@pytest.mark.parametrize("change,status", [
    (dict(batch=0), INVALID), (dict(batch=16385), INVALID), (dict(kv_lens=None), INVALID),
    (dict(new_lens=None), INVALID), (dict(table=None), INVALID), (dict(qo=None), INVALID),
    (dict(kv=None), INVALID), (dict(used=None), INVALID), (dict(indices=None), INVALID),
    (dict(slots=None), INVALID), (dict(positions=None), INVALID), (dict(free=None), INVALID),
    (dict(page=0), INVALID), (dict(num_pages=0), INVALID), (dict(max_pages=0), INVALID),
    (dict(stride=15), INVALID), (dict(stride=1 << 36), INVALID),
    (dict(page=1 << 16, num_pages=1 << 15), INVALID),               # pool rows past 2^31 - 1
    (dict(num_free=-1), INVALID), (dict(indices_len=-1), INVALID), (dict(slots_len=-1), INVALID),
    (dict(indices_len=2**31 - 1), INVALID), (dict(slots_len=2**31 - 1), INVALID),
    (dict(indices=ptr(4)), INVALID), (dict(slots=ptr(2)), INVALID), (dict(kv_lens=ptr(1)), INVALID),
    (dict(ws=None), INVALID), (dict(ws=ptr(16)), INVALID), (dict(ws_bytes=255), WS_SMALL)])
def test_page_map_refusals(lib, change, status):
    assert lib.mla_page_map(*{**MAP, **change}.values(), None) == status


APPEND = dict(kv=ptr(), stride=576, weight=ptr(), eps=1e-6, table=ptr(), max_pos=128, inter=1,
              positions=ptr(), slots=ptr(), tokens=4, cache=ptr(), scale=ptr(), rows=64, dense=None,
              q=ptr(), qt=1024, qh=64, out=ptr(4096), ot=1024, oh=64, heads=16, ws=ptr(), ws_bytes=256)


@pytest.mark.parametrize("change,status", [
    (dict(kv=None), INVALID), (dict(kv=ptr(8)), INVALID), (dict(stride=568), INVALID),
    (dict(stride=577), INVALID), (dict(stride=-576), INVALID), (dict(weight=None), INVALID),
    (dict(weight=ptr(2)), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(table=None), INVALID), (dict(table=ptr(4)), INVALID),
    (dict(max_pos=0), INVALID), (dict(positions=None), INVALID), (dict(slots=None), INVALID),
    (dict(tokens=-1), INVALID), (dict(cache=None), INVALID), (dict(cache=ptr(8)), INVALID),
    (dict(scale=None), INVALID), (dict(rows=0), INVALID), (dict(rows=2**31), INVALID),
    (dict(dense=ptr(2)), INVALID), (dict(dense=ptr(), stride=640), INVALID),   # in place, strided
    (dict(heads=-1), INVALID), (dict(q=None), INVALID), (dict(out=None), INVALID),
    (dict(q=ptr(8)), INVALID), (dict(qt=1020), INVALID), (dict(qh=60), INVALID),
    (dict(oh=56), INVALID), (dict(ot=32), INVALID), (dict(out=ptr(), ot=2048), INVALID),
    (dict(ws=None), INVALID), (dict(ws_bytes=128), WS_SMALL)])
def test_kv_append_refusals(lib, change, status):
    args = {**APPEND, **change}
    assert lib.mla_kv_append(*args.values(), None) == status
    if "scale" not in change:
        del args["scale"]
        assert lib.mla_kv_append_bf16kv(*args.values(), None) == status


def test_kv_append_of_no_tokens_launches_nothing(lib):
    args = {**APPEND, "tokens": 0, "kv": None, "slots": None}
    assert lib.mla_kv_append(*args.values(), None) == 0


def prefill_args(made, **change):
    args = dict(q=ptr(), qt=16 * 192, qh=192, kn=ptr(), knt=16 * 256, knh=256, kr=ptr(), krt=576, v=ptr(),
                vt=16 * 256, vh=256, total_kv=512, qo=ptr(), kv=ptr(), scale=0.1, causal=1, out=ptr(),
                lse=None, stream=None, plan=ctypes.byref(made), ws=ptr(), ws_bytes=made.ws_bytes)
    return {**args, **change}.values()


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INVALID), (dict(q=ptr(8)), INVALID), (dict(qt=100), INVALID), (dict(qh=184), INVALID),
    (dict(kn=None), INVALID), (dict(knt=4), INVALID), (dict(knh=120), INVALID), (dict(kr=None), INVALID),
    (dict(krt=56), INVALID), (dict(krt=66), INVALID), (dict(v=None), INVALID), (dict(v=ptr(2)), INVALID),
    (dict(vt=0), INVALID), (dict(vh=1 << 36), INVALID), (dict(total_kv=-1), INVALID),
    (dict(total_kv=2**31), INVALID), (dict(qo=None), INVALID), (dict(kv=None), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(out=None), INVALID), (dict(out=ptr(8)), INVALID),
    (dict(lse=ptr(2)), INVALID), (dict(ws=None), INVALID), (dict(ws=ptr(128)), INVALID),
    (dict(plan=None), INVALID), (dict(ws_bytes=0), WS_SMALL)])
def test_prefill_refusals(lib, change, status):
    plan = binding.mla_prefill_plan(2, 64, 8192, 16, 152)
    assert plan.splits > 1
    assert lib.mla_prefill_fwd(*prefill_args(plan, **change)) == status


def test_prefill_refuses_a_changed_plan(lib):
    for field, value in [("splits", 1), ("tiles", 99), ("abi_version", 4), ("ws_lse_offset", 0),
                         ("num_heads", 0), ("batch", 0), ("total_q", -1), ("num_sms", 0)]:
        plan = binding.mla_prefill_plan(2, 64, 8192, 16, 152)
        setattr(plan, field, value)
        assert lib.mla_prefill_fwd(*prefill_args(plan)) == INVALID, field


def test_prefill_of_no_queries_launches_nothing(lib):
    plan = binding.mla_prefill_plan(2, 0, 8192, 16, 152)
    assert plan.tiles == 0 and lib.mla_prefill_fwd(*prefill_args(plan, q=None, out=None)) == 0


@pytest.mark.parametrize("batch,total,kv,heads,sms", [(1, 1, 1, 1, 152), (1, 100, 100, 16, 152),
                                                      (1, 64, 8256, 16, 152), (12, 12000, 2047, 16, 152),
                                                      (256, 256, 8192, 16, 152), (1, 16384, 16384, 16, 152),
                                                      (3, 1000, 70000, 1, 40), (7, 5, 900, 2, 1)])
def test_prefill_plan(lib, batch, total, kv, heads, sms):
    p = binding.mla_prefill_plan(batch, total, kv, heads, sms)
    # any cut of the queries into rows fits the planned blocks
    rng = np.random.default_rng(batch + total)
    for _ in range(20):
        cuts = np.sort(rng.integers(0, total + 1, size=batch - 1))
        rows = np.diff(np.concatenate([[0], cuts, [total]]))
        assert int((-(-rows // 256)).sum()) <= p.tiles
    blocks = p.tiles * heads
    assert p.splits >= 1 and (p.splits == 1 or (blocks * p.splits <= sms and 4 * p.splits <= -(-kv // 128)))
    if p.splits > 1:
        rows = p.splits * total * heads
        assert p.ws_lse_offset >= 4 and p.ws_partial_offset >= p.ws_lse_offset + 4 * rows
        assert p.ws_bytes >= p.ws_partial_offset + 4 * 128 * rows
        assert p.ws_lse_offset % 256 == 0 and p.ws_partial_offset % 256 == 0


def test_prefill_plan_refusals(lib):
    p = ctypes.byref(binding.mla_prefill_plan_t())
    for args in [(0, 1, 1, 1), (1, -1, 1, 1), (1, 1, -1, 1), (1, 1, 1, 0), (1, 1, 1, 1025), (65537, 1, 1, 1)]:
        assert lib.mla_prefill_plan(*args, 152, p) == INVALID
    assert lib.mla_prefill_plan(1, 1, 1, 1, 152, None) == INVALID
    assert lib.mla_prefill_plan(1, 2**31 - 1, 1, 1024, 152, p) == INVALID   # blocks past 2^31 - 1 are refused or fit


MERGE = dict(parts=ptr(), lses=ptr(), n=2, rows=8, dim=128, out=ptr(), lse=None)


@pytest.mark.parametrize("change", [dict(parts=None), dict(lses=None), dict(out=None), dict(n=0), dict(n=65),
                                    dict(rows=-1), dict(rows=2**31), dict(dim=0), dict(dim=12), dict(dim=1032),
                                    dict(parts=ptr(8)), dict(out=ptr(8)), dict(lses=ptr(2)), dict(lse=ptr(1))])
def test_merge_refusals(lib, change):
    assert lib.mla_attn_merge(*{**MERGE, **change}.values(), None) == INVALID


def test_merge_of_no_rows_launches_nothing(lib):
    assert lib.mla_attn_merge(*{**MERGE, "rows": 0, "parts": None}.values(), None) == 0


def test_binding_refuses_cpu_tensors(lib):
    torch = pytest.importorskip("torch")
    i, f, h = torch.zeros(4, dtype=torch.int32), torch.zeros(4), torch.zeros(4, 576, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        binding.mla_page_map(i, i, i.view(4, 1), i, i, i, i, i, i, i, page_size=1, num_pages=1, workspace=f)
    with pytest.raises(TypeError):
        binding.mla_kv_append_bf16kv(h, h[0, :512], f, i, i, h, workspace=f)
    with pytest.raises(TypeError):                                  # a bf16 cache is not e4m3 codes
        binding.mla_kv_append(h, h[0, :512], f, i, i, h, f[:1], workspace=f)
    with pytest.raises(TypeError):
        binding.mla_attn_merge(h.view(1, 4, 576), f, h)
    plan = binding.mla_prefill_plan(1, 4, 4, 1, 152)
    with pytest.raises(TypeError):
        binding.mla_prefill_fwd(h, h, h, h, i, i, h, plan=plan, workspace=f)


# ---------------------------------------------------------------- pins of the oracle
def test_oracle_page_map_by_hand():
    table = np.array([[7, 5, -1], [-1, -1, -1], [2, -1, -1]])
    got = page_map_ref([5, 0, 3], [4, 0, 1], table, [9, 1, 4], 4)
    assert got["table"].tolist() == [[7, 5, 9], [-1, -1, -1], [2, -1, -1]]
    assert got["pages_used"] == 1 and got["kv_indptr"].tolist() == [0, 9, 9, 13]
    assert got["qo_indptr"].tolist() == [0, 4, 4, 5]
    assert got["kv_indices"].tolist() == [28, 29, 30, 31, 20, 21, 22, 23, 36, 8, 9, 10, 11]
    assert got["slots"].tolist() == [21, 22, 23, 36, 11] and got["positions"].tolist() == [5, 6, 7, 8, 3]


def test_oracle_rotation_is_a_rotation():
    rng = np.random.default_rng(1)
    x, angle = rng.standard_normal((3, 64)), rng.uniform(0, 6, (3, 32))
    for inter in (True, False):
        y = rotate_ref(x, np.cos(angle), np.sin(angle), inter)
        assert np.allclose(rotate_ref(y, np.cos(angle), -np.sin(angle), inter), x)
        assert np.allclose((y * y).sum(1), (x * x).sum(1))
    pair = rotate_ref(np.eye(64)[0], np.full(32, 0.0), np.ones(32), True)
    assert pair[1] == 1.0 and np.count_nonzero(pair) == 1           # (1, 0) turned by 90 degrees


def test_oracle_row_has_unit_mean_square():
    rng = np.random.default_rng(2)
    row = kv_row_ref(rng.standard_normal((4, 576)) * 9, np.ones(512), 0.0, np.ones((4, 32)), np.zeros((4, 32)), True)
    assert np.allclose((row[:, :512] ** 2).mean(1), 1.0)


def test_oracle_pieces_merge_to_the_whole():
    rng = np.random.default_rng(3)
    q, kn, kr, v = (rng.standard_normal(s) for s in ((5, 2, 192), (9, 2, 128), (9, 64), (9, 2, 128)))
    whole, lse, _, _ = prefill_ref(q, kn, kr, v, [0, 5], [0, 9], 0.1, False)
    parts = [prefill_ref(q, kn[a:b], kr[a:b], v[a:b], [0, 5], [0, b - a], 0.1, False) for a, b in ((0, 4), (4, 9))]
    out, l2, _ = merge_ref(np.stack([p[0] for p in parts]), np.stack([p[1] for p in parts]))
    assert np.allclose(out, whole) and np.allclose(l2, lse)
    # causal: the last query sees all keys, the first of five on nine keys sees five
    c, cl, _, _ = prefill_ref(q, kn, kr, v, [0, 5], [0, 9], 0.1, True)
    assert np.allclose(c[4], whole[4]) and np.allclose(cl[4], lse[4])
    first, fl, _, _ = prefill_ref(q[:1], kn[:5], kr[:5], v[:5], [0, 1], [0, 5], 0.1, False)
    assert np.allclose(c[0], first[0]) and np.allclose(cl[0], fl[0])
