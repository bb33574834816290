"""The decode step's log-sum-exps, and a shared prefix joined to the rows' own tokens.

Scores are float32 sums of up to 2 x 576 products: within 2^-14 of the largest sum |q||k| / 24;
the e4m3 form's query terms add 2^-22 of the token's largest magnitude times sum |k| / 24; the
exponentials and their sum stay below 2^-18.  The joined output has three bf16 roundings of
2^-8 (the two pieces', the result's) and two of probabilities: 2^-6 of the 2-norm bounds them."""
import numpy as np
import pytest
import torch

from mla_decode_attention_08_gb300 import binding
from oracle.long_context import attend_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(built_library):
    binding.load_library(built_library)


def f64(t):
    return t.double().cpu().numpy()


def i32(a):
    return torch.tensor([int(x) for x in a], dtype=torch.int32, device="cuda")


def check(q, keys_of, kv, n, lse, out):
    for b in range(len(kv) - 1):
        keys = keys_of(b)
        length = len(keys)
        t = slice(b * n, (b + 1) * n)
        seen = [length - n + 1 + i for i in range(n)]
        ref, ref_lse = attend_ref(q[t], keys, seen)
        empty = ref_lse == -np.inf
        assert (lse[t][empty] == -np.inf).all() and (out[t][empty] == 0).all()
        if empty.all():
            continue
        spread = (np.abs(q[t]) @ np.abs(keys).T / 24).max(axis=2)
        low = np.abs(q[t]).max(axis=(1, 2))[:, None] * np.abs(keys).sum(axis=1).max() / 24
        e = 2.0**-14 * spread + 2.0**-22 * low + 2.0**-18
        off = np.abs(lse[t][~empty] - ref_lse[~empty])
        assert (off <= (e + 2.0**-22 * np.abs(ref_lse))[~empty]).all(), (b, off.max())


@pytest.mark.parametrize("cache", ["e4m3", "paged", "bf16", "mxfp4"])
@pytest.mark.parametrize("n", [1, 2, 3, 4])
@pytest.mark.parametrize("lens", [[1], [3, 0, 129, 640, 2], [2000, 2500], [300] * 40])
def test_lse(cache, n, lens):
    if cache == "mxfp4" and n > 1:
        pytest.skip("one query token a row")
    g = torch.Generator(device="cuda").manual_seed(n + len(lens))
    rows, batch = sum(lens) + 1, len(lens)
    kv = np.concatenate([[0], np.cumsum(lens)])
    q = (1.5 * torch.randn(batch * n, 16, 576, generator=g, device="cuda")).bfloat16()
    x = torch.randn(rows, 576, generator=g, device="cuda").bfloat16()
    out = torch.full((batch * n, 16, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    plain, lse = torch.empty_like(out), torch.full((batch * n, 16), 7.0, device="cuda")
    plans = [binding.mla_decode_plan(batch, max(lens), qo_len=n), binding.mla_decode_plan(batch, max(lens), qo_len=n, persistent=True)]
    qo = i32(range(0, batch * n + 1, n))
    scale, index = torch.full((1,), 1 / 60, device="cuda"), None
    if cache in ("e4m3", "paged"):
        pool = (x.float() * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
        values = f64(pool.float()) * float(scale)
        index = torch.randperm(rows, generator=g, device="cuda").to(torch.int32) if cache == "paged" else None
        call = lambda out, **m: binding.mla_decode_fwd(q, pool, scale, qo, i32(kv), out, kv_indices=index, **m)
    elif cache == "bf16":
        values = f64(x)
        call = lambda out, **m: binding.mla_decode_fwd_bf16kv(q, x, qo, i32(kv), out, **m)
    else:
        fp4 = torch.empty(rows, 288, dtype=torch.uint8, device="cuda")
        scales = torch.empty(rows, 18, dtype=torch.uint8, device="cuda")
        binding.mla_mxfp4_quantize(x, fp4, scales)
        grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device="cuda")
        codes = torch.stack([fp4 & 15, fp4 >> 4], dim=2).flatten(1).long()
        values = f64(grid[codes] * torch.exp2(scales.float() - 127).repeat_interleave(32, dim=1))
        call = lambda out, **m: binding.mla_decode_fwd_mxfp4(q, fp4, scales, qo, i32(kv), out, **m)
    for plan in plans:
        ws = binding.new_workspace(plan)
        call(plain, plan=plan, workspace=ws)
        call(out, plan=plan, workspace=ws, lse=lse)
        torch.cuda.synchronize()
        assert binding.mla_decode_read_error(ws) == 0
        assert torch.equal(out, plain)
        rows_of = lambda b: values[kv[b]:kv[b + 1]] if index is None else values[index[kv[b]:kv[b + 1]].cpu().numpy()]
        check(f64(q), rows_of, kv, n, f64(lse), f64(out))
        lse.fill_(7.0)


def test_lse_of_another_shape_is_refused():
    plan = binding.mla_decode_plan(1, 16)
    ws = binding.new_workspace(plan)
    q, out = (torch.zeros(1, 16, d, dtype=torch.bfloat16, device="cuda") for d in (576, 512))
    pool, scale = torch.zeros(16, 576, dtype=torch.uint8, device="cuda"), torch.ones(1, device="cuda")
    for lse in (torch.empty(1, 15, device="cuda"), torch.empty(16, 1, device="cuda"), torch.empty(1, 16, 1, device="cuda")):
        with pytest.raises(ValueError):
            binding.mla_decode_fwd(q, pool, scale, i32([0, 1]), i32([0, 4]), out, plan=plan, workspace=ws, lse=lse)
    with pytest.raises(TypeError):
        binding.mla_decode_fwd(q, pool, scale, i32([0, 1]), i32([0, 4]), out, plan=plan, workspace=ws,
                               lse=torch.empty(1, 16, dtype=torch.float64, device="cuda"))


@pytest.mark.parametrize("n", [1, 3])
def test_a_shared_prefix_joined_to_the_rows_own_tokens(n):
    """Pages of two prefixes and of the rows' own tokens in one pool: the decode step over
    all of a row's tokens, in 64 bits, against the three calls."""
    g = torch.Generator(device="cuda").manual_seed(n)
    prefix, own = [700, 130], [[50, 3, 128, 260], [4, 90, 300]]
    rows = 4000
    pool = (torch.randn(rows, 576, generator=g, device="cuda") * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
    scale = torch.full((1,), 1 / 60, device="cuda")
    place = torch.randperm(rows, generator=g, device="cuda").to(torch.int32)
    batch = sum(map(len, own))
    q = (1.2 * torch.randn(batch * n, 16, 576, generator=g, device="cuda")).bfloat16()
    flat = [x for group in own for x in group]
    kv_prefix = np.concatenate([[0], np.cumsum(prefix)])
    kv_own = np.concatenate([[0], np.cumsum(flat)])
    i_prefix, i_own = place[:kv_prefix[-1]], place[kv_prefix[-1]:kv_prefix[-1] + kv_own[-1]]
    parts = torch.empty(2, batch * n, 16, 512, dtype=torch.bfloat16, device="cuda")
    lses = torch.empty(2, batch * n, 16, device="cuda")
    out = torch.empty(batch * n, 16, 512, dtype=torch.bfloat16, device="cuda")
    shared = binding.mla_shared_plan(2, batch * n, max(prefix))
    step = binding.mla_decode_plan(batch, max(flat), qo_len=n)
    ws = [binding.new_workspace(p) for p in (shared, step)]
    qo_groups = i32(np.concatenate([[0], np.cumsum([n * len(x) for x in own])]))
    binding.mla_shared_fwd(q, pool, scale, qo_groups, i32(kv_prefix), parts[0], plan=shared, workspace=ws[0],
                           kv_indices=i_prefix, lse=lses[0])
    binding.mla_decode_fwd(q, pool, scale, i32(range(0, batch * n + 1, n)), i32(kv_own), parts[1], plan=step,
                           workspace=ws[1], kv_indices=i_own, lse=lses[1])
    binding.mla_attn_merge(parts, lses, out)
    torch.cuda.synchronize()
    assert all(binding.mla_decode_read_error(w) == 0 for w in ws)
    values, got = f64(pool.float()) * float(scale), f64(out)
    b = 0
    for group, members in enumerate(own):
        head = i_prefix[kv_prefix[group]:kv_prefix[group + 1]].cpu().numpy()
        for length in members:
            keys = values[np.concatenate([head, i_own[kv_own[b]:kv_own[b + 1]].cpu().numpy()])]
            ref, _ = attend_ref(f64(q[b * n:(b + 1) * n]), keys, [len(keys) - n + 1 + i for i in range(n)])
            assert np.linalg.norm(got[b * n:(b + 1) * n] - ref) <= 2.0**-6 * np.linalg.norm(ref), b
            b += 1
