"""The operators around the decode step together, as a serving loop uses them: maps
from lengths, new tokens into the paged cache, the prompt's attention in one piece
and in chunks over its prefix, then decode steps over the same cache."""
import numpy as np
import pytest
import torch

from mla_decode_attention_08_gb300 import binding
from oracle.attention import mla_decode_ref
from oracle.ops import page_map_ref, prefill_ref

from .gpu_util import assert_close

pytestmark = pytest.mark.gpu

HEADS, PAGE, EPS = 16, 16, 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib(built_library):
    binding.load_library(built_library)


def f64(t):
    return t.double().cpu().numpy()


class Server:
    """Three requests over one paged e4m3 cache."""

    def __init__(self, seed=0, rows=3, pages=64, max_pages=24):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        dev = dict(dtype=torch.int32, device="cuda")
        self.rows, self.pages = rows, pages
        self.lens = torch.zeros(rows, **dev)
        self.table = torch.full((rows, max_pages), -1, **dev)
        self.free = torch.randperm(pages, generator=self.g, device="cuda").int()
        self.cache = torch.zeros((pages * PAGE, 576), dtype=torch.uint8, device="cuda")
        self.scale = torch.tensor([8.0 / 448.0], device="cuda")
        self.weight = (1 + 0.1 * self.rand(512)).bfloat16()
        angle = torch.arange(512, device="cuda")[:, None] * 10000.0 ** (-torch.arange(32, device="cuda") / 32)
        self.rope = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
        self.w_k = (self.rand(HEADS, 128, 512) * 512 ** -0.5).bfloat16()
        self.w_v = (self.rand(HEADS, 128, 512) * 512 ** -0.5).bfloat16()
        self.ws = torch.zeros(binding.STEP_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")

    def rand(self, *s):
        return torch.randn(s, generator=self.g, device="cuda")

    def step(self, new, slots_len=None):
        """Maps of a step that adds ``new[b]`` tokens to row b; moves the lengths and the free list on."""
        dev = dict(dtype=torch.int32, device="cuda")
        new = torch.tensor(new, **dev)
        want = page_map_ref(self.lens.tolist(), new.tolist(), f64(self.table), self.free.tolist(), PAGE)
        total, fresh = int((self.lens + new).sum()), int(new.sum())
        n = slots_len or fresh
        out = {"qo": torch.empty(self.rows + 1, **dev), "kv": torch.empty(self.rows + 1, **dev),
               "indices": torch.empty(total, **dev), "slots": torch.empty(n, **dev),
               "positions": torch.empty(n, **dev), "used": torch.empty(1, **dev)}
        binding.mla_page_map(self.lens, new, self.table, self.free, *out.values(), page_size=PAGE,
                             num_pages=self.pages, workspace=self.ws)
        assert np.array_equal(out["indices"].cpu().numpy(), want["kv_indices"])
        assert np.array_equal(out["slots"].cpu().numpy()[:fresh], want["slots"])
        self.lens = self.lens + new
        self.free = self.free[int(out["used"]):].contiguous()
        return out

    def append(self, maps, q=None, q_out=None, dense=True):
        t = maps["slots"].numel()
        kv = (self.rand(t, 2112) * 0.8).bfloat16()[:, 1536:]
        latent = torch.empty((t, 576), dtype=torch.bfloat16, device="cuda") if dense else None
        binding.mla_kv_append(kv, self.weight, self.rope, maps["positions"], maps["slots"], self.cache, self.scale,
                              workspace=self.ws, eps=EPS, q_pe=q, q_out=q_out, latent_out=latent)
        return latent

    def expand(self, latent):
        k = torch.einsum("tc,hdc->thd", latent[:, :512].float(), self.w_k.float())
        v = torch.einsum("tc,hdc->thd", latent[:, :512].float(), self.w_v.float())
        return torch.cat([k, v], 2).bfloat16()

    def prefill(self, q, e, rope, qo, kv, causal=True, lse=None):
        out = torch.empty((q.shape[0], HEADS, 128), dtype=torch.bfloat16, device="cuda")
        plan = binding.mla_prefill_plan(qo.numel() - 1, q.shape[0], e.shape[0], HEADS)
        ws = binding.new_workspace(plan)
        binding.mla_prefill_fwd(q, e[..., :128], rope, e[..., 128:], qo, kv, out, plan=plan, workspace=ws,
                                causal=causal, lse=lse)
        assert binding.mla_decode_read_error(ws) == 0
        return out

    def decode(self, maps, q, qo_len=1):
        plan = binding.mla_decode_plan(self.rows, 24 * PAGE, qo_len=qo_len)
        ws = binding.new_workspace(plan)
        out = torch.empty((q.shape[0], HEADS, 512), dtype=torch.bfloat16, device="cuda")
        binding.mla_decode_fwd(q, self.cache, self.scale, maps["qo"], maps["kv"], out, plan=plan, workspace=ws,
                               kv_indices=maps["indices"])
        assert binding.mla_decode_read_error(ws) == 0
        ref = mla_decode_ref(f64(q), self.cache.cpu().numpy(), np.float32(self.scale.item()), maps["qo"].cpu().numpy(),
                             maps["kv"].cpu().numpy(), maps["indices"].cpu().numpy())
        assert_close(f64(out), ref)
        return out


def test_prompts_then_decode_steps():
    s = Server()
    maps = s.step([130, 1, 77])
    q = s.rand(208, HEADS, 192).bfloat16()
    latent = s.append(maps, q[..., 128:], q[..., 128:])          # the queries' rotation in place
    e = s.expand(latent)
    lse = torch.empty((208, HEADS), device="cuda")
    out = s.prefill(q, e, latent[:, 512:], maps["qo"], maps["kv"], lse=lse)
    want, want_lse, reach, spread = prefill_ref(f64(q), f64(e[..., :128]), f64(latent[:, 512:]), f64(e[..., 128:]),
                                                maps["qo"].tolist(), maps["kv"].tolist(), 192 ** -0.5, True)
    err = 2.0 ** -16 * (spread + 1)
    assert (np.abs(f64(out) - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + err[..., None]) * reach).all()
    assert (np.abs(f64(lse) - want_lse) <= err + 2.0 ** -22 * np.abs(want_lse)).all()
    for new in ([1, 1, 1], [1, 1, 1], [2, 2, 2]):                # single tokens, then a two-token draft
        maps = s.step(new, slots_len=sum(new) + 2)               # a padded launch: the last two tokens are skipped
        n = sum(new)
        q = s.rand(n + 2, HEADS, 576).bfloat16()
        pe = s.rand(n + 2, HEADS, 64).bfloat16()
        before = q[n:].clone()
        s.append(maps, pe, q[..., 512:], dense=False)
        assert torch.equal(q[n:], before)
        s.decode(maps, q[:n].contiguous(), qo_len=new[0])
    assert binding.mla_decode_read_error(s.ws) == 0


def test_a_prompt_in_chunks_equals_the_whole():
    """The second chunk attends its prefix (no mask) and itself (causal); the pieces
    merge to what one call over all keys gives.  Each side is within its own rounding
    of the exact result, and the pieces' bf16 outputs add one more: 3 roundings."""
    s = Server(seed=1, rows=1)
    n, cut = 300, 170
    maps = s.step([n])
    q = s.rand(n, HEADS, 192).bfloat16()
    latent = s.append(maps, q[..., 128:], q[..., 128:])
    e, rope = s.expand(latent), latent[:, 512:]
    whole_lse = torch.empty((n, HEADS), device="cuda")
    whole = s.prefill(q, e, rope, maps["qo"], maps["kv"], lse=whole_lse)
    dev = dict(dtype=torch.int32, device="cuda")
    ind = lambda m: torch.tensor([0, m], **dev)  # noqa: E731
    m = n - cut
    lses = torch.empty((2, m, HEADS), device="cuda")
    parts = torch.stack([s.prefill(q[cut:], e[:cut], rope[:cut], ind(m), ind(cut), False, lses[0]),
                         s.prefill(q[cut:], e[cut:], rope[cut:], ind(m), ind(m), True, lses[1])])
    out, lse = torch.empty_like(parts[0]), torch.empty((m, HEADS), device="cuda")
    binding.mla_attn_merge(parts, lses, out, lse_out=lse)
    assert np.linalg.norm(f64(out) - f64(whole[cut:])) <= 3 * 2.0 ** -8 * np.linalg.norm(f64(whole[cut:]))
    assert np.abs(f64(lse) - f64(whole_lse[cut:])).max() <= 1e-4
    assert np.array_equal(f64(whole[:cut]), f64(s.prefill(q[:cut], e[:cut], rope[:cut], ind(cut), ind(cut))))


def test_expanded_and_absorbed_forms_agree():
    """The last token of a prompt by prefill, and by a decode step whose query carries the
    key expansion: q_latent = q_nope W_k, out = out_latent W_v.  (The decode step scales by
    1/sqrt(576), so its query is sqrt(3) times the prompt's.)  Roundings to bf16 on the way:
    the query, the expanded key, its score's probability, the value and both outputs on
    either side, each 2^-8 at most and scores of a few units; the cache's e4m3 codes move a
    latent value by up to 2^-4, independent from key to key and dim to dim."""
    s = Server(seed=2, rows=1)
    n = 200
    q = s.rand(n, HEADS, 192).bfloat16()
    maps = s.step([n])
    latent = s.append(maps, q[..., 128:], q[..., 128:])
    e = s.expand(latent)
    out = s.prefill(q, e, latent[:, 512:], maps["qo"], maps["kv"])[-1]
    absorbed = torch.einsum("hd,hdc->hc", q[-1, :, :128].float(), s.w_k.float())
    dq = (3 ** 0.5 * torch.cat([absorbed, q[-1, :, 128:].float()], 1)).bfloat16()[None]
    one = {"qo": torch.tensor([0, 1], dtype=torch.int32, device="cuda"), "kv": maps["kv"], "indices": maps["indices"]}
    lat = s.decode(one, dq)[0].float()
    got = torch.einsum("hc,hdc->hd", lat, s.w_v.float())
    assert np.linalg.norm(f64(got) - f64(out)) <= 2.0 ** -4 * np.linalg.norm(f64(out))


def test_calls_without_tokens_do_nothing():
    bf16, dev = torch.bfloat16, "cuda"
    s = Server(seed=3)
    none = torch.empty(0, dtype=torch.int32, device=dev)
    before = s.cache.clone()
    binding.mla_kv_append(torch.empty((0, 576), dtype=bf16, device=dev), s.weight, s.rope, none, none, s.cache, s.scale,
                          workspace=s.ws, q_pe=torch.empty((0, 16, 64), dtype=bf16, device=dev),
                          q_out=torch.empty((0, 16, 64), dtype=bf16, device=dev))
    assert torch.equal(s.cache, before)
    plan = binding.mla_prefill_plan(2, 0, 100, HEADS)
    ind = torch.zeros(3, dtype=torch.int32, device=dev)
    empty = lambda *shape: torch.empty(shape, dtype=bf16, device=dev)  # noqa: E731
    binding.mla_prefill_fwd(empty(0, HEADS, 192), empty(5, HEADS, 128), empty(5, 64), empty(5, HEADS, 128), ind, ind,
                            empty(0, HEADS, 128), plan=plan, workspace=binding.new_workspace(plan))
    # queries without any key tensor rows: zeros
    plan = binding.mla_prefill_plan(1, 3, 0, HEADS)
    out = torch.full((3, HEADS, 128), 7.0, dtype=bf16, device=dev)
    binding.mla_prefill_fwd(s.rand(3, HEADS, 192).bfloat16(), empty(0, HEADS, 128), empty(0, 64), empty(0, HEADS, 128),
                            torch.tensor([0, 3], dtype=torch.int32, device=dev), ind[:2], out, plan=plan,
                            workspace=binding.new_workspace(plan))
    assert (out == 0).all()
    binding.mla_attn_merge(empty(2, 0, 128), torch.empty((2, 0), device=dev), empty(0, 128))
