"""gtq_chunk_attn where its fp16 operands come to the ends of their range."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import decode_attention_13_b200 as gtq  # noqa: E402
from tests import layout  # noqa: E402
from tests.serving import Cache, workspace  # noqa: E402
from tests.test_gpu_chunk import CHUNK_REL_L2  # noqa: E402

pytestmark = pytest.mark.gpu


class Head(Cache):
    """Reads heads of a cache that a test made itself."""

    def __init__(self, plan, hkv, kb, vb, tiles):
        self.hkv, self.kb, self.vb, self.pairing = hkv, kb, vb, 0
        self.tb, self.tiles, self.bits = layout.tile_bytes(kb, vb), tiles, gtq.gtq_get_bits(plan)


@pytest.mark.parametrize("n", [20, 100, 250])         # one tile of rows, two, pairs of CTAs
@pytest.mark.parametrize("mass", [0.9, 0.99, 0.999, 0.9999])
def test_a_sink_of_small_value_before_a_long_context(n, mass):
    # one token takes `mass` of every row and has a value of almost nothing, so the others, each 2^-18 to 2^-28 of it,
    # make up the row; enough heads that no call is split over the tokens (a split has a maximum of its own).  The sink
    # stands out in two RoPE blocks whose codes are the widest: logits are held to their low parts there
    B, hkv, gq, T = 8, 18, 2, 16384
    rng = np.random.default_rng(int(mass * 1e4) + n)
    loud = [3, 67, 20, 84]
    std = np.full(128, 0.02)
    std[loud] = 0.5
    u = np.zeros((B, hkv, 128))
    u[..., loud] = rng.choice([-0.5, 0.5], (B, hkv, 4))
    logit = np.log(mass / (1 - mass) * T)
    g = torch.Generator(device="cuda").manual_seed(n)
    k = torch.randn((B, hkv, T, 128), generator=g, device="cuda") * torch.tensor(std, dtype=torch.float32, device="cuda")
    k[:, :, 0] = torch.from_numpy(logit * np.sqrt(128.0) / 8.0 * u).float().cuda()
    v = torch.randn((B, hkv, T, 128), generator=g, device="cuda") * 0.3 + 1.0
    v[:, :, 0] *= 0.01
    q = 8.0 * np.repeat(u, gq, 1)[:, :, None, :] + 0.05 * rng.standard_normal((B, hkv * gq, n, 128))
    q, k, v = torch.from_numpy(q.astype(np.float16)).cuda(), k.half(), v.half()
    plan = gtq.gtq_alloc_bits(gtq.make_config(B, hkv * gq, hkv, 4, 4, T), k, T)
    packed = torch.empty(plan.packed_bytes, dtype=torch.uint8, device="cuda")
    gtq.gtq_quantize_pack(plan, k, v, 0, T, packed)
    out = torch.empty_like(q)
    need = gtq.gtq_chunk_workspace(plan, T, n)
    assert need == 256, "the call is split"
    gtq.gtq_chunk_attn(plan, packed, T, q, out, workspace(need))
    torch.cuda.synchronize()
    assert gtq.gtq_status(plan) == gtq.GTQ_OK
    rows = np.arange(0, n, max(1, n // 7))
    for b, h in ((0, 0), (7, 13)):
        K, V = Head(plan, hkv, 4, 4, T // 64).dequantised(packed, None, b, h, T)
        hs = slice(h * gq, (h + 1) * gq)
        s = q[b, hs][:, rows].double().cpu().numpy() @ K.T / np.sqrt(128.0)
        s = np.where(np.arange(T) <= (T - n + rows)[:, None], s, -np.inf)
        p = np.exp(s - s.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        ref, got = p @ V, out[b, hs][:, rows].double().cpu().numpy()
        e = np.linalg.norm(got - ref, axis=-1) / np.linalg.norm(ref, axis=-1)
        assert e.max() <= CHUNK_REL_L2, (b, h, p[..., 0].mean(), e.max())
