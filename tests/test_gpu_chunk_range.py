"""gtq_chunk_attn where its fp16 operands come to the ends of their range."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import decode_attention_13_b200 as gtq  # noqa: E402
from tests import layout  # noqa: E402
from tests.serving import Cache, probabilities, workspace  # noqa: E402
from tests.test_gpu_chunk import CHUNK_REL_L2, run_chunk, same  # noqa: E402

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


def weights_of(c, q, n):
    w = torch.zeros((c.B, c.hkv, c.cap), device="cuda")
    gtq.gtq_attn_weights(c.plan, c.packed, c.cap, q, w, workspace(gtq.gtq_weights_workspace(c.plan, c.cap, n)),
                         layout=c.layout)
    torch.cuda.synchronize()
    assert gtq.gtq_status(c.plan) == gtq.GTQ_OK
    return w


@pytest.mark.parametrize("n", [3, 20, 40, 90])
@pytest.mark.parametrize("size", [2e4, 6e4])
def test_queries_near_the_end_of_fp16(n, size):
    # one group's turned query has nearly all of its length in one coordinate: entries of +-size, signed like a row of the
    # group's rotation.  The keys are so small that logits stay mild
    from oracle import allocation, rotation

    c = Cache([300], 1, 8, 3, 3, seed=5, scale=1e-3)
    group = max(allocation.groups(c.bits[0, 0], 128, 0), key=lambda g: g.m)
    R = rotation.key_rotation(group.m)
    q = np.zeros((1, 8, n, 128))
    rows = np.random.default_rng(n).integers(0, group.m, (8, n))
    q[0][..., list(group.coords)] = np.where(R[rows] < 0, -size, size)
    K, V = c.K[0][0], c.V[0][0]
    # (the most that a logit varies by, brought to 4)
    spread = np.abs(q[0] @ K.T).max() / np.sqrt(128.0)
    c = Cache([300], 1, 8, 3, 3, seed=5, scale=1e-3 * 4.0 / spread)
    assert group == max(allocation.groups(c.bits[0, 0], 128, 0), key=lambda g: g.m)
    K, V = c.K[0][0], c.V[0][0]
    qd = torch.from_numpy(q.astype(np.float16)).cuda()
    p = probabilities(q[0], K, n, True)
    # A coordinate's term: half a step, 2^-11, for the query, the centroid and the element each, and 2^-25 of the element's
    # unit, 8 / sqrt(m), for an element (and its centroid's 2^-25 an eighth of the norm at most) among the subnormals
    off = 0.0
    for g in allocation.groups(c.bits[0, 0], 128, 0):
        turned = np.abs(q[0][..., list(g.coords)] @ rotation.key_rotation(g.m).T)
        k = np.abs(K[:, list(g.coords)] @ rotation.key_rotation(g.m).T)
        norm = np.linalg.norm(K[:, list(g.coords)], axis=-1).max()
        off = off + (3 * 2.0 ** -11 * turned @ k.T + (2.0 ** -25 * 8.0 / np.sqrt(g.m) * (1 + norm)) * turned.sum(-1)[..., None])
    off = (off / np.sqrt(128.0)).max()      # of any logit, in nats; a weight changes by twice that, relatively
    out = run_chunk(c, qd, n, None, True)
    ref, got = p @ V, out[0].double().cpu().numpy()
    e = np.linalg.norm(got - ref, axis=-1)
    most = np.linalg.norm(V, axis=-1).max()
    assert np.all(e <= CHUNK_REL_L2 * np.linalg.norm(ref, axis=-1) + np.expm1(2 * off) * most), (off, e.max())
    w = weights_of(c, qd, n)[0, 0].double().cpu().numpy()
    sums = p.sum((0, 1))
    assert np.all(np.abs(w - sums) <= np.expm1(2 * off) * sums + 1e-5 * sums.max()), off


@pytest.mark.parametrize("n", [3, 20, 40, 90])     # each form of the kernel; 9000 tokens are split, 200 are not
@pytest.mark.parametrize("length", [200, 9000])
@pytest.mark.parametrize("sign", [1, -1])
def test_infinite_queries_stay_in_their_rows(n, length, sign):
    c = Cache([length], 1, 8, 3, 3, seed=n)
    q = c.queries(n, seed=n)
    want, weights = run_chunk(c, q, n, None, True), weights_of(c, q, n)
    for dim in (0, 77, 127):
        bad = q.clone()
        bad[0, 5, n // 2, dim] = sign * float("inf")
        got = run_chunk(c, bad, n, None, True)
        assert bool(got[0, 5, n // 2].isnan().all())
        got[0, 5, n // 2] = want[0, 5, n // 2]
        assert torch.equal(got, want)
        seen = length - n + n // 2 + 1
        w = weights_of(c, bad, n)
        assert bool(w[0, 0, :seen].isnan().all())
        assert torch.equal(w[0, 0, seen:], weights[0, 0, seen:])


@pytest.mark.parametrize("n", [1, 2])      # 8 and 16 rows: weights come from kept scores, one token from the decode kernel
@pytest.mark.parametrize("length", [200, 9000])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_odd_queries_of_few_rows(n, length, value):
    c = Cache([length], 1, 8, 3, 3, seed=1)
    q = c.queries(n, seed=n)
    want, weights = run_chunk(c, q, n, None, True), weights_of(c, q, n)
    bad = q.clone()
    bad[0, 5, 0, 77] = value
    got, w, seen = run_chunk(c, bad, n, None, True), weights_of(c, bad, n), length - n + 1
    assert bool(w[0, 0, :seen].isnan().all()) and torch.equal(w[0, 0, seen:], weights[0, 0, seen:])
    if n > 1:
        assert bool(got[0, 5, 0].isnan().all())
    got[0, 5, 0] = want[0, 5, 0]
    assert same(got, want, n, c)


@pytest.mark.parametrize("n", [20, 100, 250])
@pytest.mark.parametrize("growth", [1.0, 2.0, 3.9, 4.1, 6.0])     # of the logits from one step of 128 tokens to the next, log2
def test_logits_that_grow_along_the_context(n, growth):
    # the reference maximum stays for some steps and moves at others, while the old tokens' weights fade.  The logits stand
    # in two RoPE blocks, whose low parts are kept: 35 log2 at most, off by 2^-20 of that
    B, hkv, gq, T = 4, 37, 2, 1024    # (enough heads that no call is split over the tokens)
    rng = np.random.default_rng(n)
    loud = [3, 67, 20, 84]
    u = np.zeros(128)
    u[loud] = 0.5
    ramp = np.minimum(growth * np.arange(T) / 128.0, 35.0) * np.log(2.0)
    k = 0.02 * rng.standard_normal((B, hkv, T, 128)) + (ramp * np.sqrt(128.0) / 8.0)[None, None, :, None] * u
    v = rng.standard_normal((B, hkv, T, 128))
    q = 8.0 * u + 0.05 * rng.standard_normal((B, hkv * gq, n, 128))
    q, k, v = (torch.from_numpy(x.astype(np.float16)).cuda() for x in (q, k, v))
    plan = gtq.gtq_alloc_bits(gtq.make_config(B, hkv * gq, hkv, 4, 4, T), k, T)
    packed = torch.empty(plan.packed_bytes, dtype=torch.uint8, device="cuda")
    gtq.gtq_quantize_pack(plan, k, v, 0, T, packed)
    out = torch.empty_like(q)
    need = gtq.gtq_chunk_workspace(plan, T, n)
    assert need == 256, "the call is split"
    gtq.gtq_chunk_attn(plan, packed, T, q, out, workspace(need))
    torch.cuda.synchronize()
    assert gtq.gtq_status(plan) == gtq.GTQ_OK
    for b, h in ((0, 0), (3, 36)):
        K, V = Head(plan, hkv, 4, 4, T // 64).dequantised(packed, None, b, h, T)
        hs = slice(h * gq, (h + 1) * gq)
        ref = probabilities(q[b, hs].float().cpu().numpy(), K, n, True) @ V
        got = out[b, hs].double().cpu().numpy()
        e = np.linalg.norm(got - ref, axis=-1) / np.linalg.norm(ref, axis=-1)
        assert e.max() <= CHUNK_REL_L2, (b, h, e.max())
