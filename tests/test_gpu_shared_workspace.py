"""Calls of changing sizes one behind the other on one stream and one workspace: it holds nothing between calls, and no
call starts to write it before the one before has read it."""

import pytest

torch = pytest.importorskip("torch")

import decode_attention_13_b200 as gtq  # noqa: E402
from tests.serving import Cache, workspace  # noqa: E402
from tests.test_gpu_chunk import run_chunk, run_weights, same  # noqa: E402

pytestmark = pytest.mark.gpu

# new tokens and bound on the lengths of the calls in their order: split over the tokens or not, every form of the kernels
CALLS = [(9, 9000), (1, 9000), (40, 300), (2, 9000), (1, 300), (80, 9000), (3, 300), (20, 9000), (1, 9000), (40, 9000)]


@pytest.mark.parametrize("seed", range(2))
def test_one_workspace_for_calls_of_all_sizes(seed):
    c = Cache([9000, 4100], 1, 8, 3, 3, seed=seed)
    sizes = [f(c.plan, T, n) for n, T in CALLS for f in (gtq.gtq_chunk_workspace, gtq.gtq_weights_workspace)]
    ws = workspace(max(sizes + [gtq.gtq_evict_workspace(c.plan, c.cap)]))
    q = {n: c.queries(n, seed=n) for n, _ in CALLS}
    # each by itself, with a workspace of its own
    want = [(run_chunk(c, q[n], n, None, True, T=T), run_weights(c, q[n], n, None, True, T=T)) for n, T in CALLS]
    w = torch.rand((2, 1, c.cap), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")
    one_ws = workspace(gtq.gtq_evict_workspace(c.plan, c.cap))

    def evict(dst, lens, space):
        gtq.gtq_evict(c.plan, c.packed, c.cap, w, 3000, dst, lens, space, n_first=4, n_recent=64, layout=c.layout)

    dst0, lens0 = torch.zeros_like(c.packed), torch.zeros_like(c.seq_lens)
    evict(dst0, lens0, one_ws)
    outs = [(torch.full_like(q[n], 77.0), torch.full((2, 1, c.cap), 77.0, device="cuda")) for n, _ in CALLS]
    moved = [(torch.zeros_like(c.packed), torch.zeros_like(lens0)) for _ in CALLS]
    torch.cuda.synchronize()
    for (n, T), (o, wo), (dst, lens) in zip(CALLS, outs, moved):
        gtq.gtq_chunk_attn(c.plan, c.packed, T, q[n], o, ws, layout=c.layout)
        gtq.gtq_attn_weights(c.plan, c.packed, T, q[n], wo, ws, layout=c.layout)
        evict(dst, lens, ws)
    torch.cuda.synchronize()
    assert gtq.gtq_status(c.plan) == gtq.GTQ_OK
    for (n, T), (o, wo), (a, b), (dst, lens) in zip(CALLS, outs, want, moved):
        assert same(o, a, n, c) and torch.equal(wo, b), (n, T)
        assert torch.equal(dst, dst0) and torch.equal(lens, lens0), (n, T)
