"""The binding of the calls around the packed cache refuses tensors of other types than the kernels read, tensors that
are not on the plan's GPU, and lists of another length than the batch, before it calls the library."""

import types

import pytest

torch = pytest.importorskip("torch")

import decode_attention_13_b200 as gtq  # noqa: E402

B, HKV, HQ, N, T, KEEP = 2, 2, 4, 3, 100, 32


def plan():
    # (no handle: a call that got past the checks would be refused by the library, with another exception)
    return types.SimpleNamespace(cfg=gtq.make_config(B, HQ, HKV, 3, 3, 128), handle=None, device=0)


def on_gpu(x):
    """A CPU tensor that says it lies on GPU 0: type checks come to their turn without one."""
    x.get_device = lambda: 0
    return x


def zeros(shape, dtype=torch.float32):
    return on_gpu(torch.zeros(shape, dtype=dtype))


def args(**kw):
    a = dict(packed=zeros((1 << 12,), torch.uint8), q=zeros((B, HQ, N, 128), torch.float16),
             out=zeros((B, HQ, N, 128), torch.float16), ws=zeros((1 << 12,), torch.uint8), chunk_lens=None,
             w=zeros((B, HKV, T)), w_in=None, dst=zeros((1 << 12,), torch.uint8), new_lens=zeros((B,), torch.int32),
             w_out=None, kept=None)
    a.update(kw)
    return types.SimpleNamespace(**a)


def chunk(a):
    gtq.gtq_chunk_attn(plan(), a.packed, T, a.q, a.out, a.ws, chunk_lens=a.chunk_lens)


def weights(a):
    gtq.gtq_attn_weights(plan(), a.packed, T, a.q, a.w, a.ws, weights_in=a.w_in, chunk_lens=a.chunk_lens)


def evict(a):
    gtq.gtq_evict(plan(), a.packed, T, a.w, KEEP, a.dst, a.new_lens, a.ws, weights_out=a.w_out, kept=a.kept)


OTHER_TYPES = [
    (chunk, dict(q=zeros((B, HQ, N, 128), torch.bfloat16), out=zeros((B, HQ, N, 128), torch.bfloat16))),
    (chunk, dict(out=zeros((B, HQ, N, 128), torch.bfloat16))),
    (chunk, dict(q=zeros((B, HQ, N, 128), torch.float32))),
    (chunk, dict(chunk_lens=zeros((B,), torch.int64))),
    (chunk, dict(chunk_lens=zeros((B,), torch.float32))),
    (weights, dict(q=zeros((B, HQ, N, 128), torch.bfloat16))),
    (weights, dict(chunk_lens=zeros((B,), torch.int64))),
    (weights, dict(w=zeros((B, HKV, T), torch.int32))),
    (weights, dict(w_in=zeros((B, HKV, T), torch.int32))),
    (evict, dict(w=zeros((B, HKV, T), torch.int32))),
    (evict, dict(w_out=zeros((B, HKV, KEEP), torch.int32))),
    (evict, dict(kept=zeros((B, HKV, KEEP), torch.float32))),
    (evict, dict(kept=zeros((B, HKV, KEEP), torch.int64))),
    (evict, dict(new_lens=zeros((B,), torch.float32))),
    (evict, dict(new_lens=zeros((B,), torch.int64))),
]


@pytest.mark.parametrize("i", range(len(OTHER_TYPES)))
def test_other_types_are_refused(i):
    call, kw = OTHER_TYPES[i]
    with pytest.raises(ValueError):
        call(args(**kw))


@pytest.mark.parametrize("lens", [(1,), (3,), (B, 2)])
def test_lists_of_another_length_are_refused(lens):
    for call in (chunk, weights):
        with pytest.raises(ValueError):
            call(args(chunk_lens=zeros(lens, torch.int32)))
    with pytest.raises(ValueError):
        evict(args(new_lens=zeros(lens, torch.int32)))


def test_lists_with_gaps_are_refused():
    every_other = on_gpu(torch.zeros((2 * B,), dtype=torch.int32)[::2])
    for call, name in ((chunk, "chunk_lens"), (weights, "chunk_lens"), (evict, "new_lens")):
        with pytest.raises(ValueError):
            call(args(**{name: every_other}))


def test_what_is_right_reaches_the_library():
    for call in (chunk, weights, evict):
        with pytest.raises(gtq.GtqError):   # the plan without a handle
            call(args(chunk_lens=zeros((B,), torch.int32), kept=zeros((B, HKV, KEEP), torch.int32),
                      w_out=zeros((B, HKV, KEEP)), w_in=zeros((B, HKV, T))))


@pytest.mark.parametrize("call,names", [
    (chunk, ("packed", "q", "out", "ws", "chunk_lens")),
    (weights, ("packed", "q", "w", "w_in", "ws", "chunk_lens")),
    (evict, ("packed", "w", "dst", "new_lens", "ws", "w_out", "kept")),
])
def test_tensors_of_the_host_or_another_gpu_are_refused(call, names):
    lens = zeros((B,), torch.int32)
    full = dict(chunk_lens=lens, kept=zeros((B, HKV, KEEP), torch.int32), w_out=zeros((B, HKV, KEEP)), w_in=zeros((B, HKV, T)))
    for name in names:
        good = getattr(args(**full), name)
        for where in (-1, 1):
            bad = good.clone()
            bad.get_device = lambda where=where: where
            with pytest.raises(ValueError):
                call(args(**dict(full, **{name: bad})))


def test_rope_takes_its_configs_type_on_the_gpu_only():
    half, full = gtq.make_rope(128, 1e4), gtq.make_rope(128, 1e4, dtype=gtq.DTYPE_FP32)
    x = {t: torch.zeros((1, 2, 3, 128), dtype=t) for t in (torch.float16, torch.bfloat16, torch.float32, torch.int32)}
    for cfg, t in ((half, torch.bfloat16), (half, torch.float32), (full, torch.float16), (full, torch.int32)):
        for kw in (dict(q=x[t]), dict(k=x[t])):
            with pytest.raises(ValueError, match="must be float"):
                gtq.gtq_rope(cfg, **kw)
    with pytest.raises(ValueError, match="GPU"):
        gtq.gtq_rope(half, x[torch.float16])


@pytest.mark.gpu
def test_rope_refuses_on_the_gpu():
    x = torch.ones((1, 2, 3, 128), dtype=torch.float16, device="cuda")
    cfg = gtq.make_rope(128, 1e4)
    for kw in (dict(q=x, q_out=x.bfloat16()), dict(q=x, positions=torch.zeros(3, dtype=torch.float64, device="cuda")),
               dict(q=x, positions=torch.zeros(3, dtype=torch.int64)), dict(q=x, k=x.float()), dict(q=x, k=x.cpu()),
               dict(q=x, q_out=torch.empty_like(x, device="cpu"))):
        with pytest.raises(ValueError):
            gtq.gtq_rope(cfg, **kw)
    torch.cuda.synchronize()
    assert bool((x == 1).all())


@pytest.mark.gpu
def test_plans_know_their_gpu():
    k = torch.randn((1, 1, 64, 128), device="cuda").half()
    p = gtq.gtq_alloc_bits(gtq.make_config(1, 1, 1, 3, 3, 64), k, 64)
    assert p.device == torch.cuda.current_device()
