"""Refusals of the calls over a plan (a plan needs a device): nothing is launched, outputs stay as they were."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import decode_attention_13_b200 as gtq  # noqa: E402
from decode_attention_13_b200 import binding  # noqa: E402
from tests.serving import Cache, workspace  # noqa: E402

pytestmark = pytest.mark.gpu

INV, UNS = gtq.GTQ_ERR_INVALID, gtq.GTQ_ERR_UNSUPPORTED


class Calls:
    def __init__(self, vb=3, n=4):
        self.c = Cache([100, 80], 2, 2, 3, vb, cap=128, seed=1)
        self.n = n
        self.q = self.c.queries(n)
        self.out = torch.full_like(self.q, 5.0)
        self.w = torch.full((2, 2, 128), 5.0, device="cuda")
        self.ws = workspace(1 << 22)

    def chunk(self, T=100, out=None, ws=None, ws_bytes=1 << 22, lay=None, packed=None, q=None, **kw):
        ch = binding._chunk(self.c.plan, self.q, self.out, None, True)
        for k, v in kw.items():
            setattr(ch, k, v)
        return ch, [self.c.plan.handle, self.c.packed.data_ptr() if packed is None else packed, T,
                    ctypes.byref(lay or self.c.layout), ctypes.byref(ch), self.q.data_ptr() if q is None else q,
                    self.out.data_ptr() if out is None else out, self.ws.data_ptr() if ws is None else ws, ws_bytes, None]

    def attn(self, **kw):
        _, args = self.chunk(**kw)
        return binding.library().gtq_chunk_attn(*args)

    def weights(self, w_out=None, w_strides=(256, 128), **kw):
        _, a = self.chunk(**kw)
        return binding.library().gtq_attn_weights(*a[:6], None, self.w.data_ptr() if w_out is None else w_out,
                                                  (ctypes.c_int64 * 2)(*w_strides), a[7], a[8], None)


BAD = [dict(T=0), dict(T=129), dict(n_tokens=0), dict(n_tokens=(1 << 20) + 1), dict(reserved=1), dict(causal=2),
       dict(chunk_lens_dev=0x1002), dict(q_strides=(ctypes.c_int64 * 4)(0, 0, 0, 2)),
       dict(q_strides=(ctypes.c_int64 * 4)(0, 4, 0, 1)), dict(q_strides=(ctypes.c_int64 * 4)(-8, 0, 0, 1)),
       dict(ws_bytes=0), dict(ws=0x1010), dict(packed=0x1004), dict(q=0x1008), dict(packed=0), dict(q=0), dict(ws=0)]


@pytest.mark.parametrize("i", range(len(BAD)))
def test_chunk_and_weights_refuse(i):
    x = Calls()
    assert x.attn(**BAD[i]) == INV
    assert x.weights(**BAD[i]) == INV
    torch.cuda.synchronize()
    assert bool((x.out == 5.0).all()) and bool((x.w == 5.0).all())


def test_more_refusals():
    x = Calls()
    assert x.attn(out=0) == INV and x.attn(out=0x1008) == INV
    assert x.attn(out_strides=(ctypes.c_int64 * 4)(0, 4, 0, 1)) == INV
    assert x.weights(w_out=0) == INV and x.weights(w_out=0x1002) == INV and x.weights(w_strides=(-1, 0)) == INV
    narrow = binding.gtq_seq_layout(x.c.seq_lens.data_ptr(), x.c.seq_lens.data_ptr(), 1)
    assert x.attn(lay=narrow) == INV and x.weights(lay=narrow) == INV
    assert Calls(vb=0).attn() == UNS     # values of a K-only plan are not in the cache
    assert gtq.gtq_chunk_workspace(x.c.plan, 0, 1) == 0 and gtq.gtq_chunk_workspace(x.c.plan, 129, 1) == 0
    assert gtq.gtq_weights_workspace(x.c.plan, 100, 0) == 0 and gtq.gtq_evict_workspace(x.c.plan, 129) == 0
    with pytest.raises(ValueError):
        gtq.gtq_chunk_attn(x.c.plan, x.c.packed, 100, x.q.float(), x.out, x.ws)
    with pytest.raises(ValueError):
        gtq.gtq_attn_weights(x.c.plan, x.c.packed, 100, x.q, x.w[:, :, :64], x.ws)
    torch.cuda.synchronize()
    assert bool((x.out == 5.0).all()) and bool((x.w == 5.0).all())


def test_evict_refuses():
    c = Cache([100, 80], 2, 2, 3, 3, cap=128, seed=1)
    w = torch.rand((2, 2, 128), device="cuda")
    dst = torch.full((c.plan.packed_bytes,), 9, dtype=torch.uint8, device="cuda")
    lens = torch.full((2,), 9, dtype=torch.int32, device="cuda")
    ws = workspace(1 << 20)

    def call(T=100, dst_p=None, dst_bytes=None, ws_p=None, ws_bytes=1 << 20, dst_lay=None, src=None, **kw):
        ev = binding.gtq_eviction(32, 1, 2, w.data_ptr(), (ctypes.c_int64 * 2)(256, 128), None,
                                  (ctypes.c_int64 * 2)(0, 0), None, lens.data_ptr())
        for k, v in kw.items():
            setattr(ev, k, v)
        return binding.library().gtq_evict(
            c.plan.handle, c.packed.data_ptr() if src is None else src, T, ctypes.byref(c.layout), ctypes.byref(ev),
            dst.data_ptr() if dst_p is None else dst_p, c.plan.packed_bytes if dst_bytes is None else dst_bytes,
            None if dst_lay is None else ctypes.byref(dst_lay), ws.data_ptr() if ws_p is None else ws_p, ws_bytes, None)

    for kw in (dict(T=0), dict(T=129), dict(keep=0), dict(keep=129), dict(n_first=-1), dict(n_recent=-1),
               dict(n_first=31), dict(n_recent=33), dict(n_first=2 ** 62, n_recent=2 ** 62), dict(weights_dev=None),
               dict(weights_dev=0x1002), dict(new_lens_dev=None), dict(kept_dev=0x1002), dict(weights_out_dev=0x1001),
               dict(w_strides=(ctypes.c_int64 * 2)(-1, 0)), dict(dst_bytes=c.plan.packed_bytes - 1), dict(ws_bytes=16),
               dict(ws_p=0x1010), dict(dst_p=0), dict(src=0), dict(dst_p=c.packed.data_ptr()),
               dict(dst_p=c.packed.data_ptr() + 64 * 1024 // 2),
               dict(keep=128, dst_lay=binding.gtq_seq_layout(None, lens.data_ptr(), 1))):
        assert call(**kw) == INV, kw
    torch.cuda.synchronize()
    assert bool((dst == 9).all()) and bool((lens == 9).all())
    with pytest.raises(ValueError):
        gtq.gtq_evict(c.plan, c.packed, 100, w[:, :, :90], 32, dst, lens, ws)
    with pytest.raises(ValueError):
        gtq.gtq_evict(c.plan, c.packed, 100, w, 32, dst, lens, ws, kept=torch.zeros((2, 2, 31), dtype=torch.int32, device="cuda"))
    assert call() == gtq.GTQ_OK


def test_outputs_that_overlap_are_refused():
    x = Calls()
    qs = x.q.stride()
    for i in range(3):  # one row of out for several of q
        s = list(x.out.stride())
        s[i] = 0
        assert x.attn(out_strides=(ctypes.c_int64 * 4)(*s)) == INV
    # in place, but in another order of dims
    assert x.attn(out=x.q.data_ptr(), out_strides=(ctypes.c_int64 * 4)(qs[0], qs[2], qs[1], 1)) == INV
    assert x.weights(w_strides=(0, 128)) == INV and x.weights(w_strides=(256, 0)) == INV
    c, w = x.c, torch.rand((2, 2, 128), device="cuda")
    ws = workspace(1 << 20)
    dst = torch.full((c.plan.packed_bytes,), 9, dtype=torch.uint8, device="cuda")
    lens = torch.full((2,), 9, dtype=torch.int32, device="cuda")
    before = c.seq_lens.clone(), w.clone()
    bad = [dict(new_lens=c.seq_lens), dict(weights_out=w), dict(weights_out=torch.zeros((1, 2, 32), device="cuda").expand(2, 2, 32))]
    for kw in bad:
        with pytest.raises(gtq.GtqError):
            gtq.gtq_evict(c.plan, c.packed, 100, w, 32, dst, kw.pop("new_lens", lens), ws, layout=c.layout, **kw)
    d = Cache([100, 80], 2, 2, 3, 3, cap=128, paged=True, seed=1)
    with pytest.raises(gtq.GtqError):  # the source's own pages
        gtq.gtq_evict(d.plan, d.packed, 100, w, 32, d.packed, lens, ws, layout=d.layout,
                      dst_layout=gtq.seq_layout(None, d.table))
    torch.cuda.synchronize()
    assert torch.equal(c.seq_lens, before[0]) and torch.equal(w, before[1])
    assert bool((dst == 9).all()) and bool((lens == 9).all())
