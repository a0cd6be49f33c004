"""gtq_evict: which tokens stay, and that their codes and norms arrive bit for bit; then the operators in a row as a
server runs them."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import decode_attention_13_b200 as gtq  # noqa: E402
from tests import layout  # noqa: E402
from tests.serving import Cache, probabilities, workspace  # noqa: E402
from tests.test_gpu_parity import DECODE_REL_L2, rel_l2  # noqa: E402

pytestmark = pytest.mark.gpu


def keepers(w, n, keep, first, recent):
    """The indices that stay of a head's n tokens, by sorting (place, then weight, then index)."""
    t = np.arange(n)
    placed = (t < first) | (t >= n - recent)
    v = np.where(np.isnan(w[:n]), -np.inf, w[:n]).astype(np.float64)
    nan = np.isnan(w[:n])
    return np.sort(np.lexsort((t, nan, -v, ~placed))[:keep])


def run_evict(c, w, keep, first, recent, T=None, dst_paged=False, give=True):
    nk = (min(keep, c.cap) + 63) // 64
    table = None
    if dst_paged:
        pages = c.B * nk + 2
        table = torch.tensor(c.rng.permutation(pages)[:c.B * nk].reshape(c.B, nk), dtype=torch.int32, device="cuda")
        dst = torch.full((pages * c.hkv * c.tb,), 0x5A, dtype=torch.uint8, device="cuda")
    else:
        dst = torch.full((c.plan.packed_bytes,), 0x5A, dtype=torch.uint8, device="cuda")
    lens = torch.full((c.B,), -5, dtype=torch.int32, device="cuda")
    kept = torch.full((c.B, c.hkv, keep), -7, dtype=torch.int32, device="cuda") if give else None
    wo = torch.full((c.B, c.hkv, keep), 77.0, device="cuda") if give else None
    ws = workspace(gtq.gtq_evict_workspace(c.plan, T or c.cap))
    gtq.gtq_evict(c.plan, c.packed, T or c.cap, w, keep, dst, lens, ws, n_first=first, n_recent=recent, layout=c.layout,
                  dst_layout=gtq.seq_layout(None, table) if dst_paged else None, weights_out=wo, kept=kept)
    torch.cuda.synchronize()
    assert gtq.gtq_status(c.plan) == gtq.GTQ_OK
    return dst, table, lens, kept, wo


def check_evict(c, w, keep, first, recent, dst, table, lens, kept, wo):
    wn = w.cpu().numpy()
    raw = dst.cpu().numpy()
    touched = np.zeros(len(raw) // c.tb, bool)
    for b, L in enumerate(c.lens):
        n = min(L, keep)
        assert int(lens[b]) == n
        for h in range(c.hkv):
            want = keepers(wn[b, h], L, keep, first, recent)
            if kept is not None:
                assert np.array_equal(kept[b, h, :n].cpu().numpy(), want), (b, h)
                assert bool((kept[b, h, n:] == -1).all())
                assert np.array_equal(wo[b, h, :n].cpu().numpy(), wn[b, h][want], equal_nan=True)
                assert bool((wo[b, h, n:] == 77.0).all())
            nt = (n + 63) // 64
            for t in range(nt):
                touched[(int(table[b, t]) * c.hkv + h) if table is not None else (b * c.hkv + h) * c.tiles + t] = True
            if not n:
                continue
            buf = c.head_bytes(dst, table, b, h, nt)
            old = c.head(c.packed, c.table, b, h, L)
            new = layout.read_head(buf, c.bits[b, h], c.kb, c.vb, nt * 64)
            for (w0, c0, n0), (w1, c1, n1) in zip(old[0], new[0]):
                assert w0 == w1 and np.array_equal(c0[want], c1[:n])
                assert np.array_equal(n0[want].view(np.uint16), n1[:n].view(np.uint16))
                assert not c1[n:].any() and not n1[n:].view(np.uint16).any()    # nothing behind the last token
            if c.vb:
                assert np.array_equal(old[1][want], new[1][:n]) and not new[1][n:].any()
                assert np.array_equal(old[2][want].view(np.uint16), new[2][:n].view(np.uint16))
            spare = buf.reshape(nt, c.tb)[:, c.tb - 1024 + 128 * len(old[0]):]
            assert not spare.any()
    assert np.all(raw.reshape(-1, c.tb)[~touched] == 0x5A)


CASES = [
    # lens, hkv, kb, vb, src paged, dst paged, keep, first, recent
    ([200], 1, 3, 3, False, False, 64, 0, 0),
    ([200], 1, 3, 3, False, False, 1, 0, 0),
    ([1], 1, 3, 3, False, False, 1, 0, 1),
    ([500, 64, 0, 130, 3], 2, 3, 2, True, True, 100, 4, 16),
    ([500, 129], 2, 3, 2, False, True, 129, 4, 125),          # only first and last tokens stay
    ([700], 1, 2, 2, True, False, 700, 0, 10),                # everything stays
    ([700, 650], 1, 2, 4, True, True, 699, 1, 1),
    ([5000], 1, 4, 3, False, True, 77, 2, 5),                 # tiles far apart: more than one batch of sources
    ([9000, 4100], 2, 3, 3, True, True, 2000, 4, 64),         # several blocks search one head
    ([40000], 1, 3, 3, False, False, 10001, 4, 300),
    ([300], 1, 1, 1, False, True, 131, 0, 3),
    ([300], 1, 8, 8, True, True, 131, 0, 3),
    ([300], 1, 6, 7, False, True, 131, 0, 3),
    ([300], 1, 5, 5, False, True, 65, 0, 3),
    ([300, 70], 2, 3, 0, True, True, 66, 1, 3),               # keys alone are coded
]


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
@pytest.mark.parametrize("kind", ["spread", "ties"])
def test_evict(case, kind):
    lens, hkv, kb, vb, src_paged, dst_paged, keep, first, recent = case
    c = Cache(lens, hkv, 2, kb, vb, paged=src_paged, seed=len(lens) + keep)
    g = torch.Generator(device="cuda").manual_seed(keep)
    w = torch.exp(3 * torch.randn((c.B, hkv, c.cap), generator=g, device="cuda"))
    if kind == "ties":
        w = torch.where(w < 1.5, torch.zeros_like(w), torch.round(w))     # many zeros, many equal
        w[..., ::7] *= -1.0                                               # -0 among the zeros, and negative weights
    for b, L in enumerate(lens):
        w[b, :, L:] = float("nan")                                        # past the length nothing is looked at
    before = c.packed.clone()
    check_evict(c, w, keep, first, recent, *run_evict(c, w, keep, first, recent, dst_paged=dst_paged))
    assert torch.equal(before, c.packed)


class Codes(Cache):
    def read(self):  # nothing of it as numbers
        pass


@pytest.mark.parametrize("keep", [50, 70000, 262144])
@pytest.mark.parametrize("kind", ["spread", "ties"])
def test_evict_from_more_tokens_than_a_block_holds(keep, kind):
    # the stretches of the blocks of a head are longer than what stays in shared memory
    c = Codes([270000], 1, 2, 1, 1, seed=keep)
    g = torch.Generator(device="cuda").manual_seed(keep)
    w = torch.exp(3 * torch.randn((1, 1, c.cap), generator=g, device="cuda"))
    if kind == "ties":
        w = torch.where(w < 1.5, torch.zeros_like(w), torch.round(w))
    check_evict(c, w, keep, 4, 30, *run_evict(c, w, keep, 4, 30))


def test_evict_from_half_a_million_tokens():
    c = Codes([530000], 1, 1, 1, 1, seed=3)
    g = torch.Generator(device="cuda").manual_seed(3)
    w = torch.round(torch.exp(3 * torch.randn((1, 1, c.cap), generator=g, device="cuda")) * 8)
    check_evict(c, w, 30000, 4, 30, *run_evict(c, w, 30000, 4, 30))


def test_evict_odd_weights():
    c = Cache([400], 2, 2, 3, 3, seed=2)
    w = torch.randn((1, 2, 400), device="cuda")
    w[0, 0, 5:50] = float("nan")
    w[0, 0, 60:70] = float("inf")
    w[0, 0, 70:300] = float("-inf")
    w[0, 1, :] = float("nan")
    for keep in (5, 80, 360):
        check_evict(c, w, keep, 1, 2, *run_evict(c, w, keep, 1, 2))


def test_evict_without_the_optional_outputs_and_with_strides():
    c = Cache([333, 280], 2, 2, 3, 3, seed=4)
    big = torch.rand((2, 2, 500), device="cuda")
    w = big[:, :, :333]
    a = run_evict(c, w, 150, 4, 8)
    b = run_evict(c, w.contiguous(), 150, 4, 8, give=False)
    assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])
    check_evict(c, w.contiguous(), 150, 4, 8, *a)


def test_evict_with_a_bound_below_the_lengths():
    # T bounds every sequence: as if each held at most T tokens
    c = Cache([500, 90], 2, 2, 3, 3, paged=True, seed=14)
    w = torch.rand((2, 2, 500), device="cuda")
    got = run_evict(c, w, 120, 4, 16, T=200, dst_paged=True)
    c.lens = [200, 90]
    check_evict(c, w, 120, 4, 16, *got)


def test_evict_far_pages():
    # from pages beyond 4 GiB of a pool to others there
    c = Cache([700, 333], 2, 2, 3, 3, paged=True, seed=15)
    w = torch.rand((2, 2, 700), device="cuda")
    page = c.hkv * c.tb
    shift, n = (5 << 30) // page, (200 + 63) // 64
    far = c.table + shift
    pool = torch.full(((shift + c.pages + 2 * n) * page,), 0x5A, dtype=torch.uint8, device="cuda")
    pool[shift * page:(shift + c.pages) * page] = c.packed
    new = shift + c.pages + torch.arange(2 * n, dtype=torch.int32, device="cuda").reshape(2, n)
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    kept = torch.zeros((2, 2, 200), dtype=torch.int32, device="cuda")
    wo = torch.full((2, 2, 200), 77.0, device="cuda")
    gtq.gtq_evict(c.plan, pool, 700, w, 200, pool, lens, workspace(gtq.gtq_evict_workspace(c.plan, 700)), n_first=4,
                  n_recent=20, layout=gtq.seq_layout(c.seq_lens, far), dst_layout=gtq.seq_layout(None, new),
                  weights_out=wo, kept=kept)
    torch.cuda.synchronize()
    assert gtq.gtq_status(c.plan) == gtq.GTQ_OK
    assert torch.equal(pool[shift * page:(shift + c.pages) * page], c.packed)
    assert bool((pool[:shift * page] == 0x5A).all())
    dst = pool[(shift + c.pages) * page:].clone()
    check_evict(c, w, 200, 4, 20, dst, new - (shift + c.pages), lens, kept, wo)


def test_evict_in_a_graph_with_growing_lengths():
    # one captured call, replayed after the lengths changed: they are read on the device
    c = Cache([600, 500], 1, 4, 3, 3, seed=8)
    w = torch.rand((2, 1, 600), device="cuda")
    dst = torch.full((c.plan.packed_bytes,), 0x5A, dtype=torch.uint8, device="cuda")
    lens = torch.zeros((2,), dtype=torch.int32, device="cuda")
    kept = torch.zeros((2, 1, 128), dtype=torch.int32, device="cuda")
    wo = torch.full((2, 1, 128), 77.0, device="cuda")
    ws = workspace(gtq.gtq_evict_workspace(c.plan, 600))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            gtq.gtq_evict(c.plan, c.packed, 600, w, 128, dst, lens, ws, n_first=2, n_recent=9, layout=c.layout,
                          weights_out=wo, kept=kept, stream=s)
        for now in ([600, 500], [90, 300]):
            c.seq_lens.copy_(torch.tensor(now, dtype=torch.int32))
            dst.fill_(0x5A)
            wo.fill_(77.0)
            g.replay()
            s.synchronize()
            c.lens = now
            check_evict(c, w, 128, 2, 9, dst, None, lens, kept, wo)


def test_a_turn_then_an_eviction_then_decode():
    """rope -> pack -> a chunk's tokens appended -> attention of the chunk -> weights -> eviction -> append -> decode."""
    B, hkv, gq, T0, n, cap, keep = 2, 2, 4, [700, 520], 24, 1024, 384
    hq = hkv * gq
    rng = np.random.default_rng(77)
    std = np.exp(-3.0 * np.arange(64) / 64)
    std[[3, 20]] *= 8
    std = np.concatenate([std, std])
    raw = lambda h: torch.from_numpy((rng.standard_normal((B, cap, h, 128)) * std).astype(np.float16)).cuda().transpose(1, 2)  # noqa: E731
    k, v = raw(hkv), torch.from_numpy(rng.standard_normal((B, hkv, cap, 128)).astype(np.float16)).cuda()
    k_rot = torch.empty((B, hkv, cap, 128), dtype=torch.float16, device="cuda")
    rope = gtq.make_rope(128, 5e5, scaling=gtq.ROPE_LLAMA3, factor=8.0, original_context=8192.0)
    gtq.gtq_rope(rope, k=k, k_out=k_rot)
    tiles = (cap + 63) // 64
    table = torch.tensor(rng.permutation(B * tiles).reshape(B, tiles), dtype=torch.int32, device="cuda")
    lens = torch.tensor(T0, dtype=torch.int32, device="cuda")
    lay = gtq.seq_layout(lens, table)
    plan = gtq.gtq_alloc_bits_ex(gtq.make_config(B, hq, hkv, 3, 3, cap), k_rot, cap, lay)
    tb = layout.tile_bytes(3, 3)
    pool = torch.full((B * tiles * hkv * tb,), 0xA5, dtype=torch.uint8, device="cuda")
    gtq.gtq_quantize_pack_ex(plan, k_rot, v, 0, cap, pool, lay)
    # a turn of n tokens: appended in pieces the append kernel and the quantizer take, then attended
    lens += n
    gtq.gtq_quantize_pack_ex(plan, k_rot, v, gtq.GTQ_T0_TAIL, n, pool, lay)
    q = raw(hq)[:, :, :n]
    pos = lens.long()[:, None] - n + torch.arange(n, device="cuda")
    q_rot = torch.empty((B, hq, n, 128), dtype=torch.float16, device="cuda")
    gtq.gtq_rope(rope, q, q_rot, positions=pos)
    out = torch.empty_like(q_rot)
    gtq.gtq_chunk_attn(plan, pool, cap, q_rot, out, workspace(gtq.gtq_chunk_workspace(plan, cap, n)), layout=lay)
    w = torch.zeros((B, hkv, cap), device="cuda")
    gtq.gtq_attn_weights(plan, pool, cap, q_rot, w, workspace(gtq.gtq_weights_workspace(plan, cap, n)), weights_in=w,
                         layout=lay)
    # appends at the tail want a table as wide as the plan's capacity
    table2 = torch.tensor(rng.permutation(B * tiles).reshape(B, tiles), dtype=torch.int32, device="cuda")
    pool2 = torch.full_like(pool, 0x5A)
    lens2 = torch.zeros_like(lens)
    kept = torch.zeros((B, hkv, keep), dtype=torch.int32, device="cuda")
    gtq.gtq_evict(plan, pool, cap, w, keep, pool2, lens2, workspace(gtq.gtq_evict_workspace(plan, cap)), n_first=4,
                  n_recent=32, layout=lay, dst_layout=gtq.seq_layout(None, table2), kept=kept)
    # the next token goes behind the kept ones: row `keep` of tensors that hold it there
    k_next = torch.empty((B, hkv, keep + 1, 128), dtype=torch.float16, device="cuda")
    v_next = torch.zeros_like(k_next)
    new = raw(hkv)[:, :, :1]
    gtq.gtq_rope(rope, k=new, k_out=k_next[:, :, keep:], positions=lens.long()[:, None])
    v_next[:, :, keep:] = v[:, :, -1:]
    lens2 += 1
    lay2 = gtq.seq_layout(lens2, table2)
    gtq.gtq_quantize_pack_ex(plan, k_next, v_next, gtq.GTQ_T0_TAIL, 1, pool2, lay2)
    qd = q_rot[:, :, -1].contiguous()
    dec = torch.empty((B, hq, 128), dtype=torch.float32, device="cuda")
    gtq.gtq_decode_attn_ex(plan, pool2, keep + 1, qd, dec, lay2)
    torch.cuda.synchronize()
    assert gtq.gtq_status(plan) == gtq.GTQ_OK

    class Held(Cache):  # reading only
        def __init__(self):
            self.hkv, self.kb, self.vb, self.pairing, self.tb, self.tiles = hkv, 3, 3, 0, tb, tiles
            self.bits = gtq.gtq_get_bits(plan)

    r = Held()
    for b in range(B):
        L = T0[b] + n
        for h in range(hkv):
            K, V = r.dequantised(pool, table, b, h, L)
            hs = slice(h * gq, (h + 1) * gq)
            p = probabilities(q_rot[b, hs].float().cpu().numpy(), K, n, True)
            assert rel_l2(out[b, hs].double().cpu().numpy(), p @ V) <= DECODE_REL_L2 + 2.0 ** -11
            want = keepers(w[b, h].cpu().numpy(), L, keep, 4, 32)
            assert np.array_equal(kept[b, h].cpu().numpy(), want)
            K2, V2 = r.dequantised(pool2, table2, b, h, keep + 1)
            assert np.array_equal(K2[:keep], K[want]) and np.array_equal(V2[:keep], V[want])
            p = probabilities(qd[b, hs].float().cpu().numpy()[:, None], K2, 1, True)
            assert rel_l2(dec[b, hs].double().cpu().numpy(), (p @ V2)[:, 0]) <= DECODE_REL_L2
