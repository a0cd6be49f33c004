"""gtq_chunk_attn and gtq_attn_weights against attention in fp64 on what the packed cache holds."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import decode_attention_13_b200 as gtq  # noqa: E402
from tests.serving import Cache, probabilities, workspace  # noqa: E402
from tests.test_gpu_parity import DECODE_REL_L2, rel_l2  # noqa: E402

pytestmark = pytest.mark.gpu

# Attention over identical packed inputs is held to the framework's decode criterion; the fp16 result adds half a step.
CHUNK_REL_L2 = DECODE_REL_L2 + 2.0 ** -11

CASES = [
    # lens, hkv, gq, kb, vb, paged, pairing, n, chunk_lens, causal
    ([64], 1, 1, 3, 3, False, 0, 1, None, True),
    ([1], 1, 4, 3, 3, False, 0, 1, None, True),
    ([300, 1, 0, 129], 2, 4, 3, 3, True, 0, 5, [5, 1, 0, 3], True),
    ([200, 7], 2, 7, 3, 2, True, 0, 1, None, True),
    ([1000], 1, 8, 2, 2, False, 0, 37, None, True),
    ([1000], 1, 8, 2, 2, False, 1, 37, None, False),
    ([513, 450], 1, 16, 4, 4, True, 1, 130, [130, 77], True),
    ([700], 2, 2, 3, 3, False, 0, 300, None, True),
    ([40, 3], 1, 3, 3, 3, False, 0, 64, [64, 64], True),     # rows before the first token see nothing
    ([130], 1, 1, 1, 1, False, 0, 3, None, True),
    ([130], 1, 2, 8, 8, True, 0, 3, None, True),
    ([257], 1, 5, 5, 6, False, 0, 17, None, True),
    ([320], 1, 6, 6, 5, False, 1, 17, None, False),
    ([320], 1, 6, 7, 7, False, 0, 9, None, True),
    ([5000], 1, 128, 3, 3, False, 0, 3, None, True),         # a group of 128 query heads
    ([9000, 2500], 1, 8, 3, 2, True, 0, 2, None, True),      # a long context: its work is split
    ([9000], 2, 4, 3, 3, False, 0, 65, None, True),
]


def run_chunk(c, q, n, cl, causal, T=None, out=None):
    out = torch.full_like(q, 77.0) if out is None else out
    ws = workspace(gtq.gtq_chunk_workspace(c.plan, T or c.cap, n))
    lens = None if cl is None else torch.tensor(cl, dtype=torch.int32, device="cuda")
    gtq.gtq_chunk_attn(c.plan, c.packed, T or c.cap, q, out, ws, layout=c.layout, chunk_lens=lens, causal=causal)
    torch.cuda.synchronize()
    assert gtq.gtq_status(c.plan) == gtq.GTQ_OK
    return out


def check_chunk(c, q, out, n, cl, causal):
    qn, on = q.float().cpu().numpy(), out.double().cpu().numpy()
    for b, L in enumerate(c.lens):
        nb = n if cl is None else cl[b]
        assert np.all(on[b, :, nb:] == 77.0)
        for h in range(c.hkv):
            hs = slice(h * c.gq, (h + 1) * c.gq)
            got = on[b, hs, :nb]
            p = probabilities(qn[b, hs, :nb], c.K[b][h], nb, causal)
            ref = p @ c.V[b][h]
            blind = p.sum(-1) == 0
            assert np.all(got[blind] == 0.0)
            if ref.size and not np.all(blind):
                assert rel_l2(got, ref) <= CHUNK_REL_L2, (b, h, rel_l2(got, ref))
                # no row is far off on its own: 8 times the bound of them all
                e = np.linalg.norm(got - ref, axis=-1)[~blind] / np.linalg.norm(ref, axis=-1)[~blind]
                assert e.max() <= 8 * CHUNK_REL_L2, (b, h, e.max())


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_chunk_against_fp64(case):
    lens, hkv, gq, kb, vb, paged, pairing, n, cl, causal = case
    c = Cache(lens, hkv, gq, kb, vb, paged=paged, pairing=pairing, seed=len(lens) + n)
    q = c.queries(n, seed=n)
    for b in range(c.B):
        if cl is not None:
            q[b, :, cl[b]:] = float("nan")      # rows a sequence does not bring are never looked at
    before = c.packed.clone()
    out = run_chunk(c, q, n, cl, causal)
    check_chunk(c, q, out, n, cl, causal)
    assert torch.equal(before, c.packed)


def test_chunk_takes_any_order_of_dims():
    c = Cache([400, 250], 2, 4, 3, 3, seed=3)
    n = 21
    q = c.queries(n, seed=4)
    want = run_chunk(c, q, n, None, True)
    # as projections leave them: [B][n][heads][128], and padded rows
    qt = torch.zeros((2, n, c.hq, 136), dtype=torch.float16, device="cuda")
    qt[..., :128] = q.transpose(1, 2)
    out = torch.full((2, n, c.hq, 128), 77.0, dtype=torch.float16, device="cuda")
    got = run_chunk(c, qt[..., :128].transpose(1, 2), n, None, True, out=out.transpose(1, 2))
    assert torch.equal(got, want)


def test_chunk_of_one_agrees_with_decode():
    c = Cache([1500, 333], 2, 4, 3, 3, paged=True, seed=6)
    q = c.queries(1, seed=8)
    out = run_chunk(c, q, 1, None, True).float()
    ref = torch.empty((2, c.hq, 128), dtype=torch.float32, device="cuda")
    gtq.gtq_decode_attn_ex(c.plan, c.packed, c.cap, q[:, :, 0].contiguous(), ref, c.layout)
    assert rel_l2(out[:, :, 0].cpu().numpy(), ref.cpu().numpy()) <= 2 * CHUNK_REL_L2


def test_chunk_with_a_bound_below_the_lengths():
    # T bounds every sequence: as if each held at most T tokens
    c = Cache([500, 90], 1, 4, 3, 3, seed=9)
    q = c.queries(6, seed=1)
    out = run_chunk(c, q, 6, None, True, T=200)
    d = Cache([500, 90], 1, 4, 3, 3, seed=9)
    d.K = [[k[:200] for k in row] for row in d.K]
    d.V = [[v[:200] for v in row] for row in d.V]
    d.lens = [200, 90]
    check_chunk(d, q, out, 6, None, True)


def test_chunk_peaked_and_flat_rows():
    # keys 20 times as large: one token takes everything; a zero query: every token the same
    c = Cache([700], 1, 4, 3, 3, seed=12, scale=20.0)
    q = c.queries(8, seed=2)
    q[:, :, 3] = 0
    out = run_chunk(c, q, 8, None, True)
    on = out.double().cpu().numpy()[0]
    p = probabilities(q.float().cpu().numpy()[0], c.K[0][0], 8, True)
    ref = p @ c.V[0][0]
    assert rel_l2(on[:, 3], ref[:, 3]) <= CHUNK_REL_L2
    # logits of hundreds leave no room for a bound on single weights, but every row stays a mean of the values: no
    # coordinate leaves their range, but for the roundings of the weights' sum and of the result (2^-10 together)
    V = c.V[0][0]
    assert np.all(np.isfinite(on))
    slack = 2.0 ** -10 * np.abs(V).max()
    assert np.all(on <= V.max(0) + slack) and np.all(on >= V.min(0) - slack)


@pytest.mark.parametrize("seed", range(3))
def test_chunk_twice_gives_the_same_bits(seed):
    c = Cache([3000, 1200], 1, 8, 3, 3, seed=seed)
    q = c.queries(11, seed=seed)
    assert torch.equal(run_chunk(c, q, 11, None, True), run_chunk(c, q, 11, None, True))


def weights_bound(c, b, h, q, rows):
    """Relative bound on a weight: scores are sums of 128 products in fp32 (or better), |error| <= 128 2^-24 times the
    sum of the products' sizes, in the row's logit and in the sum that it is divided by; those sums run over the
    tokens, the weights' over the rows; exp adds a few units."""
    s = np.max(np.linalg.norm(q, axis=-1)) * np.max(np.linalg.norm(c.K[b][h], axis=-1)) / np.sqrt(128.0)
    return 2 * 128 * 2.0 ** -24 * s + (rows + c.lens[b] + 16) * 2.0 ** -24


def run_weights(c, q, n, cl, causal, w_in=None, w_out=None, T=None):
    T = T or c.cap
    w_out = torch.full((c.B, c.hkv, c.cap), 77.0, device="cuda") if w_out is None else w_out
    ws = workspace(gtq.gtq_weights_workspace(c.plan, T, n))
    lens = None if cl is None else torch.tensor(cl, dtype=torch.int32, device="cuda")
    gtq.gtq_attn_weights(c.plan, c.packed, T, q, w_out, ws, weights_in=w_in, layout=c.layout, chunk_lens=lens,
                         causal=causal)
    torch.cuda.synchronize()
    assert gtq.gtq_status(c.plan) == gtq.GTQ_OK
    return w_out


WEIGHT_CASES = [i for i, x in enumerate(CASES) if x[7] * x[2] <= 2000] + [-1, -2]


@pytest.mark.parametrize("i", WEIGHT_CASES)
def test_weights_against_fp64(i):
    if i < 0:  # keys alone are coded
        lens, hkv, gq, kb, vb, paged, pairing, n, cl, causal = [700, 65], 2, 4, 3, 0, i == -2, 0, 9, [9, 2], True
    else:
        lens, hkv, gq, kb, vb, paged, pairing, n, cl, causal = CASES[i]
    c = Cache(lens, hkv, gq, kb, vb, paged=paged, pairing=pairing, seed=len(lens) + n)
    q = c.queries(n, seed=n)
    qn = q.float().cpu().numpy()
    for b in range(c.B):
        if cl is not None:
            q[b, :, cl[b]:] = float("nan")
    w_in = torch.rand((c.B, c.hkv, c.cap), device="cuda") if n % 2 else None
    got = run_weights(c, q, n, cl, causal, w_in).double().cpu().numpy()
    for b, L in enumerate(lens):
        nb = n if cl is None else cl[b]
        assert np.all(got[b, :, L:] == 77.0)
        for h in range(hkv):
            x = qn[b, h * gq:(h + 1) * gq, :nb]
            ref = probabilities(x, c.K[b][h], nb, causal).sum((0, 1)) if nb else np.zeros(L)
            start = 0.0 if w_in is None else w_in[b, h, :L].double().cpu().numpy()
            if L == 0:
                continue
            tol = (weights_bound(c, b, h, x, nb * gq) if nb else 0.0) * ref + 2.0 ** -24 * (start + ref) + 1e-30
            assert np.all(np.abs(got[b, h, :L] - (start + ref)) <= tol), (b, h)


def test_weights_add_up_in_place_over_steps():
    c = Cache([600], 2, 4, 3, 3, seed=21)
    q = c.queries(4, seed=5)
    w = torch.zeros((1, 2, 600), device="cuda")
    for i in range(4):   # one row at a time; not causal, so that each sees the whole cache
        run_weights(c, q[:, :, i:i + 1], 1, None, False, w, w)
    whole = run_weights(c, q, 4, None, False, None, torch.zeros_like(w))
    # 4 against 1 additions per token, the same weights
    assert torch.allclose(w, whole, rtol=8 * 2.0 ** -24, atol=0)
    # every row's weights sum to 1
    assert torch.allclose(whole.double().sum(-1), torch.full((1, 2), 16.0, dtype=torch.float64, device="cuda"),
                          rtol=1e-4)


def test_strided_weights_and_a_graph():
    c = Cache([300, 200], 2, 4, 3, 3, paged=True, seed=31)
    q = c.queries(3, seed=6)
    want = run_weights(c, q, 3, None, True)
    attn = run_chunk(c, q, 3, None, True)
    big = torch.full((2, 2, 512), 77.0, device="cuda")
    out = torch.full_like(q, 77.0)
    w1 = workspace(gtq.gtq_weights_workspace(c.plan, c.cap, 3))
    w2 = workspace(gtq.gtq_chunk_workspace(c.plan, c.cap, 3))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            gtq.gtq_attn_weights(c.plan, c.packed, c.cap, q, big[:, :, :300], w1, layout=c.layout, stream=s)
            gtq.gtq_chunk_attn(c.plan, c.packed, c.cap, q, out, w2, layout=c.layout, stream=s)
        for _ in range(3):
            g.replay()
    s.synchronize()
    assert torch.equal(big[:, :, :300], want) and bool((big[:, :, 300:] == 77.0).all())
    assert torch.equal(out, attn)


def test_two_calls_at_once_on_one_plan():
    # the plan is only read; each call has a workspace of its own
    c = Cache([4000, 2000], 1, 8, 3, 3, seed=41)
    qs = [c.queries(9, seed=50 + i) for i in range(2)]
    want = [run_chunk(c, q, 9, None, True) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    outs = [torch.empty_like(q) for q in qs]
    ws = [workspace(gtq.gtq_chunk_workspace(c.plan, c.cap, 9)) for _ in qs]
    torch.cuda.synchronize()
    for _ in range(4):
        for q, s, o, w in zip(qs, streams, outs, ws):
            gtq.gtq_chunk_attn(c.plan, c.packed, c.cap, q, o, w, layout=c.layout, stream=s)
    torch.cuda.synchronize()
    for o, x in zip(outs, want):
        assert torch.equal(o, x)


PAIRS = [
    # lens, hkv, gq, kb, vb, paged, n, chunk_lens, causal: more than 256 rows of a KV head
    ([65], 1, 4, 3, 3, True, 65, None, True),                         # the last row sees a tile and one token
    ([64, 129, 1], 2, 8, 3, 2, True, 40, [40, 17, 1], True),          # sequences of one half, of less, of one token
    ([700, 0, 333], 1, 3, 2, 2, True, 171, [171, 9, 86], True),       # 257 and 258 rows beside none
    ([450], 1, 8, 8, 8, True, 65, None, False),
    ([450, 190], 1, 8, 6, 5, False, 129, [129, 100], True),
    ([8000, 130], 1, 8, 3, 3, True, 33, None, True),                  # split, and a sequence that ends in the first part
    ([300], 1, 128, 1, 1, False, 5, None, True),
    ([50], 1, 2, 3, 3, True, 200, None, True),                        # most rows stand before the first token
    ([700, 0, 333], 1, 8, 2, 2, True, 120, [120, 3, 65], True),       # 960 rows, 24 of none, 520
    ([450], 1, 8, 8, 8, True, 60, None, False),
    ([450, 190], 2, 8, 6, 5, False, 60, [60, 33], False),
    ([300], 1, 128, 1, 1, False, 4, None, True),
    ([9000], 1, 4, 4, 4, True, 250, None, True),                      # split, several tiles of rows
]


@pytest.mark.parametrize("case", PAIRS, ids=[str(i) for i in range(len(PAIRS))])
def test_many_rows_against_fp64(case):
    lens, hkv, gq, kb, vb, paged, n, cl, causal = case
    c = Cache(lens, hkv, gq, kb, vb, paged=paged, seed=len(lens) + n)
    q = c.queries(n, seed=n)
    for b in range(c.B):
        if cl is not None:
            q[b, :, cl[b]:] = float("nan")
    out = run_chunk(c, q, n, cl, causal)
    check_chunk(c, q, out, n, cl, causal)
    # in place
    ws = workspace(gtq.gtq_chunk_workspace(c.plan, c.cap, n))
    lens_dev = None if cl is None else torch.tensor(cl, dtype=torch.int32, device="cuda")
    gtq.gtq_chunk_attn(c.plan, c.packed, c.cap, q, q, ws, layout=c.layout, chunk_lens=lens_dev, causal=causal)
    for b in range(c.B):
        nb = n if cl is None else cl[b]
        assert torch.equal(q[b, :, :nb], out[b, :, :nb])


@pytest.mark.parametrize("n", [3, 20, 40, 90])   # each form of the kernel; 9000 tokens are split, 200 are not
@pytest.mark.parametrize("length", [200, 9000])
def test_nan_queries_stay_in_their_rows(n, length):
    c = Cache([length], 1, 8, 3, 3, seed=n)
    q = c.queries(n, seed=n)
    want = run_chunk(c, q, n, None, True)
    weights = run_weights(c, q, n, None, True)
    bad = q.clone()
    bad[0, 5, n // 2, 77] = float("nan")
    got = run_chunk(c, bad, n, None, True)
    assert bool(got[0, 5, n // 2].isnan().all())
    got[0, 5, n // 2] = want[0, 5, n // 2]
    assert torch.equal(got, want)
    seen = length - n + n // 2 + 1
    w = run_weights(c, bad, n, None, True)
    assert bool(w[0, 0, :seen].isnan().all()) and bool(w[0, 0, seen:].isfinite().all())
    assert bool((w[0, 0, seen:] == weights[0, 0, seen:]).all())


def test_many_rows_in_a_graph_whose_lengths_change():
    c = Cache([500, 260], 1, 8, 3, 3, paged=True, seed=17)
    n = 40
    q = c.queries(n, seed=3)
    out = torch.empty_like(q)
    cl = torch.tensor([n, n], dtype=torch.int32, device="cuda")
    ws = workspace(gtq.gtq_chunk_workspace(c.plan, c.cap, n))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            gtq.gtq_chunk_attn(c.plan, c.packed, c.cap, q, out, ws, layout=c.layout, chunk_lens=cl, stream=s)
    K, V = c.K, c.V
    for lens, rows in (([500, 260], [40, 40]), ([77, 0], [1, 40]), ([129, 260], [33, 0])):
        c.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        cl.copy_(torch.tensor(rows, dtype=torch.int32))
        out.fill_(77.0)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            g.replay()
        s.synchronize()
        c.lens = lens
        c.K = [[k[:x] for k in row] for row, x in zip(K, lens)]
        c.V = [[v[:x] for v in row] for row, x in zip(V, lens)]
        check_chunk(c, q, out, n, rows, True)


def test_one_token_of_empty_and_absent_sequences():
    c = Cache([0, 200, 64], 2, 4, 3, 3, paged=True, seed=61)
    q = c.queries(1, seed=62)
    for cl in (None, [1, 0, 1]):
        check_chunk(c, q, run_chunk(c, q, 1, cl, True), 1, cl, True)


def same(a, b, n, c):
    """The same bits; for one token, whose decode kernel adds its parts up as its blocks end, two fp32 results differ by
    the roundings of sums in another order: of T weights times values (weights sum to 1: each rounding is at most 2^-24
    of the largest value) and of 128 in the rotation, twice; and the fp16 ones by those and half a step, twice."""
    if n > 1:
        return torch.equal(a, b)
    a, b = a.double(), b.double()
    largest = max(np.abs(v).max() for row in c.V for v in row if v.size)
    return bool(((a - b).abs() <= 2 * 2.0 ** -11 * b.abs() + 2 * (max(c.lens) + 128) * 2.0 ** -24 * largest).all())


def test_far_pages():
    # the same pages beyond 4 GiB of a pool
    c = Cache([300, 130], 2, 4, 3, 3, paged=True, seed=71)
    page = c.hkv * c.tb
    shift = (5 << 30) // page
    pool = torch.empty((shift + c.pages) * page, dtype=torch.uint8, device="cuda")
    pool[shift * page:] = c.packed
    far_table = c.table + shift     # (a layout holds addresses, not tensors)
    far = gtq.seq_layout(c.seq_lens, far_table)
    for n in (1, 7, 40, 80):    # 4 to 320 rows
        q = c.queries(n, seed=n)
        want, w_want = run_chunk(c, q, n, None, True), run_weights(c, q, n, None, True)
        near = c.packed, c.layout
        c.packed, c.layout = pool, far
        try:
            got, w_got = run_chunk(c, q, n, None, True), run_weights(c, q, n, None, True)
        finally:
            c.packed, c.layout = near
        assert same(got, want, n, c) and torch.equal(w_got, w_want)


def test_far_heads():
    # a capacity whose second head lies beyond 4 GiB
    c = Cache([300], 2, 4, 3, 3, seed=73)
    cap = (5 << 30) // c.tb * 64
    plan = gtq.gtq_alloc_bits_ex(gtq.make_config(1, c.hq, 2, 3, 3, cap), c.k, 300, c.layout)
    packed = torch.empty(plan.packed_bytes, dtype=torch.uint8, device="cuda")
    gtq.gtq_quantize_pack_ex(plan, c.k, c.v, 0, 300, packed, c.layout)
    for n in (1, 7, 80):
        q = c.queries(n, seed=n)
        want, w_want = run_chunk(c, q, n, None, True, T=300), run_weights(c, q, n, None, True)
        out, w = torch.empty_like(q), torch.full_like(w_want, 77.0)
        gtq.gtq_chunk_attn(plan, packed, 300, q, out, workspace(gtq.gtq_chunk_workspace(plan, 300, n)), layout=c.layout)
        gtq.gtq_attn_weights(plan, packed, 300, q, w, workspace(gtq.gtq_weights_workspace(plan, 300, n)), layout=c.layout)
        torch.cuda.synchronize()
        assert gtq.gtq_status(plan) == gtq.GTQ_OK
        assert same(out, want, n, c) and torch.equal(w[:, :, :300], w_want[:, :, :300])
