"""Operators around the packed cache, in plain torch operations and as library calls, for timing and comparison.

    rope      rotary positions of queries and keys, before they are coded or attended
    chunk     attention of a chunk of new tokens (or one) over the packed cache
    weights   attention weights that a chunk gives every cached token, added up
    evict     the cached tokens with the largest weights, moved into a smaller cache

With ``own`` false, ``run`` computes an operator in elementary torch operations; with ``own`` true it makes the
library's calls.  ``prepare`` writes the packed caches itself, from the layout that include/gtq.h describes.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
TILE = 64
TAG_KEY, TAG_VALUE = 0x4B, 0x56


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decode step's queries and keys of 16 sequences: a launch and little else
        dict(name="rope_decode", op="rope", B=16, hq=28, hkv=4, T=1, d=128, rot=128, dtype="fp16", half=True,
             theta=1e4, scaling="none", factor=1.0, context=16384, backward=False),
        # a 32K prompt's queries and keys, frequencies scaled for a longer context than the training one
        dict(name="rope_prompt", op="rope", B=1, hq=32, hkv=8, T=32768, d=128, rot=128, dtype="fp16", half=True,
             theta=5e5, scaling="llama3", factor=8.0, context=8192, backward=False),
        # the gradient's way through, fp32, half of the head rotated, neighbours paired, an odd number of tokens
        dict(name="rope_gradient", op="rope", B=2, hq=16, hkv=2, T=4099, d=128, rot=64, dtype="fp32", half=False,
             theta=1e6, scaling="yarn", factor=4.0, context=32768, backward=True),
        # a small ragged batch over pages, one sequence with no new token, wide codes
        dict(name="chunk_ragged", op="chunk", B=3, hq=8, hkv=2, T=1000, n=37, kb=4, vb=4, half=False, paged=True,
             ragged=True, causal=True),
        # a decode step of 16 sequences of their own lengths over pages: one new token each
        dict(name="chunk_token", op="chunk", B=16, hq=28, hkv=4, T=16384, n=1, kb=3, vb=2, half=True, paged=True,
             ragged=True, causal=True),
        # five drafted tokens verified against a 128K context
        dict(name="chunk_draft", op="chunk", B=1, hq=16, hkv=2, T=131072, n=5, kb=3, vb=3, half=True, paged=False,
             ragged=False, causal=True),
        # a user's next turn of 1000 tokens over a 32K conversation
        dict(name="chunk_turn", op="chunk", B=1, hq=32, hkv=8, T=32768, n=1000, kb=2, vb=2, half=True, paged=True,
             ragged=False, causal=True),
        # one piece of a long prompt that is taken in piece by piece
        dict(name="chunk_prompt", op="chunk", B=1, hq=16, hkv=2, T=131072, n=1024, kb=3, vb=3, half=True, paged=False,
             ragged=False, causal=True),
        # a decode step's weights, added to what the earlier steps gave
        dict(name="weights_token", op="weights", B=1, hq=16, hkv=2, T=131072, n=1, kb=3, vb=3, half=True, paged=False,
             ragged=False, causal=True, add=True),
        # the last 32 tokens of a prompt look back over all of it
        dict(name="weights_window", op="weights", B=1, hq=32, hkv=8, T=32768, n=32, kb=2, vb=2, half=True, paged=True,
             ragged=False, causal=True, add=False),
        # a serving batch over its page budget: every sequence down to 4096 tokens
        dict(name="evict_pages", op="evict", B=16, hq=28, hkv=4, T=16384, kb=3, vb=2, half=True, paged=True,
             ragged=True, keep=4096, first=4, recent=256),
        # a 128K prompt cut to an eighth before decoding starts
        dict(name="evict_prompt", op="evict", B=1, hq=16, hkv=2, T=131072, kb=3, vb=3, half=True, paged=False,
             ragged=False, keep=16384, first=4, recent=1024),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "chunk", "chunk", "weights", "evict"])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 7, 8])
    half = rng.random() < 0.7
    if op == "rope":
        B, T = _log_int(rng, 1, 16), _log_int(rng, 1, 32768)
        T = max(1, min(T, 1000000 // (B * (hq + hkv))))
        d = rng.choice([64, 128, 128, 128])
        return dict(op=op, B=B, hq=hq, hkv=hkv, T=T, d=d, rot=rng.choice([d, d, d // 2]), dtype=rng.choice(["fp16", "fp32"]),
                    half=half, theta=rng.choice([1e4, 5e5, 1e6]), scaling=rng.choice(["none", "linear", "llama3", "yarn"]),
                    factor=rng.choice([2.0, 4.0, 8.0]), context=rng.choice([8192, 16384, 32768]), backward=rng.random() < 0.4)
    B = _log_int(rng, 1, 16)
    T = max(64, min(_log_int(rng, 64, 131072), 1048576 // (B * hkv)))
    kb, vb = rng.choice([2, 3, 3, 4]), rng.choice([2, 2, 3, 4])
    case = dict(op=op, B=B, hq=hq, hkv=hkv, T=T, kb=kb, vb=vb, half=half, paged=rng.random() < 0.5, ragged=B > 1)
    if op == "evict":
        recent = _log_int(rng, 1, min(256, T // 4))
        keep = max(recent + 4, _log_int(rng, max(1, T // 16), T))
        return dict(case, keep=keep, first=rng.choice([0, 4]), recent=recent)
    most = 1024 if op == "chunk" else 64
    n = _log_int(rng, 1, most)
    n = max(1, min(n, T, (1 << 31) // (B * hq * T)))
    case = dict(case, n=n, causal=rng.random() < 0.8)
    return case if op == "chunk" else dict(case, add=rng.random() < 0.5)


# ---------------------------------------------------------------- the quantizer's tables (host, 64 bits)

def _lloyd_max(b):
    """Centroids and thresholds of the 2**b level quantizer of N(0, 1) with the least mean squared error: Newton on
    c_k = mean of the cell between the midpoints of the neighbouring centroids."""
    n = 1 << b
    erfc = np.vectorize(math.erfc)
    phi = lambda x: np.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)  # noqa: E731

    def cells(c):
        t = 0.5 * (c[1:] + c[:-1])
        tail = 0.5 * erfc(np.abs(t) / math.sqrt(2))  # the mass beyond |t|
        lo, hi = np.concatenate([[-np.inf], t]), np.concatenate([t, [np.inf]])
        tl, th = np.concatenate([[0.0], tail]), np.concatenate([tail, [0.0]])
        # the mass of a cell, without cancellation: by the upper tails on the right, the lower ones on the left
        p = np.where(lo >= 0, tl - th, np.where(hi <= 0, th - tl, 1 - tl - th))
        f = phi(t)
        return t, f, p

    # start where a quantizer of many levels has its centroids: equal masses of the density's cube root, N(0, 3)
    x, u = np.linspace(-8, 8, 20001), (np.arange(n) + 0.5) / n
    c = math.sqrt(3.0) * np.interp(u, 0.5 * erfc(-x / math.sqrt(2)), x)
    for step in range(300):
        t, f, p = cells(c)
        fl, fh = np.concatenate([[0.0], f]), np.concatenate([f, [0.0]])
        m = (fl - fh) / p
        if step < 200 and b <= 3 or step < 20:
            c = m
            continue
        tl, th = np.concatenate([[0.0], t]), np.concatenate([t, [0.0]])
        dl = fl * (m - tl) / p  # dm/dlo
        dh = fh * (th - m) / p  # dm/dhi
        J = np.eye(n) - np.diag(0.5 * (dl + dh))
        J[np.arange(1, n), np.arange(n - 1)] -= 0.5 * dl[1:]
        J[np.arange(n - 1), np.arange(1, n)] -= 0.5 * dh[:-1]
        new = c - np.linalg.solve(J, c - m)
        done = np.max(np.abs(new - c)) < 1e-14
        c = new if np.all(np.diff(new) > 0) else m
        if done:
            break
    c = 0.5 * (c - c[::-1])
    t, f, p = cells(c)
    return c, t, 1.0 - float(np.sum(p * c * c))


def _rotation(m, tag, seed=0):
    """The seeded m x m orthogonal matrix of tag: Q of a Gaussian's QR, diag(R) > 0."""
    with np.errstate(over="ignore"):
        k = np.arange(1, 2 * m * m + 1, dtype=np.uint64)
        z = np.uint64((seed ^ (tag << 48) ^ (m << 32)) & 0xFFFFFFFFFFFFFFFF) + k * np.uint64(0x9E3779B97F4A7C15)
        z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
        z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
        z = (z ^ (z >> np.uint64(31))) >> np.uint64(11)
    u1, u2 = (z[0::2].astype(np.float64) + 0.5) * 2.0 ** -53, z[1::2].astype(np.float64) * 2.0 ** -53
    q, r = np.linalg.qr((np.sqrt(-2 * np.log(u1)) * np.cos(2 * np.pi * u2)).reshape(m, m))
    return q * np.where(np.diag(r) < 0, -1.0, 1.0)[None, :]


_made = {}


def _constants():
    if not _made:
        lm = [(np.zeros(1), np.zeros(0), 1.0)] + [_lloyd_max(b) for b in range(1, 9)]
        _made["centroids"] = [x[0] for x in lm]
        _made["thresholds"] = [x[1].astype(np.float32) for x in lm]
        _made["distortion"] = [x[2] for x in lm]
        _made["rv"] = _rotation(128, TAG_VALUE)
        _made["rk"] = {}
    return _made


def _key_rotation(m):
    rk = _constants()["rk"]
    if m not in rk:
        rk[m] = _rotation(m, TAG_KEY)
    return rk[m]


def _widths(energy, kb):
    """Bits of every RoPE block of one head: one at a time to the block that gains the most."""
    dist = _constants()["distortion"]
    b = np.zeros(64, np.int64)
    gain = energy * (dist[0] - dist[1])
    for _ in range(64 * kb):
        i = int(np.argmax(gain))
        b[i] += 1
        gain[i] = energy[i] * (dist[b[i]] - dist[b[i] + 1]) if b[i] < 8 else -1.0
    return b


def _tile_bytes(kb, vb):
    return 1024 * (kb + vb) + 128 + 1024


def _tables(energy, case):
    """What the layout and the rotations of a plan with these energies are, head by head."""
    kb, vb = case["kb"], case["vb"]
    H = energy.shape[0]
    j = np.arange(64)
    t = dict(bits=np.zeros((H, 64), np.int64), width=np.zeros((H, 128), np.int64), group=np.zeros((H, 128), np.int64),
             scale=np.zeros((H, 128)), start=np.zeros((H, 64, 128), np.int64), M=np.zeros((H, 128, 128)), groups=[])
    for h in range(H):
        b = _widths(energy[h].copy(), kb)
        t["bits"][h] = b
        pos, off, groups = 0, 0, []
        for w in range(8, 0, -1):
            blocks = np.flatnonzero(b == w)
            if not len(blocks):
                continue
            m = 2 * len(blocks)
            dims = np.stack([blocks, blocks + 64] if case["half"] else [2 * blocks, 2 * blocks + 1], 1).ravel()
            r = np.arange(m)
            t["width"][h, pos:pos + m], t["group"][h, pos:pos + m], t["scale"][h, pos:pos + m] = w, len(groups), m ** -0.5
            t["M"][h, pos:pos + m, dims] = _key_rotation(m).T
            t["start"][h, :, pos:pos + m] = (8 * off + (r // 2) * 128 * w + (r % 2) * w)[None, :] + (
                (j & 7) * 16 * w + 2 * (j >> 3) * w)[:, None]
            groups.append((w, pos, m, dims))
            pos, off = pos + m, off + 16 * w * (m // 2)
        t["groups"].append(groups)
    d = np.arange(128)
    p = (d >> 4) * 32 + (d & 7) * 4
    t["vstart"] = 8192 * kb + (p[None, :] + ((j & 7) >> 1)[:, None]) * 32 * vb + vb * (
        8 * (j >> 4)[:, None] + 4 * ((j >> 3) & 1)[:, None] + 2 * ((d >> 3) & 1)[None, :] + (j & 1)[:, None])
    norm = 16 * ((j & 7) * 8 + (j >> 3))  # bit of token j's norm in a row of 64 norms
    t["vnorm"] = 8192 * (kb + vb) + norm
    t["knorm"] = 8192 * (kb + vb) + 1024 + 1024 * np.arange(8)[:, None] + norm[None, :]
    return t


# ---------------------------------------------------------------- what a program has in hand

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _scales(seed, H):
    """Standard deviation of the RoPE blocks of H heads: a decay of their own each, and two blocks that stand out."""
    rng = np.random.RandomState(seed % (2 ** 31))
    s = np.exp(-rng.uniform(1, 5, (H, 1)) * np.arange(64)[None, :] / 64)
    for h in range(H):
        s[h, rng.choice(64, 2, replace=False)] *= 8
    return s


def _dims(s, half):
    """Per-dim values of per-block ones."""
    return np.concatenate([s, s], -1) if half else np.repeat(s, 2, -1)


def _i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32, device=DEV)


def _write_bits(bits, start, code, width):
    """bits[tile][bit]: puts code[tile][...] (width[...] bits each) at start[...]."""
    for k in range(8):
        on = width > k
        if bool(on.any()):
            bits[:, (start + k)[on]] = ((code[:, on] >> k) & 1).to(torch.uint8)


def _cache(case, seed):
    """A packed cache of random keys and values (post-RoPE), its tables, and the plan where the library's calls need it."""
    B, hkv, T, kb, vb = case["B"], case["hkv"], case["T"], case["kb"], case["vb"]
    H, nt, tb = B * hkv, (T + 63) // 64, _tile_bytes(case["kb"], case["vb"])
    rng = np.random.RandomState((seed * 7 + 3) % (2 ** 31))
    gen = _generator(seed)
    c = _constants()
    s = _scales(seed, H)
    tab = _tables(2.0 * s * s, case)
    std = torch.tensor(_dims(s, case["half"]), dtype=torch.float32, device=DEV)
    thr = [torch.tensor(t, device=DEV) for t in c["thresholds"]]
    vstart = torch.tensor(tab["vstart"], device=DEV)
    rv = torch.tensor(c["rv"], dtype=torch.float32, device=DEV)
    tiles = torch.zeros((H, nt, tb), dtype=torch.uint8, device=DEV)
    eight = torch.tensor([1 << i for i in range(8)], dtype=torch.uint8, device=DEV)

    def put_norm(bits, at, n):
        v = n.to(torch.float16).view(torch.int16).to(torch.int32) & 0xFFFF
        for k in range(16):
            bits[:, at + k] = ((v >> k) & 1).to(torch.uint8)

    for h in range(H):
        x = torch.randn((nt * 64, 128), generator=gen, device=DEV) * std[h]
        code = torch.zeros((nt * 64, 128), dtype=torch.int64, device=DEV)
        bits = torch.zeros((nt, tb * 8), dtype=torch.uint8, device=DEV)
        for gi, (w, pos, m, dims) in enumerate(tab["groups"][h]):
            y = x[:, torch.tensor(dims, device=DEV)]
            n = y.norm(dim=1)
            y = (y * (math.sqrt(m) / n)[:, None]) @ torch.tensor(_key_rotation(m).T, dtype=torch.float32, device=DEV)
            code[:, pos:pos + m] = torch.bucketize(y, thr[w])
            put_norm(bits, torch.tensor(tab["knorm"][gi], device=DEV), n.view(nt, 64))
        _write_bits(bits, torch.tensor(tab["start"][h], device=DEV), code.view(nt, 64, 128),
                    torch.tensor(tab["width"][h], device=DEV).expand(64, 128))
        v = torch.randn((nt * 64, 128), generator=gen, device=DEV)
        n = v.norm(dim=1)
        y = (v * (math.sqrt(128) / n)[:, None]) @ rv.T
        _write_bits(bits, vstart, torch.bucketize(y, thr[vb]).view(nt, 64, 128), torch.full((64, 128), vb, device=DEV))
        put_norm(bits, torch.tensor(tab["vnorm"], device=DEV), n.view(nt, 64))
        tiles[h] = (bits.view(nt, tb, 8) * eight).sum(-1, dtype=torch.uint8)
        del bits
    lens = rng.randint(max(1, T // 4), T + 1, B) if case["ragged"] else np.full(B, T)
    st = dict(case=case, tab=tab, T=T, lens=_i32(lens), table=None, tile_bytes=tb, std=std)
    if case["paged"]:  # pages in a random order, three of them nobody's
        pages = rng.permutation(B * nt + 3)[:B * nt].reshape(B, nt)
        pool = torch.zeros((B * nt + 3, hkv, tb), dtype=torch.uint8, device=DEV)
        pool[torch.tensor(pages, device=DEV)] = tiles.view(B, hkv, nt, tb).transpose(1, 2)
        st["packed"], st["table"] = pool.view(-1), _i32(pages)
    else:
        st["packed"] = tiles.view(-1)
    # the tables on the device, for the plain form
    st["start"] = torch.tensor(tab["start"], dtype=torch.int64, device=DEV)
    st["width"] = torch.tensor(tab["width"], dtype=torch.int64, device=DEV)
    st["group"] = torch.tensor(tab["group"], dtype=torch.int64, device=DEV)
    st["scale"] = torch.tensor(tab["scale"], dtype=torch.float32, device=DEV)
    st["M"] = torch.tensor(tab["M"], dtype=torch.float32, device=DEV)
    st["rv"] = rv
    st["vstart"] = vstart
    st["knorm"] = torch.tensor(tab["knorm"], device=DEV)
    st["vnorm"] = torch.tensor(tab["vnorm"], device=DEV)
    st["centroids"] = torch.tensor(np.concatenate([[0.0]] + c["centroids"][1:]), dtype=torch.float32, device=DEV)
    if own:  # the handle that a serving program keeps for each layer; only the library can make it
        import decode_attention_13_b200 as gtq

        cfg = gtq.make_config(B, case["hq"], hkv, kb, vb, T,
                              rope_pairing=gtq.PAIRING_HALF if case["half"] else gtq.PAIRING_INTERLEAVED)
        st["plan"] = gtq.gtq_alloc_bits_from_energy(cfg, (2.0 * s * s).reshape(B, hkv, 64))
        st["layout"] = gtq.seq_layout(st["lens"], st["table"])
    return st, gen, rng


def _prepare_rope(case, seed):
    gen = _generator(seed)
    B, T, d = case["B"], case["T"], case["d"]
    dt = torch.float16 if case["dtype"] == "fp16" else torch.float32
    rng = np.random.RandomState((seed * 7 + 5) % (2 ** 31))
    st = dict(case=case)
    for name, h in (("q", case["hq"]), ("k", case["hkv"])):  # as a projection leaves them: [B][T][heads][d]
        st[name] = torch.randn((B, T, h, d), generator=gen, device=DEV).to(dt).transpose(1, 2)
        st[name + "_out"] = torch.empty((B, T, h, d), dtype=dt, device=DEV).transpose(1, 2)
    start = rng.randint(0, case["context"], B)
    st["pos"] = torch.tensor(start[:, None] + np.arange(T)[None, :], dtype=torch.int64, device=DEV)
    if own:
        import decode_attention_13_b200 as gtq

        kind = dict(none=gtq.ROPE_PLAIN, linear=gtq.ROPE_LINEAR, llama3=gtq.ROPE_LLAMA3, yarn=gtq.ROPE_YARN)[case["scaling"]]
        low, high = (1.0, 4.0) if case["scaling"] == "llama3" else (1.0, 32.0)
        st["rope"] = gtq.make_rope(d, case["theta"], rotary_dim=case["rot"],
                                   rope_pairing=gtq.PAIRING_HALF if case["half"] else gtq.PAIRING_INTERLEAVED,
                                   dtype=gtq.DTYPE_FP16 if case["dtype"] == "fp16" else gtq.DTYPE_FP32, scaling=kind,
                                   factor=case["factor"], original_context=case["context"], low_freq=low, high_freq=high,
                                   magnitude=_magnitude(case), backward=case["backward"])
    return st


def _magnitude(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "yarn" else 1.0


def prepare(case, seed):
    if case["op"] == "rope":
        return _prepare_rope(case, seed)
    st, gen, rng = _cache(case, seed)
    B, hq, hkv, T = case["B"], case["hq"], case["hkv"], case["T"]
    if case["op"] == "evict":
        # weights as many steps leave them: a few tokens hold most, many hold nothing at all
        w = torch.exp(4 * torch.randn((B, hkv, T), generator=gen, device=DEV) - 8)
        st["w"] = torch.where(w < 1e-4, torch.zeros_like(w), w)
        keep = case["keep"]
        nk = (keep + 63) // 64
        st["w_out"] = torch.zeros((B, hkv, keep), device=DEV)
        st["kept"] = torch.zeros((B, hkv, keep), dtype=torch.int32, device=DEV)
        st["new_lens"] = torch.zeros((B,), dtype=torch.int32, device=DEV)
        st["dst_table"] = None
        st["dst"] = torch.zeros_like(st["packed"])
        if case["paged"]:
            pages = rng.permutation(B * nk + 2)[:B * nk].reshape(B, nk)
            st["dst_table"] = _i32(pages)
            st["dst"] = torch.zeros(((B * nk + 2) * hkv * st["tile_bytes"],), dtype=torch.uint8, device=DEV)
        if own:
            import decode_attention_13_b200 as gtq

            st["dst_layout"] = gtq.seq_layout(None, st["dst_table"]) if case["paged"] else None
            st["workspace"] = torch.empty((gtq.gtq_evict_workspace(st["plan"], T),), dtype=torch.uint8, device=DEV)
        return st
    n = case["n"]
    q = torch.randn((B, n, hq, 128), generator=gen, device=DEV) * st["std"].view(B, 1, hkv, 1, 128).expand(
        B, n, hkv, hq // hkv, 128).reshape(B, n, hq, 128)
    st["q"] = q.to(torch.float16).transpose(1, 2)  # [B][heads][n][128], as a projection leaves it
    # new tokens of every sequence; in a ragged batch of several rows some bring fewer, or none
    cl = np.full(B, n)
    if case["ragged"] and n > 1:
        cl = rng.randint(0, n + 1, B)
        cl[rng.randint(B)] = n
    st["chunk_lens"] = _i32(cl)
    if case["op"] == "chunk":
        st["out"] = torch.zeros((B, n, hq, 128), dtype=torch.float16, device=DEV).transpose(1, 2)
    else:
        st["w_in"] = torch.rand((B, hkv, T), generator=gen, device=DEV) if case["add"] else None
        st["w_out"] = torch.zeros((B, hkv, T), device=DEV)
    if own:
        import decode_attention_13_b200 as gtq

        size = gtq.gtq_chunk_workspace if case["op"] == "chunk" else gtq.gtq_weights_workspace
        st["workspace"] = torch.empty((size(st["plan"], T, n),), dtype=torch.uint8, device=DEV)
    return st


# ---------------------------------------------------------------- one pass

def run(state):
    return dict(rope=_rope, chunk=_chunk, weights=_weights, evict=_evict)[state["case"]["op"]](state)


def _frequencies(case):
    """Angle per position of every rotated pair, in 64 bits."""
    r, f = case["rot"], case["factor"]
    i = torch.arange(r // 2, dtype=torch.float64, device=DEV)
    w = case["theta"] ** (-2.0 * i / r)
    if case["scaling"] == "linear":
        w = w / f
    elif case["scaling"] == "llama3":  # short waves stay, long ones are stretched, a ramp between
        turns = case["context"] * w / (2 * math.pi)
        s = ((turns - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        w = (1 - s) * w / f + s * w
    elif case["scaling"] == "yarn":  # the ramp runs over the pairs' indices
        at = lambda turns: r * math.log(case["context"] / (turns * 2 * math.pi)) / (2 * math.log(case["theta"]))  # noqa: E731
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), r - 1)
        s = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        w = s * w / f + (1 - s) * w
    return w


def _rope(st):
    case = st["case"]
    if own:
        import decode_attention_13_b200 as gtq

        gtq.gtq_rope(st["rope"], st["q"], st["q_out"], st["k"], st["k_out"], positions=st["pos"])
        return {"q": st["q_out"], "k": st["k_out"]}
    r = case["rot"]
    a = st["pos"].to(torch.float64)[:, None, :, None] * _frequencies(case)
    cos = (torch.cos(a) * _magnitude(case)).to(torch.float32)
    sin = (torch.sin(a) * _magnitude(case)).to(torch.float32)
    if case["backward"]:
        sin = -sin
    got = {}
    for name in ("q", "k"):
        x = st[name].to(torch.float32)
        x0, x1 = (x[..., :r // 2], x[..., r // 2:r]) if case["half"] else (x[..., 0:r:2], x[..., 1:r:2])
        y0, y1 = x0 * cos - x1 * sin, x1 * cos + x0 * sin
        y = torch.cat([y0, y1], -1) if case["half"] else torch.stack([y0, y1], -1).flatten(-2)
        got[name] = torch.cat([y, x[..., r:]], -1).to(st[name].dtype)
    return got


def _tiles(st, packed, table):
    """[heads][tiles][bytes] of a cache, from its pages where it has some."""
    case = st["case"]
    B, hkv, tb = case["B"], case["hkv"], st["tile_bytes"]
    if table is None:
        return packed.view(B * hkv, -1, tb)
    return packed.view(-1, hkv, tb)[table.long()].transpose(1, 2).reshape(B * hkv, -1, tb)


def _codes(tiles, start, width):
    """Codes at bit start[...] (below 8 bits wide) of every tile: two bytes each."""
    H, nt, tb = tiles.shape
    at = (start >> 3).reshape(start.shape[0], 1, -1).expand(H, nt, -1)
    two = torch.gather(tiles, 2, at).to(torch.int32) | (torch.gather(tiles, 2, (at + 1).clamp(max=tb - 1)).to(torch.int32) << 8)
    two = two >> (start & 7).reshape(start.shape[0], 1, -1).to(torch.int32)
    mask = ((1 << width) - 1).to(torch.int32)
    return two.view(H, nt * 64, 128) & mask.reshape(mask.shape[0], 1, -1)


def _keys(st, tiles):
    """Keys in their groups' rotated bases: [heads][tokens][128]."""
    H, nt, _ = tiles.shape
    code = _codes(tiles, st["start"], st["width"])
    base = torch.where(st["width"] > 0, (1 << st["width"]) - 1, 0)  # first centroid of the width
    k = st["centroids"][(code + base[:, None, :]).long()]
    halves = tiles.view(torch.float16)
    norm = halves[:, :, (st["knorm"] >> 4).flatten()].view(H, nt, 8, 64).permute(0, 1, 3, 2).reshape(H, nt * 64, 8)
    norm = torch.gather(norm.to(torch.float32), 2, st["group"][:, None, :].expand(H, nt * 64, 128))
    # a position of no width has the centroid 0; the norms of groups that are not there are anything
    return torch.where(st["scale"][:, None, :] > 0, k * norm * st["scale"][:, None, :], 0.0)


def _values(st, tiles):
    H, nt, _ = tiles.shape
    vb = st["case"]["vb"]
    code = _codes(tiles, st["vstart"][None], torch.full((1, 128), vb, device=DEV))
    norm = tiles.view(torch.float16)[:, :, st["vnorm"] >> 4].reshape(H, nt * 64, 1).to(torch.float32)
    return st["centroids"][(code + ((1 << vb) - 1)).long()] * norm * 128 ** -0.5


def _probabilities(st, tiles):
    """Softmax over the tokens of every row of the chunk: [heads][group rows x n][tokens]; rows with nothing to see are 0."""
    case = st["case"]
    B, hq, hkv, n = case["B"], case["hq"], case["hkv"], case["n"]
    k = _keys(st, tiles)
    q = st["q"].to(torch.float32).reshape(B * hkv, -1, 128) @ st["M"].transpose(1, 2)
    s = (q @ k.transpose(1, 2)) * 128 ** -0.5
    s = s.view(B, hkv, hq // hkv, n, -1)
    t = torch.arange(s.shape[-1], device=DEV)
    i = torch.arange(n, device=DEV)
    lens, cl = st["lens"].long(), st["chunk_lens"].long()
    end = lens[:, None] - cl[:, None] + i[None, :] + 1 if case["causal"] else lens[:, None].expand(B, n)
    seen = (t < torch.minimum(end, lens[:, None])[..., None]) & (i < cl[:, None])[..., None]
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(s - top)
    return (p / p.sum(-1, keepdim=True).clamp(min=1e-30)).view(B * hkv, -1, p.shape[-1])


def _chunk(st):
    case = st["case"]
    B, hq, hkv, n = case["B"], case["hq"], case["hkv"], case["n"]
    if own:
        import decode_attention_13_b200 as gtq

        gtq.gtq_chunk_attn(st["plan"], st["packed"], st["T"], st["q"], st["out"], st["workspace"], layout=st["layout"],
                           chunk_lens=st["chunk_lens"], causal=case["causal"])
        return st["out"]
    tiles = _tiles(st, st["packed"], st["table"])
    o = (_probabilities(st, tiles) @ _values(st, tiles)) @ st["rv"]
    brings = torch.arange(n, device=DEV) < st["chunk_lens"].long()[:, None]
    return torch.where(brings[:, None, :, None], o.view(B, hq, n, 128).to(torch.float16), st["out"])


def _weights(st):
    case = st["case"]
    B, hkv, T = case["B"], case["hkv"], case["T"]
    if own:
        import decode_attention_13_b200 as gtq

        gtq.gtq_attn_weights(st["plan"], st["packed"], st["T"], st["q"], st["w_out"], st["workspace"], weights_in=st["w_in"],
                             layout=st["layout"], chunk_lens=st["chunk_lens"], causal=case["causal"])
        return st["w_out"]
    p = _probabilities(st, _tiles(st, st["packed"], st["table"])).sum(1).view(B, hkv, -1)[..., :T]
    held = torch.arange(T, device=DEV) < st["lens"].long()[:, None]
    return torch.where(held[:, None], p if st["w_in"] is None else st["w_in"] + p, st["w_out"])


def _token_bits(st):
    """Bit of a tile that holds bit i of token j, [heads][64][bits of a token]: every bit but the spare norms is there."""
    case, tab = st["case"], st["tab"]
    kb, vb, H = case["kb"], case["vb"], tab["bits"].shape[0]
    key = torch.cat([torch.cat([st["start"][h][:, st["width"][h] > k] + k for k in range(8)], 1)[None] for h in range(H)])
    val = torch.cat([st["vstart"] + k for k in range(vb)], 1)
    vn = st["vnorm"][:, None] + torch.arange(16, device=DEV)
    kn = (st["knorm"].T[:, :, None] + torch.arange(16, device=DEV)).flatten(1)
    return torch.cat([key, torch.cat([val, vn, kn], 1)[None].expand(H, -1, -1)], 2)


def _evict(st):
    case = st["case"]
    B, hkv, T, keep = case["B"], case["hkv"], case["T"], case["keep"]
    if own:
        import decode_attention_13_b200 as gtq

        gtq.gtq_evict(st["plan"], st["packed"], T, st["w"], keep, st["dst"], st["new_lens"], st["workspace"],
                      n_first=case["first"], n_recent=case["recent"], layout=st["layout"], dst_layout=st["dst_layout"],
                      weights_out=st["w_out"], kept=st["kept"])
        return {"dst": st["dst"], "lens": st["new_lens"], "kept": st["kept"], "weights": st["w_out"]}
    H, tb, nk = B * hkv, st["tile_bytes"], (keep + 63) // 64
    lens = st["lens"].long()
    t = torch.arange(T, device=DEV)
    # the order of preference: tokens that stay by their place, then the others by weight, then those that are not there
    rank = torch.where(t < lens[:, None], 1, 0)
    rank = torch.where((rank == 1) & ((t < case["first"]) | (t >= lens[:, None] - case["recent"])), 2, rank)
    by_weight = torch.argsort(st["w"], dim=-1, descending=True, stable=True)
    by_rank = torch.argsort(torch.gather(rank[:, None].expand(B, hkv, T), 2, by_weight), dim=-1, descending=True, stable=True)
    new = lens.clamp(max=keep)
    best = torch.gather(by_weight, 2, by_rank)[..., :keep]
    if best.shape[-1] < keep:
        best = torch.cat([best, best.new_zeros((B, hkv, keep - best.shape[-1]))], -1)
    there = torch.arange(keep, device=DEV) < new[:, None, None]
    kept = torch.where(there, best, T).sort(-1).values
    source = torch.where(there, kept, 0)
    # the packed cache, token by token in bits, then the kept ones laid out again
    tiles = _tiles(st, st["packed"], st["table"])
    where = _token_bits(st)
    nb = where.shape[2]
    eight = torch.arange(8, dtype=torch.uint8, device=DEV)
    bits = ((tiles[..., None] >> eight) & 1).view(H, tiles.shape[1], tb * 8)
    bits = torch.gather(bits, 2, where.view(H, 1, -1).expand(H, tiles.shape[1], -1)).view(H, -1, nb)
    pad = nk * 64 - keep
    some = torch.nn.functional.pad(source, (0, pad)).view(H, nk * 64)
    is_there = torch.nn.functional.pad(there.expand(B, hkv, keep), (0, pad)).reshape(H, nk * 64)
    bits = torch.gather(bits, 1, some[..., None].expand(H, nk * 64, nb)) * is_there[..., None]
    # norms of groups that a head does not have are 0 in the new cache
    n_groups = st["group"].amax(1) + 1
    spare = torch.arange(8, device=DEV) >= n_groups[:, None]
    bits[:, :, nb - 128:] *= ~spare.repeat_interleave(16, 1)[:, None]
    laid = torch.zeros((H, nk, tb * 8), dtype=torch.uint8, device=DEV)
    laid.scatter_(2, where.view(H, 1, -1).expand(H, nk, -1), bits.view(H, nk, 64 * nb))
    laid = (laid.view(H, nk, tb, 8) << eight).sum(-1, dtype=torch.uint8).view(B, hkv, nk, tb)
    used = torch.arange(nk, device=DEV) * 64 < new[:, None]
    dst = st["dst"].clone()
    if st["dst_table"] is None:
        d = dst.view(B, hkv, -1, tb)
        d[:, :, :nk] = torch.where(used[:, None, :, None], laid, d[:, :, :nk])
    else:
        d = dst.view(-1, hkv, tb)
        at = st["dst_table"].long()
        d[at] = torch.where(used[:, :, None, None], laid.transpose(1, 2), d[at])
    weights = torch.where(there, torch.gather(st["w"], 2, source), st["w_out"])
    return {"dst": dst, "lens": new.to(torch.int32), "kept": torch.where(there, kept, -1).to(torch.int32), "weights": weights}


# ---------------------------------------------------------------- what a pass cannot do without

def _held(case):
    return case["T"] * (0.625 if case["ragged"] else 1.0)  # tokens of a sequence: lengths are even in [T/4, T]


def work(case):
    B, hq, hkv, T = case["B"], case["hq"], case["hkv"], case["T"]
    if case["op"] == "rope":
        values = B * T * (hq + hkv) * case["d"]
        return {"bytes": 2.0 * values * (2 if case["dtype"] == "fp16" else 4) + 8 * B * T,
                "flops": 3.0 * B * T * (hq + hkv) * case["rot"]}
    held = _held(case)
    # per token and head: codes and the norms, 7 key groups among the heads' usual 6 to 8
    key, value = 16.0 * case["kb"] + 14, 16.0 * case["vb"] + 2
    if case["op"] == "evict":
        kept = min(case["keep"], held)
        return {"bytes": B * hkv * (4 * held + kept * (2 * (key + value) + 8)), "flops": B * hkv * held}
    rows = B * hq * case["n"] * (0.5 if case["ragged"] and case["n"] > 1 else 1.0)
    turn = 2.0 * 128 * 128  # a row into a rotated basis, or out of one
    if case["op"] == "chunk":
        return {"bytes": B * hkv * held * (key + value) + rows * 512, "flops": rows * (4.0 * 128 * held + 2 * turn)}
    return {"bytes": B * hkv * held * (key + (8 if case["add"] else 4)) + rows * 256,
            "flops": rows * (2.0 * 128 * held + turn)}


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_rope(st):
    case = st["case"]
    r, f, L = case["rot"], case["factor"], case["context"]
    freq = []
    for i in range(r // 2):
        w = case["theta"] ** (-2.0 * i / r)
        if case["scaling"] == "linear":
            w /= f
        elif case["scaling"] == "llama3":
            wave = 2 * math.pi / w
            if wave > L / 1.0:
                w /= f
            elif wave >= L / 4.0:
                s = (L / wave - 1.0) / 3.0
                w = (1 - s) * w / f + s * w
        elif case["scaling"] == "yarn":
            a, b = (r * math.log(L / (x * 2 * math.pi)) / (2 * math.log(case["theta"])) for x in (32.0, 1.0))
            a, b = max(math.floor(a), 0), min(math.ceil(b), r - 1)
            s = min(1.0, max(0.0, (i - a) / max(b - a, 0.001)))
            w = w / f * s + w * (1 - s)
        freq.append(w)
    turn = torch.polar(torch.full((), _magnitude(case), dtype=torch.float64, device=DEV),
                       st["pos"].double()[..., None] * torch.tensor(freq, dtype=torch.float64, device=DEV))
    if case["backward"]:
        turn = turn.conj()
    got = {}
    for name in ("q", "k"):
        x = st[name].double()
        y = x.clone()
        a = torch.arange(r // 2, device=DEV)
        a, b = (a, a + r // 2) if case["half"] else (2 * a, 2 * a + 1)
        z = torch.complex(x[..., a], x[..., b]) * turn[:, None]
        y[..., a], y[..., b] = z.real, z.imag
        got[name] = y
    return got


def _exact_head(st, h):
    """Keys [tokens][128] in the original basis and values, of one head, from the bytes of its tiles."""
    case, tab, c = st["case"], st["tab"], _constants()
    kb, vb, hkv, tb = case["kb"], case["vb"], case["hkv"], st["tile_bytes"]
    b, hh = divmod(h, hkv)
    nt = (case["T"] + 63) // 64
    packed = st["packed"].view(-1, tb)
    rows = torch.arange(nt, device=DEV) + h * nt if st["table"] is None else st["table"][b].long() * hkv + hh
    raw = packed[rows]
    bits = ((raw.long()[:, :, None] >> torch.arange(8, device=DEV)) & 1).view(nt, -1)

    def number(at, w):  # w bits from at, little-endian
        return sum(bits[:, at + k] << k for k in range(w))

    K = torch.zeros((nt, 64, 128), dtype=torch.float64, device=DEV)
    slot_byte = 0
    for gi, (w, pos, m, dims) in enumerate(tab["groups"][h]):
        y = torch.zeros((nt, 8, 8, m), dtype=torch.float64, device=DEV)  # u, g: token g + 8 u
        cb = torch.tensor(c["centroids"][w], device=DEV)
        for s in range(m // 2):
            for e in range(2):
                at = 8 * slot_byte + (torch.arange(8, device=DEV)[None, :] * 16 + 2 * torch.arange(8, device=DEV)[:, None] + e) * w
                y[..., 2 * s + e] = cb[number(at.flatten(), w)].view(nt, 8, 8)
            slot_byte += 16 * w
        o = 1024 * (kb + vb) + 128 + 128 * gi
        n = raw[:, o:o + 128].contiguous().view(torch.float16).double().view(nt, 8, 8).transpose(1, 2)
        y = (y * (n / math.sqrt(m))[..., None]).view(nt, 64, m) @ torch.tensor(_key_rotation(m), device=DEV)
        K[:, :, torch.tensor(dims, device=DEV)] = y
    V = torch.zeros((nt, 64, 128), dtype=torch.float64, device=DEV)
    cb = torch.tensor(c["centroids"][vb], device=DEV)
    x = torch.arange(32, device=DEV)
    for p in range(256):
        i, g, q = p >> 5, (p >> 2) & 7, p & 3
        at = 8192 * kb + p * 32 * vb + x * vb
        V[:, 16 * (x >> 3) + 2 * q + (x & 1) + 8 * ((x >> 2) & 1), 16 * i + g + 8 * ((x >> 1) & 1)] = cb[number(at, vb)]
    o = 1024 * (kb + vb)
    n = raw[:, o:o + 128].contiguous().view(torch.float16).double().view(nt, 8, 8).transpose(1, 2).reshape(nt, 64, 1)
    V = (V * n).view(-1, 128) @ torch.tensor(c["rv"], device=DEV) / math.sqrt(128)
    return K.view(-1, 128), V


def _exact_attention(st, chunk):
    case = st["case"]
    B, hq, hkv, n, T = case["B"], case["hq"], case["hkv"], case["n"], case["T"]
    g = hq // hkv
    got = (torch.zeros((B, hq, n, 128), dtype=torch.float64, device=DEV) if chunk else
           torch.zeros((B, hkv, T), dtype=torch.float64, device=DEV))
    lens, cl = st["lens"].tolist(), st["chunk_lens"].tolist()
    for b in range(B):
        for h in range(hkv):
            K, V = _exact_head(st, b * hkv + h)
            K, V = K[:lens[b]], V[:lens[b]]
            for i0 in range(0, cl[b], 64):
                i1 = min(i0 + 64, cl[b])
                q = st["q"][b, h * g:(h + 1) * g, i0:i1].double()
                s = q @ K.T / math.sqrt(128)
                if case["causal"]:
                    last = torch.arange(i0, i1, device=DEV) + lens[b] - cl[b]
                    s = s.masked_fill(torch.arange(lens[b], device=DEV) > last[:, None], -math.inf)
                p = torch.nan_to_num(torch.softmax(s, -1), nan=0.0)
                if chunk:
                    got[b, h * g:(h + 1) * g, i0:i1] = p @ V
                else:
                    got[b, h, :lens[b]] += p.sum((0, 1))
            if not chunk and st["w_in"] is not None:
                got[b, h, :lens[b]] += st["w_in"][b, h, :lens[b]].double()
    return got


def _exact_evict(st):
    """What stays, by sorting each head's tokens on the host; the codes that move are whole numbers and need no more."""
    case = st["case"]
    keep, lens, w = case["keep"], st["lens"].tolist(), st["w"].double().cpu().numpy()
    kept = np.full(w.shape[:2] + (keep,), -1, np.int64)
    weights = np.zeros(kept.shape)
    for b, n in enumerate(lens):
        t = np.arange(n)
        by_place = (t < case["first"]) | (t >= n - case["recent"])
        for h in range(case["hkv"]):
            best = np.sort(np.lexsort((t, -w[b, h, :n], ~by_place))[:keep])
            kept[b, h, :len(best)], weights[b, h, :len(best)] = best, w[b, h, best]
    return {"dst": None, "lens": np.minimum(lens, keep), "kept": kept, "weights": weights}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(st)
    return _exact_evict(st) if case["op"] == "evict" else _exact_attention(st, case["op"] == "chunk")
