"""A packed cache made by the library, and what it holds read back in fp64 (for the tests of the operators around it)."""

import numpy as np
import torch

import decode_attention_13_b200 as gtq
from decode_attention_13_b200 import synth
from oracle import allocation, quantize
from tests import layout


class Cache:
    """Ragged batch of sequences coded by the library; K[b][h], V[b][h]: fp64 [len_b, 128] as attention sees them."""

    def __init__(self, lens, hkv=2, gq=4, kb=3, vb=3, cap=None, paged=False, pairing=0, seed=0, scale=1.0):
        self.lens, self.B, self.hkv, self.gq, self.hq = list(lens), len(lens), hkv, gq, hkv * gq
        self.kb, self.vb, self.pairing = kb, vb, pairing
        self.cap = cap or max(max(lens), 1)
        self.lay = synth.layer((seed, 91), self.B, hkv, gq, self.cap, theta=1e4)
        self.k = torch.from_numpy(self.lay["k"]).cuda() * scale
        self.v = torch.from_numpy(self.lay["v"]).cuda()
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.cfg = gtq.make_config(self.B, self.hq, hkv, kb, vb, self.cap, rope_pairing=pairing)
        self.tb = layout.tile_bytes(kb, vb)
        self.tiles = (self.cap + 63) // 64
        self.table, self.pages = None, None
        self.rng = np.random.default_rng(seed + 5)
        if paged:
            self.pages = self.B * self.tiles + 3
            perm = self.rng.permutation(self.pages)[:self.B * self.tiles].reshape(self.B, self.tiles)
            self.table = torch.tensor(perm, dtype=torch.int32, device="cuda")
        self.layout = gtq.seq_layout(self.seq_lens, self.table)
        self.plan = gtq.gtq_alloc_bits_ex(self.cfg, self.k, self.cap, self.layout)
        nbytes = self.pages * hkv * self.tb if paged else self.plan.packed_bytes
        self.packed = torch.full((nbytes,), 0xA5, dtype=torch.uint8, device="cuda")
        gtq.gtq_quantize_pack_ex(self.plan, self.k, self.v if vb else None, 0, self.cap, self.packed, self.layout)
        self.bits = gtq.gtq_get_bits(self.plan)
        self.read()

    def head_bytes(self, packed, table, b, h, tiles):
        p = packed.cpu().numpy()
        if table is None:
            i = (b * self.hkv + h) * self.tiles * self.tb
            return p[i:i + tiles * self.tb]
        return layout.gather_paged_head(p, table[b].cpu().numpy(), self.hkv, h, tiles, self.tb)

    def head(self, packed, table, b, h, n):
        """(codes by group, value codes, value norms) of the first n tokens of a head."""
        buf = self.head_bytes(packed, table, b, h, (n + 63) // 64)
        return layout.read_head(buf, self.bits[b, h], self.kb, self.vb, n)

    def dequantised(self, packed, table, b, h, n):
        if n == 0:
            return np.zeros((0, 128)), np.zeros((0, 128))
        keys, vc, vn = self.head(packed, table, b, h, n)
        by_width = {g.width: g.coords for g in allocation.groups(self.bits[b, h], 128, self.pairing)}
        kg = [quantize.CodedGroup(w, by_width[w], c, n16, n16.astype(np.float64), False) for w, c, n16 in keys]
        K = quantize.dequantize_keys(kg, 128, n)
        if not self.vb:
            return K, None
        vg = quantize.CodedGroup(self.vb, tuple(range(128)), vc, vn, vn.astype(np.float64), False)
        return K, quantize.dequantize_values(vg)

    def read(self):
        got = [[self.dequantised(self.packed, self.table, b, h, n) for h in range(self.hkv)]
               for b, n in enumerate(self.lens)]
        self.K = [[x[0] for x in row] for row in got]
        self.V = [[x[1] for x in row] for row in got]

    def queries(self, n, seed=0):
        """fp16 [B, hq, n, 128] drawn like the cache's keys' heads."""
        lay = synth.layer((seed, 17), self.B, self.hkv, self.gq, 1, theta=1e4)
        rng = np.random.default_rng(seed + 23)
        std = np.abs(lay["q"].astype(np.float64)) + 0.1
        q = rng.standard_normal((self.B, self.hq, n, 128)) * std[:, :, None, :]
        return torch.from_numpy(q.astype(np.float16)).cuda()


def probabilities(q, K, n_b, causal):
    """Softmax rows [heads, n_b, tokens] in fp64 of q [heads, n_b, 128] over K; rows that see nothing are 0."""
    n = K.shape[0]
    s = q.astype(np.float64) @ K.T / np.sqrt(128.0)
    if causal:
        last = n - n_b + np.arange(n_b)
        s = np.where(np.arange(n)[None, None, :] <= last[None, :, None], s, -np.inf)
    if n == 0:
        return s
    top = s.max(-1, keepdims=True)
    p = np.exp(s - np.where(np.isfinite(top), top, 0.0))
    z = p.sum(-1, keepdims=True)
    return np.where(z > 0, p / np.where(z > 0, z, 1.0), 0.0)


def workspace(nbytes):
    return torch.full((max(int(nbytes), 256),), 0xFF, dtype=torch.uint8, device="cuda")
