"""The four-bit serving path as a program runs it: block manager, rotation, prompt attention, cache
writes, copy-on-write, decode steps, a second chunk of a prompt over gathered context, a swap to host
memory and back.  Every attention output against the fp64 oracle on what the cache stands for.

Tolerance: attention outputs here are averages of values below 4 in size with errors of a few roundings
of 2^-11 (weights and output) and of 8/15 * 2^-11 of a row's span (cached values): 2e-3 * 4."""
import numpy as np
import pytest
import torch

from oracle import attention as oracle_attention
from oracle import int4_cache as o4
from paged_kv_cache_73_gb300 import binding as pkv

pytestmark = pytest.mark.gpu

H, HK, D, B = 6, 2, 64, 8
SCALE = D ** -0.5
ATOL = 8e-3


class Model:
    """One layer's projections stood in for by random rows; per sequence the fp64 rows its cache holds."""

    def __init__(self, dev):
        self.dev, self.rng = dev, np.random.default_rng(3)
        self.inv = 10000.0 ** (-np.arange(D // 2) / (D // 2))
        self.freq = pkv.rope_frequencies(self.inv, dev)
        self.w = [torch.from_numpy((1 + 0.1 * self.rng.standard_normal(D)).astype(np.float16)).to(dev) for _ in range(2)]
        self.bm = pkv.BlockManager(64, B, list(self.rng.permutation(64)))
        self.k = torch.zeros(pkv.int4_cache_shape(64, HK, B, D), dtype=torch.uint8, device=dev)
        self.v = torch.zeros_like(self.k)
        self.rows = {}

    def project(self, positions):
        """Rotated q and k, and v, of tokens at the given positions."""
        qkv = torch.from_numpy(self.rng.standard_normal((len(positions), H + 2 * HK, D)).astype(np.float16)).to(self.dev)
        pos = torch.tensor(positions, dtype=torch.int32, device=self.dev)
        q, k = pkv.qk_norm_rope(qkv[:, :H], qkv[:, H:H + HK], pos, self.freq, *self.w)
        return q, k, qkv[:, H + HK:]

    def write(self, k, v, slots, owners):
        pkv.reshape_and_cache_int4(k, v, self.k, self.v, torch.as_tensor(slots, device=self.dev), B)
        for x, kind in ((k, 0), (v, 1)):
            n, s, z = o4.quantise_rows(x.cpu().numpy())
            stored = z.astype(np.float64)[..., None] + s.astype(np.float64)[..., None] * n
            for t, seq in enumerate(owners):
                self.rows.setdefault(seq, ([], []))[kind].append(stored[t])

    def cached(self, seq):
        return [np.repeat(np.stack(r), H // HK, axis=1) for r in self.rows[seq]]

    def decode(self, seqs, q):
        tables, lens = self.bm.block_tables(seqs, 16)
        out = pkv.paged_attention_decode_int4(q, self.k, self.v, torch.from_numpy(tables).to(self.dev),
                                              torch.from_numpy(lens).to(self.dev), SCALE, B)
        assert pkv.device_error() == 0
        for i, seq in enumerate(seqs):
            k, v = self.cached(seq)
            assert len(k) == lens[i]
            want = oracle_attention.contiguous_attention(q[i].cpu().numpy(), k, v, SCALE)
            assert np.abs(out[i].cpu().numpy() - want).max() <= ATOL
        return out

    def step(self, seqs):
        """One token of every sequence: positions, slots (and copies), write, decode."""
        q, k, v = self.project([len(self.rows[s][0]) for s in seqs])
        slots, pairs = self.bm.append_slots(seqs)
        if len(pairs):
            pkv.copy_blocks_int4([self.k], [self.v], torch.from_numpy(pairs).to(self.dev), B)
        self.write(k, v, slots, seqs)
        return self.decode(seqs, q), len(pairs)


def test_serving_path(cuda_device):
    m = Model(cuda_device)
    # the prompts of two requests, packed
    lens = {1: 37, 2: 90}
    q, k, v = m.project([t for n in lens.values() for t in range(n)])
    start = torch.tensor([0, 37, 127], dtype=torch.int32, device=cuda_device)
    out = pkv.prompt_attention(q, k, v, start, SCALE, 90)
    want = o4.prompt_attention(q.cpu().numpy(), k.cpu().numpy(), v.cpu().numpy(), [0, 37, 127], [0, 37, 127], SCALE)
    assert np.abs(out.cpu().numpy() - want).max() <= ATOL
    slots = np.concatenate([m.bm.add_seq(s, n) for s, n in lens.items()])
    m.write(k, v, slots, [s for s, n in lens.items() for _ in range(n)])

    # two samples of request 1 share its blocks until they write
    m.bm.fork(1, 3)
    m.rows[3] = ([*m.rows[1][0]], [*m.rows[1][1]])
    copies = [m.step([1, 2, 3])[1] for _ in range(4)]
    assert copies[0] == 1 and sum(copies[1:]) == 0           # 37 tokens: the fifth block is partly filled

    # a second chunk of request 2: its context back as fp16 rows, its own tokens after them
    n, past = 20, len(m.rows[2][0])
    q, k, v = m.project(list(range(past, past + n)))
    table, _ = m.bm.block_table(2)
    t = np.arange(past)
    ck, cv = pkv.gather_cache_int4(m.k, m.v, torch.from_numpy(np.array(table)[t // B] * B + t % B).to(cuda_device), B)
    keys, values = torch.cat([ck, k]), torch.cat([cv, v])
    out = pkv.prompt_attention(q, keys, values, torch.tensor([0, n], dtype=torch.int32, device=cuda_device), SCALE, n,
                               key_start=torch.tensor([0, past + n], dtype=torch.int32, device=cuda_device))
    kc, vc = m.cached(2)
    fresh = [np.repeat(x.cpu().numpy().astype(np.float64), H // HK, axis=1) for x in (k, v)]
    for i in range(n):
        want = oracle_attention.contiguous_attention(q[i].cpu().numpy(), np.concatenate([kc, fresh[0][:i + 1]]),
                                                     np.concatenate([vc, fresh[1][:i + 1]]), SCALE)
        assert np.abs(out[i].cpu().numpy() - want).max() <= ATOL
    slots, pairs = m.bm.extend(2, n)
    assert len(pairs) == 0
    m.write(k, v, slots, [2] * n)
    m.step([1, 2, 3])

    # request 2 is preempted to host memory and comes back to other blocks
    q, _, _ = m.project([0])
    before = m.decode([2], q)
    host_bm = pkv.BlockManager(32, B)
    host = [torch.zeros(pkv.int4_cache_shape(32, HK, B, D), dtype=torch.uint8).pin_memory() for _ in range(2)]
    pairs = torch.from_numpy(m.bm.swap(host_bm, [2])).to(cuda_device)
    pkv.swap_blocks_int4([m.k], [m.v], host[:1], host[1:], pairs, B)
    m.step([3, 1])                                            # its blocks are used meanwhile
    back = torch.from_numpy(host_bm.swap(m.bm, [2])).to(cuda_device)
    pkv.swap_blocks_int4(host[:1], host[1:], [m.k], [m.v], back, B)
    assert torch.equal(m.decode([2], q), before)
    m.step([2, 3, 1])


def test_decode_step_in_one_graph(cuda_device):
    """Rotation, write and attention of a step captured together and replayed with new inputs."""
    m = Model(cuda_device)
    dev = cuda_device
    q, k, v = m.project(list(range(30)))
    m.write(k, v, m.bm.add_seq(7, 30), [7] * 30)
    qkv = torch.zeros(1, H + 2 * HK, D, dtype=torch.float16, device=dev)
    pos = torch.zeros(1, dtype=torch.int32, device=dev)
    slot = torch.full((1,), -1, dtype=torch.int64, device=dev)
    tables = torch.full((1, 16), -1, dtype=torch.int32, device=dev)
    lens = torch.zeros(1, dtype=torch.int32, device=dev)

    def step():
        q, k = pkv.qk_norm_rope(qkv[:, :H], qkv[:, H:H + HK], pos, m.freq, *m.w)
        pkv.reshape_and_cache_int4(k, qkv[:, H + HK:], m.k, m.v, slot, B)
        return q, k, pkv.paged_attention_decode_int4(q, m.k, m.v, tables, lens, SCALE, B)

    step()                                                    # nothing: no slot, no context
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, k, out = step()
    for i in range(5):
        slots, _ = m.bm.append_slots([7])
        t, n = m.bm.block_tables([7], 16)
        qkv.copy_(torch.from_numpy(m.rng.standard_normal((1, H + 2 * HK, D)).astype(np.float16)))
        pos.fill_(30 + i)
        slot.copy_(torch.from_numpy(slots))
        tables.copy_(torch.from_numpy(t))
        lens.copy_(torch.from_numpy(n))
        graph.replay()
        torch.cuda.synchronize()
        assert pkv.device_error() == 0
        for x, kind in ((k, 0), (qkv[:, H + HK:], 1)):
            nn, s, z = o4.quantise_rows(x.cpu().numpy())
            m.rows[7][kind].append((z.astype(np.float64)[..., None] + s.astype(np.float64)[..., None] * nn)[0])
        kc, vc = m.cached(7)
        want = oracle_attention.contiguous_attention(q[0].cpu().numpy(), kc, vc, SCALE)
        assert np.abs(out[0].cpu().numpy() - want).max() <= ATOL
