"""Speculative steps that never return to the host: room for the drafted tokens
(pa_pages_update, pa_copy_pages), their rows appended to a block-scaled cache, each
drafted token decoded over its own context, the drafts verified, the rest cut by the
next step.  Every call against its 64-bit oracle on the step's own inputs, the whole
captured in one graph and replayed, and the tree form with pa_compact_kv."""
import numpy as np
import pytest
import torch

import speclib
from paged_kv_cache_251_gb300 import pa

pytestmark = pytest.mark.gpu

N, T, H, K, D, BS, VOCAB = 6, 3, 8, 2, 64, 16, 300


class Loop:
    """A model of random tables: a token's rows depend on the token and its position alone."""

    def __init__(self, code, blocks=60):
        g = torch.Generator(device="cuda").manual_seed(1)
        rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.embed = {n: rand(VOCAB, h, D) for n, h in (("q", H), ("k", K), ("v", K))}
        self.place = {n: rand(512, h, D) for n, h in (("q", H), ("k", K), ("v", K))}
        self.head = rand(H * D, VOCAB) * 0.15
        self.width = 12
        i32 = dict(dtype=torch.int32, device="cuda")
        lens = torch.tensor([0, 5, 16, 17, 30, 1], **i32)
        self.lens, self.reserved = lens.clone(), lens.clone()
        self.tables = torch.full((N, self.width), -1, **i32)
        self.refs = torch.zeros(blocks, **i32)
        order = torch.randperm(blocks, generator=torch.Generator().manual_seed(2))
        at = 0
        for s, n in enumerate(lens.tolist()):
            have = -(-n // BS)
            self.tables[s, :have] = order[at:at + have].int().cuda()
            at += have
        # two rows share a last block, a prompt cache holds another
        self.tables[3, :2] = self.tables[4, :2]
        for b in self.tables[self.tables >= 0].tolist():
            self.refs[b] += 1
        self.refs[int(self.tables[1, 0])] += 1
        self.pools = [torch.zeros((blocks, K, BS, D), device="cuda").to(code) for _ in range(2)]
        self.pools += [torch.zeros((blocks, K), device="cuda") for _ in range(2)]
        # what the contexts hold already
        tok = torch.randint(0, VOCAB, (N, 64), generator=g, device="cuda")
        for s, n in enumerate(lens.tolist()):
            pos = torch.arange(n, device="cuda")
            slots = self.tables[s].long()[pos // BS] * BS + pos % BS
            self._append(tok[s if s != 3 else 4, :n], pos, slots)
        self.root = torch.randint(0, VOCAB, (N,), generator=g, device="cuda")
        self.new_tables, self.new_refs = torch.empty_like(self.tables), torch.empty_like(self.refs)
        self.pairs, self.status = torch.empty((N, 2), dtype=torch.int64, device="cuda"), torch.zeros(4, **i32)
        self.out = [torch.empty(N, **i32), torch.empty((N, T), **i32), torch.empty((N, T + 1), **i32)]
        self.attn = torch.empty((N * (T + 1), H, D), device="cuda")
        self.drafts = torch.empty((N, T), **i32)
        self.draft_probs = torch.empty((N, T, VOCAB), device="cuda")
        self.uniforms = torch.empty((N, T + 1), device="cuda")
        self.err = torch.zeros(1, **i32)
        self.keep = {}

    def _append(self, tokens, pos, slots):
        rows = {n: (self.embed[n][tokens] + self.place[n][pos]).contiguous() for n in "kv"}
        pa.pa_append_kv_block_quant(rows["k"], rows["v"], slots.contiguous(), *self.pools)

    def draw(self, seed):
        """The step's drafts (from a draft model near the target's taste) and random numbers."""
        g = torch.Generator(device="cuda").manual_seed(seed)
        logits = torch.randn((N, T, VOCAB), generator=g, device="cuda")
        self.draft_probs.copy_(logits.softmax(-1))
        self.drafts.copy_(torch.multinomial(self.draft_probs.view(N * T, VOCAB), 1, generator=g).view(N, T))
        self.uniforms.copy_(torch.rand((N, T + 1), generator=g, device="cuda"))

    def step(self):
        grow = self.lens + (T + 1)
        self.keep["grow"] = grow
        pa.pa_pages_update(self.new_tables, self.new_refs, self.pairs, self.status, self.tables, self.refs, self.reserved,
                           self.lens, grow, BS, err_word=self.err)
        pa.pa_copy_pages(self.pairs, self.pools, err_word=self.err)
        tokens = torch.cat([self.root[:, None], self.drafts.long()], 1)
        pos = self.lens.long()[:, None] + torch.arange(T + 1, device="cuda")
        slots = (self.new_tables.long().gather(1, pos // BS) * BS + pos % BS).view(-1)
        rows = {n: (self.embed[n][tokens] + self.place[n][pos]).view(N * (T + 1), -1, D).contiguous() for n in "qkv"}
        pa.pa_append_kv_block_quant(rows["k"], rows["v"], slots, *self.pools, err_word=self.err)
        lens = (pos + 1).view(-1).int()
        tables = self.new_tables.repeat_interleave(T + 1, 0)
        pa.pa_decode_block_quant(self.attn, rows["q"], *self.pools, tables, lens, err_word=self.err)
        probs = (self.attn.view(N, T + 1, H * D) @ self.head).softmax(-1)
        pa.pa_verify_drafts(*self.out, probs, self.drafts, self.uniforms, draft_probs=self.draft_probs,
                            err_word=self.err)
        self.keep.update(rows=rows, slots=slots, lens=lens, tables=tables, probs=probs)
        # the next step's state
        n = self.out[0]
        self.root.copy_(self.out[2].long().gather(1, n[:, None].long())[:, 0])
        self.lens.add_(n + 1)
        self.reserved.copy_(grow)
        self.tables.copy_(self.new_tables)
        self.refs.copy_(self.new_refs)

    def state(self):
        return [self.lens, self.reserved, self.tables, self.refs, self.root, *self.pools]


@pytest.mark.parametrize("code", [torch.int8, torch.float8_e4m3fn])
def test_steps_against_the_oracles(code):
    loop = Loop(code)
    for step in range(5):
        loop.draw(100 + step)
        before = [x.clone() for x in loop.state()]
        loop.step()
        torch.cuda.synchronize()
        assert loop.err.item() == 0
        want = speclib.pages_update(before[2].tolist(), before[3].tolist(), before[1].tolist(), None, before[0].tolist(),
                                    loop.keep["grow"].tolist(), BS)
        assert [loop.new_tables.tolist(), loop.new_refs.tolist(), loop.pairs.tolist(), loop.status.tolist()] == list(want)
        pools = [p.cpu() for p in before[5:]]
        for a, b in loop.pairs.tolist():
            if a >= 0:
                for p in pools:
                    p.view(torch.uint8 if p.dtype == code else p.dtype)[b] = \
                        p.view(torch.uint8 if p.dtype == code else p.dtype)[a].clone()
        rows = loop.keep["rows"]
        want = speclib.append_block_quant(rows["k"].cpu(), rows["v"].cpu(), loop.keep["slots"].cpu(), *pools)
        for got, w in zip(loop.pools, want):
            assert torch.equal(got.cpu().double(), w)
        want = speclib.decode_block_quant(rows["q"].cpu(), *[p.cpu() for p in loop.pools], loop.keep["tables"].cpu(),
                                          loop.keep["lens"].cpu())
        # scores up to 60 in fp32 sums of 64 products (64 * 60 * 2^-24) and 22-bit weights, of |v| up to 8
        assert (loop.attn.cpu().double() - want).abs().max() <= 8 * (64 * 60 * 2.0 ** -24 + 2.0 ** -21)
        want = speclib.verify(loop.keep["probs"].double().cpu().numpy(), loop.draft_probs.double().cpu().numpy(),
                              loop.drafts.cpu().numpy(), loop.uniforms.cpu().numpy())
        for got, w in zip(loop.out, want):
            np.testing.assert_array_equal(got.cpu().numpy(), w)


def test_the_same_steps_from_a_graph():
    eager, graphed = Loop(torch.int8), Loop(torch.int8)
    eager.draw(7), graphed.draw(7)
    eager.step(), graphed.step()  # (the first of each outside the graph)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed.step()
    for a, b in zip(graphed.state(), eager.state()):  # (capturing ran nothing)
        b_bytes, a_bytes = b.view(torch.uint8) if b.element_size() == 1 else b, a.view(torch.uint8) if a.element_size() == 1 else a
        assert torch.equal(a_bytes, b_bytes)
    for step in range(6):
        eager.draw(50 + step), graphed.draw(50 + step)
        eager.step()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager.state() + eager.out, graphed.state() + graphed.out):
            assert torch.equal(a, b)
    assert eager.err.item() == graphed.err.item() == 0


def test_tree_attention_verification_and_commit():
    """A tree over a 16-bit cache: attention of its tokens, verification, and the accepted ones moved
    together by the list that verification wrote."""
    g = torch.Generator().manual_seed(3)
    n, t, lens = 4, 7, [20, 33, 16, 50]
    parents = torch.tensor([[-1, -1, 0, 0, 1, 2, 4]] * n, dtype=torch.int32)
    need = [-(-(x + t) // BS) for x in lens]
    tables = torch.arange(sum(need), dtype=torch.int32).split(need)
    width = max(need)
    tables = torch.stack([torch.cat([x, torch.full((width - len(x),), -1, dtype=torch.int32)]) for x in tables])
    kc, vc = (torch.randn((sum(need), K, BS, 128), generator=g).half().cuda() for _ in range(2))
    q = torch.randn((n, t, 8, 128), generator=g).half().cuda()
    out = torch.empty((n, t, 8, 128), device="cuda")
    base = torch.tensor(lens, dtype=torch.int32, device="cuda")
    pa.pa_decode_tree(out, q, kc, vc, tables.cuda(), base + t, tree_mask=pa.tree_mask_from_parents(parents).cuda())
    probs = torch.cat([torch.rand((n, 1, 90), generator=g).cuda().softmax(-1),
                       (out.view(n, t, -1)[:, :, :90]).softmax(-1)], 1)
    tokens = torch.multinomial(probs[:, 0], t, replacement=True).int()
    res = [torch.empty(s, dtype=torch.int32, device="cuda") for s in ((n,), (n, t), (n, t + 1))]
    draft = probs[:, :t].contiguous()
    pa.pa_verify_drafts(*res, probs, tokens, torch.rand((n, t + 1), generator=g).cuda(), draft_probs=draft,
                        parents=parents.cuda())
    before = kc.clone(), vc.clone()
    pa.pa_compact_kv(kc, vc, res[1].view(n, 1, t), res[0], tables.cuda(), base_lens=base)
    torch.cuda.synchronize()
    assert (res[0] > 0).any()
    for s in range(n):
        for i in range(int(res[0][s])):
            src, dst = lens[s] + int(res[1][s, i]), lens[s] + i
            a, b = int(tables[s, src // BS]), int(tables[s, dst // BS])
            for now, old in zip((kc, vc), before):
                assert torch.equal(now[b, :, dst % BS], old[a, :, src % BS])
