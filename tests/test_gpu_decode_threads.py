"""The decoding operators from several host threads at once, each on a stream, cache and workspaces of its own
(needs a gfx950 GPU): every result is that of the same calls made one after another."""
from __future__ import annotations

import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def cr():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rotation_w4a4_quantized_convrot_amd as mod
    mod.load_library()
    return mod


class Program:
    """Prompts of its own sizes and a few steps of one token: every kernel that splits, stages or prepares."""

    def __init__(self, cr, seed):
        gen = torch.Generator().manual_seed(seed)
        self.cr, self.D, self.Hq, self.H, self.page = cr, (64, 128, 256)[seed % 3], 8, 2, 32
        self.prompt = [40 + 17 * seed, 1300 + 100 * seed]
        hidden, out = 512, (self.Hq + 2 * self.H) * self.D
        w = (torch.randn((out, hidden), generator=gen) * 0.05).to(torch.bfloat16).to(DEV)
        self.layer = cr.ConvLinearW4A16.from_linear(w, group_size=(256, 1024, 0)[seed % 3], scale_group=(32, 64, 128)[seed % 3])
        self.inv = cr.convrot_rotary_frequencies(self.D).to(DEV)
        used = [-(-(n + 4) // self.page) for n in self.prompt]
        ids = torch.randperm(sum(used), generator=gen).to(torch.int32)
        table = torch.full((2, max(used)), -1, dtype=torch.int32)
        table[0, :used[0]], table[1, :used[1]] = ids[:used[0]], ids[used[0]:]
        self.table, self.pages = table.to(DEV), sum(used)
        self.xs = [torch.randn((n, hidden), generator=gen).to(torch.bfloat16).to(DEV) for n in (sum(self.prompt), 2, 2, 2)]
        # what a step needs is made before any thread starts
        self.steps = []
        for step, x in enumerate(self.xs):
            n = self.prompt if step == 0 else [1, 1]
            lens = [p + step for p in self.prompt]
            pos = torch.cat([torch.arange(a - b, a) for a, b in zip(lens, n)])
            self.steps.append((pos.to(DEV), torch.tensor([0, n[0], sum(n)], dtype=torch.int32, device=DEV),
                               torch.tensor(lens, dtype=torch.int32, device=DEV), max(n), max(lens)))

    def run(self):
        cr, out = self.cr, []
        cache = cr.KVCache8bit(self.pages, self.page, self.H, self.D, 16, device=DEV)
        for x, (pos, cu, lens, new, longest) in zip(self.xs, self.steps):
            rows = self.layer(x).view(-1, self.Hq + 2 * self.H, self.D)
            q, k, v = rows.split((self.Hq, self.H, self.H), dim=1)
            cr.convrot_rotary(q, k, pos, self.inv, q_out=q, k_out=k)
            cache.append(k, v, cu, lens, self.table, new)
            out.append(cache.attention(q, cu, lens, self.table, max_new=new, max_len=longest))
        return out + list(cache.read(torch.stack((lens[0] * 0, lens[0], lens.sum())).to(torch.int32), lens, self.table,
                                     tokens=sum(self.prompt) + 6))


def test_decoding_from_several_threads(cr):
    print("\n[case] decoding operators from four threads", flush=True)
    programs = [Program(cr, seed) for seed in range(4)]
    want = [p.run() for p in programs]
    torch.cuda.synchronize()
    got, errors = [[] for _ in programs], []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(5):
                    got[i].append(programs[i].run())
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(programs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for mine, ref in zip(got, want):
        for run in mine:
            for a, b in zip(run, ref):
                assert torch.equal(a.view(torch.int16), b.view(torch.int16))
