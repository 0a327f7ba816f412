"""The eviction's launch follows the table's width and the number of sequences: CTAs per sequence, threads
per CTA, numbers held in registers, in shared memory or read again.  The choice is the same in all."""
import random
import subprocess
import sys

import pytest
import torch

import mla_causal_attention_gb300 as mla
from mla_causal_attention_gb300 import binding
from mla_causal_attention_gb300.build import ROOT
from test_evict import pages, run_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,positions,most", [
    (70, 32768, 9000),     # 2 CTAs of 1024 threads
    (77, 16384, 16384),    # one of 1024, two rounds of rows
    (152, 16384, 5000),
    (100, 8192, 8192),     # 2 of 512
    (152, 8192, 8192),
    (153, 8192, 4097),     # one of 1024
    (19, 32768, 20000),    # 8 of 512
    (39, 32768, 32768),    # 2 of 1024
    (36, 65536, 32768),    # 4 of 1024
    (38, 65536, 32768),    # 2 of 1024
    (37, 262144, 20000),   # 8 of 1024, three waves
    (3, 65536, 65536),     # 16 of 512
    (3, 131072, 70000),    # 16 of 1024
    (64, 131072, 8192),    # a table far wider than the sequences
    (1, 4096, 4096), (1, 4112, 4100),
])
@pytest.mark.parametrize("kind", ["plain", "odd"])
def test_choice_in_every_launch(B, positions, most, kind):
    r = random.Random(B + positions)
    lens = [r.randint(0, most) for _ in range(B - 1)] + [most]
    budgets = [r.randint(0, 1 + n) for n in lens]
    wide = positions // 16 - max(pages(n, 16) for n in lens)
    run_case(lens, budgets, 3, 17, 16, kind, B, K=max(1, max(map(min, lens, budgets))), extra=wide)


def test_freed_pages_are_listed_as_the_table_has_them():
    ws = mla.Workspace("cuda:0")
    i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    w = torch.rand(8, 16, device="cuda")

    def call(table):
        p = mla.mla_paged_evict(w, i(table), i([60, 64, 33]), i([20, 16, 32]), workspace=ws)
        return p.freed[:int(p.n_freed)].tolist(), mla.mla_attn_get_status(ws)

    # shared pages come up for each sequence that lets go of them
    assert call([[0, 1, 2, 3], [4, 1, 2, 2], [0, 1, 5, -1]]) == ([2, 3, 1, 2, 2, 5], 0)
    # and so do entries that are no pages, with the status to say so
    freed, status = call([[0, 1, 2, -1], [4, 8, 6, 7], [0, 1, 5, -1]])
    assert freed == [2, -1, 8, 6, 7, 5] and status == binding.MlaStatus.ERR_PAGE


def test_a_process_whose_first_choice_is_captured():
    """What the launch asks the device (attributes, clusters at once) it can ask within a capture."""
    code = """
import torch
import mla_causal_attention_gb300 as mla
i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
B, width = 70, 2048
w = torch.rand(B * 4, 16, device="cuda")
table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
table[:, :4] = torch.arange(B * 4, device="cuda", dtype=torch.int32).view(B, 4)
lens, budget = i([60] * B), i([20] * B)
out = (i([[0] * 20] * B), i([0] * B), i([0] * (B * width)), i([0]))
ws = mla.Workspace("cuda:0")
mla.mla_rope_apply(torch.rand(1, 2, device="cuda"), i([0]), torch.rand(1, 2, device="cuda"), workspace=ws)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    mla.mla_paged_evict(w, table, lens, budget, 2, 3, out=out, workspace=ws)
g.replay()
torch.cuda.synchronize()
v = w.view(B, 64)[:, 2:57]
best = v.topk(15).indices.sort().values + 2
want = torch.cat((i([[0, 1]] * B), best.to(torch.int32), i([[57, 58, 59]] * B)), 1)
print(torch.equal(out[0], want), out[1].unique().tolist(), int(out[3]), mla.mla_attn_get_status(ws))
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.stdout.split() == ["True", "[20]", "140", "0"], r.stdout + r.stderr
