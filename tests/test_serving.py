"""The paged-cache operators together, as a server uses them: packed prompts are planned, appended
and attended to; drafted trees follow on the same pages; the accepted path is kept and the next
step goes on from there.  Every attention result is compared with its definition in 64 bits on the
cache as it then is."""
import random

import pytest
import torch

import mla_causal_attention_gb300 as mla
from mla_causal_attention_gb300.workloads import softmax_scale_192
from paged_helpers import pages, random_parents, rotate64, tree_reference

pytestmark = pytest.mark.gpu

SCALE = softmax_scale_192()
PAGE, WIDTH, POOL = 16, 40, 120


def _i(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


class _Server:
    """Buffers of three sequences, one pool, one free list."""

    def __init__(self, H, seed):
        self.g = torch.Generator("cpu").manual_seed(seed)
        self.r = random.Random(seed)
        self.H = H
        ids = list(range(POOL))
        self.r.shuffle(ids)
        self.free, self.head = ids, 0
        nan = lambda n: torch.full((POOL, PAGE, n), float("nan"), dtype=torch.bfloat16,  # noqa: E731
                                   device="cuda")
        self.c_pages, self.pe_pages = nan(512), nan(64)
        self.table = _i([[-1] * WIDTH] * 3)
        self.w = self.normal(H * 256, 512).div(512 ** 0.5)
        self.rope = mla.mla_rope_table(1000)

    def normal(self, *s):
        return torch.randn(*s, generator=self.g).to(torch.bfloat16).cuda()

    def step(self, ctx, new, parents=None, tokens=None):
        """Plans, appends and attends to new tokens; returns (plan, inputs, output)."""
        T = tokens or sum(new)
        par = None if parents is None else _i(parents + [-1] * (T - len(parents)))
        p = mla.mla_paged_plan(_i(ctx), _i(new), self.table, _i(self.free), _i([self.head]), PAGE,
                               POOL, T, parent=par)
        x = dict(c=self.normal(T, 512), pe=self.normal(T, 64), q_nope=self.normal(T, self.H, 128),
                 q_raw=self.normal(T, self.H, 64))
        q = mla.mla_latent_append(x["c"], x["pe"], p.slots, self.c_pages, self.pe_pages,
                                  positions=p.positions, rope_table=self.rope, q_pe=x["q_raw"])
        out = mla.mla_latent_tree_fwd(x["q_nope"], q, self.c_pages, self.pe_pages, self.table,
                                      p.kv_len, p.cu_q, p.draft_mask, self.w, SCALE)
        torch.cuda.synchronize()
        assert mla.mla_attn_get_status() == 0
        self.head = int(p.free_next)
        x["q_pe"] = q
        used = sum(new)
        # the rotated queries and keys are those of the tokens' positions
        want = rotate64(x["q_raw"], self.rope, p.positions)[:used]
        assert bool(((q[:used].double() - want).abs() <= want.abs() * 2 ** -7 + 1e-5).all())
        d = dict(q_nope=x["q_nope"], q_pe=q, c_pages=self.c_pages, pe_pages=self.pe_pages,
                 block_table=self.table, kv_len=p.kv_len, cu_q=p.cu_q, draft_mask=p.draft_mask,
                 w_kvb=self.w)
        ref, spread, mixed = tree_reference(d, SCALE)
        err = (out.double() - ref).abs()[:used]
        assert float(err.norm() / ref[:used].norm()) <= 0.0045  # four roundings to bf16
        assert not bool((err > 2 ** -8 * (7 * spread + mixed)[:used] + 1e-30).any())
        return p, x, out


@pytest.mark.parametrize("H,seed", [(16, 0), (64, 1)])
def test_prompts_then_drafted_trees(H, seed):
    s = _Server(H, seed)
    lens = [70, 1, 200]
    p, x, out = s.step([0, 0, 0], lens, tokens=288)
    T = sum(lens)
    assert p.slots[T:].tolist() == [-1] * 17

    # The same prompts through the packed prompt attention, with each head's keys and values made
    # from the latent rows (rounded to bf16, as a projection's output is) and the rotated keys
    # read back from the cache.
    kv = (x["c"][:T].float() @ s.w.float().T).bfloat16().view(T, H, 256)
    k_pe = s.pe_pages.view(-1, 64)[p.slots[:T].long()]
    packed = mla.mla_attn_varlen_fwd(x["q_nope"][:T], x["q_pe"][:T], kv[..., :128], k_pe,
                                     kv[..., 128:], p.cu_q, SCALE)
    # Rounded keys and values add their 2^-8 to the weights' and the output's: five roundings
    # between the two results and the exact one, each at most 2^-8 / sqrt(3) in the 2-norm, on
    # both sides: sqrt(4 + 4) * 2^-8 / sqrt(3) = 0.0064.
    rel = float((packed.double() - out[:T].double()).norm() / out[:T].double().norm())
    assert rel <= 0.0064

    # the projection of the packed rows, each a row of its own
    w_o = s.normal(128, H * 128).div((H * 128) ** 0.5)
    y = mla.mla_oproj_fwd(out[:T].view(T, H, 1, 128), w_o)
    want = out[:T].reshape(T, -1).double() @ w_o.double().T
    assert float((y.view(T, 128).double() - want).norm() / want.norm()) <= 2 ** -8

    ctx = list(lens)
    for _ in range(3):
        new = [s.r.randint(1, 20) for _ in ctx]
        parents = [random_parents(s.r, n) for n in new]
        p, x, out = s.step(ctx, new, [q for t in parents for q in t], tokens=64)
        cu = p.cu_q.tolist()
        # Accept a path from the root: its rows move up behind the cached ones, the pages past
        # the new end go back to the free list.
        free = []
        for b, n in enumerate(new):
            path, at = [0], 0
            while True:
                kids = [i for i in range(n) if parents[b][i] == at]
                if not kids or len(path) == 4:
                    break
                at = s.r.choice(kids)
                path.append(at)
            rows = p.slots[[cu[b] + i for i in path]].long()
            to = p.slots[cu[b]:cu[b] + len(path)]
            mla.mla_latent_append(s.c_pages.view(-1, 512)[rows], s.pe_pages.view(-1, 64)[rows], to,
                                  s.c_pages, s.pe_pages)
            ctx[b] += len(path)
            held, had = pages(ctx[b], PAGE), pages(int(p.kv_len[b]), PAGE)
            free += s.table[b, held:had].tolist()
            s.table[b, held:had] = -1
        s.free, s.head = free + s.free[s.head:], 0
    assert sorted(s.free + [q for row in s.table.tolist() for q in row if q >= 0]) == list(range(POOL))


def test_two_streams_at_once():
    """Two servers' steps in flight at the same time, each on a stream and a workspace of its own."""
    from paged_helpers import tree_case
    cases = [tree_case(60, 20, 64, (0, 900), (1, 30), 32, True),
             tree_case(61, 5, 64, (2000, 3000), (1, 5), 64, False)]
    streams = [torch.cuda.Stream() for _ in cases]
    spaces = [mla.Workspace() for _ in cases]

    def call(d, out, **kw):
        return mla.mla_latent_tree_fwd(d["q_nope"], d["q_pe"], d["c_pages"], d["pe_pages"],
                                       d["block_table"], d["kv_len"], d["cu_q"], d["draft_mask"],
                                       d["w_kvb"], SCALE, out=out, **kw)

    want = [call(d, None, workspace=w).clone() for d, w in zip(cases, spaces)]
    torch.cuda.synchronize()
    outs = [torch.zeros_like(w) for w in want]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(60):
        for d, o, s, w in zip(cases, outs, streams, spaces):
            call(d, o, stream=s, workspace=w)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
    for w in spaces:
        assert mla.mla_attn_get_status(workspace=w) == 0


def test_a_graph_outlives_its_workspace_growing():
    """A graph captured with the default workspace, then larger calls, then the graph again."""
    from paged_helpers import tree_case
    small = tree_case(62, 3, 8, (100, 400), (1, 9), 32, True)
    large = tree_case(63, 30, 64, (0, 300), (1, 40), 32, True)

    def call(d, **kw):
        return mla.mla_latent_tree_fwd(d["q_nope"], d["q_pe"], d["c_pages"], d["pe_pages"],
                                       d["block_table"], d["kv_len"], d["cu_q"], d["draft_mask"],
                                       d["w_kvb"], SCALE, **kw)

    ws = mla.Workspace()
    want = call(small, workspace=ws).clone()
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(small, out=out, workspace=ws)
    call(large, workspace=ws)
    assert len(ws.outgrown) == 1
    other = torch.full_like(ws.outgrown[0], 255)  # where the first buffer would have been reused
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert bool((other == 255).all())
    small["kv_len"][0] = 0  # below its new tokens: in the status word of the captured call's buffer
    g.replay()
    assert mla.mla_attn_get_status(workspace=ws) == mla.MlaStatus.ERR_KVLEN
    assert mla.mla_attn_get_status(workspace=ws) == 0


def test_workspaces_of_another_device_are_refused():
    """Before anything is launched: the kernels write to the workspace."""
    from paged_helpers import tree_case
    ws = mla.Workspace("cpu")
    ws.buf = torch.zeros(1 << 28, dtype=torch.uint8)
    d = tree_case(64, 2, 8, (10, 40), (1, 3), 32, True)
    x = torch.zeros((1, 8, 4, 128), dtype=torch.bfloat16, device="cuda")
    rot = torch.zeros((1, 8, 4, 64), dtype=torch.bfloat16, device="cuda")
    w_o = torch.zeros((7168, 8 * 128), dtype=torch.bfloat16, device="cuda")
    i = torch.zeros(1, dtype=torch.int32, device="cuda")
    c = torch.zeros((1, 16, 512), dtype=torch.bfloat16, device="cuda")
    for call in (
            lambda: mla.mla_latent_tree_fwd(d["q_nope"], d["q_pe"], d["c_pages"], d["pe_pages"],
                                            d["block_table"], d["kv_len"], d["cu_q"],
                                            d["draft_mask"], d["w_kvb"], SCALE, workspace=ws),
            lambda: mla.mla_paged_plan(i, i, i[None], i, i, 16, 1, 1, workspace=ws),
            lambda: mla.mla_latent_append(c[0, :1], c[0, :1, :64].contiguous(), i, c,
                                          c[..., :64].contiguous(), workspace=ws),
            lambda: mla.mla_attn_fwd(x, rot, x, rot[:, 0], x, None, 0, SCALE, workspace=ws),
            lambda: mla.mla_oproj_fwd(x, w_o, workspace=ws)):
        with pytest.raises(ValueError, match="workspace is on cpu"):
            call()
    torch.cuda.synchronize()
