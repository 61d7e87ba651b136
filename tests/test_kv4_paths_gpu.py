"""Every path of kv4_fwd (8 and 16 rows a warp, 16 and 32 a block, pages expanded):
where one ends and the next begins, over workspaces that held anything, and as captured
graphs of later lengths.  Tolerances as in test_kv4_edges_gpu."""
import pytest
import torch

from test_kv4_edges_gpu import ROWS, close, wanted
from test_kv4_gpu import Batch, U, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import attention_blackwell_gb300 as fa
    fa.lib()
    return fa


@pytest.mark.parametrize("small", [False, True])
@pytest.mark.parametrize("d,hq,n", [(64, 4, 16), (64, 5, 13), (128, 8, 8), (128, 4, 32), (128, 3, 43), (256, 12, 11), (256, 4, 64), (256, 1, 257)])
def test_rows_at_the_change_of_path(fa, d, hq, n, small):
    """Up to d rows of a request and key/value head from the codes, more of them from
    expanded pages, or, where the workspace is short of that, from the codes as well."""
    rows = hq * n
    b = Batch(2 * hq, 2, d, 16, [300, 90, 700], [n, 1, n], seed=rows)
    W, T = len(b.table[0]), b.T
    ws = fa.kv4_workspace(3, 2 * hq, 2, T, W, 16, 1 if small else n, d)
    full = fa.kv4_workspace(3, 2 * hq, 2, T, W, 16, n, d).numel()
    assert (full > fa.kv4_workspace(3, 2 * hq, 2, T, W, 16, 1, d).numel()) == (rows > d)
    o, lse = b.run(fa, workspace=ws)
    assert fa.device_status() == 0
    close(b, o, lse, wanted(b), 2.0 ** -10 if small or rows <= d else U)


# A kernel's rows, and prompts over expanded pages.
PATHS = ROWS + [(64, 8, 2, 40), (128, 8, 2, 40), (256, 8, 2, 70)]


@pytest.mark.parametrize("d,hq,hkv,n", PATHS)
def test_what_a_workspace_held_does_not_matter(fa, d, hq, hkv, n):
    b = Batch(hq, hkv, d, 16, [3000, 17, 900, 0, 2000], [n, 1, n, 1, 1], seed=9 + d, tail=2)
    b.table[2][5] = -1
    ws = fa.kv4_workspace(5, hq, hkv, b.T, len(b.table[0]), 16, n, d)
    out, lse = torch.full((b.T, hq, d), 5.0, dtype=torch.bfloat16, device="cuda"), torch.full((hq, b.T), 5.0, device="cuda")
    first = [x.clone() for x in b.run(fa, workspace=ws, out=out, lse=lse)]
    b.check(fa, *first)
    for fill in (0, 255, 127):
        ws.fill_(fill)
        o, l = b.run(fa, workspace=ws, out=out, lse=lse)
        assert torch.equal(o, first[0]) and torch.equal(l, first[1])
    assert (out[-2:] == 5).all() and (lse[:, -2:] == 5).all()


@pytest.mark.parametrize("d,hq,hkv,n", PATHS)
def test_a_graph_serves_other_lengths_and_offsets(fa, d, hq, hkv, n):
    b = Batch(hq, hkv, d, 16, [700, 80, 5], [n, 1, n], seed=5 + d, tail=1)
    for x in (b.ks, b.vs):
        x[x == 0xFC] = 0x60                          # lengths change below
    args, cu = list(b.args()), i32(b.cu)
    ws = fa.kv4_workspace(3, hq, hkv, b.T, len(b.table[0]), 16, n, d)
    out, lse = torch.empty(b.T, hq, d, dtype=torch.bfloat16, device="cuda"), torch.empty(hq, b.T, device="cuda")
    run = lambda: fa.kv4_fwd(*args, cu_seqlens=cu, max_seqlen=n, alpha=b.alpha, out=out, lse=lse, workspace=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for s, n3 in (([700, 80, 5], [n, 1, n]), ([7, 0, 1], [1, n, n]), ([300, 66, 4], [n, n, 1]), ([650, 1, 0], [0, n, 0])):
        b.s, b.n, b.cu = s, n3, [0, n3[0], n3[0] + n3[1], sum(n3)]
        args[-1].copy_(i32(s))
        cu.copy_(i32(b.cu))
        out.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        b.check(fa, out, lse)
        assert (out[sum(n3):] == 9).all()
