"""Embedding lookup with scaling and its gradient by sorted tokens (through the
C ABI).  The lookup is one float32 product rounded once: bit for bit.  A row of
the gradient is a float32 sum of its n terms: within n 2^-24 of their absolute
sum (and one rounding of the scaling)."""
import pytest
import torch

from oracle import sequence as seq

pytestmark = pytest.mark.gpu
TD = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def built():
    from protein_structure_models_b200 import build
    build.build()


def rnd(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


def indices(T, V, how, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if how == "one":                       # every token the same
        return torch.full((T,), V // 2, dtype=torch.int32, device="cuda")
    if how == "outside":                   # half of them outside [0, V), at the ends of int32 too
        i = torch.randint(-V - 1, 2 * V + 1, (T,), generator=g, device="cuda", dtype=torch.int64)
        i[::7] = 2 ** 31 - 1
        i[3::7] = -2 ** 31
        return i.int()
    if how == "sorted":
        return torch.sort(torch.randint(0, V, (T,), generator=g, device="cuda")).values.int()
    if how == "skew":
        return (torch.rand(T, generator=g, device="cuda") ** 4 * V).long().clamp(max=V - 1).int()
    return torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)


def check(idx, V, C, dtype, scale=1.0, seed=3):
    import protein_structure_models_b200 as fw
    table, d = rnd((V, C), TD[dtype], seed), rnd((*idx.shape, C), TD[dtype], seed + 1)
    out = fw.embedding(idx, table, scale=scale)["out"]
    ok = (idx >= 0) & (idx < V)
    sc = torch.tensor(scale, dtype=torch.float32, device="cuda")
    assert torch.equal(out, ((table.float() * sc)[idx.long().clamp(0, V - 1)] * ok[..., None]).to(out.dtype))
    g = fw.embedding_backward(idx, d, V, scale=scale)["table"]
    scale = float(sc)
    want = seq.embedding_backward(idx, d, V, scale)
    n = torch.bincount(idx[ok].cpu().long(), minlength=V).double()[:, None]
    tol = abs(scale) * n * 2.0 ** -24 * seq.embedding_backward(idx, d.abs(), V, 1.0) + want.abs() * 2.0 ** -23
    assert g.dtype == torch.float32 and ((g.cpu().double() - want).abs() <= tol).all()
    assert (g.cpu()[n[:, 0] == 0] == 0).all()
    return table, d, out, g


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,C", [(1, 1, 1), (1, 5, 8), (31, 3, 7), (33, 1, 16), (513, 21, 256), (2049, 64, 20), (4096, 300, 1),
                                   (5000, 255, 128), (5000, 256, 33), (3000, 257, 8), (20000, 70000, 12), (6000, 100000, 4),
                                   (700, 9, 1032), (300, 40, 3001), (70000, 64, 16), (128, 700, 264), (127, 3, 131),
                                   (129, 40, 24), (90, 20000, 40)])
@pytest.mark.parametrize("how", ["even", "one", "outside", "skew"])
def test_against_the_definition(dtype, T, V, C, how):
    check(indices(T, V, how), V, C, dtype, scale=2.5)


def test_sorted_tokens_and_shapes():
    check(indices(9000, 500, "sorted"), 500, 64, "f32", scale=-0.37)
    check(indices(3 * 5 * 7, 11, "even").view(3, 5, 7), 11, 24, "bf16", scale=16.0)


def test_nothing_to_look_up():
    import protein_structure_models_b200 as fw
    idx = torch.empty(0, dtype=torch.int32, device="cuda")
    assert fw.embedding(idx, rnd((4, 8), torch.float32, 1))["out"].shape == (0, 8)
    g = fw.embedding_backward(idx, torch.empty(0, 8, device="cuda"), 4)["table"]
    assert (g == 0).all()


def test_values_pass_as_they_are():
    """NaN and infinities reach only the rows that they belong to; a skipped token's gradient is never used."""
    import protein_structure_models_b200 as fw
    idx = torch.tensor([0, -1, 2, 0, 7, 3], dtype=torch.int32, device="cuda")
    d = torch.ones(6, 8, device="cuda")
    d[1] = float("nan")
    d[4] = float("inf")
    d[2] = float("nan")
    g = fw.embedding_backward(idx, d, 4)["table"]
    assert (g[0] == 2).all() and (g[1] == 0).all() and g[2].isnan().all() and (g[3] == 1).all()


@pytest.mark.parametrize("C", [16, 30])
def test_unaligned_guards_repeats_graph(C):
    import protein_structure_models_b200 as fw
    T, V = 3000, 50
    idx = indices(T, V, "skew")
    table, d, out, g = check(idx, V, C, "bf16")
    b = torch.empty(T * C + 1, dtype=torch.bfloat16, device="cuda")
    b[1:] = d.view(-1)
    gb = torch.full((V * C + 129,), 5.0, device="cuda")
    gv = gb[65:65 + V * C].view(V, C)
    need = fw.embedding_backward_workspace_size(T, V, C)
    ws = torch.full((need + 512,), 9, dtype=torch.uint8, device="cuda")
    fw.embedding_backward(idx, b[1:].view(T, C), V, workspace=ws[256:256 + need], grads={"table": gv})
    assert torch.equal(gv, g) and (gb[:65] == 5).all() and (gb[65 + V * C:] == 5).all()
    assert (ws[:256] == 9).all() and (ws[256 + need:] == 9).all()
    assert torch.equal(fw.embedding_backward(idx, d, V)["table"], g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, r = fw.embedding(idx, table)["out"], fw.embedding_backward(idx, d, V)["table"]
    idx.copy_(indices(T, V, "even", 5))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, fw.embedding(idx, table)["out"]) and torch.equal(r, fw.embedding_backward(idx, d, V)["table"])


def test_output_beyond_32_bit_offsets():
    import protein_structure_models_b200 as fw
    T, V, C = 2 ** 21 + 5, 3, 1024
    idx = indices(T, V, "even")
    out = fw.embedding(idx, rnd((V, C), torch.bfloat16, 1).clone())["out"]
    table = rnd((V, C), torch.bfloat16, 1)
    for rows in (slice(0, 64), slice(T - 64, T), slice(2 ** 20, 2 ** 20 + 64)):
        assert torch.equal(out[rows], table[idx[rows].long()])
    g = fw.embedding_backward(idx, torch.ones_like(out), V)["table"]
    n = torch.bincount(idx.long(), minlength=V).float()
    assert torch.equal(g, n[:, None].expand(V, C))          # whole numbers below 2^24: exact


def test_refusals():
    import protein_structure_models_b200 as fw
    from protein_structure_models_b200 import FipaError
    idx, table = indices(5, 4, "even"), rnd((4, 8), torch.float32, 0)
    for a in ((idx.long(), table), (idx, table.half()), (idx.cpu(), table), (idx, table.t())):
        with pytest.raises(ValueError):
            fw.embedding(*a)
    with pytest.raises(FipaError) as e:
        fw.embedding(idx, table, scale=float("inf"))
    assert e.value.status == 1
    d = torch.ones(5, 8, device="cuda")
    with pytest.raises(ValueError):
        fw.embedding_backward(idx[:4], d, 4)
    with pytest.raises(FipaError) as e:
        fw.embedding_backward(idx, d, 4, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 3
    for bad in ((5, 0, 8), (2 ** 30 + 1, 4, 8), (5, 4, 70000)):
        with pytest.raises(FipaError):
            fw.embedding_backward_workspace_size(*bad)
