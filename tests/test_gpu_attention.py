"""Differential attention, distance bias and dropout on the GPU against the 64-bit oracle (needs an MI355X).

Every element has its own tolerance: the oracle's first-order roundoff bound
for 32-bit arithmetic, plus half a step of the storage type where an output is
rounded to it, plus 2% for the higher orders.
"""
import ctypes as ct
import dataclasses

import numpy as np
import pytest
import torch

import synth
from oracle import attention as oa
from tests.helpers import grid_box

pytestmark = pytest.mark.gpu

eg = pytest.importorskip("equivariant_gnn_electronic_amd")
from equivariant_gnn_electronic_amd import _lib  # noqa: E402

SEED, STEP, SITE = 0x1234_5678_9ABC_DEF1, 42, 9


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def rng_state(dev, step=STEP):
    return torch.tensor([SEED, step], dtype=torch.int64, device=dev)


def within(got, want, bound, store, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    half = 0.0 if store is None else torch.finfo(store).eps / 2
    tol = 1.02 * (bound + half * (np.abs(want) + bound)) + 1e-37
    assert got.shape == want.shape, what
    over = np.abs(got - want) > tol
    assert not np.any(over) and np.all(np.isfinite(got)), (
        f"{what}: {int(over.sum())} of {over.size} beyond the bound, worst {np.max(np.abs(got - want) / tol):.3g} of it")


@dataclasses.dataclass
class Case:
    degrees: tuple
    n_src: int
    lmax: int
    C: int
    H: int
    D: int
    dtype: str = "f32"
    bias: bool = True
    mask: bool = False
    p: float = 0.0


def varied(seed, n, mean):
    rng = np.random.default_rng(seed)
    return tuple(int(x) for x in rng.integers(0, 2 * mean + 1, n))


CASES = {
    "one_edge": Case((1,), 1, 0, 1, 1, 1),
    "no_edges": Case((0, 0, 0), 2, 1, 4, 2, 4),
    "cell": Case(varied(1, 20, 12), 24, 2, 8, 2, 8),
    "empty_rows": Case((0, 3, 0, 1, 64, 0), 9, 1, 16, 4, 4, mask=True),
    "invariants": Case(varied(2, 30, 20), 30, 0, 64, 8, 16, mask=True, p=0.1),
    "hfo2_shape": Case(varied(3, 12, 90), 40, 4, 64, 8, 16, p=0.1),
    "gst_shape": Case(varied(4, 10, 70), 30, 4, 128, 8, 32, "bf16", mask=True, p=0.2),
    "odd": Case(varied(5, 15, 20), 17, 3, 30, 3, 10, mask=True, p=0.25),
    "odd_bf16": Case(varied(6, 15, 20), 17, 2, 21, 7, 5, "bf16", mask=True, p=0.5),
    "one_head_wide": Case(varied(7, 6, 30), 11, 1, 256, 1, 256),
    "many_heads": Case(varied(8, 6, 40), 11, 1, 64, 32, 4, p=0.3),
    "many_heads_bf16": Case(varied(9, 6, 40), 11, 0, 256, 32, 64, "bf16"),
    "degree8": Case(varied(10, 5, 10), 7, 8, 24, 3, 8),
    # rows beyond every block limit (64 edges with 32 heads, 256 with 8, 512 with 2), some cut at a window's border
    "readout": Case((1500,), 300, 1, 16, 8, 8, "bf16", bias=False),
    "long_rows": Case((5, 512, 1024, 3, 700, 0, 256, 1), 90, 1, 16, 8, 8, mask=True, p=0.1),
    "long_rows_many_heads": Case((64, 65, 130, 2, 300), 40, 0, 64, 32, 4, p=0.1),
    "long_rows_two_maps": Case((513, 1, 1100), 50, 2, 6, 1, 3),
    # a small graph is not cut: one block walks its long row in steps
    "steps_in_a_row": Case((700, 3, 0, 300) + (20,) * 36, 60, 1, 16, 8, 8, p=0.2),
    "steps_in_a_row_bf16": Case((900,) + (15,) * 40, 60, 2, 32, 4, 8, "bf16", mask=True),
    # many rows: cut at 4,096 edges only, so blocks take steps and pieces are joined
    "many_rows_and_a_long_one": Case((3,) * 500 + (9000,) + (2, 0, 5) * 200, 300, 0, 8, 2, 4, p=0.1),
    # long rows next to each other, several of them joined by one block
    "neighbouring_long_rows": Case((3,) * 600 + (4200, 4100, 1, 4300) + (2,) * 700, 9, 1, 16, 4, 8, p=0.1),
    # some hundred rows of several steps each, and a few that are cut at 512 edges
    "some_hundred_rows": Case((300,) * 258 + (900, 513), 50, 0, 16, 16, 4, p=0.1),
    # few rows of many edges: pieces longer than the shortest, none left over at the end
    "few_rows_of_many_edges": Case((140_000, 1), 50, 0, 2, 1, 2),
    # long component-free rows: slices that meet a few heads each
    "wide_invariants": Case(varied(12, 9, 20), 15, 0, 1024, 16, 128, p=0.1),
    "wide_invariants_bf16": Case(varied(13, 9, 20), 15, 0, 1024, 32, 64, "bf16"),
    # vectors that hold several heads, more than 16 of them
    "mixed_heads": Case(varied(14, 8, 30), 20, 1, 64, 32, 2, p=0.1),
    "mixed_heads_bf16": Case(varied(15, 8, 30), 20, 3, 48, 16, 4, "bf16", mask=True),
    # half vectors
    "pairs": Case(varied(16, 8, 30), 20, 2, 36, 6, 6),
    "quads_bf16": Case(varied(17, 8, 30), 20, 2, 32, 8, 4, "bf16"),
    # one source in every edge: the backward's long rows
    "one_source": Case(varied(11, 40, 60), 1, 1, 16, 2, 8, p=0.1),
}


def make(case, dev, seed=5):
    g = torch.Generator().manual_seed(seed)
    E, K = sum(case.degrees), (case.lmax + 1) ** 2
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[case.dtype]
    n_dst = len(case.degrees)
    t = dict(row_ptr=torch.tensor([0, *np.cumsum(case.degrees)], dtype=torch.int32),
             src=torch.randint(case.n_src, (E,), generator=g).int(),
             q=torch.randn(n_dst, case.H, 2, case.D, generator=g).to(dt),
             k=torch.randn(case.n_src, case.H, 2, case.D, generator=g).to(dt),
             v=torch.randn(case.n_src, K, case.C, generator=g).to(dt),
             lam=torch.rand(case.H, generator=g) * 0.6 + 0.2,
             bias=torch.randn(E, 2 * case.H, generator=g) if case.bias else None,
             mask=(torch.rand(E, generator=g) > 0.2).to(torch.uint8) if case.mask else None,
             grad_out=torch.randn(n_dst, K, case.C, generator=g))
    d = {n: None if x is None else x.to(dev) for n, x in t.items()}
    d["graph"] = eg.Graph.from_csr(d["row_ptr"], d["src"], n_src=case.n_src, group=True)
    d["desc"] = eg.attn_desc(case.lmax, case.C, case.H, case.D, drop_p=case.p, site=SITE,
                             storage=eg.EGNN_BF16 if case.dtype == "bf16" else eg.EGNN_F32)
    d["rng"] = rng_state(dev) if case.p else None
    d["dt"] = dt
    return d


def host(t):
    return None if t is None else (t.float() if t.dtype == torch.bfloat16 else t).cpu().numpy()


def oracle_of(case, d, grad=True, **over):
    E = sum(case.degrees)
    factors = oa.keep_factors(np.arange(E * case.H).reshape(E, case.H), case.p, SEED, STEP, SITE) if case.p else None
    a = {n: over.get(n, host(d[n])) for n in ("row_ptr", "src", "q", "k", "v", "lam", "bias", "mask")}
    return oa.attention_bounds(**a, scale=float(np.float32(case.D ** -0.5)), factors=factors,
                               grad_out=host(d["grad_out"]) if grad else None)


def forward(d, **kw):
    return eg.egnn_diff_attention_fwd(d["desc"], d["graph"], d["q"], d["k"], d["v"], d["lam"], bias=d["bias"],
                                      mask=d["mask"], rng=d["rng"], **kw)


NAMES = ("grad_q", "grad_k", "grad_v", "grad_lam", "grad_bias")


def backward(d, buf):
    return dict(zip(NAMES, eg.egnn_diff_attention_bwd(d["desc"], d["graph"], d["q"], d["k"], d["v"], d["lam"], buf,
                                                      d["grad_out"], rng=d["rng"])))


@pytest.mark.parametrize("name", list(CASES))
def test_attention_forward_backward(dev, name):
    print(f"[attention] {name}", flush=True)
    case = CASES[name]
    d = make(case, dev)
    infer, _ = forward(d)
    buf = eg.AttnBuffers(d["desc"], d["graph"])
    out, _ = forward(d, buffers=buf)
    got = backward(d, buf)
    torch.cuda.synchronize()
    res, bnd = oracle_of(case, d)
    within(host(out), res["out"], bnd["out"], d["dt"], "out")
    assert torch.equal(infer, out)
    for n in NAMES:
        within(host(got[n]), res[n], bnd[n], None, n)
    # again on the same buffers: bit-identical
    out2, _ = forward(d, buffers=buf)
    again = backward(d, buf)
    assert torch.equal(out, out2) and all(torch.equal(got[n], again[n]) for n in NAMES)


@pytest.mark.parametrize("name", ["cell", "gst_shape", "odd"])
def test_attention_gradients_against_differences(dev, name):
    """<grad, direction> against the forward's central difference in 64 bits (the oracle's forward), and the GPU's own
    forward moved the same way: the gradient is that of what the forward computes."""
    case = CASES[name]
    d = make(case, dev)
    buf = eg.AttnBuffers(d["desc"], d["graph"])
    forward(d, buffers=buf)
    got = backward(d, buf)
    rng = np.random.default_rng(3)
    h = 1e-5
    for n in ("q", "k", "v", "lam", "bias"):
        if d[n] is None:
            continue
        base = host(d[n]).astype(np.float64)
        dirn = rng.standard_normal(base.shape)
        G = host(d["grad_out"]).astype(np.float64)
        up, dn = (np.sum(oracle_of(case, d, grad=False, **{n: base + s * h * dirn})[0]["out"] * G) for s in (1, -1))
        res, bnd = oracle_of(case, d)
        want = (up - dn) / (2 * h)
        g = host(got["grad_" + n]).astype(np.float64).reshape(base.shape)
        # the gradient's own bound along the direction, and the difference's error (third order, and 64-bit rounding)
        tol = 1.02 * np.sum(bnd["grad_" + n].reshape(base.shape) * np.abs(dirn)) + 1e-6 * np.abs(want) + 1e-5
        assert abs(np.sum(g * dirn) - want) <= tol, (n, np.sum(g * dirn), want, tol)


@pytest.mark.parametrize("name", ["empty_rows", "long_rows"])
def test_masked_places_may_hold_anything(dev, name):
    """NaN and infinities in the keys, values and biases of edges that take no part leave every output as it is."""
    case = CASES[name]
    d = make(case, dev)
    E = sum(case.degrees)
    # source 0 is poisoned and all its edges are masked
    gone = d["src"] == 0
    d["mask"][gone] = 0
    buf = eg.AttnBuffers(d["desc"], d["graph"])
    clean, _ = forward(d, buffers=buf)
    clean_g = backward(d, buf)
    d["k"][0], d["v"][0] = float("nan"), float("inf")
    d["bias"][gone] = float("nan")
    out, _ = forward(d, buffers=buf)
    g = backward(d, buf)
    assert torch.equal(out, clean)
    assert all(torch.equal(g[n], clean_g[n]) for n in NAMES)
    # masked by a bias of -inf instead: the same
    d["mask"] = torch.ones(E, dtype=torch.uint8, device=dev) if d["mask"] is None else d["mask"]
    keep = d["mask"].clone()
    d["mask"] = None
    d["bias"][keep == 0] = float("-inf")
    out, _ = forward(d, buffers=buf)
    g = backward(d, buf)
    assert torch.equal(out, clean)
    assert all(torch.equal(g[n], clean_g[n]) for n in NAMES)
    # and by a source outside the list
    d["mask"] = keep
    d["src"][gone] = torch.where(torch.arange(int(gone.sum()), device=dev) % 2 == 0, -1, case.n_src).int()
    out, _ = forward(d, buffers=buf)
    assert torch.equal(out, clean)


def test_lowest_bias_is_a_number_not_a_mask(dev):
    """A row whose every bias is the type's lowest value is still a softmax: its products drown, so it is uniform; beside
    ordinary entries the lowest ones vanish."""
    case = dataclasses.replace(CASES["cell"], p=0.0)
    d = make(case, dev)
    low = torch.finfo(torch.float32).min
    ptr = d["row_ptr"].cpu().numpy()
    r = int(np.argmax(case.degrees))
    d["bias"][ptr[r]:ptr[r + 1]] = low
    d["bias"][0] = low
    out, _ = forward(d)
    res, bnd = oracle_of(case, d)
    n = ptr[r + 1] - ptr[r]
    v = host(d["v"]).astype(np.float64)[host(d["src"])[ptr[r]:ptr[r + 1]]]
    w = np.repeat(1.0 - host(d["lam"]).astype(np.float64), case.C // case.H)
    # uniform weights: (1 - lam)/n, each sum of n terms in fp32
    tol = (n + 12) * oa.U32 * (1 + np.repeat(host(d["lam"]), case.C // case.H)) * np.abs(v).mean(0)
    assert np.all(np.abs(host(out)[r] - w * v.mean(0)) <= 1.02 * tol)
    others = [i for i in range(len(case.degrees)) if i != r and not (ptr[i] == 0 and ptr[i + 1] > 0)]
    within(host(out)[others], res["out"][others], bnd["out"][others], None, "other rows")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strided_and_unaligned_rows(dev, dtype):
    """q, k, v as parts of one projection give the packed results bit for bit; at an odd offset (single elements
    instead of vectors) they stay inside the bound."""
    case = dataclasses.replace(CASES["hfo2_shape"], degrees=varied(3, 40, 25), dtype=dtype, lmax=0)
    d = make(case, dev)
    buf = eg.AttnBuffers(d["desc"], d["graph"])
    out, _ = forward(d, buffers=buf)
    got = backward(d, buf)
    H, D, C, n = case.H, case.D, case.C, case.n_src
    res, bnd = oracle_of(case, d)
    for shift in (0, 1):
        wide = torch.full((n, 4 * H * D + C + 8), float("nan"), dtype=d["dt"], device=dev)
        o = shift
        parts = {}
        for name, width in (("q", 2 * H * D), ("k", 2 * H * D), ("v", C)):
            wide[:, o:o + width] = d[name].reshape(n, width)
            parts[name] = wide[:, o:o + width].view(d[name].shape)
            o += width
        e = dict(d, **parts)
        out2, _ = forward(e, buffers=buf)
        got2 = backward(e, buf)
        if shift == 0:
            assert torch.equal(out, out2) and all(torch.equal(got[m], got2[m]) for m in NAMES)
        within(host(out2), res["out"], bnd["out"], d["dt"], "out")
        for m in NAMES:
            within(host(got2[m]), res[m], bnd[m], None, m)


def test_offsets_beyond_32_bits(dev):
    """Rows 2^27 elements apart (an array of more than 4 GB): bit-identical to packed rows."""
    case = dataclasses.replace(CASES["cell"], degrees=varied(1, 12, 12), n_src=12, lmax=0, C=16)
    d = make(case, dev)
    buf = eg.AttnBuffers(d["desc"], d["graph"])
    out, _ = forward(d, buffers=buf)
    got = backward(d, buf)
    far = {}
    for n in ("q", "k", "v"):
        rows, width = d[n].shape[0], d[n][0].numel()
        a = torch.empty((rows - 1) * 2**27 + width, device=dev).as_strided((rows, width), (2**27, 1))
        a.copy_(d[n].view(rows, width))
        far[n] = a.as_strided(d[n].shape, (2**27, *d[n].stride()[1:]))
    e = dict(d, **far)
    out2, _ = forward(e, buffers=buf)
    got2 = backward(e, buf)
    assert torch.equal(out, out2) and all(torch.equal(got[m], got2[m]) for m in NAMES)


def test_unsorted_sources_and_doubled_edges(dev):
    """Sources in any order and the same edge twice: the graph need only be grouped by destination."""
    case = dataclasses.replace(CASES["hfo2_shape"], degrees=(90, 150, 200, 40) * 8, n_src=300)
    d = make(case, dev)
    d["src"][5:9] = d["src"][4]
    d["graph"] = eg.Graph.from_csr(d["row_ptr"], d["src"], n_src=case.n_src, group=True)
    buf = eg.AttnBuffers(d["desc"], d["graph"])
    out, _ = forward(d, buffers=buf)
    got = backward(d, buf)
    res, bnd = oracle_of(case, d)
    within(host(out), res["out"], bnd["out"], d["dt"], "out")
    for n in NAMES:
        within(host(got[n]), res[n], bnd[n], None, n)


def test_no_edges_without_operands(dev):
    """A graph without edges through the C ABI with every operand NULL that the header lets be: gradients of zero."""
    g = _lib.EgnnGraph()
    ptr = torch.zeros(4, dtype=torch.int32, device=dev)
    g.n_dst, g.n_src, g.n_edges = 3, 3, 0
    g.row_ptr = g.src_ptr = ptr.data_ptr()
    d = eg.attn_desc(1, 8, 2, 4)
    s, i, t = (ct.c_size_t() for _ in range(3))
    lib = _lib.load()
    assert lib.egnn_diff_attention_sizes(ct.byref(d), ct.byref(g), ct.byref(s), ct.byref(i), ct.byref(t)) == 0
    ws = torch.empty(max(i.value, t.value, 1), dtype=torch.uint8, device=dev)
    outs = [torch.full(sh, 9.0, device=dev) for sh in ((3, 4, 8), (3, 2, 2, 4), (3, 2, 2, 4), (3, 4, 8), (2,))]
    st = ct.c_void_p(torch.cuda.current_stream().cuda_stream)
    p = lambda x: ct.c_void_p(x.data_ptr())  # noqa: E731
    assert lib.egnn_diff_attention_fwd(ct.byref(d), ct.byref(g), None, None, None, None, None, None, None, p(outs[0]),
                                       None, p(ws), ws.numel(), st) == 0
    assert lib.egnn_diff_attention_bwd(ct.byref(d), ct.byref(g), None, None, None, None, None, None, None,
                                       *map(p, outs[1:]), None, p(ws), ws.numel(), st) == 0
    torch.cuda.synchronize()
    assert all(bool((o == 0).all()) for o in outs)


def test_rows_of_a_longer_array(dev):
    """q, k and v may hold more rows than the graph; out behind the last row stays as it was."""
    case = CASES["cell"]
    d = make(case, dev)
    out, _ = forward(d)
    longer = {n: torch.cat([d[n], torch.full_like(d[n][:3], float("nan"))]) for n in ("q", "k", "v")}
    room = torch.full((out.shape[0] + 2, *out.shape[1:]), 7.0, dtype=out.dtype, device=dev)
    out2, _ = forward(dict(d, **longer), out=room[:out.shape[0]])
    assert torch.equal(out, out2) and bool((room[out.shape[0]:] == 7.0).all())


GUARD = 1 << 16


@pytest.mark.parametrize("name", ["cell", "odd", "long_rows", "gst_shape", "many_heads", "no_edges"])
def test_nothing_is_written_outside_the_buffers(dev, name):
    case = CASES[name]
    d = make(case, dev)
    desc, g = d["desc"], d["graph"]
    saved, infer, train = eg.egnn_diff_attention_sizes(desc, g)
    raws = []

    def guarded(nbytes):
        raw = torch.full((2 * GUARD + max(nbytes, 16),), 0xA5, dtype=torch.uint8, device=dev)
        raws.append((raw, nbytes))
        return ct.c_void_p(raw.data_ptr() + GUARD)

    p = lambda t: None if t is None else ct.c_void_p(t.data_ptr())  # noqa: E731
    n_dst, n_src, E, K = g.n_dst, g.n_src, g.n_edges, (case.lmax + 1) ** 2
    size = 2 if case.dtype == "bf16" else 4
    gs, lib = g.c_struct(), _lib.load()
    st = ct.c_void_p(torch.cuda.current_stream().cuda_stream)
    ins = (p(d["q"]), p(d["k"]), p(d["v"]), p(d["lam"]))
    for keep in (None, guarded(saved)):
        n = infer if keep is None else train
        assert lib.egnn_diff_attention_fwd(ct.byref(desc), ct.byref(gs), *ins, p(d["bias"]), p(d["mask"]), p(d["rng"]),
                                           guarded(n_dst * K * case.C * size), keep, guarded(n), n, st) == 0
    outs = [guarded(4 * n) for n in (2 * n_dst * case.H * case.D, 2 * n_src * case.H * case.D, n_src * K * case.C,
                                     case.H, 2 * E * case.H)]
    assert lib.egnn_diff_attention_bwd(ct.byref(desc), ct.byref(gs), *ins, p(d["rng"]), keep, p(d["grad_out"]), *outs,
                                       guarded(train), train, st) == 0
    torch.cuda.synchronize()
    for raw, n in raws:
        assert bool((raw[:GUARD] == 0xA5).all()) and bool((raw[GUARD + n:] == 0xA5).all())


def test_other_stream_and_captured_step(dev):
    """A training step on a side stream, then captured and replayed with new steps of the generator: every replay equals
    the eager result of its step."""
    case = dataclasses.replace(CASES["hfo2_shape"], degrees=varied(3, 30, 30))
    d = make(case, dev)
    buf = eg.AttnBuffers(d["desc"], d["graph"])
    drop = eg.dropout_desc(case.lmax, case.C, 0.3, share="degree", site=4)
    table = torch.randn(8, 2 * case.H, device=dev)
    d["graph"].dist = torch.rand(sum(case.degrees), device=dev) * 8
    borders = eg.egnn_distance_borders(8, 4, 4.0, 8.0).to(dev)

    def step():
        d["bias"] = eg.egnn_distance_bias_fwd(d["graph"], borders, table)
        out, _ = forward(d, buffers=buf)
        y = eg.egnn_dropout_fwd(drop, out, d["rng"], residual=out)
        g = backward(dict(d, grad_out=eg.egnn_dropout_bwd(drop, d["grad_out"], d["rng"])), buf)
        gt = eg.egnn_distance_bias_bwd(d["graph"], borders, g["grad_bias"])
        return [y, gt, *(g[n] for n in NAMES)]

    eager = {}
    for s in (1, 2, 3):
        d["rng"].copy_(rng_state(dev, s))
        eager[s] = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        on_side = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(on_side, eager[3]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for s in (2, 1, 3, 2):
        d["rng"].copy_(rng_state(dev, s))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, eager[s])), s
    assert not torch.equal(eager[1][0], eager[2][0])


def test_block_of_a_network(dev):
    """Bias, attention, dropout with a residual and the SO(2) layer in a row on a built graph, and back, against the oracle
    chained the same way."""
    from oracle import layer as olayer
    from oracle import neighbors as onb
    cfg = synth.CONFIGS["tiny_l4"]
    s = synth.make_structure(cfg)
    lo, box = grid_box(s)
    g = eg.egnn_build_graph(torch.from_numpy(s.pos).to(dev), s.n_dst, lo, box, s.periodic_mask, s.r_cut)
    x, ws = synth.make_layer_inputs(cfg)
    H, D, C, K, N, p = 2, 4, cfg.C, cfg.K, s.n_dst, 0.25
    rng = np.random.default_rng(6)
    q, k = (rng.standard_normal((N, H, 2, D)).astype(np.float32) for _ in range(2))
    lam = np.asarray([0.3, 0.6], np.float32)
    table = rng.standard_normal((12, 2 * H)).astype(np.float32)
    G = synth.make_cotangent(cfg, N)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    borders = eg.egnn_distance_borders(12, 6, 2.5, 5.0)
    state = rng_state(dev)
    ad = eg.attn_desc(cfg.lmax, C, H, D, drop_p=p, site=1)
    dd = eg.dropout_desc(cfg.lmax, C, p, share="degree", site=2)
    ld = eg.layer_desc(cfg.lmax, cfg.mmax, C, cfg.n_rbf, cfg.r_cut)
    xt, w = up(x), up(ws[0])
    geom = eg.egnn_edge_geom(ld, g)
    bias = eg.egnn_distance_bias_fwd(g, borders.to(dev), up(table))
    att, buf = eg.egnn_diff_attention_fwd(ad, g, up(q), up(k), xt, up(lam), bias=bias, rng=state,
                                          buffers=eg.AttnBuffers(ad, g))
    y = eg.egnn_dropout_fwd(dd, att, state, residual=xt)
    lb = eg.LayerBuffers(ld, g)
    (z, _), lb = eg.egnn_layer_fwd(ld, g, geom, w, y, buffers=lb)
    gy, gw = eg.egnn_layer_bwd(ld, g, geom, w, y, lb, up(G))
    ga = eg.egnn_dropout_bwd(dd, gy, state)
    gq, gk, gv, gl, gb = eg.egnn_diff_attention_bwd(ad, g, up(q), up(k), xt, up(lam), buf, ga, rng=state)
    gt = eg.egnn_distance_bias_bwd(g, borders.to(dev), gb)
    gx = gv + gy
    torch.cuda.synchronize()

    og = onb.build_graph(s.pos, N, s.box, s.periodic_mask, s.r_cut)
    E = len(og["src"])
    dist = g.dist.cpu().numpy()
    f_att = oa.keep_factors(np.arange(E * H).reshape(E, H), p, SEED, STEP, 1)
    f_drop = oa.dropout_factors(N, cfg.lmax, C, "degree", p, SEED, STEP, 2)
    obias = oa.bias_forward(dist, borders.numpy(), table)
    args = dict(row_ptr=og["row_ptr"], src=og["src"], q=q, k=k, v=x, lam=lam, scale=D ** -0.5, bias=obias, factors=f_att)
    oy = x.astype(np.float64) + f_drop * oa.attention_forward(**args)
    od = olayer.LayerDesc(cfg.lmax, cfg.mmax, C, cfg.n_rbf, cfg.r_cut)
    w64 = ws[0].astype(np.float64)
    fwd = olayer.layer_forward(og, oy, w64, od)
    dy, dw = olayer.layer_backward(og, oy, w64, od, fwd, G.astype(np.float64))
    res, _ = oa.attention_bounds(**args, grad_out=f_drop * dy)

    def rel(a, b):
        return np.linalg.norm(host(a).astype(np.float64) - b) / np.linalg.norm(b)

    # the layer's own parity tolerance carries through the chain
    for name, a, b in (("z", z, fwd["x_out"]), ("gw", gw, dw), ("gq", gq, res["grad_q"]), ("gk", gk, res["grad_k"]),
                       ("gx", gx, res["grad_v"] + dy), ("gl", gl, res["grad_lam"]),
                       ("gt", gt, oa.bias_backward(dist, borders.numpy(), res["grad_bias"]))):
        assert rel(a, b) <= 1e-4, (name, rel(a, b))


# ---------------------------------------------------------------------- bias

@pytest.mark.parametrize("E,B,M", [(1, 1, 1), (63, 2, 1), (64, 33, 6), (1000, 32, 16), (4097, 1024, 64), (777, 512, 32),
                                   (5000, 7, 64), (300, 64, 24), (2500, 100, 63)])
def test_distance_bias(dev, E, B, M):
    print(f"[bias] {E} {B} {M}", flush=True)
    g = torch.Generator().manual_seed(E + B)
    borders = eg.egnn_distance_borders(B, max(1, B // 2), 4.0, 8.0)
    dist = torch.rand(E, generator=g) * 10
    if B > 1:  # values on a border, beyond the last, and no number at all
        n = min(E, B - 1)
        dist[:n] = borders[:n]
    dist[-1] = float("nan")
    table, G = torch.randn(B, M, generator=g), torch.randn(E, M, generator=g)
    graph = eg.Graph.from_csr(torch.tensor([0, E], dtype=torch.int32, device=dev),
                              torch.zeros(E, dtype=torch.int32, device=dev))
    graph.dist = dist.to(dev)
    out = eg.egnn_distance_bias_fwd(graph, borders.to(dev), table.to(dev))
    gt = eg.egnn_distance_bias_bwd(graph, borders.to(dev), G.to(dev))
    b = oa.buckets(dist.numpy(), borders.numpy())
    assert torch.equal(out.cpu(), table[torch.from_numpy(b)])
    want = oa.bias_backward(dist.numpy(), borders.numpy(), G.numpy())
    # a sum of n terms in any order: (n - 1) roundings of partial sums, each at most the sum of magnitudes
    mag = oa.bias_backward(dist.numpy(), borders.numpy(), G.abs().numpy())
    n = np.bincount(b, minlength=B)[:, None]
    within(gt.cpu().numpy(), want, n * oa.U32 * mag, None, "grad_table")
    assert torch.equal(gt, eg.egnn_distance_bias_bwd(graph, borders.to(dev), G.to(dev)))


@pytest.mark.parametrize("E,B,M", [(1_000_003, 20, 1), (1_000_003, 20, 2), (600_007, 40, 5), (600_007, 64, 9),
                                   (600_007, 48, 12), (400_013, 500, 16)])
def test_distance_bias_gradient_over_many_chunks(dev, E, B, M):
    """Every round size of the gradient, waves that take several chunks, the last of them ragged."""
    print(f"[bias gradient] {E} {B} {M}", flush=True)
    g = torch.Generator().manual_seed(M)
    borders = eg.egnn_distance_borders(B, B // 2, 4.0, 8.0)
    dist, G = torch.rand(E, generator=g) * 10, torch.randn(E, M, generator=g)
    graph = eg.Graph.from_csr(torch.tensor([0, E], dtype=torch.int32, device=dev),
                              torch.zeros(E, dtype=torch.int32, device=dev))
    graph.dist = dist.to(dev)
    gt = eg.egnn_distance_bias_bwd(graph, borders.to(dev), G.to(dev))
    b = oa.buckets(dist.numpy(), borders.numpy())
    n = np.bincount(b, minlength=B)[:, None]
    sums = [np.stack([np.bincount(b, t[:, c].double().numpy(), B) for c in range(M)], 1) for t in (G, G.abs())]
    # a sum of n terms in any order: (n - 1) roundings of partial sums, each at most the sum of magnitudes
    within(gt.cpu().numpy(), sums[0], n * oa.U32 * sums[1], None, "grad_table")
    assert torch.equal(gt, eg.egnn_distance_bias_bwd(graph, borders.to(dev), G.to(dev)))
    # integers add without rounding: an edge lost or counted twice shows
    ones = torch.ones(E, M, device=dev)
    assert np.array_equal(eg.egnn_distance_bias_bwd(graph, borders.to(dev), ones).cpu().numpy(),
                          np.broadcast_to(n.astype(np.float32), (B, M)))
    # what is not a number stays in its bucket
    ones[E // 2] = float("nan")
    bad = torch.isnan(eg.egnn_distance_bias_bwd(graph, borders.to(dev), ones)).cpu().numpy()
    assert bad[b[E // 2]].all() and bad.sum() == M


def test_distance_bias_without_edges(dev):
    graph = eg.Graph.from_csr(torch.zeros(2, dtype=torch.int32, device=dev), torch.zeros(0, dtype=torch.int32, device=dev))
    graph.dist = torch.zeros(0, device=dev)
    borders = eg.egnn_distance_borders(4, 2, 1.0, 2.0).to(dev)
    assert eg.egnn_distance_bias_fwd(graph, borders, torch.ones(4, 3, device=dev)).shape == (0, 3)
    assert bool((eg.egnn_distance_bias_bwd(graph, borders, torch.zeros(0, 3, device=dev)) == 0).all())


# ------------------------------------------------------------------- dropout

@pytest.mark.parametrize("share", ["channel", "degree", "row"])
@pytest.mark.parametrize("rows,lmax,C", [(1, 0, 1), (5, 0, 190), (70, 0, 64), (9, 1, 7), (33, 2, 8), (21, 3, 50),
                                         (13, 4, 128), (4, 5, 16), (6, 6, 64), (3, 7, 24), (2, 8, 40),
                                         (100, 0, 3), (50, 0, 1), (41, 0, 13), (9, 5, 10), (3, 7, 9), (2, 8, 41)])
def test_dropout(dev, rows, lmax, C, share):
    print(f"[dropout] {rows} {lmax} {C} {share}", flush=True)
    gen = torch.Generator().manual_seed(rows + C)
    K, p = (lmax + 1) ** 2, 0.3
    x, r = torch.randn(rows, K, C, generator=gen), torch.randn(rows, K, C, generator=gen)
    f = oa.dropout_factors(rows, lmax, C, share, p, SEED, STEP, SITE)
    state = rng_state(dev)
    for dt, storage in ((torch.float32, eg.EGNN_F32), (torch.bfloat16, eg.EGNN_BF16)):
        desc = eg.dropout_desc(lmax, C, p, share=share, site=SITE, storage=storage)
        xs, rs = x.to(dt), r.to(dt)
        want = xs.double().numpy() * f
        y = eg.egnn_dropout_fwd(desc, xs.to(dev), state)
        # the factor is rounded to fp32, then the product, then storage
        within(host(y), want, 2 * oa.U32 * np.abs(want), dt, "y")
        assert bool(((y == 0).cpu() == torch.from_numpy(f == 0)).all())
        yr = eg.egnn_dropout_fwd(desc, xs.to(dev), state, residual=rs.to(dev))
        sum_ = rs.double().numpy() + want
        within(host(yr), sum_, oa.U32 * (np.abs(want) + np.abs(sum_)) + oa.U32 * np.abs(want), dt, "y + residual")
        inplace = xs.to(dev)
        eg.egnn_dropout_fwd(desc, inplace, state, residual=rs.to(dev), out=inplace)
        assert torch.equal(inplace, yr)
        # bytes at an odd element: single elements instead of vectors, the same values
        wide = torch.empty(x.numel() + 1, dtype=dt, device=dev)[1:].view(x.shape)
        wide.copy_(xs)
        assert torch.equal(eg.egnn_dropout_fwd(desc, wide, state), y)
        gx = eg.egnn_dropout_bwd(desc, x.to(dev), state)
        within(host(gx), x.double().numpy() * f, 2 * oa.U32 * np.abs(x.double().numpy() * f), None, "grad_x")


def test_dropout_hides_dropped_values_and_passes_others(dev):
    desc = eg.dropout_desc(0, 64, 0.5, site=SITE)
    f = oa.dropout_factors(8, 0, 64, "channel", 0.5, SEED, STEP, SITE)
    x = torch.ones(8, 1, 64)
    x[torch.from_numpy(f == 0)] = float("nan")
    r = torch.full_like(x, 3.0)
    y = eg.egnn_dropout_fwd(desc, x.to(dev), rng_state(dev), residual=r.to(dev)).cpu().numpy()
    assert np.array_equal(y, np.where(f == 0, 3.0, 5.0))
    keep = eg.dropout_desc(2, 5, 0.0)
    z = torch.randn(3, 9, 5, device=dev)
    assert torch.equal(eg.egnn_dropout_fwd(keep, z, None), z) and torch.equal(eg.egnn_dropout_bwd(keep, z, None), z)
