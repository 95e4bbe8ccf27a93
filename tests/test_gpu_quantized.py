"""Rows to 8-bit integers and products of 8-bit integers against their definitions in 64 bits.

Tolerances.  Whole numbers are compared for equality: the fp64 quotient 127 x / a rounds as the exact
one does (254 |x| and (2 q + 1) a are integers below 2^32 times one power of two, so a quotient that
is no tie is more than 2^-26 from one, against fp64's 2^-47 here).  A product's sum is exact; its
conversion to fp32 and its two scales round three times (a relative 2^-24 each), the last rounding
is Y's type's half step (and half its smallest subnormal)."""

from fractions import Fraction

import numpy as np
import pytest
import torch

import expanded_rank_matrix_amd as erm

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def quantized(x):
    """(q, scale) of a matrix by the definition, on the CPU in 64 bits."""
    x = x.cpu().double()
    a = x.abs().amax(1)
    q = torch.round(x * 127 / torch.where(a > 0, a, torch.ones_like(a))[:, None])
    return q.to(torch.int8), (a / 127).float()


def close(y, want, dtype):
    """y (of dtype) within the tolerance above of the 64-bit values."""
    f = torch.finfo(dtype)
    tol = want.abs() * (3.01 * 2.0**-24 + (f.eps / 2 if dtype != torch.float32 else 0)) + f.smallest_normal * f.eps / 2
    off = (y.cpu().double() - want).abs()
    assert not (off > tol).any(), f"worst {float((off / tol).max()):.3g} of the tolerance"


def rand(rows, n, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((rows, n), generator=g) * scale).to(dtype)


def rand_i8(rows, n, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-128, 128, (rows, n), generator=g, dtype=torch.int8)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,n", [(1, 1), (3, 7), (5, 64), (4, 1000), (9, 1024), (2, 1025), (7, 2560), (3, 9728),
                                    (2, 10240), (2, 10241), (1, 40000), (1027, 33), (6, 8), (5, 9), (6, 15),
                                    (3, 4096), (3, 4097), (2, 4104)])
def test_quantize_matches_definition(rows, n, dtype):
    x = rand(rows, n, TYPES[dtype], 17 + rows + n)
    q, s = erm.quantize_rows(x.cuda())
    wq, ws = quantized(x)
    assert torch.equal(q.cpu(), wq)
    assert torch.equal(s.cpu(), ws)


def test_quantize_borders_are_exact():
    """Values next to and on the borders between two whole numbers, checked in whole numbers."""
    rng = np.random.default_rng(5)
    rows = []
    for _ in range(64):
        a = np.float32(rng.uniform(1, 2)) * np.float32(2.0) ** int(rng.integers(-20, 20))
        t = (rng.integers(0, 126, 96) + 0.5) / 127 * float(a)
        x = t.astype(np.float32)
        step = rng.integers(-2, 3, 96)
        x = np.where(step > 0, np.nextafter(x, np.float32(np.inf)), np.where(step < 0, np.nextafter(x, np.float32(0)), x))
        x *= rng.choice([-1, 1], 96).astype(np.float32)
        rows.append(np.concatenate([x.astype(np.float32), [a]]))
    rows.append(np.concatenate([np.arange(96, dtype=np.float32) + 0.5, [np.float32(127)]]))  # ties
    x = np.stack(rows).astype(np.float32)
    q, _ = erm.quantize_rows(torch.from_numpy(x).cuda())
    q = q.cpu().numpy()
    for i in range(x.shape[0]):
        a = Fraction(float(np.max(np.abs(x[i]))))
        assert [round(127 * Fraction(float(v)) / a) for v in x[i]] == q[i].tolist(), i  # Fraction rounds ties to even


def test_quantize_extreme_rows():
    tiny = torch.finfo(torch.float32).smallest_normal
    x = torch.zeros((8, 300))
    x[1, 5] = float("nan")
    x[2, 5], x[2, 6] = float("inf"), 1.0
    x[3] = torch.linspace(-1, 1, 300) * 3.4e38
    x[4] = torch.linspace(-1, 1, 300) * tiny
    x[5] = torch.linspace(-1, 1, 300) * tiny * 2**-20
    x[6] = 1.0
    x[7] = torch.linspace(-1, 1, 300) * 2.0**-100
    q, s = erm.quantize_rows(x.cuda())
    q, s = q.cpu(), s.cpu()
    assert s[0] == 0 and not q[0].any()
    assert torch.isnan(s[1:3]).all() and not q[1:3].any()
    wq, ws = quantized(x[3:])
    assert torch.equal(q[3:], wq) and torch.equal(s[3:], ws)


def test_quantize_strided_and_offset_rows():
    base = rand(6, 501, torch.bfloat16, 3).cuda()
    x = base[:, 3:404]
    room = torch.full((6, 450), 99, dtype=torch.int8, device="cuda")
    out = (room[:, 1:402], torch.empty(6, device="cuda"))
    q, s = erm.quantize_rows(x, out=out)
    wq, ws = quantized(x)
    assert torch.equal(q.cpu(), wq) and torch.equal(s.cpu(), ws)
    assert (room[:, 0] == 99).all() and (room[:, 402:] == 99).all()


def check_product(tokens, n, m, xd, yd, seed=0, W=None, X=None):
    W = rand_i8(m, n, seed + 1) if W is None else W
    sw = rand(1, m, torch.float32, seed + 2)[0].abs() * 1e-3
    if xd == "i8":
        X = rand_i8(tokens, n, seed) if X is None else X
        sx = rand(1, tokens, torch.float32, seed + 3)[0].abs()
        q, s = X.cpu(), sx
        y = erm.apply_quantized(W.cuda(), sw.cuda(), X.cuda(), sx.cuda(), out_dtype=TYPES[yd])
    else:
        X = rand(tokens, n, TYPES[xd], seed) if X is None else X
        q, s = quantized(X)
        y = erm.apply_quantized(W.cuda(), sw.cuda(), X.cuda(), out_dtype=TYPES[yd])
    want = (q.double() @ W.cpu().double().t()) * s.double()[:, None] * sw.double()
    assert y.dtype == TYPES[yd] and tuple(y.shape) == (tokens, m)
    close(y, want, TYPES[yd])
    return y


@pytest.mark.parametrize("xd,yd", [("i8", "f32"), ("i8", "bf16"), ("i8", "f16"), ("bf16", "bf16"), ("f16", "f16"),
                                   ("f32", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("tokens,n,m", [(1, 1, 1), (1, 16, 16), (2, 63, 17), (15, 64, 33), (16, 2560, 256), (17, 65, 100),
                                        (31, 127, 48), (32, 128, 129), (33, 129, 130), (64, 300, 200), (65, 1021, 70),
                                        (128, 128, 128), (130, 257, 259), (200, 640, 513)])
def test_product_matches_definition(tokens, n, m, xd, yd):
    check_product(tokens, n, m, xd, yd, seed=tokens + n + m)


@pytest.mark.parametrize("tokens,n,m,xd,yd", [(1, 2560, 2560, "bf16", "bf16"), (5, 9728, 2560, "i8", "f32"),
                                              (300, 2560, 1000, "bf16", "bf16"), (513, 1021, 2051, "f16", "f16"),
                                              (2, 131071, 40, "i8", "f32"), (70, 131071, 33, "i8", "f32"),
                                              (1100, 512, 2600, "i8", "bf16"),
                                              # ends of the row length within a stage of the tiles, whole
                                              # and split, direct and through registers
                                              (40, 16, 70, "i8", "f32"), (70, 48, 200, "i8", "f32"), (300, 144, 140, "i8", "bf16"),
                                              (300, 272, 300, "i8", "f16"), (70, 2559, 300, "i8", "f32"), (40, 5001, 130, "i8", "f32"),
                                              (100, 4096, 500, "bf16", "bf16"), (260, 2577, 250, "f32", "f32"),
                                              (33, 4112, 129, "i8", "f32"), (8, 2560, 100, "bf16", "bf16"),
                                              (7, 1000, 50, "f32", "f32"), (6, 130, 33, "f16", "f16")])
def test_product_larger_sizes(tokens, n, m, xd, yd):
    check_product(tokens, n, m, xd, yd, seed=tokens)


@pytest.mark.parametrize("tokens", [3, 40])
def test_product_largest_sums(tokens):
    """All codes -128 at the largest length: the sums reach 2^31 - 2^14."""
    n, m = 131071, 20
    q = torch.full((tokens, n), -128, dtype=torch.int8)
    check_product(tokens, n, m, "i8", "f32", W=torch.full((m, n), -128, dtype=torch.int8), X=q)


@pytest.mark.parametrize("tokens", [1, 20, 70])
def test_product_bad_tokens_stay_alone(tokens):
    x = rand(tokens + 2, 200, torch.float32, 11)
    x[0, 7], x[1, 8] = float("nan"), float("-inf")
    W, sw = rand_i8(90, 200, 1).cuda(), torch.ones(90, device="cuda")
    y = erm.apply_quantized(W, sw, x.cuda())
    assert torch.isnan(y[:2]).all()
    assert torch.equal(y[2:], erm.apply_quantized(W, sw, x[2:].contiguous().cuda()))
    assert not erm.apply_quantized(W, sw, torch.zeros((tokens, 200), device="cuda")).any()


@pytest.mark.parametrize("tokens", [7, 30, 150])
def test_product_strided_offset_out_and_single(tokens):
    room_w = rand_i8(75, 333, 4).cuda()
    W = room_w[:, 5:306]
    sw = torch.rand(75, device="cuda")
    X = rand(tokens, 400, torch.bfloat16, 6).cuda()[:, 1:302]
    room = torch.full((tokens + 1, 100), 7.0, device="cuda")
    y = erm.apply_quantized(W, sw, X, out=room[:tokens, 3:78])
    plain = erm.apply_quantized(W.contiguous(), sw, X.contiguous(), out_dtype=torch.float32)
    assert torch.equal(y, plain)
    assert (room[:, :3] == 7).all() and (room[:, 78:] == 7).all() and (room[tokens:] == 7).all()
    one = erm.apply_quantized(W, sw, X[0], out_dtype=torch.float32)
    assert one.shape == (75,) and torch.equal(one, plain[0])


@pytest.mark.parametrize("tokens", [3, 40, 90])
def test_product_rows_far_apart(tokens):
    """Row distances of 2^24 and more: offsets within a tile pass 32 bits."""
    room = torch.zeros(((1 << 24) + 32) * 300, dtype=torch.int8, device="cuda")
    W = torch.as_strided(room, (300, 160), ((1 << 24) + 16, 1), 5 * 16)
    W.copy_(rand_i8(300, 160, 1))
    X, sw, sx = rand_i8(tokens, 160, 2).cuda(), torch.rand(300, device="cuda"), torch.rand(tokens, device="cuda")
    y = erm.apply_quantized(W, sw, X, sx)
    assert torch.equal(y, erm.apply_quantized(W.contiguous(), sw, X, sx))


def test_offsets_past_32_bits():
    """70 000 x 32 768: element offsets of the tokens' rows, the codes and Y pass 2^31."""
    rows, n = 70000, 32768
    few = rand(64, n, torch.bfloat16, 5).cuda()
    q, s = erm.quantize_rows(few.repeat((rows + 63) // 64, 1)[:rows])
    wq, ws = erm.quantize_rows(few)
    assert torch.equal(q[:64], wq) and torch.equal(q[69952:], wq[:48]) and torch.equal(s[69952:], ws[:48])
    W, sw = rand_i8(n, 64, 6).cuda(), torch.rand(n, device="cuda")
    X, sx = q[:, :64], s
    y = erm.apply_quantized(W, sw, X, sx, out_dtype=torch.bfloat16)
    want = erm.apply_quantized(W, sw, X[:64].contiguous(), sx[:64].contiguous(), out_dtype=torch.bfloat16)
    assert torch.equal(y[:64], want) and torch.equal(y[69952:], want[:48])


def test_product_independent_of_batch():
    """The same token gives the same bits alone, in a small and in a large batch."""
    x = rand(300, 777, torch.bfloat16, 2).cuda()
    W, sw = rand_i8(333, 777, 3).cuda(), torch.rand(333, device="cuda")
    y = erm.apply_quantized(W, sw, x)
    for t in (1, 5, 17, 40, 100):
        assert torch.equal(erm.apply_quantized(W, sw, x[:t]), y[:t]), t


def test_product_empty():
    W, sw = rand_i8(5, 6, 0).cuda(), torch.rand(5, device="cuda")
    assert erm.apply_quantized(W, sw, torch.zeros((0, 6), device="cuda")).shape == (0, 5)
    q, s = erm.quantize_rows(torch.zeros((0, 6), device="cuda"))
    assert q.shape == (0, 6) and s.shape == (0,)


def test_product_streams_and_graph():
    x = [rand(t, 500, torch.bfloat16, t).cuda() for t in (4, 90)]
    W, sw = rand_i8(210, 500, 3).cuda(), torch.rand(210, device="cuda")
    want = [erm.apply_quantized(W, sw, v) for v in x]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(4):
        for v, s in zip(x, streams):
            got.append(erm.apply_quantized(W, sw, v, stream=s))
    torch.cuda.synchronize()
    for k, y in enumerate(got):
        assert torch.equal(y, want[k % 2])
    static = x[1].clone()
    erm.apply_quantized(W, sw, static)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = erm.apply_quantized(W, sw, static)
    for k in range(4):
        static.copy_(x[1] * (k + 1))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, erm.apply_quantized(W, sw, static)), k


def test_product_two_graphs_and_two_threads():
    """Two captured graphs with workspaces of their own, replayed at once; two host threads at once."""
    import threading

    W, sw = rand_i8(300, 3001, 3).cuda(), torch.rand(300, device="cuda")
    x = [rand(t, 3001, torch.bfloat16, t).cuda() for t in (70, 100)]
    want = [erm.apply_quantized(W, sw, v) for v in x]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for v in x:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(erm.apply_quantized(W, sw, v))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for r in range(5):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w), r
    got = [[], []]

    def work(i):
        with torch.cuda.stream(streams[i]):
            for _ in range(20):
                got[i].append(erm.apply_quantized(W, sw, x[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in (0, 1):
        assert len(got[i]) == 20 and all(torch.equal(y, want[i]) for y in got[i])


def test_binding_refusals():
    W, sw = rand_i8(8, 16, 0).cuda(), torch.ones(8, device="cuda")
    X = torch.zeros((3, 16), device="cuda")
    q, s = erm.quantize_rows(X)
    bad = [lambda: erm.apply_quantized(W.float(), sw, X), lambda: erm.apply_quantized(W, sw.double(), X),
           lambda: erm.apply_quantized(W, sw[:7], X), lambda: erm.apply_quantized(W, sw, X[:, :15]),
           lambda: erm.apply_quantized(W, sw, X.double()), lambda: erm.apply_quantized(W, sw, X, s),
           lambda: erm.apply_quantized(W, sw, q), lambda: erm.apply_quantized(W, sw, q, s[:2]),
           lambda: erm.apply_quantized(W, sw, X, out_dtype=torch.int8),
           lambda: erm.apply_quantized(W, sw, X, out=torch.empty((3, 9), device="cuda")),
           lambda: erm.apply_quantized(W, sw, X, out=torch.empty((3, 8), device="cuda"), out_dtype=torch.float16),
           lambda: erm.apply_quantized(W, sw, X.t().contiguous().t()), lambda: erm.apply_quantized(W, sw, X.cpu()),
           lambda: erm.apply_quantized(W, sw, X[:1].expand(3, 16)), lambda: erm.apply_quantized(W, sw, X[None]),
           lambda: erm.quantize_rows(X.double()), lambda: erm.quantize_rows(X[0]),
           lambda: erm.quantize_rows(X, out=(q[:2], s)), lambda: erm.quantize_rows(X, out=(q, s[:2]))]
    for k, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {k} was not refused")
    big = torch.zeros((1, 131072), dtype=torch.int8, device="cuda")
    with pytest.raises(erm.ExterndError) as e:
        erm.apply_quantized(big, sw[:1], big, torch.ones(1, device="cuda"))
    assert e.value.status == erm.EINVAL


def test_product_of_more_tiles_than_a_launch_holds():
    """2^29 + 300 tokens by one channel: 2^22 + 3 tiles of 128 rows."""
    tokens, n = 2**29 + 300, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    X = torch.randint(-128, 128, (tokens, n), generator=g, device="cuda", dtype=torch.int8)
    sx = torch.rand(tokens, generator=g, device="cuda")
    W, sw = rand_i8(1, n, 2).cuda(), torch.rand(1, device="cuda")
    room = torch.full((tokens, 2), 7.0, device="cuda")
    y = erm.apply_quantized(W, sw, X, sx, out=room[:, 1:])
    assert (room[:, 0] == 7).all()
    for t in range(0, tokens, 1 << 24):
        total = (X[t:t + (1 << 24)].int() * W.int()).sum(1)  # below 2^19: exact in fp32
        assert torch.equal(y[t:t + (1 << 24), 0], total.float() * sw * sx[t:t + (1 << 24)]), t


def test_missing_tensors_are_refused():
    X, W, sw = torch.zeros((3, 16), device="cuda"), rand_i8(8, 16, 0).cuda(), torch.ones(8, device="cuda")
    q = torch.empty((3, 16), dtype=torch.int8, device="cuda")
    for call in (lambda: erm.quantize_rows(None), lambda: erm.quantize_rows(X, out=(q, None)),
                 lambda: erm.quantize_rows(X, out=(None, sw[:3])), lambda: erm.apply_quantized(None, sw, X),
                 lambda: erm.apply_quantized(W, None, X), lambda: erm.apply_quantized(W, sw, None)):
        with pytest.raises(ValueError):
            call()


def test_outputs_beside_the_inputs_and_over_them():
    """X and Y as columns of one matrix (rows of one pitch) stay allowed; an output over an input is not."""
    for tokens in (1, 5, 40):
        room = torch.zeros((tokens, 500), dtype=torch.bfloat16, device="cuda")
        x = rand(tokens, 250, torch.bfloat16, tokens).cuda()
        room[:, :250] = x
        W, sw = rand_i8(250, 250, 1).cuda(), torch.rand(250, device="cuda")
        y = erm.apply_quantized(W, sw, room[:, :250], out=room[:, 250:])
        assert torch.equal(y, erm.apply_quantized(W, sw, x)) and torch.equal(room[:, :250], x)
        q = room.view(torch.int8)[:, 500:750]
        erm.quantize_rows(room[:, :250], out=(q, torch.empty(tokens, device="cuda")))
        assert torch.equal(q, erm.quantize_rows(x)[0]) and torch.equal(room[:, :250], x)
        for call in (lambda: erm.apply_quantized(W, sw, x, out=x), lambda: erm.apply_quantized(W, sw, room[:, :250], out=room[:, 249:499]),
                     lambda: erm.quantize_rows(x, out=(x.view(torch.int8)[:, :250], torch.empty(tokens, device="cuda")))):
            with pytest.raises(erm.ExterndError):
                call()


def test_more_rows_than_a_launch():
    """Quantisation runs of 2^23 rows; runs of 65535 groups of 32 tokens of rows too short for tiles."""
    rows = 2**23 + 3
    x = rand(4096, 3, torch.float32, 1)
    pick = torch.arange(rows) % 4093
    q, s = erm.quantize_rows(x[pick].cuda())
    wq, ws = quantized(x)
    assert torch.equal(q.cpu(), wq[pick]) and torch.equal(s.cpu(), ws[pick])
    tokens = 32 * 65535 + 5
    X, W, sw = rand_i8(4096, 7, 2), rand_i8(3, 7, 3), torch.rand(3)
    pick = torch.arange(tokens) % 4093
    sx = torch.rand(tokens)
    y = erm.apply_quantized(W.cuda(), sw.cuda(), X[pick].cuda(), sx.cuda())
    close(y, (X.double() @ W.double().t())[pick] * sx.double()[:, None] * sw.double(), torch.float32)
