"""w4a16_experts_gemm against a 64-bit product with the dequantized weights,
and a run of the operators of a layer of experts together.

Tolerance: the element-wise bound of the W4A16 product (parity.py), one bf16
rounding of an fp32 sum of K terms.
"""
import numpy as np
import pytest

from bit_gemm_quant_b200 import synth
from parity import assert_y_elementwise, dev_bf16, dev_f32, host_bf16_as_f64

SYM, ASYM = 0, 1


@pytest.fixture(scope="module")
def w4():
    from bit_gemm_quant_b200 import build
    build.build()
    import bit_gemm_quant_b200 as w4
    w4.lib()
    return w4


def dequantize(q, s, z, g):
    """W^ in fp64 [E, N, K] from the packed arrays (numpy), each value one bf16 rounding."""
    E, N, KW = q.shape
    u = np.empty((E, N, KW * 8))
    for i in range(8):
        u[..., i::8] = (q >> (4 * (i // 2) + 16 * (i % 2))) & 15
    G = s.shape[2]
    zp = np.full(s.shape, 8.0) if z is None else np.stack([(z[..., j // 8] >> (4 * (j % 8))) & 15 for j in range(G)], -1)
    w = (u.reshape(E, N, G, g) - zp[..., None]) * s.astype(np.float64)[..., None]
    return synth.bf16_bits_to_f32(synth.to_bf16_bits(w.reshape(E, N, -1).astype(np.float32))).astype(np.float64)


class Layer:
    """E quantized weights [N, K] on the device, and their values."""

    def __init__(self, w4, E, N, K, g, mode, seed=0):
        import torch
        packed = [w4.quant_pack(dev_bf16(synth.weights(seed * 1000 + e, N, K, 0.02, 0.01, 5.0)), g, mode) for e in range(E)]
        self.q, self.s = (torch.stack([p[i] for p in packed]) for i in (0, 1))
        self.z = torch.stack([p[2] for p in packed]) if mode == ASYM else None
        self.g, self.mode = g, mode
        u32 = lambda t: None if t is None else t.cpu().numpy().view(np.uint32)
        self.w = dequantize(u32(self.q), self.s.cpu().numpy(), u32(self.z), g)

    def __call__(self, w4, X, offsets, **kw):
        return w4.experts_gemm(X, self.q, self.s, self.z, self.g, self.mode, offsets, **kw)


def reference(layer, x, rows, offsets):
    """(Y, sum |x w|) of the sorted rows; rows: the row of x behind each."""
    N = layer.w.shape[1]
    Y, A = np.zeros((len(rows), N)), np.zeros((len(rows), N))
    for e in range(len(offsets) - 1):
        lo, hi = offsets[e], offsets[e + 1]
        xe = x[rows[lo:hi]]
        Y[lo:hi], A[lo:hi] = xe @ layer.w[e].T, np.abs(xe) @ np.abs(layer.w[e]).T
    return Y, A


def plan_of(ids, E):
    """(offsets, order) of ids [T, k], -1 for none."""
    flat = ids.reshape(-1)
    order = np.concatenate([np.flatnonzero(flat == e) for e in range(E)]).astype(np.int32)
    offsets = np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(E)])]).astype(np.int32)
    return offsets, np.concatenate([order, np.full(flat.size - order.size, -1, np.int32)])


def random_ids(T, E, k, seed, skew=0.0):
    rng = np.random.default_rng([T, E, k, seed])
    return np.argsort(-(rng.standard_normal((T, E)) + skew * np.arange(E)), axis=1)[:, :k].astype(np.int32)


def check(w4, layer, ids, gather, seed=0, stream=None):
    import torch
    E, N, K = layer.w.shape
    T, k = ids.shape
    P = T * k
    offsets, order = plan_of(ids, E)
    X = synth.activations(seed + 5, T if gather else P, K, 0.01, 40.0)
    out = torch.full((P + 2, N), 777.0, dtype=torch.bfloat16, device="cuda")
    kw = dict(order=torch.from_numpy(order).cuda(), top_k=k) if gather else {}
    got = layer(w4, dev_bf16(X), torch.from_numpy(offsets).cuda(), out=out[1:-1], stream=stream, **kw)
    torch.cuda.synchronize()
    assert w4.w4_device_error() == 0
    rows = order // k if gather else np.arange(P)
    n = offsets[-1]
    x = synth.bf16_bits_to_f32(X).astype(np.float64)
    if n:
        Y, A = reference(layer, x, rows[:n], offsets)
        assert_y_elementwise(host_bf16_as_f64(got)[:n], Y, A, K)
    assert (out[0] == 777).all() and (out[n + 1:] == 777).all(), "rows that are nobody's were written"
    return got


# (E, N, K, group, mode, T, k): one pair; tiles of one channel; k-blocks of half
# a group's length; few rows an expert and many; ragged everything
CASES = [(1, 16, 128, 128, SYM, 1, 1), (2, 1, 32, 32, ASYM, 1, 2), (4, 40, 320, 64, ASYM, 3, 2), (3, 129, 96, 32, SYM, 5, 1),
         (8, 300, 1408, 128, ASYM, 1, 2), (16, 64, 512, 64, SYM, 20, 4), (64, 48, 256, 32, ASYM, 16, 8),
         (5, 200, 544, 32, ASYM, 100, 2), (4, 260, 640, 128, SYM, 200, 2), (40, 130, 288, 32, ASYM, 150, 6),
         (2, 512, 1024, 128, ASYM, 700, 1), (3, 136, 2048, 64, SYM, 333, 2), (100, 32, 128, 64, ASYM, 64, 3),
         (8, 256, 512, 128, ASYM, 1500, 2), (6, 1000, 4096, 128, ASYM, 9, 3),
         # the widest tiles: whole and ragged ones, stored whole or element by element
         (2, 136, 512, 64, SYM, 1100, 1), (2, 300, 416, 32, ASYM, 1300, 1), (1, 77, 256, 128, ASYM, 600, 1),
         (3, 128, 1088, 64, ASYM, 1000, 2), (1, 40, 32, 32, SYM, 768, 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("E,N,K,g,mode,T,k", CASES)
def test_product_by_expert(w4, E, N, K, g, mode, T, k, gather):
    layer = Layer(w4, E, N, K, g, mode, seed=E)
    check(w4, layer, random_ids(T, E, k, 0), gather)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [4, 13, 40, 90, 600, 3700])
def test_uneven_plans(w4, T):
    """All rows at one expert; experts without rows at either end; no rows at all;
    some tokens without an expert."""
    layer = Layer(w4, 7, 136, 384, 64, ASYM, seed=3)
    for e in (0, 3, 6):
        check(w4, layer, np.full((T, 1), e, np.int32), True)
    check(w4, layer, random_ids(T, 7, 2, 1, skew=1.5), True)
    ids = random_ids(T, 7, 3, 2)
    ids[::3] = -1
    check(w4, layer, ids, True)
    check(w4, layer, np.full((T, 2), -1, np.int32), True)
    check(w4, layer, np.full((T, 2), -1, np.int32), False)


@pytest.mark.gpu
@pytest.mark.parametrize("counts", [
    (1, 15, 16, 17, 31, 33, 48, 64, 65, 100, 112, 113, 127, 128, 129, 0, 144, 257),
    (255, 256, 257, 241, 240, 16, 1, 272, 600, 513),
    (5, 5, 5, 5), (6, 6, 6, 6), (0, 0, 23, 1),
], ids=["tiles_128", "tiles_256", "streaming", "few_rows", "few_rows_one_expert"])
def test_rows_around_a_tile_and_an_mma(w4, counts):
    """Experts whose last tile ends around the multiples of 16 that an MMA is
    wide, around a tile, and averages on either side of the two kernels' limit."""
    layer = Layer(w4, len(counts), 200, 320, 32, ASYM, seed=12)
    ids = np.repeat(np.arange(len(counts), dtype=np.int32), counts)
    check(w4, layer, np.random.default_rng(5).permutation(ids)[:, None], True)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 40, 400])
def test_same_bits_again_and_on_another_stream(w4, T):
    import torch
    layer = Layer(w4, 8, 264, 640, 128, ASYM, seed=4)
    ids = random_ids(T, 8, 2, 3)
    first = check(w4, layer, ids, True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = check(w4, layer, ids, True, stream=side)
    assert torch.equal(first[: T * 2], again[: T * 2])


@pytest.mark.gpu
def test_a_given_workspace(w4):
    """A workspace of the stated size serves calls in turn; a smaller one is refused."""
    import torch
    layer = Layer(w4, 4, 136, 384, 64, ASYM, seed=12)
    need = w4.w4a16_experts_workspace_bytes(400, 4, 384, 1)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")          # NaN in every place
    for seed in (1, 2):
        ids = random_ids(200, 4, 2, seed)
        offsets, order = (torch.from_numpy(a).cuda() for a in plan_of(ids, 4))
        X = dev_bf16(synth.activations(seed, 200, 384))
        want = layer(w4, X, offsets, order=order, top_k=2)
        assert torch.equal(layer(w4, X, offsets, order=order, top_k=2, workspace=ws), want)
        with pytest.raises(w4.W4Error):
            layer(w4, X, offsets, order=order, top_k=2, workspace=ws[:-256])


@pytest.mark.gpu
def test_tensors_on_another_device(w4):
    """Calls on tensors of a device that is not the current one."""
    import torch
    if torch.cuda.device_count() < 2:
        pytest.skip("one GPU")
    layer = Layer(w4, 4, 136, 384, 64, ASYM, seed=13)
    ids = random_ids(30, 4, 2, 3)
    offsets, order = (torch.from_numpy(a).cuda() for a in plan_of(ids, 4))
    X = dev_bf16(synth.activations(3, 30, 384))
    want = layer(w4, X, offsets, order=order, top_k=2)
    to = lambda t: t.to("cuda:1")
    got = w4.experts_gemm(to(X), to(layer.q), to(layer.s), to(layer.z), 64, ASYM, to(offsets), order=to(order), top_k=2)
    assert got.device.index == 1 and torch.equal(got.cpu(), want.cpu())
    with pytest.raises(ValueError):
        w4.experts_gemm(X, to(layer.q), layer.s, layer.z, 64, ASYM, offsets, order=order, top_k=2)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [2, 300])
def test_a_wrong_plan_stays_inside_the_arrays(w4, T):
    """Offsets and rows out of range are taken as the nearest ends: the call
    returns, reports nothing and writes no row behind P."""
    import torch
    layer = Layer(w4, 4, 72, 256, 64, SYM, seed=5)
    X = dev_bf16(synth.activations(1, T, 256))
    out = torch.full((2 * T + 1, 72), 777.0, dtype=torch.bfloat16, device="cuda")
    order = torch.full((2 * T,), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    order[::2] = -5
    for offsets in ([0, -7, 10 ** 9, 3, 2 ** 31 - 1], [5, 4, 3, 2, 1], [-1] * 5):
        layer(w4, X, torch.tensor(offsets, dtype=torch.int32, device="cuda"), order=order, top_k=2, out=out[:-1])
        torch.cuda.synchronize()
    assert (out[-1] == 777).all() and w4.w4_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T,lo,hi", [(2, 0x401, 0x402), (300, 0x101, 0x106)], ids=["streaming", "tensor_core"])
def test_wait_runs_out_then_next_call_is_correct(w4, T, lo, hi):
    """The failure path without a fault (test_failure_path.py): a wait that runs
    out is reported, nothing hangs, and the next calls are right (a leaked
    tensor-memory allocation would stall them)."""
    from test_failure_path import run_with_short_limit
    layer = Layer(w4, 8, 520, 1024, 128, ASYM, seed=10)
    ids = random_ids(T, 8, 2, 5)
    offsets, order = plan_of(ids, 8)
    import torch
    X = dev_bf16(synth.activations(2, T, 1024))
    off, order = torch.from_numpy(offsets).cuda(), torch.from_numpy(order).cuda()
    for _ in range(3):
        code = run_with_short_limit(w4, lambda: layer(w4, X, off, order=order, top_k=2))
        assert lo <= code <= hi, hex(code)
        check(w4, layer, ids, True)


@pytest.mark.gpu
def test_calls_at_once(w4):
    """Layers on two streams at the same time give the bits that each gives alone."""
    import torch
    layer = Layer(w4, 8, 520, 1024, 64, ASYM, seed=11)
    jobs = []
    for T in (3, 200, 5, 500):
        ids = random_ids(T, 8, 2, T)
        offsets, order = (torch.from_numpy(a).cuda() for a in plan_of(ids, 8))
        X = dev_bf16(synth.activations(T, T, 1024))
        jobs.append((X, offsets, order, layer(w4, X, offsets, order=order, top_k=2)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [[layer(w4, X, off, order=order, top_k=2, stream=streams[i % 2]) for i, (X, off, order, _) in enumerate(jobs)]
               for _ in range(4)]
        torch.cuda.synchronize()
        for r in got:
            for y, job in zip(r, jobs):
                assert torch.equal(y, job[3])


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 64])
def test_arrays_past_32_bits(w4, T):
    """Codes of more than 2^32 bytes: the last expert's weights are at their end."""
    import torch
    E, N, K, g = 9, 131072, 8192, 128
    q = torch.zeros(E, N, K // 8, dtype=torch.int32, device="cuda")
    s = torch.zeros(E, N, K // g, dtype=torch.float16, device="cuda")
    packed = w4.quant_pack(dev_bf16(synth.weights(77, 200, K, 0.02)), g, SYM)
    q[-1, -200:], s[-1, -200:] = packed[0], packed[1]
    X = dev_bf16(synth.activations(78, T, K))
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[-1] = T
    Y = w4.experts_gemm(X, q, s, None, g, SYM, offsets)
    want = w4.gemm(X, packed[0], packed[1], None, g, SYM).double()
    # two sums of the same terms in fp32, in another order, each rounded to bf16: two half steps of 2^-8
    # and K 2^-22 of the terms' magnitudes (parity.py), those below 2^5 of the result's scale here
    diff = (Y[:, -200:].double() - want).norm() / want.norm()
    assert diff <= 2 * 2.0 ** -8 + 2 * K * 2.0 ** -22 * 2 ** 5
    assert (Y[:, :-200] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [2, 60], ids=["streaming", "tensor_core"])
@pytest.mark.parametrize("K,g", [(320, 64), (32, 32), (96, 32), (544, 32), (640, 128), (512, 128)])
def test_infinities_in_x(w4, K, g, T):
    """An infinity in a row gives an infinity of the weight's sign, NaN where the weight is 0, in that row alone:
    wherever it stands, the last columns of a K that is no whole stage among them."""
    layer = Layer(w4, 3, 72, K, g, ASYM, seed=14)
    ids = random_ids(T, 3, 1, 7)
    offsets, order = plan_of(ids, 3)
    assert (T <= 15) == (w4.w4a16_experts_workspace_bytes(T, 3, K, 1) == 0)      # the kernel that is meant
    for cols in ((K - 1,), (K - 32,), (0,), (K // 2, K - 3)):
        bits = synth.activations(21, T, K)
        for i, c in enumerate(cols):
            bits[i % T, c] = 0xFF80 if i else 0x7F80                             # +inf in row 0, -inf in row 1
        x = synth.bf16_bits_to_f32(bits).astype(np.float64)
        got = host_bf16_as_f64(layer(w4, dev_bf16(bits), torch_from(offsets), order=torch_from(order), top_k=1))
        for i, row in enumerate(order):
            e = ids[row, 0]
            if np.isinf(x[row]).any():
                c = int(np.argmax(np.isinf(x[row])))
                with np.errstate(invalid="ignore"):
                    want = x[row, c] * layer.w[e][:, c]
                assert np.array_equal(got[i], want, equal_nan=True), (cols, row)
            else:
                assert_y_elementwise(got[i:i + 1], x[row:row + 1] @ layer.w[e].T,
                                     np.abs(x[row:row + 1]) @ np.abs(layer.w[e]).T, K)


def torch_from(a):
    import torch
    return torch.from_numpy(a).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["rmsnorm", "rmsnorm_mxfp8", "route", "experts_gemm", "combine"])
def test_inputs_dropped_behind_a_call_on_a_side_stream(w4, name):
    """With stream= the inputs' memory is not handed out again before the kernel has read them, although the
    caller drops them right behind the call."""
    import torch
    T, K, E, k, N = 64, 512, 8, 2, 136
    layer = Layer(w4, E, N, K, 64, ASYM, seed=15)
    ids = random_ids(T, E, k, 1)
    n = lambda *shape: torch.randn(*shape, device="cuda")
    offsets, order = (torch.from_numpy(a).cuda() for a in plan_of(ids, E))
    pos = torch.argsort(order.long()).int().view(T, k)
    x, r, gamma = n(T, K).bfloat16(), n(T, K).bfloat16(), n(K).bfloat16()
    calls = {
        "rmsnorm": (w4.rmsnorm, (x, gamma, 1e-6, r), {}),
        "rmsnorm_mxfp8": (w4.rmsnorm_mxfp8, (x, gamma, 1e-6, r), {}),
        "route": (w4.route, (n(T, E), k), dict(scoring=w4.SIGMOID, bias=n(E), n_groups=4, topk_groups=3, group_top=2)),
        "experts_gemm": (w4.experts_gemm, (x, layer.q, layer.s, layer.z, 64, ASYM, offsets, order, k), {}),
        "combine": (w4.combine, (n(T * k, N).bfloat16(), pos, n(T, k)), dict(add=n(T, N).bfloat16())),
    }
    fn, args, kw = calls[name]
    want = [t.clone() for t in flat(fn(*args, **kw))]
    side = torch.cuda.Stream()
    fn(*args, **kw, stream=side)
    zeros = lambda: [torch.empty_like(args[0]).zero_() for _ in range(64)]
    zeros()                                              # (nothing below has to wait for memory or a kernel's code)
    copy = lambda v: v.clone() if isinstance(v, torch.Tensor) else v
    args2, kw2 = [copy(v) for v in args], {key: copy(v) for key, v in kw.items()}
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)                   # some 50 ms: the call below is still to come
    got = fn(*args2, stream=side, **kw2)
    del args2, kw2
    fill = zeros()                                       # on the current stream, at once
    torch.cuda.synchronize()
    assert len(fill) == 64
    for a, b in zip(flat(got), want):
        assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 90])
def test_a_given_stream_under_capture(w4, T):
    """stream= naming the capturing stream, inputs dropped behind the calls that read them."""
    import torch
    layer = Layer(w4, 8, 136, 512, 64, ASYM, seed=17)
    x, r, gamma, gate, bias = layer_inputs(w4, T, 512, 0, 8, 5)
    side = torch.cuda.Stream()

    def run(stream):
        y, h = w4.rmsnorm(x, gamma, 1e-6, residual=r, stream=stream)
        plan = w4.route(y.float() @ gate, 2, scoring=w4.SIGMOID, bias=bias, stream=stream)
        a = layer(w4, y, plan.offsets, order=plan.order, top_k=2, stream=stream)
        return w4.combine(a, plan.pos, plan.weights, stream=stream), h

    want = run(None)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        got = run(side)
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    assert w4.w4_device_error() == 0


def flat(v):
    import torch
    return [v] if isinstance(v, torch.Tensor) else [t for t in v if t is not None]


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 64], ids=["streaming", "tensor_core"])
def test_values_past_32_bits(w4, T):
    """Each value of a product whose weights lie behind 2^32 bytes of codes, within one rounding of the exact sum;
    other weights stand where an index cut to 32 bits would read."""
    import torch
    E, N, K, g, n = 9, 131072, 8192, 128, 200
    q = torch.zeros(E, N, K // 8, dtype=torch.int32, device="cuda")
    s = torch.zeros(E, N, K // g, dtype=torch.float16, device="cuda")
    last = w4.quant_pack(dev_bf16(synth.weights(77, n, K, 0.02)), g, SYM)
    decoy = w4.quant_pack(dev_bf16(synth.weights(78, n, K, 0.02)), g, SYM)
    wrapped = (E * N * (K // 2) - 2 ** 32) // (K // 2)      # this row of codes lies 2^32 bytes in front of the end
    q.view(E * N, -1)[wrapped - n:wrapped], s.view(E * N, -1)[wrapped - n:wrapped] = decoy[0], decoy[1]
    q[-1, -n:], s[-1, -n:] = last[0], last[1]
    bits = synth.activations(79, T, K)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[-1] = T
    got = w4.experts_gemm(dev_bf16(bits), q, s, None, g, SYM, offsets)
    w = dequantize(last[0].cpu().numpy().view(np.uint32)[None], last[1].cpu().numpy()[None], None, g)[0]
    x = synth.bf16_bits_to_f32(bits).astype(np.float64)
    assert_y_elementwise(host_bf16_as_f64(got[:, -n:]), x @ w.T, np.abs(x) @ np.abs(w).T, K)
    assert (got[:, :-n] == 0).all()


# ------------------------------------------------- the operators together --

def forward(w4, x, r, gamma, gate, up, down, k, bias):
    """One layer of experts as a decoder runs it; every tensor it makes, in order."""
    import torch
    y, h = w4.rmsnorm(x, gamma, 1e-6, residual=r)
    plan = w4.route(y.float() @ gate, k, scoring=w4.SIGMOID, bias=bias, n_groups=4, topk_groups=2, group_top=2, scale=1.5)
    a = up(w4, y, plan.offsets, order=plan.order, top_k=k)
    F = a.shape[1] // 2
    b = (torch.nn.functional.silu(a[:, :F].float()) * a[:, F:].float()).bfloat16()
    c = down(w4, b, plan.offsets)
    out = w4.combine(c, plan.pos, plan.weights, add=h)
    codes, scales, _ = w4.rmsnorm_mxfp8(out, gamma, 1e-6)
    return dict(y=y, h=h, plan=plan, a=a, b=b, c=c, out=out, codes=codes, scales=scales)


def layer_inputs(w4, T, K, F, E, seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = lambda *shape: torch.randn(*shape, generator=g, device="cuda")
    return (n(T, K).bfloat16(), n(T, K).bfloat16(), (1 + 0.1 * n(K)).bfloat16(), n(K, E) / K ** 0.5, 0.1 * n(E))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 13, 260])
def test_a_layer_of_experts(w4, T):
    """Each operator against 64 bits on what the one before it gave."""
    import test_parity_norm as norm
    import test_parity_route as rt
    K, F, E, k = 256, 96, 16, 3
    up, down = Layer(w4, E, 2 * F, K, 128, ASYM, seed=6), Layer(w4, E, K, F, 32, SYM, seed=7)
    x, r, gamma, gate, bias = layer_inputs(w4, T, K, F, E, T)
    o = forward(w4, x, r, gamma, gate, up, down, k, bias)
    host = host_bf16_as_f64
    h = host(x) + host(r)
    y = h / np.sqrt((h * h).mean(1, keepdims=True) + 1e-6) * host(gamma)
    norm.between(host(o["y"]), y, norm.bf16, "y")
    logits = (o["y"].float() @ gate).cpu().numpy().astype(np.float64)
    ids, weights = rt.choose(logits, k, True, bias.cpu().numpy(), 4, 2, 2, True, 1.5)
    assert np.array_equal(o["plan"].ids.cpu().numpy(), ids)
    offsets, order, pos = rt.plan(ids, E)
    Y, A = reference(up, host(o["y"]), order // k, offsets)
    assert_y_elementwise(host(o["a"]), Y, A, K)
    Y, A = reference(down, host(o["b"]), np.arange(T * k), offsets)
    assert_y_elementwise(host(o["c"]), Y, A, F)
    terms = host(o["c"])[pos] * weights.astype(np.float32).astype(np.float64)[..., None]
    hh = host(o["h"])
    ref, mag = hh + terms.sum(1), np.abs(hh) + np.abs(terms).sum(1)
    # the weights used on the device are rounded as these are, up to one fp32 step (2^-23)
    e = (k + 2) * 2.0 ** -24 * mag + 2.0 ** -23 * mag
    assert (np.abs(host(o["out"]) - ref) <= 2.0 ** -8 * (np.abs(ref) + e) + e).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 24, 150])
def test_a_layer_captured_and_replayed(w4, T):
    """The whole layer in a CUDA graph: replays with other inputs, and so other
    plans, give the bits of eager calls; two graphs do not disturb each other."""
    import torch
    K, F, E, k = 256, 128, 8, 2
    up, down = Layer(w4, E, 2 * F, K, 64, ASYM, seed=8), Layer(w4, E, K, F, 64, ASYM, seed=9)
    inputs = [layer_inputs(w4, T, K, F, E, s) for s in (1, 2, 3)]
    static = [t.clone() for t in inputs[0]]
    run = lambda a: forward(w4, a[0], a[1], a[2], a[3], up, down, k, a[4])
    run(static)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = run(static)
        graphs.append((g, got))
    for a in inputs + inputs[:1]:
        for t, v in zip(static, a):
            t.copy_(v)
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        want = run(a)
        for _, got in graphs:
            for name in ("y", "h", "out", "codes", "scales"):
                assert torch.equal(got[name], want[name]), name
            for u, v in zip(got["plan"], want["plan"]):
                assert torch.equal(u, v)
    assert w4.w4_device_error() == 0


# ------------------------------------------------------------- refusals --

FAKE = 1 << 20


def call(w4, X=FAKE, R=64, offsets=FAKE, order=FAKE, k=2, E=8, P=64, N=64, K=256, q=FAKE, s=FAKE, z=None, g=128, mode=0,
         Y=FAKE, ws=None, wbytes=0):
    return w4.w4a16_experts_gemm(X, R, offsets, order, k, E, P, N, K, q, s, z, g, mode, Y, ws, wbytes, None)


@pytest.mark.parametrize("bad", [
    dict(X=None), dict(offsets=None), dict(q=None), dict(s=None), dict(Y=None), dict(R=0), dict(k=0), dict(E=0),
    dict(E=1025), dict(P=0), dict(N=0), dict(K=0), dict(K=192), dict(g=16), dict(mode=2), dict(mode=0x100),
    dict(mode=0x201), dict(mode=1), dict(z=FAKE), dict(order=None, R=63), dict(X=FAKE + 8), dict(q=FAKE + 4),
    dict(s=FAKE + 1), dict(offsets=FAKE + 2), dict(order=FAKE + 2), dict(mode=1, z=FAKE + 2), dict(Y=FAKE + 1),
    dict(N=1 << 61), dict(P=4096, ws=FAKE, wbytes=4096 * 512 - 1), dict(P=4096, wbytes=4096 * 512),
    dict(P=4096, ws=FAKE + 128, wbytes=4096 * 512)])
def test_refusals(w4, bad):
    assert call(w4, **bad) == w4.W4_ERR_INVALID_ARG


@pytest.mark.parametrize("big", [dict(N=1 << 29, ws=FAKE, wbytes=1 << 40), dict(P=(1 << 23) + 1, ws=FAKE, wbytes=1 << 40),
                                 dict(R=1 << 31, order=FAKE, ws=FAKE, wbytes=1 << 40)])
def test_unsupported(w4, big):
    assert call(w4, **big) == w4.W4_ERR_UNSUPPORTED


def test_workspace_bytes(w4):
    assert w4.w4a16_experts_workspace_bytes(4096, 8, 256, 1) == 4096 * 512
    assert w4.w4a16_experts_workspace_bytes(4096, 8, 256, 0) == 0       # the rows are sorted already
    assert w4.w4a16_experts_workspace_bytes(8, 8, 256, 1) == 0          # the GEMV reads them in place
    assert w4.w4a16_experts_workspace_bytes(0, 8, 256, 1) == 0
    assert w4.w4a16_experts_workspace_bytes(1 << 40, 8, 1 << 40, 1) == 0


def test_helper_refusals(w4):
    import torch
    X = torch.zeros(4, 256, dtype=torch.bfloat16)
    q, s = torch.zeros(2, 16, 32, dtype=torch.int32), torch.zeros(2, 16, 2, dtype=torch.float16)
    offsets = torch.zeros(3, dtype=torch.int32)
    for args in ((X, q, s, None, 128, 0, offsets), (X, q[0], s, None, 128, 0, offsets), (X, q, s, None, 0, 0, offsets),
                 (X.float(), q, s, None, 128, 0, offsets)):
        with pytest.raises(ValueError):
            w4.experts_gemm(*args)
