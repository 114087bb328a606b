"""The 8-bit (block-128) quantisers, product and linear layer against the float64
oracle, through the public Python layer and the C ABI.

Gates (from the arithmetic):
* codes and scales are bit-exact: S is a power of two and v / S is exact on both sides;
* whole numbers whose sums stay below 2^24 (times one power of two) come out exact in
  float32, whatever the order of the sums: any misplaced element, block or scale shows;
* real data, float32 results: products are exact, and each of the K additions is off by
  at most one unit of 2^-23 of the partial sum (rounded or truncated), so
  |y - y64| <= K 2^-23 sum |a||b| + half a step of y's type;
* bf16 results: beside that, a group of 8 products loses at most one unit of 2^-13 of
  its largest for each of the others, 7 * 2^-13 max|a||b| <= 7 * 2^-13 * (sum over the
  group), and a bound for y is 7 * 2^-13 of sum |a||b|; half a step of bf16 is added.
"""

import numpy as np
import pytest
import torch

from oracle import fp8 as O
from wam_asp_w4a4_amd import binding as B
from wam_asp_w4a4_amd.fp8 import Fp8Layer, Fp8Tensor, quantize

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def to_device(a, dtype="f32", ld=None):
    """A float64 array as a device matrix of row stride ld, and its values as float64."""
    t = torch.from_numpy(np.ascontiguousarray(a)).to(TYPES[dtype])
    if ld:
        wide = torch.full((t.shape[0], ld), 77.0, dtype=t.dtype)
        wide[:, :t.shape[1]] = t
        return wide.to(DEV)[:, :t.shape[1]], t.double().numpy()
    return t.to(DEV), t.double().numpy()


def host(t):
    return t.double().cpu().numpy()


def check_codes(q, codes, bytes_):
    np.testing.assert_array_equal(q.codes.cpu().numpy(), codes)
    np.testing.assert_array_equal(q.scales.cpu().numpy(), O.layout_scales(bytes_))


def data(rng, M, K):
    """Magnitudes over 2^-30 .. 2^30, a block of zeros, and values at every border."""
    v = rng.standard_normal((M, K)) * np.exp2(rng.integers(-30, 31, (M, -(-K // 128)))).repeat(128, 1)[:, :K]
    v[-1, :min(K, 128)] = 0.0
    special = [448.0, -17.0, 18.0, 19.0, 2.0 ** -10, -3 * 2.0 ** -10, -0.0, 2.0 ** -11]
    v[0, :min(K, 8)] = special[:K]
    if K > 8:
        v[0, 8:128] = 0.25
    return v


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,K,ld", [(1, 1, None), (1, 128, None), (3, 127, None), (5, 129, 200),
                                    (130, 640, None), (257, 1000, 1008), (64, 1001, 1001),
                                    (300, 513, None)])
def test_quantisers_are_bit_exact(M, K, ld, dtype):
    print(f"quantise {M}x{K} ld={ld} {dtype}", flush=True)
    x, v = to_device(data(np.random.default_rng(M + K), M, K), dtype, ld)
    codes, s = O.quantize(v)
    q = quantize(x)
    check_codes(q, codes, s)
    check_codes(quantize(x, transpose=True), *O.quantize(v.T))
    layer = Fp8Layer.pack(x)
    check_codes(layer, *O.quantize(v, square=True))
    check_codes(Fp8Tensor(K, M, layer.codes_t, layer.scales_t), *O.quantize(v.T, square=True))
    got = host(q.dequantize())
    np.testing.assert_array_equal(got, O.values(codes, s, K))   # float32 holds every one here
    np.testing.assert_array_equal(host(q.dequantize("bf16")), got)


def test_values_without_a_code_and_extremes():
    v = np.zeros((4, 256))
    v[0, :4] = [np.nan, -np.inf, 3.0, np.inf]
    v[1, :3] = [2.0 ** -149, -2.0 ** -126, 2.0 ** -130]
    v[2, :2] = [3.4028234663852886e38, -1e30]
    v[3, 128:] = np.nan
    x, v = to_device(v)
    q = quantize(x)
    codes, s = O.quantize(v)
    nan = np.isnan(v) | np.isinf(v)
    got = q.codes.cpu().numpy()
    assert ((got & 0x7F) == 0x7F)[nan].all()
    np.testing.assert_array_equal(got[~nan], codes[~nan])
    np.testing.assert_array_equal(q.scales.cpu().numpy(), O.layout_scales(s))
    back = host(q.dequantize())
    assert np.isnan(back[nan]).all()
    np.testing.assert_array_equal(back[~nan], np.float32(O.values(codes, s, 256))[~nan])
    # a row with a NaN or infinity spoils its own results only
    w, _ = to_device(np.ones((20, 256)))
    for rows in (4, 40):   # the few-row kernel and the tiles
        y = Fp8Layer.pack(w).forward(torch.cat([x, torch.ones((rows - 4, 256), device=DEV)]))
        assert torch.isnan(y[[0, 3]]).all() and torch.isfinite(y[1]).all()
        assert torch.isfinite(y[4:]).all()


# every kernel: few rows, 32 x 32 tiles, tiles of 64, 128 (whole and split) and 256 (whole, the
# last ones in quarters or halves)
SHAPES = [(1, 16, 1), (1, 33, 128), (5, 100, 129), (16, 4096, 1024), (16, 40, 4224), (17, 16, 640),
          (33, 65, 127), (64, 64, 8192), (100, 130, 1537), (256, 1024, 1024), (777, 515, 300),
          (1920, 1793, 256), (3500, 3330, 640), (4100, 3900, 130), (4100, 4700, 200), (1500, 3500, 2050),
          (1000, 1003, 385), (520, 515, 33000)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product_of_whole_numbers_is_exact(M, N, K):
    """|a|, |b| <= 4 times a power of two for each block: sums of K <= 33000 products stay
    below 2^24 units of the smallest."""
    print(f"product {M}x{N}x{K}", flush=True)
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    nb = -(-K // 128)
    ka = rng.integers(-2, 2, nb).repeat(128)[:K]

    def matrix(rows):
        return rng.integers(-4, 5, (rows, K))

    a = matrix(M) * np.exp2(ka)
    b = matrix(N) * np.exp2(-ka)        # so that every product is a whole number
    x, _ = to_device(a, "bf16")
    w, _ = to_device(b, "bf16")
    bias = rng.integers(-50, 50, N)
    xa = torch.from_numpy(a).to(DEV)
    want = xa @ torch.from_numpy(b).to(DEV).t() + torch.from_numpy(bias).to(DEV).double()
    layer = Fp8Layer.pack(w, torch.from_numpy(bias).float().to(DEV), backward=False)
    y = layer.forward(x, "f32")
    assert torch.equal(y.double(), want)
    assert torch.equal(layer.forward(x, "bf16"), want.float().bfloat16())
    assert torch.equal(layer.forward(quantize(x), "f32"), y)
    assert torch.equal(Fp8Layer(N, K, layer.codes, layer.scales, None, None, None).forward(x, "f32").double(),
                       want - torch.from_numpy(bias).to(DEV).double())


def far_apart(rng, K):
    """The columns, one of a block of 128 and at most 200 of them, at which both operands
    hold +-256 beside the +-1 of all others: products of 2^16 next to ones of 1."""
    blocks = np.linspace(0, -(-K // 128) - 1, min(200, -(-K // 128))).astype(int)
    return np.unique(np.minimum(128 * blocks + rng.integers(0, 128, blocks.size), K - 1))


def signs(rng, rows, cols):
    return (rng.integers(0, 2, (rows, cols), dtype=np.int8) * 2 - 1).astype(np.float32)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_float32_results_are_summed_in_float32(M, N, K):
    """Products 16 bits apart within eight consecutive ones, which the 8-bit instruction's
    14-bit window would drop.  All magnitudes together are below 200 * 2^16 + 33000 < 2^24:
    float32 sums of any order are exact."""
    print(f"float32 sums {M}x{N}x{K}", flush=True)
    rng = np.random.default_rng(M + N + K)
    big = far_apart(rng, K)
    a, b = signs(rng, M, K), signs(rng, N, K)
    a[:, big] *= 256
    b[:, big] *= 256
    x, w = (torch.from_numpy(v).to(DEV) for v in (a, b))
    want = x.double() @ w.double().t()
    layer = Fp8Layer.pack(w, backward=False)
    for xt in (x, x.bfloat16(), quantize(x)):
        assert torch.equal(layer.forward(xt, "f32").double(), want)


@pytest.mark.parametrize("y_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K,dtype,ld", [(1, 1030, 1024, "bf16", None), (7, 64, 1000, "f32", 1003),
                                            (16, 256, 4096, "bf16", 4104), (200, 300, 2000, "f32", None),
                                            (256, 1024, 4096, "bf16", None), (2000, 1700, 515, "bf16", 520)])
def test_layer_against_the_oracle(M, N, K, dtype, ld, y_dtype):
    print(f"layer {M}x{N}x{K} {dtype} -> {y_dtype}", flush=True)
    rng = np.random.default_rng(K + M)
    x, xv = to_device(rng.standard_normal((M, K)) * np.exp(rng.standard_normal((1, K))), dtype, ld)
    w, wv = to_device(rng.standard_normal((N, K)) / np.sqrt(K), dtype)
    b = rng.standard_normal(N).astype(np.float32)
    layer = Fp8Layer.pack(w, torch.from_numpy(b).to(DEV))
    y = layer.forward(x, y_dtype)
    qx, qw = O.held(xv), O.held(wv, square=True)
    want = qx @ qw.T + b
    half, window = (2.0 ** -8, 7 * 2.0 ** -13) if y_dtype == "bf16" else (2.0 ** -24, 0.0)
    bound = (K * 2.0 ** -23 + window) * (np.abs(qx) @ np.abs(qw).T) + 2.0 ** -23 * np.abs(b)
    assert (np.abs(host(y) - want) <= bound + half * (np.abs(want) + bound)).all()
    # the row quantiser and the product in two calls: the same bits
    assert torch.equal(layer.forward(quantize(x), y_dtype), y)
    # and on every call, into the caller's buffers, whatever they held
    out, ws = torch.full_like(y, 3.0), layer.workspace(M).fill_(255)
    assert layer.forward(x, y_dtype, ws, out) is out and torch.equal(out, y)


GRADS = [(1, 24, 16, "f32"), (130, 100, 200, "bf16"), (16, 1000, 33, "f32"), (300, 16, 130, "bf16"),
         (257, 515, 640, "f32"), (1024, 256, 512, "bf16"), (2048, 2100, 1792, "bf16"),
         # small products of one launch: 32 x 32 tiles with 64 x 64 ones, 64 x 64 ones only
         (300, 2000, 1300, "bf16"), (1200, 2000, 1300, "f32")]


@pytest.mark.parametrize("M,N,K,dtype", GRADS)
def test_gradients_against_the_oracle(M, N, K, dtype):
    print(f"gradients {M}x{N}x{K} {dtype}", flush=True)
    rng = np.random.default_rng(M + 2 * N + 3 * K)
    x, xv = to_device(rng.standard_normal((M, K)) * 3, dtype, K + 8)
    dy, dv = to_device(rng.standard_normal((M, N)) * 1e-3 * np.exp(rng.standard_normal((M, 1))), dtype, N + 3)
    w, wv = to_device(rng.standard_normal((N, K)), dtype)
    layer = Fp8Layer.pack(w, torch.zeros(N, device=DEV))
    dx, dw, db = layer.backward(dy, x)
    wx, ww, wb = O.backward(dv, xv, wv)
    half, window = (2.0 ** -8, 7 * 2.0 ** -13) if dtype == "bf16" else (2.0 ** -24, 0.0)

    def near(got, want, terms, mass, step):
        bound = (terms * 2.0 ** -23 + (window if step > 1e-3 else 0.0)) * mass
        assert (np.abs(host(got) - want) <= bound + step * (np.abs(want) + bound)).all()

    near(dx, wx, N, np.abs(O.held(dv)) @ np.abs(O.held(wv, True)), half)
    near(dw, ww, M, np.abs(O.held(dv.T)) @ np.abs(O.held(xv.T)).T, 2.0 ** -24)
    near(db, wb, M, np.abs(dv).sum(axis=0), 2.0 ** -24)
    assert dx.dtype == TYPES[dtype] and dw.dtype == db.dtype == torch.float32
    # each alone is the same, and the ones that nobody asks for are absent
    one = layer.backward(dy)
    assert torch.equal(one[0], dx) and one[1] is None and torch.equal(one[2], db)
    two = layer.backward(dy, x, need_dx=False, need_db=False, dw_dtype="bf16")
    assert two[0] is None and two[2] is None and two[1].dtype == torch.bfloat16
    near(two[1], ww, M, np.abs(O.held(dv.T)) @ np.abs(O.held(xv.T)).T * (1 + 7 * 2.0 ** -13 / (M * 2.0 ** -23)), 2.0 ** -8)
    three = layer.backward(dy, need_dx=False, workspace=layer.workspace(M, backward=True).fill_(255))
    assert three[0] is three[1] is None and torch.equal(three[2], db)


@pytest.mark.parametrize("M,N,K", [shape[:3] for shape in GRADS])
def test_float32_gradients_are_summed_in_float32(M, N, K):
    """As in the forward: dx sums over N and dw over M, at most 200 * 2^16 + 2100 * 2^8 < 2^24."""
    print(f"float32 gradients {M}x{N}x{K}", flush=True)
    rng = np.random.default_rng(M + N + K)
    x, dy, w = signs(rng, M, K), signs(rng, M, N), signs(rng, N, K)
    m, n = far_apart(rng, M), far_apart(rng, N)
    dy[m] = signs(rng, m.size, N) * 256
    x[m] *= 256
    dy[:, n] = signs(rng, M, n.size) * 256
    w[n] *= 256
    x, dy, w = (torch.from_numpy(v).to(DEV) for v in (x, dy, w))
    dx, dw, db = Fp8Layer.pack(w, torch.zeros(N, device=DEV)).backward(dy, x)
    assert torch.equal(dx.double(), dy.double() @ w.double())
    assert torch.equal(dw.double(), dy.double().t().contiguous() @ x.double())
    assert torch.equal(db.double(), dy.double().sum(0))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(1, 4096, 1024), (16, 14336, 4096), (3, 130, 200), (20000, 16, 1300), (5000, 9, 70),
                                   (256, 1024, 1024), (700, 2000, 1300)])
def test_each_gradient_alone_has_the_same_bits(M, N, K, dtype):
    """Which kernel a product takes depends on its own sizes, not on what else is asked for."""
    print(f"alone {M}x{N}x{K} {dtype}", flush=True)
    torch.manual_seed(M + N + K)
    layer = Fp8Layer.pack(torch.randn((N, K), device=DEV), torch.zeros(N, device=DEV))
    x, dy = torch.randn((M, K), device=DEV).to(TYPES[dtype]), torch.randn((M, N), device=DEV).to(TYPES[dtype])
    for dw_dtype in ("f32", "bf16"):
        dx, dw, db = layer.backward(dy, x, dw_dtype=dw_dtype)
        for need_dx, need_dw, need_db in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 0, 1), (0, 1, 1), (1, 1, 0)):
            got = layer.backward(dy, x if need_dw else None, need_dx=need_dx, need_db=need_db, dw_dtype=dw_dtype)
            for name, g, want, need in zip(("dx", "dw", "db"), got, (dx, dw, db), (need_dx, need_dw, need_db)):
                assert (g is not None) == bool(need)
                assert g is None or torch.equal(g, want), (name, dw_dtype, need_dx, need_dw, need_db)
    if M > 16:     # above the few-row kernel's rows, the product of the same operands
        back = Fp8Layer(K, N, layer.codes_t, layer.scales_t, None, None, None)
        assert torch.equal(back.forward(quantize(dy), dtype), dx)


def test_gradients_against_differences():
    """Whole numbers: the layer is linear in them, so differences are exact."""
    rng = np.random.default_rng(5)
    M, N, K = 40, 70, 150
    x, w, dy = (rng.integers(-4, 5, s).astype(float) for s in ((M, K), (N, K), (M, N)))
    xt, wt, dt = (to_device(a)[0] for a in (x, w, dy))
    layer = Fp8Layer.pack(wt)
    dx, dw, _ = layer.backward(dt, xt)
    d = rng.integers(-2, 3, x.shape)
    dt_ = torch.from_numpy(d).float().to(DEV)
    diff = (layer.forward(xt + dt_).double() - layer.forward(xt).double()) * dt.double()
    assert diff.sum().item() == (dx.double() * dt_.double()).sum().item()
    d = torch.from_numpy(rng.integers(-2, 3, w.shape)).float().to(DEV)
    diff = (Fp8Layer.pack(wt + d).forward(xt).double() - layer.forward(xt).double()) * dt.double()
    assert diff.sum().item() == (dw.double() * d.double()).sum().item()


def test_empty_batches():
    layer = Fp8Layer.pack(torch.ones((40, 200), device=DEV), torch.ones(40, device=DEV))
    assert layer.forward(torch.empty((0, 200), device=DEV)).shape == (0, 40)
    assert quantize(torch.empty((0, 200), device=DEV)).codes.shape == (0, 256)
    dx, dw, db = layer.backward(torch.empty((0, 40), device=DEV), torch.empty((0, 200), device=DEV))
    assert dx.shape == (0, 200) and not dw.any() and not db.any()
    for N, K in ((2000, 1300), (4000, 2000)):   # the tiled kernels
        layer = Fp8Layer.pack(torch.ones((N, K), device=DEV), torch.ones(N, device=DEV))
        dx, dw, db = layer.backward(torch.empty((0, N), device=DEV), torch.empty((0, K), device=DEV))
        assert dx.shape == (0, K) and not dw.any() and not db.any()


def test_neighbouring_memory_is_untouched():
    """Ragged outputs inside a larger buffer: nothing around them is written."""
    for M, N, K in [(3, 19, 70), (70, 37, 200), (300, 261, 129)]:
        print(f"neighbours {M}x{N}x{K}", flush=True)
        layer = Fp8Layer.pack(torch.randn((N, K), device=DEV))
        x = torch.randn((M, K), device=DEV)
        buf = torch.full((M * N + 64,), 7.0, device=DEV)
        y = layer.forward(x, y=buf[32:32 + M * N].view(M, N))   # 16-byte aligned, ragged rows
        z = torch.full((M * N + 64,), 7.0, device=DEV)
        layer.forward(x, y=z[3:3 + M * N].view(M, N))           # aligned to its elements only
        assert torch.equal(z[3:3 + M * N].view(M, N), y)
        assert (buf[:32] == 7).all() and (buf[32 + M * N:] == 7).all()
        assert (z[:3] == 7).all() and (z[3 + M * N:] == 7).all()


def test_captured_calls_replay_like_eager_ones():
    layer = Fp8Layer.pack(torch.randn((512, 1024), device=DEV), torch.randn(512, device=DEV))
    for M in (4, 256):
        x, dy = torch.randn((M, 1024), device=DEV), torch.randn((M, 512), device=DEV)
        ws, wb = layer.workspace(M), layer.workspace(M, backward=True)
        y = torch.empty((M, 512), device=DEV)
        layer.forward(x, workspace=ws, y=y)
        layer.backward(dy, x, workspace=wb)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer.forward(x, workspace=ws, y=y)
            grads = layer.backward(dy, x, workspace=wb)
        for i in range(4):
            x.copy_(torch.randn((M, 1024), device=DEV) * (i + 1))
            dy.copy_(torch.randn((M, 512), device=DEV))
            want_y, want = layer.forward(x), layer.backward(dy, x)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want_y)
            assert all(torch.equal(a, b) for a, b in zip(grads, want))


def test_calls_on_another_stream():
    layer = Fp8Layer.pack(torch.randn((300, 700), device=DEV))
    x = torch.randn((500, 700), device=DEV)
    want = layer.forward(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [layer.forward(x, stream=side.cuda_stream) for _ in range(4)]
    with torch.cuda.stream(side):
        got.append(layer.forward(x))
    side.synchronize()
    assert all(torch.equal(g, want) for g in got)


def _busy():
    """Some milliseconds of work on the current stream."""
    a = torch.ones((8192, 8192), dtype=torch.bfloat16, device=DEV)
    b = torch.empty_like(a)
    for _ in range(12):
        torch.mm(a, a, out=b)


@pytest.mark.parametrize("other", ["a side stream", "the default stream"])
def test_memory_of_calls_on_another_stream(other):
    """The current stream is behind: blocks that it freed are still to be written by it, and a
    result is still to be read.  Neither may be handed to a call on another stream."""
    from wam_asp_w4a4_amd.norm import gated_norm, gated_norm_backward
    M, N, K = 500, 300, 700
    w, bias = torch.randn((N, K), device=DEV), torch.randn(N, device=DEV)
    x, x2, dy = (torch.randn((M, k), device=DEV) for k in (K, K, N))
    layer = Fp8Layer.pack(w, bias)

    def calls(x, stream=None):
        q = quantize(x, stream=stream)
        p = Fp8Layer.pack(w, bias, stream=stream)
        h, n = gated_norm(x, x, post="rms", stream=stream)
        _, c = gated_norm(x, out="fp8", stream=stream)
        g = gated_norm_backward(x, x, x, x, post="rms", weight=w[0], stream=stream)
        return [layer.forward(x, stream=stream), *layer.backward(dy, x, stream=stream), q.codes, q.scales,
                q.dequantize(stream=stream), p.codes, p.scales, p.codes_t, p.scales_t, h, n, c.codes, c.scales,
                g.dx, g.dy, g.weight]

    want, want2 = calls(x), calls(x2)
    torch.cuda.synchronize()
    side, cur = torch.cuda.Stream(), torch.cuda.default_stream()
    if other == "the default stream":
        side, cur = cur, side
        assert side.cuda_stream == 0
    cur.wait_stream(side)
    with torch.cuda.stream(cur):
        _busy()
        for _ in range(2):
            trash = [torch.empty_like(t) for t in want for _ in range(2)]
            for t in trash:
                t.fill_(3)
            del trash, t
        got = calls(x, side.cuda_stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        # read late, on the current stream, and freed before that
        _busy()
        late = [t.clone() for t in got]
        del got
        again = calls(x2, side.cuda_stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(late, want))
        assert all(torch.equal(a, b) for a, b in zip(again, want2))


def test_the_c_calls_refuse_a_small_workspace():
    layer = Fp8Layer.pack(torch.ones((64, 8192), device=DEV))
    x = torch.ones((64, 8192), device=DEV)
    need = B.asp_fp8_workspace_bytes(64, 64, 8192)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    y = torch.empty((64, 64), device=DEV)
    with pytest.raises(B.ASPError) as ei:
        B.asp_fp8_forward(x, 0, 8192, 64, 64, 8192, layer.codes, layer.scales, None, y, 0, ws, need - 1)
    assert ei.value.status == 5


def test_module_trains():
    """Fp8Linear under autograd gives Fp8Layer.backward's gradients; frozen and trainable."""
    from wam_asp_w4a4_amd.linear import Fp8Linear
    lin = torch.nn.Linear(300, 130).to(DEV)
    x = torch.randn((3, 40, 300), device=DEV, requires_grad=True)
    dy = torch.randn((3, 40, 130), device=DEV)
    layer = Fp8Layer.pack(lin.weight.detach(), lin.bias.detach())
    want = layer.backward(dy.view(120, 130), x.detach().view(120, 300))
    for trainable in (False, True):
        m = Fp8Linear.from_linear(lin, trainable=trainable)
        x.grad = lin.weight.grad = None
        y = m(x)
        assert torch.equal(y, layer.forward(x.detach().view(120, 300)).view(3, 40, 130))
        y.backward(dy)
        assert torch.equal(x.grad.view(120, 300), want[0])
        if trainable:
            assert torch.equal(lin.weight.grad, want[1]) and torch.equal(m.bias.grad, want[2])
        with torch.no_grad():
            assert torch.equal(m(x), y)
    with pytest.raises(RuntimeError, match="capture"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            m(x)
    torch.cuda.synchronize()
    assert torch.equal(m(x), y)


@pytest.mark.parametrize("M", [5, 150, 3000])
def test_float32_sums_are_a_choice_in_every_direction(M):
    """bf16 activations with a float32 y and dx: the sums of the float32 call on the same values."""
    from wam_asp_w4a4_amd.linear import Fp8Linear
    lin = torch.nn.Linear(1000, 700).to(DEV)
    x = torch.randn((M, 1000), device=DEV).bfloat16().requires_grad_()
    dy = torch.randn((M, 700), device=DEV).bfloat16()
    layer = Fp8Layer.pack(lin.weight.detach(), lin.bias.detach())
    want = layer.backward(dy.float(), x.detach().float())
    got = layer.backward(dy, x.detach(), dx_dtype="f32")
    assert got[0].dtype == torch.float32 and all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(layer.backward(dy.float(), dx_dtype="bf16")[0], layer.backward(dy)[0])
    for trainable in (False, True):
        m = Fp8Linear.from_linear(lin, trainable=trainable, y_dtype="f32")
        x.grad = None
        y = m(x)
        assert y.dtype == torch.float32 and torch.equal(y, layer.forward(x.detach().float()))
        with torch.no_grad():
            assert torch.equal(m(x), y)
        y.backward(dy.float())
        assert torch.equal(x.grad, want[0].bfloat16())
    m = Fp8Linear(weight=torch.nn.Parameter(lin.weight.detach().bfloat16()), y_dtype="f32")
    m(x).backward(dy.float())
    want = Fp8Layer.pack(m.weight.detach()).backward(dy.float(), x.detach().float())
    assert torch.equal(m.weight.grad, want[1].bfloat16())


def test_module_takes_broadcast_and_transposed_inputs():
    from wam_asp_w4a4_amd.linear import Fp8Linear
    m = Fp8Linear.from_linear(torch.nn.Linear(200, 70).to(DEV), trainable=True)
    x = torch.randn((1, 200), device=DEV, requires_grad=True)
    plain = x.detach().expand(40, 200).contiguous().requires_grad_()
    y = m(x.expand(40, 200))
    assert torch.equal(y, m(plain))
    dy = torch.randn((40, 70), device=DEV)
    y.backward(dy)
    m(plain).backward(dy)
    assert torch.allclose(x.grad, plain.grad.sum(0, keepdim=True), rtol=1e-5, atol=1e-5)
    z = torch.randn((200, 40), device=DEV)
    assert torch.equal(m(z.t()), m(z.t().contiguous()))


def test_offsets_past_32_bits():
    """Whole numbers, whose sums are exact: the far rows of a large call and the same rows alone."""
    def whole(M, K):
        return torch.randint(-4, 5, (M, K), dtype=torch.int8, device=DEV).bfloat16()

    M, N, K = 600_000, 130, 4000        # x and its codes past 2^31 elements
    x, dy = whole(M, K), whole(M, N)
    layer = Fp8Layer.pack(whole(N, K))
    y = layer.forward(x, "f32")
    assert torch.equal(y[-300:], layer.forward(x[-300:].contiguous(), "f32"))
    dx, dw, _ = layer.backward(dy, x)
    assert torch.equal(dx[-300:], layer.backward(dy[-300:].contiguous())[0])
    want = torch.zeros((N, K), device=DEV, dtype=torch.float64)
    for i in range(0, M, 100_000):
        want += (dy[i:i + 100_000].float().t() @ x[i:i + 100_000].float()).double()   # below 2^24
    assert torch.equal(dw.double(), want)
    assert torch.equal(quantize(x).dequantize("bf16")[-300:], x[-300:])
    del x, dy, y, dx, dw, want

    M, N, K = 70_000, 40_000, 130       # y past 2^31 elements
    x = whole(M, K)
    layer = Fp8Layer.pack(whole(N, K), backward=False)
    y = layer.forward(x, "f32")
    assert torch.equal(y[-300:], layer.forward(x[-300:].contiguous(), "f32"))
    y = layer.forward(x)
    assert torch.equal(y[-300:], layer.forward(x[-300:].contiguous()))


def test_one_row_of_the_longest_k():
    K = 1 << 20
    x = torch.randint(-2, 3, (40, K), dtype=torch.int8, device=DEV).bfloat16()
    w = torch.randint(-2, 3, (20, K), dtype=torch.int8, device=DEV).bfloat16()
    layer = Fp8Layer.pack(w, backward=False)
    want = x.float() @ w.float().t()     # whole numbers up to 2^22: exact in any order
    assert torch.equal(layer.forward(x, "f32"), want)
    assert torch.equal(layer.forward(x[:1], "f32"), want[:1])


def test_two_captured_calls_and_two_streams_share_a_layer():
    """Each call has a workspace of its own: graphs replayed at once and eager calls on two
    streams do not disturb each other."""
    layer = Fp8Layer.pack(torch.randn((1024, 1024), device=DEV), torch.randn(1024, device=DEV))
    xs = [torch.randn((M, 1024), device=DEV) for M in (200, 700)]
    want = [(layer.forward(x), layer.backward(x, x)) for x in xs]
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in xs]
    for x in xs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append((layer.forward(x), layer.backward(x, x)))
        graphs.append(graph)

    def same(a, b):
        return torch.equal(a[0], b[0]) and all(torch.equal(s, t) for s, t in zip(a[1], b[1]))

    for _ in range(5):
        torch.cuda.synchronize()
        eager = []
        for x, graph, stream in zip(xs, graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(outs, want))
        for x, stream in zip(xs, streams):
            with torch.cuda.stream(stream):
                eager.append((layer.forward(x), layer.backward(x, x)))
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(eager, want))
