"""8-bit integer quantisation and linear on the GPU: codes, scales and outputs to the last bit (the
sums are exact integers), at every cut, and the calls a serving loop makes."""
import numpy as np
import pytest
import torch

import gemv_dg_bf16_gb300 as dg
from tests import _ref_more as R

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _x(M, K, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, K), generator=g) * scale
    x[:, ::97] *= 17.0
    return x.to(BF)


def _w(N, K, seed):
    g = torch.Generator().manual_seed(seed)
    w = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int16).to(torch.int8)
    return w, torch.rand((N,), generator=g) * 1e-2 + 1e-4


def _bits(y):
    return y.cpu().view(torch.int16).numpy()


def _check(x, w, sw, **kw):
    y = dg.dg_gemv_i8_rowscale(x.cuda(), w.cuda(), sw.cuda(), **kw)
    want = R.i8_linear(R.f32(x), w.numpy(), sw.numpy())
    np.testing.assert_array_equal(_bits(y), want)
    return y


@pytest.mark.parametrize("M,K", [(1, 16), (3, 48), (2, 1024), (5, 1040), (1, 4096), (7, 4112), (4, 16400), (1300, 272),
                                 (1300, 4096), (1217, 1040), (2, 65552), (1, 140000), (20000, 32)])
def test_quantisation_to_the_bit(M, K):
    x = _x(M, K, M + K)
    q, s = dg.dg_quant_i8_rowscale(x.cuda())
    wq, ws = R.i8_codes(R.f32(x))
    np.testing.assert_array_equal(q.cpu().numpy(), wq)
    np.testing.assert_array_equal(s.cpu().numpy(), ws)


def test_quantisation_of_extremes():
    x = torch.zeros((9, 64), dtype=BF)
    x[1, 3] = float("inf")
    x[2, 4] = float("nan")
    x[2, 5] = 1.0
    x[3] = 3.3e38
    x[4, :2] = torch.tensor([2.0 ** -133, -2.0 ** -130])     # below the floor: codes 0
    x[5, :3] = torch.tensor([2.0 ** -100, -2.0 ** -101, 2.0 ** -120])
    x[6] = torch.arange(64) / 63 * 127                         # ties, and the largest itself
    x[7] = -1.0
    x[8, :4] = torch.tensor([64.0, 1.0, -3.0, 0.25])
    q, s = dg.dg_quant_i8_rowscale(x.cuda())
    wq, ws = R.i8_codes(R.f32(x))
    np.testing.assert_array_equal(q.cpu().numpy(), wq)
    np.testing.assert_array_equal(s.cpu().numpy(), ws)       # (NaN where NaN)
    assert q[0].abs().max() == 0 and s[0] == np.float32(2.0 ** -100) * (np.float32(1) / np.float32(127))
    assert q[8, :4].tolist() == [127, 2, -6, 0] and torch.isnan(s[1:3]).all() and q[1:3].abs().max() == 0


@pytest.mark.parametrize("M", [1, 2, 3, 8, 9, 16, 17, 32, 33, 64, 65, 100, 128, 129, 257, 512])
@pytest.mark.parametrize("N,K", [(1, 16), (129, 144), (300, 1040), (128, 4096)])
def test_linear_to_the_bit(M, N, K):
    _check(_x(M, K, M * 7 + N), *_w(N, K, N + K))


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (16, 4099, 2064), (5, 2050, 12288), (77, 4099, 1616), (200, 8208, 528), (512, 1283, 4096), (16, 20480, 4112), (31, 24576, 4096),
                                   (3, 17, 33008), (40, 260, 16384)])
def test_linear_of_ragged_and_long_shapes(M, N, K):
    _check(_x(M, K, M), *_w(N, K, N + K))


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 9, 16])
@pytest.mark.parametrize("N,K", [(1, 16), (7, 48), (129, 144), (300, 1040), (1300, 4096), (2050, 2064), (40, 12288)])
def test_every_family_gives_the_same_bits(M, N, K):
    x, (w, sw) = _x(M, K, M * 7 + N), _w(N, K, N + K)
    for variant, most in ((dg.DG_VAR_CC_WARP, 4), (dg.DG_VAR_TC, 512)):
        if M <= most:
            _check(x, w, sw, choice=dg.Choice.make(variant))


def test_tokens_without_room_are_refused():
    x, (w, sw) = _x(17, 64, 1), _w(8, 64, 2)
    for x, K, variant in ((x, 64, dg.DG_VAR_CC_WARP), (_x(5, 64, 1), 64, dg.DG_VAR_CC_WARP), (_x(4, 65536, 1), 65536, dg.DG_VAR_CC_WARP)):
        w, sw = _w(8, K, 2)
        with pytest.raises(dg.DGError) as e:
            dg.dg_gemv_i8_rowscale(x.cuda(), w.cuda(), sw.cuda(), choice=dg.Choice.make(variant))
        assert e.value.status == dg.DG_ERR_UNSUPPORTED_SHAPE
        _check(x, w, sw)


def test_every_cut_gives_the_same_bits():
    """Any cut of K and of the tokens, any stages."""
    for M, N, K in ((3, 260, 2064), (40, 384, 3088), (150, 130, 1296), (512, 1000, 400), (200, 20000, 160), (17, 40000, 1168)):
        x, (w, sw) = _x(M, K, M), _w(N, K, N)
        xc, wc, sc = x.cuda(), w.cuda(), sw.cuda()
        want = R.i8_linear(R.f32(x), w.numpy(), sw.numpy())
        ws = dg.workspace(dg.DG_OP_GEMV_I8, M, N, K)
        for tg in (0, 16, 32, 48, 64, 80, 112, 128):
            for ns in (0, 1, 2, 3, 5, 8):
                for st in (0, 2, 4):
                    if tg == 128 and M > 112 and ns > 1:
                        continue                                  # (no room for the sums of a split: refused)
                    y = dg.dg_gemv_i8_rowscale(xc, wc, sc, ws=ws, choice=dg.Choice.make(dg.DG_VAR_TC, st, tg, ns))
                    np.testing.assert_array_equal(_bits(y), want, err_msg=str((M, tg, ns, st)))
        assert dg.dg_device_status(ws) == 0


@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (64, 256, 128), (100, 257, 1040), (129, 130, 1296), (512, 1000, 400), (200, 20000, 160),
                                   (77, 4099, 2064), (300, 40000, 1168), (512, 20000, 2176)])
def test_pairs_of_ctas_give_the_same_bits(M, N, K):
    x, (w, sw) = _x(M, K, M), _w(N, K, N)
    xc, wc, sc = x.cuda(), w.cuda(), sw.cuda()
    want = R.i8_linear(R.f32(x), w.numpy(), sw.numpy())
    ws = dg.workspace(dg.DG_OP_GEMV_I8, M, N, K)
    for cut in ((0, 0, 0, 2), (6, 0, 1, 2), (0, 0, 0, 1), (0, 0, 1, 0), (0, 64, 0, 2), (0, 96, 1, 2), (0, 128, 0, 2)):
        if cut[1] > (M + 15) // 16 * 16:
            continue
        for _ in range(3):
            y = dg.dg_gemv_i8_rowscale(xc, wc, sc, ws=ws, choice=dg.Choice.make(dg.DG_VAR_TC, *cut))
            np.testing.assert_array_equal(_bits(y), want, err_msg=str(cut))
    assert dg.dg_device_status(ws) == 0


@pytest.mark.parametrize("K", [1024, 8192, 131072])
def test_largest_sums_are_exact(K):
    """All products of one sign at their largest: K * 127 * 128, past 2^24 from K = 1040 on, next to 2^31 at the longest."""
    x = torch.ones((3, K), dtype=BF)
    x[1] = -1.0
    x[2, 1::2] = -1.0
    w = torch.full((5, K), -128, dtype=torch.int8)
    w[1] = 127
    w[2, ::2] = 127
    w[3, 1:] = 0
    w[4, :K - 1] = 1
    _check(x, w, torch.tensor([1.0, 1e-3, 0.7, 3.0, 1e-9]))
    for ns in (1, 3, 8):
        _check(x, w, torch.tensor([1.0, 1e-3, 0.7, 3.0, 1e-9]), choice=dg.Choice.make(dg.DG_VAR_TC, 0, 0, ns))


def test_tokens_do_not_meet():
    """Non-finite and all-zero tokens, each in its own row only; every row's bits are those it has alone."""
    M, N, K = 37, 200, 1168
    x, (w, sw) = _x(M, K, 1), _w(N, K, 2)
    x[3, 5] = float("nan")
    x[11, K - 1] = float("-inf")
    x[20] = 0
    x[21] *= 1e30
    y = dg.dg_gemv_i8_rowscale(x.cuda(), w.cuda(), sw.cuda())
    assert torch.isnan(y[3]).all() and torch.isnan(y[11]).all() and (y[20] == 0).all()
    fine = [m for m in range(M) if m not in (3, 11)]
    np.testing.assert_array_equal(_bits(y)[fine], R.i8_linear(R.f32(x), w.numpy(), sw.numpy())[fine])
    for m in (0, 21, 36):
        one = dg.dg_gemv_i8_rowscale(x[m:m + 1].cuda(), w.cuda(), sw.cuda())
        assert torch.equal(one[0], y[m])


def test_scales_of_any_size():
    x, (w, _) = _x(4, 64, 5), _w(6, 64, 6)
    _check(x, w, torch.tensor([0.0, 1e-45, 3e38, -2.0, float("inf"), 1e-30]))
    _check((x.float() * 2.0 ** -110).to(BF), w, torch.tensor([1.0, 1e10, 1e30, 1e-10, 1e-38, 2.0]))


def test_weights_quantised_here_give_the_linear_of_their_values():
    M, N, K = 6, 150, 512
    x, w = _x(M, K, 8), _x(N, K, 9, 0.05)
    q, s = dg.dg_quant_i8_rowscale(w.cuda())
    y = dg.dg_gemv_i8_rowscale(x.cuda(), q, s).float().cpu().double()
    ref = x.double() @ w.double().T
    # each operand within half a code of its row's scale, on both sides, and the output's rounding
    ax, aw = x.double().abs().amax(1) / 127, w.double().abs().amax(1) / 127
    bound = (0.5 * ax[:, None] * w.double().abs().sum(1)[None] + 0.5 * aw[None] * x.double().abs().sum(1)[:, None]
             + 0.25 * K * ax[:, None] * aw[None]) * (1 + 2.0 ** -20) + ref.abs() * 2.0 ** -7
    assert ((y - ref).abs() <= bound).all()


def test_streams_graph_and_shared_workspace():
    M, N, K = 4, 256, 1024
    (w, sw) = _w(N, K, 3)
    xs = [_x(M, K, 20 + i) for i in range(4)]
    want = [R.i8_linear(R.f32(x), w.numpy(), sw.numpy()) for x in xs]
    wc, sc = w.cuda(), sw.cuda()
    ws = dg.workspace(dg.DG_OP_GEMV_I8, M, N, K)
    x = torch.empty((M, K), dtype=BF, device="cuda")
    ys = [torch.empty((M, N), dtype=BF, device="cuda") for _ in xs]
    x.copy_(xs[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = dg.dg_gemv_i8_rowscale(x, wc, sc, stream=side)
    side.synchronize()
    np.testing.assert_array_equal(_bits(y), want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.dg_gemv_i8_rowscale(x, wc, sc, y=ys[0], ws=ws)
        x.neg_()
        dg.dg_gemv_i8_rowscale(x, wc, sc, y=ys[1], ws=ws)
    for i in (1, 2, 3):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(_bits(ys[0]), want[i])
        assert torch.equal(ys[1], -ys[0])
    xd = [t.cuda() for t in xs]
    for i in range(4):
        dg.dg_gemv_i8_rowscale(xd[i], wc, sc, y=ys[i], ws=ws)
    torch.cuda.synchronize()
    for i in range(4):
        np.testing.assert_array_equal(_bits(ys[i]), want[i])
    assert dg.dg_device_status(ws) == 0


def test_weights_written_in_front_of_the_linear():
    """Weights quantised right ahead of the linear that reads them, over and over in one buffer."""
    M, N, K = 2, 2048, 1024
    x = _x(M, K, 1).cuda()
    q = torch.empty((N, K), dtype=torch.int8, device="cuda")
    s = torch.empty((N,), device="cuda")
    src = [(_x(N, K, 30 + i)).cuda() for i in range(6)]
    ws = dg.workspace(dg.DG_OP_GEMV_I8, M, N, K)
    want = []
    for w in src:
        a, b = dg.dg_quant_i8_rowscale(w)
        torch.cuda.synchronize()
        want.append(dg.dg_gemv_i8_rowscale(x, a, b))
        torch.cuda.synchronize()
    got = []
    for w in src:
        dg.dg_quant_i8_rowscale(w, q=q, s=s)
        got.append(dg.dg_gemv_i8_rowscale(x, q, s, ws=ws))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_sweep_and_table(tmp_path):
    M, N, K = 2, 256, 512
    path = str(tmp_path / "t.json")
    dg.dg_sweep([(dg.DG_OP_GEMV_I8, M, N, K, 0)], path, reps=3)
    x, (w, sw) = _x(M, K, 1), _w(N, K, 2)
    dg.dg_table_load(path)
    try:
        assert dg.dg_select(dg.DG_OP_GEMV_I8, M, N, K).from_table == 1
        _check(x, w, sw)
    finally:
        dg.dg_table_clear()


def test_batch_invariant_mode_changes_no_bits():
    x, (w, sw) = _x(20, 2048, 1), _w(300, 2048, 2)
    dg.dg_set_numerics(dg.DG_NUMERICS_BATCH_INVARIANT)
    try:
        _check(x, w, sw)
    finally:
        dg.dg_set_numerics(dg.DG_NUMERICS_FASTEST)


def test_bad_choices_are_refused():
    x, (w, sw) = _x(2, 64, 1), _w(8, 64, 2)
    xc, wc, sc = x.cuda(), w.cuda(), sw.cuda()
    for bad in ((dg.DG_VAR_CC_BULK,), (dg.DG_VAR_CC_WARP, 4, 8), (dg.DG_VAR_TC, 1), (dg.DG_VAR_TC, 3), (dg.DG_VAR_TC, 10), (dg.DG_VAR_TC, 0, 40), (dg.DG_VAR_TC, 0, 144), (dg.DG_VAR_TC, 0, 0, 9), (dg.DG_VAR_TC, 0, 0, -1), (dg.DG_VAR_TC, 0, -16),
                (dg.DG_VAR_MMA, 1), (dg.DG_VAR_TC, 0, 0, 0, 3), (dg.DG_VAR_TC, 0, 0, 0, 0, 1), (dg.DG_VAR_TC, 4, 0, 0, 2),
                (dg.DG_VAR_TC, 0, 48, 0, 2), (dg.DG_VAR_TC, 0, 0, 2, 2)):
        with pytest.raises(dg.DGError) as e:
            dg.dg_gemv_i8_rowscale(xc, wc, sc, choice=dg.Choice.make(*bad))
        assert e.value.status == dg.DG_ERR_BAD_VARIANT, bad
    _check(x, w, sw)
