"""The gated projection and the adapters at sizes where a CTA takes several tiles, where the adapters' gradients run on the
side stream, where K is split over eight CTAs, and at the sizes of large layers (sampled rows)."""
import numpy as np
import pytest
import torch

import oracle as O
from nvfp4_bit_microscaled_b200 import api, synth
from tests import _nvfp4_ref as R
from tests import test_gpu_gated as D
from tests import test_gpu_lora as G
from tests import test_gpu_projections as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from nvfp4_bit_microscaled_b200 import build
    build.build()
    api.read_device_error(clear=True)
    yield
    torch.cuda.synchronize()
    assert api.read_device_error(clear=True) == 0


# ------------------------------------------------------------------ several tiles for each CTA
@pytest.mark.parametrize("M,C,F", [(2100, 64, 4096), (700, 320, 7680)])   # 288 and 180 tiles for 74 pairs
def test_gated_tiles_in_turn(M, C, F):
    x = D._activations(M, C, M)
    w, wq = D._weight(2 * F, C, C)
    xq, _ = api.quantize(x.cuda(), api.ROW, api.amax(x.cuda()))
    GU, tgu, H, th = D._gated_ref(R.decode_bf16(x, "row"), R.decode_bf16(w, "2d"), "silu")
    first = None
    for _ in range(3):
        gu, amax = torch.zeros(M, 2 * F, dtype=torch.bfloat16, device="cuda"), torch.full((1,), 9e9, device="cuda")
        h = api.gated_gemm(xq, wq, H=torch.zeros(M, F, dtype=torch.bfloat16, device="cuda"), GU=gu, amax_out=amax)
        if first is None:
            R.assert_within(R.f64(gu), GU, tgu, "G | U")
            R.assert_within(R.f64(h), H, th, "H")
            first = (h, gu)
        assert float(amax) == float(h.float().abs().max())
        assert torch.equal(h, first[0]) and torch.equal(gu, first[1])
    assert torch.equal(api.gated_gemm(xq, wq), first[0])


@pytest.mark.parametrize("T,C,F", [(256, 64, 10240), (1152, 128, 2304)])   # 320 and 324 tiles for 296 CTAs
@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_gated_gradient_tiles_in_turn(T, C, F, name):
    x, w, dh = D._activations(T, C, T), synth.weights(2 * F, C, F), synth.gradients(T, F, 9)
    ws = api.GatedWorkspace(T, C, F, "cuda")
    _, gu = api.gated_fwd(x.cuda(), w.cuda(), ws, D.ACTS[name])
    seed, first = 2 ** 40 + 7, None
    for _ in range(3):
        got = api.gated_bwd(dh.cuda(), gu, ws, seed, D.ACTS[name])
        row, col = ws.tensor("dy_row"), ws.tensor("dy_col")
        got = (*got, row.data.clone(), row.scales.clone(), col.data.clone(), col.scales.clone())
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(got, first))
    d = D._grad_ref(R.f64(dh), R.f64(gu), name).astype(np.float32)
    cols = np.arange(T // 16)[None, :] * 2 * F + np.arange(2 * F)[:, None]
    D._same_codes(row, *R.quantize_f32(d, seed, 0, np.arange(d.size // 16).reshape(T, -1))[:2], "row copy")
    D._same_codes(col, *R.quantize_f32(R.rht_columns(d), seed, 1, cols)[:2], "column copy")
    for y, a, b in ((got[0], row, "w_col"), (got[1], col, "x_col")):
        want, tol = D._product(R.decode(a), R.decode(ws.tensor(b)))
        R.assert_within(R.f64(y), want, tol + (R.BF16 * (np.abs(want) + tol) if y.dtype == torch.bfloat16 else 0), b)


def _check_adapters(b, x, dy, seed, repeats=3):
    """lora_fwd and lora_bwd of the batch against the 64-bit forms, the same bytes each time: (Y, V, dX, dA, dB)."""
    n, A, B = b["n"], R.f64(b["A"]), R.f64(b["B"])
    first = None
    for _ in range(repeats):
        out = [torch.full((b["T"], w), 7.0, dtype=torch.bfloat16, device="cuda") for w in (b["cout"], b["cin"])]
        V = torch.full((b["T"], b["rank"]), 3.0, device="cuda")
        api.lora_fwd(x, b["row"], b["ad"], *b["seg"], Y=out[0], V=V)
        _, dA, dB = api.lora_bwd(dy, x, V, b["col"], b["ad"], *b["seg"], seed, dX=out[1])
        got = (out[0], V, out[1], dA, dB)
        first = first or got
        assert all(torch.equal(p, q) for p, q in zip(got, first))
    xs, dys = R.f64(x), R.f64(dy)
    xs[n:], dys[n:] = 0, 0
    sides = ((out[0], x, xs, A, B, b["row"], {}),
             (out[1], dy, dys, B.transpose(0, 2, 1), A.transpose(0, 2, 1), b["col"], dict(sr=True, seed=seed)))
    for y, data, d, one, two, weight, how in sides:
        codes = R.decode_bf16(data[:n].cpu().contiguous(), "row", **how)
        want, tol = P._projected(b, d, one, two, codes, R.decode(weight), P.TERMS)
        R.assert_within(R.f64(y)[:n], want, tol, "forward" if not how else "backward")
        assert (y[n:] == 7.0).all()
    # dA and dB: U and V in 16 bits of FP32 sums, FP32 accumulation, BF16
    u, ua, _, _ = G._low_rank(b, dys, B.transpose(0, 2, 1), A.transpose(0, 2, 1))
    v = R.f64(V)
    for i in range(b["count"]):
        rows = np.concatenate([np.arange(lo, hi) for lo, hi, k in zip(b["ptr"], b["ptr"][1:], b["ids"]) if k == i] or [[]]).astype(int)
        want = u[rows].T @ xs[rows]
        tol = ((P.TERMS + R.GEMM_REL) * np.abs(u[rows]) + G.F32_SUM * ua[rows]).T @ np.abs(xs[rows])
        R.assert_within(R.f64(dA[i]), want, tol + R.BF16 * (np.abs(want) + tol), f"dA {i}")
        want = dys[rows].T @ v[rows]
        tol = (P.TERMS + R.GEMM_REL) * (np.abs(dys[rows]).T @ np.abs(v[rows]))
        R.assert_within(R.f64(dB[i]), want, tol + R.BF16 * (np.abs(want) + tol), f"dB {i}")
    return got


LENGTHS = [300, 1, 255, 256, 200, 100, 700, 512, 277]
IDS = [-1, 0, 1, -1, 2, 0, -1, 1, 3]   # tiles with no slab, one and several, in turn


@pytest.mark.parametrize("cin,cout,rank", [(64, 4096, 40), (4096, 64, 16), (192, 2624, 128)])
@pytest.mark.parametrize("large", [1.0, 3e33])   # the third adapter out of proportion: its tiles take no slabs
def test_adapter_tiles_in_turn(cin, cout, rank, large):
    b = G._make(LENGTHS, IDS, cin, cout, rank, 4, 9, seed=3)
    b["scale"][2] *= large
    b["ad"] = api.LoraAdapters(b["ad"].A, b["ad"].B, b["scale"].cuda())
    _check_adapters(b, b["X"], b["dY"], 11)


# ------------------------------------------------------------------ K split over eight CTAs
@pytest.mark.parametrize("lengths,ids,rank", [([300, 1, 0, 211], [1, 0, 1, -1], 16), ([129], [0], 128), ([40, 100, 77, 3], [0, 1, 2, -1], 72)])
def test_first_low_rank_product_split_over_a_cluster(lengths, ids, rank):
    b = G._make(lengths, ids, 4160, 4224, rank, 3, 5, seed=rank)
    _check_adapters(b, b["X"], b["dY"], 2, repeats=2)


# ------------------------------------------------------------------ gradients on the side stream
def test_adapter_gradients_beside_the_product():
    # T (Cin + Cout) rank above 2^28: dA and dB run on the library's second stream beside dX's product
    lengths, T, C, rank = [900, 0, 33, 800, 1, 560], 2300, 512, 128
    assert T * 2 * C * rank > 2 ** 28
    b = G._make(lengths, [0, 2, 1, -1, 2, 0], C, C, rank, 3, 6, seed=9)
    c = dict(b)   # other ranges in the same tensors
    c["ptr"], c["ids"] = [0, 10, 700, 700, 1500, 2299, 2300], [1, 0, 0, 2, 2, -1]
    c["n"], c["seg"] = 2300, (G._i32(c["ptr"]), G._i32(c["ids"]))
    x, dy = b["X"].clone(), b["dY"].clone()
    x[2294:], dy[2294:] = 0.5, 1e-3
    want = [_check_adapters(b, x, dy, 4), _check_adapters(c, x, dy, 4)]

    def run(seg, ws, out):
        api.lora_fwd(x, b["row"], b["ad"], *seg, Y=out[0], V=out[1], ws=ws[0])
        api.lora_bwd(dy, x, out[1], b["col"], b["ad"], *seg, 4, dX=out[2], dA=out[3], dB=out[4], ws=ws[1])

    def fresh():
        return ((api.LoraWorkspace(b["T"], 6, b["ad"], "cuda"), api.LoraWorkspace(b["T"], 6, b["ad"], "cuda", backward=True)),
                [torch.full_like(t, 3.0 if i == 1 else 7.0) for i, t in enumerate(want[0])])

    # two streams at once (they share the side stream), one workspace each
    streams, kept = [torch.cuda.Stream(), torch.cuda.Stream()], []
    torch.cuda.synchronize()
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            ws, out = fresh()
            run((b, c)[i % 2]["seg"], ws, out)
            kept.append((out, ws))
    torch.cuda.synchronize()
    for i, (out, _) in enumerate(kept):
        assert all(torch.equal(p, q) for p, q in zip(out, want[i % 2]))
    # captured twice in a row, replayed with either batch's ranges
    seg = tuple(t.clone() for t in b["seg"])
    ws, out = fresh()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(seg, ws, out)
        run(seg, ws, out)
    for i in (1, 0, 1):
        for t, s in zip(seg, (b, c)[i]["seg"]):
            t.copy_(s)
        for k, t in enumerate(out):
            t.fill_(3.0 if k == 1 else 7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want[i]))


# ------------------------------------------------------------------ large layers, sampled rows
def _sample(T, rng, always):
    return np.unique(np.concatenate([rng.integers(0, T, 24), always])).astype(np.int64)


@pytest.mark.parametrize("T", [1, 48, 1777])
def test_fullsize_gated_serving(T):
    C, F = 5120, 10240
    x = D._activations(T, C, T)
    w = synth.weights(2 * F, C, 1, device="cuda")
    wq = api.quantize(w, api.TWO_D, api.amax(w), col_out=False)[0]
    h = api.gated_apply(x.cuda(), wq)
    rows = _sample(T, np.random.default_rng(T), [0, T - 1])
    a = O.amax(x)
    c, s = O.quantize_row(x[rows].contiguous(), a)
    _, _, H, th = D._gated_ref(R.decode_parts(c, s, O.global_scales(a)[1]), R.decode(wq), "silu")
    R.assert_within(R.f64(h[torch.from_numpy(rows).cuda()]), H, th, "H")


@pytest.mark.parametrize("T", [64, 4100])
def test_fullsize_adapters(T):
    cin, cout, rank, count = 8192, 8192, 64, 8
    lengths = [1] * T if T == 64 else [1000, 1, 2000, 0, 37, 1062]
    b = G._make(lengths, [i % 9 - 1 for i in range(len(lengths))], cin, cout, rank, count, 0, seed=1)
    V = torch.zeros(T, rank, device="cuda")
    Y = api.lora_fwd(b["X"], b["row"], b["ad"], *b["seg"], V=V)
    dX, dA, dB = api.lora_bwd(b["dY"], b["X"], V, b["col"], b["ad"], *b["seg"], 6)
    x, dy = b["x"][:, :cin].contiguous(), b["dy"][:, :cout].contiguous()
    A, B = R.f64(b["A"]), R.f64(b["B"])
    ids = np.repeat(b["ids"], lengths)
    rows = _sample(T, np.random.default_rng(2), [0, T - 1])
    at = torch.from_numpy(rows).cuda()
    for got, data, one, two, weight, sr in ((Y, x, A, B, b["row"], False), (dX, dy, B.transpose(0, 2, 1), A.transpose(0, 2, 1), b["col"], True)):
        a, d = O.amax(data), R.f64(data[rows])
        if sr:   # the draws are those of the rows' places in the whole tensor
            c, s = zip(*[O.quantize_row(data[r:r + 1].contiguous(), a, sr=True, seed=6, row0=int(r)) for r in rows])
            c, s = np.concatenate(c), np.concatenate(s)
        else:
            c, s = O.quantize_row(data[rows].contiguous(), a)
        part = dict(b, T=len(rows), n=len(rows), ptr=list(range(len(rows) + 1)), ids=ids[rows].tolist())
        want, tol = P._projected(part, d, one, two, R.decode_parts(c, s, O.global_scales(a)[1]), R.decode(weight), P.TERMS)
        R.assert_within(R.f64(got[at]), want, tol, "backward" if sr else "forward")
    own = np.flatnonzero(ids == 2)
    u, v, xs, ds = b["scale"][2].double().numpy() * (R.f64(dy)[own] @ B[2]), R.f64(V)[own], R.f64(x)[own], R.f64(dy)[own]
    ua = float(b["scale"][2]) * (np.abs(ds) @ np.abs(B[2]))
    cols = np.arange(0, cin, 97)
    want = u.T @ xs[:, cols]
    tol = ((P.TERMS + R.GEMM_REL) * np.abs(u) + G.F32_SUM * ua).T @ np.abs(xs[:, cols])
    R.assert_within(R.f64(dA[2])[:, cols], want, tol + R.BF16 * (np.abs(want) + tol), "dA")
    want = ds[:, cols].T @ v
    tol = (P.TERMS + R.GEMM_REL) * (np.abs(ds[:, cols]).T @ np.abs(v))
    R.assert_within(R.f64(dB[2])[cols], want, tol + R.BF16 * (np.abs(want) + tol), "dB")


def test_fullsize_gated_training():
    T, C, F, seed = 4096, 2560, 10240, 77
    x, w = D._activations(T, C, 1), synth.weights(2 * F, C, 2, device="cuda")
    dh = synth.gradients(T, F, 3)
    ws = api.GatedWorkspace(T, C, F, "cuda")
    h, gu = api.gated_fwd(x.cuda(), w, ws)
    dX, dW = api.gated_bwd(dh.cuda(), gu, ws, seed, dw_dtype=api.OUT_BF16)
    rng = np.random.default_rng(4)
    rows = _sample(T, rng, [0, T - 1])
    at = torch.from_numpy(rows).cuda()
    a = O.amax(x)
    c, s = O.quantize_row(x[rows].contiguous(), a)
    GU, tgu, H, th = D._gated_ref(R.decode_parts(c, s, O.global_scales(a)[1]), R.decode(ws.tensor("w_row")), "silu")
    R.assert_within(R.f64(gu[at]), GU, tgu, "G | U")
    R.assert_within(R.f64(h[at]), H, th, "H")
    # the gradients' row copy: the row of the largest gradient is among the sampled ones, so that they share its scale
    g, u = gu[:, :F].double(), gu[:, F:].double()
    sig = torch.sigmoid(g)
    d = torch.cat([dh.cuda().double() * u * (sig * (1 + g * (1 - sig))), dh.cuda().double() * g * sig], 1)
    rows = _sample(T, rng, [int(d.abs().amax(1).argmax()), T - 1])
    dr = d[torch.from_numpy(rows).cuda()].float().cpu().numpy()
    q = ws.tensor("dy_row")
    codes, sf, dec = R.quantize_f32(dr, seed, 0, rows[:, None] * (2 * F // 16) + np.arange(2 * F // 16)[None, :])
    assert abs(float(q.global_scale) / float(dec) - 1) < 2.0 ** -18
    got_codes, got_sf = R.codes_of(q)[rows], R.scales_of(q)[rows]
    assert (got_codes != codes).sum() <= 4 + 16 * (1 + codes.size / 16 / 2 ** 14) + codes.size / 2 ** 14
    assert (got_sf != sf).sum() <= 1 + codes.size / 16 / 2 ** 12
    # the products of the copies as stored
    want, tol = D._product(R.decode_parts(got_codes, got_sf, float(q.global_scale)), R.decode(ws.tensor("w_col")))
    R.assert_within(R.f64(dX[torch.from_numpy(rows).cuda()]), want, tol + R.BF16 * (np.abs(want) + tol), "dX")
    q = ws.tensor("dy_col")
    some = np.sort(rng.choice(2 * F, 64, replace=False))
    part = R.decode_parts(R.codes_of(q)[some], R.scales_of(q)[some], float(q.global_scale))
    want, tol = D._product(part, R.decode(ws.tensor("x_col")))
    R.assert_within(R.f64(dW[torch.from_numpy(some).cuda()]), want, tol + R.BF16 * (np.abs(want) + tol), "dW")
