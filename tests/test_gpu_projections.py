"""The gated projection and the adapters where their kernels meet: clusters, overlapping launches, the side stream, many
tiles for each CTA, and the ends of the value range."""
import numpy as np
import pytest
import torch

import oracle as O
from nvfp4_bit_microscaled_b200 import api, synth
from tests import _nvfp4_ref as R
from tests import test_gpu_lora as G

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


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _copies(w):
    return api.quantize(w, api.TWO_D, api.amax(w))


@pytest.mark.parametrize("T,C", [(2, 256), (40, 512), (100, 1088)])
def test_few_rows_quantizer_clusters_under_load(T, C):
    # clusters of 1, 8 and 16 CTAs take X's amax together; beside them other streams keep the SMs busy, so that the
    # CTAs of a cluster begin apart: the same bytes every time
    w = synth.weights(512, C, 1).cuda()
    row, _ = _copies(w)
    ad = api.LoraAdapters((torch.randn(2, 16, C) / 16).bfloat16().cuda(), torch.randn(2, 512, 16).bfloat16().cuda(),
                          torch.ones(2, device="cuda"))
    seg = _i32([0, T // 2, T]), _i32([1, 0])
    xs = [synth.activations(T, C, 10 + i, outlier_scale=20.0 * (i + 1)).cuda() for i in range(3)]
    want = [(api.gated_apply(x, row), api.lora_fwd(x, row, ad, *seg)) for x in xs]
    torch.cuda.synchronize()
    streams, noise, got = [torch.cuda.Stream() for _ in range(3)], torch.randn(2048, 2048, device="cuda"), []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for i in range(60):
        with torch.cuda.stream(streams[2]):
            noise = noise * 0.999
        with torch.cuda.stream(streams[i % 2]):
            got.append((api.gated_apply(xs[i % 3], row), api.lora_fwd(xs[i % 3], row, ad, *seg)))
    torch.cuda.synchronize()
    for i, (h, y) in enumerate(got):
        assert torch.equal(h, want[i % 3][0]) and torch.equal(y, want[i % 3][1])


@pytest.mark.parametrize("ptr,rows", [([0, 1000, 100, 900], 1000), ([0, 900, 130, 890, 140, 880], 900),
                                      ([0, 2500, 0, 2400, 3, 2000, 500], 2500), ([700, 0, 700, 0, 700], 700)])
def test_overlapping_ranges_share_numbers_of_blocks(ptr, rows):
    # ranges that decrease: several requests claim the same 128-row items of the first low-rank product, which a cluster
    # works on together (K = 4096: eight CTAs).  The numbers are wrong, but nothing hangs and nothing out of the batch
    # is written
    cin, cout, S = 4096, 128, len(ptr) - 1
    row, col = _copies(synth.weights(cout, cin, 1).cuda())
    g = torch.Generator().manual_seed(2)
    ad = api.LoraAdapters((torch.randn(3, 16, cin, generator=g) / 64).bfloat16().cuda(),
                          torch.randn(3, cout, 16, generator=g).bfloat16().cuda(), torch.ones(3, device="cuda"))
    x, dy = synth.activations(rows, cin, 3).cuda(), synth.gradients(rows, cout, 4).cuda()
    seg = _i32(ptr), _i32([i % 4 - 1 for i in range(S)])
    Y = torch.full((rows + 64, cout), 7.0, dtype=torch.bfloat16, device="cuda")
    dX = torch.full((rows + 64, cin), 7.0, dtype=torch.bfloat16, device="cuda")
    V = torch.zeros(rows + 64, 16, device="cuda")
    V[rows:] = 7.0
    for _ in range(5):
        api.lora_fwd(x, row, ad, *seg, Y=Y[:rows], V=V[:rows])
        api.lora_bwd(dy, x, V[:rows].clone(), col, ad, *seg, 1, dX=dX[:rows])
        torch.cuda.synchronize()
        assert api.read_device_error(clear=True) == 0
        assert (Y[rows:] == 7.0).all() and (dX[rows:] == 7.0).all() and (V[rows:] == 7.0).all()


@pytest.mark.parametrize("rows", [130, 300, 1500])
@pytest.mark.parametrize("lengths", ["one", "many", "none"])
def test_zero_batches_after_a_flagged_one(rows, lengths):
    # a batch of zeros has no maximum to record; the NaN that the batch before left in the same workspace is not its own
    cin, cout, S = 256, 192, 40
    row, _ = _copies(synth.weights(cout, cin, 1).cuda())
    ad = api.LoraAdapters(torch.randn(2, 16, cin).bfloat16().cuda(), torch.randn(2, cout, 16).bfloat16().cuda(),
                          torch.ones(2, device="cuda"))
    n = 0 if lengths == "none" else rows
    at = [min(n, 3 * i) for i in range(S)] + [n] if lengths == "many" else [0] * S + [n]
    seg, ws = (_i32(at), _i32([i % 3 - 1 for i in range(S)])), api.LoraWorkspace(rows, S, ad, "cuda")
    full = (_i32([0] * S + [rows]), seg[1])
    zero, bad = torch.zeros(rows, cin, dtype=torch.bfloat16, device="cuda"), synth.activations(rows, cin, 2).cuda()
    bad[7, 3] = float("nan")
    Y, Z = (torch.full((rows, cout), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for _ in range(20):
        api.lora_fwd(bad, row, ad, *full, Y=Y, ws=ws)
        Z.fill_(7.0)
        api.lora_fwd(zero, row, ad, *seg, Y=Z, ws=ws)
        assert Y.isnan().all() and (Z[:n] == 0).all() and (Z[n:] == 7.0).all()


@pytest.mark.parametrize("lengths,rank,cin,cout", [([1] * 20, 16, 320, 256), ([60, 40], 128, 192, 256),
                                                   ([1] * 190, 16, 128, 192), ([150, 3, 200], 32, 1088, 320)])
def test_adapters_alternate_in_one_workspace(lengths, rank, cin, cout):
    # what a launch makes for the next ones (transposed adapters, rows of each adapter, the operand's scale) is written
    # anew in each call of a captured chain: every call gives what it gives alone
    T, S = sum(lengths), len(lengths)
    row, col = _copies(synth.weights(cout, cin, 1).cuda())
    sets = []
    for i in range(3):
        g = torch.Generator().manual_seed(i)
        ad = api.LoraAdapters((torch.randn(130, rank, cin, generator=g) * 0.1).bfloat16().cuda(),
                              (torch.randn(130, cout, rank, generator=g) * 0.1).bfloat16().cuda(),
                              (torch.rand(130, generator=g) + 0.5).cuda())
        seg = (_i32(np.concatenate([[0], np.cumsum(lengths)]).tolist()),
               torch.randint(-1, 130, (S,), generator=g, dtype=torch.int32).cuda())
        x, dy = synth.activations(T, cin, 5 + i).cuda(), (synth.gradients(T, cout, 8 + i) * 10.0 ** (2 * i)).cuda()
        out = dict(Y=torch.zeros(T, cout, dtype=torch.bfloat16, device="cuda"), V=torch.zeros(T, rank, device="cuda"),
                   dX=torch.zeros(T, cin, dtype=torch.bfloat16, device="cuda"), dA=torch.zeros_like(ad.A), dB=torch.zeros_like(ad.B))
        sets.append((ad, seg, x, dy, out))
    spaces = api.LoraWorkspace(T, S, sets[0][0], "cuda"), api.LoraWorkspace(T, S, sets[0][0], "cuda", backward=True)

    def step(ad, seg, x, dy, o):
        api.lora_fwd(x, row, ad, *seg, Y=o["Y"], V=o["V"], ws=spaces[0])
        api.lora_bwd(dy, x, o["V"], col, ad, *seg, 3, dX=o["dX"], dA=o["dA"], dB=o["dB"], ws=spaces[1])

    want = []
    for s in sets:
        step(*s)
        torch.cuda.synchronize()
        want.append({k: v.clone() for k, v in s[4].items()})
        assert all(v.float().abs().max() > 0 for v in want[-1].values())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for s in sets:
            step(*s)
    for _ in range(5):
        for s in sets:
            for v in s[4].values():
                v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for s, w in zip(sets, want):
            for k, v in s[4].items():
                assert torch.equal(v, w[k]), k


def _projected(b, x, first, second, codes, weight, terms):
    """Wanted rows and their bound: the quantized product (FP32 accumulation), the low-rank product of V in `terms`
    roundings' accuracy (FP32 accumulation, V's own FP32 sum), one rounding to BF16."""
    n = b["n"]
    _, va, low, la = G._low_rank(b, x, first, second)
    lva = np.zeros_like(low)
    for lo, hi, i in zip(b["ptr"], b["ptr"][1:], b["ids"]):
        if 0 <= i < b["count"]:
            lva[lo:hi] = va[lo:hi] @ np.abs(second[i]).T
    want = codes @ weight.T + low[:n]
    tol = R.GEMM_REL * (np.abs(codes) @ np.abs(weight).T) + (terms + R.GEMM_REL) * la[:n] + G.F32_SUM * lva[:n]
    return want, tol + R.BF16 * (np.abs(want) + tol)


# V is summed in FP32.  Few rows keep it so; the tiles take it as two BF16 terms, the second a rounding of what the
# first leaves: 2^-8 of 2^-8
TERMS = 2.0 ** -16


@pytest.mark.parametrize("zero_weight", [False, True])
@pytest.mark.parametrize("case", [2, 4, 5, 8, 9, 10, 11, 14, 16, 17, 20, 23])
def test_the_low_rank_product_is_rounded_once(case, zero_weight):
    b = G._make(*G.CASES[case], seed=40 + case)
    n, cin, cout = b["n"], b["cin"], b["cout"]
    if zero_weight:
        b["row"], b["col"] = _copies(torch.zeros(cout, cin, dtype=torch.bfloat16, device="cuda"))
    x, dy = R.f64(b["x"][:, :cin]), R.f64(b["dy"][:, :cout])
    x[n:], dy[n:] = 0, 0
    A, B = R.f64(b["A"]), R.f64(b["B"])
    V = torch.zeros(b["T"], b["rank"], device="cuda")
    Y = api.lora_fwd(b["X"], b["row"], b["ad"], *b["seg"], V=V)
    codes = R.decode_bf16(b["x"][:n, :cin].contiguous(), "row")
    want, tol = _projected(b, x, A, B, codes, R.decode(b["row"]), TERMS)
    R.assert_within(R.f64(Y)[:n], want, tol, "Y")
    dX, _, _ = api.lora_bwd(b["dY"], b["X"], V, b["col"], b["ad"], *b["seg"], 5)
    codes = R.decode_bf16(b["dy"][:n, :cout].contiguous(), "row", sr=True, seed=5)
    want, tol = _projected(b, dy, B.transpose(0, 2, 1), A.transpose(0, 2, 1), codes, R.decode(b["col"]), TERMS)
    R.assert_within(R.f64(dX)[:n], want, tol, "dX")


EXTREMES = {   # scales of x (or dy), w, the last adapter's scale, its B (forward) or A (backward)
    "product 1e-34": (1e-17, 1e-17, 1.0, 1.0),
    "product 1e-38": (1e-19, 1e-19, 1.0, 1.0),
    "decode scale 0": (1e-24, 1e-25, 1.0, 1.0),
    "subnormal scale": (1.0, 2e-34, 1.0, 1.0),   # 2688 / max|W| is finite, the decode scale max|W| / 2688 no normal number
    "large adapter": (1.0, 1.0, 3e33, 1.0),
    "large by small": (1.0, 1.0, 3e35, 1e-33),
}


@pytest.mark.parametrize("name", EXTREMES)
@pytest.mark.parametrize("lengths,ids,cin,cout,rank,count,pad", [
    ([129], [0], 128, 64, 16, 1, 0),
    ([300, 1, 0, 211], [1, 0, 1, -1], 576, 320, 128, 2, 17),
    ([200, 56, 300, 3], [0, 0, 1, -1], 192, 832, 40, 2, 4),      # the last adapter in the later tiles only
    ([70], [0], 128, 192, 128, 1, 3),
    ([1] * 190, [i % 131 - 1 for i in range(190)], 128, 192, 8, 130, 0),
])
def test_low_rank_sums_where_the_decode_scale_is_small(name, lengths, ids, cin, cout, rank, count, pad):
    # V divided by the quantized product's decode scale leaves FP32's range although every output is inside it
    sx, sw, ss, se = EXTREMES[name]
    b = G._make(lengths, ids, cin, cout, rank, count, pad, seed=len(lengths))
    n = b["n"]
    b["x"], b["dy"] = (b["x"].float() * sx).bfloat16(), (b["dy"].float() * sx).bfloat16()
    b["scale"][-1] *= ss
    w = (b["w"].float() * sw).bfloat16().cuda()
    row, col = _copies(w)
    V = torch.zeros(b["T"], rank, device="cuda")
    for forward in (True, False):
        A, B = b["A"].clone(), b["B"].clone()
        (B if forward else A)[-1] *= se
        ad = api.LoraAdapters(A.cuda(), B.cuda(), b["scale"].cuda())
        A, B = R.f64(A), R.f64(B)
        width, out = (cin, cout) if forward else (cout, cin)
        data = (b["x"] if forward else b["dy"])[:, :width]
        got = torch.full((b["T"], out), 7.0, dtype=torch.bfloat16, device="cuda")
        if forward:
            api.lora_fwd(data.cuda(), row, ad, *b["seg"], Y=got, V=V)
            weight, first, second = R.decode(row), A, B
        else:
            dA, dB = api.lora_bwd(data.cuda(), torch.ones(b["T"], cin, dtype=torch.bfloat16, device="cuda"), V.clamp(-1, 1), col, ad,
                                  *b["seg"], 5, dX=got)[1:]
            assert dA.isfinite().all() and dB.isfinite().all()
            weight, first, second = R.decode(col), B.transpose(0, 2, 1), A.transpose(0, 2, 1)
        codes = R.decode_bf16(data[:n].contiguous(), "row", **({} if forward else dict(sr=True, seed=5)))
        d = R.f64(data)
        d[n:] = 0
        want, tol = _projected(b, d, first, second, codes, weight, TERMS)
        # the decode scale is an FP32 product: half of a subnormal's step, times the sum of the code products; and half
        # of a BF16 subnormal's step in the output, and of an FP32 one's in each low-rank product
        sa, sb = float(O.global_scales(O.amax(data[:n].contiguous()))[1]), float(row.global_scale)
        tol = tol + 2.0 ** -150 * (np.abs(codes) / sa) @ (np.abs(weight) / sb).T + 2.0 ** -134 + rank * 2.0 ** -149
        R.assert_within(R.f64(got)[:n], want, tol, f"forward {forward}")
        assert (got[n:] == 7.0).all()


@pytest.mark.parametrize("bad", [float("inf"), -3.39e38])
@pytest.mark.parametrize("others", [2, 300])
def test_infinite_sums_have_infinite_gradients(others, bad):
    # an adapter of a single row: its gradients are products of two numbers, and where U or V is infinite so are they,
    # with their sign.  -3.39e38, BF16's lowest, makes sums that FP32 cannot hold either
    b = G._make([others, 1], [0, 1], 128, 192, 16, 2)
    n = b["n"]
    A, B = b["A"].clone(), b["B"].clone()
    A[1, 3, 7], B[1, 5, 9] = bad, bad
    x, dy = b["X"].clone(), b["dY"].clone()
    x[n - 1, 7], dy[n - 1, 5] = 32.0, -64.0
    ad = api.LoraAdapters(A.cuda(), B.cuda(), b["ad"].scale)
    V = torch.zeros(b["T"], 16, device="cuda")
    api.lora_fwd(x, b["row"], ad, *b["seg"], V=V)
    assert V[n - 1, 3].item() == np.sign(bad) * np.inf and V[n - 1, [i for i in range(16) if i != 3]].isfinite().all()
    _, dA, dB = api.lora_bwd(dy, x, V, b["col"], ad, *b["seg"], 1)
    for got, j, z, sign in ((dA[1], 9, x[n - 1], -np.sign(bad)), (dB[1].t(), 3, dy[n - 1], np.sign(bad))):
        got, z = R.f64(got), R.f64(z)
        assert (got[j][z != 0] == sign * np.sign(z[z != 0]) * np.inf).all()
        assert np.isfinite(np.delete(got, j, 0)).all()
    assert dA[0].isfinite().all() and dB[0].isfinite().all()
