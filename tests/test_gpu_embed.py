"""Token embedding and its gradient on the GPU against the fp64 definitions:
types, odd sizes and addresses, padding and out-of-range ids, runs of every
length around the sorting tiles and the summing chunks, accumulation, the
same bits on every run."""

import numpy as np
import pytest
import torch

from ends_common import DEV, U, Guarded, f64, to_dev, within
from oracle import ends
from uniform_noise_diffusion_amd import binding as B

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float32]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,H,V,skew", [(1, 1, 1, 0), (1, 128, 1024, 0), (5, 7, 3, 1),
                                        (257, 2816, 500, 0), (33, 2053, 60, 3), (9, 4104, 11, 5),
                                        (0, 64, 4, 0)])
def test_embed_is_the_scaled_row(dtype, n, H, V, skew):
    rng = np.random.default_rng(n * 7 + H)
    T, _ = to_dev(rng.standard_normal((V, H)), dtype, skew)
    ids = rng.integers(-2, V + 2, n).astype(np.int32)  # negative and too large ones among them
    out = Guarded((n, H), dtype, skew)
    B.mdlm_embed(torch.from_numpy(ids).to(DEV), T.t, 1.7, out.t)
    # one fp32 product, one rounding: exact
    want = T.t.cpu().float() * np.float32(1.7)
    ok = torch.from_numpy((ids >= 0) & (ids < V))
    rows = want[torch.from_numpy(np.where(ok, ids, 0)).long()]
    want = torch.where(ok[:, None], rows, torch.zeros(())).to(dtype)
    assert torch.equal(out.t.cpu(), want)
    assert out.intact() and T.intact()


def test_embed_keeps_leading_dimensions_and_nonfinite_rows():
    T = torch.tensor([[float("inf"), 1.0, float("nan")], [2.0, -0.5, 4.0]], device=DEV)
    ids = torch.tensor([[[0, 1], [1, -1]]], dtype=torch.int32, device=DEV)
    out = torch.empty(1, 2, 2, 3, device=DEV)
    B.mdlm_embed(ids, T, 2.0, out)
    o = out.cpu()
    assert o[0, 0, 0, 0] == float("inf") and torch.isnan(o[0, 0, 0, 2])
    assert torch.equal(o[0, 0, 1], torch.tensor([4.0, -1.0, 8.0]))
    assert torch.equal(o[0, 1, 1], torch.zeros(3))  # no token: zeros, whatever row 0 holds


def draw_ids(rng, kind, n, V):
    """Ids whose sorted runs have the lengths that can go wrong."""
    if kind == "absorb":  # half of the tokens one id
        ids = rng.integers(0, V, n)
        ids[rng.random(n) < 0.5] = V - 1
    elif kind == "one":  # a single run
        ids = np.full(n, min(3, V - 1))
    elif kind == "distinct":
        ids = rng.permutation(max(n, V))[:n] % V
    elif kind == "few":  # long runs that start and end inside chunks
        ids = rng.integers(0, min(V, 5), n)
    elif kind == "uniform":
        ids = rng.integers(0, V, n)
    elif kind == "none":  # no token at all
        ids = rng.choice([-1, -7, V, V + 100], n)
    else:  # "padded": a tail without tokens, some ids too large
        ids = rng.integers(-1, V + 1, n)
        ids[n - n // 3:] = -1
    return ids.astype(np.int32)


def check_grad(ids, n, H, V, dtype, accumulate, scale, seed, skew=0):
    rng = np.random.default_rng(seed)
    g, g64 = to_dev(rng.standard_normal((n, H)), dtype, skew)
    start = rng.standard_normal((V, H)).astype(np.float32)
    d = Guarded((V, H), torch.float32, skew, torch.from_numpy(start))
    dev_ids = torch.from_numpy(ids).to(DEV)
    B.mdlm_embed_grad(dev_ids, g.t, scale, d.t, accumulate)
    want, size = ends.embed_grad(ids, g64, V, float(np.float32(scale)),
                                 start.astype(np.float64) if accumulate else None)
    count = np.bincount(ids[(ids >= 0) & (ids < V)], minlength=V)[:, None]
    # a run of m terms: fewer than m roundings on any term's way into the sum
    # (chunks and partial rows only shorten it), the scale, the last addition
    within(f64(d.t), want, (count + 2) * U * size, (n, H, V, accumulate))
    assert d.intact() and g.intact()
    if accumulate:  # rows without a token keep their bits
        idle = torch.from_numpy(count[:, 0] == 0)
        assert torch.equal(d.t.cpu()[idle], torch.from_numpy(start)[idle])
    return d.t, g.t, dev_ids


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("kind", ["absorb", "one", "distinct", "few", "none", "padded"])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 33, 47, 49, 1023, 1024, 1025, 2500])
def test_embed_grad_runs(dtype, accumulate, kind, n):
    V, H = 700, 24
    ids = draw_ids(np.random.default_rng(n), kind, n, V)
    check_grad(ids, n, H, V, dtype, accumulate, 1.5, n + 1)


@pytest.mark.parametrize("n,H,V,dtype,kind", [
    (4096, 264, 9000, torch.bfloat16, "absorb"),
    (16384, 40, 9000, torch.bfloat16, "absorb"),   # sixteen tiles: one merge
    (16385, 40, 9000, torch.bfloat16, "absorb"),   # two merges, the longer chunks
    (40000, 33, 300, torch.float32, "few"),
    (20000, 40, 60, torch.float32, "uniform"),     # hundreds of cut runs
    (33000, 300, 9000, torch.bfloat16, "absorb"),  # a cut run of 500 chunks
    (8193, 24, 400, torch.float32, "absorb"),      # the sorted runs merged in LDS
    (32769, 16, 40000, torch.float32, "padded"),   # and in memory
    (70001, 16, 70000, torch.float32, "distinct"),
    (600000, 8, 5000, torch.float32, "absorb"),    # two merges in memory
    (3000, 1, 50, torch.float32, "few"),
    (300, 1001, 400, torch.bfloat16, "padded"),
    (200, 2816, 90, torch.bfloat16, "few"),
    (64, 9000, 20, torch.float32, "few"),
])
def test_embed_grad_sizes(n, H, V, dtype, kind):
    ids = draw_ids(np.random.default_rng(n), kind, n, V)
    for accumulate in (False, True):
        check_grad(ids, n, H, V, dtype, accumulate, 0.75, n, skew=3 if H % 8 else 0)


def test_embed_grad_run_borders():
    """One run of every length from 1 to 70 at every offset within a chunk of
    16, between single tokens."""
    V, H = 4000, 8
    for off in range(16):
        ids, v = [], 1
        for _ in range(off):
            ids.append(0)  # the shift of everything behind
        for length in range(1, 71):
            ids += [v] * length
            v += 1
        rng = np.random.default_rng(off)
        ids = np.array(ids, dtype=np.int32)
        rng.shuffle(ids)
        check_grad(ids, len(ids), H, V, torch.float32, off % 2 == 0, 1.0, off)


@pytest.mark.parametrize("accumulate", [False, True])
def test_embed_grad_of_few_tokens_and_long_rows(accumulate):
    """Up to 1,024 tokens on both sides of the 2^20 entries up to which one
    launch does it all, and the sorted list at its shortest."""
    for n, H, V in ((1, 1 << 20, 3), (1, (1 << 20) + 8, 3), (3, 400_000, 2), (17, 70_000, 4),
                    (33, 33_000, 5), (100, 10_400, 30), (255, 4112, 40), (256, 4096, 40),
                    (257, 4096, 40), (1000, 1100, 90), (1024, 1024, 90), (1025, 1024, 90)):
        for kind in ("absorb", "few"):
            ids = draw_ids(np.random.default_rng(n), kind, n, V)
            check_grad(ids, n, H, V, torch.bfloat16, accumulate, 1.25, n)


def test_embed_grad_of_few_tokens_runs():
    """Runs of 1 to 40 tokens, in one launch, in a table on both sides of the
    size that the launch clears itself."""
    for V in (41, 300_000):
        ids = np.repeat(np.arange(41), np.arange(41)).astype(np.int32)
        np.random.default_rng(V).shuffle(ids)
        check_grad(ids, len(ids), 60, V, torch.float32, False, -0.5, V)
        check_grad(ids, len(ids), 60, V, torch.float32, True, -0.5, V)


def test_embed_grad_of_few_tokens_into_narrow_rows():
    """Tables on both sides of the 512 clearing blocks up to which one launch
    also clears the table, and long ones of short rows."""
    for H, V in ((8, 64 * 512), (8, 64 * 512 + 1), (256, 64 * 512), (256, 64 * 512 + 1),
                 (1, 500_000), (3, 300_000)):
        ids = draw_ids(np.random.default_rng(V), "padded", 90, V)
        ids[:2] = 0, V - 1
        check_grad(ids, 90, H, V, torch.float32, False, 0.75, H, skew=3 if H % 8 else 0)


def test_embed_grad_no_tokens():
    d = torch.full((10, 12), 7.0, device=DEV)
    ids, g = torch.empty(0, dtype=torch.int32, device=DEV), torch.empty(0, 12, device=DEV)
    B.mdlm_embed_grad(ids, g, 1.0, d, accumulate=True)
    assert bool((d == 7.0).all())
    B.mdlm_embed_grad(ids, g, 1.0, d)
    assert not d.any()


def test_embed_grad_padding_hides_nonfinite_gradients():
    ids = torch.tensor([2, -1, 2, 9], dtype=torch.int32, device=DEV)
    g = torch.ones(4, 5, device=DEV)
    g[1], g[3] = float("nan"), float("inf")
    d = torch.empty(4, 5, device=DEV)
    B.mdlm_embed_grad(ids, g, 1.0, d)
    want = torch.zeros(4, 5)
    want[2] = 2.0
    assert torch.equal(d.cpu(), want)


def test_embed_grad_same_bits_every_run_and_given_workspace():
    n, H, V = 9000, 136, 2000
    ids = draw_ids(np.random.default_rng(0), "absorb", n, V)
    first, g, dev_ids = check_grad(ids, n, H, V, torch.bfloat16, False, 1.0, 5)
    need = B.mdlm_embed_grad_workspace_bytes(n, H)
    for fill in (0, 255):  # contents on entry are ignored
        ws = torch.full((need,), fill, dtype=torch.uint8, device=DEV)
        again = torch.empty_like(first)
        B.mdlm_embed_grad(dev_ids, g, 1.0, again, workspace=ws)
        assert torch.equal(first.view(torch.int32), again.view(torch.int32))
    with pytest.raises(B.MdlmError, match="workspace"):
        B.mdlm_embed_grad(dev_ids, g, 1.0, first, workspace=ws[:need - 1])


def test_embed_binding_refusals():
    ids = torch.zeros(4, dtype=torch.int32, device=DEV)
    T = torch.zeros(8, 16, device=DEV)
    out = torch.zeros(4, 16, device=DEV)
    with pytest.raises(TypeError):
        B.mdlm_embed(ids.long(), T, 1.0, out)
    with pytest.raises(TypeError):
        B.mdlm_embed(ids, T, 1.0, out.bfloat16())
    with pytest.raises(TypeError):
        B.mdlm_embed(ids, T.half(), 1.0, out.half())
    with pytest.raises(ValueError):
        B.mdlm_embed(ids, T, 1.0, out[:3])
    with pytest.raises(ValueError):
        B.mdlm_embed(ids, T.t().contiguous().t(), 1.0, out)
    with pytest.raises(ValueError):
        B.mdlm_embed(ids.cpu(), T, 1.0, out)
    with pytest.raises(B.MdlmError):
        B.mdlm_embed(ids, T, float("nan"), out)
    with pytest.raises(TypeError):
        B.mdlm_embed_grad(ids, out, 1.0, T.bfloat16())
    with pytest.raises(ValueError):
        B.mdlm_embed_grad(ids[:3], out, 1.0, T)
    with pytest.raises(ValueError):
        B.mdlm_embed_grad(ids, out.cpu(), 1.0, T)
    with pytest.raises(TypeError):
        B.mdlm_embed_grad(ids, out, 1.0, T, workspace=torch.zeros(1 << 20, device=DEV))


def test_checking_mode_reports_ids_past_the_table():
    ids = torch.tensor([0, 7, -1], dtype=torch.int32, device=DEV)
    T, out = torch.ones(7, 8, device=DEV), torch.full((3, 8), 5.0, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    B.mdlm_check_tokens(ids, 7, status)
    assert int(status) == B.MDLM_CHECK_TOKEN
    status.zero_()
    B.mdlm_check_tokens(ids, 8, status)
    assert int(status) == 0
    prev = B.mdlm_set_checking(True)
    try:
        with pytest.raises(B.MdlmError, match="ids"):
            B.mdlm_embed(ids, T, 1.0, out)
        with pytest.raises(B.MdlmError, match="ids"):
            B.mdlm_embed_grad(ids, out, 1.0, T)
        torch.cuda.synchronize()
        assert bool((out == 5.0).all()) and bool((T == 1.0).all())
        ids[1] = 6
        B.mdlm_embed(ids, T, 1.0, out)
        assert bool((out[:2] == 1.0).all()) and not out[2].any()
    finally:
        B.mdlm_set_checking(prev)
