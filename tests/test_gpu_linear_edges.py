"""Linear products on the GPU where rows, values or extents are out of the ordinary, against the 64-bit
references and bounds of ffn_reference.py."""
import pytest
import torch

from test_gpu_linear import check_backward, check_forward, draw

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16

# rows before the first group, rows of each group, rows after the last: a segment of each kind that
# ends inside a tile, groups up to and past the 64 segments looked at together, no group with rows,
# few rows a group and many
LEADING = [(30, [40, 50], 0), (1, [300], 40), (129, [0, 70, 0, 257], 5), (7, [1] * 61, 0), (0, [1] * 62, 9),
           (5, [1] * 62, 9), (5, [1] * 63, 0), (33, [2, 0, 1] * 43, 7), (200, [0, 0, 0], 0), (700, [3000, 1, 2500], 300)]


@pytest.mark.parametrize("before,counts,after", LEADING, ids=[str(i) for i in range(len(LEADING))])
@pytest.mark.parametrize("N,K", [(136, 200), (384, 1024), (2056, 520)])
def test_rows_before_the_first_group(gpu, before, counts, after, N, K):
    """offsets[0] > 0 (a slice of a longer list of offsets): the rows before it are of no group.  Whatever
    they hold, their rows of y, pre and dx are zero and no gradient of w or b sees them."""
    M = before + sum(counts) + after
    t = draw(M, N, K, groups=len(counts), seed=M)
    off = torch.tensor([before] + counts, device="cuda").cumsum(0).to(torch.int32)
    for rows in (slice(0, before), slice(M - after, M)):
        t["x"][rows], t["dy"][rows], t["residual"][rows] = float("nan"), float("inf"), float("nan")
    for act in ("none", "silu"):
        pre = check_forward(gpu, t, act, off, save_pre=act != "none")
        check_backward(gpu, t, pre, act, off)


def test_a_slice_of_the_experts(gpu):
    """The products of experts 2 .. 4 alone, from a slice of all the offsets."""
    counts = [70, 31, 0, 150, 64, 90]
    t = draw(sum(counts), 264, 200, groups=6)
    off = torch.tensor([0] + counts, device="cuda").cumsum(0).to(torch.int32)
    part = dict(t, w=t["w"][2:5], bias=t["bias"][2:5])
    pre = check_forward(gpu, part, "gelu", off[2:6], save_pre=True)
    check_backward(gpu, part, pre, "gelu", off[2:6])
    assert (pre[:101] == 0).all() and (pre[315:] == 0).all()


def test_every_row_before_the_first_group(gpu):
    t = draw(90, 64, 72, groups=2)
    off = torch.tensor([400, 500, 600], dtype=torch.int32, device="cuda")
    assert (gpu.glu_linear(t["x"], t["w"], t["bias"], t["residual"], offsets=off) == 0).all()
    for g in gpu.glu_linear_bwd(t["dy"], t["x"], t["w"], offsets=off, bias=True):
        assert (g == 0).all()


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_erf"])
@pytest.mark.parametrize("M,N,K", [(3, 136, 200), (150, 136, 200), (900, 520, 1032), (4000, 4008, 904)])
def test_nan_reaches_the_gradients(gpu, act, M, N, K):
    """A NaN of the bias makes its column of the pre-activation NaN, so that column of dp, its element of db,
    its row of dw and all of dx; a NaN in a row of x, that row of dx and all of dw and db.  Nothing
    else changes.  Few rows, sums split over workgroups and each tile size."""
    t = draw(M, N, K)

    def run():
        y, pre = gpu.glu_linear(t["x"], t["w"], t["bias"], act=act, save_pre=True)
        return (y, pre) + gpu.glu_linear_bwd(t["dy"], t["x"], t["w"], pre=pre, act=act, bias=True)

    def nan(t):
        return torch.isnan(t.float())

    y, pre, dx, dw, db = run()
    rest, keep = [i for i in range(N) if i != 5], t["bias"][5].item()
    t["bias"][5] = float("nan")
    y2, pre2, dx2, dw2, db2 = run()
    assert nan(y2[:, 5]).all() and nan(pre2[:, 5]).all() and nan(dx2).all() and nan(dw2[5]).all() and nan(db2[5])
    assert torch.equal(pre2[:, rest], pre[:, rest]) and torch.equal(dw2[rest], dw[rest]) and torch.equal(db2[rest], db[rest])
    t["bias"][5] = keep
    t["x"][1, 7] = float("nan")
    y2, pre2, dx2, dw2, db2 = run()
    rest = [i for i in range(M) if i != 1]
    assert nan(y2[1]).all() and nan(pre2[1]).all() and nan(dx2[1]).all() and nan(dw2).all() and nan(db2).all()
    assert torch.equal(pre2[rest], pre[rest]) and torch.equal(dx2[rest], dx[rest])


def test_the_saved_pre_activation_is_clamped(gpu):
    """Finite values past FP16's range and infinities are saved as its largest values, rounding at the edge
    of the range included; subnormals stay."""
    v = torch.tensor([65504.0, 65510.0, 65530.0, 1e6, 3e38, float("inf"), 1e-7, 6e-8, 1e-30, 0.0], device="cuda")
    p = torch.cat([v, -v]).to(BF16)
    bias = torch.zeros(24, device="cuda", dtype=BF16)
    bias[:20] = p
    want = bias.double().clamp(-65504, 65504).to(torch.float16)
    for M in (2, 40):
        x = torch.zeros(M, 8, device="cuda", dtype=BF16)
        w = torch.zeros(24, 8, device="cuda", dtype=BF16)
        _, pre = gpu.glu_linear(x, w, bias, act="gelu", save_pre=True)
        assert torch.equal(pre, want.expand(M, 24))


def test_sum_over_2_to_the_30_rows(gpu):
    """The gradient of w summed over 2^30 rows in 256 parts (17 GB an operand): rows that count lie at both
    ends and around the bounds of the last parts, each a power of two, so that the sum is exact and
    shows which of them are missing or counted twice."""
    M, part = 1 << 30, 1 << 22
    at = [0, 1, part - 1, part, 127 * part - 1, 127 * part, 254 * part, 255 * part - 1, 255 * part, 255 * part + 70000,
          M - 65, M - 1]
    x = torch.zeros(M, 8, device="cuda", dtype=BF16)
    dy = torch.zeros(M, 8, device="cuda", dtype=BF16)
    for i, row in enumerate(at):
        dy[row, i % 8] = 1.0
        x[row, i // 8] = 2.0 ** i
    _, dw, _ = gpu.glu_linear_bwd(dy, x, torch.zeros(8, 8, device="cuda", dtype=BF16), need_dx=False)
    want = torch.zeros(8, 8, device="cuda", dtype=BF16)
    for i in range(len(at)):
        want[i % 8, i // 8] = 2.0 ** i
    assert torch.equal(dw, want)
