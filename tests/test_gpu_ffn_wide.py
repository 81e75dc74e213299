"""The products of include/forge_ffn.h on tiles of 256 columns, which they take where there are more than 128 of them: every
height of tile, with a last column tile half as wide, for every form that is kept."""
import pytest
import torch

from tests import ffn_ref as R
from tests import test_gpu_ffn as G

pytestmark = pytest.mark.gpu
BF, FP8, I8 = G.BF, G.FP8, G.I8
lib, _name = G.lib, G._name


def groups(sizes, rest, tile, columns):
    """(rows, ends) of groups of these sizes and `rest` rows of no group, that make more than 128 wide tiles of every
    height."""
    ends = torch.tensor(sizes).cumsum(0).to(torch.int32)
    tiles = sum(-(-n // tile) for n in [*sizes, rest])
    assert tiles * -(-columns // 256) > 128
    assert {-(-((n - 1) % tile + 1) // 64) for n in sizes if n} == {1, 2, 3, 4}
    return int(ends[-1]) + rest, ends


def fixed(monkeypatch, ends):
    monkeypatch.setattr(G, "ends_of", lambda T, E, seed: ends.clone())


# the host's bound on the tiles is below 128 for the first groups, above for the second
BLOCK = [([30, 100, 150, 210, 0, 224, 224 + 64], 24, 4224), ([224, 448, 60, 120, 190, 700, 225], 44, 4224)]


@pytest.mark.parametrize("sizes,rest,N", BLOCK)
@pytest.mark.parametrize("KB", [1, 2, 4, 5, 63, 64, 65, 68, 129])
def test_block_product_exact(lib, sizes, rest, N, KB):
    """Whole numbers and scales that are powers of two, so exact: products of at most 9 with scales of 1 / 4 to 4 add up to
    KB * 128 * 9 * 4 at most, 2.4 million times their unit of 1 / 4, below 2^24.  Contractions of whole fours of blocks and
    others, past 64 and 128 blocks."""
    T, ends = groups(sizes, rest, 224, N)
    E, K = len(sizes), 128 * KB
    g = torch.Generator(device="cuda").manual_seed(KB)
    whole = lambda *shape: torch.randint(-3, 4, shape, generator=g, device="cuda").float().to(FP8)  # noqa: E731
    power = lambda *shape: 2.0 ** torch.randint(-1, 2, shape, generator=g, device="cuda").float()  # noqa: E731
    X, W, xs, ws = whole(T, K), whole(E, N, K), power(T, KB), power(E, N // 128, KB)
    Y = torch.full((T, N), float("nan"), dtype=BF, device="cuda")
    lib.grouped_block_gemm(X, xs, W, ws, ends.cuda(), Y)
    x = X.double() * xs.double().repeat_interleave(128, 1)
    want = torch.zeros(T, N, dtype=R.F64, device="cuda")
    for e, (a, b) in enumerate(R.spans(ends, T)[0]):
        want[a:b] = x[a:b] @ R.weight_value(W[e], ws[e]).t().contiguous()
    assert torch.equal(Y, want.to(BF))


@pytest.mark.parametrize("K", [512, 640])
def test_block_product(lib, monkeypatch, K):
    """Every code of e4m3, scales of any size."""
    sizes, rest, N = BLOCK[0]
    T, ends = groups(sizes, rest + 1, 224, N)
    fixed(monkeypatch, ends)
    G.test_block_product(lib, T, len(sizes), N, K)


def test_block_product_scales_beside_16_bytes(lib):
    """The same bits, whether four scales of a row lie on 16 bytes or not."""
    sizes, rest, N = BLOCK[0]
    T, ends = groups(sizes, rest, 224, N)
    K, ends = 128 * 68, ends.cuda()
    g = torch.Generator().manual_seed(1)
    X, W = G.codes((T, K), 1).cuda(), G.codes((len(sizes), N, K), 2).cuda()
    xs, ws = torch.rand(T, K // 128, generator=g).cuda(), torch.rand(len(sizes), N // 128, K // 128, generator=g).cuda()
    Y = [torch.empty(T, N, dtype=BF, device="cuda") for _ in range(2)]
    lib.grouped_block_gemm(X, xs, W, ws, ends, Y[0])
    beside = torch.empty(xs.numel() + 4, device="cuda")[1:1 + xs.numel()].view(xs.shape)
    assert beside.data_ptr() % 16 == 4
    lib.grouped_block_gemm(X, beside.copy_(xs), W, ws, ends, Y[1])
    assert torch.equal(Y[0], Y[1]) and bool(Y[0].isfinite().all())


GATED = [([40, 100, 150, 250, 0, 256, 256 + 64], 24), ([256, 512, 60, 128, 190, 700, 257], 45)]


@pytest.mark.parametrize("sizes,rest", GATED)
@pytest.mark.parametrize("K", [128, 640])
@pytest.mark.parametrize("kind", [None, FP8, I8])
def test_gated_dgrad(lib, monkeypatch, sizes, rest, K, kind):
    T, ends = groups(sizes, rest, 256, 4224)
    assert T % 2 == 0
    fixed(monkeypatch, ends)
    G.test_grouped_gated_dgrad(lib, T, len(sizes), 4224, K, kind)


@pytest.mark.parametrize("sizes,rest", GATED)
@pytest.mark.parametrize("K", [128, 640])
@pytest.mark.parametrize("kind", ["none", BF, FP8, I8])
def test_gated(lib, monkeypatch, sizes, rest, K, kind):
    """A wide tile takes 128 gate and 128 up rows of the stacked weight: 17 for 2176 columns of H."""
    T, ends = groups(sizes, rest, 256, 2 * 2176)
    fixed(monkeypatch, ends)
    G.test_grouped_gated(lib, T, len(sizes), 2176, K, kind)
