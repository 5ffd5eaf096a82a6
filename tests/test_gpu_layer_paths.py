"""GPU tests of the mixture of experts at sizes that take its other kernels: activations in several chunks (a row of x or
of what passes between the products does not fit beside the rest), one token whose experts' activations do not fit
together, one token of many experts."""
import pytest

torch = pytest.importorskip("torch")
import bit_integer_gemm_amd as lb  # noqa: E402
import test_gpu_layer as layer  # noqa: E402
from test_gpu_layer import BF, HF, experts, gen  # noqa: E402

pytestmark = pytest.mark.gpu

# T, E, k, H, I, group
CHUNKS = [(17, 4, 2, 2304, 1056, 32),   # both products; an expert's tokens in two passes, rows that end inside a line
          (40, 3, 2, 2560, 1280, 128),  # the same in up to three passes
          (5, 2, 2, 7168, 64, 64),      # the first product, two and one registers of rows
          (3, 2, 1, 11264, 96, 32),
          (12, 2, 1, 64, 2592, 32),     # the second, in two planes of more than 8 rows, of up to 8 and up to 4
          (8, 2, 2, 64, 2304, 64),
          (2, 3, 2, 128, 8704, 128)]
TOKEN = [(1, 8, 8, 256, 4096, 32),      # its experts' activations do not fit together: three launches
         (1, 16, 12, 128, 2816, 64),
         (1, 4, 2, 128, 19456, 128),    # and not even one expert's two planes
         (1, 200, 4, 256, 64, 64), (1, 129, 1, 128, 96, 32), (1, 300, 7, 128, 64, 64),   # more than 128 experts, than 256
         (1, 1000, 8, 64, 32, 32), (1, 1024, 64, 96, 32, 32)]

# as many pairs of a token and an expert as experts, and around five for every four, where the search for those met ends
SHARED = [(16, 16, 1, 128, 64, 32), (19, 16, 1, 128, 64, 32), (20, 16, 1, 128, 64, 32), (21, 16, 1, 128, 64, 32),
          (13, 64, 6, 128, 96, 32), (14, 64, 6, 128, 96, 32), (30, 200, 8, 64, 64, 32), (32, 200, 8, 64, 64, 32)]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("T,E,k,H,I,group", CHUNKS + TOKEN + SHARED)
def test_moe_w4(dtype, T, E, k, H, I, group):
    layer.test_moe_w4(dtype, T, E, k, H, I, group)


def one_token(E, H=64, seed=0):
    g = gen(E + seed)
    wr, up, down = experts(E, H, 32, 32, BF, g)
    x = torch.randn(1, H, generator=g).to(BF)
    out = torch.empty(1, H, dtype=BF, device="cuda")

    def run(k, renorm=False):
        ids = torch.empty(1, k, dtype=torch.int32, device="cuda")
        weights = torch.empty(1, k, device="cuda")
        lb.lb_moe_w4(x.cuda(), *(a.cuda() for a in (wr, up[0], up[1], down[0], down[1])), out, top_k=k, renorm=renorm, ids=ids,
                     weights=weights)
        return out.cpu(), ids.cpu()[0].tolist(), weights.cpu()[0]

    return x, wr, up, down, run


@pytest.mark.parametrize("E", [12, 100, 128, 200, 256, 1000])
def test_one_token_ties(E):
    """Equal logits: the lowest expert first; and behind one that is larger."""
    x, wr, up, down, run = one_token(E)
    wr[:] = wr[0]
    for k in (1, 5, min(E, 64)):
        out, ids, weights = run(k)
        assert ids == list(range(k))
        want, _, p, _, _, bound = layer.moe_ref(x, wr, up, down, k, False, 1.0)
        layer.check_output(out, want, bound, BF)
        assert ((weights.double() - p[0]).abs() <= p[0] * (E + 40) * layer.STEP).all()   # (equal logits are equal in fp32)
    last = E - 1
    wr[last] = 2 * x[0] / x[0].norm()
    assert (x[0].double() @ wr[last].double()) > (x[0].double() @ wr[0].double()) + 1
    assert run(4)[1] == [last, 0, 1, 2]


@pytest.mark.parametrize("E", [12, 200, 1000])
@pytest.mark.parametrize("renorm", [False, True])
def test_one_token_not_finite(E, renorm):
    """A NaN among the logits comes first and spoils the token; the chosen are k different experts all the same."""
    x, wr, up, down, run = one_token(E, seed=1)
    wr[E // 2, 3] = wr[2, 5] = float("nan")
    out, ids, weights = run(5, renorm)
    order = torch.sort(x.double() @ wr.double().T, dim=1, descending=True, stable=True).indices[0]
    rest = [e for e in order.tolist() if e not in (2, E // 2)]
    assert ids == [2, E // 2] + rest[:3]
    assert out.isnan().all() and weights.isnan().all()
    x[0, 7] = float("inf")
    out, ids, _ = run(5, renorm)
    assert not out.isfinite().any() and len(set(ids)) == 5 and all(0 <= e < E for e in ids)
