"""What a plan keeps on the device is there when the call that sets it returns, for runs on any
stream: work that waits on the default stream does not hold it up."""
import pytest
import torch

from persistent_stream_matmul_gb300 import _binding as B
from moe_util import normal
from test_scaled_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _ready():
    from gpu_util import ensure_built
    ensure_built()


def keep_busy():
    """Work of some 200 ms on the default stream; an event behind it."""
    done = torch.cuda.Event()
    torch.cuda._sleep(400_000_000)
    done.record()
    return done


def test_words_of_a_scaled_plan():
    """A plan whose words another plan of the same size has just left, with its unit 0 told to give up."""
    c = Case(96, 1024, 8192, seed=1)
    want = c.run().clone()
    out, stream = torch.zeros_like(want), torch.cuda.Stream()
    c.plan.set_option(B.GEMM_SCALED_OPT_INJECT_GIVE_UP, 0)
    args = (c.M, c.N, c.K, 0, 0, c.code, B.GEMM_ROW_MAJOR, B.GEMM_COL_MAJOR, B.GEMM_SCALE_VECTOR, B.GEMM_SCALE_BLOCK)
    torch.cuda.synchronize()
    c.plan.close()
    done = keep_busy()
    plan = B.ScaledPlan(*args)
    plan.run(c.a, c.sa, c.b, c.sb, out, c.ws, stream)
    stream.synchronize()
    assert not done.query()  # the default stream is still busy
    torch.cuda.synchronize()
    assert plan.last_status(stream) == B.GEMM_OK
    assert torch.equal(out, want)


def test_words_of_a_grouped_plan():
    G, rows, N, K = 2, 64, 512, 4096
    A, Bm = normal((rows, K), torch.bfloat16, 1), normal((G, K, N), torch.bfloat16, 2)
    off = torch.tensor([0, 30, rows], dtype=torch.int32, device="cuda")
    make = lambda: B.GroupedPlan(B.GEMM_GROUPED_ROWS, G, rows, N, K, B.GEMM_BF16, B.GEMM_ROW_MAJOR)  # noqa: E731
    p, stream = make(), torch.cuda.Stream()
    ws = torch.empty(max(16, p.workspace_size), dtype=torch.uint8, device="cuda")
    want, out = (torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    p.run(A, Bm, want, off, ws)
    p.set_option(B.GEMM_GROUPED_OPT_INJECT_GIVE_UP, 0)
    torch.cuda.synchronize()
    p.close()
    done = keep_busy()
    q = make()
    q.run(A, Bm, out, off, ws, stream)
    stream.synchronize()
    assert not done.query()
    torch.cuda.synchronize()
    assert q.last_status(stream) == B.GEMM_OK
    assert torch.equal(out, want)


def test_timeout_of_a_new_plan_is_kept():
    """The status of a 16-bit product's plan: a run that timed out while the default stream was still
    behind the plan's creation."""
    from gpu_util import Workspace
    M, N, K = 128, 128, 4096
    A, Bm, C = normal((M, K), torch.float16, 1), normal((K, N), torch.float16, 2), torch.zeros(M, N, dtype=torch.float16, device="cuda")
    options = dict(tile_n=128, grid=4, wait_limit_us=2000)
    p, stream = B.Plan(M, N, K, B.GEMM_F16, 0, 0, "streamk", **options), torch.cuda.Stream()
    ws = Workspace().get(p.workspace_size)
    p.run(A, Bm, C, ws)
    assert p.last_status() == B.GEMM_OK
    done = keep_busy()
    q = B.Plan(M, N, K, B.GEMM_F16, 0, 0, "streamk", inject_skip_post=1, **options)
    q.run(A, Bm, C, ws, stream)
    stream.synchronize()
    assert not done.query()
    torch.cuda.synchronize()
    assert q.last_status(stream) == B.GEMM_ERR_TIMEOUT
    assert q.last_status(stream) == B.GEMM_OK
