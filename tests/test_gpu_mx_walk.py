"""GPU parity of the walking blocks of moe_norm_join_mx: shapes whose blocks take three
rows and more.  An SM holds at most 32 blocks and 2048 threads, and a walking block has
sixteen columns a thread, so the grid is at most min(32, 2048 / threads) blocks per SM."""
import pytest
import torch

from tests import dense_ref as R
from tests import mx_ref as X
from tests.test_gpu_mx import BF, DEV, EPS, F4, F8, F32, check_join, make, new_mx

pytestmark = pytest.mark.gpu
rvq = pytest.importorskip("moe_expert_ffn_router_gb300")


def three_rows(d):
    """Rows of which every walking block takes three or more, and some one more still (up to
    1024 columns only more than 4096 rows walk, and these are more)."""
    threads = -(-d // 512) * 32
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return 3 * sms * min(32, 2048 // threads) + 77


def stale_shared_memory():
    """A launch that leaves NaNs and large numbers all over every SM's shared memory: its
    rows pass through there."""
    n, d = 1216, 7168
    y = torch.full((n, d), 3.0e38, device=DEV)
    y[::2] = float("nan")
    rvq.moe_norm_join_mx(y, n, d, None, *new_mx(n, d, F8), h=y, eps=EPS)


WIDTHS = [8, 72, 264, 512, 520, 1096, 2056, 7168, 8192]
GATES = [("token", True, 0.5), ("channel", True, 1.0), ("full", False, 0.8125),
         ("none", False, 1.0), ("scalar", True, 1.0)]


@pytest.mark.parametrize("gate,post,alpha", GATES)
@pytest.mark.parametrize("d", WIDTHS)
def test_rows_of_a_walk(d, gate, post, alpha):
    """Every row against the definition, in the types that have an instance."""
    n = three_rows(d)
    kinds = [(F32, F32, F32, F8), (BF, BF, BF, F4)] if gate != "full" else \
        [(F32, BF, BF, F4), (BF, F32, F32, F8)]
    for hdt, ydt, wdt, fmt in kinds:
        s = make(n, d, hdt, ydt, wdt, gate, post, seed=d)
        stale_shared_memory()
        check_join(s, n, d, alpha, post, hdt, BF, fmt)


@pytest.mark.parametrize("d", [72, 512, 1096, 7168])
def test_walk_without_h(d):
    """Rows of zeros take the place of an absent h; no gains, no h_out."""
    n = three_rows(d)
    s = make(n, d, F32, F32, F32, "token", True, seed=d, with_h=False, gains=False)
    stale_shared_memory()
    check_join(s, n, d, 1.0, True, F32, F32, F8, ("xn", "rstd"))


@pytest.mark.parametrize("gate", ["token", "full"])
@pytest.mark.parametrize("d", [72, 512, 1096, 7168])
def test_walk_in_place(d, gate):
    """h_out over h and xn over y while the rows behind are on their way in."""
    n = three_rows(d)
    s = make(n, d, F32, F32, F32, gate, True, seed=d + 1)
    want = {k: None if v is None else v.clone() for k, v in s.items()}
    c2, s2, xn = check_join(want, n, d, 0.75, True, F32, F32, F8)
    h_out = torch.empty((n, d), device=DEV)
    rvq.moe_norm_join_mx(want["y"], n, d, h_out, *new_mx(n, d, F8), h=want["h"], alpha=0.75,
                         gate=want["gate"], w_post=want["w_post"], w_pre=want["w_pre"], eps=EPS)
    codes, scales = new_mx(n, d, F8)
    stale_shared_memory()
    rvq.moe_norm_join_mx(s["y"], n, d, s["h"], codes, scales, xn=s["y"], h=s["h"], alpha=0.75,
                         gate=s["gate"], w_post=s["w_post"], w_pre=s["w_pre"], eps=EPS)
    assert torch.equal(codes, c2) and torch.equal(scales, s2)
    assert torch.equal(s["y"], xn) and torch.equal(s["h"], h_out)


@pytest.mark.parametrize("d", [72, 512, 1096, 7168])
def test_walk_non_finite_rows(d):
    """NaN and infinity make their own rows NaN and none of those that a block takes
    before or after them."""
    n = three_rows(d)
    s = make(n, d, F32, F32, F32, "token", True, seed=d + 2)
    bad = torch.zeros(n, dtype=torch.bool, device=DEV)
    bad[::5] = True
    s["y"][::10, d - 1] = float("nan")
    s["h"][5::10, 3] = float("inf")
    codes, scales = new_mx(n, d, F8)
    rvq.moe_norm_join_mx(s["y"], n, d, None, codes, scales, h=s["h"], gate=s["gate"],
                         w_post=s["w_post"], w_pre=s["w_pre"], eps=EPS)
    byte, blocks = X.from_tiles(scales, n, d), -(-d // 32)
    # an infinity alone is NaN in its own block and 0 elsewhere in its row
    assert (byte[::10, :blocks] == 255).all() and (byte[5::10, 0] == 255).all()
    assert (byte[~bad] < 255).all() and (byte[:, blocks:] == 0).all()
    good = {k: v if v is None or v.shape[0] != n else v[~bad].contiguous() for k, v in s.items()}
    m = good["y"].shape[0]
    c2, s2 = new_mx(m, d, F8)
    rvq.moe_norm_join_mx(good["y"], m, d, None, c2, s2, h=good["h"], gate=good["gate"],
                         w_post=s["w_post"], w_pre=s["w_pre"], eps=EPS)
    assert torch.equal(codes.view(n, -1)[~bad].view(-1), c2)
    assert torch.equal(byte[~bad], X.from_tiles(s2, m, d))


@pytest.mark.parametrize("d", [72, 512, 1096])
def test_walk_streams_and_graph(d):
    """Two calls at once on two streams, and a captured call replayed on new rows: the
    rows of the definition."""
    n = three_rows(d)
    ins = [make(n, d, F32, BF, F32, "token", True, seed=60 + i) for i in range(2)]
    alone = [check_join(s, n, d, 1.0, True, F32, BF, F8)[:2] for s in ins]

    def call(s, q, **kw):
        rvq.moe_norm_join_mx(s["y"], n, d, None, *q, h=s["h"], gate=s["gate"], w_post=s["w_post"],
                             w_pre=s["w_pre"], eps=EPS, **kw)

    together = [new_mx(n, d, F8) for _ in ins]
    streams = [torch.cuda.Stream() for _ in ins]
    stale_shared_memory()
    torch.cuda.synchronize()
    for _ in range(4):
        for s, q, st in zip(ins, together, streams):
            call(s, q, stream=st)
    torch.cuda.synchronize()
    for a, b in zip(alone, together):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    s, q = {k: None if v is None else v.clone() for k, v in ins[0].items()}, new_mx(n, d, F8)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(s, q)
    for i in (1, 0):
        for k, v in ins[i].items():
            s[k].copy_(v)
        stale_shared_memory()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(q[0], alone[i][0]) and torch.equal(q[1], alone[i][1])


def test_walk_agrees_with_the_row_kernel():
    """The same rows through both kernels: 1/rms within the error of two orders of a sum
    (64 half steps each and one of its division)."""
    n, d = three_rows(512), 512
    s = make(n, d, F32, F32, F32, "channel", True, seed=3)
    rstd = torch.empty((2, n), device=DEV)
    stale_shared_memory()
    rvq.moe_norm_join_mx(s["y"], n, d, None, *new_mx(n, d, F8), h=s["h"], gate=s["gate"],
                         w_post=s["w_post"], w_pre=s["w_pre"], eps=EPS, rstd=rstd)
    m = 4096                      # a block per row up to here
    few = torch.empty((2, m), device=DEV)
    for r0 in (0, n - m):
        rvq.moe_norm_join_mx(s["y"][r0:r0 + m], m, d, None, *new_mx(m, d, F8), h=s["h"][r0:r0 + m],
                             gate=s["gate"], w_post=s["w_post"], w_pre=s["w_pre"], eps=EPS,
                             rstd=few)
        rel = (rstd[:, r0:r0 + m] / few - 1).abs().max()
        assert rel <= 260 * R.U32, rel
