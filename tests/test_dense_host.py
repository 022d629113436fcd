"""Host side of the dense operators (no GPU): workspace sizes and refusals
before any launch, in the library and in the binding."""
import ctypes
import os

import pytest
import torch

import moe_expert_ffn_router_gb300 as rvq

lib = rvq._lib
A = 0x10000000       # fake, aligned "device" addresses far apart (never dereferenced)
B, C, D, E_, F = (A + i * 0x10000000 for i in range(1, 6))
OK, EINVAL, EALIGN, ENOMEM = 0, 1, 2, 3
F32, BF16, F16 = 0, 1, 2


def up256(v):
    return (v + 255) // 256 * 256


def test_workspace_sizes():
    for n, r, c in ((1, 8, 8), (7, 256, 512), (4096, 2048, 7168)):
        assert rvq.moe_linear_workspace_bytes(n, r, c) >= 256
        assert rvq.moe_gated_linear_workspace_bytes(n, r, c) >= 256
        # dp (16 bits) of each matrix and one bias partial per 32 tokens
        for f, m in ((rvq.moe_linear_workspace_bytes, 1), (rvq.moe_gated_linear_workspace_bytes, 2)):
            assert f(n, r, c, True) >= 256 + m * n * r * 2 + (n + 31) // 32 * m * r * 4
        assert rvq.moe_norm_join_workspace_bytes(n, c) >= 256 + 4 * 3 * c
    for n, r, c in ((0, 8, 8), (1, 12, 8), (1, 8, 12), (1, 0, 8), (-1, 8, 8)):
        assert rvq.moe_linear_workspace_bytes(n, r, c) == 0
        assert rvq.moe_gated_linear_workspace_bytes(n, r, c, True) == 0
    assert rvq.moe_norm_join_workspace_bytes(0, 8) == 0
    assert rvq.moe_norm_join_workspace_bytes(1, 12) == 0
    assert rvq.moe_norm_join_workspace_bytes(1, 16384 + 8) == 0


LIN = dict(x=A, ldx=64, w=B, ldw=64, bias=None, dt=BF16, n=4, rows=32, cols=64, act=0, alpha=1.0,
           res=None, rdt=F32, ldr=0, out=C, odt=BF16, ldo=32, pre=None, ws=D, wsb=1 << 20, st=None)


def lin(**kw):
    return lib.moe_linear(*{**LIN, **kw}.values())


def test_linear_refusals():
    for bad in (dict(n=0), dict(rows=12), dict(cols=60), dict(rows=0), dict(dt=F32), dict(dt=3),
                dict(act=5), dict(act=-1), dict(x=None), dict(w=None), dict(out=None),
                dict(ldx=56), dict(ldx=68), dict(ldw=0), dict(ldo=31), dict(odt=7),
                dict(res=E_, rdt=5, ldr=32), dict(res=E_, ldr=24), dict(ws=None), dict(ws=D + 16),
                dict(out=A), dict(out=B + 64), dict(out=A + 4 * 64 * 2 - 16),
                dict(res=C, rdt=F32, ldr=32), dict(res=C + 16, rdt=BF16, ldr=32),
                dict(res=C, rdt=BF16, ldr=40), dict(pre=C)):
        assert lin(**bad) == EINVAL, bad
    for bad in (dict(x=A + 2), dict(w=B + 8), dict(out=C + 4), dict(bias=E_ + 2), dict(pre=E_ + 4),
                dict(res=E_ + 8, ldr=32)):
        assert lin(**bad) == EALIGN, bad
    assert lin(wsb=255) == ENOMEM
    assert b"workspace" in lib.rvq_last_error()


GAT = dict(x=A, ldx=64, wg=B, wu=B + 0x10000, ldw=64, bg=None, bu=None, dt=BF16, n=4, rows=32,
           cols=64, act=2, out=C, ldo=32, pre=None, ws=D, wsb=1 << 20, st=None)


def test_gated_refusals():
    def gat(**kw):
        return lib.moe_gated_linear(*{**GAT, **kw}.values())

    for bad in (dict(n=0), dict(rows=4), dict(cols=4), dict(dt=F32), dict(act=9), dict(x=None),
                dict(wg=None), dict(wu=None), dict(out=None), dict(ldw=60), dict(ldo=16),
                dict(out=A), dict(out=B), dict(out=B + 0x10000), dict(pre=C), dict(ws=None)):
        assert gat(**bad) == EINVAL, bad
    for bad in (dict(x=A + 2), dict(wu=B + 8), dict(out=C + 8), dict(bg=E_ + 8), dict(bu=E_ + 8),
                dict(pre=E_ + 8)):
        assert gat(**bad) == EALIGN, bad
    assert gat(wsb=0) == ENOMEM


def test_backward_refusals():
    base = dict(do=A, ldd=32, x=B, ldx=64, w=C, ldw=64, pre=D, dt=BF16, n=4, rows=32, cols=64,
                act=2, alpha=1.0, dx=E_, lddx=64, dw=F, lddw=64, db=None, ws=F + 0x10000000,
                wsb=1 << 20, st=None)

    def back(**kw):
        return lib.moe_linear_backward(*{**base, **kw}.values())

    for bad in (dict(do=None), dict(pre=None), dict(dx=None, dw=None), dict(x=None), dict(w=None),
                dict(lddx=32), dict(lddw=65), dict(dx=A), dict(dx=C), dict(dw=B), dict(dx=B),
                dict(dw=A), dict(n=0), dict(dt=F32), dict(ws=None)):
        assert back(**bad) == EINVAL, bad
    for bad in (dict(do=A + 2), dict(dx=E_ + 8), dict(dw=F + 8), dict(db=A + 4), dict(pre=D + 4)):
        assert back(**bad) == EALIGN, bad
    assert back(wsb=rvq.moe_linear_workspace_bytes(4, 32, 64, True) - 1) == ENOMEM
    gb = dict(do=A, ldd=32, x=B, ldx=64, wg=C, wu=C + 0x10000, ldw=64, pre=D, dt=BF16, n=4,
              rows=32, cols=64, act=2, dx=E_, lddx=64, dwg=F, dwu=F + 0x10000, lddw=64, dbg=None,
              dbu=None, ws=F + 0x10000000, wsb=1 << 20, st=None)

    def gback(**kw):
        return lib.moe_gated_linear_backward(*{**gb, **kw}.values())

    for bad in (dict(do=None), dict(pre=None), dict(dwu=None), dict(dwg=None), dict(dwu=F),
                dict(dx=None, dwg=None, dwu=None), dict(wu=None), dict(dx=C), dict(dwg=B),
                dict(dx=B), dict(lddw=60)):
        assert gback(**bad) == EINVAL, bad
    assert gback(wsb=rvq.moe_gated_linear_workspace_bytes(4, 32, 64, True) - 1) == ENOMEM


def test_join_refusals():
    base = dict(h=A, hdt=F32, y=B, ydt=BF16, n=4, d=64, alpha=1.0, gate=None, kind=0, gdt=F32,
                post=1, wpost=None, wpre=None, wdt=F32, eps=1e-6, ho=C, xn=D, xdt=BF16, rstd=None,
                st=None)

    def join(**kw):
        return lib.moe_norm_join(*{**base, **kw}.values())

    for bad in (dict(n=0), dict(d=60), dict(d=16392), dict(hdt=3), dict(ydt=-1), dict(gdt=4),
                dict(wdt=9), dict(xdt=3), dict(y=None), dict(kind=2), dict(gate=E_, kind=0),
                dict(gate=E_, kind=5), dict(post=0, wpost=E_), dict(eps=-1.0),
                dict(eps=float("nan")), dict(ho=None, xn=None), dict(ho=B), dict(xn=A),
                dict(xn=C), dict(ho=A + 16), dict(xn=B + 32)):
        assert join(**bad) == EINVAL, bad
    for bad in (dict(h=A + 4), dict(y=B + 2), dict(gate=E_ + 2, kind=3), dict(wpost=E_ + 4),
                dict(wpre=E_ + 4), dict(ho=C + 8), dict(xn=D + 8), dict(rstd=E_ + 4)):
        assert join(**bad) == EALIGN, bad
    bb = dict(dho=A, dxn=B, xdt=BF16, h=C, hdt=F32, y=D, ydt=BF16, n=4, d=64, alpha=1.0, gate=None,
              kind=0, gdt=F32, post=1, wpost=None, wpre=None, wdt=F32, rstd=E_, dh=F, dy=None,
              dgate=None, dwpost=None, dwpre=None, ws=F + 0x10000000, wsb=1 << 20, st=None)

    def back(**kw):
        return lib.moe_norm_join_backward(*{**bb, **kw}.values())

    for bad in (dict(dho=None, dxn=None), dict(dh=None), dict(rstd=None), dict(dgate=F + 0x1000),
                dict(h=None), dict(post=0, dwpost=F + 0x1000), dict(dxn=None, dwpre=F + 0x1000),
                dict(dh=B), dict(dy=A), dict(dy=F), dict(ws=None), dict(n=0)):
        assert back(**bad) == EINVAL, bad
    assert back(dh=F + 4) == EALIGN and back(rstd=E_ + 4) == EALIGN
    assert back(wsb=512) == ENOMEM


def test_other_calls_still_refuse_fp16():
    """RVQ_F16 is the dense operators' own type code."""
    assert lib.rvq_lut_build(A, A, F16, 1, 16, B, None) == EINVAL
    assert lib.moe_router_logits(A, None, A, F16, 1, 64, 512, B, None) == EINVAL
    assert lib.moe_rms_norm(A, F16, 1, 64, ctypes.c_float(1e-6), B, F32, None) == EINVAL
    assert lib.moe_combine(A, A, 2, 2, 8, A, F16, B, None) == EINVAL


def test_binding_refusals():
    """Shapes, types and layouts the binding can see are refused there."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(32, 64, dtype=torch.bfloat16)
    out = torch.zeros(4, 32, dtype=torch.bfloat16)
    ws = torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="shape"):
        rvq.moe_linear(x, w, 5, 32, 64, out, ws)
    with pytest.raises(ValueError, match="not contiguous"):
        rvq.moe_linear(torch.zeros(64, 4, dtype=torch.bfloat16).t(), w, 4, 32, 64, out, ws)
    with pytest.raises(TypeError, match="dtype"):
        rvq.moe_linear(x, w.half(), 4, 32, 64, out, ws)
    with pytest.raises(TypeError, match="unsupported"):
        rvq.moe_linear(x, w, 4, 32, 64, out.double(), ws)
    with pytest.raises(ValueError, match="bias"):
        rvq.moe_linear(x, w, 4, 32, 64, out, ws, bias=torch.zeros(31, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="pitches"):
        rvq.moe_gated_linear(x, w, torch.zeros(32, 128, dtype=torch.bfloat16)[:, :64], 4, 32, 64,
                             out, ws)
    y = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="broadcast"):
        rvq.moe_norm_join(y, 4, 64, y.clone(), None, gate=torch.zeros(3, 1))
    with pytest.raises(ValueError, match="gate"):
        rvq.moe_norm_join(y, 4, 64, y.clone(), None, gate=torch.zeros(64, 4).t())
    assert [rvq._gate_kind(g, 4, 64) for g in
            (None, torch.zeros(1), torch.zeros(4, 1), torch.zeros(64), torch.zeros(1, 64),
             torch.zeros(4, 64))] == [0, 1, 2, 3, 3, 4]


@pytest.mark.parametrize("n", [1, 4, 300])
def test_gradients_refuse_racing_overlaps(n):
    """The products of a gradient call may run in one launch: a gradient over an
    input of the other product, or over another gradient, is refused."""
    at = [A + i * 0x10000000 for i in range(16)]
    base = dict(do=at[0], ldd=32, x=at[1], ldx=64, w=at[2], ldw=64, pre=at[3], dt=BF16, n=n,
                rows=32, cols=64, act=2, alpha=1.0, dx=at[4], lddx=64, dw=at[5], lddw=64,
                db=at[6], ws=at[7], wsb=1, st=None)

    def back(**kw):
        return lib.moe_linear_backward(*{**base, "wsb": 1 << 24, **kw}.values())

    assert lib.moe_linear_backward(*base.values()) == ENOMEM   # else it is accepted
    last = (32 * 64 - 8) * 2        # the last 16 bytes of w and dw
    for bad in (dict(dw=at[2]), dict(dw=at[2] + last), dict(dw=at[2] - last), dict(dw=at[4]),
                dict(dx=at[5] + 64), dict(db=at[4]), dict(db=at[5] + last), dict(db=at[2]),
                dict(db=at[1]), dict(db=at[0]), dict(db=at[0], act=0, pre=None)):
        assert back(**bad) == EINVAL, bad
        assert b"overlaps" in lib.rvq_last_error(), bad
    base = dict(do=at[0], ldd=32, x=at[1], ldx=64, wg=at[2], wu=at[3], ldw=64, pre=at[4], dt=BF16,
                n=n, rows=32, cols=64, act=2, dx=at[5], lddx=64, dwg=at[6], dwu=at[7], lddw=64,
                dbg=at[8], dbu=at[9], ws=at[10], wsb=1, st=None)

    def gback(**kw):
        return lib.moe_gated_linear_backward(*{**base, "wsb": 1 << 24, **kw}.values())

    assert lib.moe_gated_linear_backward(*base.values()) == ENOMEM
    for bad in (dict(dwg=at[2]), dict(dwg=at[3]), dict(dwu=at[2] + last), dict(dwu=at[3]),
                dict(dwg=at[5]), dict(dwu=at[5]), dict(dx=at[7] - 16), dict(dbg=at[5]),
                dict(dbg=at[6]), dict(dbg=at[2]), dict(dbu=at[7] + last), dict(dbu=at[3]),
                dict(dbu=at[8]), dict(dbu=at[8] + 48), dict(dbg=at[1])):
        assert gback(**bad) == EINVAL, bad
        assert b"overlaps" in lib.rvq_last_error(), bad


@pytest.mark.parametrize("n", [1, 4, 300])
def test_outputs_over_inputs_are_refused(n):
    """The saved pre-activations and the biases too: some blocks still read what
    others write."""
    at = [A + i * 0x10000000 for i in range(16)]
    base = dict(x=at[0], ldx=64, w=at[1], ldw=64, bias=at[2], dt=BF16, n=n, rows=32, cols=64,
                act=2, alpha=1.0, res=at[3], rdt=BF16, ldr=32, out=at[4], odt=BF16, ldo=32,
                pre=at[5], ws=at[6], wsb=1, st=None)
    assert lib.moe_linear(*base.values()) == ENOMEM    # else it is accepted
    for bad in (dict(pre=at[0]), dict(pre=at[1]), dict(pre=at[1] + (32 * 64 - 8) * 2),
                dict(pre=at[2]), dict(pre=at[3]), dict(pre=at[4]), dict(out=at[2]),
                dict(out=at[2] + 48), dict(out=at[0]), dict(out=at[5])):
        assert lib.moe_linear(*{**base, "wsb": 1 << 24, **bad}.values()) == EINVAL, bad
        assert b"overlaps" in lib.rvq_last_error(), bad
    base = dict(x=at[0], ldx=64, wg=at[1], wu=at[2], ldw=64, bg=at[3], bu=at[4], dt=BF16, n=n,
                rows=32, cols=64, act=2, out=at[5], ldo=32, pre=at[6], ws=at[7], wsb=1, st=None)
    assert lib.moe_gated_linear(*base.values()) == ENOMEM
    half = n * 32 * 4               # bytes of pre's first plane
    for bad in (dict(pre=at[0]), dict(pre=at[1]), dict(pre=at[2]), dict(pre=at[2] - half),
                dict(pre=at[3]), dict(pre=at[4] - half), dict(pre=at[5] - half),
                dict(out=at[3]), dict(out=at[4] + 48), dict(out=at[6]), dict(out=at[6] + half)):
        assert lib.moe_gated_linear(*{**base, "wsb": 1 << 24, **bad}.values()) == EINVAL, bad
        assert b"overlaps" in lib.rvq_last_error(), bad


@pytest.mark.parametrize("n,d", [(4, 64), (1000, 264)])
def test_join_refuses_racing_overlaps(n, d):
    """Rows are read before they are written by the block that owns them, so an
    output may take the place of rows of its type; any other overlap is refused."""
    at = [A + i * 0x10000000 for i in range(16)]
    base = dict(h=at[0], hdt=F32, y=at[1], ydt=F32, n=n, d=d, alpha=1.0, gate=at[2], kind=4,
                gdt=F32, post=1, wpost=at[3], wpre=at[4], wdt=F32, eps=1e-6, ho=at[5], xn=at[6],
                xdt=F32, rstd=at[7], st=None)
    row = d * 4
    for bad in (dict(ho=at[2] + row), dict(xn=at[2] + row), dict(ho=at[2], gdt=BF16),
                dict(ho=at[2], kind=3), dict(xn=at[2], kind=2), dict(ho=at[2], kind=1),
                dict(ho=at[3]), dict(xn=at[4] + 16), dict(rstd=at[0]), dict(rstd=at[1] + row),
                dict(rstd=at[2]), dict(rstd=at[3]), dict(rstd=at[5]), dict(rstd=at[6] + row),
                dict(xn=at[5] + row), dict(ho=at[0] + row), dict(xn=at[1] - row)):
        assert lib.moe_norm_join(*{**base, **bad}.values()) == EINVAL, bad
        assert b"overlaps" in lib.rvq_last_error(), bad
    base = dict(dho=at[0], dxn=at[1], xdt=F32, h=at[2], hdt=F32, y=at[3], ydt=F32, n=n, d=d,
                alpha=1.0, gate=at[4], kind=4, gdt=F32, post=1, wpost=at[5], wpre=at[6], wdt=F32,
                rstd=at[7], dh=at[8], dy=at[9], dgate=at[10], dwpost=at[11], dwpre=at[12],
                ws=at[13], wsb=1, st=None)

    def back(**kw):
        return lib.moe_norm_join_backward(*{**base, **kw}.values())

    ok = (dict(), dict(dh=at[0]), dict(dh=at[1]), dict(dh=at[2]), dict(dh=at[3], dy=at[2]),
          dict(dy=at[4], dgate=at[3]), dict(dgate=at[4]), dict(kind=2, dgate=at[4]),
          dict(kind=3, dgate=at[4]), dict(kind=1, dgate=at[4]), dict(dwpost=at[5], dwpre=at[6]))
    for kw in ok:
        assert back(**kw) == ENOMEM, kw     # past the checks of overlaps
    for bad in (dict(dh=at[2] + row), dict(dh=at[3] + row), dict(dh=at[4] + row),
                dict(dy=at[2] + row), dict(dy=at[3] - row), dict(dh=at[2], hdt=F32, dy=at[2]),
                dict(dh=at[3], ydt=BF16), dict(dh=at[4], kind=3), dict(dy=at[4], kind=2),
                dict(dgate=at[8]), dict(dgate=at[9] + row), dict(dgate=at[2] + row),
                dict(dgate=at[4] + row), dict(dgate=at[7]), dict(dgate=at[5]),
                dict(dgate=at[7], kind=2), dict(dgate=at[3] + 16, kind=2),
                dict(dgate=at[8], kind=3), dict(dgate=at[9], kind=1), dict(dwpost=at[8]),
                dict(dwpre=at[9] + row), dict(dwpost=at[12]), dict(dwpre=at[10]),
                dict(dh=at[5]), dict(dy=at[6]), dict(dh=at[7]), dict(dgate=at[11], kind=3)):
        assert back(**bad, wsb=1 << 26) == EINVAL, bad
        assert b"overlaps" in lib.rvq_last_error(), bad


def test_no_read_only_loads_beside_a_running_kernel():
    """The dense operators' kernels are launched programmatically: their blocks may be
    resident while the kernel before them writes what they will read.  The read-only
    path (ld.global.nc, __ldg) is defined for data that no one writes meanwhile."""
    csrc = os.path.join(os.path.dirname(rvq.__file__), "csrc")
    files = [f for f in sorted(os.listdir(csrc)) if f.startswith(("dense", "join", "norm_join"))]
    assert len(files) >= 10
    for f in files:
        code = open(os.path.join(csrc, f)).read()
        assert "__ldg(" not in code and "global.nc" not in code and "__restrict__" not in code, f


@pytest.mark.parametrize("rows,cols", [(2048, 7168), (7168, 2048), (1000, 2048), (256, 512),
                                       (360, 688), (264, 7168), (8, 8)])
@pytest.mark.parametrize("backward", [False, True])
def test_a_workspace_serves_fewer_tokens(rows, cols, backward):
    """A program allocates for its largest batch: no smaller batch needs more, nor
    does the forward call need more than the gradients."""
    tokens = sorted(set(list(range(1, 520, 7)) + [2 ** i + j for i in range(8, 15) for j in (-1, 0, 1)]
                        + list(range(512, 5000, 97))))
    for f in (rvq.moe_linear_workspace_bytes, rvq.moe_gated_linear_workspace_bytes):
        need = [f(n, rows, cols, backward) for n in tokens]
        assert all(a <= b for a, b in zip(need, need[1:]))
        assert all(f(n, rows, cols) <= b for n, b in zip(tokens, need))
    need = [rvq.moe_norm_join_workspace_bytes(n, cols) for n in tokens]
    assert all(a <= b for a, b in zip(need, need[1:]))


def test_shared_expert_types_are_refused_where_they_are_built():
    """Not in the first call: a weight type that the products do not take, mixed types,
    and fp16 experts in a stack, whose normed stream is bf16."""
    from moe_expert_ffn_router_gb300.layer import SharedExpert, SharedExpertStack

    def expert(*dtypes):
        shapes = ((16, 32), (16, 32), (32, 16))
        return SharedExpert(*(torch.zeros(s, dtype=t) for s, t in zip(shapes, dtypes)), device="cpu")

    bf, hf, f32 = torch.bfloat16, torch.float16, torch.float32
    for bad in ((f32, f32, f32), (bf, bf, hf), (hf, bf, hf)):
        with pytest.raises(TypeError, match="bf16 or fp16"):
            expert(*bad)
    layer = type("Layer", (), dict(d=32))()
    SharedExpertStack([(layer, expert(bf, bf, bf), {})])
    with pytest.raises(TypeError, match="block 1"):
        SharedExpertStack([(layer, expert(bf, bf, bf), {}), (layer, expert(hf, hf, hf), {})])


def test_columns_of_one_wider_matrix_do_not_overlap():
    """Matrices of one pitch that lie beside each other in a wider one are accepted (the
    next refusal is the workspace's); a shared column, or another pitch, is not."""
    # x in columns 0 .. 63, out 64 .. 95, the residual 96 .. 127 of 128, 300 rows
    beside = dict(n=300, x=A, ldx=128, out=A + 128, ldo=128, res=A + 192, rdt=BF16, ldr=128, wsb=1)
    assert lin(**beside) == ENOMEM
    assert lin(**{**beside, "n": 1}) == ENOMEM
    # a narrow fp32 output in the same bytes: columns 64 .. 127 of 256 bytes
    assert lin(**{**beside, "res": None, "odt": F32, "ldo": 64}) == ENOMEM
    for bad in (dict(out=A + 112), dict(out=A + 144), dict(res=A + 176), dict(ldo=136),
                dict(ldr=120), dict(out=A + 240), dict(x=A + 16), dict(odt=F32, ldo=64)):
        assert lin(**{**beside, **bad}) == EINVAL, bad
    # the gradients of two halves of a matrix [rows][2 cols], into such a matrix
    both = dict(do=A, ldd=32, x=B, ldx=64, wg=C, wu=C + 128, ldw=128, pre=D, dt=BF16, n=40, rows=32,
                cols=64, act=2, dx=E_, lddx=64, dwg=F, dwu=F + 128, lddw=128, dbg=None, dbu=None,
                ws=F + 0x10000000, wsb=1, st=None)
    assert lib.moe_gated_linear_backward(*both.values()) == ENOMEM
    for bad in (dict(dwu=F + 112), dict(dwu=F + 144), dict(dx=C + 128, lddx=128),
                dict(dwg=C, dwu=F)):
        assert lib.moe_gated_linear_backward(*{**both, **bad}.values()) == EINVAL, bad


def test_plan_of_a_product():
    """What the planner says without a GPU: shapes are checked, decode batches stream
    the weights, many tokens take whole tiles, gradients report both products."""
    out = (ctypes.c_int32 * 7)()
    for bad in ((0, 0, 0, 8, 8), (0, 1, 1, 12, 8), (1, 0, 1, 8, 0)):
        assert lib.rvq_selftest_dense_plan(*bad, out) == EINVAL
    assert lib.rvq_selftest_dense_plan(0, 0, 1, 8, 8, None) == EINVAL
    for gated in (False, True):
        assert rvq.rvq_selftest_dense_plan(gated, False, 1, 2048, 7168) == (False, [("stream", 0, 0)])
        joint, ((way, cut, cols),) = rvq.rvq_selftest_dense_plan(gated, False, 4096, 2048, 7168)
        assert (joint, way, cut) == (False, "tiles", 1) and cols % 32 == 0
        joint, ways = rvq.rvq_selftest_dense_plan(gated, True, 1, 2048, 7168)
        assert not joint and [w[0] for w in ways] == ["stream", "tiles"]
        assert len(rvq.rvq_selftest_dense_plan(gated, True, 4096, 2048, 7168)[1]) == 2
