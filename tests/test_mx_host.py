"""Host side of the microscaled operators (no GPU): sizes and refusals before any
launch, in the library and in the binding; the tests' own definition of the formats."""
import pytest
import torch

import moe_expert_ffn_router_gb300 as rvq
from tests import mx_ref as X

lib = rvq._lib
A = 0x10000000       # fake, aligned "device" addresses far apart (never dereferenced)
B, C, D, E_, F = (A + i * 0x10000000 for i in range(1, 6))
OK, EINVAL, EALIGN, ENOMEM = 0, 1, 2, 3
F32, BF16, F16 = 0, 1, 2
F8, F4 = rvq.MOE_MX_F8, rvq.MOE_MX_F4


def test_sizes():
    assert rvq.moe_mx_code_bytes(F8, 1, 8) == 128 and rvq.moe_mx_code_bytes(F4, 1, 8) == 64
    assert rvq.moe_mx_code_bytes(F8, 5, 136) == 5 * 256
    assert rvq.moe_mx_code_bytes(F4, 2048, 7168) == 2048 * 3584
    assert rvq.moe_mx_scale_bytes(1, 8) == 512 and rvq.moe_mx_scale_bytes(129, 136) == 4 * 512
    assert rvq.moe_mx_scale_bytes(2048, 7168) == 2048 * 7168 // 32
    # past 2^31 and 2^32 bytes
    assert rvq.moe_mx_code_bytes(F8, 1 << 20, 1 << 16) == 1 << 36
    for r, c in ((0, 8), (-1, 8), (1, 0), (1, 12), (1 << 24, 8), (1, 1 << 24), (1 << 23, 1 << 23)):
        assert rvq.moe_mx_code_bytes(F8, r, c) == 0 and rvq.moe_mx_scale_bytes(r, c) == 0
    assert rvq.moe_mx_code_bytes(2, 1, 8) == 0


def test_quantize_refusals():
    base = dict(x=A, ldx=64, xdt=BF16, rows=4, cols=64, fmt=F8, codes=B, scales=C, st=None)

    def q(**kw):
        return lib.moe_mx_quantize(*{**base, **kw}.values())

    for bad in (dict(rows=0), dict(cols=60), dict(cols=0), dict(xdt=3), dict(x=None), dict(ldx=56),
                dict(ldx=65), dict(fmt=2), dict(fmt=-1), dict(codes=None), dict(scales=None),
                dict(codes=A), dict(scales=A + 480), dict(scales=B + 512 - 32),
                dict(codes=A - 4 * 128 + 32), dict(codes=C + 480)):
        assert q(**bad) == EINVAL, bad
    for bad in (dict(x=A + 8), dict(codes=B + 16), dict(scales=C + 16)):
        assert q(**bad) == EALIGN, bad
    assert b"aligned" in lib.rvq_last_error()


def test_dequantize_refusals():
    base = dict(codes=A, scales=B, fmt=F4, rows=4, cols=64, out=C, odt=BF16, ldo=64, st=None)

    def q(**kw):
        return lib.moe_mx_dequantize(*{**base, **kw}.values())

    for bad in (dict(rows=0), dict(cols=4), dict(odt=9), dict(out=None), dict(ldo=32), dict(fmt=7),
                dict(codes=None), dict(scales=None), dict(out=A + 192), dict(out=B)):
        assert q(**bad) == EINVAL, bad
    for bad in (dict(out=C + 8), dict(codes=A + 16), dict(scales=B + 8)):
        assert q(**bad) == EALIGN, bad


def test_join_refusals():
    base = dict(h=A, hdt=F32, y=B, ydt=BF16, n=4, d=64, alpha=1.0, gate=None, kind=0, gdt=F32,
                post=1, wpost=None, wpre=None, wdt=F32, eps=1e-6, ho=C, xn=D, xdt=BF16, fmt=F8,
                codes=E_, scales=F, rstd=None, st=None)

    def join(**kw):
        return lib.moe_norm_join_mx(*{**base, **kw}.values())

    for bad in (dict(n=0), dict(d=60), dict(d=16392), dict(hdt=3), dict(ydt=-1), dict(y=None),
                dict(kind=2), dict(gate=E_, kind=0), dict(post=0, wpost=A + 0x100000),
                dict(eps=-1.0), dict(eps=float("inf")), dict(fmt=3), dict(codes=None),
                dict(scales=None), dict(ho=B), dict(xn=A), dict(ho=C, xn=C), dict(codes=A),
                dict(codes=B), dict(codes=C), dict(codes=D), dict(scales=E_), dict(scales=C),
                dict(rstd=C), dict(rstd=E_), dict(wpre=E_), dict(wpre=C),
                dict(gate=F, kind=2), dict(ho=A + 16)):
        assert join(**bad) == EINVAL, bad
    for bad in (dict(h=A + 4), dict(y=B + 8), dict(ho=C + 8), dict(xn=D + 8), dict(codes=E_ + 16),
                dict(scales=F + 16), dict(wpre=E_ + 0x100008), dict(rstd=A + 0x100004)):
        assert join(**bad) == EALIGN, bad


def test_binding_refusals():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    codes, scales = torch.zeros(512, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)
    with pytest.raises(ValueError, match="x: shape"):
        rvq.moe_mx_quantize(x, 4, 72, codes, scales)
    with pytest.raises(ValueError, match="codes"):
        rvq.moe_mx_quantize(x, 4, 64, codes[:256], scales)
    with pytest.raises(ValueError, match="codes scales"):
        rvq.moe_mx_quantize(x, 4, 64, codes, scales[:256])
    with pytest.raises(TypeError, match="codes"):
        rvq.moe_mx_quantize(x, 4, 64, codes.view(torch.int8), scales)
    with pytest.raises(TypeError, match="unsupported dtype"):
        rvq.moe_mx_quantize(x.double(), 4, 64, codes, scales)
    with pytest.raises(ValueError, match="contiguous"):
        rvq.moe_mx_dequantize(codes, scales, 4, 64, x.t().contiguous().t())
    with pytest.raises(ValueError, match="y"):
        rvq.moe_norm_join_mx(x, 4, 128, None, codes, scales)


def test_definition():
    """The tests' formats: every value a fixed point, ties, ends, padding, layout."""
    v4 = X.values(F4)
    assert v4.tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6]
    v8 = X.values(F8)
    assert v8[126] == 448 and v8[1] == 2.0 ** -9 and torch.isnan(v8[127])
    for t, v in ((torch.float8_e4m3fn, v8),):
        assert torch.equal(torch.arange(256, dtype=torch.uint8).view(t).double().nan_to_num(-1),
                           v.nan_to_num(-1))
    for fmt, v in ((F8, v8), (F4, v4)):
        f = v[torch.isfinite(v)]
        assert torch.equal(X.round_code(f, fmt), f)
    assert X.round_code(torch.tensor([.25, .75, 2.5, 3.5, 5., 7.]).double(), F4).tolist() == \
        [0, 1, 2, 4, 4, 6]
    x = torch.zeros((130, 136))
    x[0, 0], x[1, 33], x[129, 135] = 3.0, -448.0, 2.0 ** -126
    for fmt in (F8, F4):
        q, b = X.quantize(x, fmt)
        assert q.shape == (130, 256) and b.shape == (130, 8)
        assert b[0, 0] == 1 - X.LEAD[fmt] + 127 and b[1, 1] == 8 - X.LEAD[fmt] + 127
        assert b[129, 4] == 0 and b[2, 3] == 0
        tiles = X.to_tiles(b)
        assert tiles.numel() == rvq.moe_mx_scale_bytes(130, 136)
        assert torch.equal(X.from_tiles(tiles, 130, 136), b)
        assert tiles[(1 * 2 + 1) * 512 + 1 * 16 + 0] == b[129, 4]
        codes = X.pack(q, fmt)
        assert codes.numel() == rvq.moe_mx_code_bytes(fmt, 130, 136)
        got = X.dequantize(codes.view(-1), tiles, 130, 136, fmt)
        # 448 over its F4 scale is 7: ends at 6
        assert got[0, 0] == 3 and got[1, 33] == (-448 if fmt == F8 else -384)
        X.check_quantized(codes, tiles, 130, 136, fmt, x.double(), torch.zeros(130, 136), "self")


def test_product_sizes():
    for f in (rvq.moe_mx_linear_workspace_bytes, rvq.moe_mx_gated_linear_workspace_bytes):
        for n, r, c in ((1, 8, 8), (7, 256, 512), (4096, 2048, 7168)):
            assert f(n, r, c) >= 256
        for n, r, c in ((0, 8, 8), (1, 12, 8), (1, 8, 12), (1, 0, 8), (-1, 8, 8), (1 << 24, 8, 8)):
            assert f(n, r, c) == 0


def test_linear_refusals():
    base = dict(x=A, xs=B, xf=F8, w=C, wsc=D, wf=F4, bias=None, n=4, rows=32, cols=64, act=0,
                alpha=1.0, res=None, rdt=F32, ldr=0, out=E_, odt=BF16, ldo=32, ws=F, wsb=1 << 20,
                st=None)

    def lin(**kw):
        return lib.moe_mx_linear(*{**base, **kw}.values())

    G = F + 0x10000000
    for bad in (dict(n=0), dict(rows=12), dict(cols=60), dict(rows=0), dict(xf=2), dict(wf=-1),
                dict(act=5), dict(act=-1), dict(x=None), dict(xs=None), dict(w=None),
                dict(wsc=None), dict(out=None), dict(ldo=24), dict(ldo=31), dict(odt=7),
                dict(res=G, rdt=5, ldr=32), dict(res=G, ldr=24), dict(ws=None), dict(ws=F + 16),
                dict(out=A), dict(out=B + 64), dict(out=A + 4 * 128 - 16), dict(out=D),
                dict(out=C + 32 * 64 - 16), dict(bias=E_),
                dict(res=E_, rdt=F32, ldr=32), dict(res=E_ + 16, rdt=BF16, ldr=32),
                dict(res=E_, rdt=BF16, ldr=40)):
        assert lin(**bad) == EINVAL, bad
    for bad in (dict(x=A + 16), dict(xs=B + 16), dict(w=C + 8), dict(wsc=D + 16), dict(out=E_ + 4),
                dict(bias=G + 4), dict(res=G + 8, ldr=32)):
        assert lin(**bad) == EALIGN, bad
    assert lin(wsb=255) == ENOMEM


def test_gated_refusals():
    G = F + 0x10000000
    base = dict(x=A, xs=A + 0x100000, xf=F8, wg=B, wgs=B + 0x100000, wu=C, wus=C + 0x100000, wf=F4,
                bg=None, bu=None, n=4, rows=32, cols=64, act=2, out=D, odt=BF16, ldo=32, codes=None,
                scales=None, of=F8, ws=F, wsb=1 << 20, st=None)

    def gat(**kw):
        return lib.moe_mx_gated_linear(*{**base, **kw}.values())

    mx = dict(out=None, codes=E_, scales=G)
    for bad in (dict(n=0), dict(rows=4), dict(cols=4), dict(xf=5), dict(wf=2), dict(act=9),
                dict(x=None), dict(wg=None), dict(wus=None), dict(out=None), dict(ldo=16),
                dict(odt=3), dict(out=A), dict(out=B), dict(out=C + 0x100000), dict(ws=None),
                dict(codes=E_, scales=G), dict(codes=E_), dict(**mx, of=2),
                dict(out=None, codes=E_), dict(out=None, scales=E_),
                dict(out=None, codes=E_, scales=E_), dict(out=None, codes=A, scales=G),
                dict(out=None, codes=E_, scales=C), dict(bg=D), dict(bu=D)):
        assert gat(**bad) == EINVAL, bad
    for bad in (dict(x=A + 16), dict(wu=C + 8), dict(out=D + 8), dict(bg=G + 8), dict(bu=G + 8),
                dict(out=None, codes=E_ + 16, scales=G)):
        assert gat(**bad) == EALIGN, bad
    assert gat(wsb=0) == ENOMEM


def test_product_binding_refusals():
    u8 = torch.uint8
    x, xs = torch.zeros(512, dtype=u8), torch.zeros(512, dtype=u8)
    w, ws_ = torch.zeros(8 * 64, dtype=u8), torch.zeros(512, dtype=u8)
    out, ws = torch.zeros((4, 8)), torch.zeros(256, dtype=u8)
    with pytest.raises(ValueError, match="x:"):
        rvq.moe_mx_linear(x[:256], xs, w, ws_, 4, 8, 64, out, ws)
    with pytest.raises(ValueError, match="w:"):
        rvq.moe_mx_linear(x, xs, w, ws_, 4, 8, 64, out, ws, wfmt=F8)
    with pytest.raises(ValueError, match="out"):
        rvq.moe_mx_linear(x, xs, w, ws_, 4, 8, 64, out[:3], ws)
    with pytest.raises(TypeError, match="bias"):
        rvq.moe_mx_linear(x, xs, w, ws_, 4, 8, 64, out, ws, bias=torch.zeros(8).double())
    with pytest.raises(ValueError, match="wu scales"):
        rvq.moe_mx_gated_linear(x, xs, w, ws_, w, ws_[:256], 4, 8, 64, out, ws)
    with pytest.raises(ValueError, match="out scales"):
        rvq.moe_mx_gated_linear(x, xs, w, ws_, w, ws_, 4, 8, 64, x, ws, out_scales=ws)


def test_tensors_of_another_device():
    """Tensors that are not on the call's device are refused before the library is
    called (here: all are on the CPU, the call would be on cuda:0)."""
    class Fake:
        device_index, cuda_stream = 0, 0

    u8 = torch.uint8
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    c, s = torch.zeros(512, dtype=u8), torch.zeros(512, dtype=u8)
    w, ws = torch.zeros(8 * 64, dtype=u8), torch.zeros(256, dtype=u8)
    out, i32 = torch.zeros((4, 8)), torch.zeros(8, dtype=torch.int32)
    st = dict(stream=Fake())
    for call in (lambda: rvq.moe_mx_quantize(x, 4, 64, c, s, **st),
                 lambda: rvq.moe_mx_dequantize(c, s, 4, 64, x, **st),
                 lambda: rvq.moe_norm_join_mx(x, 4, 64, None, c, s, **st),
                 lambda: rvq.moe_mx_linear(c, s, w, s, 4, 8, 64, out, ws, **st),
                 lambda: rvq.moe_mx_gated_linear(c, s, w, s, w, s, 4, 8, 64, out, ws, **st),
                 lambda: rvq.moe_route_scored(out, 4, 8, 2, i32, out[:1], i32.new_zeros(9), i32,
                                              ws, **st),
                 lambda: rvq.moe_route_scored_backward(out[:1], out, i32, 4, 8, 2, out, **st)):
        with pytest.raises(ValueError, match="on cpu, the call on cuda:0"):
            call()
