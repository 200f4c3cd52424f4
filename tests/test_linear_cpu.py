"""Host-side checks of the target model's dense side that need no GPU: every refusal comes back before the
device is touched (no kernel is launched here), and the plain forms of the tests hold against each other."""
import os

import pytest

import speculative_decoding_verification_59_gb300 as sv

FAKE, WS = 1 << 20, 1 << 24          # aligned addresses that are never dereferenced
F32, BF16, E4M3 = sv.SPEC_DTYPE_F32, sv.SPEC_DTYPE_BF16, sv.SPEC_DTYPE_E4M3
INVALID, DTYPE, ALIGN = sv.SPEC_ERR_INVALID_ARG, sv.SPEC_ERR_UNSUPPORTED_DTYPE, sv.SPEC_ERR_MISALIGNED


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(sv.lib_path()):
        import __graft_entry__
        __graft_entry__.build()
    return sv.load_library()


def norm(**kw):
    a = dict(x=FAKE, xt=BF16, xs=256, res=FAKE, st=BF16, rs=256, w=FAKE, eps=1e-6, rows=3, dim=256, sum=FAKE, ss=256, out=FAKE,
             ot=BF16, scale=None, pitch=0)
    a.update(kw)
    return sv.load_library().spec_add_norm(*a.values(), None)


def act(**kw):
    a = dict(gate=FAKE, up=FAKE, t=BF16, gs=512, us=512, act=0, rows=3, dim=256, out=FAKE, ot=BF16, scale=None, pitch=0)
    a.update(kw)
    return sv.load_library().spec_gated_act(*a.values(), None)


def quantize(**kw):
    a = dict(x=FAKE, t=BF16, xs=256, rows=3, dim=256, high=1, out=FAKE, scale=FAKE, pitch=4)
    a.update(kw)
    return sv.load_library().spec_quantize_e4m3(*a.values(), None)


def matmul(**kw):
    a = dict(x=FAKE, xld=256, xs=FAKE, xss=4, w=FAKE, wld=256, ws=FAKE, wss=2, M=3, N=200, K=256, out=FAKE, ot=BF16, old=200, work=WS,
             wb=1 << 30)
    a.update(kw)
    return sv.load_library().spec_matmul_e4m3(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(xt=E4M3), DTYPE), (dict(st=E4M3), DTYPE), (dict(ot=9), DTYPE), (dict(x=None), INVALID), (dict(out=None), INVALID),
    (dict(rows=-1), INVALID), (dict(dim=0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(res=None), INVALID),                       # a sum of nothing
    (dict(ot=E4M3), INVALID), (dict(ot=E4M3, scale=FAKE, pitch=2), INVALID), (dict(rows=1 << 27), INVALID),
    (dict(x=FAKE + 2), ALIGN), (dict(xs=260), ALIGN), (dict(xt=F32, xs=258), ALIGN), (dict(res=FAKE + 8), ALIGN),
    (dict(rs=257), ALIGN), (dict(sum=FAKE + 4), ALIGN), (dict(ss=4), ALIGN), (dict(w=FAKE + 2), ALIGN), (dict(dim=252), ALIGN),
    (dict(ot=E4M3, scale=FAKE, pitch=4, dim=248), ALIGN), (dict(out=FAKE + 8), ALIGN), (dict(ot=E4M3, scale=FAKE + 2, pitch=4), ALIGN),
    (dict(ss=248), INVALID), (dict(ss=0), INVALID), (dict(ss=-128), INVALID),           # rows of the sum that overlap
    (dict(rows=0), sv.SPEC_OK), (dict(rows=0, x=None, out=None), sv.SPEC_OK)])
def test_add_norm_refusals(kw, want):
    assert norm(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(t=E4M3), DTYPE), (dict(ot=7), DTYPE), (dict(gate=None), INVALID), (dict(up=None), INVALID), (dict(act=2), INVALID),
    (dict(act=-1), INVALID), (dict(rows=-3), INVALID), (dict(dim=-8), INVALID), (dict(ot=E4M3), INVALID), (dict(out=None), INVALID),
    (dict(gate=FAKE + 4), ALIGN), (dict(up=FAKE + 8), ALIGN), (dict(gs=500), ALIGN), (dict(us=511), ALIGN), (dict(dim=12), ALIGN),
    (dict(ot=E4M3, scale=FAKE, pitch=3, dim=24), ALIGN), (dict(rows=0), sv.SPEC_OK)])
def test_gated_act_refusals(kw, want):
    assert act(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(t=E4M3), DTYPE), (dict(x=None), INVALID), (dict(out=None), INVALID), (dict(scale=None), INVALID), (dict(high=64), INVALID),
    (dict(high=0), INVALID), (dict(pitch=2), INVALID), (dict(high=128, pitch=1), INVALID), (dict(rows=-1), INVALID),
    (dict(dim=0), INVALID), (dict(dim=24), ALIGN), (dict(x=FAKE + 8), ALIGN), (dict(xs=250), ALIGN), (dict(out=FAKE + 1), ALIGN),
    (dict(rows=0), sv.SPEC_OK)])
def test_quantize_refusals(kw, want):
    assert quantize(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(ot=E4M3), DTYPE), (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(K=0), INVALID), (dict(x=None), INVALID),
    (dict(xs=None), INVALID), (dict(w=None), INVALID), (dict(ws=None), INVALID), (dict(out=None), INVALID), (dict(work=None), INVALID),
    (dict(xld=240), INVALID), (dict(wld=240), INVALID), (dict(old=199), INVALID), (dict(xss=2), INVALID), (dict(wss=1), INVALID),
    (dict(xld=264), ALIGN), (dict(wld=260), ALIGN), (dict(x=FAKE + 8), ALIGN), (dict(w=FAKE + 4), ALIGN), (dict(xs=FAKE + 4), ALIGN),
    (dict(xss=6), ALIGN), (dict(ws=FAKE + 2), ALIGN), (dict(out=FAKE + 1), ALIGN), (dict(ot=F32, out=FAKE + 2), ALIGN),
    (dict(work=WS + 64), ALIGN), (dict(wb=16), sv.SPEC_ERR_WORKSPACE_TOO_SMALL), (dict(K=2147483647, xld=1 << 31, wld=1 << 31, wss=1 << 30), INVALID),
    (dict(xld=1 << 41), INVALID), (dict(M=0, x=None), sv.SPEC_OK), (dict(N=0, w=None), sv.SPEC_OK)])
def test_matmul_refusals(kw, want):
    assert matmul(**kw) == want


def test_matmul_workspace():
    size = sv.load_library().spec_matmul_workspace_size
    assert size(-1, 4, 4) == 0 and size(4, -1, 4) == 0 and size(4, 4, 0) == 0
    assert size(0, 4, 4) >= 256 and size(512, 4096, 4096) >= 256


def test_helpers_refuse_tensors_that_are_not_on_a_gpu():
    torch = pytest.importorskip("torch")
    x = torch.zeros((2, 128), dtype=torch.bfloat16)
    q = torch.zeros((2, 128), dtype=torch.uint8).view(torch.float8_e4m3fn)
    for call in (lambda: sv.add_norm(x), lambda: sv.gated_act(x), lambda: sv.quantize_e4m3(x),
                 lambda: sv.matmul_e4m3(q, torch.ones(2, 1), q, torch.ones(1, 1))):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError, match="torch tensor"):
        sv.add_norm(x.float().numpy())
    with pytest.raises(ValueError, match="act must be"):
        sv.gated_act(x, act="relu")
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        sv.add_norm(x, dtype=torch.float16)
    for call in (sv.add_norm, sv.gated_act):
        with pytest.raises(ValueError, match="without e4m3"):
            call(x, e4m3=True, dtype=torch.float32)


def test_plain_forms():
    torch = pytest.importorskip("torch")
    import linear_ref as R
    x, xs, w, ws = R.problem(1, 5, 130, 144, device="cpu")
    ref, mags = R.matmul(x, xs, w, ws)
    assert ref.shape == (5, 130) and (mags >= ref.abs()).all()
    want = sum(float(x[3, k]) * float(xs[3, k // 128]) * float(w[129, k]) * float(ws[1, k // 128]) for k in range(144))
    assert abs(ref[3, 129] - want) <= 1e-9 * mags[3, 129]
    # a block's order of magnitude wrong, or its neighbour's scale, is seen
    y = torch.randn((4, 256), dtype=torch.float64)
    top = R.block_top(y)
    q = (y * (448 / top).repeat_interleave(128, 1)).to(torch.float32).to(torch.float8_e4m3fn)
    R.check_e4m3(q, (top / 448).float(), y)
    with pytest.raises(AssertionError):
        R.check_e4m3(q, (top / 448).float().flip(1), y)
    with pytest.raises(AssertionError):
        R.check_e4m3(q.roll(1, 1), (top / 448).float(), y)
