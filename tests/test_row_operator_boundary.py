"""Host-side argument checks of the log-probability and distillation entry
points (no GPU): fake addresses, so a call that passed its checks would reach a
launch.  The same checks run under ASan and UBSan below."""
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import lm_head_fp32_amd as lmh  # noqa: E402
from lm_head_fp32_amd import build as hbuild  # noqa: E402

OK, DTYPE, SHAPE, NULL, ALIGN, ALIAS = 0, 1, 2, 3, 4, 5
BF16, FP32, FP16 = lmh.LMH_BF16, lmh.LMH_FP32, lmh.LMH_FP16
MAX = 2 ** 63 - 1
# fake, 16-byte aligned device addresses far apart
Z, Y, T, LP, H, RK, TL, TT, ST, WS, G, GL, GH, TV = (0x1000000000 * (i + 1) for i in range(14))


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(lmh.library_path()):
        pytest.skip("liblmhead.so not built")
    return lmh.lib()


def _call(fn, order, base, **kw):
    assert set(kw) <= set(order), kw
    d = {**base, **kw}
    return fn(*(d[k] for k in order))


FWD = "z ld dt n V y ign t ts k lp h rk tl tt st ws wsb stream".split()
FWD_OK = dict(z=Z, ld=104, dt=FP32, n=10, V=100, y=Y, ign=-100, t=T, ts=1, k=6, lp=LP, h=H, rk=RK, tl=TL, tt=TT,
              st=ST, ws=WS, wsb=1 << 20, stream=None)


def test_logprobs_refusals(L):
    def f(**kw):
        return _call(L.lmhead_logprobs, FWD, FWD_OK, **kw)

    assert f(dt=FP16) == DTYPE and f(dt=7) == DTYPE
    for bad in (dict(n=-1), dict(n=MAX), dict(V=0), dict(V=-1), dict(V=MAX), dict(V=2 ** 30 + 1, ld=2 ** 30 + 4), dict(k=-1), dict(k=65), dict(V=5, k=6),
                dict(ld=96), dict(wsb=-1), dict(ts=2), dict(ts=-1), dict(ld=MAX // 4 * 4)):
        assert f(**bad) == SHAPE, bad
    for bad in (dict(z=None), dict(st=None), dict(tl=None), dict(tt=None), dict(y=None),
                dict(y=None, lp=None), dict(y=None, rk=None)):
        assert f(**bad) == NULL, bad
    for bad in (dict(z=Z + 4), dict(ld=102), dict(dt=BF16, ld=108), dict(y=Y + 2), dict(t=T + 1), dict(lp=LP + 2),
                dict(h=H + 1), dict(rk=RK + 2), dict(tl=TL + 2), dict(tt=TT + 1), dict(st=ST + 8), dict(ws=WS + 8)):
        assert f(**bad) == ALIGN, bad
    for bad in (dict(lp=Z), dict(h=LP + 4), dict(rk=Y), dict(tl=T), dict(tt=TL + 8), dict(st=LP),
                dict(st=Z + 16), dict(rk=T + 36)):
        assert f(**bad) == ALIAS, bad
    assert f(n=0, z=None, st=None, ws=None) == OK
    # the workspace of a few long rows
    need = L.lmhead_logprobs_workspace_bytes(2, 200000, 6)
    far = dict(n=2, V=200000, ld=200000)
    assert need > 0 and L.lmhead_logprobs_workspace_bytes(2, 100, 6) == 0
    assert f(**far, wsb=need - 1) == SHAPE and f(**far, ws=None) == NULL
    assert f(**far, ws=Z) == ALIAS and f(**far, ws=TL - 16) == ALIAS
    assert L.lmhead_logprobs_workspace_bytes(4, 0, 0) == -SHAPE
    assert L.lmhead_logprobs_workspace_bytes(-1, 8, 0) == -SHAPE
    assert L.lmhead_logprobs_workspace_bytes(4, 8, 9) == -SHAPE
    assert L.lmhead_logprobs_workspace_bytes(4, 100, 65) == -SHAPE
    for n in (0, 1, 8192, 2 ** 31 - 1):
        for V in (1, 2047, 131072, 2 ** 30):
            for k in (0, 1, 64):
                if k <= V:
                    assert L.lmhead_logprobs_workspace_bytes(n, V, k) >= 0


BWD = "z ld dt st y ign t ts gl gls gh ghs g ldg gt n V stream".split()
BWD_OK = dict(z=Z, ld=104, dt=FP32, st=ST, y=Y, ign=-100, t=T, ts=0, gl=GL, gls=1, gh=GH, ghs=0, g=G, ldg=104,
              gt=BF16, n=10, V=100, stream=None)


def test_logprobs_bwd_refusals(L):
    def f(**kw):
        return _call(L.lmhead_logprobs_bwd, BWD, BWD_OK, **kw)

    assert f(dt=FP16) == DTYPE and f(gt=FP16) == DTYPE
    for bad in (dict(n=-1), dict(V=0), dict(V=MAX), dict(ld=96), dict(ldg=96), dict(ts=2), dict(gls=3), dict(ghs=-1)):
        assert f(**bad) == SHAPE, bad
    for bad in (dict(z=None), dict(g=None), dict(st=None)):
        assert f(**bad) == NULL, bad
    for bad in (dict(z=Z + 8), dict(g=G + 8), dict(ldg=108), dict(st=ST + 4), dict(y=Y + 1), dict(t=T + 2),
                dict(gl=GL + 2), dict(gh=GH + 3)):
        assert f(**bad) == ALIGN, bad
    for bad in (dict(g=Z), dict(g=Z + 16), dict(g=Z, gt=FP32, ldg=108), dict(g=ST), dict(g=Y), dict(g=GL + 16),
                dict(g=GH - 16), dict(g=T)):
        assert f(**bad) == ALIAS, bad
    assert f(n=0, z=None, g=None, st=None) == OK


DF = "z ld dt n V y ldy v ldv vt k tail t ts loss st ws wsb stream".split()
DF_OK = dict(z=Z, ld=104, dt=FP32, n=10, V=100, y=Y, ldy=8, v=TV, ldv=7, vt=BF16, k=6, tail=0, t=T, ts=1, loss=LP,
             st=ST, ws=WS, wsb=1 << 20, stream=None)
DB = "z ld dt st y ldy v ldv vt k tail t ts gl gls g ldg gt n V stream".split()
DB_OK = dict(z=Z, ld=104, dt=FP32, st=ST, y=Y, ldy=8, v=TV, ldv=7, vt=BF16, k=6, tail=1, t=T, ts=1, gl=GL, gls=1,
             g=G, ldg=104, gt=FP32, n=10, V=100, stream=None)
DU = "z ld dt n V y ldy v ldv vt k tail t ts gl gls loss st g ldg gt ws wsb stream".split()
DU_OK = {**DF_OK, **DB_OK}


@pytest.mark.parametrize("name,order,base", [("lmhead_distill_fwd", DF, DF_OK), ("lmhead_distill_bwd", DB, DB_OK),
                                             ("lmhead_distill_fused", DU, DU_OK)])
def test_distill_refusals(L, name, order, base):
    fn = getattr(L, name)

    def f(**kw):
        return _call(fn, order, base, **kw)

    def only(*cases):
        return [c for c in cases if set(c) <= set(order)]

    for bad in only(dict(dt=FP16), dict(vt=FP16), dict(gt=FP16)):
        assert f(**bad) == DTYPE, bad
    for bad in only(dict(n=-1), dict(n=MAX), dict(V=0), dict(V=MAX), dict(k=-1), dict(k=257), dict(ld=96),
                    dict(ldy=5), dict(ldv=5), dict(ldy=MAX), dict(ts=2), dict(gls=2), dict(ldg=96),
                    dict(wsb=-1)):
        assert f(**bad) == SHAPE, bad
    for bad in only(dict(z=None), dict(y=None), dict(v=None), dict(st=None), dict(g=None),
                    dict(gl=None)):
        assert f(**bad) == NULL, bad
    for bad in only(dict(z=Z + 4), dict(ld=102), dict(y=Y + 2), dict(v=TV + 1), dict(v=TV + 2, vt=FP32),
                    dict(t=T + 2), dict(st=ST + 8), dict(loss=LP + 1), dict(gl=GL + 2),
                    dict(g=G + 4), dict(ldg=102), dict(gt=BF16, ldg=108)):
        assert f(**bad) == ALIGN, bad
    out = "g" if "g" in order else "st"
    for bad in only({out: Y}, {out: TV}, {out: T}, {out: Z + 16}, dict(loss=ST + 4),
                    dict(loss=Y + 4), dict(g=GL), dict(g=Z, gt=BF16), dict(g=Z, ldg=108), dict(st=G),
                    dict(st=TV)):
        if name == "lmhead_distill_bwd" and "st" in bad and bad["st"] != G:
            continue  # an input there
        if G in bad.values() and "g" not in order:
            continue
        assert f(**bad) == ALIAS, bad
    if "ws" in order:  # the workspace of a few long rows
        need = L.lmhead_distill_workspace_bytes(2, 200000)
        far = dict(n=2, V=200000, ld=200000, **({"ldg": 200000} if "ldg" in order else {}))
        assert need > 0 and L.lmhead_distill_workspace_bytes(10, 100) == 0
        assert f(**far, wsb=need - 1) == SHAPE and f(**far, ws=None) == NULL and f(**far, ws=WS + 8) == ALIGN
        for at in [Z, ST, Y, TV - 16] + ([G] if "g" in order else []):
            assert f(**far, ws=at) == ALIAS, at
    empty = {k: None for k in ("z", "y", "v", "st", "ws", "g", "gl") if k in order}
    assert f(n=0, **empty) == OK


def test_distill_workspace(L):
    assert L.lmhead_distill_workspace_bytes(4, 0) == -SHAPE
    assert L.lmhead_distill_workspace_bytes(-4, 8) == -SHAPE
    for n in (0, 1, 8192, 2 ** 31 - 1):
        for V in (1, 2047, 131072, 2 ** 30):
            assert L.lmhead_distill_workspace_bytes(n, V) >= 0


def test_python_arguments():
    """What the binding refuses before it reaches the library."""
    z = torch.zeros(4, 8)
    i = torch.zeros(4, dtype=torch.int32)
    for bad in (lambda: lmh.lmhead_logprobs(z, i), lambda: lmh.lmhead_logprobs(z.half(), i),
                lambda: lmh.lmhead_logprobs_bwd(z, z, i, z), lambda: lmh.lmhead_logprobs_bwd(z.int(), z, i, z),
                lambda: lmh.lmhead_distill_fwd(z, i[:, None], z), lambda: lmh.lmhead_distill_fwd(z.long(), i, z),
                lambda: lmh.lmhead_distill_bwd(z, z, i[:, None], z, None),
                lambda: lmh.lmhead_distill_fused(z, i[:, None], z, None)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(lmh.LmheadError):
        lmh.lmhead_logprobs_workspace_bytes(4, 8, 9)
    with pytest.raises(lmh.LmheadError):
        lmh.lmhead_distill_workspace_bytes(4, 0)
    # values per row
    with pytest.raises(TypeError):
        lmh._per_row(1.5, "temperature", 4)
    with pytest.raises(TypeError):
        lmh._per_row(z.double(), "temperature", 32)
    with pytest.raises(TypeError):
        lmh._per_row(z, "temperature", 32)
    assert lmh._per_row(None, "temperature", 4) == (None, 0)
    assert lmh._row_out(False, "rank", torch.int32, (4,), z) == (None, None)


def test_these_checks_pass_under_the_sanitizers():
    if os.environ.get("LMH_SANITIZED_CHILD"):
        pytest.skip("already inside the sanitized run")
    if not os.path.exists(hbuild.HOSTSAN_LIB):
        pytest.skip("liblmhead_hostsan.so not built (build() makes it)")
    rt = hbuild.sanitizer_runtime()
    if not rt:
        pytest.skip("clang's ASan runtime is not installed")
    code = ("import sys\n"
            f"sys.path.insert(0, {ROOT!r})\n"
            "import lm_head_fp32_amd as lmh\n"
            f"lmh._LIB_PATH = {hbuild.HOSTSAN_LIB!r}\n"
            "import pytest\n"
            f"sys.exit(pytest.main(['-q', '-s', '-p', 'no:cacheprovider', {os.path.abspath(__file__)!r}]))\n")
    env = dict(os.environ, LD_PRELOAD=rt, ASAN_OPTIONS="detect_leaks=0", LMH_SANITIZED_CHILD="1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env=env, capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert " passed" in r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr
