"""Host-side argument checks of the adapter and beam entry points (no GPU):
fake addresses, so a call that passed its checks would reach a launch.  The
same checks run under ASan and UBSan below."""
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
X, W, A, B, ID, SC, OUT, WS, G, DX, DA, DB = (0x1000000000 * (i + 1) for i in range(12))


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(lmh.library_path()):
        pytest.skip("liblmhead.so not built")
    return lmh.lib()


def _call(fn, order, base, **kw):
    assert set(kw) <= set(order), kw
    d = {**base, **kw}
    return fn(*(d[k] for k in order))


LOGITS = ("x ldx W ldw A lda sa B ldb sb ids scale n r out ldo dt M K V ws wsb stream").split()
LOGITS_OK = dict(x=X, ldx=64, W=W, ldw=64, A=A, lda=64, sa=512, B=B, ldb=8, sb=8 * 104, ids=ID, scale=SC,
                 n=3, r=8, out=OUT, ldo=104, dt=FP32, M=10, K=64, V=100, ws=WS, wsb=1 << 20, stream=None)


def test_logits_lora_refusals(L):
    def f(**kw):
        return _call(L.lmhead_logits_lora, LOGITS, LOGITS_OK, **kw)

    assert f(dt=FP16) == DTYPE and f(dt=9) == DTYPE
    for bad in (dict(M=-1), dict(K=-1), dict(V=-1), dict(r=0), dict(r=129), dict(n=-1), dict(n=MAX),
                dict(M=MAX), dict(wsb=-1), dict(wsb=16), dict(ldx=56), dict(ldw=56), dict(lda=56),
                dict(ldb=0), dict(ldo=96), dict(sa=504), dict(sb=8), dict(sa=MAX // 8 * 8),
                dict(sb=-8), dict(lda=MAX // 8 * 8)):
        assert f(**bad) == SHAPE, bad
    for bad in (dict(x=None), dict(W=None), dict(A=None), dict(B=None), dict(ids=None), dict(out=None),
                dict(ws=None)):
        assert f(**bad) == NULL, bad
    for bad in (dict(x=X + 2), dict(A=A + 8), dict(B=B + 8), dict(ids=ID + 2), dict(scale=SC + 1),
                dict(ws=WS + 8), dict(ldx=68), dict(lda=68), dict(ldb=12), dict(sa=516), dict(sb=836),
                dict(ldo=102), dict(dt=BF16, ldo=108)):
        assert f(**bad) == ALIGN, bad
    for bad in (dict(out=X), dict(out=A), dict(out=B), dict(out=ID - 400), dict(out=SC - 16),
                dict(ws=X), dict(ws=OUT), dict(ws=A), dict(ws=W + 16), dict(out=W + 32)):
        assert f(**bad) == ALIAS, bad
    # empty outputs touch nothing
    assert f(M=0, x=None, ids=None, out=None, ws=None) == OK
    assert f(V=0, W=None, B=None, out=None, ws=None) == OK


BWD = ("g ldg x ldx A lda sa B ldb sb ids scale n r dX lddx dA ldda sda dB lddb sdb acc M K V ws wsb "
       "stream").split()
BWD_OK = dict(g=G, ldg=104, x=X, ldx=64, A=A, lda=64, sa=512, B=B, ldb=8, sb=8 * 104, ids=ID, scale=SC,
              n=3, r=8, dX=DX, lddx=64, dA=DA, ldda=64, sda=512, dB=DB, lddb=8, sdb=832, acc=0, M=10,
              K=64, V=100, ws=WS, wsb=1 << 30, stream=None)


def test_lora_bwd_refusals(L):
    def f(**kw):
        return _call(L.lmhead_lora_bwd, BWD, BWD_OK, **kw)

    for bad in (dict(M=-1), dict(r=0), dict(r=129), dict(n=-1), dict(n=2 ** 23), dict(M=2 ** 22 + 1, wsb=MAX),
                dict(wsb=-5), dict(wsb=100), dict(ldg=96), dict(lddx=60), dict(ldda=60), dict(lddb=4),
                dict(sda=508), dict(sdb=4), dict(V=2 ** 31 - 1, n=2), dict(sda=MAX // 4 * 4)):
        assert f(**bad) == SHAPE, bad
    for bad in (dict(g=None), dict(x=None), dict(A=None), dict(B=None), dict(ids=None), dict(ws=None)):
        assert f(**bad) == NULL, bad
    for bad in (dict(g=G + 2), dict(dX=DX + 4), dict(dA=DA + 4), dict(dB=DB + 8), dict(lddx=66),
                dict(ldda=66), dict(lddb=10), dict(sda=514), dict(sdb=834), dict(ws=WS + 4)):
        assert f(**bad) == ALIGN, bad
    for bad in (dict(dX=X), dict(dA=A), dict(dB=B), dict(dX=G), dict(dB=DX), dict(dA=DB + 16),
                dict(ws=DX), dict(ws=G), dict(dX=ID - 16)):
        assert f(**bad) == ALIAS, bad
    # nothing asked for
    assert f(dX=None, dA=None, dB=None, ws=None) == OK


SEL = "z ld dt B W V s fin eos k os op ot of ws wsb stream".split()
SEL_OK = dict(z=X, ld=104, dt=FP32, B=5, W=4, V=100, s=SC, fin=ID, eos=2, k=6, os=OUT, op=A, ot=B, of=DX,
              ws=WS, wsb=1 << 20, stream=None)


def test_beam_select_refusals(L):
    def f(**kw):
        return _call(L.lmhead_beam_select, SEL, SEL_OK, **kw)

    assert f(dt=FP16) == DTYPE
    for bad in (dict(B=-1), dict(W=0), dict(W=65), dict(V=0), dict(k=0), dict(k=65), dict(V=1, k=5),
                dict(V=2 ** 29), dict(ld=96), dict(wsb=-1), dict(wsb=64), dict(B=MAX), dict(V=MAX),
                dict(B=2 ** 23 + 1), dict(B=2 ** 22, V=20000)):
        assert f(**bad) == SHAPE, bad
    for bad in ("z", "s", "os", "op", "ot", "of", "ws"):
        assert f(**{bad: None}) == NULL, bad
    for bad in (dict(z=X + 4), dict(ld=102), dict(s=SC + 2), dict(os=OUT + 1), dict(op=A + 2),
                dict(ot=B + 2), dict(ws=WS + 8), dict(dt=BF16, ld=100)):
        assert f(**bad) == ALIGN, bad
    for bad in (dict(os=X), dict(op=OUT), dict(ot=A + 4), dict(of=ID), dict(os=SC), dict(ws=X),
                dict(ws=SC & ~15), dict(op=SC), dict(of=SC), dict(os=ID),
                dict(k=4, os=SC + 4), dict(k=4, of=ID + 1), dict(k=4, os=SC, of=SC + 4),
                dict(k=4, of=ID, op=ID), dict(k=4, os=SC, ws=SC)):
        assert f(**bad) == ALIAS, bad
    assert f(B=0, z=None, s=None, ws=None) == OK
    assert L.lmhead_beam_select_workspace_bytes(1, 65, 10, 1) == -SHAPE
    assert L.lmhead_beam_select_workspace_bytes(0, 4, 10, 1) == 0


RE = "s so sr sh d do dr dh p l no B wi wo h T pb stream".split()
RE_OK = dict(s=X, so=40960, sr=2048, sh=512, d=OUT, do=40960, dr=2048, dh=512, p=ID, l=SC, no=2, B=5, wi=4,
             wo=4, h=4, T=64, pb=8, stream=None)


def test_beam_reorder_refusals(L):
    def f(**kw):
        return _call(L.lmhead_beam_reorder, RE, RE_OK, **kw)

    for bad in (dict(no=-1), dict(B=-1), dict(wi=-1), dict(wo=65), dict(wi=65), dict(h=-1), dict(T=-1),
                dict(pb=-1), dict(so=-8), dict(dr=-8), dict(dh=511), dict(dr=2047), dict(do=40959),
                dict(dr=0), dict(wi=0), dict(so=MAX), dict(do=MAX), dict(T=2 ** 31 - 1, pb=2 ** 31 - 1),
                dict(B=2 ** 31 - 1), dict(no=2 ** 31), dict(dr=512, dh=512)):
        assert f(**bad) == SHAPE, bad
    for bad in ("s", "d", "p"):
        assert f(**{bad: None}) == NULL, bad
    assert f(p=ID + 2) == ALIGN and f(l=SC + 1) == ALIGN
    for bad in (dict(d=X, dr=4096, do=81920), dict(d=X, wo=3), dict(d=X + 1), dict(d=ID), dict(d=SC),
                dict(s=OUT + 64), dict(d=X, do=40968)):
        assert f(**bad) == ALIAS, bad
    for none in ("no", "B", "wo", "h", "T", "pb"):
        assert f(**{none: 0}) == OK, none


def test_beam_reorder_of_long_runs(L):
    """A run of one position (a whole row of a state without lengths) is bound
    by the launch and the spans, not by 31 bits."""
    def f(pb, **kw):
        far = dict(no=1, h=1, T=1, sr=pb, dr=pb, so=0, do=0, d=X + 2 ** 46, p=2 ** 50, l=None, pb=pb)
        return _call(L.lmhead_beam_reorder, RE, RE_OK, **{**far, **kw})

    # the sizes pass: what is refused is the missing parent, or the overlap
    for pb in (2 ** 31 - 1, 2 ** 31, 2 ** 31 + 1, 2 ** 33 - 4096, 2 ** 39):
        assert f(pb, p=None) == NULL, pb
    assert f(2 ** 31, B=1, d=X + 2 ** 31) == ALIAS
    assert f(2 ** 31, B=1, p=X + 2 ** 46 + 2 ** 33 - 8) == ALIAS
    # past the launch, past the spans, past 64 bits
    assert f(2 ** 34, B=1) == SHAPE
    for pb, T in ((2 ** 44 + 1, 1), (2 ** 43, 3), (2 ** 62, 2), (2 ** 62, 2 ** 31 - 1), (MAX, 1), (MAX, MAX)):
        assert f(pb, T=T, B=1) == SHAPE, (pb, T)


def test_workspace_sizes(L):
    """Every size, zero included, has a workspace size (no division by a size)."""
    for M in (0, 1, 16, 17, 256, 257, 4096, 2 ** 22):
        for K in (0, 1, 255, 8192):
            for V in (0, 1, 257, 32768):
                for r in (1, 16, 17, 64, 128):
                    for dt in (FP32, BF16):
                        assert L.lmhead_logits_lora_workspace_bytes(M, K, V, r, dt) >= 0
                    for n in (0, 1, 300):
                        assert L.lmhead_lora_bwd_workspace_bytes(M, K, V, r, n) > 0
    assert L.lmhead_logits_lora_workspace_bytes(2 ** 22 + 1, 8, 8, 8, FP32) == -SHAPE
    assert L.lmhead_logits_lora_workspace_bytes(8, 8, 8, 8, FP16) == -DTYPE
    assert L.lmhead_lora_bwd_workspace_bytes(8, 8, 2 ** 31 - 1, 8, 2) == -SHAPE
    # the grouping of the tokens reads every id for every adapter
    assert L.lmhead_lora_bwd_workspace_bytes(2 ** 22, 8, 8, 8, 2 ** 17 - 2) > 0
    assert L.lmhead_lora_bwd_workspace_bytes(2 ** 22, 8, 8, 8, 2 ** 17 - 1) == -SHAPE


def test_python_arguments():
    """What the binding refuses before it reaches the library."""
    cpu = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        lmh.lmhead_logits_lora(cpu, cpu, cpu[None], cpu[None], torch.zeros(4, dtype=torch.int32))
    with pytest.raises(TypeError):
        lmh.lmhead_lora_bwd(cpu, cpu, cpu[None], cpu[None], torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError):
        lmh.lmhead_beam_select(cpu.float(), torch.zeros(4))
    with pytest.raises(TypeError):
        lmh.lmhead_beam_select(cpu.half(), torch.zeros(2, 2))
    with pytest.raises(TypeError):
        lmh.lmhead_beam_reorder(cpu, torch.zeros(2, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        lmh.lmhead_beam_reorder(cpu, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError):
        lmh.lmhead_beam_reorder(cpu, torch.zeros(2, 2, dtype=torch.int32), beam_dim=5)
    with pytest.raises(ValueError):
        lmh.lmhead_beam_reorder(cpu, torch.zeros(2, 2, dtype=torch.int32), lengths=torch.zeros(2))
    with pytest.raises(lmh.LmheadError):
        lmh.lmhead_logits_lora_workspace_bytes(4, 8, 8, 200)
    with pytest.raises(lmh.LmheadError):
        lmh.lmhead_lora_bwd_workspace_bytes(-1, 8, 8, 4, 1)
    with pytest.raises(lmh.LmheadError):
        lmh.lmhead_beam_select_workspace_bytes(1, 4, 1, 5)


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
