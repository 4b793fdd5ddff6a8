"""Host-side contract of the other token mixers (CPU only: every call below is refused before a kernel is
launched), and the same under AddressSanitizer and UndefinedBehaviorSanitizer."""
import ctypes
import os
import re
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CLANG = "/opt/rocm/llvm/bin/clang"
A = 0x10000  # an aligned address that is never read


@pytest.fixture(scope="module")
def G():
    import gated_delta_rule_34_amd as G

    return G


def test_exports_every_declared_symbol(G):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "gdn_hybrid.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(gdn_[a-z0-9_]+)\s*\(", src)))
    assert set(names) == set(G.HYBRID_EXPORTED)
    for n in names:
        assert hasattr(ctypes.CDLL(G.LIB_PATH), n), n
        assert G.layer._fn(n) is not None


def call(G, name, p, *args):
    return G.layer._fn(name)(ctypes.byref(p), *args)


def filled(p, v, kw):
    for k, x in {**v, **kw}.items():
        setattr(p, k, x)
    return p


def glr(G, **kw):
    return filled(G.gdn_glr_problem(), {"N": 2, "T": 64, "T_total": 128, "channels": 256, "dtype": G.GDN_BF16, "rate": 8.0, "lambda": A}, kw)


V, O = (A, 256), [(k * A, 256) for k in range(2, 6)]


def glr_fwd(G, p, x=V, r=V, i=V, h0=None, y=O[0], hT=None, sv=None, ws=(A, 1 << 40)):
    return call(G, "gdn_glr_fwd", p, *x, *r, *i, h0, *y, hT, sv, *ws, 0)


def glr_bwd(G, p, sv=A, dy=V, dhT=None, dx=O[0], dr=O[1], di=O[2], dlam=None, dh0=None, ws=(A, 1 << 40)):
    return call(G, "gdn_glr_bwd", p, *V, *V, *V, sv, *dy, dhT, *dx, *dr, *di, dlam, dh0, *ws, 0)


def glr_dec(G, p, x=V, state=9 * A, slots=2, idx=None, y=V):
    return call(G, "gdn_glr_decode", p, *x, *V, *V, state, slots, idx, *y, 0)


def test_recurrence_refusals(G):
    E, U, L, W = G.GDN_EINVAL, G.GDN_EUNSUPPORTED, G.GDN_EALIGN, G.GDN_EWORKSPACE
    for kw, want in ((dict(channels=12), E), (dict(channels=0), E), (dict(channels=-8), E), (dict(dtype=2), U), (dict(rate=0.0), E),
                     (dict(rate=-1.0), E), (dict(rate=float("nan")), E), (dict(rate=float("inf")), E), (dict(N=-1), E), (dict(T=63), E),
                     (dict(T_total=-1), E), ({"lambda": None}, E), ({"lambda": A + 4}, L), (dict(fresh=A + 2), L), (dict(cu_seqlens=A + 2), L),
                     (dict(N=0, T_total=5, cu_seqlens=A), E), (dict(N=1, T=1 << 29, T_total=1 << 29), E), (dict(N=1 << 23, T=0, T_total=0), E),
                     (dict(N=2**31 - 1, T=0, T_total=0), E), (dict(N=1 << 21, T=0, T_total=0), E), (dict(channels=2**31 - 8), E)):
        p = glr(G, **kw)
        assert glr_fwd(G, p) == want, kw
        assert glr_bwd(G, p) == want, kw
        assert G.gdn_glr_state_bytes(p) == 0 and G.gdn_glr_fwd_workspace_bytes(p) == 0 and G.gdn_glr_bwd_workspace_bytes(p) == 0
    p = glr(G)
    assert glr_fwd(G, p, x=(None, 256)) == E and glr_fwd(G, p, r=(A, 255)) == E and glr_fwd(G, p, y=(A * 2, 260)) == L
    assert glr_fwd(G, p, i=(A + 8, 256)) == L and glr_fwd(G, p, x=(A, 1 << 60)) == E and glr_fwd(G, p, y=(A, 512)) == E
    assert glr_fwd(G, p, h0=A + 4) == L and glr_fwd(G, p, hT=A + 8) == L and glr_fwd(G, p, h0=A, hT=A) == E and glr_fwd(G, p, sv=A + 4) == L
    for rs in (1 << 22, 1 << 61, 1 << 62, -8):
        assert glr_fwd(G, p, x=(A, rs)) == E and glr_bwd(G, p, dy=(A, rs)) == E
    one = glr(G, N=1, T=1 << 16, T_total=1 << 16)
    need = G.gdn_glr_fwd_workspace_bytes(one)  # one sequence of few channels is cut into segments
    assert need > 0 and glr_fwd(G, one, ws=(None, 0)) == W and glr_fwd(G, one, ws=(A, need - 1)) == W and glr_fwd(G, one, ws=(A + 16, need)) == L
    need = G.gdn_glr_bwd_workspace_bytes(p)
    assert need > 0 and glr_bwd(G, p, ws=(A, need - 1)) == W and glr_bwd(G, p, sv=None) == E and glr_bwd(G, p, sv=A + 4) == L
    assert glr_bwd(G, p, dhT=A, dh0=A) == E and glr_bwd(G, p, dx=(2 * A, 8)) == E and glr_bwd(G, p, dlam=A + 2) == L
    assert glr_bwd(G, p, dr=O[0]) == E and glr_bwd(G, p, di=(A, 512)) == E and glr_bwd(G, p, dy=(A, 8)) == E


def test_recurrence_token_refusals(G):
    E, L = G.GDN_EINVAL, G.GDN_EALIGN
    one = dict(N=2, T=1, T_total=2)
    assert glr_dec(G, glr(G)) == E and glr_dec(G, glr(G, **one, cu_seqlens=A)) == E
    p = glr(G, **one)
    assert glr_dec(G, p, slots=1) == E and glr_dec(G, p, slots=-1, idx=A) == E and glr_dec(G, p, state=None) == E
    assert glr_dec(G, p, state=A + 4) == L and glr_dec(G, p, idx=A + 2) == L and glr_dec(G, p, y=(A, 8)) == E
    assert glr_dec(G, p, y=(A, 512)) == E and glr_dec(G, p, state=A) == E


def rope(G, **kw):
    return filled(G.gdn_qk_rope_problem(), dict(rows=4, Hq=4, Hk=2, D=64, rot=32, adjacent=0, eps=1e-6, rope_scale=1.0, dtype=G.GDN_BF16,
                                                positions=A, freq=A), kw)


def test_rotation_refusals(G):
    E, U, L, W = G.GDN_EINVAL, G.GDN_EUNSUPPORTED, G.GDN_EALIGN, G.GDN_EWORKSPACE

    def fwd(p, q=(A, 256), k=(2 * A, 128), qo=(A, 256), ko=(2 * A, 128)):
        return call(G, "gdn_qk_rope_fwd", p, *q, *k, *qo, *ko, 0)

    def bwd(p, dq=(3 * A, 256), dk=(4 * A, 128), dwq=A, dwk=None, ws=(A, 1 << 30)):
        return call(G, "gdn_qk_rope_bwd", p, A, 256, 2 * A, 128, A, 256, 2 * A, 128, *dq, *dk, dwq, dwk, *ws, 0)

    def cache(p, qo=(A, 256), kp=5 * A, vp=6 * A, pages=4, page=16, where=A, v=(7 * A, 128)):
        return call(G, "gdn_qk_rope_cache", p, A, 256, 2 * A, 128, *v, *qo, kp, vp, pages, page, where, 0)

    for kw, want in ((dict(rows=-1), E), (dict(Hq=0), E), (dict(Hk=0), E), (dict(D=0), E), (dict(D=24, rot=16), U), (dict(D=272), U), (dict(rot=8), U),
                     (dict(rot=80), E), (dict(rot=-16), E), (dict(dtype=3), U), (dict(eps=-1.0), E), (dict(eps=float("nan")), E),
                     (dict(rope_scale=float("inf")), E), (dict(positions=None), E), (dict(freq=None), E), (dict(positions=A + 2), L),
                     (dict(freq=A + 4), L), (dict(wq=A + 4), L), (dict(wk=A + 8), L), (dict(rows=1 << 40), E), (dict(Hq=2**31 - 1), E)):
        p = rope(G, **kw)
        assert fwd(p) == want and bwd(p) == want and cache(p) == want, kw
        assert G.gdn_qk_rope_bwd_workspace_bytes(p) == 0
    p = rope(G)
    assert fwd(p, q=(None, 256)) == E and fwd(p, k=(2 * A, 127)) == E and fwd(p, ko=(2 * A + 2, 128)) == L
    assert fwd(p, qo=(2 * A, 256)) == E and fwd(p, ko=(A, 128)) == E and fwd(p, qo=(A, 264)) == E and fwd(p, qo=(3 * A, 256), ko=(3 * A, 128)) == E
    assert bwd(p, dq=(2 * A, 256)) == E and bwd(p, dk=(A, 256)) == E and bwd(p, dk=(3 * A, 128)) == E and bwd(p, dq=(A, 264)) == E
    assert bwd(p, ws=(None, 0)) == W and bwd(p, ws=(A, G.gdn_qk_rope_bwd_workspace_bytes(p) - 1)) == W and bwd(p, ws=(A + 64, 1 << 30)) == L
    assert bwd(p, dwk=A) == E and bwd(p, dwq=A + 1) == L
    assert cache(p, kp=None) == E and cache(p, vp=A * 5) == E and cache(p, kp=5 * A + 8) == L and cache(p, where=None) == E and cache(p, where=A + 2) == L
    assert cache(p, pages=-1) == E and cache(p, page=0) == E and cache(p, pages=1 << 30, page=2) == E and cache(p, v=(None, 128)) == E
    assert cache(p, kp=7 * A) == E and cache(p, qo=(7 * A, 256)) == E and cache(p, vp=A) == E and cache(p, qo=(5 * A, 256)) == E
    assert cache(rope(G, Hk=4), pages=1 << 30, page=1, v=(7 * A, 256)) == E  # rows of heads past 32 bits


def paged(G, **kw):
    return filled(G.gdn_paged_problem(), dict(N=2, Hq=8, Hk=2, D=64, page_size=16, n_pages=10, max_pages=5, max_len=80, window=0, scale=0.125,
                                              dtype=G.GDN_BF16, page_table=A, lens=A), kw)


def test_attention_refusals(G):
    E, U, L, W = G.GDN_EINVAL, G.GDN_EUNSUPPORTED, G.GDN_EALIGN, G.GDN_EWORKSPACE

    def run(p, q=(A, 512), kp=2 * A, vp=3 * A, out=(4 * A, 512), lse=None, ws=(A, 1 << 40)):
        return call(G, "gdn_paged_attn_decode", p, *q, kp, vp, *out, lse, *ws, 0)

    for kw, want in ((dict(N=-1), E), (dict(Hq=7), E), (dict(Hq=0), E), (dict(Hk=0), E), (dict(D=48), U), (dict(D=512), U), (dict(dtype=7), U),
                     (dict(page_size=0), E), (dict(n_pages=-1), E), (dict(n_pages=1 << 30, page_size=4), E), (dict(max_pages=-1), E),
                     (dict(max_len=81), E), (dict(max_len=-1), E), (dict(window=-1), E), (dict(scale=float("nan")), E), (dict(page_table=None), E),
                     (dict(lens=None), E), (dict(page_table=A + 2), L), (dict(lens=A + 1), L), (dict(N=1 << 24), E),
                     (dict(Hk=8, n_pages=1 << 29, page_size=2), E), (dict(N=1 << 21), E),
                     (dict(N=1, max_pages=2**27 - 1, max_len=2**31 - 16), E), (dict(N=1, max_pages=2**27 - 1, max_len=2**30 + 1), E)):
        p = paged(G, **kw)
        assert run(p) == want, kw
        assert G.gdn_paged_attn_workspace_bytes(p) == 0
    p = paged(G)
    assert run(p, q=(None, 512)) == E and run(p, q=(A, 511)) == E and run(p, out=(4 * A, 516)) == L and run(p, kp=None) == E and run(p, vp=3 * A + 8) == L
    assert run(p, out=(A, 512)) == E and run(p, out=(2 * A, 512)) == E and run(p, lse=A + 2) == L
    long = paged(G, max_pages=1 << 12, max_len=1 << 16, n_pages=1 << 13)
    need = G.gdn_paged_attn_workspace_bytes(long)
    assert need > 0 and run(long, ws=(None, 0)) == W and run(long, ws=(A, need - 1)) == W and run(long, ws=(A + 64, need)) == L


def test_binding_without_gpu(G):
    import torch

    t = torch.zeros(8)
    for f in (lambda: G.make_glr_problem(1, 1, 8, lam=t), lambda: G.make_glr_problem(1, 1, 8, lam=None),
              lambda: G.make_qk_rope_problem(1, 1, 1, 16, positions=t.int(), freq=t.double()), lambda: G.make_qk_rope_problem(1, 1, 1, 16),
              lambda: G.make_paged_problem(t.int()[None], t.int(), 1, 1, 32, page_size=1), lambda: G.make_paged_problem(None, None, 1, 1, 32, page_size=1),
              lambda: G.gdn_qk_rope_fwd(rope(G), t, t, t, t), lambda: G.gdn_glr_fwd(glr(G), None, t, t, None, t, None, None, None)):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(TypeError):
        G.gdn_glr_state_bytes(rope(G))


def _asan_runtime():
    r = subprocess.run([CLANG, "-print-file-name=libclang_rt.asan-x86_64.so"], capture_output=True, text=True)
    path = r.stdout.strip()
    return path if r.returncode == 0 and os.path.isabs(path) and os.path.exists(path) else None


def test_under_sanitizers(tmp_path):
    """This file's other tests against a host-only build of hybrid_abi.cpp whose launchers are stubs."""
    if os.environ.get("GDN_LIBRARY"):
        pytest.skip("already that run")
    rt = _asan_runtime() if os.path.exists(CLANG) else None
    if not (os.path.exists(HIPCC) and rt):
        pytest.skip("no hipcc / clang sanitizer runtime")
    csrc, san = os.path.join(ROOT, "gated_delta_rule_34_amd", "csrc"), os.path.join(ROOT, "tests", "sanitize")
    lib = str(tmp_path / "libgdn_sanitized.so")
    subprocess.run([HIPCC, "-xhip", "--offload-host-only", "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
                    "-shared-libasan", "-fno-omit-frame-pointer", "-g", "-O1", "-std=c++17", "-fPIC", "-shared", f"-I{ROOT}/include", f"-I{csrc}",
                    os.path.join(csrc, "gdn_abi.cpp"), os.path.join(csrc, "hybrid", "hybrid_abi.cpp"), os.path.join(san, "gdn_host_stubs.cpp"),
                    os.path.join(san, "hybrid_host_stubs.cpp"), "-o", lib], check=True)
    env = dict(os.environ, LD_PRELOAD=rt, GDN_LIBRARY=lib, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:verify_asan_link_order=0",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", os.path.abspath(__file__)], env=env, cwd=ROOT,
                       capture_output=True, text=True, timeout=600)
    tail = (r.stdout + r.stderr)[-4000:]
    assert r.returncode == 0 and " passed" in r.stdout, tail
    assert "ERROR: AddressSanitizer" not in tail and "runtime error" not in tail, tail
