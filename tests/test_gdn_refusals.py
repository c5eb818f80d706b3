"""What the recurrent calls and the 4-bit cache format refuse, before anything is launched (CPU)."""
import ctypes as C

import pytest
import torch

import tree_speculative_decoding_array_gb300 as tsv
from tree_speculative_decoding_array_gb300 import _abi

PTR = 0x1000


def gdn(**kw):
    d = _abi.GdnDesc()
    f = dict(n_layers=1, B=1, T=4, HK=2, HV=4, DK=128, DV=128, norm_eps=1e-6, scale=0.0)
    f.update({k: v for k, v in kw.items() if k in f})
    for k, v in f.items():
        setattr(d, k, v)
    for name in ("q", "k", "v", "g", "beta", "state", "state_out", "o"):
        getattr(d, name)[0] = kw.get(name, PTR)
    return d


def calls(d, anc=PTR, path=PTR, cu=PTR, max_len=1):
    lib = tsv.load()
    vp = C.c_void_p
    return dict(verify=lambda: lib.tsv_gdn_tree_verify(C.byref(d), vp(anc), None, None),
                commit=lambda: lib.tsv_gdn_commit(C.byref(d), vp(path), vp(path), None, None),
                scan=lambda: lib.tsv_gdn_scan(C.byref(d), vp(cu), max_len, None, None))


@pytest.fixture(autouse=True)
def no_error_left_behind():
    yield
    assert calls(gdn(B=0))["scan"]() == _abi.OK  # a call that succeeds clears this thread's reason


@pytest.mark.parametrize("kw, status, word", [
    (dict(n_layers=0), _abi.ECAPACITY, b"n_layers"), (dict(n_layers=65), _abi.ECAPACITY, b"n_layers"),
    (dict(HK=3), _abi.EINVAL, b"HK=3"), (dict(HK=0), _abi.EINVAL, b"HK=0"), (dict(B=-1), _abi.EINVAL, b"B=-1"),
    (dict(DK=96), _abi.EUNSUPPORTED, b"96"), (dict(DV=256), _abi.EUNSUPPORTED, b"256"),
    (dict(norm_eps=-1.0), _abi.EINVAL, b"norm_eps"), (dict(norm_eps=float("nan")), _abi.EINVAL, b"norm_eps"),
    (dict(scale=float("inf")), _abi.EINVAL, b"scale"), (dict(state=0), _abi.EINVAL, b"state"),
    (dict(k=0), _abi.EINVAL, b"null"), (dict(beta=0), _abi.EINVAL, b"null"), (dict(v=PTR + 8), _abi.EINVAL, b"16-byte"),
    (dict(state=PTR + 4), _abi.EINVAL, b"16-byte"), (dict(g=PTR + 2), _abi.EINVAL, b"4-byte"),
    (dict(B=1 << 30, HV=4), _abi.ECAPACITY, b"units"),
])
def test_every_call_refuses(kw, status, word):
    for name, call in calls(gdn(**kw)).items():
        assert call() == status, name
        assert word in tsv.load().tsv_last_error(), name


def test_what_each_call_needs():
    lib = tsv.load()
    for T in (0, 65, -1):
        d = gdn(T=T)
        assert calls(d)["verify"]() == _abi.ECAPACITY and calls(d)["commit"]() == _abi.ECAPACITY
    assert calls(gdn(T=-1))["scan"]() == _abi.ECAPACITY
    assert calls(gdn(q=0))["verify"]() == _abi.EINVAL and calls(gdn(o=0))["scan"]() == _abi.EINVAL
    assert calls(gdn(state_out=0))["commit"]() == _abi.EINVAL and calls(gdn(state_out=0))["scan"]() == _abi.EINVAL
    assert calls(gdn(), anc=0)["verify"]() == _abi.EINVAL
    assert calls(gdn(), path=0)["commit"]() == _abi.EINVAL
    assert calls(gdn(), cu=0)["scan"]() == _abi.EINVAL
    assert calls(gdn(), max_len=5)["scan"]() == _abi.EINVAL and b"max_len" in lib.tsv_last_error()
    assert calls(gdn(), max_len=-1)["scan"]() == _abi.EINVAL
    for name, call in calls(gdn(B=0, q=0, k=0, state=0)).items():  # an empty batch reads nothing
        assert call() == _abi.OK, name


def test_four_bit_caches_need_their_scales():
    lib = tsv.load()
    a = _abi.AttnDesc()
    a.n_layers, a.B, a.T, a.HQ, a.HKV, a.D, a.kv_dtype, a.s_cap, a.max_kv_len = 1, 1, 2, 4, 2, 128, tsv.I4_G64, 8, 8
    for f in ("q", "k", "v", "o"):
        getattr(a, f)[0] = PTR
    a.kv_len = a.anc = PTR
    assert lib.tsv_tree_verify_attention(C.byref(a), None, 0, None, None) == _abi.EINVAL
    assert b"4-bit" in lib.tsv_last_error()
    a.k_scale[0], a.v_scale[0] = PTR, PTR + 4
    assert lib.tsv_tree_verify_attention(C.byref(a), None, 0, None, None) == _abi.EINVAL
    kv = _abi.KvDesc()
    kv.n_layers, kv.B, kv.HKV, kv.D, kv.s_cap, kv.kv_dtype = 1, 1, 2, 128, 8, tsv.I4_G64
    kv.k[0] = kv.v[0] = PTR
    vp = C.c_void_p(PTR)
    assert lib.tsv_kv_gather_positions(C.byref(kv), vp, vp, vp, 2, None, None) == _abi.EINVAL
    assert lib.tsv_gather_positions(C.byref(kv), vp, vp, vp, 2, None, None) == _abi.EINVAL
    ap = _abi.AppendDesc()
    ap.n_layers, ap.B, ap.T, ap.HQ, ap.HKV, ap.D, ap.s_cap, ap.kv_dtype = 1, 1, 2, 4, 2, 128, 8, tsv.I4_G64
    ap.rot_dim, ap.rope_base, ap.depth = 64, 1e4, PTR
    for f in ("q_in", "q_out", "k_new", "v_new", "k", "v"):
        getattr(ap, f)[0] = PTR
    assert lib.tsv_tree_append(C.byref(ap), vp, None, None) == _abi.EINVAL
    for bad in (3, 5, -1):  # a weight format, an unknown one
        a.kv_dtype = kv.kv_dtype = ap.kv_dtype = bad
        assert lib.tsv_tree_verify_attention(C.byref(a), None, 0, None, None) == _abi.EUNSUPPORTED
        assert lib.tsv_kv_gather_positions(C.byref(kv), vp, vp, vp, 2, None, None) == _abi.EUNSUPPORTED
        assert lib.tsv_gather_positions(C.byref(kv), vp, vp, vp, 2, None, None) == _abi.EUNSUPPORTED
        assert lib.tsv_tree_append(C.byref(ap), vp, None, None) == _abi.EUNSUPPORTED


@pytest.mark.parametrize("D, HQ, path", [(256, 4, 0), (256, 64, 0), (256, 64, 2), (128, 4, 1)])
def test_four_bit_attention_needs_an_aligned_workspace(D, HQ, path):
    lib = tsv.load()
    a = _abi.AttnDesc()
    a.n_layers, a.B, a.T, a.HQ, a.HKV, a.D, a.kv_dtype, a.s_cap, a.max_kv_len = 1, 1, 2, HQ, 2, D, tsv.I4_G64, 4096, 4096
    a.splits, a.path = 4, path
    for f in ("q", "k", "v", "o", "k_scale", "v_scale"):
        getattr(a, f)[0] = PTR
    a.kv_len = a.anc = PTR
    need = lib.tsv_attention_workspace_size(C.byref(a))
    assert need > 0
    assert lib.tsv_tree_verify_attention(C.byref(a), C.c_void_p(PTR), need - 1, None, None) == _abi.ECAPACITY
    assert lib.tsv_tree_verify_attention(C.byref(a), C.c_void_p(PTR + 8), need, None, None) == _abi.EINVAL
    assert b"aligned" in lib.tsv_last_error()


def test_the_binding_checks_its_tensors():
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    f = lambda *s: torch.zeros(*s)  # noqa: E731
    args = lambda **kw: [kw.get(n, d) for n, d in (  # noqa: E731
        ("q", [bf(1, 2, 1, 128)]), ("k", [bf(1, 2, 1, 128)]), ("v", [bf(1, 2, 2, 128)]), ("g", [f(1, 2, 2)]),
        ("beta", [f(1, 2, 2)]), ("state", [f(1, 2, 128, 128)]))]
    with pytest.raises(ValueError, match="CUDA"):
        tsv.gdn_desc(*args())
    with pytest.raises(ValueError, match="same length"):
        tsv.gdn_desc(*args(g=[]))
    with pytest.raises(ValueError, match="must be"):
        tsv.gdn_desc(*args(k=[bf(2, 128)]))
    with pytest.raises(ValueError, match="sequences"):
        tsv.gdn_desc(*args(state=[f(3, 2, 128, 128)]))


def test_struct_layout_matches_header(tmp_path):
    import os
    import shutil
    import subprocess

    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    names = [f for f, _ in _abi.GdnDesc._fields_]
    src = ['#include <stdio.h>', '#include <stddef.h>', '#include "tsv.h"', "int main(void){",
           'printf("%zu\\n", sizeof(tsv_gdn_desc));']
    src += [f'printf("%zu\\n", offsetof(tsv_gdn_desc, {f}));' for f in names] + ["return 0;}"]
    (tmp_path / "a.c").write_text("\n".join(src))
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), "-I", "/usr/local/cuda/include", str(tmp_path / "a.c"),
                    "-o", str(tmp_path / "a")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "a")], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [C.sizeof(_abi.GdnDesc)] + [getattr(_abi.GdnDesc, f).offset for f in names]
