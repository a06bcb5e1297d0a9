"""The entry points of gdn_layer.h reject bad arguments on the host before any
HIP call (so these run without a GPU), and their host layer runs clean under
AddressSanitizer and UndefinedBehaviorSanitizer."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

import gated_deltanet_tree_gdn_amd as gdn
from gated_deltanet_tree_gdn_amd import layer

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gdn_layer.h")
FAKE = 0x10000  # never dereferenced: every call below fails before touching it


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(gdn.LIB_PATH):
        pytest.fail("libgdn_tree.so is not built: run __graft_entry__.build()")
    return layer.layer_library()


def status(code):
    return gdn.STATUS[code]


def test_exports_every_declared_symbol(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(gdn_[a-z0-9_]+)\s*\(", text))
    assert names == set(layer.LAYER_EXPORTS)
    for n in names:
        assert hasattr(lib, n), n


def seq(**kw):
    d = dict(B=2, T=100, H_k=2, H_v=4, d_k=128, d_v=128, qkv_dtype=0, o_dtype=1, n_slots=2, qk_l2norm=0, q_scale=1.0,
             l2_eps=1e-6, q_stride=256, k_stride=256, v_stride=512)
    d.update(kw)
    return layer.SeqDims(**d)


PREFILL = ["q", "k", "v", "g", "beta", "cu_seqlens", "slot", "has_state", "S", "o", "seq_status", "workspace"]


def prefill(lib, d, nbytes=None, **over):
    a = dict.fromkeys(PREFILL, FAKE)
    a.update(over)
    if nbytes is None:
        nbytes = lib.gdn_prefill_workspace_bytes(d) if d is not None else 0
    return status(lib.gdn_prefill(d, *(a[n] for n in PREFILL), nbytes, None))


BAD_SEQ = [
    (dict(B=-1), "GDN_ERR_SHAPE"), (dict(B=65536), "GDN_ERR_SHAPE"), (dict(H_k=0), "GDN_ERR_SHAPE"),
    (dict(H_v=3), "GDN_ERR_SHAPE"), (dict(H_v=65536), "GDN_ERR_SHAPE"), (dict(B=60000, H_v=400), "GDN_ERR_SHAPE"),
    (dict(d_k=96), "GDN_ERR_SHAPE"), (dict(d_v=32), "GDN_ERR_SHAPE"), (dict(n_slots=-1), "GDN_ERR_SHAPE"),
    (dict(l2_eps=-1.0), "GDN_ERR_SHAPE"), (dict(l2_eps=float("nan")), "GDN_ERR_SHAPE"),
    (dict(q_stride=-8), "GDN_ERR_SHAPE"), (dict(k_stride=1 << 25), "GDN_ERR_SHAPE"), (dict(v_stride=513), "GDN_ERR_ALIGN"),
    (dict(qkv_dtype=2), "GDN_ERR_DTYPE"), (dict(o_dtype=-1), "GDN_ERR_DTYPE"),
]


@pytest.mark.parametrize("kw,code", BAD_SEQ + [(dict(T=-1), "GDN_ERR_SHAPE")])
def test_prefill_rejects_dims(lib, kw, code):
    assert prefill(lib, seq(**kw), nbytes=1 << 40) == code
    assert lib.gdn_last_error().decode()


@pytest.mark.parametrize("kw,code", BAD_SEQ)
def test_decode_rejects_dims(lib, kw, code):
    assert status(lib.gdn_decode(seq(**kw), *[FAKE] * 8, None)) == code


@pytest.mark.parametrize("name", ["q", "k", "v", "g", "beta", "cu_seqlens", "S", "o"])
def test_prefill_rejects_null_and_misaligned(lib, name):
    assert prefill(lib, seq(), **{name: None}) == "GDN_ERR_NULL"
    assert name in lib.gdn_last_error().decode()
    assert prefill(lib, seq(), **{name: FAKE + 4}) == "GDN_ERR_ALIGN"


def test_prefill_optional_arguments_and_workspace(lib):
    for name in ("slot", "has_state", "seq_status"):
        assert prefill(lib, seq(), **{name: FAKE + 8}) == "GDN_ERR_ALIGN"
    need = lib.gdn_prefill_workspace_bytes(seq())
    assert need > 0 and need % 256 == 0
    assert prefill(lib, seq(), workspace=None) == "GDN_ERR_WORKSPACE"
    assert prefill(lib, seq(), nbytes=need - 1) == "GDN_ERR_WORKSPACE"
    assert prefill(lib, seq(), workspace=FAKE + 16) == "GDN_ERR_ALIGN"
    assert prefill(lib, seq(n_slots=1), slot=None) == "GDN_ERR_SHAPE"
    assert prefill(lib, None) == "GDN_ERR_NULL"
    assert prefill(lib, seq(B=0), **dict.fromkeys(PREFILL)) == "GDN_OK"
    assert lib.gdn_prefill_workspace_bytes(None) == 0
    assert lib.gdn_prefill_workspace_bytes(seq(B=0)) == lib.gdn_prefill_workspace_bytes(seq(T=0)) == 0


def test_prefill_workspace_grows_with_tokens_and_sequences(lib):
    """room for every packing: T / 64 + B chunks of every value head"""
    per = [lib.gdn_prefill_workspace_bytes(seq(T=t, B=b)) for t, b in ((6400, 1), (12800, 1), (6400, 101))]
    assert 1.9 < per[1] / per[0] < 2.0 and 1.9 < per[2] / per[0] < 2.1


def test_decode_rejects_pointers(lib):
    for i in range(8):
        args = [FAKE] * 8
        args[i] = FAKE + 4
        assert status(lib.gdn_decode(seq(), *args, None)) == "GDN_ERR_ALIGN"
        args[i] = None
        want = "GDN_ERR_NULL" if i != 5 else None  # slot may be NULL
        if want:
            assert status(lib.gdn_decode(seq(), *args, None)) == want
    args = [FAKE] * 8
    args[5] = None
    assert status(lib.gdn_decode(seq(n_slots=1), *args, None)) == "GDN_ERR_SHAPE"
    assert status(lib.gdn_decode(None, *[FAKE] * 8, None)) == "GDN_ERR_NULL"
    assert status(lib.gdn_decode(seq(B=0), *[None] * 8, None)) == "GDN_OK"


def add_dims(**kw):
    d = dict(T=3, D=100, x_dtype=0, res_dtype=1, y_dtype=0, scale=1.0, eps=1e-6, weight_offset=0.0, x_stride=100,
             res_stride=100, h_stride=100, y_stride=100)
    d.update(kw)
    return layer.AddNormDims(**d)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), "GDN_ERR_SHAPE"), (dict(D=0), "GDN_ERR_SHAPE"), (dict(D=16385), "GDN_ERR_SHAPE"),
    (dict(eps=-1.0), "GDN_ERR_SHAPE"), (dict(x_stride=-1), "GDN_ERR_SHAPE"), (dict(y_stride=99), "GDN_ERR_SHAPE"),
    (dict(h_stride=99), "GDN_ERR_SHAPE"), (dict(x_dtype=3), "GDN_ERR_DTYPE"), (dict(res_dtype=3), "GDN_ERR_DTYPE"),
    (dict(y_dtype=3), "GDN_ERR_DTYPE"),
])
def test_add_norm_rejects_dims(lib, kw, code):
    assert status(lib.gdn_add_norm(add_dims(**kw), *[FAKE] * 7, None)) == code


def test_add_norm_rejects_pointers(lib):
    for i in range(7):
        args = [FAKE + 64 * j for j in range(7)]
        args[i] += 4 if i in (2, 3, 4) else 1  # weights in 16-byte pieces, rows wherever their elements may be
        assert status(lib.gdn_add_norm(add_dims(), *args, None)) == "GDN_ERR_ALIGN"
        args[i] = None
        if i in (0, 2, 6):
            assert status(lib.gdn_add_norm(add_dims(), *args, None)) == "GDN_ERR_NULL"
    args = [FAKE] * 7  # h in place of residual with another stride
    assert status(lib.gdn_add_norm(add_dims(h_stride=128), *args, None)) == "GDN_ERR_SHAPE"
    assert status(lib.gdn_add_norm(None, *args, None)) == "GDN_ERR_NULL"
    assert status(lib.gdn_add_norm(add_dims(T=0), *[None] * 7, None)) == "GDN_OK"


def gated_dims(**kw):
    d = dict(T=3, H=2, d=64, o_dtype=1, z_dtype=0, y_dtype=0, gate=1, eps=1e-6, o_stride=128, z_stride=128, y_stride=128)
    d.update(kw)
    return layer.GatedNormDims(**d)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), "GDN_ERR_SHAPE"), (dict(H=0), "GDN_ERR_SHAPE"), (dict(d=0), "GDN_ERR_SHAPE"),
    (dict(d=16385), "GDN_ERR_SHAPE"), (dict(gate=0), "GDN_ERR_SHAPE"), (dict(gate=2), "GDN_ERR_SHAPE"),
    (dict(eps=float("nan")), "GDN_ERR_SHAPE"), (dict(o_stride=-1), "GDN_ERR_SHAPE"), (dict(z_stride=-1), "GDN_ERR_SHAPE"),
    (dict(y_stride=127), "GDN_ERR_SHAPE"), (dict(o_dtype=5), "GDN_ERR_DTYPE"), (dict(z_dtype=5), "GDN_ERR_DTYPE"),
    (dict(y_dtype=5), "GDN_ERR_DTYPE"),
])
def test_gated_norm_rejects_dims(lib, kw, code):
    assert status(lib.gdn_gated_norm(gated_dims(**kw), FAKE, FAKE + 16, FAKE, FAKE + 32, None)) == code


def test_gated_norm_rejects_pointers(lib):
    for i in range(4):
        args = [FAKE + 64 * j for j in range(4)]
        args[i] += 4 if i == 2 else 1  # the weight in 16-byte pieces, rows wherever their elements may be
        assert status(lib.gdn_gated_norm(gated_dims(), *args, None)) == "GDN_ERR_ALIGN"
        args[i] = None
        assert status(lib.gdn_gated_norm(gated_dims(), *args, None)) == "GDN_ERR_NULL"
    assert status(lib.gdn_gated_norm(gated_dims(), FAKE, FAKE + 16, FAKE, FAKE, None)) == "GDN_ERR_SHAPE"  # in place, other dtype
    assert status(lib.gdn_gated_norm(None, *[FAKE] * 4, None)) == "GDN_ERR_NULL"
    assert status(lib.gdn_gated_norm(gated_dims(T=0), *[None] * 4, None)) == "GDN_OK"


def linear_dims(**kw):
    d = dict(M=3, N=5, K=64, res_dtype=0, y_dtype=0, act=0, scale=1.0, x_stride=64, w_stride=64, res_stride=5, y_stride=5)
    d.update(kw)
    return layer.LinearDims(**d)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), "GDN_ERR_SHAPE"), (dict(N=-1), "GDN_ERR_SHAPE"), (dict(K=-1), "GDN_ERR_SHAPE"),
    (dict(act=4), "GDN_ERR_SHAPE"), (dict(act=-1), "GDN_ERR_SHAPE"), (dict(x_stride=-1), "GDN_ERR_SHAPE"),
    (dict(w_stride=-1), "GDN_ERR_SHAPE"), (dict(res_stride=-1), "GDN_ERR_SHAPE"), (dict(y_stride=4), "GDN_ERR_SHAPE"),
    (dict(y_dtype=2), "GDN_ERR_DTYPE"), (dict(res_dtype=2), "GDN_ERR_DTYPE"),
])
def test_linear_rejects_dims(lib, kw, code):
    assert status(lib.gdn_linear(linear_dims(**kw), FAKE, FAKE, FAKE, FAKE + 16, FAKE, FAKE, 1 << 40, None)) == code


def test_linear_rejects_pointers(lib):
    for i in range(5):
        args = [FAKE + 64 * j for j in range(5)]
        args[i] += 4
        assert status(lib.gdn_linear(linear_dims(), *args, FAKE, 1 << 40, None)) == "GDN_ERR_ALIGN"
        args[i] = None
        if i in (0, 1, 4):
            assert status(lib.gdn_linear(linear_dims(), *args, FAKE, 1 << 40, None)) == "GDN_ERR_NULL"
    in_place = (FAKE, FAKE, None, FAKE, FAKE, FAKE, 1 << 40, None)
    assert status(lib.gdn_linear(linear_dims(res_dtype=1), *in_place)) == "GDN_ERR_SHAPE"
    assert status(lib.gdn_linear(linear_dims(res_stride=8), *in_place)) == "GDN_ERR_SHAPE"
    assert status(lib.gdn_linear(None, *in_place)) == "GDN_ERR_NULL"
    for kw in (dict(M=0), dict(N=0)):
        assert status(lib.gdn_linear(linear_dims(**kw), *[None] * 6, 0, None)) == "GDN_OK"
    assert lib.gdn_linear_workspace_bytes(None) == 0


def test_binding_has_no_cpu_fallback():
    src = open(layer.__file__).read()
    assert "oracle" not in src and "numpy" not in src


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not installed")
def test_layer_host_code_under_sanitizers(tmp_path):
    exe = str(tmp_path / "layer_driver")
    csrc = os.path.join(ROOT, "gated_deltanet_tree_gdn_amd", "csrc")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                        "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I", os.path.join(ROOT, "include"), "-I", csrc,
                        os.path.join(csrc, "gdn_layer_api.cpp"),
                        os.path.join(ROOT, "tests", "sanitize", "layer_driver.cpp"), "-o", exe],
                       capture_output=True, text=True)
    if r.returncode != 0 and "cannot find" in r.stderr and "asan" in r.stderr.lower():
        pytest.skip("sanitizer runtime not installed")
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60,
                       env=dict(os.environ, UBSAN_OPTIONS="print_stacktrace=1"))
    assert r.returncode == 0, r.stdout + r.stderr
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr
